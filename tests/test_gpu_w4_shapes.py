"""The 4-bit layer in every shape of its two kernels that a plan chooses, against
the same sum in 64 bits with the tolerance of the other tests (test_gpu_w4).

w4_few: each count of row blocks and warps, CTAs that take several tiles of
output channels, so that weights, scales and sums pass from tile to tile, with
units of input channels fewer than the warps, fewer than the ring and many, and
rows of scales copied by vectors and singly.  w4_many: each count of row blocks
and output channels a CTA, x copied as it lies and through registers."""
import re

import pytest
import torch

from test_gpu_w4 import DT, cl, weights64  # noqa: F401  (cl: the fixture)

pytestmark = pytest.mark.gpu

FEW = [
    # rows, c_in, c_out, group, dtype, act, (blocks of eight rows, warps)
    (1, 100, 14600, 32, "bf16", "none", (1, 8)),        # one unit: most warps have none
    (3, 1000, 14600, 64, "bf16", "relu", (1, 8)),
    (1, 5003, 14601, 128, "f32", "none", (1, 8)),       # five units a warp
    (1, 8192, 14600, 128, "bf16", "mish", (1, 8)),      # eight; scales by vectors
    (1, 8192, 14600, 32, "bf16", "none", (1, 8)),
    (8, 4096, 14592, 32, "bf16", "none", (1, 16)),
    (2, 18432, 4900, 128, "bf16", "none", (1, 16)),
    (1, 18700, 4901, 32, "f32", "none", (1, 8)),        # sixteen warps do not fit
    (2, 7400, 4901, 64, "f32", "mish", (1, 16)),
    (16, 700, 14600, 64, "bf16", "relu", (2, 8)),
    (14, 2300, 4900, 32, "bf16", "none", (2, 16)),
    (11, 1900, 4901, 64, "f32", "none", (2, 8)),
    (13, 777, 9800, 32, "f32", "relu", (2, 16)),
    (21, 260, 14600, 128, "bf16", "mish", (4, 8)),
    (32, 900, 9800, 128, "bf16", "none", (4, 16)),
    (17, 100, 9800, 64, "f32", "none", (4, 8)),
    (20, 515, 9800, 64, "f32", "none", (4, 16)),
]
MANY = [
    # ... (blocks of eight rows, times 16 output channels a CTA)
    (70, 1000, 40, 64, "bf16", "none", (1, 2)),
    (1, 41761, 9692, 32, "bf16", "none", (1, 4)),
    (2, 38064, 19405, 64, "bf16", "none", (1, 8)),
    (37, 333, 1603, 64, "bf16", "relu", (2, 2)),
    (9, 7123, 9747, 32, "bf16", "none", (2, 4)),
    (15, 4201, 19687, 32, "bf16", "none", (2, 8)),
    (33, 520, 3169, 128, "bf16", "none", (4, 2)),
    (33, 521, 3169, 32, "bf16", "mish", (4, 2)),        # more of a turn's x than the registers hold
    (45, 304, 5057, 32, "bf16", "none", (4, 4)),
    (25, 1805, 19687, 32, "bf16", "none", (4, 8)),
    (43, 1000, 10012, 128, "bf16", "none", (8, 4)),
    (43, 1001, 10012, 64, "bf16", "none", (8, 4)),
    (74, 500, 10240, 64, "bf16", "relu", (8, 8)),
    (130, 77, 10233, 32, "bf16", "none", (8, 8)),
    (33, 400, 21, 32, "f32", "none", (1, 2)),
    (1, 19813, 10253, 32, "f32", "none", (1, 4)),
    (3, 19200, 20507, 32, "f32", "none", (1, 8)),
    (53, 260, 1239, 64, "f32", "mish", (2, 2)),
    (37, 777, 3217, 128, "f32", "none", (2, 4)),
    (12, 2404, 20107, 32, "f32", "none", (2, 8)),
    (40, 515, 5180, 64, "f32", "none", (4, 4)),
    (40, 300, 9700, 32, "f32", "relu", (4, 8)),
    (47, 390, 19579, 128, "f32", "none", (8, 8)),
    (200, 130, 9000, 64, "f32", "none", (8, 8)),
]


def against_64_bits(cl, plan, rows, ci, co, group, dtype, act):  # noqa: F811
    g = torch.Generator("cuda").manual_seed(rows + ci)
    x = torch.randn(rows, ci, device="cuda", generator=g).to(DT[dtype])
    codes = torch.randint(0, 256, (co, (ci + 1) // 2), device="cuda", generator=g, dtype=torch.uint8)
    scales = (0.01 + 0.02 * torch.rand(co, -(-ci // group), device="cuda", generator=g)).to(DT[dtype])
    bias = 0.1 * torch.randn(co, device="cuda", generator=g)
    buf = torch.full((rows * co + 64,), 9.0, dtype=DT[dtype], device="cuda")
    y = buf[:rows * co].view(rows, co)
    packed = plan.pack(codes)
    plan.run(x, packed, scales, bias, y)
    again = torch.empty_like(y)
    plan.run(x, packed, scales, bias, again)
    assert torch.equal(y, again) and bool((buf[rows * co:] == 9).all())
    for i in range(0, co, 1024):
        w = weights64(codes[i:i + 1024], scales[i:i + 1024], ci, group)
        z = x.double() @ w.t() + bias[i:i + 1024].double()
        size = x.double().abs() @ w.abs().t() + bias[i:i + 1024].double().abs()
        tol = (ci / 16 + scales.shape[1] + 16) * 2.0 ** -23 * size
        if act == "relu":
            z = z.clamp(min=0)
        elif act == "mish":
            tol = 1.1 * tol + 2e-6 * (1 + z.abs())
            z = z * torch.tanh(torch.nn.functional.softplus(z))
        if dtype == "bf16":
            tol = tol + 2.0 ** -8 * z.abs()
        err = (y[:, i:i + 1024].double() - z).abs()
        assert (err <= tol).all(), (i, float((err / tol).max()), int((err > tol).sum()))


@pytest.mark.parametrize("rows,ci,co,group,dtype,act,shape", FEW)
def test_x_in_shared_memory(cl, rows, ci, co, group, dtype, act, shape):  # noqa: F811
    plan = cl.W4Plan(rows, ci, co, group, dtype, act)
    m = re.search(r"x in shared memory rows=(\d+)x8 warps=(\d+) tiles=(\d+) ctas=(\d+)$", plan.describe())
    assert m and (int(m[1]), int(m[2])) == shape, plan.describe()
    assert int(m[3]) > int(m[4])                          # tiles than CTAs
    against_64_bits(cl, plan, rows, ci, co, group, dtype, act)


@pytest.mark.parametrize("rows,ci,co,group,dtype,act,shape", MANY)
def test_x_in_turns(cl, rows, ci, co, group, dtype, act, shape):  # noqa: F811
    plan = cl.W4Plan(rows, ci, co, group, dtype, act)
    m = re.search(r"x in turns rows=(\d+)x8 warps=8 wc=(\d+) ", plan.describe())
    assert m and (int(m[1]), int(m[2])) == shape, plan.describe()
    against_64_bits(cl, plan, rows, ci, co, group, dtype, act)


def test_the_lists_hold_every_shape():
    few = {(c[4],) + c[6] for c in FEW}
    assert few == {(t, n, w) for t in ("bf16", "f32") for n in (1, 2, 4) for w in (8, 16)}
    many = {(c[4],) + c[6] for c in MANY}
    assert many == ({("bf16", n, w) for n in (1, 2, 4, 8) for w in (2, 4, 8)} - {("bf16", 8, 2)} |
                    {("f32", n, w) for n in (1, 2, 4, 8) for w in (2, 4, 8)} - {("f32", 4, 2), ("f32", 8, 2), ("f32", 8, 4)})
