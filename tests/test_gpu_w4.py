"""The pointwise layer with 4-bit weights against the same sum in 64 bits.

Tolerance: products are exact in fp32 and sums run in fp32 on the tensor
core, c_in / 16 steps of 2^-23 at most relative to the running sum of
magnitudes, then the groups': (c_in / 16 + groups + 16) 2^-23 of
sum |w x| + |bias|; a bf16 result adds 2^-8 of its size; the activations
2e-6 (1 + |z|)."""
import pytest
import torch

pytestmark = pytest.mark.gpu
DT = {"f32": torch.float32, "bf16": torch.bfloat16}


@pytest.fixture(scope="module")
def cl():
    from convolution_nhwc_implicit_gb300 import build
    build.build()
    import convolution_nhwc_implicit_gb300 as cl
    return cl


def inputs(rows, ci, co, group, dtype, seed=0):
    g = torch.Generator("cpu").manual_seed(seed)
    x = torch.randn(rows, ci, generator=g).to(DT[dtype])
    codes = torch.randint(0, 256, (co, (ci + 1) // 2), generator=g, dtype=torch.int64).to(torch.uint8)
    scales = (0.01 + 0.02 * torch.rand(co, -(-ci // group), generator=g)).to(DT[dtype])
    bias = 0.1 * torch.randn(co, generator=g)
    return x, codes, scales, bias


def weights64(codes, scales, ci, group):
    q = torch.stack([codes & 15, codes >> 4], dim=2).flatten(1)[:, :ci].double() - 8
    return q * scales.double().repeat_interleave(group, dim=1)[:, :ci]


def check(y, x, w, bias, act, dtype, ng):
    z = x.double() @ w.t() + bias.double()
    size = x.double().abs() @ w.abs().t() + bias.double().abs()
    tol = (x.shape[1] / 16 + ng + 16) * 2.0 ** -23 * size
    ref = z
    if act == "relu":
        ref = z.clamp(min=0)
    elif act == "mish":
        ref = z * torch.tanh(torch.nn.functional.softplus(z))
        tol = 1.1 * tol + 2e-6 * (1 + z.abs())
    if dtype == "bf16":
        tol = tol + 2.0 ** -8 * ref.abs()
    err = (y.double().cpu() - ref).abs()
    assert (err <= tol).all(), (float((err / tol).max()), int((err > tol).sum()))


CASES = [
    # rows, c_in, c_out, group, dtype, act
    (1, 1, 1, 32, "bf16", "none"),
    (1, 31, 3, 32, "f32", "none"),
    (1, 1024, 1000, 128, "bf16", "none"),
    (1, 4096, 48, 64, "bf16", "mish"),
    (2, 129, 17, 128, "bf16", "relu"),        # a last group and a last unit of one channel
    (5, 640, 100, 64, "f32", "mish"),
    (8, 264, 33, 32, "bf16", "none"),         # whole eights, not whole groups
    (9, 264, 33, 32, "bf16", "none"),         # ... a second block of rows
    (13, 2047, 61, 32, "f32", "relu"),        # odd channels: single loads
    (17, 333, 16, 64, "bf16", "mish"),
    (32, 512, 64, 128, "f32", "none"),
    (33, 256, 40, 64, "bf16", "relu"),
    (64, 200, 24, 32, "f32", "none"),
    (65, 384, 31, 128, "bf16", "none"),       # a second CTA of rows
    (150, 96, 20, 32, "f32", "none"),
    (1, 8192, 160, 128, "f32", "none"),
    (3, 12288, 32, 32, "bf16", "none"),
]


@pytest.mark.parametrize("rows,ci,co,group,dtype,act", CASES)
def test_against_64_bits(cl, rows, ci, co, group, dtype, act):
    x, codes, scales, bias = inputs(rows, ci, co, group, dtype)
    plan = cl.W4Plan(rows, ci, co, group, dtype, act)
    packed = plan.pack(codes.cuda())
    buf = torch.full((rows * co + 64,), 9.0, dtype=DT[dtype], device="cuda")
    y = buf[:rows * co].view(rows, co)
    plan.run(x.cuda(), packed, scales.cuda(), bias.cuda(), y)
    check(y, x, weights64(codes, scales, ci, group), bias, act, dtype, scales.shape[1])
    assert bool((buf[rows * co:] == 9).all())


def test_every_code_in_every_place(cl):
    """Unit inputs read each weight back exactly: rows of the identity pick a
    channel, so y is the weight itself (|code - 8| times a power of two)."""
    ci, co, group = 192, 40, 64
    g = torch.Generator("cpu").manual_seed(5)
    codes = torch.randint(0, 256, (co, ci // 2), generator=g, dtype=torch.int64).to(torch.uint8)
    scales = torch.pow(2.0, torch.randint(-3, 4, (co, 3), generator=g).float())
    want = weights64(codes, scales, ci, group)
    for dtype in ("bf16", "f32"):
        plan = cl.W4Plan(ci, ci, co, group, dtype)
        y = torch.empty(ci, co, device="cuda", dtype=DT[dtype])
        plan.run(torch.eye(ci, device="cuda", dtype=DT[dtype]), plan.pack(codes.cuda()), scales.to(DT[dtype]).cuda(), None, y)
        assert torch.equal(y.double().cpu(), want.t())


def test_fp32_rows_keep_their_digits(cl):
    """fp32 rows are split in three bf16 parts: values of 24 significant bits,
    the largest fp32 among them, come through a weight of one exactly."""
    ci = 128
    g = torch.Generator("cpu").manual_seed(6)
    vals = torch.randn(64, generator=g) * torch.pow(2.0, torch.randint(-60, 60, (64,), generator=g).float())
    vals[0], vals[1], vals[2] = 3.402823466e38, -3.402823466e38, 1.0 + 2.0 ** -23
    x = torch.zeros(64, ci)
    x[torch.arange(64), torch.arange(64)] = vals
    codes = torch.full((16, ci // 2), 0x99, dtype=torch.uint8)  # every weight is 1
    plan = cl.W4Plan(64, ci, 16, 128, "f32")
    y = torch.empty(64, 16, device="cuda")
    plan.run(x.cuda(), plan.pack(codes.cuda()), torch.ones(16, 1, device="cuda"), None, y)
    assert torch.equal(y.cpu(), vals[:, None].expand(64, 16))


def test_non_finite_rows(cl):
    """An infinity or a NaN reaches its own row's outputs and no other's."""
    x, codes, scales, bias = inputs(9, 256, 32, 64, "f32", 7)
    codes = codes | 0x11                                # no weight is zero: (odd code - 8) is odd
    x[2, 17], x[5, 200] = float("inf"), float("nan")
    plan = cl.W4Plan(9, 256, 32, 64, "f32")
    y = torch.empty(9, 32, device="cuda")
    plan.run(x.cuda(), plan.pack(codes.cuda()), scales.cuda(), bias.cuda(), y)
    y = y.cpu()
    assert torch.isinf(y[2]).all() and torch.isnan(y[5]).all()
    assert torch.isfinite(y[[0, 1, 3, 4, 6, 7, 8]]).all()


@pytest.mark.parametrize("co,ci,group,dtype", [(5, 100, 32, "f32"), (33, 255, 64, "bf16"), (4, 512, 128, "bf16"), (1, 1, 32, "f32")])
def test_quantize(cl, co, ci, group, dtype):
    g = torch.Generator("cpu").manual_seed(8)
    w = (torch.randn(co, ci, generator=g) * 0.05).to(DT[dtype])
    w[0, :min(ci, group)] = 0                            # a group of zeros
    codes, scales = cl.w4_quantize(w.cuda(), group)
    ng = -(-ci // group)
    wide = torch.zeros(co, ng * group)
    wide[:, :ci] = w.float()
    s = (wide.view(co, ng, group).abs().amax(dim=2) / 7).to(DT[dtype])
    assert torch.equal(scales.cpu(), s)
    sf = s.float().repeat_interleave(group, dim=1)[:, :ci]
    q = torch.where(sf > 0, torch.round(w.float() / torch.where(sf > 0, sf, torch.ones_like(sf))).clamp(-8, 7), torch.zeros_like(sf))
    c = codes.cpu()
    got = torch.stack([c & 15, c >> 4], dim=2).flatten(1)[:, :ci].float() - 8
    assert torch.equal(got, q)


def test_streams_graph_and_refusals(cl):
    x, codes, scales, bias = (t.cuda() for t in inputs(3, 256, 32, 64, "bf16", 9))
    plan = cl.W4Plan(3, 256, 32, 64, "bf16", "mish")
    packed = plan.pack(codes)
    a, b, c = (torch.zeros(3, 32, device="cuda", dtype=torch.bfloat16) for _ in range(3))
    plan.run(x, packed, scales, bias, a)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    plan.run(x, packed, scales, bias, b, stream=s)
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        plan.run(x, packed, scales, bias, c)
    g.replay()
    torch.cuda.synchronize()
    assert torch.equal(a, b) and torch.equal(a, c)
    with pytest.raises(TypeError):
        plan.run(x.float(), packed, scales, bias, a)
    with pytest.raises(ValueError):
        plan.run(x[:2], packed, scales, bias, a)
    with pytest.raises(ValueError):
        plan.run(x, codes, scales, bias, a)
    with pytest.raises(ValueError):
        plan.run(x, packed, scales[:, :2], bias, a)
    with pytest.raises(ValueError):
        plan.run(x.t().contiguous().t(), packed, scales, bias, a)
    with pytest.raises(TypeError):
        plan.run(x, packed, scales, bias.bfloat16(), a)
    lib = cl.load_library()
    p = [t.data_ptr() for t in (x, packed, scales, bias, a)]
    assert lib.conv_run_w4(plan.handle, None, p[1], p[2], p[3], p[4], None) == -1
    assert lib.conv_run_w4(plan.handle, p[0], p[1] + 4, p[2], p[3], p[4], None) == -4
    assert lib.conv_run_w4(plan.handle, p[0], p[1], p[2], p[3], p[0], None) == -5
    assert lib.conv_run(plan.handle, p[0], p[1], None, p[4], None) == -9
    assert lib.conv_run_groupnorm(plan.handle, p[0], 0, None, None, p[4], 0, None, None, None, None) == -9
    assert cl.W4Plan(0, 64, 64).run(x[:0, :64].contiguous(), torch.empty(4096, dtype=torch.uint8, device="cuda"),
                                    torch.empty(64, 1, device="cuda", dtype=torch.bfloat16), None,
                                    torch.empty(0, 64, device="cuda", dtype=torch.bfloat16)) is None
