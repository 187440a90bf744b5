"""Infinities and NaN through the 4-bit layer: every output is finite, NaN or an
infinity where the formula in 64 bits is, for each activation, type and kernel.
Weights that hold them are quantised to groups that answer NaN, not zero."""
import pytest
import torch

from test_gpu_w4 import DT, cl, inputs, weights64  # noqa: F401  (cl: the fixture)

pytestmark = pytest.mark.gpu


def kind(v):
    """0 finite, 1 NaN, 2 and 3 the infinities."""
    return v.isnan() * 1 + (v == float("inf")) * 2 + (v == float("-inf")) * 3


@pytest.mark.parametrize("rows", [1, 9, 40])   # x whole in shared memory, or in turns
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("act", ["none", "relu", "mish"])
def test_kinds_of_answers(cl, rows, dtype, act):  # noqa: F811
    x, codes, scales, bias = inputs(rows, 256, 48, 64, dtype, 7)
    codes = codes | 0x11                      # no weight is zero: (odd code - 8) is odd
    if rows > 1:
        x[2, 17], x[5, 200], x[6, 3] = float("inf"), float("nan"), float("-inf")
    else:
        x[0, 9] = float("nan")
    scales[7, 1], bias[9] = float("nan"), float("nan")
    bias[11], bias[12] = float("inf"), float("-inf")
    plan = cl.W4Plan(rows, 256, 48, 64, dtype, act)
    assert ("in turns" in plan.describe()) == (rows > 32)
    y = torch.empty(rows, 48, device="cuda", dtype=DT[dtype])
    plan.run(x.cuda(), plan.pack(codes.cuda()), scales.cuda(), bias.cuda(), y)
    z = x.double() @ weights64(codes, scales, 256, 64).t() + bias.double()
    if act == "relu":
        z = z.clamp(min=0)
    elif act == "mish":
        z = z * torch.tanh(torch.nn.functional.softplus(z))
    assert torch.equal(kind(y.cpu().double()), kind(z))

@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("what", [float("nan"), float("inf"), float("-inf")])
def test_quantised_weights(cl, dtype, what):  # noqa: F811
    g = torch.Generator("cpu").manual_seed(3)
    w = torch.randn(32, 200, generator=g).to(DT[dtype])
    clean_codes, clean_scales = cl.w4_quantize(w.cuda(), 64)
    w[3, 70], w[17, 199], w[20, 0] = what, what, what
    codes, scales = cl.w4_quantize(w.cuda(), 64)
    at = torch.zeros(32, 4, dtype=torch.bool)
    at[3, 1] = at[17, 3] = at[20, 0] = True
    assert torch.equal(~torch.isfinite(scales.cpu()), at)
    assert torch.equal(scales.cpu()[~at], clean_scales.cpu()[~at])
    same = ~at.repeat_interleave(32, dim=1)[:, :100]      # (64 channels are 32 bytes)
    assert torch.equal(codes.cpu()[same], clean_codes.cpu()[same])
    plan = cl.W4Plan(2, 200, 32, 64, dtype)
    y = torch.empty(2, 32, device="cuda", dtype=DT[dtype])
    plan.run(torch.randn(2, 200, generator=g).to(DT[dtype]).cuda(), plan.pack(codes), scales, None, y)
    assert torch.equal(y.cpu().isnan(), at.any(dim=1).expand(2, 32))
