"""Infinities and NaN through the 4-bit layer: every output is finite, NaN or an
infinity where the formula in 64 bits is, for each activation, type and kernel."""
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
