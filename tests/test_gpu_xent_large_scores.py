"""The class loss of scores in the hundreds: exponentials are of differences,
not of scores and maxima each multiplied by log2 e first, whose rounding grows
with the scores."""
import pytest
import torch

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def cl():
    from convolution_nhwc_implicit_gb300 import build
    build.build()
    import convolution_nhwc_implicit_gb300 as cl
    return cl


@pytest.mark.parametrize("classes", [300, 1000])
def test_lse_is_rounded_once(cl, classes):
    """Scores are exact (one product of few bits a class).  lse = m + log s: m
    is exact; a term of s, e^(l - m), is off by its exponent's two roundings,
    |l - m| 2^-23 of it (at most 2^-23 / e of 1), and by the exponential's 2^-21;
    s by at most 48 additions of 2^-24 more: 2^-18 of it in all.  log s <= 7 is
    off by its own 2^-22, and the sum is rounded once."""
    n, d = 512, 8
    g = torch.Generator("cpu").manual_seed(1)
    x, w = torch.zeros(n, d), torch.zeros(classes, d)
    x[:, 0] = 8.0
    x[:, 1] = 0.25 * torch.randint(-16, 17, (n,), generator=g)
    w[:, 0] = 0.5 * torch.randint(150, 256, (classes,), generator=g)
    w[:, 1] = 1.0 * torch.randint(-8, 9, (classes,), generator=g)
    x, w = x.bfloat16(), w.bfloat16()
    z = x.double() @ w.double().t()
    assert z.max() > 500 and torch.equal(z.float().double(), z)
    want = torch.logsumexp(z, dim=1)
    t = z.argmax(dim=1).to(torch.int32)
    plan = cl.ClassLossPlan(n, d, classes)
    loss, lse, row = torch.empty((), device="cuda"), torch.empty(n, device="cuda"), torch.empty(n, device="cuda")
    plan.run(x.cuda(), w.cuda(), t.cuda(), loss, lse, row)
    spacing = 2.0 ** (torch.floor(torch.log2(want)) - 23)
    err = (lse.double().cpu() - want).abs()
    assert (err <= 0.5 * spacing + 2.0 ** -18 + 7 * 2.0 ** -22).all(), float((err / spacing).max())


def test_gradient_of_a_confident_row(cl):
    """Two classes eight apart, the label the likelier: g = exp(l - lse) - 1 is
    small and keeps its digits, lse being what the caller gives.  g is off by
    the exponential's 2^-21 and its rounding to bf16 (2^-8), dx by the sum of
    those times |w| and its own rounding (2^-8)."""
    n, d = 256, 8
    x, w = torch.zeros(n, d), torch.zeros(2, d)
    x[:, 0] = 8.0
    x[:, 1] = 0.25 * torch.arange(n).remainder(64)
    w[0, 0], w[1, 0], w[0, 1], w[1, 1] = 90.0, 89.0, 1.0, 1.0
    x, w = x.bfloat16(), w.bfloat16()
    t = torch.zeros(n, dtype=torch.int32)
    z = x.double() @ w.double().t()
    lse = torch.logsumexp(z, dim=1).float()
    g = torch.exp(z - lse.double()[:, None])
    g[:, 0] -= 1
    eg = 2.0 ** -21 + 2.0 ** -8 * g.abs()
    want = g @ w.double() / n
    tol = eg @ w.double().abs() / n + 2.0 ** -8 * want.abs()
    plan = cl.ClassLossPlan(n, d, 2)
    dx, dw = torch.empty_like(x).cuda(), torch.empty_like(w).cuda()
    plan.run_backward(x.cuda(), w.cuda(), t.cuda(), lse.cuda(), dx, dw)
    err = (dx.double().cpu() - want).abs()
    assert (err <= tol).all(), float((err / tol.clamp(min=1e-300)).max())
    want = g.t() @ x.double() / n
    tol = eg.t() @ x.double().abs() / n + 2.0 ** -8 * want.abs()
    err = (dw.double().cpu() - want).abs()
    assert (err <= tol).all(), float((err / tol.clamp(min=1e-300)).max())
