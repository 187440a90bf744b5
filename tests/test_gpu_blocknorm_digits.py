"""The gradient of the norms around a block where a mean is far above the spread.

Rows are 1000 + d and 1000 - d with d whole multiples of 2^-14, an fp32 number's
step there: their mean is 1000 exactly, and so is every difference from it.  With
those statistics given (r rounded to fp32 first), a normalised value is one
product, off by u = 2^-24 of itself; everything else as in test_gpu_blocknorm.py.
(Formed as v r - m r its error would be that of m r, 2^14 u.)"""
import pytest
import torch
from test_gpu_blocknorm import U, back64, cl, close, draw, mean  # noqa: F401

pytestmark = pytest.mark.gpu

SHAPES = [(2, 3, 5, 8), (1, 9, 7, 64), (2, 6, 7, 264), (1, 5, 5, 2056), (3, 40, 40, 96), (1, 1, 40, 8192)]


def far(shape, seed, wide):
    """Maps, and their normalised values and statistics: m exact, r an fp32 number."""
    n, h, w, c = shape
    g = torch.Generator("cuda").manual_seed(seed)
    d = torch.randint(1, 1 << 11, (n, h, w, c // 2), generator=g, device="cuda").double() * 2.0 ** -14
    v = torch.cat([1000 + d, 1000 - d], dim=-1)
    buf = torch.full((n, h, w, c + wide), 7.0, device="cuda")
    buf[..., wide:] = v.float()
    assert torch.equal(buf[..., wide:].double(), v)
    r = (1 / torch.sqrt(mean((v - 1000) ** 2) + 1e-5)).float()
    return buf[..., wide:], (v - 1000) * r.double(), r


def statistics(shape, which, r):
    s = torch.zeros(*shape[:3], 4, device="cuda")
    s[..., 1], s[..., 3] = 1.0, 1.0
    s[..., 2 * which], s[..., 2 * which + 1] = 1000.0, r[..., 0]
    return s


@pytest.mark.parametrize("shape", SHAPES)
@pytest.mark.parametrize("wide", [0, 1])
def test_norm_after_the_block(cl, shape, wide):  # noqa: F811
    x, hat, r = far(shape, 1, wide)
    c = shape[3]
    gamma = 1 + 0.3 * draw((1, 1, 1, c), torch.float32, 2).view(c)
    dz = (hat / gamma.double()).float() + draw(shape, torch.float32, 3, std=0.1)   # (along the normalised values)
    plan = cl.BlockNormPlan(*shape, "none", "layer", 1e-5, "f32")
    dx, dg, db = torch.empty(shape, device="cuda"), torch.empty(c, device="cuda"), torch.empty(c, device="cuda")
    plan.run_backward(x, None, statistics(shape, 1, r), None, dz, dx, None, pre_gamma=gamma, dpre_gamma=dg, dpre_beta=db)
    e = dz.double() * gamma.double()
    ref, tol = back64(e, U * e.abs(), hat, U * hat.abs(), r.double(), torch.zeros_like(hat), "layer")
    close(dx, ref, tol, False, "dx")
    terms = dz.double() * hat
    close(dg, terms.sum(dim=(0, 1, 2)), 301 * U * terms.abs().sum(dim=(0, 1, 2)), False, "dg")


@pytest.mark.parametrize("shape", SHAPES)
@pytest.mark.parametrize("wide", [0, 1])
def test_norm_of_the_block(cl, shape, wide):  # noqa: F811
    f, hat, r = far(shape, 4, wide)
    n, c = shape[0], shape[3]
    gamma, scale = (1 + 0.3 * draw((1, 1, 1, c), torch.float32, 5 + i).view(c) for i in range(2))
    k = gamma.double() * scale.double()
    dy = (hat / k).float() + draw(shape, torch.float32, 7, std=0.1)
    x = draw(shape, torch.float32, 8)
    plan = cl.BlockNormPlan(*shape, "layer", "none", 1e-5, "f32")
    dx, df, dg = torch.empty(shape, device="cuda"), torch.empty(shape, device="cuda"), torch.empty(c, device="cuda")
    plan.run_backward(x, f, statistics(shape, 0, r), dy, None, dx, df, scale=scale, post_gamma=gamma, dpost_gamma=dg)
    assert torch.equal(dx, dy)
    v = dy.double() * k
    ref, tol = back64(v, 3 * U * v.abs(), hat, U * hat.abs(), r.double(), torch.zeros_like(hat), "layer")
    close(df, ref, tol, False, "df")
    terms = dy.double() * hat * scale.double()
    close(dg, terms.sum(dim=(0, 1, 2)), 303 * U * terms.abs().sum(dim=(0, 1, 2)), False, "dg")
