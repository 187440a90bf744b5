"""Group norm's gradient with Mish where gamma makes z huge: Mish' is 1 above
and 0 below (to fp32), whatever z is."""
import pytest
import torch

from test_gpu_groupnorm import DT, U, cl, close, draw, reference  # noqa: F401  (cl: the fixture)

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("shape,groups", [((2, 6, 6, 24), 4), ((1, 160, 160, 64), 4)])   # one launch, two launches
@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("size", [1e8, 1e12, 1e18])
def test_slope_far_out(cl, shape, groups, dtype, size):  # noqa: F811
    """dz = dy or 0, off by 2e-6 of it; the sums by 64 u of their terms more;
    xhat as in the other tests; values whose |z| is below 1e4 may take any
    slope between (none lies there unless xhat does, within 1e4 / size)."""
    n, h, w, c = shape
    x, dy = draw(shape, DT[dtype], 1), draw(shape, DT[dtype], 2, mean=0.1, std=0.3)
    gamma = torch.full((c,), size)
    plan = cl.GroupNormPlan(*shape, groups, 1e-5, dtype, "mish")
    y, dx = torch.empty_like(x), torch.empty_like(x)
    mean, rstd = (torch.empty(n, groups, device="cuda") for _ in range(2))
    dg, db = (torch.empty(c, device="cuda") for _ in range(2))
    ga = gamma.cuda()
    plan.run(x, ga, None, y, mean, rstd)
    plan.run_backward(x, ga, None, mean, rstd, dy, dx, dg, db)
    v = x.double().cpu().reshape(n, h * w, groups, c // groups)
    r = reference(x, None, None, groups, 1e-5, "none")
    xh = r["z"]
    exh = r["ztol"]
    dyv = dy.double().cpu().reshape(v.shape)
    near = xh.abs() <= 1e4 / size + exh       # the side may be either
    dz = torch.where(xh > 0, dyv, torch.zeros_like(dyv))
    edz = 2e-6 * dz.abs() + torch.where(near, dyv.abs() * 1.2, torch.zeros_like(dyv)) + 64 * U * dz.abs()
    close(db, dz.sum(dim=(0, 1)).reshape(c), edz.sum(dim=(0, 1)).reshape(c), False, "dbeta")
    close(dg, (dz * xh).sum(dim=(0, 1)).reshape(c), (edz * xh.abs() + dz.abs() * exh).sum(dim=(0, 1)).reshape(c), False, "dgamma")
    gh = dz * size
    m1, m2 = gh.mean(dim=(1, 3), keepdim=True), (gh * xh).mean(dim=(1, 3), keepdim=True)
    want = r["rstd"] * (gh - m1 - xh * m2)
    em1 = (edz * size).mean(dim=(1, 3), keepdim=True)
    em2 = (edz * size * xh.abs() + gh.abs() * exh).mean(dim=(1, 3), keepdim=True)
    tol = r["rstd"] * (edz * size + em1 + xh.abs() * em2 + exh * m2.abs() + 4e-6 * (gh.abs() + m1.abs() + (xh * m2).abs()))
    close(dx, want, tol, dtype == "bf16", "dx", near)
    y64 = torch.where(xh > 0, xh * size, torch.zeros_like(xh))
    close(y, y64, size * exh * 1.5 + 2e-6 * y64.abs(), dtype == "bf16", "y", near)
