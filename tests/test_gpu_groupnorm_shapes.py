"""Group norm where a CTA of a cluster holds more than 256 channels, so that a
call's addresses choose between one launch and two, and batches of more images
than the card holds CTAs, whose gradient joins the channels' sums of a run an
image; against 64 bits with the tolerances of the other tests."""
import pytest
import torch

from test_gpu_groupnorm import DT, U, cl, close, draw, reference  # noqa: F401  (cl: the fixture)

pytestmark = pytest.mark.gpu


def against_64_bits(cl, plan, shape, groups, dtype, act, wide=0, off=0):  # noqa: F811
    n, h, w, c = shape
    dt = DT[dtype]
    x, dy = draw(shape, dt, 1, wide, off), draw(shape, dt, 2, wide, off, 0.1, 0.3)
    gen = torch.Generator("cpu").manual_seed(3)
    gamma, beta = 1 + 0.3 * torch.randn(c, generator=gen), 0.3 * torch.randn(c, generator=gen)
    ref = reference(x, gamma, beta, groups, 1e-5, act, dy)
    y, dx = draw(shape, dt, 4, wide, off), draw(shape, dt, 5, wide, off)
    mean, rstd = (torch.full((n, groups), 9.0, device="cuda") for _ in range(2))
    dg, db = (torch.full((c,), 9.0, device="cuda") for _ in range(2))
    ga, be = gamma.cuda(), beta.cuda()
    plan.run(x, ga, be, y, mean, rstd)
    plan.run_backward(x, ga, be, mean, rstd, dy, dx, dg, db)
    torch.cuda.synchronize()
    bf = dtype == "bf16"
    big = x.double().abs().max().cpu()
    close(mean, ref["mean"], 4 * U * big, False, "mean")
    close(rstd, ref["rstd"], 4e-6 * ref["rstd"] + 8 * U * big * U * big * ref["rstd"] ** 3, False, "rstd")
    close(y, ref["y"], 1.5 * ref["ztol"], bf, "y")
    close(dg, ref["dgamma"], ref["dgamma_tol"], False, "dgamma")
    close(db, ref["dbeta"], ref["dbeta_tol"], False, "dbeta")
    close(dx, ref["dx"], ref["dx_tol"], bf, "dx", ref["kink"])
    for t in (y, dx):
        if wide:
            whole = t._base
            assert bool((whole[..., :off] == 7).all()) and bool((whole[..., off + c:] == 7).all())


@pytest.mark.parametrize("n,h,w,c,groups,dtype,act", [
    (2, 6, 5, 744, 8, "bf16", "mish"),       # one CTA block of all eight groups
    (3, 10, 9, 1800, 6, "bf16", "relu"),     # two groups a CTA
    (1, 7, 7, 2072, 7, "bf16", "none"),      # one group a CTA
    (2, 4, 4, 1500, 5, "bf16", "mish"),      # 4-byte vectors at the widest
    (1, 5, 4, 2048, 1, "bf16", "relu"),      # as many vectors as threads
    (2, 9, 8, 780, 3, "f32", "mish"),
    (1, 5, 5, 1024, 1, "f32", "none"),
    (4, 6, 6, 1040, 4, "f32", "relu"),
    (9, 4, 5, 744, 8, "bf16", "mish"),       # ... the gradient in two launches
])
@pytest.mark.parametrize("wide,off", [(0, 0), (16, 8), (6, 2), (5, 3)])
def test_wide_clusters(cl, n, h, w, c, groups, dtype, act, wide, off):  # noqa: F811
    plan = cl.GroupNormPlan(n, h, w, c, groups, 1e-5, dtype, act)
    assert plan.describe().split(" forward: ")[1].startswith("clusters") and plan.workspace_bytes > 0, plan.describe()
    against_64_bits(cl, plan, (n, h, w, c), groups, dtype, act, wide, off)


@pytest.mark.parametrize("n,h,w,c,groups,dtype,act", [
    (310, 3, 3, 1024, 32, "bf16", "mish"),   # more images than the gradient's CTAs: a run an image
    (460, 2, 3, 200, 8, "f32", "relu"),
    (460, 7, 5, 33, 3, "f32", "none"),
    (150, 20, 20, 96, 12, "bf16", "relu"),   # two runs an image
    (1000, 1, 1, 64, 4, "bf16", "none"),
])
def test_many_images(cl, n, h, w, c, groups, dtype, act):  # noqa: F811
    plan = cl.GroupNormPlan(n, h, w, c, groups, 1e-5, dtype, act)
    assert " px" in plan.describe().split("gradient: ")[1], plan.describe()
    against_64_bits(cl, plan, (n, h, w, c), groups, dtype, act)
