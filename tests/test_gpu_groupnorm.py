"""Group norm with an activation against a plain 64-bit form of the same
formulas, forward and gradient, and the gradient against differences of the
forward run.

Tolerances, with u = 2^-24: the mean is off by at most a few roundings of the
largest value, 4 u max|x|, which moves z by that times |gamma| rstd; rstd and
the remaining operations are relative, bounded by 2e-6 (1 + |z|) (the fast
exponential of bf16 maps included); a bf16 result adds its rounding, 2^-8 of
its size.  ReLU's derivative jumps at z = 0: values whose z lies within the
forward tolerance of 0 may take either side and are left out of dx's
comparison and allowed for in the sums.  Sums of products are allowed 64 u of
their terms' absolute sum (chains of at most 64 additions, joined pairwise)."""
import pytest
import torch

pytestmark = pytest.mark.gpu
U = 2.0 ** -24
DT = {"f32": torch.float32, "bf16": torch.bfloat16}


@pytest.fixture(scope="module")
def cl():
    from convolution_nhwc_implicit_gb300 import build
    build.build()
    import convolution_nhwc_implicit_gb300 as cl
    return cl


def act64(z, act):
    if act == "relu":
        return z.clamp(min=0), (z > 0).double()
    if act == "mish":
        sp = torch.nn.functional.softplus(z)
        t = torch.tanh(sp)
        return z * t, t + z * (1 - t * t) * torch.sigmoid(z)
    return z, torch.ones_like(z)


def reference(x, gamma, beta, groups, eps, act, dy=None):
    """Everything in 64 bits on the CPU; maps as [n, hw, g, cg]."""
    n, h, w, c = x.shape
    v = x.double().cpu().reshape(n, h * w, groups, c // groups)
    ga = (torch.ones(c) if gamma is None else gamma.cpu()).double().view(1, 1, groups, -1)
    be = (torch.zeros(c) if beta is None else beta.cpu()).double().view(1, 1, groups, -1)
    mean = v.mean(dim=(1, 3), keepdim=True)
    rstd = 1 / torch.sqrt(((v - mean) ** 2).mean(dim=(1, 3), keepdim=True) + eps)
    xh = (v - mean) * rstd
    z = xh * ga + be
    y, d = act64(z, act)
    out = dict(y=y, mean=mean, rstd=rstd, z=z)
    big = v.abs().amax(dim=(1, 3), keepdim=True)
    out["ztol"] = 2e-6 * (1 + z.abs()) + 4 * U * big * rstd * ga.abs()
    if dy is not None:
        g = dy.double().cpu().reshape(v.shape)
        dz = g * d
        out["dgamma"], out["dbeta"] = (dz * xh).sum(dim=(0, 1)).reshape(c), dz.sum(dim=(0, 1)).reshape(c)
        gh = dz * ga
        m1, m2 = gh.mean(dim=(1, 3), keepdim=True), (gh * xh).mean(dim=(1, 3), keepdim=True)
        out["dx"] = rstd * (gh - m1 - xh * m2)
        # errors: dz by its derivative's change over ztol (|act''| <= 1.5) and 2e-6, xhat by ztol / |gamma|
        kink = (z.abs() <= 2 * out["ztol"]) & (act == "relu")
        edz = g.abs() * (3 * out["ztol"] + 4e-6) if act == "mish" else 4e-6 * dz.abs()
        exh = 2e-6 * (1 + xh.abs()) + 4 * U * big * rstd
        jump = torch.where(kink, g.abs(), torch.zeros_like(g))
        out["dbeta_tol"] = (edz + jump + 64 * U * dz.abs()).sum(dim=(0, 1)).reshape(c)
        out["dgamma_tol"] = ((edz + jump + 64 * U * dz.abs()) * xh.abs() + dz.abs() * exh).sum(dim=(0, 1)).reshape(c)
        em1 = ((edz + jump + 64 * U * dz.abs()) * ga.abs()).mean(dim=(1, 3), keepdim=True)
        em2 = ((edz + jump + 64 * U * dz.abs()) * ga.abs() * xh.abs() + gh.abs() * exh).mean(dim=(1, 3), keepdim=True)
        out["dx_tol"] = rstd * (edz * ga.abs() + em1 + xh.abs() * em2 + exh * m2.abs() + 4e-6 * (gh.abs() + m1.abs() + (xh * m2).abs()))
        out["kink"] = kink
    return out


def close(got, ref, tol, bf16, what, skip=None):
    got = got.double().cpu().reshape(ref.shape)
    lim = tol + (ref.abs() * 2.0 ** -8 if bf16 else 0) + 1e-30
    bad = ~((got - ref).abs() <= lim)
    if skip is not None:
        bad &= ~skip
    assert not bad.any(), (what, int(bad.sum()), float(((got - ref).abs() / lim)[bad].max()))


def draw(shape, dt, seed, wide=0, off=0, mean=0.5, std=1.0):
    n, h, w, c = shape
    g = torch.Generator("cpu").manual_seed(seed)
    v = (torch.randn(n, h, w, c, generator=g) * std + mean).to(dt)
    if wide == 0:
        return v.cuda()
    buf = torch.full((n, h, w, c + wide), 7.0, dtype=dt, device="cuda")
    buf[..., off:off + c] = v.cuda()
    return buf[..., off:off + c]


CASES = [
    # n, h, w, c, groups, dtype, act, wide, off
    (1, 1, 1, 1, 1, "f32", "none", 0, 0),            # one value a group: xhat = 0
    (2, 1, 1, 32, 32, "bf16", "mish", 0, 0),
    (3, 1, 1, 64, 4, "bf16", "none", 0, 0),          # one pixel
    (1, 7, 7, 512, 32, "bf16", "relu", 0, 0),
    (2, 5, 3, 60, 6, "f32", "relu", 0, 0),           # groups of ten
    (2, 5, 3, 60, 6, "bf16", "mish", 0, 0),          # ... 4-byte vectors
    (3, 9, 11, 33, 3, "bf16", "none", 0, 0),         # odd channels
    (3, 9, 11, 33, 11, "f32", "mish", 0, 0),         # groups of three
    (1, 13, 17, 24, 8, "bf16", "mish", 0, 0),        # groups end inside a vector
    (2, 20, 20, 128, 1, "bf16", "relu", 0, 0),       # one group: layer norm of the image
    (2, 20, 20, 40, 40, "f32", "mish", 0, 0),        # a group a channel
    (1, 3, 5, 2056, 8, "bf16", "none", 0, 0),        # more vectors than the CTA threads
    (1, 2, 2, 8192, 32, "f32", "relu", 0, 0),        # the most channels
    (1, 3, 3, 8191, 1, "bf16", "mish", 0, 0),
    (4, 40, 40, 64, 16, "bf16", "mish", 64, 64),     # slice of a concatenated buffer
    (2, 10, 10, 48, 6, "bf16", "relu", 13, 5),       # a slice at odd addresses
    (2, 10, 10, 48, 6, "f32", "mish", 3, 1),
    (1, 160, 160, 32, 8, "bf16", "mish", 0, 0),
    (5, 31, 33, 96, 12, "f32", "none", 0, 0),
    (2, 130, 131, 33, 3, "bf16", "mish", 0, 0),      # maps too large for shared memory: odd channels
    (1, 150, 151, 66, 6, "f32", "relu", 2, 1),       # ... a slice at odd addresses
    (3, 120, 120, 60, 6, "bf16", "none", 0, 0),
    (2, 90, 90, 512, 4, "bf16", "mish", 0, 0),       # ... groups of 128 channels
    (1, 100, 100, 300, 300, "f32", "mish", 0, 0),    # more groups than a CTA stages runs of
    (9, 12, 12, 64, 8, "bf16", "relu", 0, 0),        # more images than a cluster holds
    (4, 40, 40, 60, 10, "f32", "mish", 0, 0),        # a last CTA with fewer groups than the others
    (6, 160, 160, 128, 32, "f32", "mish", 0, 0),     # more than one pass over L2
]


@pytest.mark.parametrize("n,h,w,c,groups,dtype,act,wide,off", CASES)
def test_forward_and_gradient(cl, n, h, w, c, groups, dtype, act, wide, off):
    shape, dt = (n, h, w, c), DT[dtype]
    x, dy = draw(shape, dt, 1, wide, off), draw(shape, dt, 2, wide, off, 0.1, 0.3)
    gen = torch.Generator("cpu").manual_seed(3)
    gamma, beta = 1 + 0.3 * torch.randn(c, generator=gen), 0.3 * torch.randn(c, generator=gen)
    ref = reference(x, gamma, beta, groups, 1e-5, act, dy)
    plan = cl.GroupNormPlan(n, h, w, c, groups, 1e-5, dtype, act)
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
    for t in (y, dx):  # nothing outside the slice was written
        if wide:
            whole = t._base
            assert bool((whole[..., :off] == 7).all()) and bool((whole[..., off + c:] == 7).all())


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_without_affine_or_statistics(cl, dtype):
    x = draw((2, 6, 5, 24), DT[dtype], 11)
    plan = cl.GroupNormPlan(2, 6, 5, 24, 4, 1e-3, dtype, "mish")
    ref = reference(x, None, None, 4, 1e-3, "mish", x)
    y, dx = torch.empty_like(x), torch.empty_like(x)
    plan.run(x, None, None, y)
    mean, rstd = (torch.empty(2, 4, device="cuda") for _ in range(2))
    plan.run(x, None, None, y, mean, rstd)
    plan.run_backward(x, None, None, mean, rstd, x, dx)
    close(y, ref["y"], 1.5 * ref["ztol"], dtype == "bf16", "y")
    close(dx, ref["dx"], ref["dx_tol"], dtype == "bf16", "dx")


def test_large_mean(cl):
    """A mean a thousand times the spread: the variance keeps its digits (each
    value is x = 1000 + r exactly in fp32; the pieces are summed about a value
    of their own)."""
    x = draw((2, 40, 40, 32), torch.float32, 21, mean=1000.0)
    ref = reference(x, None, None, 4, 1e-5, "none")
    plan = cl.GroupNormPlan(2, 40, 40, 32, 4, 1e-5, "f32", "none")
    y, mean, rstd = torch.empty_like(x), torch.empty(2, 4, device="cuda"), torch.empty(2, 4, device="cuda")
    plan.run(x, None, None, y, mean, rstd)
    close(rstd, ref["rstd"], 4e-6 * ref["rstd"], False, "rstd")
    close(y, ref["y"], 1.5 * ref["ztol"], False, "y")


def test_constant_and_non_finite_groups(cl):
    """Equal values give beta (variance 0, eps alone below the root); a NaN or
    an infinity spoils its own group only."""
    x = draw((2, 4, 4, 16), torch.float32, 31)
    x[0, :, :, 0:4] = 3.25
    x[1, 2, 1, 5] = float("nan")
    x[1, 0, 0, 9] = float("inf")
    beta = torch.linspace(-1, 1, 16, device="cuda")
    plan = cl.GroupNormPlan(2, 4, 4, 16, 4, 1e-5, "f32", "relu")
    y = torch.empty_like(x)
    plan.run(x, None, beta, y)
    y = y.cpu()
    assert torch.equal(y[0, :, :, 0:4], beta.cpu()[0:4].clamp(min=0).expand(4, 4, 4))
    assert torch.isnan(y[1, :, :, 4:8]).all() and torch.isnan(y[1, :, :, 8:12]).any()
    assert torch.isfinite(y[0]).all() and torch.isfinite(y[1, :, :, 0:4]).all() and torch.isfinite(y[1, :, :, 12:]).all()


@pytest.mark.parametrize("act", ["none", "mish"])
def test_gradient_against_differences(cl, act):
    """sum(dx v) against (L(x + e v) - L(x - e v)) / 2 e with L = sum(y dy), and
    the same for gamma and beta.  The difference is off by e^2/6 of the third
    derivative (of order 10 |dy| |v|^3 rstd^3 here) and by the forward run's
    rounding over e: 2e-3 of the sum of |dx v| covers both at e = 2^-7."""
    shape, c = (2, 6, 6, 24), 24
    x, dy, v = draw(shape, torch.float32, 41), draw(shape, torch.float32, 42, mean=0.0), draw(shape, torch.float32, 43, mean=0.0)
    ga, be = (draw((1, 1, 1, c), torch.float32, s).reshape(c) for s in (44, 45))
    vg, vb = (draw((1, 1, 1, c), torch.float32, s).reshape(c) for s in (46, 47))
    plan = cl.GroupNormPlan(*shape, 4, 1e-5, "f32", act)
    mean, rstd = (torch.empty(2, 4, device="cuda") for _ in range(2))

    def loss(xx, gg, bb):
        y = torch.empty_like(x)
        plan.run(xx, gg, bb, y, mean, rstd)
        return float((y.double() * dy.double()).sum())

    e = 2.0 ** -7
    loss(x, ga, be)
    dx, dg, db = torch.empty_like(x), torch.empty(c, device="cuda"), torch.empty(c, device="cuda")
    plan.run_backward(x, ga, be, mean, rstd, dy, dx, dg, db)
    for grad, d, at in ((dx, v, lambda s: (x + s * e * v, ga, be)), (dg, vg, lambda s: (x, ga + s * e * vg, be)),
                        (db, vb, lambda s: (x, ga, be + s * e * vb))):
        diff = (loss(*at(1)) - loss(*at(-1))) / (2 * e)
        terms = grad.double() * d.double()
        assert abs(float(terms.sum()) - diff) <= 2e-3 * float(terms.abs().sum()), act


def test_offsets_past_31_bits(cl):
    """Pixels whose element offsets pass 2^31 (a small slice of a very wide buffer)."""
    c, pitch, w = 16, (1 << 25) + 8, 70
    buf = torch.empty(1, 1, w, pitch, dtype=torch.bfloat16, device="cuda")
    x = buf[..., 8:8 + c]
    x.copy_(draw((1, 1, w, c), torch.bfloat16, 51))
    y = buf[..., 1024:1024 + c]
    ref = reference(x, None, None, 2, 1e-5, "relu", x)
    plan = cl.GroupNormPlan(1, 1, w, c, 2, 1e-5, "bf16", "relu")
    mean, rstd = (torch.empty(1, 2, device="cuda") for _ in range(2))
    plan.run(x, None, None, y, mean, rstd)
    close(y, ref["y"], 1.5 * ref["ztol"], True, "y")
    dx = buf[..., 2048:2048 + c]
    plan.run_backward(x, None, None, mean, rstd, x, dx)
    close(dx, ref["dx"], ref["dx_tol"], True, "dx", ref["kink"])


def test_streams_graph_and_repeat(cl):
    """The same bits on another stream, in a replayed graph and run after run."""
    shape = (4, 20, 20, 64)
    x, dy = draw(shape, torch.bfloat16, 61), draw(shape, torch.bfloat16, 62)
    plan = cl.GroupNormPlan(*shape, 8, 1e-5, "bf16", "mish")

    def outs():
        return [torch.zeros_like(x), torch.zeros(4, 8, device="cuda"), torch.zeros(4, 8, device="cuda"),
                torch.zeros_like(x), torch.zeros(64, device="cuda"), torch.zeros(64, device="cuda")]

    def go(o, stream=None):
        plan.run(x, None, None, o[0], o[1], o[2], stream=stream)
        plan.run_backward(x, None, None, o[1], o[2], dy, o[3], o[4], o[5], stream=stream)

    a, b, c, d = outs(), outs(), outs(), outs()
    go(a)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    go(b, stream=s)
    with torch.cuda.stream(s):
        go(c)
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        go(d)
    g.replay()
    g.replay()
    torch.cuda.synchronize()
    for other in (b, c, d):
        assert all(torch.equal(p, q) for p, q in zip(a, other))


def test_refusals(cl):
    x = draw((2, 4, 4, 16), torch.bfloat16, 71)
    plan = cl.GroupNormPlan(2, 4, 4, 16, 4, 1e-5, "bf16", "relu")
    y = torch.empty_like(x)
    st = torch.empty(2, 4, device="cuda")
    with pytest.raises(TypeError):
        plan.run(x.float(), None, None, y)
    with pytest.raises(ValueError):
        plan.run(x[:1], None, None, y)
    with pytest.raises(ValueError):
        plan.run(x.cpu(), None, None, y)
    with pytest.raises(ValueError):
        plan.run(x, None, None, None)
    with pytest.raises(ValueError):
        plan.run(x.permute(0, 2, 1, 3), None, None, y)
    with pytest.raises(ValueError):
        plan.run(x, torch.ones(8, device="cuda"), None, y)
    with pytest.raises(TypeError):
        plan.run(x, torch.ones(16, device="cuda", dtype=torch.bfloat16), None, y)
    with pytest.raises(cl.ConvError) as e:
        plan.run(x, None, None, x)
    assert e.value.code == -5
    buf = torch.zeros(2, 4, 4, 32, device="cuda", dtype=torch.bfloat16)
    with pytest.raises(cl.ConvError) as e:  # slices that share channels
        plan.run(buf[..., :16], None, None, buf[..., 8:24])
    assert e.value.code == -5
    plan.run(buf[..., :16], None, None, buf[..., 16:])  # and slices that share none
    with pytest.raises(ValueError):
        plan.run_backward(x, None, None, None, st, x, y)
    with pytest.raises(cl.ConvError) as e:
        plan.run_backward(x, None, None, st, st, y, y)
    assert e.value.code == -5
    lib = cl.load_library()
    args = [plan.handle, x.data_ptr(), 0, None, None, y.data_ptr(), 0, None, None, None, None]
    assert plan.workspace_bytes == 0 and lib.conv_run_groupnorm(*args) == 0
    assert lib.conv_run_groupnorm(*(args[:2] + [8] + args[3:])) == -9          # a pitch below the channels
    assert lib.conv_run_groupnorm(*(args[:1] + [x.data_ptr() + 1] + args[2:])) == -4
    big = cl.GroupNormPlan(1, 160, 160, 64, 4)
    xb, yb = torch.zeros(2, 1, 160, 160, 64, device="cuda", dtype=torch.bfloat16)
    assert big.workspace_bytes > 0
    big.run(xb, None, None, yb)
    args = [big.handle, xb.data_ptr(), 0, None, None, yb.data_ptr(), 0, None, None, None, None]
    assert lib.conv_run_groupnorm(*args) == -1                                 # no workspace
    assert lib.conv_run_groupnorm(*(args[:9] + [xb.data_ptr(), None])) == -5   # a workspace over x
    assert lib.conv_run(plan.handle, x.data_ptr(), x.data_ptr(), None, y.data_ptr(), None) == -9
    assert plan.algo == "groupnorm" and plan.launches >= 1 and plan.describe().startswith("groupnorm")
    plan.check_device_status()


def test_empty_batch(cl):
    plan = cl.GroupNormPlan(0, 4, 4, 16, 4)
    x = torch.empty(0, 4, 4, 16, device="cuda", dtype=torch.bfloat16)
    st, dg = torch.empty(0, 4, device="cuda"), torch.full((16,), 5.0, device="cuda")
    plan.run(x, None, None, x.clone(), st, st.clone())
    plan.run_backward(x, None, None, st, st.clone(), x.clone(), x.clone(), dg, None)
    assert not dg.any()
