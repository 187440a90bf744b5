"""The norms before and after a block against a plain 64-bit form of their
formulas, forward and gradient, and the gradient against differences of the
forward run.

Tolerances, with u = 2^-24, follow the formulas.  A sum over a row's channels
is off by at most 40 u of its terms' absolute sum (16 additions in a thread, 5
between lanes, up to 16 between warps), so a mean by em = 40 u mean|v|, and a
reciprocal deviation, half of whose relative error is that of its positive sum,
by 30 u of itself; a value normalised by r (em + 2 u |v|) + 32 u |v^|.  Errors
are carried on through each further formula, a few u for its own operations
(those of the second norm's input enter its mean, and through the root of their
mean square its deviation).  Sums over pixels are allowed 300 u of their terms'
absolute sum (at most 256 additions in a row, then joined) besides the terms'
own errors.  A bf16 result adds its rounding, 2^-8 of its size."""
import pytest
import torch

pytestmark = pytest.mark.gpu
U = 2.0 ** -24
DT = {"f32": torch.float32, "bf16": torch.bfloat16}
PARAMS = ("scale", "gate", "post_gamma", "post_beta", "pre_gamma", "pre_beta")


@pytest.fixture(scope="module")
def cl():
    from convolution_nhwc_implicit_gb300 import build
    build.build()
    import convolution_nhwc_implicit_gb300 as cl
    return cl


def mean(v):
    return v.mean(dim=-1, keepdim=True)


def norm64(v, err, kind, eps):
    """Normalised values, m, r, and what each normalised value and r (relative) may be off by."""
    m = mean(v) if kind == "layer" else torch.zeros_like(v[..., :1])
    if kind == "none":
        return v, m, torch.ones_like(m), err, torch.zeros_like(m)
    r = 1 / torch.sqrt(mean((v - m) ** 2) + eps)
    em = 40 * U * mean(v.abs()) + mean(err) if kind == "layer" else 0.0
    rel = 30 * U + r * torch.sqrt(mean((err + em) ** 2))
    hat = (v - m) * r
    return hat, m, r, r * (err + em + 2 * U * v.abs()) + hat.abs() * (rel + 2 * U), rel


def back64(d, ed, hat, ehat, r, rel, kind):
    """The gradient at a norm's input, and what it may be off by."""
    if kind == "none":
        return d, ed
    m1 = mean(d) if kind == "layer" else torch.zeros_like(r)
    m2 = mean(d * hat)
    e1 = mean(ed + 42 * U * d.abs()) if kind == "layer" else 0.0
    e2 = mean(ed * hat.abs() + d.abs() * ehat + 42 * U * (d * hat).abs())
    out = r * (d - m1 - hat * m2)
    size = d.abs() + m1.abs() + (hat * m2).abs()
    return out, r * (ed + e1 + hat.abs() * e2 + ehat * m2.abs() + (4 * U + rel) * size)


def reference(x, f, w, post, pre, eps, dy=None, dz=None, grad=False):
    n, h, wd, c = x.shape
    p = {k: None if w.get(k) is None else w[k].double() for k in PARAMS}
    one = torch.ones(c, dtype=torch.float64, device=x.device)

    def at(k, other):
        return other * one if p[k] is None else p[k]

    x = x.double()
    scale, g1, b1, g2, b2 = at("scale", 1), at("post_gamma", 1), at("post_beta", 0), at("pre_gamma", 1), at("pre_beta", 0)
    gate = torch.ones(n, 1, 1, c, dtype=torch.float64, device=x.device) if p["gate"] is None else p["gate"].view(n, 1, 1, c)
    out, tol = {}, {}
    if f is None:
        y, ey = x, torch.zeros_like(x)
    else:
        uh, m1, r1, euh, rel1 = norm64(f.double(), torch.zeros_like(x), post, eps)
        u = g1 * uh + b1
        k = scale * gate
        y = x + k * u
        ey = (k * g1).abs() * euh + 5 * U * (x.abs() + (k * b1).abs() + (k * g1 * uh).abs())
        out["y"], tol["y"] = y, ey
        out["m1"], out["r1"] = m1, r1
        tol["m1"], tol["r1"] = 42 * U * mean(f.double().abs()), rel1 * r1
    yh, m2, r2, eyh, rel2 = norm64(y, ey, pre, eps)
    if pre != "none":
        out["z"] = g2 * yh + b2
        tol["z"] = g2.abs() * eyh + 3 * U * ((g2 * yh).abs() + b2.abs())
        out["m2"], out["r2"] = m2, r2
        tol["m2"], tol["r2"] = 42 * U * mean(y.abs()) + mean(ey), rel2 * r2
    if not grad:
        return out, tol
    t = torch.zeros_like(x) if dy is None else dy.double()
    et = torch.zeros_like(x)
    if dz is not None:
        dz = dz.double()
        d, ed = back64(dz * g2, U * (dz * g2).abs(), yh, eyh, r2, rel2, pre)
        t, et = t + d, ed + 2 * U * (t.abs() + d.abs())
        for name, v, e in (("dpre_gamma", dz * yh, dz.abs() * eyh), ("dpre_beta", dz, torch.zeros_like(dz))):
            out[name], tol[name] = v.sum(dim=(0, 1, 2)), (e + 300 * U * v.abs()).sum(dim=(0, 1, 2))
    out["dx"], tol["dx"] = t, et
    if f is not None:
        v = k * g1 * t
        ev = (k * g1).abs() * et + 4 * U * v.abs()
        out["df"], tol["df"] = back64(v, ev, uh, euh, r1, rel1, post)
        A, B = (t * uh).sum(dim=(1, 2)), t.sum(dim=(1, 2))
        eA = (et * uh.abs() + t.abs() * euh + 300 * U * (t * uh).abs()).sum(dim=(1, 2))
        eB = (et + 300 * U * t.abs()).sum(dim=(1, 2))
        inner, einner = g1 * A + b1 * B, g1.abs() * eA + b1.abs() * eB
        size = (g1 * A).abs() + (b1 * B).abs()
        gate = gate.view(n, c)
        out["dgate"], tol["dgate"] = scale * inner, scale.abs() * (einner + 4 * U * size)
        out["dscale"], tol["dscale"] = (gate * inner).sum(0), (gate.abs() * (einner + 300 * U * size)).sum(0)
        out["dpost_gamma"], tol["dpost_gamma"] = (scale * gate * A).sum(0), (scale * gate).abs().mul(eA + 300 * U * A.abs()).sum(0)
        out["dpost_beta"], tol["dpost_beta"] = (scale * gate * B).sum(0), (scale * gate).abs().mul(eB + 300 * U * B.abs()).sum(0)
    return out, tol


def close(got, ref, tol, bf16, what):
    got = got.double().reshape(ref.shape)
    lim = tol * 1.05 + (ref.abs() * 2.0 ** -8 if bf16 else 2 * U * ref.abs()) + 1e-30
    bad = ~((got - ref).abs() <= lim)
    assert not bad.any(), (what, int(bad.sum()), float(((got - ref).abs() / lim)[bad].max()))


def draw(shape, dt, seed, wide=0, off=0, mean=0.0, std=1.0):
    n, h, w, c = shape
    g = torch.Generator("cuda").manual_seed(seed)
    v = torch.randn(n, h, w, c, generator=g, device="cuda") * std + mean
    if wide == 0:
        return v.to(dt)
    buf = torch.full((n, h, w, c + wide), 7.0, dtype=dt, device="cuda")
    buf[..., off:off + c] = v.to(dt)
    return buf[..., off:off + c]


def parameters(n, c, post, pre, gate, seed=100):
    g = torch.Generator("cuda").manual_seed(seed)

    def r(*shape):
        return torch.randn(*shape, generator=g, device="cuda")

    return dict(scale=0.5 + 0.2 * r(c), gate=torch.sigmoid(r(n, c)) if gate else None,
                post_gamma=None if post == "none" else 1 + 0.3 * r(c), post_beta=0.3 * r(c) if post == "layer" else None,
                pre_gamma=None if pre == "none" else 1 + 0.3 * r(c), pre_beta=0.3 * r(c) if pre == "layer" else None)


def grads_of(w):
    return {"d" + k: None if v is None else torch.full_like(v, 9.0) for k, v in w.items()}


CASES = [
    # n, h, w, c, post, pre, dtype, gate, wide, off
    (1, 1, 1, 1, "rms", "rms", "f32", False, 0, 0),
    (3, 2, 5, 2, "layer", "layer", "f32", True, 0, 0),
    (1, 1, 1, 512, "none", "layer", "bf16", False, 0, 0),
    (2, 7, 7, 512, "layer", "layer", "bf16", True, 0, 0),
    (2, 5, 3, 60, "rms", "layer", "bf16", True, 0, 0),         # 4-byte vectors
    (3, 9, 11, 33, "layer", "rms", "bf16", False, 0, 0),       # odd channels
    (3, 9, 11, 61, "layer", "layer", "f32", True, 0, 0),
    (2, 31, 33, 8, "layer", "rms", "bf16", True, 0, 0),        # a lane a row
    (2, 13, 17, 24, "rms", "rms", "bf16", False, 0, 0),        # lanes without channels
    (4, 20, 20, 256, "rms", "rms", "bf16", True, 0, 0),
    (1, 40, 41, 128, "layer", "layer", "f32", False, 0, 0),
    (2, 6, 7, 264, "layer", "layer", "bf16", False, 0, 0),     # two warps, one nearly empty
    (2, 6, 7, 520, "rms", "layer", "bf16", True, 0, 0),        # three warps
    (2, 10, 10, 1000, "layer", "rms", "f32", True, 0, 0),
    (1, 9, 9, 1023, "layer", "layer", "bf16", True, 0, 0),
    (1, 5, 5, 2056, "rms", "rms", "bf16", True, 0, 0),         # nine warps: one row a CTA
    (2, 3, 5, 4096, "layer", "layer", "bf16", True, 0, 0),
    (1, 3, 3, 4104, "rms", "layer", "bf16", False, 0, 0),      # sixteen channels a thread
    (2, 3, 4, 8192, "layer", "rms", "bf16", True, 0, 0),
    (1, 2, 5, 8191, "layer", "layer", "bf16", True, 0, 0),
    (1, 2, 5, 8192, "layer", "layer", "f32", True, 0, 0),
    (1, 2, 3, 6001, "rms", "rms", "f32", False, 0, 0),
    (3, 20, 20, 510, "layer", "rms", "bf16", True, 0, 0),      # sixteen channels a thread, a warp a row
    (1, 40, 30, 300, "rms", "rms", "f32", False, 1, 0),
    (2, 25, 25, 512, "layer", "none", "bf16", False, 0, 0),
    (4, 20, 20, 64, "layer", "rms", "bf16", True, 64, 64),     # a slice of a concatenated buffer
    (2, 10, 10, 48, "layer", "layer", "bf16", False, 13, 5),   # a slice at odd addresses
    (2, 10, 10, 48, "rms", "rms", "f32", True, 3, 1),
    (700, 1, 1, 96, "layer", "layer", "bf16", True, 0, 0),     # a pixel an image: whole images, more than CTAs
    (350, 3, 3, 40, "rms", "layer", "f32", True, 0, 0),
    (3, 50, 50, 64, "none", "rms", "bf16", True, 0, 0),        # runs of an image
    (4, 8, 8, 96, "layer", "layer", "bf16", True, 0, 0),       # a cluster: four images of few rows
    (1, 10, 50, 256, "rms", "rms", "bf16", False, 0, 0),       # ... four sets of rows a CTA, the last one short
    (1, 1, 9, 3001, "layer", "rms", "f32", True, 0, 0),        # ... a row at a time
    (5, 3, 2, 70, "rms", "layer", "bf16", True, 0, 0),         # more images than that
    (1, 80, 80, 256, "none", "none", "bf16", True, 0, 0),      # a gated residual add
    (2, 30, 30, 32, "layer", "none", "f32", True, 0, 0),
    (2, 160, 160, 64, "rms", "layer", "bf16", False, 0, 0),
]


def buffers(shape, dt, wide, off):
    return [draw(shape, dt, 50 + i, wide, off) for i in range(4)]  # y, z, dx, df


@pytest.mark.parametrize("n,h,w,c,post,pre,dtype,gate,wide,off", CASES)
def test_forward_and_gradient(cl, n, h, w, c, post, pre, dtype, gate, wide, off):
    shape, dt, bf = (n, h, w, c), DT[dtype], dtype == "bf16"
    x, f = draw(shape, dt, 1, wide, off, 0.4, 0.8), draw(shape, dt, 2, wide, off, -0.3, 2.0)
    dy, dz = draw(shape, dt, 3, wide, off, 0.1, 0.5), draw(shape, dt, 4, wide, off, 0.1, 0.5)
    has_z = pre != "none"
    p = parameters(n, c, post, pre, gate)
    ref, tol = reference(x, f, p, post, pre, 1e-5, dy, dz if has_z else None, True)
    y, z, dx, df = buffers(shape, dt, wide, off)
    stats = torch.full((n, h, w, 4), 9.0, device="cuda")
    d = grads_of(p)
    plan = cl.BlockNormPlan(n, h, w, c, post, pre, 1e-5, dtype)
    plan.run(x, f, y, z if has_z else None, stats, **p)
    back = {k: v for k, v in p.items() if k != "pre_beta"}
    plan.run_backward(x, f, stats, dy, dz if has_z else None, dx, df, **back, **d)
    torch.cuda.synchronize()
    close(y, ref["y"], tol["y"], bf, "y")
    for k, name in enumerate(("m1", "r1", "m2", "r2")):
        if name in ref:
            close(stats[..., k:k + 1], ref[name], tol[name], False, name)
    if has_z:
        close(z, ref["z"], tol["z"], bf, "z")
    close(dx, ref["dx"], tol["dx"], bf, "dx")
    close(df, ref["df"], tol["df"], bf, "df")
    for k, v in d.items():
        if v is not None:
            close(v, ref[k], tol[k], False, k)
    for t in (y, z, dx, df):  # nothing outside the slice was written
        if wide:
            whole = t._base
            assert bool((whole[..., :off] == 7).all()) and bool((whole[..., off + c:] == 7).all())


@pytest.mark.parametrize("dtype,c", [("bf16", 96), ("f32", 50)])
@pytest.mark.parametrize("pre", ["layer", "rms"])
def test_without_a_block(cl, dtype, c, pre):
    """f None: the norm before the first block, and its gradient added to the stream's."""
    shape, dt = (2, 9, 8, c), DT[dtype]
    x, dy, dz = draw(shape, dt, 11, mean=0.3), draw(shape, dt, 12), draw(shape, dt, 13)
    p = parameters(2, c, "none", pre, False)
    p["scale"] = None
    plan = cl.BlockNormPlan(*shape, "none", pre, 1e-5, dtype)
    z, dx, stats = torch.empty_like(x), torch.empty_like(x), torch.empty(2, 9, 8, 4, device="cuda")
    plan.run(x, None, None, z, stats, pre_gamma=p["pre_gamma"], pre_beta=p["pre_beta"])
    dg, db = torch.empty(c, device="cuda"), torch.empty(c, device="cuda")
    for stream_grad in (dy, None):
        ref, tol = reference(x, None, p, "none", pre, 1e-5, stream_grad, dz, True)
        plan.run_backward(x, None, stats, stream_grad, dz, dx, None, pre_gamma=p["pre_gamma"], dpre_gamma=dg, dpre_beta=db)
        close(z, ref["z"], tol["z"], dtype == "bf16", "z")
        close(dx, ref["dx"], tol["dx"], dtype == "bf16", "dx")
        close(dg, ref["dpre_gamma"], tol["dpre_gamma"], False, "dg")
        close(db, ref["dpre_beta"], tol["dpre_beta"], False, "db")


@pytest.mark.parametrize("post,pre", [("layer", "layer"), ("rms", "rms"), ("none", "layer")])
def test_without_parameters(cl, post, pre):
    shape = (2, 6, 5, 48)
    x, f, dy, dz = (draw(shape, torch.bfloat16, 20 + i) for i in range(4))
    plan = cl.BlockNormPlan(*shape, post, pre)
    ref, tol = reference(x, f, {}, post, pre, 1e-5, None, dz, True)
    y, z, dx, df = buffers(shape, torch.bfloat16, 0, 0)
    stats = torch.empty(2, 6, 5, 4, device="cuda")
    plan.run(x, f, None, z, stats)         # without the stream
    plan.run(x, f, y, z)                   # without statistics
    ds = torch.empty(48, device="cuda")
    plan.run_backward(x, f, stats, None, dz, dx, df, dscale=ds)
    for name, t in (("y", y), ("z", z), ("dx", dx), ("df", df)):
        close(t, ref[name], tol[name], True, name)
    close(ds, ref["dscale"], tol["dscale"], False, "dscale")


# A row of two CTAs: units of one and several rows, images one after another in a
# pair of CTAs, odd channels and addresses, and what a call may leave out.
PAIRS = [
    # n, h, w, c, post, pre, dtype, gate, wide, off, f, dy, dz
    (1, 1, 200, 8192, "layer", "layer", "bf16", False, 0, 0, True, True, True),
    (1, 1, 200, 4097, "rms", "layer", "bf16", False, 0, 0, True, True, True),
    (160, 1, 1, 5000, "layer", "rms", "bf16", True, 0, 0, True, True, True),
    (90, 3, 1, 4104, "layer", "layer", "f32", True, 0, 0, True, True, True),
    (3, 7, 11, 4352, "layer", "layer", "f32", True, 0, 0, True, True, True),
    (1, 1, 160, 6002, "layer", "rms", "bf16", False, 0, 0, True, True, True),
    (1, 1, 160, 4099, "layer", "layer", "bf16", True, 13, 5, True, True, True),
    (1, 1, 160, 7001, "rms", "rms", "f32", True, 3, 1, True, True, True),
    (1, 1, 160, 5120, "layer", "none", "bf16", False, 0, 0, True, True, False),
    (1, 1, 160, 5120, "none", "layer", "bf16", True, 0, 0, True, True, True),
    (1, 1, 160, 5121, "none", "none", "bf16", True, 0, 0, True, True, False),
    (1, 1, 160, 5120, "layer", "layer", "bf16", False, 0, 0, True, False, True),
    (1, 1, 160, 5121, "rms", "rms", "f32", True, 0, 0, True, False, True),
    (1, 1, 160, 5120, "none", "layer", "bf16", False, 0, 0, False, True, True),
    (1, 1, 160, 5122, "none", "rms", "bf16", False, 0, 0, False, False, True),
]


@pytest.mark.parametrize("n,h,w,c,post,pre,dtype,gate,wide,off,has_f,has_dy,has_dz", PAIRS)
def test_gradient_of_rows_of_two_ctas(cl, n, h, w, c, post, pre, dtype, gate, wide, off, has_f, has_dy, has_dz):
    shape, dt, bf = (n, h, w, c), DT[dtype], dtype == "bf16"
    x, f = draw(shape, dt, 31, wide, off, 0.4, 0.8), draw(shape, dt, 32, wide, off, -0.3, 2.0) if has_f else None
    dy = draw(shape, dt, 33, wide, off, 0.1, 0.5) if has_dy else None
    dz = draw(shape, dt, 34, wide, off, 0.1, 0.5) if has_dz else None
    p = parameters(n, c, post, pre, gate)
    if not has_f:
        p.update(scale=None, gate=None, post_gamma=None, post_beta=None)
    ref, tol = reference(x, f, p, post, pre, 1e-5, dy, dz, True)
    y, z, dx, df = buffers(shape, dt, wide, off)
    stats = torch.full((n, h, w, 4), float("nan"), device="cuda")   # (what a norm leaves out stays so)
    plan = cl.BlockNormPlan(n, h, w, c, post, pre, 1e-5, dtype)
    plan.run(x, f, y if has_f else None, z if has_dz else None, stats, **p)
    d = grads_of(p)
    args = (x, f, stats, dy, dz, dx, df if has_f else None)
    plan.run_backward(*args, **{k: v for k, v in p.items() if k != "pre_beta"}, **d)
    first = [t.clone() for t in (dx, df, *d.values()) if t is not None]
    plan.run_backward(*args, **{k: v for k, v in p.items() if k != "pre_beta"}, **d)
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(first, (t for t in (dx, df, *d.values()) if t is not None)))
    close(dx, ref["dx"], tol["dx"], bf, "dx")
    if has_f:
        close(df, ref["df"], tol["df"], bf, "df")
    for k, v in d.items():
        if v is not None:
            close(v, ref[k], tol[k], False, k)
    for t in (dx, df):
        if wide:
            whole = t._base
            assert bool((whole[..., :off] == 7).all()) and bool((whole[..., off + c:] == 7).all())


# One row at a time and images one after another in a CTA: a thread adds its own
# sums, writes the gate's gradient, and either may lie on no 16 bytes.
OWN = [
    # n, h, w, c, post, pre, dtype, parameters' address off by elements
    (1300, 1, 1, 264, "layer", "layer", "bf16", 0),
    (1300, 1, 1, 264, "layer", "layer", "bf16", 1),
    (5000, 1, 1, 256, "rms", "layer", "bf16", 3),      # a warp a row
    (200, 2, 1, 2056, "layer", "rms", "f32", 2),
    (200, 1, 1, 2058, "layer", "layer", "bf16", 1),    # 4-byte vectors
    (200, 1, 1, 2057, "rms", "rms", "f32", 0),
    (160, 1, 1, 4104, "layer", "layer", "bf16", 1),    # two CTAs a row
    (160, 1, 1, 8192, "layer", "rms", "f32", 3),
]


@pytest.mark.parametrize("n,h,w,c,post,pre,dtype,shift", OWN)
def test_gradient_of_many_small_gated_images(cl, n, h, w, c, post, pre, dtype, shift):
    shape, dt, bf = (n, h, w, c), DT[dtype], dtype == "bf16"
    x, f = draw(shape, dt, 61, mean=0.4, std=0.8), draw(shape, dt, 62, mean=-0.3, std=2.0)
    dy, dz = draw(shape, dt, 63, mean=0.1, std=0.5), draw(shape, dt, 64, mean=0.1, std=0.5)

    def moved(t):
        if t is None:
            return None
        buf = torch.full((t.numel() + 8,), 9.0, device="cuda")
        buf[shift:shift + t.numel()] = t.flatten()
        return buf[shift:shift + t.numel()].view(t.shape)

    p = {k: moved(v) for k, v in parameters(n, c, post, pre, True).items()}
    d = {k: moved(v) for k, v in grads_of(p).items()}
    ref, tol = reference(x, f, p, post, pre, 1e-5, dy, dz, True)
    y, z, dx, df = buffers(shape, dt, 0, 0)
    stats = torch.empty(n, h, w, 4, device="cuda")
    plan = cl.BlockNormPlan(n, h, w, c, post, pre, 1e-5, dtype)
    plan.run(x, f, y, z, stats, **p)
    plan.run_backward(x, f, stats, dy, dz, dx, df, **{k: v for k, v in p.items() if k != "pre_beta"}, **d)
    torch.cuda.synchronize()
    close(y, ref["y"], tol["y"], bf, "y")
    close(z, ref["z"], tol["z"], bf, "z")
    close(dx, ref["dx"], tol["dx"], bf, "dx")
    close(df, ref["df"], tol["df"], bf, "df")
    for k, v in d.items():
        if v is not None:
            close(v, ref[k], tol[k], False, k)
            assert bool((v._base[:shift] == 9).all()) and bool((v._base[shift + v.numel():] == 9).all())


def test_rows_of_two_ctas_on_two_streams_and_in_graphs(cl):
    """Two gradients at once, then captured on two streams and replayed together: the bits of one alone."""
    shape = (1, 1, 400, 5120)
    plan = cl.BlockNormPlan(*shape, "layer", "rms")
    sides = []
    for i in range(2):
        x, f, dy, dz = (draw(shape, torch.bfloat16, 70 + 10 * i + j) for j in range(4))
        y, z, dx, df = (torch.empty_like(x) for _ in range(4))
        stats = torch.empty(1, 1, 400, 4, device="cuda")
        p = parameters(1, 5120, "layer", "rms", True, seed=80 + i)
        d = grads_of(p)
        plan.run(x, f, y, z, stats, **p)
        kw = {**{k: v for k, v in p.items() if k != "pre_beta"}, **d}
        run = (lambda a, k: lambda: plan.run_backward(*a, **k))((x, f, stats, dy, dz, dx, df), kw)
        sides.append((run, [dx, df] + [v for v in d.values() if v is not None]))
    alone = []
    for run, outs in sides:
        run()
        torch.cuda.synchronize()
        alone.append([t.clone() for t in outs])

    def check():
        torch.cuda.synchronize()
        for (_, outs), ref in zip(sides, alone):
            assert all(torch.equal(a, b) for a, b in zip(outs, ref))
            for t in outs:
                t.fill_(3.0)
        torch.cuda.synchronize()

    check()
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    for (run, _), st in zip(sides, streams):
        with torch.cuda.stream(st):
            for _ in range(3):
                run()
    check()
    graphs = []
    for run, _ in sides:
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            run()
        graphs.append(g)
    for _ in range(2):
        for g, st in zip(graphs, streams):
            with torch.cuda.stream(st):
                g.replay()
        check()


@pytest.mark.parametrize("c", [520, 8192])
@pytest.mark.parametrize("pre", ["layer", "rms"])
def test_gradient_that_cancels(cl, c, pre):
    """dz along the normalised stream, and dy against what is left: dY is a rounding of
    its terms.  (The bounds count each term's roundings, not dY's alone: a sum of
    dY's terms apart, 22 roundings deep, is inside dY's own 34 a term.)"""
    shape = (1, 1, 100, c)
    x, f = draw(shape, torch.float32, 41, mean=0.4), draw(shape, torch.float32, 42, mean=-0.3, std=2.0)
    p = parameters(1, c, "layer", pre, False)
    plan = cl.BlockNormPlan(*shape, "layer", pre, 1e-5, "f32")
    y, z, dx, df = (torch.empty_like(x) for _ in range(4))
    stats = torch.empty(1, 1, 100, 4, device="cuda")
    plan.run(x, f, y, z, stats, **p)
    y64 = y.double()
    m = mean(y64) if pre == "layer" else 0.0
    hat = (y64 - m) / torch.sqrt(mean((y64 - m) ** 2) + 1e-5)
    noise = draw(shape, torch.float32, 43)
    for dz, dy in (((hat / p["pre_gamma"]).float(), None), (noise, None)):
        if dz is noise:
            dy = (-reference(x, f, p, "layer", pre, 1e-5, None, dz, True)[0]["dx"]).float()
        ref, tol = reference(x, f, p, "layer", pre, 1e-5, dy, dz, True)
        plan.run_backward(x, f, stats, dy, dz, dx, df, **{k: v for k, v in p.items() if k != "pre_beta"})
        close(dx, ref["dx"], tol["dx"], False, "dx")
        close(df, ref["df"], tol["df"], False, "df")


def test_in_place(cl):
    """y over x, z over f; dx over dy, df over dz: the bits of separate buffers."""
    for shape, dtype in (((2, 9, 9, 256), "bf16"), ((2, 5, 5, 8192), "bf16"), ((3, 7, 7, 33), "f32"), ((2, 21, 20, 255), "bf16"),
                         ((2, 30, 30, 66), "bf16")):
        n, h, w, c = shape
        x, f, dy, dz = (draw(shape, DT[dtype], 30 + i) for i in range(4))
        p = parameters(n, c, "layer", "rms", True)
        plan = cl.BlockNormPlan(*shape, "layer", "rms", dtype=dtype)
        y, z, dx, df = buffers(shape, DT[dtype], 0, 0)
        stats, st2 = (torch.empty(n, h, w, 4, device="cuda") for _ in range(2))
        plan.run(x, f, y, z, stats, **p)
        xs, fs = x.clone(), f.clone()
        plan.run(xs, fs, xs, fs, st2, **p)
        assert torch.equal(xs, y) and torch.equal(fs, z) and torch.equal(st2, stats)
        back = {k: v for k, v in p.items() if k != "pre_beta"}
        d, d2 = grads_of(p), grads_of(p)
        plan.run_backward(x, f, stats, dy, dz, dx, df, **back, **d)
        dys, dzs = dy.clone(), dz.clone()
        plan.run_backward(x, f, stats, dys, dzs, dys, dzs, **back, **d2)
        assert torch.equal(dys, dx) and torch.equal(dzs, df)
        xs, fs = x.clone(), f.clone()
        plan.run_backward(xs, fs, stats, dy, dz, fs, xs, **back)
        assert torch.equal(fs, dx) and torch.equal(xs, df)
        assert all(torch.equal(d[k], d2[k]) for k in d if d[k] is not None)


@pytest.mark.parametrize("post,pre,gate", [("layer", "layer", True), ("rms", "rms", False), ("none", "layer", True)])
def test_gradient_against_differences(cl, post, pre, gate):
    """sum(grad v) against (L(+e v) - L(-e v)) / 2 e, L = sum(y dy + z dz).  The
    difference is off by e^2/6 of the third derivative (of order 10 |grad| |v|^3
    r^3 here) and by the forward run's rounding over e: 3e-3 of the sum of
    |grad v| covers both at e = 2^-8."""
    shape, (n, c) = (2, 5, 4, 24), (2, 24)
    x, f, dy, dz = (draw(shape, torch.float32, 40 + i, std=1.0 + 0.5 * i % 2) for i in range(4))
    p = parameters(n, c, post, pre, gate)
    plan = cl.BlockNormPlan(*shape, post, pre, 1e-5, "f32")
    stats = torch.empty(2, 5, 4, 4, device="cuda")

    def loss(x, f, **p):
        y, z = torch.empty_like(x), torch.empty_like(x)
        plan.run(x, f, y, z, stats, **p)
        return float((y.double() * dy.double()).sum() + (z.double() * dz.double()).sum())

    e = 2.0 ** -8
    args = dict(x=x, f=f, **p)
    loss(**args)
    dx, df, d = torch.empty_like(x), torch.empty_like(x), grads_of(p)
    plan.run_backward(x, f, stats, dy, dz, dx, df, **{k: v for k, v in p.items() if k != "pre_beta"}, **d)
    for name, grad in [("x", dx), ("f", df)] + [(k[1:], v) for k, v in d.items() if v is not None]:
        v = torch.randn(grad.shape, generator=torch.Generator("cuda").manual_seed(99), device="cuda")
        diff = (loss(**{**args, name: args[name] + e * v}) - loss(**{**args, name: args[name] - e * v})) / (2 * e)
        terms = grad.double() * v.double()
        assert abs(float(terms.sum()) - diff) <= 3e-3 * float(terms.abs().sum()), name


def test_large_mean_and_constant_rows(cl):
    """A mean a thousand times the spread keeps its digits; equal values give beta."""
    shape = (1, 4, 4, 200)
    x = draw(shape, torch.float32, 60, mean=1000.0)
    x[0, 1, 2] = 3.25
    beta = torch.linspace(-1, 1, 200, device="cuda")
    plan = cl.BlockNormPlan(*shape, "none", "layer", 1e-5, "f32")
    z = torch.empty_like(x)
    plan.run(x, None, None, z, pre_beta=beta)
    ref, tol = reference(x, None, {"pre_beta": beta}, "none", "layer", 1e-5)
    # (the constant row: 200 * 3.25 is exact, its mean within a rounding of 3.25)
    assert bool(((z[0, 1, 2] - beta).abs() <= 4 * U * 3.25 * 1e-5 ** -0.5).all())
    keep = torch.ones(16, dtype=torch.bool, device="cuda")
    keep[6] = False
    close(z.view(16, 200)[keep], ref["z"].view(16, 200)[keep], tol["z"].view(16, 200)[keep], False, "z")


def test_non_finite_rows_stay_their_own(cl):
    shape = (2, 6, 6, 40)
    x, f, dy, dz = (draw(shape, torch.bfloat16, 70 + i) for i in range(4))
    clean_x = x.clone()
    x[0, 2, 3, 5] = float("nan")
    x[1, 1, 1, 0] = float("inf")
    plan = cl.BlockNormPlan(*shape, "rms", "layer")
    stats, st2 = (torch.empty(2, 6, 6, 4, device="cuda") for _ in range(2))
    y, z, dx, df = buffers(shape, torch.bfloat16, 0, 0)
    y2, z2, dx2, df2 = buffers(shape, torch.bfloat16, 0, 0)
    plan.run(x, f, y, z, stats)
    plan.run(clean_x, f, y2, z2, st2)
    plan.run_backward(x, f, stats, dy, dz, dx, df)
    plan.run_backward(clean_x, f, st2, dy, dz, dx2, df2)
    rows = torch.ones(2, 6, 6, dtype=torch.bool, device="cuda")
    rows[0, 2, 3] = rows[1, 1, 1] = False
    assert torch.isnan(z[0, 2, 3]).all() and torch.isnan(z[1, 1, 1]).any() and torch.isnan(dx[0, 2, 3]).all()
    for a, b in ((y, y2), (z, z2), (dx, dx2), (df, df2)):
        assert torch.equal(a[rows], b[rows])


def test_offsets_past_31_bits(cl):
    """Pixels whose element offsets pass 2^31 (a small slice of a very wide buffer)."""
    c, pitch, w = 16, (1 << 25) + 8, 70
    buf = torch.empty(1, 1, w, pitch, dtype=torch.bfloat16, device="cuda")
    maps = [buf[..., 1024 * i + 8:1024 * i + 8 + c] for i in range(8)]
    x, f, dy, dz, y, z, dx, df = maps
    for i, m in enumerate(maps[:4]):
        m.copy_(draw((1, 1, w, c), torch.bfloat16, 80 + i))
    plan = cl.BlockNormPlan(1, 1, w, c, "layer", "layer")
    stats = torch.empty(1, 1, w, 4, device="cuda")
    ref, tol = reference(x, f, {}, "layer", "layer", 1e-5, dy, dz, True)
    plan.run(x, f, y, z, stats)
    plan.run_backward(x, f, stats, dy, dz, dx, df)
    for name, t in (("y", y), ("z", z), ("dx", dx), ("df", df)):
        close(t, ref[name], tol[name], True, name)


@pytest.mark.parametrize("gate", [False, True])
def test_streams_graph_and_repeat(cl, gate):
    """The same bits on another stream, in a replayed graph and run after run."""
    shape = (4, 20, 20, 64)
    x, f, dy, dz = (draw(shape, torch.bfloat16, 90 + i) for i in range(4))
    p = parameters(4, 64, "layer", "rms", gate)
    plan = cl.BlockNormPlan(*shape, "layer", "rms")
    back = {k: v for k, v in p.items() if k != "pre_beta"}

    def outs():
        return buffers(shape, torch.bfloat16, 0, 0) + [torch.zeros(4, 20, 20, 4, device="cuda")], grads_of(p)

    def go(o, stream=None):
        (y, z, dx, df, stats), d = o
        plan.run(x, f, y, z, stats, stream=stream, **p)
        plan.run_backward(x, f, stats, dy, dz, dx, df, stream=stream, **back, **d)

    a, b, c, d, e = (outs() for _ in range(5))
    go(a)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    go(b, stream=s)
    with torch.cuda.stream(s):
        go(c)
    torch.cuda.synchronize()
    graphs = [torch.cuda.CUDAGraph(), torch.cuda.CUDAGraph()]
    for g, o in zip(graphs, (d, e)):  # two graphs whose scratch comes from their own pools
        with torch.cuda.graph(g):
            go(o)
    with torch.cuda.stream(s):
        graphs[0].replay()
    graphs[1].replay()
    graphs[1].replay()
    torch.cuda.synchronize()
    for other in (b, c, d, e):
        assert all(torch.equal(p, q) for p, q in zip(a[0], other[0]))
        assert all(torch.equal(a[1][k], other[1][k]) for k in a[1] if a[1][k] is not None)


def test_refusals(cl):
    shape = (2, 4, 4, 16)
    x, f, dz = (draw(shape, torch.bfloat16, 110 + i) for i in range(3))
    y, z, dx, df = buffers(shape, torch.bfloat16, 0, 0)
    plan = cl.BlockNormPlan(*shape, "rms", "layer")
    stats = torch.empty(2, 4, 4, 4, device="cuda")
    v, gate = torch.ones(16, device="cuda"), torch.ones(2, 16, device="cuda")
    plan.run(x, f, y, z, stats)
    for bad in (x.float(), x[:1], x.cpu(), x.permute(0, 2, 1, 3), None):
        with pytest.raises((TypeError, ValueError)):
            plan.run(bad, f, y, z)
    for kw in (dict(scale=gate), dict(gate=v), dict(post_gamma=v.bfloat16()), dict(stats=stats[:1])):
        with pytest.raises((TypeError, ValueError)):
            plan.run(x, f, y, z, **kw)

    def code(call, *a, **kw):
        with pytest.raises(cl.ConvError) as e:
            call(*a, **kw)
        return e.value.code

    assert code(plan.run, x, f, y, None) == -1                     # no z
    assert code(plan.run, x, None, None, z) == -9                  # no f under a norm of it
    assert code(plan.run, x, f, y, y) == -5
    buf = torch.zeros(2, 4, 4, 32, device="cuda", dtype=torch.bfloat16)
    assert code(plan.run, buf[..., :16], f, buf[..., 8:24], z) == -5
    assert code(plan.run, buf[..., :16], f, y, buf[..., 8:24]) == -5
    plan.run(buf[..., :16], f, buf[..., :16], buf[..., 16:])        # slices that share none, and the stream in place
    none = cl.BlockNormPlan(*shape, "none", "none")
    assert code(none.run, x, f, y, z) == -9 and code(none.run, x, f, None, None) == -1
    assert code(none.run, x, f, y, None, post_gamma=v) == -9 and code(none.run, x, f, y, None, pre_beta=v) == -9
    assert code(none.run, x, None, y, None) == -9
    assert code(plan.run_backward, x, f, stats, None, None, dx, df) == -1
    assert code(plan.run_backward, x, f, stats, None, dz, dx, None) == -1
    assert code(plan.run_backward, x, f, stats, None, dz, dx, dx) == -5
    assert code(plan.run_backward, x, f, stats, None, dz, dx, df, dgate=gate) == -9
    assert code(plan.run_backward, x, f, stats, None, dz, dx, df, dscale=v, scale=v) == -5
    assert code(plan.run_backward, x, f, stats, None, dz, dx, df, dscale=v, dpre_beta=v) == -5
    assert code(none.run_backward, x, f, stats, y, None, dx, df, dpost_beta=v) == -9
    with pytest.raises(ValueError):
        plan.run_backward(x, f, None, None, dz, dx, df)
    lib = cl.load_library()
    args = [plan.handle, x.data_ptr(), 0, f.data_ptr(), 0, None, y.data_ptr(), 0, z.data_ptr(), 0, None, None]
    assert lib.conv_run_blocknorm(*args) == 0
    assert lib.conv_run_blocknorm(*(args[:2] + [8] + args[3:])) == -9
    assert lib.conv_run_blocknorm(*(args[:1] + [x.data_ptr() + 1] + args[2:])) == -4
    assert lib.conv_run_blocknorm(*(args[:10] + [stats.data_ptr() + 4, None])) == -4
    assert lib.conv_run_blocknorm(*(args[:10] + [y.data_ptr(), None])) == -5
    back = [plan.handle, x.data_ptr(), 0, f.data_ptr(), 0, None, stats.data_ptr(), None, 0, dz.data_ptr(), 0, dx.data_ptr(), 0,
            df.data_ptr(), 0, None]
    assert plan.workspace_bytes_backward == 0 and lib.conv_run_blocknorm_bwd(*back, None, None) == 0
    big = cl.BlockNormPlan(1, 160, 160, 64, "rms", "layer")
    m = torch.zeros(5, 1, 160, 160, 64, device="cuda", dtype=torch.bfloat16)
    st = torch.zeros(1, 160, 160, 4, device="cuda")
    big.run(m[0], m[1], None, m[2], st)
    big.run_backward(m[0], m[1], st, None, m[2], m[3], m[4], dscale=torch.empty(64, device="cuda"))
    back = [big.handle, m[0].data_ptr(), 0, m[1].data_ptr(), 0, None, st.data_ptr(), None, 0, m[2].data_ptr(), 0, m[3].data_ptr(), 0,
            m[4].data_ptr(), 0, None]
    assert big.workspace_bytes_backward > 0 and lib.conv_run_blocknorm_bwd(*back, None, None) == -1  # no workspace
    assert lib.conv_run_blocknorm_bwd(*back, m[0].data_ptr(), None) == -5                            # one over x
    assert lib.conv_run(plan.handle, x.data_ptr(), x.data_ptr(), None, y.data_ptr(), None) == -9
    assert plan.algo == "blocknorm" and plan.launches == 1 and plan.describe().startswith("blocknorm")
    plan.check_device_status()


@pytest.mark.parametrize("shape", [(200, 1, 2, 2056), (400, 1, 1, 1024), (170, 2, 2, 40), (160, 1, 3, 4200)])
def test_gradients_not_asked_for_change_nothing(cl, shape):
    """Images that a CTA takes one after the other: the bits of every gradient do
    not depend on which others are asked for."""
    n, h, w, c = shape
    x, f, dy, dz = (draw(shape, torch.bfloat16, 120 + i) for i in range(4))
    p = parameters(n, c, "layer", "layer", True)
    back = {k: v for k, v in p.items() if k != "pre_beta"}
    plan = cl.BlockNormPlan(*shape, "layer", "layer")
    _, _, dx, df = buffers(shape, torch.bfloat16, 0, 0)
    stats = torch.empty(n, h, w, 4, device="cuda")
    plan.run(x, f, torch.empty_like(x), torch.empty_like(x), stats, **p)
    every = grads_of(p)
    plan.run_backward(x, f, stats, dy, dz, dx, df, **back, **every)
    ref, tol = reference(x, f, p, "layer", "layer", 1e-5, dy, dz, True)
    for k, v in every.items():
        close(v, ref[k], tol[k], False, k)
    for _ in range(3):
        for k in every:
            one, (dx2, df2) = torch.full_like(every[k], 9.0), (torch.empty_like(x), torch.empty_like(x))
            plan.run_backward(x, f, stats, dy, dz, dx2, df2, **back, **{k: one})
            assert torch.equal(one, every[k]) and torch.equal(dx, dx2) and torch.equal(df, df2), k


def test_empty_batch(cl):
    plan = cl.BlockNormPlan(0, 4, 4, 16)
    x = torch.empty(0, 4, 4, 16, device="cuda", dtype=torch.bfloat16)
    st, d = torch.empty(0, 4, 4, 4, device="cuda"), torch.full((16,), 5.0, device="cuda")
    gate = torch.empty(0, 16, device="cuda")
    plan.run(x, x.clone(), x.clone(), x.clone(), st)
    plan.run_backward(x, x.clone(), st, x.clone(), x.clone(), x.clone(), x.clone(), gate=gate, dgate=gate.clone(), dscale=d)
    assert not d.any()
