"""Loss of a class head over many classes and its gradient, against the same
formulas in 64 bits, and the gradient against differences of the loss.

Tolerances.  A score is a sum of D exact products in fp32: off by at most
el = (D / 16 + 8) 2^-23 sum |x w| (the tensor core joins 16 products a step).
lse is off by the scores' largest error and 4e-6 of exponentials and sums, a
row's loss by twice that.  g is off by g's own change (its probability times
the relative error e^(2 el) - 1 and 4e-6) and its rounding to bf16 (eight
significant bits: half the spacing of such numbers at g, 2^-8 of its power of
two); a gradient by the sum of those errors times |w| (or |x|), by its fp32 sum
(2^-20 of the terms' sizes) and by its rounding to bf16 (2^-8 of it)."""
import pytest
import torch

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def cl():
    from convolution_nhwc_implicit_gb300 import build
    build.build()
    import convolution_nhwc_implicit_gb300 as cl
    return cl


def inputs(n, d, v, seed=0, scale=1.0):
    g = torch.Generator("cpu").manual_seed(seed)
    x = torch.randn(n, d, generator=g).to(torch.bfloat16)
    w = (scale * torch.randn(v, d, generator=g) / d ** 0.5).to(torch.bfloat16)
    t = torch.randint(0, v, (n,), generator=g, dtype=torch.int64).to(torch.int32)
    return x.cuda(), w.cuda(), t.cuda()


def reference(x, w, t, dloss=1.0):
    """64 bits; errors as in the head of this file."""
    xd, wd = x.double(), w.double()
    z = xd @ wd.t()
    size = xd.abs() @ wd.abs().t()
    el = ((x.shape[1] / 16 + 8) * 2.0 ** -23 * size).amax(dim=1)
    lse = torch.logsumexp(z, dim=1)
    on = (t >= 0) & (t < w.shape[0])
    at = torch.where(on, t, torch.zeros_like(t)).long()[:, None]
    row = torch.where(on, lse - z.gather(1, at)[:, 0], torch.zeros_like(lse))
    count = max(1, int(on.sum()))
    p = torch.exp(z - lse[:, None])
    g = p.clone()
    g.scatter_add_(1, at, -torch.ones_like(g[:, :1]))
    eg = p * (4 * el[:, None] + 4e-6)
    eg = eg + torch.exp2(torch.floor(torch.log2((g.abs() + eg).clamp(min=1e-300)))) * 2.0 ** -8
    s = dloss / count
    m = on.double()[:, None] * s
    g, eg = g * m, eg * m.abs()
    out = dict(lse=lse, lse_tol=el + 4e-6 * (1 + lse.abs()), row=row, row_tol=2 * el + 8e-6 * (1 + lse.abs()), loss=row.sum() / count)
    out["loss_tol"] = (out["row_tol"] * on).sum() / count + 1e-30
    out["dx"], out["dw"] = g @ wd, g.t() @ xd
    out["dx_tol"] = (eg + 2.0 ** -20 * g.abs()) @ wd.abs() + out["dx"].abs() * 2.0 ** -8
    out["dw_tol"] = (eg + 2.0 ** -20 * g.abs()).t() @ xd.abs() + out["dw"].abs() * 2.0 ** -8
    return out


def close(got, ref, tol, what):
    lim = tol + 1e-36
    err = (got.double() - ref).abs()
    bad = ~(err <= lim)
    assert not bad.any(), (what, int(bad.sum()), bad.numel(), float((err / lim)[bad].max()))


def run(cl, x, w, t, piece=0, dloss=None):
    n, d = x.shape
    v = w.shape[0]
    plan = cl.ClassLossPlan(n, d, v, piece)
    loss, lse, row = (torch.full(s, 7.0, device="cuda") for s in ((), (n,), (n,)))
    plan.run(x, w, t, loss, lse, row)
    dx, dw = torch.full_like(x, 7.0), torch.full_like(w, 7.0)
    plan.run_backward(x, w, t, lse, dx, dw, dloss)
    plan.check_device_status()
    return plan, dict(loss=loss, lse=lse, row=row, dx=dx, dw=dw)


CASES = [
    # rows, features, classes, piece
    (1, 8, 1, 0),                  # one class: loss 0, no gradient
    (1, 64, 300, 0),               # a single row
    (2, 1, 5, 0),                  # one feature
    (3, 33, 77, 0),                # odd features: padded copies
    (20, 512, 1000, 0),
    (64, 1024, 4096, 0),           # products in many runs
    (255, 40, 257, 0),             # a class past a tile
    (257, 130, 513, 0),            # rows, features and classes past their tiles
    (1000, 256, 300, 0),
    (300, 64, 2000, 512),          # pieces, the last one short
    (130, 77, 1300, 256),          # pieces with padded copies
    (40, 96, 3000, 1024),          # pieces, few rows
    (513, 264, 2100, 768),
    (5, 2048, 20000, 0),
    (40, 96, 12000, 4096),         # pieces with products in runs, the last piece with fewer runs
    (3000, 48, 600, 0),            # dw in runs
]


@pytest.mark.parametrize("n,d,v,piece", CASES)
def test_against_64_bits(cl, n, d, v, piece):
    x, w, t = inputs(n, d, v, scale=2.0)
    if n > 2:
        t[1], t[n - 1] = -1, v      # two rows that are left out
    ref = reference(x, w, t)
    plan, out = run(cl, x, w, t, piece)
    for k in ("lse", "row", "loss", "dx", "dw"):
        close(out[k], ref[k], ref[k + "_tol"], (k, plan.describe()))


def test_confident_and_wide_scores(cl):
    """Scores from -200 to 200: maxima far apart between tiles, probabilities
    of one and of zero."""
    x, w, t = inputs(70, 128, 900, 3, scale=50.0)
    ref = reference(x, w, t)
    plan, out = run(cl, x, w, t, 256)
    for k in ("lse", "row", "loss", "dx", "dw"):
        close(out[k], ref[k], ref[k + "_tol"], k)


def test_labels_left_out(cl):
    """No labelled row: loss and gradients are 0.  Labels far outside the
    classes are read as none."""
    x, w, t = inputs(30, 64, 500, 4)
    out = run(cl, x, w, torch.full_like(t, -100), 256)[1]
    assert float(out["loss"]) == 0 and not out["dx"].any() and not out["dw"].any() and not out["row"].any()
    t2 = t.clone()
    t2[::2] = torch.tensor([-2 ** 31, 2 ** 31 - 1, -1, 500, 12345], dtype=torch.int32, device="cuda").repeat(3)
    ref = reference(x, w, t2)
    out = run(cl, x, w, t2, 256)[1]
    for k in ("lse", "row", "loss", "dx", "dw"):
        close(out[k], ref[k], ref[k + "_tol"], k)
    assert not out["dx"][::2].any()


def test_every_row_the_same_label(cl):
    x, w, t = inputs(400, 64, 300, 5)
    t.fill_(299)
    ref = reference(x, w, t)
    out = run(cl, x, w, t)[1]
    for k in ("loss", "dx", "dw"):
        close(out[k], ref[k], ref[k + "_tol"], k)


def test_incoming_gradient(cl):
    x, w, t = inputs(50, 72, 600, 6)
    d = torch.tensor(-3.5, device="cuda")
    ref = reference(x, w, t, -3.5)
    out = run(cl, x, w, t, 0, d)[1]
    for k in ("dx", "dw"):
        close(out[k], ref[k], ref[k + "_tol"], k)


def test_non_finite_rows(cl):
    """A NaN in a row spoils the loss and that row's lse, and no other row's."""
    x, w, t = inputs(300, 64, 700, 7)
    x[5, 3] = float("nan")
    out = run(cl, x, w, t)[1]
    rest = torch.arange(300, device="cuda") != 5
    assert torch.isnan(out["lse"][5]) and torch.isnan(out["loss"]) and torch.isfinite(out["lse"][rest]).all()
    assert torch.isnan(out["dx"][5]).all() and torch.isfinite(out["dx"][rest]).all()


def test_gradient_against_differences(cl):
    """loss(w + h) - loss(w - h) against sum dw 2h along a step h of which both
    ends are bf16 numbers, and the same for x.  The difference is off by the
    third derivative (of order |h|^3, below 1e-3 of it here), the gradient by
    its roundings (2^-8 of g, 2^-8 of itself): 1e-2 of the terms' sizes."""
    x, w, t = inputs(60, 48, 400, 8)
    plan, out = run(cl, x, w, t)
    for which, grad in (("x", out["dx"]), ("w", out["dw"])):
        base = x if which == "x" else w
        # along the gradient, so that the difference is far above the loss's rounding
        step = grad.float() / grad.float().norm() * 0.5 * float(base.float().std())
        hi, lo = (base.float() + step).to(torch.bfloat16), (base.float() - step).to(torch.bfloat16)
        vals = []
        for b in (hi, lo):
            loss = torch.empty((), device="cuda")
            plan.run(b if which == "x" else x, b if which == "w" else w, t, loss)
            vals.append(float(loss))
        terms = grad.double() * (hi.double() - lo.double())
        assert abs(float(terms.sum()) - (vals[0] - vals[1])) <= 1e-2 * float(terms.abs().sum())


def test_offsets_past_31_bits(cl):
    """Class rows past element 2^31 of w and dw."""
    n, d, v = 4, 2048, 1_060_000
    x = inputs(n, d, 1, 10)[0]
    w = torch.empty(v, d, dtype=torch.bfloat16, device="cuda")
    w.normal_(0, 0.02, generator=torch.Generator("cuda").manual_seed(1))
    t = torch.tensor([v - 1, 0, v - 2, 1_050_000], dtype=torch.int32, device="cuda")
    plan = cl.ClassLossPlan(n, d, v)
    loss, lse = torch.empty((), device="cuda"), torch.empty(n, device="cuda")
    dx, dw = torch.empty_like(x), torch.empty_like(w)
    plan.run(x, w, t, loss, lse)
    plan.run_backward(x, w, t, lse, dx, dw)
    plan.check_device_status()
    z = torch.cat([x.float() @ c.float().t() for c in w.split(65536)], dim=1).double()
    ref = torch.logsumexp(z, dim=1)
    assert (lse.double() - ref).abs().max() < 1e-4
    assert abs(float(loss) - float((ref - z[torch.arange(n), t.long()]).mean())) < 1e-4
    p = torch.exp(z - ref[:, None])
    p[torch.arange(n), t.long()] -= 1
    rows = torch.tensor([0, 5, 1_048_575, 1_048_576, 1_050_000, v - 2, v - 1], device="cuda")
    want = p[:, rows].t() / n @ x.double()
    tol = p[:, rows].abs().t() / n @ x.double().abs() * 2.0 ** -7 + 1e-12
    assert ((dw[rows].double() - want).abs() <= tol).all()


def test_streams_graph_and_repeat(cl):
    x, w, t = inputs(300, 128, 3000, 11)
    plan = cl.ClassLossPlan(300, 128, 3000, 1024)

    def outs():
        return [torch.zeros((), device="cuda"), torch.zeros(300, device="cuda"), torch.zeros_like(x), torch.zeros_like(w)]

    def go(o, stream=None):
        plan.run(x, w, t, o[0], o[1], stream=stream)
        plan.run_backward(x, w, t, o[1], o[2], o[3], stream=stream)

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
    plan.check_device_status()


def test_refusals(cl):
    x, w, t = inputs(16, 64, 100, 12)
    plan = cl.ClassLossPlan(16, 64, 100)
    loss, lse = torch.empty((), device="cuda"), torch.empty(16, device="cuda")
    with pytest.raises(TypeError):
        plan.run(x.float(), w, t, loss, lse)
    with pytest.raises(TypeError):
        plan.run(x, w, t.long(), loss, lse)
    with pytest.raises(ValueError):
        plan.run(x, w[:50], t, loss, lse)
    with pytest.raises(ValueError):
        plan.run(x, w, t, torch.empty(1, device="cuda"), lse)
    with pytest.raises(ValueError):
        plan.run(x.t().contiguous().t(), w, t, loss, lse)
    with pytest.raises(ValueError):
        plan.run_backward(x, w, t, None, x.clone(), w.clone())
    with pytest.raises(cl.ConvError) as e:
        plan.run_backward(x, w, t, lse, x, w.clone())
    assert e.value.code == -5
    lib = cl.load_library()
    ws = torch.empty(plan.workspace_bytes, dtype=torch.uint8, device="cuda")
    a = [plan.handle, x.data_ptr(), w.data_ptr(), t.data_ptr(), loss.data_ptr(), None, lse.data_ptr(), ws.data_ptr(), None]
    assert lib.conv_run_xent(*a) == 0
    assert lib.conv_run_xent(*(a[:1] + [None] + a[2:])) == -1
    assert lib.conv_run_xent(*(a[:7] + [None, None])) == -1
    assert lib.conv_run_xent(*(a[:2] + [w.data_ptr() + 2] + a[3:])) == -4
    assert lib.conv_run(plan.handle, x.data_ptr(), w.data_ptr(), None, lse.data_ptr(), None) == -9
    assert plan.algo == "xent" and plan.describe().startswith("xent")
    torch.cuda.synchronize()


def test_no_rows(cl):
    plan = cl.ClassLossPlan(0, 64, 100)
    x, w = torch.empty(0, 64, device="cuda", dtype=torch.bfloat16), torch.ones(100, 64, device="cuda", dtype=torch.bfloat16)
    t, loss = torch.empty(0, device="cuda", dtype=torch.int32), torch.full((), 5.0, device="cuda")
    plan.run(x, w, t, loss)
    assert float(loss) == 0
    dw = torch.ones_like(w)
    plan.run_backward(x, w, t, torch.empty(0, device="cuda"), x.clone(), dw)
    assert not dw.any()
