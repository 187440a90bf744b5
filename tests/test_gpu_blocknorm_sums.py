"""Sums of the gradient of the norms around a block: gradients that cancel, with a
gate and every parameter's gradient, and sums over thousands of rows a thread.

Bounds as in test_gpu_blocknorm.py, which allows a sum over pixels 300 u of its
terms' absolute sum.  A thread adds its rows one after another, a rounding each,
so where it has more of them than those 300 cover, as many u as rows are added."""
import pytest
import torch
from test_gpu_blocknorm import DT, U, buffers, cl, close, draw, grads_of, mean, parameters, reference  # noqa: F401

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("c", [520, 4096, 4104, 8192])
@pytest.mark.parametrize("post,pre", [("layer", "layer"), ("rms", "rms"), ("none", "layer")])
@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_gradients_that_cancel_under_a_gate(cl, c, post, pre, dtype):  # noqa: F811
    """dz along the normalised stream, and dy against what dz leaves."""
    shape, dt, bf = (3, 5, 7, c), DT[dtype], dtype == "bf16"
    x, f = draw(shape, dt, 1, mean=0.4), draw(shape, dt, 2, mean=-0.3, std=2.0)
    p = parameters(3, c, post, pre, True)
    back = {k: v for k, v in p.items() if k != "pre_beta"}
    plan = cl.BlockNormPlan(*shape, post, pre, 1e-5, dtype)
    y, z, dx, df = buffers(shape, dt, 0, 0)
    stats = torch.empty(3, 5, 7, 4, device="cuda")
    plan.run(x, f, y, z, stats, **p)
    y64 = reference(x, f, p, post, pre, 1e-5)[0]["y"]
    m = mean(y64) if pre == "layer" else 0.0
    hat = (y64 - m) / torch.sqrt(mean((y64 - m) ** 2) + 1e-5)
    noise = draw(shape, dt, 3)
    for dz, dy in (((hat / p["pre_gamma"].double()).to(dt), None), (noise, None)):
        if dz is noise:
            dy = (-reference(x, f, p, post, pre, 1e-5, None, dz, True)[0]["dx"]).to(dt)
        ref, tol = reference(x, f, p, post, pre, 1e-5, dy, dz, True)
        d = grads_of(p)
        plan.run_backward(x, f, stats, dy, dz, dx, df, **back, **d)
        close(dx, ref["dx"], tol["dx"], bf, "dx")
        close(df, ref["df"], tol["df"], bf, "df")
        for k, v in d.items():
            if v is not None:
                close(v, ref[k], tol[k], False, k)


@pytest.mark.parametrize("rows,c,ctas,gate", [
    (76 * 1500, 8192, 76, False),      # rows of two CTAs, one at a time
    (152 * 1200, 4096, 152, False),    # one row at a time
    (152 * 1200, 4096, 152, True),     # ... images of three rows one after another
])
def test_thousands_of_rows_a_thread(cl, rows, c, ctas, gate):  # noqa: F811
    n = rows // 3 if gate else 1
    shape = (n, 1, rows // n, c)
    gates = torch.rand(n, c, device="cuda", generator=torch.Generator("cuda").manual_seed(9)) if gate else None
    p = dict(parameters(1, c, "rms", "layer", False), gate=gates)
    back = {k: v for k, v in p.items() if k != "pre_beta"}
    maps = [torch.empty(shape, device="cuda", dtype=torch.bfloat16) for _ in range(7)]
    x, f, dy, dz, z, dx, df = maps
    g = torch.Generator("cuda").manual_seed(10)
    for i, t in enumerate((x, f, dy, dz)):
        t.normal_(0.1 + 0.1 * i, 0.5, generator=g)
    stats = torch.empty(*shape[:3], 4, device="cuda")
    plan = cl.BlockNormPlan(*shape, "rms", "layer")
    assert f"gradient: {ctas}, gated {n if gate else ctas} in {ctas}" in plan.describe()
    plan.run(x, f, None, z, stats, **p)
    d = grads_of(p)
    plan.run_backward(x, f, stats, dy, dz, dx, df, **back, **d)
    ref, tol = {}, {}
    step = (1 << 24) // c // 3 * 3
    for a in range(0, rows, step):
        b = min(rows, a + step)
        part = {k: v for k, v in p.items() if k != "gate"}
        if gate:
            part["gate"] = gates[a // 3:b // 3]
        one = [t.view(rows, c)[a:b].view(*((b - a) // 3 if gate else 1, 1, 3 if gate else b - a, c)) for t in (x, f, dy, dz)]
        r, t = reference(one[0], one[1], part, "rms", "layer", 1e-5, one[2], one[3], True)
        close(dx.view(rows, c)[a:b], r["dx"].view(-1, c), t["dx"].view(-1, c), True, "dx")
        close(df.view(rows, c)[a:b], r["df"].view(-1, c), t["df"].view(-1, c), True, "df")
        for k in d:
            if d[k] is None:
                continue
            if k == "dgate":
                close(d[k][a // 3:b // 3], r[k], t[k], False, k)
                continue
            # (300 u of the absolute sum of terms are in the bound: scaled, they bound that sum)
            more = rows / ctas / 300
            ref[k], tol[k] = ref.get(k, 0) + r[k], tol.get(k, 0) + t[k] * (1 + more)
    for k in ref:
        close(d[k], ref[k], tol[k], False, k)
