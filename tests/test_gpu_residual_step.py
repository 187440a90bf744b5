"""A training step through the operators together, as they would be used: the
norm before the first block, a residual block (pointwise layer, the norm of its
output, gate, residual scale and residual add, the norm after it), the class
loss, all gradients back to the input, and their clipping.

Every stage is compared with 64 bits from the tensors that it was given itself
(the bf16 maps between the stages are inputs of the next one), so that each has
its own tolerance: bf16 results 2^-8 of their size and, for the sums in fp32 that
they are of, 2^-14 of the largest (rows of 96 to 1000 terms, 40 to 1000 u of
their absolute sum, u = 2^-24, which is at most 16 times the result's largest
here); fp32 sums over pixels 2^-12 of their largest."""
import pytest
import torch

pytestmark = pytest.mark.gpu
N, H, W, C, CLASSES = 3, 10, 9, 96, 1000
PIX = N * H * W


@pytest.fixture(scope="module")
def cl():
    from convolution_nhwc_implicit_gb300 import build
    build.build()
    import convolution_nhwc_implicit_gb300 as cl
    return cl


def near(got, ref, what):
    tol = 2.0 ** -8 * ref.abs() + 2.0 ** -14 * ref.abs().max() if got.dtype is torch.bfloat16 else 2.0 ** -12 * ref.abs().max()
    bad = (got.double() - ref).abs() > tol
    assert not bad.any(), (what, int(bad.sum()), float(((got.double() - ref).abs() / tol).max()))


def layer_norm(v, gamma, beta):
    return torch.nn.functional.layer_norm(v, (C,), gamma, beta, 1e-5)


def rms_norm(v, gamma):
    return v / torch.sqrt((v * v).mean(dim=-1, keepdim=True) + 1e-5) * gamma


def step(cl, t, out, stream=None):
    first, block, layer, loss_of, clip = t["plans"]
    first.run(t["x"], None, None, out["s"], out["st1"], pre_gamma=t["g0"], pre_beta=t["b0"], stream=stream)
    layer.run(out["s"], t["v"], t["bias"], out["f"], stream=stream)
    w = dict(scale=t["scale"], gate=t["gate"], post_gamma=t["g1"], pre_gamma=t["g2"])
    block.run(t["x"], out["f"], out["y"], out["z"], out["st2"], pre_beta=t["b2"], stream=stream, **w)
    loss_of.run(out["z"].view(PIX, C), t["head"], t["target"], out["loss"], out["lse"], stream=stream)
    loss_of.run_backward(out["z"].view(PIX, C), t["head"], t["target"], out["lse"], out["dz"].view(PIX, C), out["dhead"], stream=stream)
    block.run_backward(t["x"], out["f"], out["st2"], t["dy"], out["dz"], out["dx"], out["df"], dscale=out["dscale"], dgate=out["dgate"],
                       dpost_gamma=out["dg1"], dpre_gamma=out["dg2"], dpre_beta=out["db2"], stream=stream, **w)
    layer.run(out["df"], t["v_back"], None, out["dz_first"], stream=stream)
    first.run_backward(t["x"], None, out["st1"], out["dx"], out["dz_first"], out["dx_all"], None, pre_gamma=t["g0"],
                       dpre_gamma=out["dg0"], dpre_beta=out["db0"], stream=stream)
    clip.run([out[k] for k in t["clipped"]], 0.5, out["length"], out=[out["c_" + k] for k in t["clipped"]], stream=stream)


def world(cl, seed):
    g = torch.Generator("cuda").manual_seed(seed)

    def r(*shape):
        return torch.randn(*shape, generator=g, device="cuda")

    b = torch.bfloat16
    t = dict(x=r(N, H, W, C).to(b), dy=(0.01 * r(N, H, W, C)).to(b), v=(r(C, 1, 1, C) / C ** 0.5).to(b), bias=0.1 * r(C),
             scale=0.5 + 0.1 * r(C), gate=torch.sigmoid(r(N, C)), g0=1 + 0.1 * r(C), b0=0.1 * r(C), g1=1 + 0.1 * r(C),
             g2=1 + 0.1 * r(C), b2=0.1 * r(C), head=(r(CLASSES, C) / C ** 0.5).to(b))
    t["v_back"] = t["v"].view(C, C).t().contiguous().view(C, 1, 1, C)
    t["target"] = torch.randint(-1, CLASSES, (PIX,), generator=g, device="cuda", dtype=torch.int32)
    t["clipped"] = ["dhead", "dg0", "db0", "dg1", "dg2", "db2", "dscale", "dgate"]
    t["plans"] = (cl.BlockNormPlan(N, H, W, C, "none", "layer"), cl.BlockNormPlan(N, H, W, C, "rms", "layer"),
                  cl.Plan(N, H, W, C, C, 1, 1, dtype="bf16"), cl.ClassLossPlan(PIX, C, CLASSES),
                  cl.GradClipPlan([(CLASSES, C)] + [(C,)] * 6 + [(N, C)], ["bf16"] + ["f32"] * 7))
    return t


def outputs():
    out = {k: torch.zeros(N, H, W, C, device="cuda", dtype=torch.bfloat16) for k in ("s", "f", "y", "z", "dz", "dx", "df", "dz_first", "dx_all")}
    out.update({k: torch.zeros(N, H, W, 4, device="cuda") for k in ("st1", "st2")})
    out.update({p + k: torch.zeros(C, device="cuda") for k in ("dg0", "db0", "dg1", "dg2", "db2", "dscale") for p in ("", "c_")})
    out.update({p + "dgate": torch.zeros(N, C, device="cuda") for p in ("", "c_")})
    out.update({p + "dhead": torch.zeros(CLASSES, C, device="cuda", dtype=torch.bfloat16) for p in ("", "c_")})
    out.update(loss=torch.zeros((), device="cuda"), lse=torch.zeros(PIX, device="cuda"), length=torch.zeros((), device="cuda"))
    return out


def test_every_stage_of_a_step(cl):
    t, out = world(cl, 1), outputs()
    step(cl, t, out)
    torch.cuda.synchronize()
    d = {k: v.double().requires_grad_() for k, v in t.items() if torch.is_tensor(v) and v.dtype is not torch.int32}
    s = layer_norm(d["x"], d["g0"], d["b0"])
    near(out["s"], s.detach(), "s")
    near(out["f"], (out["s"].double() @ d["v"].view(C, C).t() + d["bias"]).detach(), "f")
    f = out["f"].double().requires_grad_()
    y = d["x"] + d["scale"] * d["gate"].view(N, 1, 1, C) * rms_norm(f, d["g1"])
    z = layer_norm(y, d["g2"], d["b2"])
    near(out["y"], y.detach(), "y")
    near(out["z"], z.detach(), "z")
    zz = out["z"].double().requires_grad_()
    loss = torch.nn.functional.cross_entropy(zz.view(PIX, C) @ d["head"].t(), t["target"].long(), ignore_index=-1)
    loss.backward()
    assert abs(float(out["loss"]) - float(loss.detach())) <= 1e-5 * float(loss.detach())
    for got, ref, what in ((out["dz"], zz.grad, "dz"), (out["dhead"], d["head"].grad, "dhead")):
        # (the loss's g is rounded to bf16: 2^-8 of the absolute sum, here within 8 times the largest result)
        assert bool(((got.double() - ref).abs() <= 2.0 ** -8 * ref.abs() + 2.0 ** -5 * ref.abs().max()).all()), what
    for v in d.values():
        v.grad = None
    torch.autograd.backward([y, z], [t["dy"].double(), out["dz"].double()])
    for name, ref in (("dx", d["x"].grad), ("df", f.grad), ("dscale", d["scale"].grad), ("dgate", d["gate"].grad), ("dg1", d["g1"].grad),
                      ("dg2", d["g2"].grad), ("db2", d["b2"].grad)):
        near(out[name], ref, name)
    near(out["dz_first"], out["df"].double() @ d["v"].detach().view(C, C), "dz_first")
    for v in d.values():
        v.grad = None
    s.backward(out["dz_first"].double())
    near(out["dx_all"], out["dx"].double() + d["x"].grad, "dx_all")
    near(out["dg0"], d["g0"].grad, "dg0")
    near(out["db0"], d["b0"].grad, "db0")
    length = torch.sqrt(sum((out[k].double() ** 2).sum() for k in t["clipped"]))
    assert abs(float(out["length"]) - float(length)) <= 2.0 ** -20 * float(length) and float(length) > 0.5
    for k in t["clipped"]:
        want = out[k].double() * (0.5 / (length + 1e-6))
        lim = (2.0 ** -8 if out[k].dtype is torch.bfloat16 else 0.0) * want.abs() + 2.0 ** -19 * want.abs() + 1e-37
        assert bool(((out["c_" + k].double() - want).abs() <= lim).all()), k


def test_two_steps_at_once_and_in_graphs(cl):
    """Two steps on two streams at once, and two captured ones replayed at once: the bits of steps alone."""
    worlds = world(cl, 2), world(cl, 3)
    want = outputs(), outputs()
    for t, o in zip(worlds, want):
        step(cl, t, o)
    streams = torch.cuda.Stream(), torch.cuda.Stream()
    both = [[outputs(), outputs()] for _ in range(4)]
    torch.cuda.synchronize()
    for pair in both:
        for t, o, st in zip(worlds, pair, streams):
            step(cl, t, o, stream=st)
    torch.cuda.synchronize()
    graphs, captured = [torch.cuda.CUDAGraph(), torch.cuda.CUDAGraph()], (outputs(), outputs())
    for g, t, o in zip(graphs, worlds, captured):
        with torch.cuda.graph(g):
            step(cl, t, o)
    for _ in range(3):
        for g, st in zip(graphs, streams):
            with torch.cuda.stream(st):
                g.replay()
    torch.cuda.synchronize()
    for pair in both + [captured]:
        for o, w in zip(pair, want):
            for k in w:
                assert torch.equal(o[k], w[k]), k
