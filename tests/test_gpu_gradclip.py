"""The global gradient norm and clipping against 64 bits.

The norm: a lane sums up to 160 squares of an item in four chains of fp32
multiply-adds, at most 40 roundings one after another and two to join them, then
fp64: the sum is off by at most 43 u of itself, u = 2^-24, its root by half of
that and a rounding, 23 u; allowed are 82 u.  The factor adds two roundings,
a product one, 27 u (allowed 83 u), and a bf16 result 2^-8 of an element."""
import math

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


def reference(grads, max_norm):
    total = math.fsum(float((g.double() ** 2).sum()) for g in grads)
    norm = math.sqrt(total)
    k = min(1.0, max_norm / (norm + 1e-6))
    return norm, k, [g.double() * k for g in grads]


def check(got, want, k, norm, ref):
    assert abs(float(norm) - ref) <= 82 * U * ref
    for a, b in zip(got, want):
        lim = (83 * U if k != 1.0 else 0.0) * b.abs() + (b.abs() * 2.0 ** -8 if a.dtype is torch.bfloat16 and k != 1.0 else 0.0)
        # (an fp32 product below the normal numbers, and a bf16 one, rounds by half a step of those)
        lim = lim + (2.0 ** -134 if a.dtype is torch.bfloat16 else 2.0 ** -150) * (k != 1.0)
        assert bool(((a.double() - b).abs() <= lim).all())


def draw(counts, dtypes, seed, std=0.1, offset=0):
    g = torch.Generator("cuda").manual_seed(seed)
    out = []
    for k, d in zip(counts, dtypes):
        buf = torch.full((k + offset + 1,), 7.0, device="cuda", dtype=DT[d])
        v = buf[offset:offset + k]
        v.copy_(torch.randn(k, generator=g, device="cuda") * std)
        out.append(v)
    return out


SETS = [
    ([1], ["f32"]),
    ([1], ["bf16"]),
    ([0, 5, 0], ["f32", "bf16", "bf16"]),
    ([7, 8, 9, 15, 16, 17], ["bf16"] * 6),
    ([3, 4, 5, 31, 33], ["f32"] * 5),
    ([255, 256, 257, 2047, 2048, 2049, 4096, 4097], ["bf16", "f32"] * 4),
    ([128 * 1000, 128, 128], ["bf16", "f32", "f32"]),
    ([1000003, 77, 500009], ["bf16", "f32", "f32"]),
    ([5_000_011], ["bf16"]),
    ([3_000_017, 12], ["f32", "bf16"]),
    ([64] * 65, ["f32"] * 65),                  # more tensors than the smallest launch takes
    ([11, 200] * 300, ["bf16", "f32"] * 300),   # ... than the middle one
    ([33] * 4000, ["bf16"] * 4000),             # ... than one launch
]


@pytest.mark.parametrize("i", range(len(SETS)))
@pytest.mark.parametrize("offset", [0, 1, 3])
def test_norm_and_clipping(cl, i, offset):
    counts, dtypes = SETS[i]
    grads = draw(counts, dtypes, i, offset=offset)
    plan = cl.GradClipPlan(counts, dtypes)
    norm = torch.full((), 9.0, device="cuda")
    full, _, _ = reference(grads, 1.0)
    for max_norm in (full * 0.3, full * 2, math.inf):
        ref, k, want = reference(grads, max_norm)
        before = [g.clone() for g in grads]
        out = draw(counts, dtypes, 50 + i, offset=(offset * 2) % 5)
        plan.run(grads, max_norm, norm, out=out)
        check(out, want, k, norm, ref)
        assert all(torch.equal(a, b) for a, b in zip(grads, before))
        for t in out + grads:  # nothing beside a tensor was written
            b = t._base
            assert bool((b[t.storage_offset() + t.numel():] == 7).all()) and bool((b[:t.storage_offset()] == 7).all())
    ref, k, want = reference(grads, full * 0.3)
    plan.run(grads, full * 0.3, norm)           # in place
    check(grads, want, k, norm, ref)


def test_no_tensors(cl):
    plan = cl.GradClipPlan([])
    norm = torch.full((), 9.0, device="cuda")
    plan.run([], 1.0, norm)
    assert float(norm) == 0.0


def test_shapes_and_mixed_places(cl):
    """Tensors of several axes; some clipped in place, others into tensors of their own."""
    grads = [t.view(s) for t, s in zip(draw([24, 60, 7], ["f32", "bf16", "f32"], 3), ((2, 3, 4), (60,), (7, 1)))]
    plan = cl.GradClipPlan([g.shape for g in grads], ["f32", "bf16", "f32"])
    ref, k, want = reference(grads, 0.1)
    out = [grads[0], torch.empty_like(grads[1]), grads[2]]
    norm = torch.empty((), device="cuda")
    plan.run(grads, 0.1, norm, out=out)
    check(out, want, k, norm, ref)


@pytest.mark.parametrize("dtype,size", [("f32", 1e25), ("f32", 1e-30), ("bf16", 1e30), ("bf16", 1e-25), ("f32", 3e-39), ("f32", 1e18)])
def test_squares_beyond_fp32(cl, dtype, size):
    """Gradients whose squares overflow or vanish in fp32 have a norm all the same, beside zeros and ordinary ones."""
    counts = [5000, 3, 4097, 9000]
    grads = draw(counts, [dtype] * 4, 5, std=size)
    grads[3].zero_()
    norm = torch.empty((), device="cuda")
    plan = cl.GradClipPlan(counts, dtype)
    # (elements of 3e-39 are fewer bits themselves: the reference has the same ones)
    for max_norm in (math.inf, 1e-3 if size > 1 else math.inf):
        ref, k, want = reference(grads, max_norm)
        out = draw(counts, [dtype] * 4, 6)
        plan.run(grads, max_norm, norm, out=out)
        check(out, want, k, norm, ref)
    grads[1][1] = 0.25  # one ordinary element among vanishing ones, or vanishing beside the others
    ref, k, want = reference(grads, math.inf)
    plan.run(grads, math.inf, norm)
    assert abs(float(norm) - ref) <= 82 * U * ref


@pytest.mark.parametrize("bad", [float("nan"), float("inf"), -float("inf")])
@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_not_finite_clips_nothing(cl, dtype, bad):
    counts = [3000, 5]
    grads = draw(counts, [dtype] * 2, 7)
    grads[0][2999] = bad
    before = [g.clone() for g in grads]
    norm = torch.empty((), device="cuda")
    plan = cl.GradClipPlan(counts, dtype)
    plan.run(grads, 0.5, norm)
    assert not math.isfinite(float(norm)) and math.isnan(float(norm)) == math.isnan(bad)
    out = [torch.empty_like(g) for g in grads]
    plan.run(grads, 0.5, norm, out=out)
    for a, b, c in zip(grads, before, out):
        assert torch.equal(a.nan_to_num(7.0), b.nan_to_num(7.0)) and torch.equal(c.nan_to_num(7.0), b.nan_to_num(7.0))


def test_a_norm_past_fp32(cl):
    """Finite gradients whose norm is above the largest fp32 number: infinite, and nothing clipped."""
    g = torch.full((100,), 3e38, device="cuda")
    norm = torch.empty((), device="cuda")
    cl.GradClipPlan([100], "f32").run([g], 1.0, norm)
    assert math.isinf(float(norm)) and bool((g == torch.tensor(3e38)).all())


def test_zeros_and_exact_border(cl):
    norm = torch.empty((), device="cuda")
    z = torch.zeros(70000, device="cuda", dtype=torch.bfloat16)
    cl.GradClipPlan([70000]).run([z], 1.0, norm)
    assert float(norm) == 0.0 and not z.any()
    g = torch.tensor([3.0, 4.0], device="cuda")
    cl.GradClipPlan([2], "f32").run([g], 6.0, norm)
    assert float(norm) == 5.0 and g.tolist() == [3.0, 4.0]
    cl.GradClipPlan([2], "f32").run([g], 2.5, norm)   # 2.5 / (5 + 1e-6), rounded once, then each product once
    k = torch.tensor(2.5 / (5 + 1e-6), dtype=torch.float64).float()
    assert float(norm) == 5.0 and g.tolist() == [float(3 * k), float(4 * k)]


def test_offsets_past_32_bits(cl):
    """A tensor of more than 2^32 bytes and 2^31 elements."""
    n = (1 << 31) + 12345
    g = torch.zeros(n, device="cuda", dtype=torch.bfloat16)
    g[-1000:] = 2.0
    g[:1000] = 1.0
    norm = torch.empty((), device="cuda")
    plan = cl.GradClipPlan([n])
    plan.run([g], 1.0, norm)
    ref = math.sqrt(5000.0)
    assert abs(float(norm) - ref) <= 82 * U * ref
    want = torch.tensor([1.0, 2.0], dtype=torch.float64) / (ref + 1e-6)
    assert bool(((g[:1000].double().cpu() - want[0]).abs() <= want[0] * 2.0 ** -7).all())
    assert bool(((g[-1000:].double().cpu() - want[1]).abs() <= want[1] * 2.0 ** -7).all())
    assert not g[1000:-1000].any()


def test_streams_graph_and_repeat(cl):
    counts, dtypes = [300001, 128, 4097], ["bf16", "f32", "f32"]
    grads = draw(counts, dtypes, 9)
    plan = cl.GradClipPlan(counts, dtypes)

    def outs():
        return [torch.zeros_like(g) for g in grads], torch.zeros((), device="cuda")

    def go(o, stream=None):
        plan.run(grads, 0.5, o[1], out=o[0], stream=stream)

    a, b, c, d, e = (outs() for _ in range(5))
    go(a)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    go(b, stream=s)
    with torch.cuda.stream(s):
        go(c)
    torch.cuda.synchronize()
    graphs = [torch.cuda.CUDAGraph(), torch.cuda.CUDAGraph()]
    for g, o in zip(graphs, (d, e)):
        with torch.cuda.graph(g):
            go(o)
    with torch.cuda.stream(s):
        graphs[0].replay()
    graphs[1].replay()
    torch.cuda.synchronize()
    for other in (b, c, d, e):
        assert torch.equal(a[1], other[1]) and all(torch.equal(p, q) for p, q in zip(a[0], other[0]))


def test_refusals(cl):
    grads = draw([64, 32], ["f32", "bf16"], 10)
    plan = cl.GradClipPlan([64, 32], ["f32", "bf16"])
    norm = torch.empty((), device="cuda")
    for bad in (grads[:1], [grads[0], None], [grads[0], grads[1].float()], [grads[0][:63], grads[1]], [grads[0].cpu(), grads[1]],
                [draw([128], ["f32"], 1)[0][::2], grads[1]]):
        with pytest.raises((TypeError, ValueError)):
            plan.run(bad, 1.0, norm)
        with pytest.raises((TypeError, ValueError)):
            plan.run(grads, 1.0, norm, out=bad)
    with pytest.raises(ValueError):
        plan.run(grads, 1.0, torch.empty(1, device="cuda"))
    with pytest.raises(ValueError):
        cl.GradClipPlan([3, 4], ["f32"])

    def code(*a, plan=plan, **kw):
        with pytest.raises(cl.ConvError) as e:
            plan.run(*a, **kw)
        return e.value.code

    for max_norm in (0.0, -1.0, float("nan")):
        assert code(grads, max_norm, norm) == -9
    same = cl.GradClipPlan([64, 64, 32], "f32")
    buf = torch.zeros(256, device="cuda")
    a, b, c = buf[:64], buf[64:128], buf[128:160]
    same.run([a, b, c], 1.0, norm)
    assert code([a, a, c], 1.0, norm, plan=same) == -5                     # a tensor twice
    assert code([a, buf[63:127], c], 1.0, norm, plan=same) == -5
    o = [torch.empty_like(t) for t in (a, b, c)]
    same.run([a, a, c], 1.0, norm, out=o)                                  # (only read: it counts twice)
    assert code([a, b, c], 1.0, norm, out=[o[0], o[0], o[2]], plan=same) == -5
    assert code([a, b, c], 1.0, norm, out=[b, a, c], plan=same) == -5
    assert code([a, b, c], 1.0, buf[10:11].view(()), plan=same) == -5
    same.run([a, b, c], 1.0, norm, out=[a, b, o[2]])
    with pytest.raises(cl.ConvError) as e:
        cl.GradClipPlan([4], "i8")
    assert e.value.code == -3
    assert plan.launches == 1 and cl.GradClipPlan([1 << 20], "f32").launches == 2
    assert plan.algo == "gradclip" and plan.describe().startswith("gradclip")
    lib = cl.load_library()
    assert lib.conv_run(plan.handle, buf.data_ptr(), buf.data_ptr(), None, o[0].data_ptr(), None) == -9
    plan.check_device_status()
