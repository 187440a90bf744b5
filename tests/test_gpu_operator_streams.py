"""Runs of one plan on two streams at once keep their scratch apart: each run's
block belongs to its own stream, and the answers are those of runs alone, bit
for bit."""
import pytest
import torch

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def cl():
    from convolution_nhwc_implicit_gb300 import build
    build.build()
    import convolution_nhwc_implicit_gb300 as cl
    return cl


def norm(cl, seed):
    """A group norm in two launches (its workspace holds the runs' results), forward and gradient."""
    g = torch.Generator("cuda").manual_seed(seed)
    x, dy = (torch.randn(2, 160, 160, 64, device="cuda", generator=g).bfloat16() for _ in range(2))
    plan = cl.GroupNormPlan(2, 160, 160, 64, 4, dtype="bf16", act="mish")
    assert plan.workspace_bytes and plan.workspace_bytes_backward

    def outs():
        return torch.empty_like(x), torch.empty_like(x), *(torch.empty(*s, device="cuda") for s in ((2, 4), (2, 4), (64,), (64,)))

    def go(o, stream=None):
        y, dx, mean, rstd, dg, db = o
        plan.run(x, None, None, y, mean, rstd, stream=stream)
        plan.run_backward(x, None, None, mean, rstd, dy, dx, dg, db, stream=stream)
        return o
    return outs, go


def loss(cl, seed):
    g = torch.Generator("cuda").manual_seed(seed)
    x, w = torch.randn(700, 128, device="cuda", generator=g).bfloat16(), torch.randn(5000, 128, device="cuda", generator=g).bfloat16()
    t = torch.randint(0, 5000, (700,), device="cuda", generator=g, dtype=torch.int32)
    plan = cl.ClassLossPlan(700, 128, 5000, 2048)

    def outs():
        return torch.empty((), device="cuda"), torch.empty(700, device="cuda"), torch.empty_like(x), torch.empty_like(w)

    def go(o, stream=None):
        out, lse, dx, dw = o
        plan.run(x, w, t, out, lse, stream=stream)
        plan.run_backward(x, w, t, lse, dx, dw, stream=stream)
        return o
    return outs, go


@pytest.mark.parametrize("make", [norm, loss])
@pytest.mark.parametrize("by_handle", [False, True])
def test_two_streams_at_once(cl, make, by_handle):
    (one_outs, one), (two_outs, two) = make(cl, 1), make(cl, 2)
    want = one(one_outs()), two(two_outs())
    # (outputs first: a block that the binding gave back between two runs may
    # still be in use on the current stream)
    to = [(one_outs(), two_outs()) for _ in range(8)]
    s = torch.cuda.Stream()
    torch.cuda.synchronize()
    got = [(one(a), two(b, stream=s.cuda_stream if by_handle else s)) for a, b in to]
    torch.cuda.synchronize()
    for pair in got:
        for a, b in zip(pair, want):
            assert all(torch.equal(p, q) for p, q in zip(a, b))


@pytest.mark.parametrize("make", [norm, loss])
def test_the_block_is_not_the_other_streams(cl, make, monkeypatch):
    """The scratch that a run on the current stream gave back (its kernels may
    still be queued) is not what a run on another stream gets next."""
    outs, go = make(cl, 3)
    s = torch.cuda.Stream()
    to = outs(), outs(), outs()
    torch.cuda.synchronize()
    took, empty = [], torch.empty

    def watch(*size, **kw):
        t = empty(*size, **kw)
        if kw.get("dtype") is torch.uint8:
            took.append((t.data_ptr(), torch.cuda.current_stream().cuda_stream))
        return t

    monkeypatch.setattr(torch, "empty", watch)
    here = torch.cuda.current_stream().cuda_stream
    go(to[0]), go(to[1], stream=s), go(to[2])
    monkeypatch.undo()
    torch.cuda.synchronize()
    assert [st for _, st in took] == [here] * 2 + [s.cuda_stream] * 2 + [here] * 2
    assert not {p for p, st in took if st == here} & {p for p, st in took if st != here}
    assert all(torch.equal(a, b) and torch.equal(a, c) for a, b, c in zip(*to))


def test_packed_and_quantised_on_another_stream(cl):
    g = torch.Generator("cuda").manual_seed(4)
    w = torch.randn(512, 1024, device="cuda", generator=g).bfloat16()
    plan = cl.W4Plan(1, 1024, 512, 64)
    codes, scales = cl.w4_quantize(w, 64)
    packed = plan.pack(codes)
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    for stream in (s, s.cuda_stream, 0):
        c2, s2 = cl.w4_quantize(w, 64, stream=stream)
        p2 = plan.pack(c2, stream=stream)
        torch.cuda.synchronize()
        assert torch.equal(c2, codes) and torch.equal(s2, scales) and torch.equal(p2, packed)
