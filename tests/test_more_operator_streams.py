"""Scratch of the norms around a block and of the gradient norm is a block of
the run's own stream, given back whatever the run answers; every tensor of a run
is on the plan's device, with that device current.  No GPU: torch's allocator,
tensors and the library are fakes."""
import ctypes

import pytest
import torch

import convolution_nhwc_implicit_gb300 as cl

CURRENT, OTHER = 100, 200
BF16, F32 = torch.bfloat16, torch.float32


class Fake:
    """A device tensor as far as the binding asks."""

    def __init__(self, shape, dtype, index=0):
        self.shape, self.dtype, self.index = torch.Size(shape), dtype, index
        self.device = torch.device("cpu" if index < 0 else f"cuda:{index}")

    def is_contiguous(self):
        return True

    def get_device(self):
        return self.index

    def data_ptr(self):
        return 4096

    def numel(self):
        return self.shape.numel()


class Stream:
    def __init__(self, handle):
        self.cuda_stream = handle


class Lib:
    """Every entry point answers `rc`; the last two arguments of each are its workspace, where it has one, and its stream."""

    def __init__(self):
        self.calls, self.rc = [], 0

    def __getattr__(self, name):
        if name == "conv_status_str":
            return lambda code: b"refused"

        def call(*args):
            self.calls.append(args)
            return self.rc
        return call


@pytest.fixture
def world(monkeypatch):
    lib, blocks = Lib(), {}

    def take(nbytes, handle):
        blocks[1 << 20 | len(blocks)] = [nbytes, handle, True]
        return max(blocks)

    def give(address):
        assert blocks[address][2]
        blocks[address][2] = False

    monkeypatch.setattr(cl, "_raw_memory_calls", lambda: (take, give))
    monkeypatch.setattr(cl, "_current_stream", lambda *a: CURRENT)
    monkeypatch.setattr(cl, "_current_device", lambda: 0)
    monkeypatch.setattr(cl, "load_library", lambda: lib)
    return lib, blocks


def plan_of(cls, **fields):
    p = object.__new__(cls)
    p._lib, p._handle, p._device = cl.load_library(), ctypes.c_void_p(), 0
    p._f32, p._dt = F32, BF16
    p.workspace_bytes = p.workspace_bytes_backward = 1024
    for k, v in fields.items():
        setattr(p, k, v)
    return p


def norm():
    return plan_of(cl.BlockNormPlan, shape=(2, 4, 5, 16), _cshape=(16,), _gshape=(2, 16), _sshape=(2, 4, 5, 4), _known={})


def forward():
    p = norm()
    m, c, g, s = (p.shape, BF16), ((16,), F32), ((2, 16), F32), ((2, 4, 5, 4), F32)
    return p.run, (m, m, m, m, s, c, g, c, c, c, c), False


def backward():
    p = norm()
    m, c, g, s = (p.shape, BF16), ((16,), F32), ((2, 16), F32), ((2, 4, 5, 4), F32)
    return p.run_backward, (m, m, s, m, m, m, m, c, g, c, c, c, c, g, c, c, c, c), True


def clip():
    p = plan_of(cl.GradClipPlan, shapes=[(3, 4), (7,)], _counts=[12, 7], _dtypes=[BF16, F32], _devices=[0, 0])
    a, b = ((3, 4), BF16), ((7,), F32)

    def run(one, two, norm, out_one, out_two, **kw):
        p.run([one, two], 1.0, norm, out=[out_one, out_two], **kw)
    return run, (a, b, ((), F32), a, b), True


@pytest.mark.parametrize("make", [forward, backward, clip])
@pytest.mark.parametrize("stream,handle", [(None, CURRENT), (Stream(OTHER), OTHER), (OTHER, OTHER), (0, 0)])
def test_scratch_belongs_to_the_stream_of_the_run(world, make, stream, handle):
    lib, blocks = world
    run, specs, scratch = make()
    run(*(Fake(*s) for s in specs), stream=stream)
    assert lib.calls[0][-1] == handle
    assert [b[:2] for b in blocks.values()] == ([[1024, handle]] if scratch else [])
    if scratch:
        assert lib.calls[0][-2] in blocks
    lib.rc = -5
    with pytest.raises(cl.ConvError):
        run(*(Fake(*s) for s in specs), stream=stream)
    assert not any(b[2] for b in blocks.values())


@pytest.mark.parametrize("make", [forward, backward, clip])
def test_every_tensor_is_checked(world, monkeypatch, make):
    lib, _ = world
    run, specs, _ = make()
    run(*(Fake(*s) for s in specs))
    for i, (shape, dtype) in enumerate(specs):
        wrong = [(Fake(shape, dtype, 1), ValueError), (Fake(shape, dtype, -1), ValueError),
                 (Fake(shape, torch.float16), TypeError), (Fake((*shape, 2), dtype), ValueError)]
        for bad, error in wrong:
            with pytest.raises(error):
                run(*(bad if j == i else Fake(*s) for j, s in enumerate(specs)))
    assert len(lib.calls) == 1
    monkeypatch.setattr(cl, "_current_device", lambda: 1)  # the same tensors, another current device
    with pytest.raises(ValueError):
        run(*(Fake(*s) for s in specs))
    assert len(lib.calls) == 1


def test_absent_tensors_keep_the_others_places(world):
    """What is not given is NULL, and what is given stays what it was."""
    class At(Fake):
        def __init__(self, at, *a):
            super().__init__(*a)
            self.at = at

        def data_ptr(self):
            return self.at

    lib, _ = world
    p = norm()
    m, c = (p.shape, BF16), ((16,), F32)
    p.run(At(1, *m), None, None, At(4, *m), pre_beta=At(9, *c))
    a = lib.calls[-1]
    assert (a[1], a[3], a[6], a[8], a[10]) == (1, None, None, 4, None)
    assert [getattr(a[5], k) for k, _ in a[5]._fields_] == [None] * 5 + [9]
    s = ((2, 4, 5, 4), F32)
    p.run_backward(At(1, *m), At(2, *m), At(3, *s), None, At(5, *m), At(6, *m), At(7, *m), pre_gamma=At(8, *c), dscale=At(9, *c))
    a = lib.calls[-1]
    assert (a[1], a[3], a[6], a[7], a[9], a[11], a[13]) == (1, 2, 3, None, 5, 6, 7)
    assert [getattr(a[5], k) for k, _ in a[5]._fields_] == [None] * 4 + [8, None]
    assert [getattr(a[15], k) for k, _ in a[15]._fields_] == [9] + [None] * 5
