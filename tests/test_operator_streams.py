"""The binding takes device memory for a run on the stream of that run.

A block that torch's allocator hands out on one stream is free only for work
ordered after that stream's: taken on another, a kernel still queued there may
be using it.  No GPU: torch's allocator and streams are stood in for by fakes
in which every block notes the stream that was current when it was taken."""
import contextlib
import ctypes

import pytest
import torch

import convolution_nhwc_implicit_gb300 as cl

CURRENT, OTHER = 100, 200


class Fake:
    """A device tensor as far as the binding asks."""

    def __init__(self, shape, dtype, made_on=CURRENT):
        self.shape, self.dtype, self.made_on = torch.Size(shape), dtype, made_on
        self.device, self.is_cuda = torch.device("cuda", 0), True

    def is_contiguous(self):
        return True

    def get_device(self):
        return 0

    def data_ptr(self):
        return 4096

    def record_stream(self, stream):
        pass


class Stream:
    """A stream object of another library: only the handle."""

    def __init__(self, handle):
        self.cuda_stream = handle


class Lib:
    """Every entry point succeeds; the last argument of each is its stream."""

    def __init__(self):
        self.streams = []

    def __getattr__(self, name):
        def call(*args):
            self.streams.append(args[-1])
            return 0
        return call


@pytest.fixture
def world(monkeypatch):
    now, made = [CURRENT], []

    @contextlib.contextmanager
    def within(stream):
        now.append(stream.cuda_stream)
        yield
        now.pop()

    def empty(*shape, dtype=None, device=None):
        made.append(Fake(shape, dtype, now[-1]))
        return made[-1]

    monkeypatch.setattr(torch, "empty", empty)
    monkeypatch.setattr(torch.cuda, "stream", within)
    monkeypatch.setattr(torch.cuda, "ExternalStream", lambda handle, device=None: Stream(handle))
    monkeypatch.setattr(torch.cuda, "default_stream", lambda device=None: Stream(0))
    monkeypatch.setattr(cl, "_current_stream", lambda *a: now[-1])
    monkeypatch.setattr(cl, "_current_device", lambda: 0, raising=False)
    lib = Lib()
    monkeypatch.setattr(cl, "load_library", lambda: lib)
    return made, lib


def plan_of(cls, **fields):
    p = object.__new__(cls)
    p._lib, p._handle, p._device = cl.load_library(), ctypes.c_void_p(), 0
    p._f32, p._dt, p._i32, p._u8 = torch.float32, torch.bfloat16, torch.int32, torch.uint8
    p.workspace_bytes = p.workspace_bytes_backward = 1024
    for k, v in fields.items():
        setattr(p, k, v)
    return p


def group_norm(stream):
    p = plan_of(cl.GroupNormPlan, shape=(1, 160, 160, 64), groups=4, _cshape=(64,), _sshape=(1, 4))
    m = Fake(p.shape, torch.bfloat16)
    s = Fake((1, 4), torch.float32)
    p.run(m, None, None, m, s, s, stream=stream)
    p.run_backward(m, None, None, s, s, m, m, stream=stream)


def class_loss(stream):
    p = plan_of(cl.ClassLossPlan, shape=(20, 64, 300))
    x, w, t = Fake((20, 64), torch.bfloat16), Fake((300, 64), torch.bfloat16), Fake((20,), torch.int32)
    loss, lse = Fake((), torch.float32), Fake((20,), torch.float32)
    p.run(x, w, t, loss, lse, stream=stream)
    p.run_backward(x, w, t, lse, x, w, stream=stream)


def pack(stream):
    p = plan_of(cl.W4Plan, shape=(1, 64, 32), packed_bytes=2048)
    return [p.pack(Fake((32, 32), torch.uint8), stream=stream)]


def quantize(stream):
    return cl.w4_quantize(Fake((32, 64), torch.bfloat16), 32, stream=stream)


@pytest.mark.parametrize("run,blocks", [(group_norm, 2), (class_loss, 2), (pack, 1), (quantize, 2)])
@pytest.mark.parametrize("stream,handle", [(None, CURRENT), (Stream(OTHER), OTHER), (OTHER, OTHER), (0, 0)])
def test_memory_belongs_to_the_stream_of_the_run(world, run, blocks, stream, handle):
    made, lib = world
    run(stream)
    assert [b.made_on for b in made] == [handle] * blocks
    assert set(lib.streams) == {handle}
