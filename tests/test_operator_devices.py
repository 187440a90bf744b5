"""A tensor of another GPU than the plan's, and a plan of another GPU than the
current one, are refused before anything is launched.  No GPU: tensors and the
library are fakes."""
import ctypes

import pytest
import torch

import convolution_nhwc_implicit_gb300 as cl


class Fake:
    def __init__(self, shape, dtype, index=0):
        self.shape, self.dtype, self.index = torch.Size(shape), dtype, index
        self.device, self.is_cuda = torch.device("cpu" if index < 0 else f"cuda:{index}"), index >= 0

    def is_contiguous(self):
        return True

    def get_device(self):
        return self.index

    def data_ptr(self):
        return 4096


class Lib:
    def __init__(self):
        self.calls = 0

    def __getattr__(self, name):
        def call(*args):
            self.calls += 1
            return 0
        return call


@pytest.fixture
def lib(monkeypatch):
    lib = Lib()
    monkeypatch.setattr(cl, "load_library", lambda: lib)
    monkeypatch.setattr(cl, "_current_stream", lambda *a: 0)
    monkeypatch.setattr(cl, "_current_device", lambda: 0, raising=False)
    return lib


BF16, F32, I32, U8 = torch.bfloat16, torch.float32, torch.int32, torch.uint8


def plan_of(cls, **fields):
    p = object.__new__(cls)
    p._lib, p._handle, p._device = cl.load_library(), ctypes.c_void_p(), 0
    p._f32, p._dt, p._i32, p._u8 = F32, BF16, I32, U8
    p.workspace_bytes = p.workspace_bytes_backward = 0
    for k, v in fields.items():
        setattr(p, k, v)
    return p


def norm():
    p = plan_of(cl.GroupNormPlan, shape=(2, 4, 4, 16), groups=4, _cshape=(16,), _sshape=(2, 4))
    m, c, s = (p.shape, BF16), ((16,), F32), ((2, 4), F32)
    return p.run, (m, c, c, m, s, s)


def norm_backward():
    p = norm()[0].__self__
    m, c, s = (p.shape, BF16), ((16,), F32), ((2, 4), F32)
    return p.run_backward, (m, c, c, s, s, m, m, c, c)


def loss():
    p = plan_of(cl.ClassLossPlan, shape=(4, 8, 30))
    return p.run, (((4, 8), BF16), ((30, 8), BF16), ((4,), I32), ((), F32), ((4,), F32), ((4,), F32))


def loss_backward():
    p = loss()[0].__self__
    return p.run_backward, (((4, 8), BF16), ((30, 8), BF16), ((4,), I32), ((4,), F32), ((4, 8), BF16), ((30, 8), BF16), ((), F32))


def w4():
    p = plan_of(cl.W4Plan, shape=(1, 64, 32), packed_bytes=2048,
                _shapes=((1, 64), (2048,), (32, 2), (32,), (1, 32)))
    return p.run, (((1, 64), BF16), ((2048,), U8), ((32, 2), BF16), ((32,), F32), ((1, 32), BF16))


def w4_pack():
    return w4()[0].__self__.pack, (((32, 32), U8),)


@pytest.mark.parametrize("make", [norm, norm_backward, loss, loss_backward, w4, w4_pack])
def test_every_tensor_is_on_the_plans_device(lib, monkeypatch, make):
    monkeypatch.setattr(torch, "empty", lambda *s, dtype=None, device=None: Fake(s, dtype))
    run, specs = make()
    run(*(Fake(*s) for s in specs))
    assert lib.calls == 1
    for i in range(len(specs)):
        for index in (1, -1):
            with pytest.raises(ValueError):
                run(*(Fake(*s, index=index if j == i else 0) for j, s in enumerate(specs)))
    assert lib.calls == 1
    monkeypatch.setattr(cl, "_current_device", lambda: 1)  # the same tensors, another current device
    with pytest.raises(ValueError):
        run(*(Fake(*s) for s in specs))
    assert lib.calls == 1


def test_quantise_takes_weights_of_the_current_device(lib, monkeypatch):
    monkeypatch.setattr(torch, "empty", lambda *s, dtype=None, device=None: Fake(s, dtype))
    cl.w4_quantize(Fake((32, 64), BF16), 32)
    assert lib.calls == 1
    for index in (1, -1):
        with pytest.raises(ValueError):
            cl.w4_quantize(Fake((32, 64), BF16, index), 32)
    assert lib.calls == 1
