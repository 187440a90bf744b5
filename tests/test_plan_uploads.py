"""What a plan puts on the device is there when the plan is returned: a run on a
stream that is not ordered after the legacy one may be the first to read it.  On
a fake runtime whose copies and fills complete when their stream is synchronised."""
import ctypes

import pytest
from fake_cuda import load


@pytest.fixture(scope="module")
def lib(tmp_path_factory):
    return load(tmp_path_factory.mktemp("fake"))


def test_gradient_norm_table(lib):
    for counts in ([5], [1 << 20, 77, 0, 4096], [33] * 4000):
        c, d, h = (ctypes.c_int64 * len(counts))(*counts), (ctypes.c_int * len(counts))(), ctypes.c_void_p()
        assert lib.conv_plan_create_gradclip(len(counts), c, d, ctypes.byref(h)) == 0
        assert lib.fake_queued() == 0
        lib.conv_plan_destroy(h)


class Shape(ctypes.Structure):
    _fields_ = [(k, ctypes.c_int32) for k in ("n", "h", "w", "c_in", "c_out", "k_h", "k_w")]


class Quant(ctypes.Structure):
    _fields_ = [("in_scale", ctypes.c_float), ("out_scale", ctypes.c_float), ("w_scales", ctypes.POINTER(ctypes.c_float))]


@pytest.mark.parametrize("algo", [0, 1])
def test_requantisation_factors_and_status_words(lib, algo):
    scales = (ctypes.c_float * 20)(*[0.5] * 20)
    s, q, h = Shape(1, 8, 8, 12, 20, 3, 3), Quant(0.1, 0.2, scales), ctypes.c_void_p()
    assert lib.conv_plan_create_ex(ctypes.byref(s), 1, 1, 1, 1, 2, 1, ctypes.byref(q), algo, ctypes.byref(h)) == 0
    assert lib.fake_queued() == 0
    lib.conv_plan_destroy(h)


def test_status_word_of_the_class_loss(lib):
    h = ctypes.c_void_p()
    assert lib.conv_plan_create_xent(100, 64, 1000, 0, 1, ctypes.byref(h)) == 0
    assert lib.fake_queued() == 0
    assert lib.conv_plan_check_device_status(h, None) == 0
    lib.fake_set_word(1)                                   # (a wait that ran out, which is told once)
    assert lib.conv_plan_check_device_status(h, None) == -7
    assert lib.fake_queued() == 0
    assert lib.conv_plan_check_device_status(h, None) == 0
    lib.conv_plan_destroy(h)


def test_status_word_of_the_fused_pair(lib):
    h = ctypes.c_void_p()
    s = Shape(1, 16, 16, 64, 64, 3, 3)
    assert lib.conv_plan_create_dwpw(ctypes.byref(s), 1, 1, 0, 1, 1, ctypes.byref(h)) == 0
    assert lib.fake_queued() == 0
    lib.conv_plan_destroy(h)
