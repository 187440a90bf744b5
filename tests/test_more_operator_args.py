"""The norms around a block and the gradient norm refuse invalid sizes and
options with the named status codes, on the host, before any CUDA call; an
empty plan pointer is refused by every entry point."""
import ctypes

import pytest


@pytest.fixture(scope="module")
def lib():
    from convolution_nhwc_implicit_gb300 import build
    build.build()
    import convolution_nhwc_implicit_gb300 as cl
    return cl.load_library()


SHAPE, UNSUPPORTED, ARG, NULL = -2, -3, -9, -1


@pytest.mark.parametrize("args,want", [
    ((-1, 4, 4, 8, 1, 1, 1e-5, 1), SHAPE),
    ((1, 0, 4, 8, 1, 1, 1e-5, 1), SHAPE),
    ((1, 4, 0, 8, 1, 1, 1e-5, 1), SHAPE),
    ((1, 4, 4, 0, 1, 1, 1e-5, 1), SHAPE),
    ((1, 4, 4, 8, 3, 1, 1e-5, 1), ARG),                # no such norm
    ((1, 4, 4, 8, 1, -1, 1e-5, 1), ARG),
    ((1, 4, 4, 8, 1, 1, -1.0, 1), ARG),
    ((1, 4, 4, 8, 1, 1, float("nan"), 1), ARG),
    ((1, 4, 4, 8, 1, 1, float("inf"), 1), ARG),
    ((1, 4, 4, 8, 1, 1, 1e-5, 3), ARG),                # no such dtype
    ((1, 4, 4, 8, 1, 1, 1e-5, 2), UNSUPPORTED),        # int8 maps
    ((1, 4, 4, 8193, 1, 1, 1e-5, 1), UNSUPPORTED),
    ((1, 1 << 15, 1 << 15, 8, 1, 1, 1e-5, 1), UNSUPPORTED),
    ((1 << 20, 1 << 5, 1 << 5, 8, 1, 1, 1e-5, 1), UNSUPPORTED),
])
def test_blocknorm_refusals(lib, args, want):
    h = ctypes.c_void_p(12345)
    assert lib.conv_plan_create_blocknorm(*args, ctypes.byref(h)) == want
    assert h.value is None
    assert lib.conv_plan_create_blocknorm(*args, None) == NULL


@pytest.mark.parametrize("counts,dtypes,want", [
    ([-1], [0], SHAPE),
    ([4, -4], [0, 0], SHAPE),
    ([4], [3], ARG),
    ([4], [-1], ARG),
    ([4, 4], [1, 2], UNSUPPORTED),                     # int8
    ([1 << 40], [0], UNSUPPORTED),
    ([1 << 39, 1 << 39], [0, 0], UNSUPPORTED),
    ([(1 << 63) - 1, (1 << 63) - 1], [0, 0], UNSUPPORTED),
])
def test_gradclip_refusals(lib, counts, dtypes, want):
    h = ctypes.c_void_p(12345)
    c, d = (ctypes.c_int64 * len(counts))(*counts), (ctypes.c_int * len(dtypes))(*dtypes)
    assert lib.conv_plan_create_gradclip(len(counts), c, d, ctypes.byref(h)) == want
    assert h.value is None
    assert lib.conv_plan_create_gradclip(len(counts), c, d, None) == NULL
    assert lib.conv_plan_create_gradclip(len(counts), None, d, ctypes.byref(h)) == NULL
    assert lib.conv_plan_create_gradclip(-1, None, None, ctypes.byref(h)) == SHAPE


def test_no_plan(lib):
    p = (ctypes.c_void_p * 1)(4096)
    assert lib.conv_run_blocknorm(None, 16, 0, 16, 0, None, 16, 0, 16, 0, None, None) == NULL
    assert lib.conv_run_blocknorm_bwd(None, 16, 0, 16, 0, None, 16, None, 0, 16, 0, 16, 0, 16, 0, None, 16, None) == NULL
    assert lib.conv_run_gradclip(None, p, None, 1.0, 16, 16, None) == NULL


def test_one_dtype_for_each_tensor():
    import convolution_nhwc_implicit_gb300 as cl
    with pytest.raises(ValueError):
        cl.GradClipPlan([3, 4], ["f32"])
