"""The operators around the layer (group norm, 4-bit pointwise) refuse invalid
sizes and options with the named status codes, on the host, before any CUDA
call; an empty plan pointer is refused by every entry point."""
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
    ((1, 0, 4, 8, 2, 1e-5, 1, 0), SHAPE),
    ((1, 4, 0, 8, 2, 1e-5, 1, 0), SHAPE),
    ((1, 4, 4, 0, 1, 1e-5, 1, 0), SHAPE),
    ((-1, 4, 4, 8, 2, 1e-5, 1, 0), SHAPE),
    ((1, 4, 4, 8, 0, 1e-5, 1, 0), SHAPE),
    ((1, 4, 4, 8, 3, 1e-5, 1, 0), SHAPE),              # groups must divide the channels
    ((1, 4, 4, 8, 2, -1.0, 1, 0), ARG),
    ((1, 4, 4, 8, 2, float("nan"), 1, 0), ARG),
    ((1, 4, 4, 8, 2, float("inf"), 1, 0), ARG),
    ((1, 4, 4, 8, 2, 1e-5, 3, 0), ARG),                # no such dtype
    ((1, 4, 4, 8, 2, 1e-5, 1, 3), ARG),                # no such activation
    ((1, 4, 4, 8, 2, 1e-5, 2, 0), UNSUPPORTED),        # int8 maps
    ((1, 4, 4, 8193, 1, 1e-5, 1, 0), UNSUPPORTED),     # more channels than fit
    ((65535, 1, 1, 8, 2, 1e-5, 1, 0), UNSUPPORTED),
    ((1, 1 << 15, 1 << 15, 8, 2, 1e-5, 1, 0), UNSUPPORTED),
])
def test_groupnorm_refusals(lib, args, want):
    h = ctypes.c_void_p(12345)
    assert lib.conv_plan_create_groupnorm(*args, ctypes.byref(h)) == want
    assert h.value is None
    assert lib.conv_plan_create_groupnorm(*args, None) == NULL


@pytest.mark.parametrize("args,want", [
    ((-1, 64, 64, 32, 1, 0), SHAPE),
    ((1, 0, 64, 32, 1, 0), SHAPE),
    ((1, 64, 0, 32, 1, 0), SHAPE),
    ((1, 64, 64, 16, 1, 0), ARG),                      # group is 32, 64 or 128
    ((1, 64, 64, 0, 1, 0), ARG),
    ((1, 64, 64, 256, 1, 0), ARG),
    ((1, 64, 64, 32, -1, 0), ARG),
    ((1, 64, 64, 32, 1, 5), ARG),
    ((1, 64, 64, 32, 2, 0), UNSUPPORTED),              # int8 activations
    ((1, 1 << 28, 64, 32, 1, 0), UNSUPPORTED),
    ((1 << 21, 64, 64, 32, 1, 0), UNSUPPORTED),
])
def test_w4_refusals(lib, args, want):
    h = ctypes.c_void_p(12345)
    assert lib.conv_plan_create_w4(*args, ctypes.byref(h)) == want
    assert h.value is None
    assert lib.conv_plan_create_w4(*args, None) == NULL


def test_w4_packing_arguments(lib):
    n = ctypes.c_size_t()
    assert lib.conv_w4_packed_bytes(128, 16, ctypes.byref(n)) == 0 and n.value == 1024
    assert lib.conv_w4_packed_bytes(129, 17, ctypes.byref(n)) == 0 and n.value == 4 * 1024
    assert lib.conv_w4_packed_bytes(0, 16, ctypes.byref(n)) == SHAPE
    assert lib.conv_w4_packed_bytes(16, 16, None) == NULL
    assert lib.conv_w4_pack(0, 16, 16, 16, None) == SHAPE
    assert lib.conv_w4_pack(64, 16, None, 16, None) == NULL
    assert lib.conv_w4_pack(64, 16, 4096, 8, None) == -4            # packed not 16-byte aligned
    assert lib.conv_w4_pack(64, 16, 4096, 4096, None) == -5         # packed over the codes
    assert lib.conv_w4_quantize(64, 0, 32, 1, 16, 16, 16, None) == SHAPE
    assert lib.conv_w4_quantize(64, 16, 33, 1, 16, 16, 16, None) == ARG
    assert lib.conv_w4_quantize(64, 16, 32, 2, 16, 16, 16, None) == UNSUPPORTED
    assert lib.conv_w4_quantize(64, 16, 32, 1, 16, None, 16, None) == NULL
    assert lib.conv_w4_quantize(64, 16, 32, 1, 17, 8192, 16384, None) == -4


def test_no_plan(lib):
    n = ctypes.c_size_t()
    assert lib.conv_plan_workspace(None, ctypes.byref(n)) == NULL
    assert lib.conv_run_groupnorm(None, 16, 0, None, None, 16, 0, None, None, None, None) == NULL
    assert lib.conv_run_groupnorm_bwd(None, 16, 0, None, None, 16, 16, 16, 0, 16, 0, None, None, None, None) == NULL
    assert lib.conv_run_w4(None, 16, 16, 16, None, 16, None) == NULL


@pytest.mark.parametrize("args,want", [
    ((-1, 64, 100, 0, 1), SHAPE),
    ((4, 0, 100, 0, 1), SHAPE),
    ((4, 64, 0, 0, 1), SHAPE),
    ((4, 64, 100, -1, 1), SHAPE),
    ((4, 64, 100, 0, 5), ARG),
    ((4, 64, 100, 0, 0), UNSUPPORTED),                 # fp32
    ((4, 64, 100, 0, 2), UNSUPPORTED),                 # int8
    ((4, 64, (1 << 24) + 1, 0, 1), UNSUPPORTED),
    (((1 << 24) + 1, 64, 100, 0, 1), UNSUPPORTED),
    ((4, (1 << 20) + 1, 100, 0, 1), UNSUPPORTED),
])
def test_xent_refusals(lib, args, want):
    h = ctypes.c_void_p(12345)
    assert lib.conv_plan_create_xent(*args, ctypes.byref(h)) == want
    assert h.value is None
    assert lib.conv_plan_create_xent(*args, None) == NULL
    assert lib.conv_run_xent(None, 16, 16, 16, 16, None, None, 16, None) == NULL
    assert lib.conv_run_xent_bwd(None, 16, 16, 16, 16, None, 16, 16, 16, None) == NULL
