"""The 4-bit layer's packing and quantising take the sizes that its plan takes,
and refuse the others on the host: their counts pass 32 bits."""
import ctypes

import pytest
import torch

SHAPE, UNSUPPORTED, ARG = -2, -3, -9
BIG = [(1 << 28, 64), (2 ** 31 - 1, 16), (64, 1 << 30), (16, 2 ** 31 - 1), (1 << 27, 1 << 14)]


@pytest.fixture(scope="module")
def cl():
    from convolution_nhwc_implicit_gb300 import build
    build.build()
    import convolution_nhwc_implicit_gb300 as cl
    return cl


@pytest.mark.parametrize("c_in,c_out", BIG)
def test_too_large(cl, c_in, c_out):
    lib, n, h = cl.load_library(), ctypes.c_size_t(77), ctypes.c_void_p()
    assert lib.conv_plan_create_w4(1, c_in, c_out, 32, 1, 0, ctypes.byref(h)) == UNSUPPORTED
    assert lib.conv_w4_packed_bytes(c_in, c_out, ctypes.byref(n)) == UNSUPPORTED
    # (addresses far apart that nothing reads: refused before any CUDA call)
    far = [i << 50 for i in range(1, 4)]
    assert lib.conv_w4_pack(c_in, c_out, far[0], far[1], None) == UNSUPPORTED
    assert lib.conv_w4_quantize(c_in, c_out, 32, 1, *far, None) == UNSUPPORTED


def test_the_largest(cl):
    lib, n = cl.load_library(), ctypes.c_size_t()
    assert lib.conv_w4_packed_bytes((1 << 28) - 1, 16, ctypes.byref(n)) == 0 and n.value == 1024 << 21
    assert lib.conv_w4_packed_bytes(1, (1 << 30) - 1, ctypes.byref(n)) == 0 and n.value == 1024 << 26


@pytest.mark.parametrize("w,group", [(torch.zeros(64), 32), (torch.zeros(2, 3, 4), 32), (torch.zeros(4, 64), 0), (torch.zeros(4, 64), -32)])
def test_quantise_refuses_shapes_and_groups(cl, w, group):
    with pytest.raises(ValueError):
        cl.w4_quantize(w, group)
