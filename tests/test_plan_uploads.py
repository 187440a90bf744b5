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
