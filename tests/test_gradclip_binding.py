"""The gradient norm's binding where there is nothing to clip: an empty list of
results is an address like any other list's.  No GPU: as in
test_more_operator_streams.py, the library and the tensors are fakes."""
import torch
from test_more_operator_streams import Fake, plan_of, world  # noqa: F401

import convolution_nhwc_implicit_gb300 as cl


def test_no_tensors_into_no_tensors(world):  # noqa: F811
    lib, _ = world
    p = plan_of(cl.GradClipPlan, shapes=[], _counts=[], _dtypes=[], _devices=[])
    for out in (None, []):
        p.run([], 1.0, Fake((), torch.float32), out=out)
        assert all(v is None or isinstance(v, int) for v in lib.calls[-1][1:3])
