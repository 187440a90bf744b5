"""The example that trains a class head on a layer's features and answers with
it in 4 bits: the loss falls below half of its start (ln of the class count)
and the 4-bit head answers like the bf16 one for most pixels."""
import importlib.util
import math
import os

import pytest

pytestmark = pytest.mark.gpu
ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


def test_class_head_example():
    from convolution_nhwc_implicit_gb300 import build
    build.build()
    spec = importlib.util.spec_from_file_location("class_head", os.path.join(ROOT, "examples", "class_head.py"))
    ex = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(ex)
    out = ex.main(steps=60, say=lambda *_: None)
    assert abs(out["losses"][0] - math.log(1000)) < 0.5
    assert out["losses"][-1] < 0.5 * out["losses"][0]
    assert out["right_bf16"] > 0.5 and out["right_w4"] > 0.8 * out["right_bf16"]
