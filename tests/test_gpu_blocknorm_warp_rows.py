"""Rows of 257 to 512 channels, of so many rows that a row is a warp's (sixteen
channels a thread), and of so few that it is not: forward against 64 bits with the
bounds of test_gpu_blocknorm.py, and the gradient from its statistics."""
import pytest
import torch
from test_gpu_blocknorm import DT, buffers, cl, close, draw, grads_of, parameters, reference  # noqa: F401

pytestmark = pytest.mark.gpu

CASES = [
    # n, h, w, c, post, pre, dtype, gate, wide, off, channels a thread
    (5, 35, 30, 510, "layer", "rms", "bf16", True, 0, 0, 16),
    (5, 35, 30, 511, "rms", "rms", "bf16", True, 0, 0, 16),
    (1, 71, 71, 511, "layer", "layer", "bf16", False, 0, 0, 16),     # (its maps end in the middle of a word)
    (1, 100, 50, 300, "rms", "rms", "f32", False, 1, 0, 8),          # (whole vectors by its channels: a slice goes by these)
    (1, 100, 50, 301, "rms", "rms", "f32", False, 1, 0, 16),
    (2, 50, 50, 257, "layer", "layer", "f32", True, 0, 0, 16),
    (2, 50, 50, 512, "layer", "layer", "bf16", False, 0, 0, 16),
    (2, 50, 50, 264, "rms", "layer", "bf16", False, 8, 8, 16),
    (2, 50, 50, 512, "layer", "none", "bf16", False, 0, 0, 16),
    (2, 50, 50, 512, "rms", "rms", "bf16", False, 0, 0, 8),
    (3, 20, 20, 510, "layer", "rms", "bf16", False, 0, 0, 8),
    (2, 25, 25, 512, "layer", "layer", "bf16", False, 0, 0, 8),
]


@pytest.mark.parametrize("n,h,w,c,post,pre,dtype,gate,wide,off,channels", CASES)
def test_rows_of_a_warp(cl, n, h, w, c, post, pre, dtype, gate, wide, off, channels):  # noqa: F811
    shape, dt, bf = (n, h, w, c), DT[dtype], dtype == "bf16"
    x, f = draw(shape, dt, 1, wide, off, 0.4, 0.8), draw(shape, dt, 2, wide, off, -0.3, 2.0)
    dy, dz = draw(shape, dt, 3, wide, off, 0.1, 0.5), draw(shape, dt, 4, wide, off, 0.1, 0.5) if pre != "none" else None
    p = parameters(n, c, post, pre, gate)
    ref, tol = reference(x, f, p, post, pre, 1e-5, dy, dz, True)
    y, z, dx, df = buffers(shape, dt, wide, off)
    stats, d = torch.full((n, h, w, 4), 9.0, device="cuda"), grads_of(p)
    plan = cl.BlockNormPlan(n, h, w, c, post, pre, 1e-5, dtype)
    assert f"channels/thread={channels} " in plan.describe()
    plan.run(x, f, y, None if dz is None else z, stats, **p)
    plan.run_backward(x, f, stats, dy, dz, dx, df, **{k: v for k, v in p.items() if k != "pre_beta"}, **d)
    close(y, ref["y"], tol["y"], bf, "y")
    for k, name in enumerate(("m1", "r1", "m2", "r2")):
        if name in ref:
            close(stats[..., k:k + 1], ref[name], tol[name], False, name)
    if dz is not None:
        close(z, ref["z"], tol["z"], bf, "z")
    close(dx, ref["dx"], tol["dx"], bf, "dx")
    close(df, ref["df"], tol["df"], bf, "df")
    for k, v in d.items():
        if v is not None:
            close(v, ref[k], tol[k], False, k)
