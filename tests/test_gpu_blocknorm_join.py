"""The one-launch gradient of the norms around a block where the last CTAs of the
cluster join no channel (the others' shares cover them all): every output against
64 bits with the bounds of test_gpu_blocknorm.py, and the same bits run after run."""
import pytest
import torch
from test_gpu_blocknorm import DT, buffers, cl, close, draw, grads_of, parameters, reference  # noqa: F401

pytestmark = pytest.mark.gpu

IDLE = [
    # n, h, w, c, dtype, gate
    (1, 28, 28, 40, "bf16", False),
    (1, 56, 56, 16, "bf16", False),
    (1, 20, 20, 144, "bf16", False),
    (1, 20, 20, 72, "f32", False),
    (1, 1, 5000, 8, "bf16", False),
    (1, 28, 28, 24, "f32", True),
    (16, 7, 7, 24, "bf16", True),
    (16, 7, 7, 88, "f32", True),
    (16, 1, 1, 8, "bf16", True),
    (16, 1, 1, 40, "f32", True),
    (9, 1, 1, 32, "bf16", True),
    (11, 2, 2, 100, "bf16", True),
    (4, 16, 16, 40, "bf16", True),
    (4, 16, 16, 40, "bf16", False),
    (3, 2, 5, 2, "f32", True),
    (16, 1, 1, 1, "f32", True),
    (16, 3, 3, 3, "bf16", True),
]


@pytest.mark.parametrize("n,h,w,c,dtype,gate", IDLE)
def test_ctas_without_channels(cl, n, h, w, c, dtype, gate):  # noqa: F811
    shape, dt, bf = (n, h, w, c), DT[dtype], dtype == "bf16"
    x, f = draw(shape, dt, 1, mean=0.4, std=0.8), draw(shape, dt, 2, mean=-0.3, std=2.0)
    dy, dz = draw(shape, dt, 3, mean=0.1, std=0.5), draw(shape, dt, 4, mean=0.1, std=0.5)
    p = parameters(n, c, "layer", "layer", gate)
    ref, tol = reference(x, f, p, "layer", "layer", 1e-5, dy, dz, True)
    plan = cl.BlockNormPlan(n, h, w, c, "layer", "layer", 1e-5, dtype)
    assert plan.workspace_bytes_backward == 0  # (one cluster, with a gate and without)
    y, z, dx, df = buffers(shape, dt, 0, 0)
    stats, first = torch.empty(n, h, w, 4, device="cuda"), None
    plan.run(x, f, y, z, stats, **p)
    for _ in range(20):
        d = grads_of(p)
        plan.run_backward(x, f, stats, dy, dz, dx, df, **{k: v for k, v in p.items() if k != "pre_beta"}, **d)
        got = [dx.clone(), df.clone()] + [v for v in d.values() if v is not None]
        first = first or got
        assert all(torch.equal(a, b) for a, b in zip(first, got))
    close(dx, ref["dx"], tol["dx"], bf, "dx")
    close(df, ref["df"], tol["df"], bf, "df")
    for k, v in d.items():
        if v is not None:
            close(v, ref[k], tol[k], False, k)
