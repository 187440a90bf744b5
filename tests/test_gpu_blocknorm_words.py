"""Maps of single bf16 values that start and end on odd and even addresses among
NaN: the bits of the same maps alone, and nothing beside them changed."""
import pytest
import torch
from test_gpu_blocknorm import cl, draw, grads_of, parameters  # noqa: F401

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("shape", [(1, 1, 1, 1), (1, 1, 1, 511), (1, 1, 2, 3), (3, 5, 7, 33), (2, 30, 20, 257), (1, 1, 300, 4097)])
@pytest.mark.parametrize("odd,wide", [(0, 0), (1, 0), (0, 1), (1, 1), (1, 6)])
def test_maps_among_nan(cl, shape, odd, wide):  # noqa: F811
    n, h, w, c = shape
    p = parameters(n, c, "layer", "rms", True)
    back = {k: v for k, v in p.items() if k != "pre_beta"}
    plan = cl.BlockNormPlan(*shape, "layer", "rms")

    def place(v):
        buf = torch.full((n * h * w * (c + wide) + 2,), float("nan"), dtype=torch.bfloat16, device="cuda")
        m = buf[odd:odd + n * h * w * (c + wide)].view(n, h, w, c + wide)[..., :c]
        m.copy_(v)
        return buf, m

    plain = [draw(shape, torch.bfloat16, 200 + i) for i in range(8)]
    both = []
    for maps, outer in ((plain, None), tuple(zip(*[(m, b) for b, m in map(place, plain)]))):
        x, f, dy, dz, y, z, dx, df = maps
        stats, d = torch.empty(n, h, w, 4, device="cuda"), grads_of(p)
        plan.run(x, f, y, z, stats, **p)
        plan.run_backward(x, f, stats, dy, dz, dx, df, **back, **d)
        both.append([y.clone(), z.clone(), stats, dx.clone(), df.clone()] + [v for v in d.values() if v is not None])
        plan.run(x, f, x, f, stats, **p)                     # in place
        both[-1] += [x.clone(), f.clone()]
        if outer is not None:
            for b, m in zip(outer, maps):
                m.fill_(float("nan"))
                assert bool(torch.isnan(b).all())            # (nothing beside the map was written)
    for a, b in zip(*both):
        assert torch.equal(a, b) and not torch.isnan(a).any()
