"""Group norm refuses every buffer that it writes over another that it reads or
writes: CTAs still read the inputs while others write."""
import itertools

import pytest
import torch

from test_gpu_groupnorm import cl  # noqa: F401  (the fixture)

pytestmark = pytest.mark.gpu
SHAPE = (1, 160, 160, 64)                     # two launches: both directions take a workspace
C, G = 64, 4


class Buffers:
    """One dense buffer: each named part of it, 512 bytes apart from the next."""

    def __init__(self, plan):
        m = SHAPE[1] * SHAPE[2] * C * 2
        sizes = dict(x=m, y=m, dy=m, dx=m, gamma=4 * C, beta=4 * C, dgamma=4 * C, dbeta=4 * C, mean=4 * G, rstd=4 * G,
                     ws=plan.workspace_bytes, wsb=plan.workspace_bytes_backward)
        self.at, o = {}, 0
        for k, n in sizes.items():
            self.at[k], o = o, o + (n + 511) // 512 * 512
        self.sizes = sizes
        self.mem = torch.zeros(o, dtype=torch.uint8, device="cuda")
        for k in ("rstd", "gamma"):
            self.mem[self.at[k]:self.at[k] + sizes[k]].view(torch.float32).fill_(1.0)
        self.base = self.mem.data_ptr()

    def __call__(self, k, moved):
        return self.base + self.at[moved.get(k, k)]


def forward(lib, plan, b, moved):
    p = lambda k: b(k, moved)  # noqa: E731
    return lib.conv_run_groupnorm(plan.handle, p("x"), 0, p("gamma"), p("beta"), p("y"), 0, p("mean"), p("rstd"), p("ws"), None)


def backward(lib, plan, b, moved):
    p = lambda k: b(k, moved)  # noqa: E731
    return lib.conv_run_groupnorm_bwd(plan.handle, p("x"), 0, p("gamma"), p("beta"), p("mean"), p("rstd"), p("dy"), 0, p("dx"), 0,
                                      p("dgamma"), p("dbeta"), p("wsb"), None)


@pytest.mark.parametrize("run,reads,writes", [
    (forward, ("x", "gamma", "beta"), ("y", "mean", "rstd", "ws")),
    (backward, ("x", "dy", "gamma", "beta", "mean", "rstd"), ("dx", "dgamma", "dbeta", "wsb")),
])
def test_nothing_written_is_shared(cl, run, reads, writes):  # noqa: F811
    lib = cl.load_library()
    plan = cl.GroupNormPlan(*SHAPE, G, dtype="bf16", act="relu")
    assert plan.workspace_bytes and plan.workspace_bytes_backward
    b = Buffers(plan)
    assert run(lib, plan, b, {}) == 0
    torch.cuda.synchronize()
    pairs = list(itertools.product(writes, reads)) + list(itertools.permutations(writes, 2))
    got = {(w, other): run(lib, plan, b, {w: other}) for w, other in pairs}
    assert all(rc == -5 for rc in got.values()), got
    shared = {(r, s): run(lib, plan, b, {r: s}) for r, s in itertools.permutations([r for r in reads if r not in ("x", "dy")], 2)
              if b.sizes[r] <= b.sizes[s]}
    assert all(rc == 0 for rc in shared.values()), shared    # inputs may
    torch.cuda.synchronize()
