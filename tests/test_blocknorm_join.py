"""The join of the one-launch gradient of the norms around a block, run on the
CPU: the function's own source, thread after thread, with the cluster's barrier
and the peers' shared memory as plain C++.  Every thread arrives, waits, arrives
and waits, and reads its peers between the first wait and the second arrival,
whatever channels its CTA joins; every channel is joined once, to the sums that
the formulas give.  Over the shapes of which the plan makes one cluster, those
whose last CTAs have no channel among them."""
import ctypes
import os
import re
import subprocess

import numpy as np
import pytest
from test_blocknorm_layout import CLUSTER, CSRC, MOST, plan, shapes, up

PRELUDE = r"""
#include <math.h>
#include <stdint.h>
#include <algorithm>
#include <vector>
using std::min;
#define __device__
#define __forceinline__ inline
struct float2 { float x, y; };
struct float4 { float x, y, z, w; };
struct Dim { unsigned x, y, z; };
static Dim threadIdx, blockIdx, gridDim, blockDim;
static constexpr uint32_t kEach = 1u << 20;            // bytes of a CTA's shared memory in the emulated window
static std::vector<std::vector<float>> sums;           // of each CTA: [SUMS][Cp]
static std::vector<int> steps;                         // 1: arrives, 2: waits, 3: reads a peer's
static void cluster_arrive() { steps.push_back(1); }
static void cluster_wait() { steps.push_back(2); }
namespace tc {
inline uint32_t smem_u32(const float *p) { return (uint32_t)((const char *)p - (const char *)sums[blockIdx.x].data()); }
inline uint32_t mapa_shared(uint32_t at, uint32_t rank) { return at + rank * kEach; }
}
static float peer_value(uint32_t at) {
    if (steps.empty() || steps.back() != 3) steps.push_back(3);
    return sums.at(at / kEach).at(at % kEach / 4);
}
"""

DRIVER = r"""
// 0, or what went wrong: 1 a thread's steps, 2 a value.
extern "C" int join_all(int ranks, int threads, int S, int N, int C, const float *all, float **p, float **d) {
    BnArgs a = {};
    a.S = S; a.N = N; a.C = C; a.Cp = (C + 3) / 4 * 4;
    a.scale = p[0]; a.gate = p[1]; a.g1 = p[2]; a.b1 = p[3];
    a.dscale = d[0]; a.dgate = d[1]; a.dg1 = d[2]; a.db1 = d[3]; a.dg2 = d[4]; a.db2 = d[5];
    gridDim = {(unsigned)ranks, 1, 1};
    blockDim = {(unsigned)threads, 1, 1};
    sums.clear();
    for (int r = 0; r < ranks; ++r) sums.emplace_back(all + (size_t)r * SUMS * a.Cp, all + (size_t)(r + 1) * SUMS * a.Cp);
    for (int r = 0; r < ranks; ++r)
        for (int t = 0; t < threads; ++t) {
            blockIdx = {(unsigned)r, 0, 0};
            threadIdx = {(unsigned)t, 0, 0};
            steps.clear();
            join_cluster(a, sums[r].data());
            if (steps != std::vector<int>({1, 2, 1, 2}) && steps != std::vector<int>({1, 2, 3, 1, 2})) return 1;
        }
    return 0;
}
"""


def piece(text, start, end):
    return text[text.index(start):text.index(end)]


@pytest.fixture(scope="module")
def lib(tmp_path_factory):
    head, body = (open(os.path.join(CSRC, f)).read() for f in ("blocknorm.cuh", "k_blocknorm_bwd.cu"))
    source = piece(head, "constexpr int kMaxC", "// Where a thread stands") + piece(body, "// What the parameters' gradients of a channel", "// Eight sums over a row")
    source = re.sub(r'asm volatile\("ld\.shared::cluster\.f32 %0, \[%1\];" : "=f"\((.*?)\) : "r"\((.*?)\) : "memory"\);', r"\1 = peer_value(\2);", source)
    assert "asm" not in source and "peer_value" in source
    tmp = tmp_path_factory.mktemp("join")
    (tmp / "join.cpp").write_text(PRELUDE + source + DRIVER)
    subprocess.run(["g++", "-std=c++17", "-O1", "-shared", "-fPIC", "-Wno-unknown-pragmas", "-o", str(tmp / "join.so"), str(tmp / "join.cpp")], check=True)
    return ctypes.CDLL(str(tmp / "join.so"))


def joined(count, seed):
    """(images, CTAs an image, threads, channels) of the one-cluster plans, each once."""
    seen = set()
    for n, hw, c, es in shapes(count, seed):
        _, _, bwd, bgate = plan(n, hw, c, es)
        for d, images in ((bwd, 0), (bgate, n)):
            if d.joined:
                seen.add((images, d.S, d.threads, c))
    return sorted(seen)


NAMED = [(0, 13, 512, 40), (16, 1, 32, 8), (16, 1, 32, 40), (9, 1, 32, 32), (0, 10, 512, 8), (11, 1, 64, 100), (16, 1, 512, 24), (3, 1, 32, 2), (1, 1, 512, 1)]


def test_every_cta_waits_between_its_arrivals(lib):
    cases = joined(500, 3)
    idle = [k for k in cases if up(k[3], max(k[0], 1) * k[1]) * (max(k[0], 1) * k[1] - 1) >= k[3]]
    assert len(idle) >= 50 and len(cases) - len(idle) >= 50
    rng = np.random.default_rng(7)
    for i, (images, each, threads, c) in enumerate(NAMED + cases):
        n, ranks, cp = max(images, 1), max(images, 1) * each, up(c, 4) * 4
        assert ranks <= CLUSTER and threads <= MOST
        f = ctypes.POINTER(ctypes.c_float)
        all_sums = rng.standard_normal((ranks, 4, cp)).astype(np.float32)
        scale, g1, b1 = (rng.standard_normal(c).astype(np.float32) if (i + j) % 3 else None for j in range(3))
        gate = rng.standard_normal((n, c)).astype(np.float32) if images else None
        given = [scale, gate, g1, b1]
        out = [np.full(s, np.nan, np.float32) for s in ((c,), (n, c), (c,), (c,), (c,), (c,))]
        if not images:
            out[1] = None
        p, d = (((f * len(v))(*(None if t is None else t.ctypes.data_as(f) for t in v))) for v in (given, out))
        assert lib.join_all(ranks, threads, each, n, c, all_sums.ctypes.data_as(f), p, d) == 0, (images, each, threads, c)
        one = np.ones(c)
        s, k, g, b = (o if t is None else t.astype(np.float64) for t, o in zip(given, (one, np.ones((n, c)), one, 0 * one)))
        A, B, G2, B2 = all_sums.astype(np.float64)[:, :, :c].reshape(n, each, 4, c).sum(1).transpose(1, 0, 2)
        gate_sum = lambda v: (k * v).sum(0)  # noqa: E731
        want = [gate_sum(g * A + b * B), s * (g * A + b * B), s * gate_sum(A), s * gate_sum(B), G2.sum(0), B2.sum(0)]
        # (sixteen sums of a few units in fp32, and products of three: within 2^-14)
        for got, ref in zip(out, want):
            if got is not None:
                assert np.abs(got - ref).max() <= 2.0 ** -14 * (1 + np.abs(ref).max()), (images, each, threads, c)
