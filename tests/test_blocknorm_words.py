"""Single bf16 values come as the words that hold them: what a row's copies read
lies between the map's first value and its last, and what is taken from the words
are the row's values.  The kernels' own source (Lane and Row of blocknorm.cuh) run
on the CPU, a thread after the other, over dense maps and slices at even and odd
addresses."""
import ctypes
import os
import random
import subprocess

import numpy as np
import pytest
from test_blocknorm_layout import CSRC, plan

PRELUDE = r"""
#include <stdint.h>
#include <string.h>
#include <type_traits>
#define __device__
#define __host__
#define __forceinline__ inline
struct float2 { float x, y; };
struct float4 { float x, y, z, w; };
static float2 make_float2(float x, float y) { return {x, y}; }
static float4 make_float4(float x, float y, float z, float w) { return {x, y, z, w}; }
struct Dim { unsigned x, y, z; };
static Dim threadIdx;
struct __nv_bfloat16 { uint16_t bits; };
struct BnArgs { int tpr, C; };
static float __uint_as_float(uint32_t u) { float f; memcpy(&f, &u, 4); return f; }
template <typename T, int VEC> struct Vec {
    static constexpr int kPairs = (VEC + 1) / 2;
    using Raw = uint16_t;
    static Raw pack(const float2 (&)[kPairs]) { return 0; }
    static void unpack(Raw, float2 (&)[kPairs]) {}
};
static uint8_t ring_bytes[1 << 20];
namespace tc { inline uint32_t smem_u32(const void *p) { return (uint32_t)((const uint8_t *)p - ring_bytes); } }
static uintptr_t from, to;      // the map's bytes
static int outside;
static void read_part(uint32_t dst, const void *src, int bytes) {
    const uintptr_t at = (uintptr_t)src;
    if (at < from || at + bytes > to || at % 4) ++outside;
    memset(ring_bytes + dst, 0, 4);
    memcpy(ring_bytes + dst, src, bytes);
}
template <int BYTES> void copy_async(uint32_t dst, const void *src) { read_part(dst, src, BYTES); }
static void copy_async_part(uint32_t dst, const void *src, int bytes) { read_part(dst, src, bytes); }
"""

DRIVER = r"""
// Reads outside the map, or -1 where a value is not the map's.
template <int K, bool CUT> int walk(uint16_t *map, int rows, long long pitch, int C, int tpr, int ctas) {
    using R = Row<__nv_bfloat16, 1, K, CUT>;
    from = (uintptr_t)map;
    to = (uintptr_t)(map + (rows - 1) * pitch + C);
    outside = 0;
    for (int row = 0; row < rows; ++row)
        for (int rank = 0; rank < ctas; ++rank)
            for (int t = 0; t < tpr; ++t) {
                threadIdx = {(unsigned)t, 0, 0};
                Lane<1, K> l(BnArgs{tpr, C});
                l.t += rank * R::NV * tpr;
                typename R::Slot *slot = R::ring(ring_bytes, 1);
                float2 got[R::P];
                R::zero(slot);
                const __nv_bfloat16 *at = (const __nv_bfloat16 *)map + row * pitch + l.first(0);
                // (as in the kernels)
                const bool bottom = CUT && row == rows - 1, late = CUT && row == 0 && l.t == 0;
                const int upto = bottom ? C - 1 : C, vector = (C - 1) / tpr, last_v = vector % R::NV, last_t = (C - 1) % tpr + (vector - last_v) * tpr;
                R::ask(l, at, slot, upto, late);
                if (bottom && l.t == last_t && !(late && upto == 0)) R::ask_last(at + last_v * tpr, slot + last_v * R::step);
                if (late) R::ask_first(at, slot, upto == 0);
                R::get(l, slot, R::odd(at), got);
                for (int v = 0; v < R::NV; ++v) {
                    const float one = v % 2 ? got[v / 2].y : got[v / 2].x;
                    const float want = l.on(v) ? __uint_as_float((uint32_t)map[row * pitch + l.first(v)] << 16) : 0.0f;
                    if (memcmp(&one, &want, 4)) return -1;
                }
            }
    return outside;
}
extern "C" int walk_map(uint16_t *map, int rows, long long pitch, int C, int tpr, int k, int ctas) {
    const bool cut = ((uintptr_t)map | (uintptr_t)(map + (rows - 1) * pitch + C)) & 3;
    if (cut) return k == 2 ? walk<2, true>(map, rows, pitch, C, tpr, ctas) : walk<1, true>(map, rows, pitch, C, tpr, ctas);
    return k == 2 ? walk<2, false>(map, rows, pitch, C, tpr, ctas) : walk<1, false>(map, rows, pitch, C, tpr, ctas);
}
"""


@pytest.fixture(scope="module")
def lib(tmp_path_factory):
    text = open(os.path.join(CSRC, "blocknorm.cuh")).read()
    source = text[text.index("// Where a thread stands"):text.index("// Rows of a part of a warp, of a warp")]
    tmp = tmp_path_factory.mktemp("words")
    (tmp / "words.cpp").write_text(PRELUDE + source + DRIVER)
    subprocess.run(["g++", "-std=c++17", "-O1", "-shared", "-fPIC", "-Wno-unknown-pragmas", "-o", str(tmp / "words.so"), str(tmp / "words.cpp")], check=True)
    out = ctypes.CDLL(str(tmp / "words.so"))
    out.walk_map.argtypes = [ctypes.c_void_p, ctypes.c_int, ctypes.c_int64] + [ctypes.c_int] * 4
    return out


def test_no_word_outside_the_map(lib):
    rng, cases = random.Random(5), []
    for c in (1, 2, 3, 7, 8, 31, 33, 48, 61, 255, 257, 511, 512, 513, 2049, 3001, 4097, 8191):
        for wide in (0, 1, 13, 64):
            cases += [(rows, c, wide, odd) for rows in (1, 2, 3, 6) for odd in (0, 1)]
    cases += [(rng.randint(1, 9), rng.randint(1, 600), rng.randint(0, 9), rng.randint(0, 1)) for _ in range(300)]
    bits = np.random.default_rng(6).integers(1, 1 << 15, 10 * (8192 + 64) + 64, dtype=np.uint16)
    assert bits.ctypes.data % 4 == 0
    for rows, c, wide, odd in cases:
        fwd, gated, bwd, bgate = plan(1, rows, c, 2)
        for d in (fwd, bwd):
            at = bits.ctypes.data + 2 * (2 * rng.randint(1, 8) + odd)
            assert lib.walk_map(at, rows, c + wide, c, d.tpr, d.k, d.ctas) == 0, (rows, c, wide, odd, d.__dict__)
