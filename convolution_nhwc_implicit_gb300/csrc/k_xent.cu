// Loss of a class head: softmax cross entropy of the class scores
// l = x w^T over many classes, and its gradient, the scores never stored.
//
//   lse_i = log sum_v exp l_iv          loss = sum_{labelled i} (lse_i - l_{i,t_i}) / count
//   g_iv = (exp(l_iv - lse_i) - [v = t_i]) for labelled rows, 0 for the others
//   dx = (dloss / count) g w            dw = (dloss / count) g^T x
//
// x [N][D] and w [V][D] bf16.  Forward 2NDV operations; the gradient 4NDV and
// 2NDV to form the scores again: the tensor cores bound it, and the bytes of w
// where rows are few.  Three tcgen05 kernels on one tile machine:
//
//   FWD   scores of a 256 x 256 tile in TMEM; each row's running maximum and
//         sum of exponentials over 128 columns go out as one (m, s) pair, and
//         a small kernel joins the pairs of a row (xent_join_kernel).
//   GRAD  the same scores for a piece of the classes; g, rounded to bf16, goes
//         to a [N][piece] workspace.
//   PROD  both products with that workspace in one launch: dx += g w_piece
//         (K = classes; fp32 partial sums between pieces) and the piece's rows
//         of dw = g^T x (K = rows).
//
// Roundings: scores, statistics and both products accumulate in fp32; g alone
// is rounded to bf16 between the products (at most 2^-8 of an element, what the
// results' own rounding costs), unscaled, so that the -1 of a label whose
// probability is small stays exact; dloss / count multiplies the fp32 sums.
// Nothing depends on the order of atomics: results repeat bit for bit.
//
// Measured on a GB300: 8192 x 1024 x 65536 with the gradient 2.5 to 2.8 ms (the
// longer in calls back to back, by the clock that the power limit leaves), 1580 to 1770
// TFLOP/s of the 8NDV that it does, 82 to 91 % of the measured burst rate; 1600 x 1024 x 32003, loss alone, 73 to 74 us, 1410
// to 1440 TFLOP/s (tensor pipe 81 % busy; its 882 tiles fill 11.6 waves of pairs, and
// the last of seven row tiles is a quarter full); 20 x 512 x 1000 with the
// gradient 25.6 us, four launches of a few K blocks each.
//
// The tile machine: a cluster of two CTAs (two SMs) computes 256 x 256 outputs
// with tcgen05.mma.cta_group::2, each CTA staging 128 rows of A and 128 of B
// per K block of 64 (32 KB a stage, six stages) and holding 128 rows of the
// accumulator, double-buffered in TMEM (2 x 256 columns).  One CTA alone with a
// 128 x 256 tile would draw 94 B a cycle from L2 at the tensor core's rate (27
// TB/s over the card, more than L2 gives); the pair draws 62.  Operands whose
// K axis is the outer one in memory (w in dx, both in dw) are staged as they
// lie, MN-major, so nothing is transposed.  Warp 0 issues the TMA loads, warp 1
// of the even CTA the MMAs, warps 2..9 drain: two warpgroups of 128 columns.
#include <cuda.h>
#include <cudaTypedefs.h>
#include <cuda_bf16.h>
#include <math.h>
#include <stdint.h>
#include <stdio.h>

#include <mutex>
#include <new>

#include "conv_internal.h"
#include "epilogue.cuh"
#include "tc_ptx.cuh"

using namespace convk;

namespace {

constexpr int kTile = 256;          // rows and columns of a tile (both CTAs)
constexpr int kBK = 64;             // K block: one 128-byte swizzle row of bf16
constexpr int kStages = 6;
constexpr uint32_t kHalf = 128 * kBK * 2;      // A or B bytes of a stage (this CTA's)
constexpr uint32_t kStage = 2 * kHalf;
constexpr uint32_t kBox = 32 * 128;            // staging of one warp: 32 rows x 64 bf16
constexpr uint32_t kSmem = 1024 + kStages * kStage + 8 * kBox + 256;
constexpr int kThreads = 320;
// K blocks of a run worth the launch that joins runs (3 us, ten blocks' time).
constexpr int kMinRun = 16;
constexpr int kGroupM = 32;         // tile rows walked before the next tile column
constexpr float kLog2e = 1.4426950408889634f;
static_assert(kSmem <= 232448, "shared memory of a CTA");

enum { FWD = 0, GRAD = 1, PROD = 2 };

struct XArgs {
    int rows, classes, d;        // N, V (of the piece in GRAD and PROD), D
    int tiles_m, tiles_n, tiles; // FWD / GRAD: row and class tiles
    int kblocks;                 // FWD / GRAD: ceil(D / 64)
    int v0, all_classes;         // first class of the piece; V
    const int *target;
    const float *lse;            // GRAD
    float2 *part;                // FWD: [2 tiles_n][rows] (max, sum of exponentials)
    float *tlogit;               // FWD: [rows], the label's score
    unsigned *counter;           // FWD clears it for the joining kernel
    const float *dloss;          // GRAD of the first piece: may be null (1)
    int first;                   // first piece: GRAD forms the scale, PROD does not read partial sums
    float *scale;                // dloss / count
    // PROD: dx tiles (K = classes, split in dx_split runs of dx_kper blocks),
    // dw tiles (K = rows, likewise); the longer kind first
    int dx_tiles, dx_tm, dx_tn, dx_kb, dx_split, dx_kper, dx_final;
    int dw_tiles, dw_tm, dw_tn, dw_kb, dw_split, dw_kper, dw_final;
    int dw_first;
    float *dx_part, *dw_part;    // fp32 partial sums, a tile's own layout
    __nv_bfloat16 *dx, *dw;
    int tma_out;                 // dx and dw rows allow TMA stores
    int *status;
};

struct Maps {
    CUtensorMap a, b, out;       // FWD / GRAD: x, w, g (store); PROD dx: g, w, dx
    CUtensorMap a2, b2, out2;    // PROD dw: g, x, dw
};

// Waits for phase `parity` of `bar`; gives up after kWaitBudgetNs or when
// another role of the CTA has, and says so in the status word.
template <bool CLUSTER = false>
__device__ __forceinline__ bool wait_bounded(uint32_t bar, uint32_t parity, volatile int *abort_flag, int *status, int code) {
    auto poll = [&]() { return CLUSTER ? tc::mbar_try_wait_cluster(bar, parity) : tc::mbar_try_wait(bar, parity); };
    if (poll()) return true;
    const unsigned long long t0 = globaltimer_ns();
    for (uint32_t i = 1;; ++i) {
        if (poll()) return true;
        if ((i & 63u) == 0u) {
            if (*abort_flag) return false;
            if (globaltimer_ns() - t0 > kWaitBudgetNs) {
                *abort_flag = 1;
                atomicExch(status, code);
                return false;
            }
        }
    }
}

// Descriptor of an MN-major operand: 128-byte rows of 64 elements along M (or
// N), one row per k, as TMA lays a [64 k][64 mn] box with the 128-byte swizzle.
// Stride byte offset: from eight k to the next eight (1024); leading byte
// offset: from 64 elements to the next 64 (the next box).
__device__ __forceinline__ uint64_t smem_desc_mnmajor(uint32_t saddr) {
    uint64_t d = 0;
    d |= (uint64_t)((saddr & 0x3FFFFu) >> 4);
    d |= (uint64_t)((64u * 128u) >> 4) << 16;
    d |= (uint64_t)(1024u >> 4) << 32;
    d |= (uint64_t)1u << 46;
    d |= (uint64_t)2u << 61;
    return d;
}

__device__ __forceinline__ float ex2(float v) {
    float r;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(v));
    return r;
}
// e^(l - v) is 2^(l log2 e - v log2 e).  With ref, v log2 e rounded (__fmul_rn,
// which no multiply-add absorbs), in the multiply-add of every l, what is left
// over is this factor of all of them: without it they are off by ref's rounding,
// which grows with |v| (1e-5 of the result at 200).  (v infinite or NaN: 1, ref
// says it.)
__device__ __forceinline__ float exp2_rest(float v, float ref) {
    return fabsf(v) < INFINITY ? ex2(-fmaf(v, kLog2e, -ref)) : 1.0f;
}
__device__ __forceinline__ uint32_t bf16_pair(float a, float b) {
    __nv_bfloat162 p = __floats2bfloat162_rn(a, b);
    return *reinterpret_cast<uint32_t *>(&p);
}

// What one tile is: its kind, place and K blocks.
struct TileAt {
    bool dw;         // PROD: a tile of dw (else of dx; FWD / GRAD: scores)
    int mi, ni, ks, kb0, kb1;
};
template <int KIND>
__device__ __forceinline__ TileAt tile_at(const XArgs &a, int tile) {
    TileAt t;
    t.ks = 0;
    if constexpr (KIND == PROD) {
        const int head = a.dw_first ? a.dw_tiles : a.dx_tiles;
        t.dw = (tile < head) == (a.dw_first != 0);
        int i = tile < head ? tile : tile - head;
        const int tn = t.dw ? a.dw_tn : a.dx_tn, tm = t.dw ? a.dw_tm : a.dx_tm;
        const int kper = t.dw ? a.dw_kper : a.dx_kper, kb = t.dw ? a.dw_kb : a.dx_kb;
        t.ni = i % tn;
        i /= tn;
        t.mi = i % tm;
        t.ks = i / tm;
        t.kb0 = t.ks * kper;
        t.kb1 = min(kb, t.kb0 + kper);
    } else {
        t.dw = false;
        const int per = kGroupM * a.tiles_n;
        const int grp = tile / per, first = grp * kGroupM;
        const int m = min(kGroupM, a.tiles_m - first), r = tile - grp * per;
        t.mi = first + r % m;
        t.ni = r / m;
        t.kb0 = 0;
        t.kb1 = a.kblocks;
    }
    return t;
}

template <int KIND>
__global__ void __launch_bounds__(kThreads, 1) xent_kernel(const __grid_constant__ Maps maps, const __grid_constant__ XArgs a) {
    extern __shared__ uint8_t smem_raw[];
    const uint32_t raw = tc::smem_u32(smem_raw);
    const uint32_t base = (raw + 1023u) & ~1023u;
    uint8_t *gbase = smem_raw + (base - raw);
    const uint32_t sOut = base + kStages * kStage;
    const uint32_t sBar = sOut + 8 * kBox;
    auto full_bar = [&](int s) { return sBar + 8u * s; };
    auto empty_bar = [&](int s) { return sBar + 8u * (kStages + s); };
    auto tfull_bar = [&](int b) { return sBar + 8u * (2 * kStages + b); };
    auto tempty_bar = [&](int b) { return sBar + 8u * (2 * kStages + 2 + b); };
    uint8_t *gmisc = gbase + (sBar - base) + 8u * (2 * kStages + 4);
    volatile uint32_t *tmem_holder = reinterpret_cast<volatile uint32_t *>(gmisc);
    volatile int *abort_flag = reinterpret_cast<volatile int *>(gmisc + 4);
    int *counts = reinterpret_cast<int *>(gmisc + 8);  // [8], one an epilogue warp

    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const uint32_t rank = tc::cluster_ctarank();
    const int unit = (int)(blockIdx.x >> 1), units = (int)(gridDim.x >> 1);

    if (threadIdx.x == 0) {
        for (int s = 0; s < kStages; ++s) {
            tc::mbar_init(full_bar(s), 1);
            tc::mbar_init(empty_bar(s), 1);
        }
        for (int b = 0; b < 2; ++b) {
            tc::mbar_init(tfull_bar(b), 1);
            tc::mbar_init(tempty_bar(b), 2 * 8);  // every epilogue warp of both CTAs
        }
        *abort_flag = 0;
        tc::fence_mbar_init();
        tc::tma_prefetch_desc(&maps.a);
        tc::tma_prefetch_desc(&maps.b);
        if (KIND != FWD) tc::tma_prefetch_desc(&maps.out);
        if (KIND == PROD) {
            tc::tma_prefetch_desc(&maps.a2);
            tc::tma_prefetch_desc(&maps.b2);
            tc::tma_prefetch_desc(&maps.out2);
        }
    }
    if (warp == 1) {
        tc::tmem_alloc_pair(tc::smem_u32((const void *)tmem_holder), 512);
        tc::tmem_relinquish_pair();
    }
    __syncwarp();
    tc::fence_before_sync();
    __syncthreads();
    tc::cluster_sync();  // the peer's barriers are initialised
    tc::fence_after_sync();
    const uint32_t tmem_base = *tmem_holder;
    pdl_trigger();
    pdl_wait();

    if (warp == 0) {
        // ------------------------------------------------ TMA producer
        if (lane == 0) {
            int stage = 0;
            uint32_t phase = 0;
            bool ok = true;
            const uint32_t full0 = tc::mapa_shared(full_bar(0), 0);
            for (int tile = unit; tile < a.tiles && ok; tile += units) {
                const TileAt t = tile_at<KIND>(a, tile);
                const int m0 = t.mi * kTile + (int)rank * 128, n0 = t.ni * kTile + (int)rank * 128;
                for (int kb = t.kb0; kb < t.kb1; ++kb) {
                    if (!wait_bounded(empty_bar(stage), phase ^ 1u, abort_flag, a.status, KSTATUS_TIMEOUT_PRODUCER)) {
                        ok = false;
                        break;
                    }
                    const uint32_t dA = base + stage * kStage, dB = dA + kHalf, fb = full0 + 8u * stage;
                    if (rank == 0) tc::mbar_arrive_expect_tx(full_bar(stage), 2u * kStage);
                    const int k0 = kb * kBK;
                    if (KIND != PROD) {
                        tc::tma_load_2d_pair(dA, &maps.a, fb, k0, m0);
                        tc::tma_load_2d_pair(dB, &maps.b, fb, k0, n0);
                    } else if (t.dw) {
                        tc::tma_load_2d_pair(dA, &maps.a2, fb, m0, k0);
                        tc::tma_load_2d_pair(dA + kHalf / 2, &maps.a2, fb, m0 + 64, k0);
                        tc::tma_load_2d_pair(dB, &maps.b2, fb, n0, k0);
                        tc::tma_load_2d_pair(dB + kHalf / 2, &maps.b2, fb, n0 + 64, k0);
                    } else {
                        tc::tma_load_2d_pair(dA, &maps.a, fb, k0, m0);
                        tc::tma_load_2d_pair(dB, &maps.b, fb, n0, k0);
                        tc::tma_load_2d_pair(dB + kHalf / 2, &maps.b, fb, n0 + 64, k0);
                    }
                    if (++stage == kStages) { stage = 0; phase ^= 1u; }
                }
            }
        }
    } else if (warp == 1) {
        // ------------------------------------------------ MMA issuer (even CTA)
        if (lane == 0 && rank == 0) {
            int stage = 0, lt = 0;
            uint32_t phase = 0;
            bool ok = true;
            for (int tile = unit; tile < a.tiles && ok; tile += units, ++lt) {
                const TileAt t = tile_at<KIND>(a, tile);
                const int buf = lt & 1;
                if (!wait_bounded<true>(tempty_bar(buf), ((uint32_t)(lt >> 1) & 1u) ^ 1u, abort_flag, a.status,
                                        KSTATUS_TIMEOUT_MMA))
                    break;
                tc::fence_after_sync();
                const uint32_t d = tmem_base + (uint32_t)(buf * kTile);
                constexpr uint32_t kIdesc = tc::idesc_bf16_f32(256, 256);
                const bool mnA = KIND == PROD && t.dw, mnB = KIND == PROD;
                const uint32_t idesc = kIdesc | (mnA ? 1u << 15 : 0u) | (mnB ? 1u << 16 : 0u);
                const uint32_t stepA = mnA ? (16u * 128u) >> 4 : 32u >> 4, stepB = mnB ? (16u * 128u) >> 4 : 32u >> 4;
                for (int kb = t.kb0; kb < t.kb1; ++kb) {
                    const uint32_t sA = base + stage * kStage, sB = sA + kHalf;
                    const uint64_t da = mnA ? smem_desc_mnmajor(sA) : tc::smem_desc_kmajor(sA, 128);
                    const uint64_t db = mnB ? smem_desc_mnmajor(sB) : tc::smem_desc_kmajor(sB, 128);
                    if (!wait_bounded(full_bar(stage), phase, abort_flag, a.status, KSTATUS_TIMEOUT_MMA)) {
                        ok = false;
                        break;
                    }
                    tc::fence_after_sync();
#pragma unroll
                    for (int k = 0; k < kBK / 16; ++k)
                        tc::mma_bf16_pair(d, da + (uint64_t)(k * stepA), db + (uint64_t)(k * stepB), idesc,
                                          (kb != t.kb0 || k != 0) ? 1u : 0u);
                    tc::mma_commit_pair(empty_bar(stage), 0x3);
                    if (++stage == kStages) { stage = 0; phase ^= 1u; }
                }
                if (ok) tc::mma_commit_pair(tfull_bar(buf), 0x3);
            }
        }
    } else {
        // ------------------------------------------------ epilogue warps 2..9
        const int ew = warp - 2, grp = ew >> 2, q = warp & 3;  // q: the TMEM lanes this warp may read
        const uint32_t tempty0 = tc::mapa_shared(tempty_bar(0), 0);
        const uint32_t sBox = sOut + (uint32_t)ew * kBox;
        uint8_t *gBox = gbase + (sBox - base);
        const int myrow = (int)rank * 128 + q * 32 + lane;     // row inside a tile
        if (KIND == FWD && blockIdx.x == 0 && threadIdx.x == 64) *a.counter = 0u;
        if (KIND == GRAD && a.first && blockIdx.x == 0) {
            // labelled rows, for the mean
            int c = 0;
            for (int i = (int)threadIdx.x - 64; i < a.rows; i += 256) {
                const int tg = a.target[i];
                c += tg >= 0 && tg < a.all_classes ? 1 : 0;
            }
            c = __reduce_add_sync(0xffffffffu, c);
            if (lane == 0) counts[ew] = c;
            tc::named_bar_sync(1, 256);
            if (threadIdx.x == 64) {
                int n = 0;
                for (int i = 0; i < 8; ++i) n += counts[i];
                *a.scale = (a.dloss ? *a.dloss : 1.0f) / (float)max(n, 1);
            }
        }
        const float scale = KIND == PROD ? *a.scale : 0.0f;
        int lt = 0;
        for (int tile = unit; tile < a.tiles; tile += units, ++lt) {
            const TileAt t = tile_at<KIND>(a, tile);
            const int buf = lt & 1;
            const int row = t.mi * kTile + myrow;              // of x / g / dx, or class of dw
            const int col0 = t.ni * kTile + grp * 128;
            // what the rows bring, read before the wait
            int tg = -1;        // the row's label inside the piece (negative or past it: none)
            bool on = false;    // a labelled row
            float ls = 0.0f;
            if (KIND != PROD && row < a.rows) {
                const int label = a.target[row];
                on = label >= 0 && label < a.all_classes;
                if (on) tg = label - a.v0;
                if (KIND == GRAD) ls = a.lse[row];
            }
            const bool got = wait_bounded(tfull_bar(buf), (uint32_t)(lt >> 1) & 1u, abort_flag, a.status, KSTATUS_TIMEOUT_EPILOGUE);
            __syncwarp();
            if (!__all_sync(0xffffffffu, got)) break;
            tc::fence_after_sync();
            const uint32_t tacc = tmem_base + ((uint32_t)(q * 32) << 16) + (uint32_t)(buf * kTile + grp * 128);
            auto release = [&]() {
                tc::fence_before_sync();
                __syncwarp();
                if (lane == 0) tc::mbar_arrive_cluster(tempty0 + 8u * buf);
            };
            if constexpr (KIND == FWD) {
                // s: sum of 2^(l log2 e - ref), ref the rounded m log2 e
                float m = -INFINITY, s = 0.0f, ref = -INFINITY;
#pragma unroll 1
                for (int c = 0; c < 128; c += 32) {
                    uint32_t r[32];
                    tc::tmem_ld_32x32(tacc + (uint32_t)c, r);
                    tc::tmem_ld_wait();
                    if (c == 96) release();
                    const int left = a.classes - (col0 + c);   // columns of the chunk that are classes
                    if (left <= 0) continue;
                    if (left < 32) {
#pragma unroll
                        for (int j = 0; j < 32; ++j)
                            if (j >= left) r[j] = 0xff800000u;
                    }
                    float top = __uint_as_float(r[0]);
#pragma unroll
                    for (int j = 1; j < 32; ++j) top = fmaxf(top, __uint_as_float(r[j]));
                    const float nm = fmaxf(m, top);
                    const float use = nm == -INFINITY ? 0.0f : __fmul_rn(nm, kLog2e);
                    float s0 = s * ex2(ref - use), s1 = 0.0f, s2 = 0.0f, s3 = 0.0f;
#pragma unroll
                    for (int j = 0; j < 32; j += 4) {
                        s0 += ex2(fmaf(__uint_as_float(r[j]), kLog2e, -use));
                        s1 += ex2(fmaf(__uint_as_float(r[j + 1]), kLog2e, -use));
                        s2 += ex2(fmaf(__uint_as_float(r[j + 2]), kLog2e, -use));
                        s3 += ex2(fmaf(__uint_as_float(r[j + 3]), kLog2e, -use));
                    }
                    s = (s0 + s1) + (s2 + s3);
                    m = nm;
                    ref = __fmul_rn(nm, kLog2e);
                    const int at = tg - (col0 + c);
                    if (on && at >= 0 && at < 32) {
                        float v = 0.0f;
#pragma unroll
                        for (int j = 0; j < 32; ++j) v = j == at ? __uint_as_float(r[j]) : v;
                        a.tlogit[row] = v;
                    }
                }
                s *= exp2_rest(m, ref);
                if (row < a.rows) a.part[(long long)(t.ni * 2 + grp) * a.rows + row] = make_float2(m, s);
            } else {
                const float ref = __fmul_rn(ls, kLog2e), rest = exp2_rest(ls, ref);
                const bool fin = KIND == PROD && (t.dw ? a.dw_final : a.dx_final) != 0;
                float *slot = nullptr;
                bool add = false;
                if constexpr (KIND == PROD) {
                    const int tm = t.dw ? a.dw_tm : a.dx_tm, tn = t.dw ? a.dw_tn : a.dx_tn;
                    const long long at = ((((long long)(t.ks * tm + t.mi) * tn + t.ni) * 2 + rank) * 2 + grp) * 4 + q;
                    slot = (t.dw ? a.dw_part : a.dx_part) + at * 4096 + lane;
                    add = !t.dw && !a.first;
                }
                const int rows_out = KIND == PROD && t.dw ? a.classes : a.rows;
                const int cols_out = KIND == PROD ? a.d : a.classes;
                const int wrow = t.mi * kTile + (int)rank * 128 + q * 32;  // the warp's first row
#pragma unroll 1
                for (int c = 0; c < 128; c += 64) {
                    uint32_t r[64];
                    tc::tmem_ld_32x32(tacc + (uint32_t)c, *reinterpret_cast<uint32_t(*)[32]>(r));
                    tc::tmem_ld_32x32(tacc + (uint32_t)c + 32u, *reinterpret_cast<uint32_t(*)[32]>(r + 32));
                    tc::tmem_ld_wait();
                    if (c == 64) release();
                    if constexpr (KIND == GRAD) {
#pragma unroll
                        for (int j = 0; j < 64; ++j) {
                            const float p = ex2(fmaf(__uint_as_float(r[j]), kLog2e, -ref)) * rest;
                            r[j] = __float_as_uint(on ? p : 0.0f);
                        }
                        const int at = tg - (col0 + c);
                        if (on && at >= 0 && at < 64) {  // (few lanes: classes are many)
#pragma unroll
                            for (int j = 0; j < 64; ++j)
                                if (j == at) r[j] = __float_as_uint(__uint_as_float(r[j]) - 1.0f);
                        }
                    } else {
                        if (add) {
#pragma unroll
                            for (int j = 0; j < 64; ++j) r[j] = __float_as_uint(__uint_as_float(r[j]) + slot[(c + j) * 32]);
                        }
                        if (!fin) {
#pragma unroll
                            for (int j = 0; j < 64; ++j) slot[(c + j) * 32] = __uint_as_float(r[j]);
                            continue;
                        }
#pragma unroll
                        for (int j = 0; j < 64; ++j) r[j] = __float_as_uint(__uint_as_float(r[j]) * scale);
                    }
                    // bf16, 32 rows x 64 columns, the 128-byte swizzle of the store's map
                    if (lane == 0) tc::bulk_wait_read0();  // the previous box has left
                    __syncwarp();
#pragma unroll
                    for (int j = 0; j < 8; ++j) {
                        uint32_t o[4];
#pragma unroll
                        for (int e = 0; e < 4; ++e)
                            o[e] = bf16_pair(__uint_as_float(r[j * 8 + 2 * e]), __uint_as_float(r[j * 8 + 2 * e + 1]));
                        const uint32_t d = sBox + (uint32_t)lane * 128u + (uint32_t)((j ^ (lane & 7)) << 4);
                        asm volatile("st.shared.v4.b32 [%0], {%1, %2, %3, %4};" ::"r"(d), "r"(o[0]), "r"(o[1]), "r"(o[2]), "r"(o[3])
                                     : "memory");
                    }
                    const int oc = col0 + c;
                    if (KIND == GRAD || a.tma_out) {
                        tc::fence_proxy_async_smem();
                        __syncwarp();
                        if (lane == 0 && wrow < rows_out && oc < cols_out) {
                            tc::tma_store_2d(KIND == PROD && t.dw ? &maps.out2 : &maps.out, sBox, oc, wrow);
                            tc::bulk_commit();
                        }
                    } else {
                        // rows that TMA cannot address: each row's 64 columns by the warp
                        __syncwarp();
                        __nv_bfloat16 *out = t.dw ? a.dw + (long long)a.v0 * a.d : a.dx;
                        const int nr = min(32, rows_out - wrow);
                        for (int i = 0; i < nr; ++i)
                            for (int j = lane; j < 64 && oc + j < cols_out; j += 32)
                                out[(long long)(wrow + i) * a.d + oc + j] = *reinterpret_cast<const __nv_bfloat16 *>(
                                    gBox + i * 128 + (((j >> 3) ^ (i & 7)) << 4) + (j & 7) * 2);
                        __syncwarp();
                    }
                }
            }
        }
        if (KIND != FWD && lane == 0) tc::bulk_wait0();  // the stores have landed
    }

    __syncwarp();
    tc::fence_before_sync();
    __syncthreads();
    tc::cluster_sync();  // neither CTA leaves while the other may use its memory
    if (warp == 1) {
        tc::fence_after_sync();
        tc::tmem_dealloc_pair(tmem_base, 512);
    }
}

// (max, sum) pairs of a row joined into lse, the row's loss, and (the last
// block, in a fixed order) the mean over the labelled rows.  32 rows a block.
__global__ void __launch_bounds__(256) xent_join_kernel(const float2 *part, int pairs, int rows, int classes, const int *target,
                                                        const float *tlogit, float *lse, float *row_loss, float *loss,
                                                        unsigned *counter) {
    __shared__ float sm[8][32], ss[8][32];
    __shared__ bool last;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int row = blockIdx.x * 32 + lane;
    pdl_trigger();
    pdl_wait();
    float m = -INFINITY, s = 0.0f;
    auto join = [&](float m2, float s2) {
        const float nm = fmaxf(m, m2);
        if (nm == -INFINITY) { s += s2; return; }  // (NaN sums stay NaN)
        s = s * ex2((m - nm) * kLog2e) + s2 * ex2((m2 - nm) * kLog2e);
        m = nm;
    };
    if (row < rows)
        for (int j = warp; j < pairs; j += 64) {  // eight pairs on their way together
            float2 v[8];
#pragma unroll
            for (int u = 0; u < 8; ++u)
                v[u] = j + 8 * u < pairs ? part[(long long)(j + 8 * u) * rows + row] : make_float2(-INFINITY, 0.0f);
#pragma unroll
            for (int u = 0; u < 8; ++u) join(v[u].x, v[u].y);
        }
    sm[warp][lane] = m;
    ss[warp][lane] = s;
    __syncthreads();
    if (warp == 0 && row < rows) {
        for (int w = 1; w < 8; ++w) join(sm[w][lane], ss[w][lane]);
        const float l = m + logf(s);
        const int t = target[row];
        lse[row] = l;
        row_loss[row] = t >= 0 && t < classes ? l - tlogit[row] : 0.0f;
    }
    __threadfence();
    __syncthreads();
    if (threadIdx.x == 0) last = atomicAdd(counter, 1u) == gridDim.x - 1;
    __syncthreads();
    if (!last) return;
    __threadfence();
    float sum = 0.0f;
    int count = 0;
    for (int i = threadIdx.x; i < rows; i += 256) {
        const int t = target[i];
        if (t >= 0 && t < classes) {
            sum += __ldcg(row_loss + i);
            ++count;
        }
    }
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) {
        sum += __shfl_xor_sync(0xffffffffu, sum, o);
        count += __shfl_xor_sync(0xffffffffu, count, o);
    }
    if (lane == 0) {
        sm[0][warp] = sum;
        ss[0][warp] = __int_as_float(count);
    }
    __syncthreads();
    if (threadIdx.x == 0) {
        sum = 0.0f;
        count = 0;
        for (int w = 0; w < 8; ++w) {
            sum += sm[0][w];
            count += __float_as_int(ss[0][w]);
        }
        *loss = sum / (float)max(count, 1);
    }
}

// Sum of a product's K runs: one warp's 32 rows x 128 columns a block of 256.
__global__ void __launch_bounds__(256) xent_finish_kernel(const float *part, int splits, int tm, int tn, int rows, int cols,
                                                          const float *scale, __nv_bfloat16 *out) {
    __shared__ float t[128][33];
    pdl_trigger();
    pdl_wait();
    const int i = blockIdx.x;  // (mi, ni, rank, grp, q)
    const int q = i & 3, grp = (i >> 2) & 1, rank = (i >> 3) & 1, ni = (i >> 4) % tn, mi = (i >> 4) / tn;
    const int r0 = mi * kTile + rank * 128 + q * 32, c0 = ni * kTile + grp * 128;
    if (r0 >= rows || c0 >= cols) return;
    const float sc = *scale;
    const long long step = (long long)tm * tn * 16 * 4096;
    const float *p = part + (long long)i * 4096;
    for (int e = threadIdx.x; e < 4096; e += 256) {
        float v = 0.0f;
        for (int k = 0; k < splits; ++k) v += p[k * step + e];
        t[e >> 5][e & 31] = v * sc;
    }
    __syncthreads();
    for (int e = threadIdx.x; e < 4096; e += 256) {
        const int r = e >> 7, c = e & 127;
        if (r0 + r < rows && c0 + c < cols) out[(long long)(r0 + r) * cols + c0 + c] = __float2bfloat16_rn(t[c][r]);
    }
}

// The rows of x and w, d values each, copied to rows of dp >= d, the rest
// zeros (rows whose length is not a multiple of eight cannot be addressed by
// TMA).  Eight values of a row a thread.
__global__ void __launch_bounds__(256) xent_pad_kernel(const __nv_bfloat16 *x, __nv_bfloat16 *xp, int rows, const __nv_bfloat16 *w,
                                                       __nv_bfloat16 *wp, int classes, int d, int dp) {
    pdl_trigger();
    pdl_wait();
    const int eights = dp / 8;
    const long long total = ((long long)rows + classes) * eights;
    for (long long i = (long long)blockIdx.x * 256 + threadIdx.x; i < total; i += (long long)gridDim.x * 256) {
        const long long r = i / eights;
        const int c = (int)(i - r * eights) * 8;
        const __nv_bfloat16 *src = r < rows ? x + r * d : w + (r - rows) * d;
        __nv_bfloat16 *dst = r < rows ? xp + r * dp : wp + (r - rows) * dp;
        uint32_t v[4] = {0u, 0u, 0u, 0u};
#pragma unroll
        for (int e = 0; e < 8; ++e)
            if (c + e < d) v[e / 2] |= (uint32_t)__bfloat16_as_ushort(src[c + e]) << (16 * (e & 1));
        *reinterpret_cast<uint4 *>(dst + c) = make_uint4(v[0], v[1], v[2], v[3]);
    }
}

// ------------------------------------------------------------------ host side
PFN_cuTensorMapEncodeTiled_v12000 encoder() {
    static PFN_cuTensorMapEncodeTiled_v12000 fn = nullptr;
    static std::once_flag once;
    std::call_once(once, [] {
        void *ptr = nullptr;
        cudaDriverEntryPointQueryResult qr;
        if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &ptr, 12000, cudaEnableDefault, &qr) == cudaSuccess &&
            qr == cudaDriverEntryPointSuccess)
            fn = reinterpret_cast<PFN_cuTensorMapEncodeTiled_v12000>(ptr);
    });
    return fn;
}

// A [rows][cols] bf16 matrix, rows `pitch` elements apart, in boxes of 64
// columns (128 bytes, swizzled) and box_rows rows; zeros outside it.
bool make_map(CUtensorMap *m, const void *p, long long cols, long long rows, long long pitch, int box_rows) {
    const cuuint64_t dims[2] = {(cuuint64_t)cols, (cuuint64_t)rows};
    const cuuint64_t strides[1] = {(cuuint64_t)pitch * 2};
    const cuuint32_t box[2] = {64, (cuuint32_t)box_rows}, ones[2] = {1, 1};
    return encoder()(m, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 2, const_cast<void *>(p), dims, strides, box, ones,
                     CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                     CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

size_t up256(size_t v) { return (v + 255) & ~(size_t)255; }
int ceil_div(long long a, long long b) { return (int)((a + b - 1) / b); }

// Workspace of a run, in order.
struct Space {
    size_t xp, wp, part, tlogit, row_loss, lse, counter, scale, g, dxp, dwp, fwd, bwd;
};
Space space_of(const conv_plan *p) {
    const XentGeom &g = p->xent;
    const long long N = p->s.n, V = p->s.c_out, D = p->s.c_in;
    Space s;
    size_t o = 0;
    auto take = [&](size_t &at, size_t bytes) { at = o; o += up256(bytes); };
    take(s.xp, g.dp != D ? (size_t)N * g.dp * 2 : 0);
    take(s.wp, g.dp != D ? (size_t)V * g.dp * 2 : 0);
    take(s.scale, 4);
    take(s.counter, 4);
    const size_t common = o;
    // forward
    take(s.part, (size_t)2 * g.tiles_n * N * 8);
    take(s.tlogit, (size_t)N * 4);
    take(s.row_loss, (size_t)N * 4);
    take(s.lse, (size_t)N * 4);
    s.fwd = o;
    // gradient
    o = common;
    take(s.g, (size_t)N * g.piece * 2);
    take(s.dxp, (g.pieces > 1 || g.dx_split > 1) ? (size_t)g.dx_split * g.tiles_m * g.tiles_d * kTile * kTile * 4 : 0);
    take(s.dwp, g.dw_split > 1 ? (size_t)g.dw_split * ceil_div(g.piece, kTile) * g.tiles_d * kTile * kTile * 4 : 0);
    s.bwd = o;
    return s;
}

const void *kernel_of(int kind) {
    return kind == FWD ? (const void *)&xent_kernel<FWD> : (kind == GRAD ? (const void *)&xent_kernel<GRAD> : (const void *)&xent_kernel<PROD>);
}

cudaError_t launch_tiles(const conv_plan *p, int kind, Maps &maps, XArgs &a, cudaStream_t st) {
    const int pairs = p->num_sms / 2;
    const int grid = 2 * (a.tiles < pairs ? a.tiles : pairs);
    void *args[] = {&maps, &a};
    return conv_launch(kernel_of(kind), dim3((unsigned)grid), dim3(kThreads), args, kSmem, st, 2);
}

// Operands as TMA can address them: as given, or padded copies.
int operands(const conv_plan *p, const Space &sp, char *ws, const void *&x, const void *&w, cudaStream_t st) {
    if (p->xent.dp == p->s.c_in) return CONV_OK;
    const __nv_bfloat16 *xs = static_cast<const __nv_bfloat16 *>(x), *wsrc = static_cast<const __nv_bfloat16 *>(w);
    __nv_bfloat16 *xp = reinterpret_cast<__nv_bfloat16 *>(ws + sp.xp), *wp = reinterpret_cast<__nv_bfloat16 *>(ws + sp.wp);
    int rows = p->s.n, classes = p->s.c_out, d = p->s.c_in, dp = p->xent.dp;
    void *args[] = {&xs, &xp, &rows, &wsrc, &wp, &classes, &d, &dp};
    const long long blocks = (((long long)rows + classes) * (dp / 8) + 255) / 256, most = 8LL * p->num_sms;
    if (conv_launch((const void *)&xent_pad_kernel, dim3((unsigned)(blocks < most ? blocks : most)), dim3(256), args, 0, st) !=
        cudaSuccess)
        return CONV_ERR_CUDA;
    x = xp;
    w = wp;
    return CONV_OK;
}

}  // namespace

extern "C" int conv_plan_create_xent(int32_t rows, int32_t c_in, int32_t classes, int32_t piece, conv_dtype_t dtype,
                                     conv_plan_t **out_plan) {
    if (!out_plan) return CONV_ERR_NULL_ARG;
    *out_plan = nullptr;
    if (rows < 0 || c_in < 1 || classes < 1 || piece < 0) return CONV_ERR_INVALID_SHAPE;
    if ((int)dtype < CONV_F32 || (int)dtype > CONV_I8) return CONV_ERR_INVALID_ARG;
    if (dtype != CONV_BF16) return CONV_ERR_UNSUPPORTED;
    // 32-bit row, class and tile indices
    if (rows > (1 << 24) || classes > (1 << 24) || c_in > (1 << 20) ||
        (long long)((rows + 255) / 256) * ((classes + 255) / 256) >= (1ll << 30))
        return CONV_ERR_UNSUPPORTED;
    conv_plan *p = new (std::nothrow) conv_plan();
    if (!p) return CONV_ERR_OOM;
    p->s = {rows, 1, 1, c_in, classes, 1, 1};
    p->stride = 1; p->groups = 1; p->dtype = dtype; p->act = CONV_ACT_NONE; p->oh = 1; p->ow = 1;
    p->y_c = classes; p->up = 1; p->algo = CONV_ALGO_XENT;
    int rc = conv_plan_bind_device(p, true);
    for (int k = FWD; k <= PROD && rc == CONV_OK; ++k) rc = conv_grant_smem_once(kernel_of(k), p->device, kSmem);
    if (rc == CONV_OK && !encoder()) rc = CONV_ERR_CUDA;
    if (rc != CONV_OK) {
        conv_plan_destroy(p);
        return rc;
    }
    XentGeom &g = p->xent;
    g.dp = (c_in + 7) / 8 * 8;
    g.tiles_m = ceil_div(rows, kTile);
    g.tiles_n = ceil_div(classes, kTile);
    g.tiles_d = ceil_div(c_in, kTile);
    // Classes of a piece: whole tiles, one at least; as many as keep g within 256
    // MB where one does (up to 524,288 rows).
    long long most = piece > 0 ? piece : (256ll << 20) / 2 / (rows > 0 ? rows : 1);
    if (most < kTile) most = kTile;
    most = most / kTile * kTile;
    const long long all = (long long)g.tiles_n * kTile;
    g.pieces = ceil_div(all, most < all ? most : all);
    g.piece = ceil_div(g.tiles_n, g.pieces) * kTile;
    g.pieces = ceil_div(all, g.piece);
    // Fewer output tiles than pairs of SMs: each product's K axis in runs, so
    // that they all work.  (Few rows and many classes have tiles enough, of dw and
    // one K block each, and dx's few long ones are then left to a few pairs:
    // 20x512x65536 with the gradient takes 351 us.)
    const int pairs = p->num_sms / 2, pt = g.piece / kTile;
    const int tiles = (g.tiles_m + pt) * g.tiles_d;
    const int kx = g.piece / kBK, kw = ceil_div(rows, kBK);
    int sx = 1, sw = 1;
    if (tiles > 0 && tiles < pairs) {
        const int want = pairs / tiles;
        sx = want < kx / kMinRun ? want : kx / kMinRun;
        if (g.pieces == 1) sw = want < kw / kMinRun ? want : kw / kMinRun;
        if (sx < 1) sx = 1;
        if (sw < 1) sw = 1;
    }
    g.dx_kper = ceil_div(kx, sx);
    g.dx_split = ceil_div(kx, g.dx_kper);
    g.dw_kper = kw > 0 ? ceil_div(kw, sw) : 1;
    g.dw_split = kw > 0 ? ceil_div(kw, g.dw_kper) : 1;
    if (rows > 0) {
        const Space sp = space_of(p);
        p->ws_bytes = sp.fwd;
        p->ws_bwd_bytes = sp.bwd;
    }
    snprintf(p->desc, sizeof(p->desc), "xent bf16 tcgen05 pair tiles=%dx%d pieces=%d x %d classes dx_split=%d dw_split=%d",
             g.tiles_m, g.tiles_n, g.pieces, g.piece, g.dx_split, g.dw_split);
    *out_plan = p;
    return CONV_OK;
}

extern "C" int conv_run_xent(const conv_plan_t *plan, const void *x, const void *w, const int32_t *target, float *loss,
                             float *row_loss, float *lse, void *workspace, void *stream) {
    if (!plan) return CONV_ERR_NULL_ARG;
    const conv_plan *p = plan;
    if (p->algo != CONV_ALGO_XENT) return CONV_ERR_INVALID_ARG;
    cudaStream_t st = (cudaStream_t)stream;
    if (!loss) return CONV_ERR_NULL_ARG;
    if ((uintptr_t)loss & 3u) return CONV_ERR_MISALIGNED;
    if (p->s.n == 0) return cudaMemsetAsync(loss, 0, 4, st) == cudaSuccess ? CONV_OK : CONV_ERR_CUDA;
    if (!x || !w || !target || !workspace) return CONV_ERR_NULL_ARG;
    if (((uintptr_t)x & 15u) || ((uintptr_t)w & 15u) || ((uintptr_t)workspace & 15u) || ((uintptr_t)target & 3u) ||
        ((uintptr_t)row_loss & 3u) || ((uintptr_t)lse & 3u))
        return CONV_ERR_MISALIGNED;
    const size_t N = (size_t)p->s.n, V = (size_t)p->s.c_out, D = (size_t)p->s.c_in;
    const void *in[3] = {x, w, target};
    const size_t inb[3] = {N * D * 2, V * D * 2, N * 4};
    const void *out[4] = {loss, row_loss, lse, workspace};
    const size_t outb[4] = {4, N * 4, N * 4, p->ws_bytes};
    for (int i = 0; i < 4; ++i) {
        for (int j = 0; j < 3; ++j)
            if (conv_overlaps(out[i], outb[i], in[j], inb[j])) return CONV_ERR_ALIASING;
        for (int j = 0; j < i; ++j)
            if (conv_overlaps(out[i], outb[i], out[j], outb[j])) return CONV_ERR_ALIASING;
    }
    const XentGeom &g = p->xent;
    const Space sp = space_of(p);
    char *ws = static_cast<char *>(workspace);
    const int rc = operands(p, sp, ws, x, w, st);
    if (rc != CONV_OK) return rc;
    alignas(64) Maps maps = {};
    if (!make_map(&maps.a, x, p->s.c_in, p->s.n, g.dp, 128) || !make_map(&maps.b, w, p->s.c_in, p->s.c_out, g.dp, 128))
        return CONV_ERR_CUDA;
    XArgs a = {};
    a.rows = p->s.n; a.classes = a.all_classes = p->s.c_out; a.d = p->s.c_in;
    a.tiles_m = g.tiles_m; a.tiles_n = g.tiles_n; a.tiles = g.tiles_m * g.tiles_n;
    a.kblocks = ceil_div(p->s.c_in, kBK);
    a.target = target;
    a.part = reinterpret_cast<float2 *>(ws + sp.part);
    a.tlogit = reinterpret_cast<float *>(ws + sp.tlogit);
    a.counter = reinterpret_cast<unsigned *>(ws + sp.counter);
    a.status = p->d_status;
    if (launch_tiles(p, FWD, maps, a, st) != cudaSuccess) return CONV_ERR_CUDA;
    float *rl = row_loss ? row_loss : reinterpret_cast<float *>(ws + sp.row_loss);
    float *ls = lse ? lse : reinterpret_cast<float *>(ws + sp.lse);
    const float2 *part = a.part;
    const float *tl = a.tlogit;
    int pairs = 2 * g.tiles_n, rows = p->s.n, classes = p->s.c_out;
    void *args[] = {&part, &pairs, &rows, &classes, &target, &tl, &ls, &rl, &loss, &a.counter};
    return conv_launch((const void *)&xent_join_kernel, dim3((unsigned)ceil_div(rows, 32)), dim3(256), args, 0, st) == cudaSuccess
               ? CONV_OK
               : CONV_ERR_CUDA;
}

extern "C" int conv_run_xent_bwd(const conv_plan_t *plan, const void *x, const void *w, const int32_t *target, const float *lse,
                                 const float *dloss, void *dx, void *dw, void *workspace, void *stream) {
    if (!plan) return CONV_ERR_NULL_ARG;
    const conv_plan *p = plan;
    if (p->algo != CONV_ALGO_XENT) return CONV_ERR_INVALID_ARG;
    cudaStream_t st = (cudaStream_t)stream;
    const size_t N = (size_t)p->s.n, V = (size_t)p->s.c_out, D = (size_t)p->s.c_in;
    if (!dw || (N && !dx)) return CONV_ERR_NULL_ARG;
    if (((uintptr_t)dw & 15u) || ((uintptr_t)dx & 15u)) return CONV_ERR_MISALIGNED;
    if (N == 0) return cudaMemsetAsync(dw, 0, V * D * 2, st) == cudaSuccess ? CONV_OK : CONV_ERR_CUDA;
    if (!x || !w || !target || !lse || !workspace) return CONV_ERR_NULL_ARG;
    if (((uintptr_t)x & 15u) || ((uintptr_t)w & 15u) || ((uintptr_t)workspace & 15u) || ((uintptr_t)target & 3u) ||
        ((uintptr_t)lse & 3u) || ((uintptr_t)dloss & 3u))
        return CONV_ERR_MISALIGNED;
    const void *in[5] = {x, w, target, lse, dloss};
    const size_t inb[5] = {N * D * 2, V * D * 2, N * 4, N * 4, 4};
    const void *out[3] = {dx, dw, workspace};
    const size_t outb[3] = {N * D * 2, V * D * 2, p->ws_bwd_bytes};
    for (int i = 0; i < 3; ++i) {
        for (int j = 0; j < 5; ++j)
            if (conv_overlaps(out[i], outb[i], in[j], inb[j])) return CONV_ERR_ALIASING;
        for (int j = 0; j < i; ++j)
            if (conv_overlaps(out[i], outb[i], out[j], outb[j])) return CONV_ERR_ALIASING;
    }
    const XentGeom &g = p->xent;
    const Space sp = space_of(p);
    char *ws = static_cast<char *>(workspace);
    const int rc = operands(p, sp, ws, x, w, st);
    if (rc != CONV_OK) return rc;
    float *scale = reinterpret_cast<float *>(ws + sp.scale);
    float *dxp = reinterpret_cast<float *>(ws + sp.dxp), *dwp = reinterpret_cast<float *>(ws + sp.dwp);
    const void *gbuf = ws + sp.g;
    const __nv_bfloat16 *wb = static_cast<const __nv_bfloat16 *>(w);
    __nv_bfloat16 *dwb = static_cast<__nv_bfloat16 *>(dw);
    const bool tma_out = D % 8 == 0;
    for (int pc = 0; pc < g.pieces; ++pc) {
        const int v0 = pc * g.piece, vn = (int)V - v0 < g.piece ? (int)V - v0 : g.piece;
        const __nv_bfloat16 *wp = wb + (long long)v0 * g.dp;
        alignas(64) Maps maps = {};
        if (!make_map(&maps.a, x, p->s.c_in, p->s.n, g.dp, 128) || !make_map(&maps.b, wp, p->s.c_in, vn, g.dp, 128) ||
            !make_map(&maps.out, gbuf, vn, p->s.n, g.piece, 32))
            return CONV_ERR_CUDA;
        XArgs a = {};
        a.rows = p->s.n; a.classes = vn; a.d = p->s.c_in; a.v0 = v0;
        a.tiles_m = g.tiles_m; a.tiles_n = ceil_div(vn, kTile); a.tiles = a.tiles_m * a.tiles_n;
        a.kblocks = ceil_div(p->s.c_in, kBK);
        a.target = target; a.lse = lse; a.dloss = dloss; a.scale = scale; a.first = pc == 0;
        a.all_classes = p->s.c_out;
        a.status = p->d_status;
        if (launch_tiles(p, GRAD, maps, a, st) != cudaSuccess) return CONV_ERR_CUDA;

        alignas(64) Maps pm = {};
        if (!make_map(&pm.a, gbuf, vn, p->s.n, g.piece, 128) || !make_map(&pm.b, wp, p->s.c_in, vn, g.dp, 64) ||
            !make_map(&pm.a2, gbuf, vn, p->s.n, g.piece, 64) || !make_map(&pm.b2, x, p->s.c_in, p->s.n, g.dp, 64))
            return CONV_ERR_CUDA;
        if (tma_out && (!make_map(&pm.out, dx, p->s.c_in, p->s.n, D, 32) ||
                        !make_map(&pm.out2, dwb + (long long)v0 * D, p->s.c_in, vn, D, 32)))
            return CONV_ERR_CUDA;
        a.tma_out = tma_out;
        a.dx = static_cast<__nv_bfloat16 *>(dx);
        a.dw = dwb;
        a.dx_part = dxp; a.dw_part = dwp;
        a.dx_tm = g.tiles_m; a.dx_tn = g.tiles_d; a.dx_kb = ceil_div(vn, kBK);
        // (runs of one length in every piece: a short last piece has fewer of
        // them, and the others keep the sums of the pieces before)
        a.dx_kper = g.dx_kper;
        a.dx_split = ceil_div(a.dx_kb, a.dx_kper);
        a.dx_tiles = a.dx_split * a.dx_tm * a.dx_tn;
        a.dx_final = pc == g.pieces - 1 && g.dx_split == 1;
        a.dw_tm = ceil_div(vn, kTile); a.dw_tn = g.tiles_d; a.dw_kb = ceil_div(p->s.n, kBK);
        a.dw_kper = g.dw_kper;
        a.dw_split = g.dw_split;
        a.dw_tiles = a.dw_split * a.dw_tm * a.dw_tn;
        a.dw_final = g.dw_split == 1;
        a.dw_first = a.dw_kper > a.dx_kper;
        a.tiles = a.dx_tiles + a.dw_tiles;
        if (launch_tiles(p, PROD, pm, a, st) != cudaSuccess) return CONV_ERR_CUDA;
        if (g.dw_split > 1) {
            const float *part = dwp;
            int rows = vn, cols = p->s.c_in;
            __nv_bfloat16 *o = dwb + (long long)v0 * D;
            void *args[] = {&part, &a.dw_split, &a.dw_tm, &a.dw_tn, &rows, &cols, &scale, &o};
            if (conv_launch((const void *)&xent_finish_kernel, dim3((unsigned)(a.dw_tm * a.dw_tn * 16)), dim3(256), args, 0, st) !=
                cudaSuccess)
                return CONV_ERR_CUDA;
        }
        if (pc == g.pieces - 1 && g.dx_split > 1) {
            const float *part = dxp;
            int rows = p->s.n, cols = p->s.c_in;
            int splits = g.pieces > 1 ? g.dx_split : a.dx_split;  // (those that were written)
            void *args[] = {&part, &splits, &a.dx_tm, &a.dx_tn, &rows, &cols, &scale, &a.dx};
            if (conv_launch((const void *)&xent_finish_kernel, dim3((unsigned)(a.dx_tm * a.dx_tn * 16)), dim3(256), args, 0, st) !=
                cudaSuccess)
                return CONV_ERR_CUDA;
        }
    }
    return CONV_OK;
}
