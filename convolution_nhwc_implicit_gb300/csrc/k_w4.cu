// Pointwise (1x1) layer on few rows with 4-bit weights and group scales:
//   y[m,co] = act( b[co] + sum_j s[co,j] sum_{k in group j} (u[co,k] - 8) x[m,k] )
// u in 0..15 is the stored code, a group `group` consecutive input channels.
//
// The weights' bytes bound it: at 4 bits a weight and one row every byte is
// used twice (two multiply-adds), so all that counts is to stream them.  The
// codes are laid out once (w4_pack_kernel) so that a warp's 16-byte loads are
// whole 512-byte runs and every lane finds in them the A operands of
// mma.sync m16n8k16: a code is turned into the bf16 number u - 8, which is
// exact (bits 0x4300 | u are 128 + u; minus 136), the products and sums are
// the tensor core's in fp32, and a group's sum is scaled in fp32 when it ends.
// Nothing is rounded to fewer bits before the result.  fp32 rows are split
// into three bf16 parts (8 + 8 + 8 bits, the whole significand), three MMAs.
// (tcgen05 would need the decoded weights written to shared memory, four
// times the streamed bytes there and back, for a product whose operand
// rows are mostly empty.)
//
// Layout: tiles of 16 output channels x 64 input channels, 512 bytes, the
// tiles of 16 output channels one after the other along k.  Lane l (g = l / 4,
// t = l % 4) owns 16 bytes: word 2 h + r holds row g + 8 r, input channels
// 32 h + 8 t + 0..7 of the tile, channel 2 i in nibble i and 2 i + 1 in nibble
// i + 4, so that (word >> 4 i) & 0x000f000f is one operand register.  k is
// padded to 128 and rows to 16 with code 8 (zero).
//
// Two kernels:
//   w4_few   x, whole, in every CTA's shared memory (as the MMA's operand rows:
//            zeros past c_in, fp32 rows already split).  A CTA's warps share 16
//            output channels, each every kWarps-th run of 128 input channels,
//            and go on to the next 16 with the loads for them already under
//            way; the warps' sums meet in shared memory in a fixed order.
//   w4_many  where x does not fit: each warp has 16 output channels of its own
//            and all of k, x passing through shared memory 128 channels at a
//            time, loaded once for all the CTA's warps.
#include <cuda_bf16.h>
#include <math.h>
#include <stdint.h>
#include <stdio.h>

#include <new>

#include "conv_internal.h"
#include "epilogue.cuh"

using namespace convk;

namespace {

constexpr int kUnit = 128;       // input channels a warp takes at a time (two tiles)
constexpr int kPad = 64;         // bytes between x rows in shared memory: 16-byte reads of eight
                                 // rows' same channels then touch every bank once
constexpr int kManyPitch = kUnit * 2 + kPad;
constexpr int kManyRows = 64;
constexpr int kFewSmem = 200 * 1024;  // x bytes that w4_few keeps (one CTA a SM)

struct W4Args {
    const void *x;
    const uint4 *w;
    const void *scales;
    const float *bias;
    void *y;
    int rows, ci, co, ng, units, act, tiles;
};

__device__ __forceinline__ void mma16816(float (&c)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0,
                                         uint32_t b1) {
    asm volatile("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
                 : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
                 : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

__device__ __forceinline__ float elem_f(float v) { return v; }
__device__ __forceinline__ float elem_f(__nv_bfloat16 v) { return __bfloat162float(v); }
template <typename T> __device__ __forceinline__ T elem_from(float v) { return convk::Elem<T>::from_f(v); }

// Codes i and i + 4 of a word as the bf16 pair (u - 8).
__device__ __forceinline__ uint32_t decode(uint32_t w, int i) {
    const uint32_t v = ((w >> (4 * i)) & 0x000f000fu) | 0x43004300u;
    const __nv_bfloat162 d = __hsub2(*reinterpret_cast<const __nv_bfloat162 *>(&v),
                                     __halves2bfloat162(__ushort_as_bfloat16(0x4308), __ushort_as_bfloat16(0x4308)));
    return *reinterpret_cast<const uint32_t *>(&d);
}

// An x row's eight consecutive channels from k on as bf16 parts: the value
// itself (bf16 rows), or three parts of eight bits each (fp32 rows); zeros at
// and past ci.
struct XBf16 {
    static constexpr int kParts = 1;
    using Elem = __nv_bfloat16;
    __device__ static __forceinline__ void load(const Elem *row, int k, int ci, bool vec, uint4 (&out)[1]) {
        out[0] = make_uint4(0u, 0u, 0u, 0u);
        if (vec && k + 8 <= ci) {
            out[0] = *reinterpret_cast<const uint4 *>(row + k);
        } else {
            uint32_t b[4] = {0u, 0u, 0u, 0u};
#pragma unroll
            for (int i = 0; i < 8; ++i)
                if (k + i < ci) b[i >> 1] |= (uint32_t)__bfloat16_as_ushort(row[k + i]) << (16 * (i & 1));
            out[0] = make_uint4(b[0], b[1], b[2], b[3]);
        }
    }
};
struct XF32 {
    static constexpr int kParts = 3;
    using Elem = float;
    // The three parts of v, cut (not rounded) to bf16's eight bits each, so
    // that no partial sum of them passes v itself: the largest fp32 values do
    // not overflow on the way.  Only the first part holds an infinity or a NaN
    // (inf - inf would make a NaN of the others).
    __device__ static __forceinline__ void split(float v, uint32_t (&p)[3]) {
        const uint32_t bits = __float_as_uint(v);
        p[0] = bits >> 16;
        const float r1 = v - __uint_as_float(bits & 0xffff0000u);
        const uint32_t b1 = __float_as_uint(r1);
        p[1] = b1 >> 16;
        p[2] = __float_as_uint(r1 - __uint_as_float(b1 & 0xffff0000u)) >> 16;
        if ((bits & 0x7f800000u) == 0x7f800000u) {
            if (bits & 0x007fffffu) p[0] = 0x7fffu;  // (a NaN whose mark the cut would lose)
            p[1] = p[2] = 0u;
        }
    }
    __device__ static __forceinline__ void load(const Elem *row, int k, int ci, bool vec, uint4 (&out)[3]) {
        float f[8];
        if (vec && k + 8 <= ci) {
            const float4 u = *reinterpret_cast<const float4 *>(row + k), v = *reinterpret_cast<const float4 *>(row + k + 4);
            f[0] = u.x; f[1] = u.y; f[2] = u.z; f[3] = u.w; f[4] = v.x; f[5] = v.y; f[6] = v.z; f[7] = v.w;
        } else {
#pragma unroll
            for (int i = 0; i < 8; ++i) f[i] = k + i < ci ? row[k + i] : 0.0f;
        }
        uint32_t b[3][4];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            uint32_t lo[3], hi[3];
            split(f[2 * i], lo);
            split(f[2 * i + 1], hi);
#pragma unroll
            for (int q = 0; q < 3; ++q) b[q][i] = lo[q] | (hi[q] << 16);
        }
#pragma unroll
        for (int q = 0; q < 3; ++q) out[q] = make_uint4(b[q][0], b[q][1], b[q][2], b[q][3]);
    }
};

// A warp's 16 output channels by 128 input channels, as loaded.
template <int GROUP>
struct Unit {
    static constexpr int kGroups = kUnit / GROUP;
    uint4 wa, wb;
    float f0[kGroups], f1[kGroups];  // scales of rows g and g + 8
    template <typename Elem>
    __device__ __forceinline__ void fetch(const uint4 *w, int u, const Elem *s0, const Elem *s1, int ng, bool on0, bool on1) {
        wa = __ldcs(w + (long long)u * 64);
        wb = __ldcs(w + (long long)u * 64 + 32);
#pragma unroll
        for (int j = 0; j < kGroups; ++j) {
            const int gi = u * kGroups + j;
            f0[j] = on0 && gi < ng ? elem_f(s0[gi]) : 0.0f;
            f1[j] = on1 && gi < ng ? elem_f(s1[gi]) : 0.0f;
        }
    }
};

// acc += the unit's products with NT blocks of eight x rows; xs: this lane's
// address in the first part's row g (of the first block), channel 8 t of the
// unit; part_step and the 8-row block's step in bytes.  on[n]: row 8 n + g exists.
template <typename X, int NT, int GROUP>
__device__ __forceinline__ void products(const Unit<GROUP> &un, float (&acc)[NT][4], const uint8_t *xs, int block_step, int part_step,
                                         const bool (&on)[NT]) {
    constexpr int kHalves = GROUP / 32;  // steps of 32 channels a scale
    float c[NT][4];
#pragma unroll
    for (int h = 0; h < 4; ++h) {
        if (h % kHalves == 0) {
#pragma unroll
            for (int n = 0; n < NT; ++n)
#pragma unroll
                for (int e = 0; e < 4; ++e) c[n][e] = 0.0f;
        }
        const uint32_t lo = h == 0 ? un.wa.x : (h == 1 ? un.wa.z : (h == 2 ? un.wb.x : un.wb.z));
        const uint32_t hi = h == 0 ? un.wa.y : (h == 1 ? un.wa.w : (h == 2 ? un.wb.y : un.wb.w));
        uint32_t p[4], q[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            p[i] = decode(lo, i);
            q[i] = decode(hi, i);
        }
#pragma unroll
        for (int n = 0; n < NT; ++n)
#pragma unroll
            for (int r = 0; r < X::kParts; ++r) {
                uint4 b = make_uint4(0u, 0u, 0u, 0u);
                if (on[n]) b = *reinterpret_cast<const uint4 *>(xs + n * block_step + r * part_step + h * 64);
                mma16816(c[n], p[0], q[0], p[1], q[1], b.x, b.y);
                mma16816(c[n], p[2], q[2], p[3], q[3], b.z, b.w);
            }
        if (h % kHalves == kHalves - 1) {
            const int j = h / kHalves;
#pragma unroll
            for (int n = 0; n < NT; ++n) {
                acc[n][0] = fmaf(un.f0[j], c[n][0], acc[n][0]);
                acc[n][1] = fmaf(un.f0[j], c[n][1], acc[n][1]);
                acc[n][2] = fmaf(un.f1[j], c[n][2], acc[n][2]);
                acc[n][3] = fmaf(un.f1[j], c[n][3], acc[n][3]);
            }
        }
    }
}

// CTAs of eight warps a SM: as many as their registers allow without spilling.
__host__ __device__ constexpr int few_ctas(int parts, int nt) { return nt * (parts == 3 ? 2 : 1) >= 4 ? 2 : 3; }

template <typename X, int NT, int GROUP, int WARPS>
__global__ void __launch_bounds__(WARPS * 32, WARPS == 8 ? few_ctas(X::kParts, NT) : 1) w4_few_kernel(W4Args a, int vec) {
    using Elem = typename X::Elem;
    constexpr int kThreads = WARPS * 32;
    extern __shared__ __align__(16) uint8_t shm[];
    float *red = reinterpret_cast<float *>(shm);  // [2][WARPS][NT * 8][16]
    constexpr int kRed = WARPS * NT * 8 * 16;
    uint8_t *xs = shm + 2 * kRed * 4;             // [parts][rows] of pitch bytes
    const int pitch = a.units * kUnit * 2 + kPad, part_step = a.rows * pitch;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, g = lane >> 2, t = lane & 3;
    pdl_trigger();
    pdl_wait();
    const Elem *x = static_cast<const Elem *>(a.x);
    const Elem *sc = static_cast<const Elem *>(a.scales);
    const int per = (a.units + WARPS - 1) / WARPS;        // steps of a warp a tile
    const int mine = ((int)gridDim.x < a.tiles ? (a.tiles - 1 - (int)blockIdx.x) / (int)gridDim.x + 1 : 1) * per;
    Unit<GROUP> un[2];
    // step j: tile blockIdx.x + (j / per) gridDim.x, unit warp + (j % per) WARPS
    int ft = blockIdx.x, fi = 0;                          // the next step to fetch
    auto fetch = [&](Unit<GROUP> &d) {
        const int u = warp + fi * WARPS, co = ft * 16 + g;
        if (ft < a.tiles && u < a.units)
            d.fetch(a.w + (long long)ft * a.units * 64 + lane, u, sc + (long long)co * a.ng, sc + (long long)(co + 8) * a.ng, a.ng,
                    co < a.co, co + 8 < a.co);
        if (++fi == per) { fi = 0; ft += gridDim.x; }
    };
    fetch(un[0]);
    fetch(un[1]);
    // x into shared memory, eight channels a thread at a time
    const int eights = a.units * (kUnit / 8);
    for (int i = threadIdx.x; i < a.rows * eights; i += kThreads) {
        const int m = i / eights, k = (i - m * eights) * 8;
        uint4 v[X::kParts];
        X::load(x + (long long)m * a.ci, k, a.ci, vec != 0, v);
#pragma unroll
        for (int r = 0; r < X::kParts; ++r) *reinterpret_cast<uint4 *>(xs + r * part_step + m * pitch + k * 2) = v[r];
    }
    __syncthreads();
    bool on[NT];
#pragma unroll
    for (int n = 0; n < NT; ++n) on[n] = n * 8 + g < a.rows;
    const uint8_t *xl = xs + g * pitch + t * 16;
    float acc[NT][4];
#pragma unroll
    for (int n = 0; n < NT; ++n)
#pragma unroll
        for (int e = 0; e < 4; ++e) acc[n][e] = 0.0f;
    int i = 0, tile = blockIdx.x, side = 0;
    auto step = [&](Unit<GROUP> &cur) {
        const int u = warp + i * WARPS;
        if (u < a.units) products<X, NT, GROUP>(cur, acc, xl + u * (kUnit * 2), 8 * pitch, part_step, on);
        fetch(cur);
        if (++i < per) return;
        i = 0;
        // the tile's sums: one barrier a tile, two sides in turn (a side is
        // written again only after the next tile's barrier)
        float *mine_red = red + side * kRed + warp * (NT * 8 * 16);
#pragma unroll
        for (int n = 0; n < NT; ++n) {
            mine_red[(n * 8 + 2 * t) * 16 + g] = acc[n][0];
            mine_red[(n * 8 + 2 * t + 1) * 16 + g] = acc[n][1];
            mine_red[(n * 8 + 2 * t) * 16 + g + 8] = acc[n][2];
            mine_red[(n * 8 + 2 * t + 1) * 16 + g + 8] = acc[n][3];
#pragma unroll
            for (int e = 0; e < 4; ++e) acc[n][e] = 0.0f;
        }
        __syncthreads();
        for (int o = threadIdx.x; o < a.rows * 16; o += kThreads) {
            const int m = o >> 4, co = tile * 16 + (o & 15);
            if (co >= a.co) continue;
            float v = 0.0f;
#pragma unroll
            for (int q = 0; q < WARPS; ++q) v += red[side * kRed + q * (NT * 8 * 16) + o];
            v = activate(v + (a.bias ? a.bias[co] : 0.0f), a.act);
            static_cast<Elem *>(a.y)[(long long)m * a.co + co] = elem_from<Elem>(v);
        }
        side ^= 1;
        tile += gridDim.x;
    };
    int j = 0;
    for (; j + 1 < mine; j += 2) {
        step(un[0]);
        step(un[1]);
    }
    if (j < mine) step(un[0]);
}

template <typename X, int GROUP, int WARPS>
__global__ void __launch_bounds__(WARPS * 32) w4_many_kernel(W4Args a, int vec) {
    using Elem = typename X::Elem;
    constexpr int kThreads = WARPS * 32, NT = kManyRows / 8;
    constexpr int kPart = kManyRows * kManyPitch, kSide = X::kParts * kPart;
    extern __shared__ __align__(16) uint8_t shm[];  // [2][parts][64] rows of kManyPitch bytes
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, g = lane >> 2, t = lane & 3;
    const int m0 = blockIdx.y * kManyRows, rows = min(kManyRows, a.rows - m0);
    const int tile = blockIdx.x * WARPS + warp;
    const bool live = tile < a.tiles;
    pdl_trigger();
    pdl_wait();
    const Elem *x = static_cast<const Elem *>(a.x) + (long long)m0 * a.ci;
    const int co = tile * 16 + g;
    const Elem *s0 = static_cast<const Elem *>(a.scales) + (long long)co * a.ng, *s1 = s0 + 8LL * a.ng;
    const uint4 *w = a.w + (long long)tile * a.units * 64 + lane;
    const bool on0 = co < a.co, on1 = co + 8 < a.co;
    auto stage = [&](int u) {
        uint8_t *dst = shm + (u & 1) * kSide;
        for (int i = threadIdx.x; i < rows * (kUnit / 8); i += kThreads) {
            const int m = i / (kUnit / 8), k = (i % (kUnit / 8)) * 8;
            uint4 v[X::kParts];
            X::load(x + (long long)m * a.ci, u * kUnit + k, a.ci, vec != 0, v);
#pragma unroll
            for (int r = 0; r < X::kParts; ++r) *reinterpret_cast<uint4 *>(dst + r * kPart + m * kManyPitch + k * 2) = v[r];
        }
    };
    bool on[NT];
    float acc[NT][4];
#pragma unroll
    for (int n = 0; n < NT; ++n) {
        on[n] = n * 8 + g < rows;
#pragma unroll
        for (int e = 0; e < 4; ++e) acc[n][e] = 0.0f;
    }
    Unit<GROUP> cur, nxt;
    if (live) cur.fetch(w, 0, s0, s1, a.ng, on0, on1);
    stage(0);
    for (int u = 0; u < a.units; ++u) {
        __syncthreads();  // unit u is staged, and everyone has left unit u - 1
        if (live && u + 1 < a.units) nxt.fetch(w, u + 1, s0, s1, a.ng, on0, on1);
        if (u + 1 < a.units) stage(u + 1);
        if (live) products<X, NT, GROUP>(cur, acc, shm + (u & 1) * kSide + g * kManyPitch + t * 16, 8 * kManyPitch, kPart, on);
        cur = nxt;
    }
    if (!live) return;
#pragma unroll
    for (int n = 0; n < NT; ++n)
#pragma unroll
        for (int e = 0; e < 4; ++e) {
            const int m = n * 8 + 2 * t + (e & 1), c = co + (e >> 1) * 8;
            if (m < rows && c < a.co)
                static_cast<Elem *>(a.y)[(long long)(m0 + m) * a.co + c] =
                    elem_from<Elem>(activate(acc[n][e] + (a.bias ? a.bias[c] : 0.0f), a.act));
        }
}

// One 32-bit word of the laid-out codes a thread.
__global__ void w4_pack_kernel(const uint8_t *codes, uint32_t *out, int ci, int co, int units, long long words) {
    pdl_trigger();
    pdl_wait();
    const long long i = (long long)blockIdx.x * blockDim.x + threadIdx.x;
    if (i >= words) return;
    const int wd = (int)(i & 3), lane = (int)(i >> 2) & 31;
    const long long tile = i >> 7;
    const int kt = (int)(tile % (2 * units));
    const long long row = tile / (2 * units) * 16 + (lane >> 2) + 8 * (wd & 1);
    const int k0 = kt * 64 + (wd >> 1) * 32 + (lane & 3) * 8;
    uint32_t v = 0x88888888u;
    if (row < co) {
        const uint8_t *src = codes + row * ((ci + 1) / 2);
#pragma unroll
        for (int j = 0; j < 8; ++j) {
            const int k = k0 + j;
            if (k < ci) {
                const uint32_t u = (src[k >> 1] >> (4 * (k & 1))) & 15u;
                const int pos = 4 * ((j >> 1) + 4 * (j & 1));
                v = (v & ~(15u << pos)) | (u << pos);
            }
        }
    }
    out[i] = v;
}

// Codes and scales of a weight row's group, one warp a group: s = max |w| / 7
// rounded to the scales' type, u = clamp(round_half_even(w / s), -8, 7) + 8.
template <typename T>
__global__ void w4_quantize_kernel(const T *w, uint8_t *codes, T *scales, int ci, int ng, int group, long long total) {
    pdl_trigger();
    pdl_wait();
    const long long i = ((long long)blockIdx.x * blockDim.x + threadIdx.x) >> 5;
    if (i >= total) return;
    const int lane = threadIdx.x & 31;
    const long long row = i / ng;
    const int k0 = (int)(i % ng) * group, k1 = min(ci, k0 + group);
    float top = 0.0f;
    for (int k = k0 + lane; k < k1; k += 32) top = fmaxf(top, fabsf(elem_f(w[row * ci + k])));
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, o));
    const T s = elem_from<T>(top / 7.0f);
    const float sf = elem_f(s);
    if (lane == 0) scales[i] = s;
    for (int k = k0 + 2 * lane; k < k1; k += 64) {
        uint32_t byte = 0;
#pragma unroll
        for (int e = 0; e < 2; ++e) {
            int q = 0;
            if (k + e < k1 && sf > 0.0f) q = max(-8, min(7, __float2int_rn(elem_f(w[row * ci + k + e]) / sf)));
            byte |= (uint32_t)(q + 8) << (4 * e);
        }
        codes[row * ((ci + 1) / 2) + (k >> 1)] = (uint8_t)byte;
    }
}

// ------------------------------------------------------------------ host side
template <typename X, int NT, int WARPS>
const void *few_group(int group) {
    return group == 32 ? (const void *)&w4_few_kernel<X, NT, 32, WARPS>
                       : (group == 64 ? (const void *)&w4_few_kernel<X, NT, 64, WARPS> : (const void *)&w4_few_kernel<X, NT, 128, WARPS>);
}
template <typename X, int WARPS>
const void *few_nt(int nt, int group) {
    switch (nt) {
    case 1: return few_group<X, 1, WARPS>(group);
    case 2: return few_group<X, 2, WARPS>(group);
    default: return few_group<X, 4, WARPS>(group);
    }
}
template <typename X, int WARPS>
const void *many_group(int group) {
    return group == 32 ? (const void *)&w4_many_kernel<X, 32, WARPS>
                       : (group == 64 ? (const void *)&w4_many_kernel<X, 64, WARPS> : (const void *)&w4_many_kernel<X, 128, WARPS>);
}
template <typename X>
const void *pick(const W4Geom &g) {
    if (g.many) return g.warps == 8 ? many_group<X, 8>(g.group) : (g.warps == 4 ? many_group<X, 4>(g.group) : many_group<X, 2>(g.group));
    return g.warps == 8 ? few_nt<X, 8>(g.nt, g.group) : few_nt<X, 16>(g.nt, g.group);
}

bool overlap(const void *a, size_t na, const void *b, size_t nb) {
    if (!a || !b || !na || !nb) return false;
    const uintptr_t a0 = (uintptr_t)a, b0 = (uintptr_t)b;
    return a0 < b0 + nb && b0 < a0 + na;
}

}  // namespace

extern "C" int conv_plan_create_w4(int32_t rows, int32_t c_in, int32_t c_out, int32_t group, conv_dtype_t dtype,
                                   conv_act_t act, conv_plan_t **out_plan) {
    if (!out_plan) return CONV_ERR_NULL_ARG;
    *out_plan = nullptr;
    if (rows < 0 || c_in < 1 || c_out < 1) return CONV_ERR_INVALID_SHAPE;
    if ((int)dtype < CONV_F32 || (int)dtype > CONV_I8) return CONV_ERR_INVALID_ARG;
    if ((int)act < CONV_ACT_NONE || (int)act > CONV_ACT_MISH) return CONV_ERR_INVALID_ARG;
    if (group != 32 && group != 64 && group != 128) return CONV_ERR_INVALID_ARG;
    if (dtype == CONV_I8) return CONV_ERR_UNSUPPORTED;
    if (c_in >= (1 << 28) || c_out >= (1 << 30) || rows >= (1 << 21) || (long long)c_in * c_out >= (1ll << 40))
        return CONV_ERR_UNSUPPORTED;
    conv_plan *p = new (std::nothrow) conv_plan();
    if (!p) return CONV_ERR_OOM;
    p->s = {rows, 1, 1, c_in, c_out, 1, 1};
    p->stride = 1; p->groups = 1; p->dtype = dtype; p->act = act; p->oh = 1; p->ow = 1;
    p->y_c = c_out; p->up = 1; p->algo = CONV_ALGO_W4;
    const int rc = conv_plan_bind_device(p, false);
    if (rc != CONV_OK) {
        conv_plan_destroy(p);
        return rc;
    }
    W4Geom &g = p->w4;
    const int parts = dtype == CONV_F32 ? 3 : 1, tiles = (c_out + 15) / 16;
    g.group = group;
    g.ng = (c_in + group - 1) / group;
    g.units = (c_in + kUnit - 1) / kUnit;
    g.nt = rows <= 8 ? 1 : (rows <= 16 ? 2 : 4);
    const long long xb = (long long)parts * rows * (g.units * (kUnit * 2) + kPad);
    // x whole in shared memory while it fits (with the warps' sums), else in
    // pieces; CTAs of 16 warps where it takes more than a third of a SM's.
    g.many = rows > 32 || xb + 2LL * 16 * g.nt * 128 * 4 > kFewSmem;
    if (g.many) {
        g.warps = 8;
        while (g.warps > 2 && (tiles + g.warps - 1) / g.warps * ((rows + kManyRows - 1) / kManyRows) < p->num_sms) g.warps /= 2;
        g.smem = 2 * parts * kManyRows * kManyPitch;
        g.grid = (tiles + g.warps - 1) / g.warps;
    } else {
        const long long red8 = 2LL * 8 * g.nt * 128 * 4;
        g.warps = xb + red8 <= 72 * 1024 ? 8 : 16;
        g.smem = (int)(xb + red8 * (g.warps / 8));
        const int wave = p->num_sms * (g.warps == 8 ? few_ctas(parts, g.nt) : 1);
        g.grid = tiles < wave ? tiles : wave;
    }
    snprintf(p->desc, sizeof(p->desc), "w4 %s group=%d %s warps=%d tiles=%d", dtype == CONV_F32 ? "f32" : "bf16", group,
             g.many ? "x in pieces" : "x in shared memory", g.warps, tiles);
    *out_plan = p;
    return CONV_OK;
}

extern "C" int conv_w4_packed_bytes(int32_t c_in, int32_t c_out, size_t *bytes) {
    if (!bytes) return CONV_ERR_NULL_ARG;
    if (c_in < 1 || c_out < 1) return CONV_ERR_INVALID_SHAPE;
    *bytes = (size_t)((c_out + 15) / 16) * ((c_in + kUnit - 1) / kUnit) * 1024;
    return CONV_OK;
}

extern "C" int conv_w4_pack(int32_t c_in, int32_t c_out, const void *codes, void *packed, void *stream) {
    size_t bytes = 0;
    const int rc = conv_w4_packed_bytes(c_in, c_out, &bytes);
    if (rc != CONV_OK) return rc;
    if (!codes || !packed) return CONV_ERR_NULL_ARG;
    if ((uintptr_t)packed & 15u) return CONV_ERR_MISALIGNED;
    if (overlap(packed, bytes, codes, (size_t)c_out * ((c_in + 1) / 2))) return CONV_ERR_ALIASING;
    long long words = (long long)(bytes / 4);
    if ((words + 255) / 256 > 0x7fffffffll) return CONV_ERR_UNSUPPORTED;
    int units = (c_in + kUnit - 1) / kUnit;
    const uint8_t *src = static_cast<const uint8_t *>(codes);
    uint32_t *dst = static_cast<uint32_t *>(packed);
    void *args[] = {&src, &dst, &c_in, &c_out, &units, &words};
    const cudaError_t e = conv_launch((const void *)&w4_pack_kernel, dim3((unsigned)((words + 255) / 256)), dim3(256), args,
                                      0, (cudaStream_t)stream);
    return e == cudaSuccess ? CONV_OK : CONV_ERR_CUDA;
}

extern "C" int conv_w4_quantize(int32_t c_in, int32_t c_out, int32_t group, conv_dtype_t dtype, const void *w, void *codes,
                                void *scales, void *stream) {
    if (c_in < 1 || c_out < 1) return CONV_ERR_INVALID_SHAPE;
    if ((int)dtype < CONV_F32 || (int)dtype > CONV_I8) return CONV_ERR_INVALID_ARG;
    if (group != 32 && group != 64 && group != 128) return CONV_ERR_INVALID_ARG;
    if (dtype == CONV_I8) return CONV_ERR_UNSUPPORTED;
    if (!w || !codes || !scales) return CONV_ERR_NULL_ARG;
    const size_t es = (size_t)conv_esize(dtype);
    if ((uintptr_t)w % es || (uintptr_t)scales % es) return CONV_ERR_MISALIGNED;
    int ng = (c_in + group - 1) / group;
    long long total = (long long)c_out * ng;
    if ((total + 7) / 8 > 0x7fffffffll) return CONV_ERR_UNSUPPORTED;
    const size_t wb = (size_t)c_in * c_out * es, cb = (size_t)c_out * ((c_in + 1) / 2), sb = (size_t)total * es;
    if (overlap(codes, cb, w, wb) || overlap(scales, sb, w, wb) || overlap(codes, cb, scales, sb)) return CONV_ERR_ALIASING;
    const void *k = dtype == CONV_F32 ? (const void *)&w4_quantize_kernel<float> : (const void *)&w4_quantize_kernel<__nv_bfloat16>;
    void *args[] = {(void *)&w, (void *)&codes, (void *)&scales, &c_in, &ng, &group, &total};
    const cudaError_t e = conv_launch(k, dim3((unsigned)((total + 7) / 8)), dim3(256), args, 0, (cudaStream_t)stream);
    return e == cudaSuccess ? CONV_OK : CONV_ERR_CUDA;
}

extern "C" int conv_run_w4(const conv_plan_t *plan, const void *x, const void *packed, const void *scales, const float *bias,
                           void *y, void *stream) {
    if (!plan) return CONV_ERR_NULL_ARG;
    const conv_plan *p = plan;
    if (p->algo != CONV_ALGO_W4) return CONV_ERR_INVALID_ARG;
    if (p->s.n == 0) return CONV_OK;
    if (!x || !packed || !scales || !y) return CONV_ERR_NULL_ARG;
    const size_t es = (size_t)conv_esize(p->dtype);
    if (((uintptr_t)packed & 15u) || (uintptr_t)x % es || (uintptr_t)scales % es || (uintptr_t)y % es || ((uintptr_t)bias & 3u))
        return CONV_ERR_MISALIGNED;
    const int ci = p->s.c_in, co = p->s.c_out, rows = p->s.n;
    size_t pb = 0;
    conv_w4_packed_bytes(ci, co, &pb);
    const size_t yb = (size_t)rows * co * es;
    if (overlap(y, yb, x, (size_t)rows * ci * es) || overlap(y, yb, packed, pb) ||
        overlap(y, yb, scales, (size_t)co * p->w4.ng * es) || overlap(y, yb, bias, (size_t)co * 4))
        return CONV_ERR_ALIASING;
    const W4Geom &g = p->w4;
    W4Args a = {x, static_cast<const uint4 *>(packed), scales, bias, y, rows, ci, co, g.ng, g.units, p->act, (co + 15) / 16};
    int vec = ci % 8 == 0 && ((uintptr_t)x & 15u) == 0 ? 1 : 0;
    const void *k = p->dtype == CONV_F32 ? pick<XF32>(g) : pick<XBf16>(g);
    if (g.smem > 48 * 1024) {
        const int rc = conv_grant_smem_once(k, p->device, g.smem);
        if (rc != CONV_OK) return rc;
    }
    void *args[] = {&a, &vec};
    const dim3 grid((unsigned)g.grid, (unsigned)(g.many ? (rows + kManyRows - 1) / kManyRows : 1));
    const cudaError_t e = conv_launch(k, grid, dim3(g.warps * 32), args, (size_t)g.smem, (cudaStream_t)stream);
    return e == cudaSuccess ? CONV_OK : CONV_ERR_CUDA;
}
