// Pointwise (1x1) layer on few rows with 4-bit weights and group scales:
//   y[m,co] = act( b[co] + sum_j s[co,j] sum_{k in group j} (u[co,k] - 8) x[m,k] )
// u in 0..15 is the stored code, a group `group` consecutive input channels.
//
// The weights' bytes bound it: at 4 bits a weight and one row every byte is
// used twice (two multiply-adds), so all that counts is to stream them.  The
// codes are laid out once (w4_pack_kernel) so that a warp's 16-byte loads are
// whole 512-byte runs and every lane finds in them the A operands of
// mma.sync m16n8k16.  A code becomes the bf16 number (u - 8) / 64, exactly, with
// one AND and one multiply-add a pair: four bits at the foot of a bf16 are the
// subnormal u 2^-133, and the four above them, which reach into the exponent,
// are 16 u 2^-133 (subnormals and the first normal binade lie on one line), so
// 2^127 or 2^123 times them is u / 64.  The products and sums are the tensor
// core's in fp32, and a group's sum is scaled in fp32 when it ends.
// Nothing is rounded to fewer bits before the result.  fp32 rows are split
// into three bf16 parts (8 + 8 + 8 bits, the whole significand; of values below
// 2^-102 the last parts pass bf16's subnormals and are cut at 2^-133), three MMAs.
// Measured on a GB300 (graph replay over changing inputs): one bf16 row through
// 8192x28672, groups of 128, 24.9 us, 4.9 TB/s of codes and scales, 72 % of the
// measured copy rate; issue slots are 64 % full and set the rest (128 input
// channels of 16 outputs cost a warp about 150 instructions, 40 of them the
// ANDs and shifts of the decoding; with a shift, an AND-OR and a
// subtraction a pair it took 33.3 us).  Groups of 32: 28.1 us.  1024x1000: 2.4
// us, of which a launch is 2.1.  64 rows of 8192x28672 143 us.
// (One or a few rows leave most of a tcgen05 tile empty.  From some tens of rows
// on this is mma.sync's rate and not the bytes: tcgen05 with the decoded weights
// in TMEM as A and x in shared memory as B was not built.)
//
// Layout: tiles of 16 output channels x 64 input channels, 512 bytes, the
// tiles of 16 output channels one after the other along k.  Lane l (g = l / 4,
// t = l % 4) owns 16 bytes: word 2 h + r holds row g + 8 r, input channels
// 32 h + 8 t + 0..7 of the tile, channel 2 i in nibble i and 2 i + 1 in nibble
// i + 4, so that (word >> 4 i) & 0x000f000f is one operand register.  k is
// padded to 128 and rows to 16 with code 8 (zero).
//
// Every warp streams its weights through a ring of shared memory slots of its
// own (cp.async, 1 KB units, kAhead on the way), so that a SM keeps ~100 KB in
// flight whatever the arithmetic does.  Two kernels:
//   w4_few   x, whole, in every CTA's shared memory (as the MMA's operand rows:
//            zeros past c_in, fp32 rows already split).  A CTA's warps share 16
//            output channels, each every WARPS-th run of 128 input channels,
//            and go on to the next 16 without a pause; the warps' sums meet in
//            shared memory in a fixed order.
//   w4_many  where x does not fit: a CTA's warps have WC times 16 output
//            channels and take k in turns of WK = 8 / WC units, x passing
//            through shared memory, loaded once for all of them.
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
constexpr int kAhead = 4;        // units of a warp's ring (a power of two)
constexpr int kPad = 64;         // bytes between x rows in shared memory: 16-byte reads of eight
                                 // rows' same channels then touch every bank once
constexpr int kSmemMost = 200 * 1024, kFewMost = 226 * 1024;

struct W4Args {
    const void *x;
    const uint4 *w;
    const void *scales;
    const float *bias;
    void *y;
    int rows, ci, co, ng, units, act, tiles;
};

// c = a b, and c += a b
__device__ __forceinline__ void mma16816_first(float (&c)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0,
                                               uint32_t b1) {
    asm volatile("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%10,%10,%10,%10};"
                 : "=f"(c[0]), "=f"(c[1]), "=f"(c[2]), "=f"(c[3])
                 : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1), "f"(0.0f));
}
__device__ __forceinline__ void mma16816(float (&c)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0,
                                         uint32_t b1) {
    asm volatile("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
                 : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
                 : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

__device__ __forceinline__ float elem_f(float v) { return v; }
__device__ __forceinline__ float elem_f(__nv_bfloat16 v) { return __bfloat162float(v); }
template <typename T> __device__ __forceinline__ T elem_from(float v) { return convk::Elem<T>::from_f(v); }
// The activation; ReLU passes a NaN on, which activate's maximum would answer with 0.
__device__ __forceinline__ float act_out(float v, int act) {
    if (act == ACT_RELU) return v < 0.0f ? 0.0f : v;
    return activate(v, act);
}

// A word's eight codes as four bf16 pairs (u - 8) / 64, pair i codes i and i + 4.
__device__ __forceinline__ void decode(uint32_t w, uint32_t (&p)[4]) {
    const uint32_t h = w >> 8;
    auto line = [](uint32_t bits, uint32_t scale) {  // bits * scale - 1/8
        uint32_t r;
        asm("fma.rn.bf16x2 %0, %1, %2, %3;" : "=r"(r) : "r"(bits), "r"(scale), "r"(0xbe00be00u));
        return r;
    };
    p[0] = line(w & 0x000f000fu, 0x7f007f00u);  // times 2^127
    p[1] = line(w & 0x00f000f0u, 0x7d007d00u);  // times 2^123
    p[2] = line(h & 0x000f000fu, 0x7f007f00u);
    p[3] = line(h & 0x00f000f0u, 0x7d007d00u);
}
constexpr float kCodeScale = 64.0f;

// An x row's eight consecutive channels from k on as bf16 parts: the value
// itself (bf16 rows), or three parts of eight bits each (fp32 rows); zeros at
// and past ci.
struct XBf16 {
    static constexpr int kParts = 1;
    using Elem = __nv_bfloat16;
    using Raw = uint4;
    __device__ static __forceinline__ Raw fetch(const Elem *row, int k, int ci, bool vec) {
        if (vec && k + 8 <= ci) return *reinterpret_cast<const uint4 *>(row + k);
        uint32_t b[4] = {0u, 0u, 0u, 0u};
#pragma unroll
        for (int i = 0; i < 8; ++i)
            if (k + i < ci) b[i >> 1] |= (uint32_t)__bfloat16_as_ushort(row[k + i]) << (16 * (i & 1));
        return make_uint4(b[0], b[1], b[2], b[3]);
    }
    __device__ static __forceinline__ void parts(const Raw &r, uint4 (&out)[1]) { out[0] = r; }
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
    struct Raw { float f[8]; };
    __device__ static __forceinline__ Raw fetch(const Elem *row, int k, int ci, bool vec) {
        Raw r;
        if (vec && k + 8 <= ci) {
            const float4 u = *reinterpret_cast<const float4 *>(row + k), v = *reinterpret_cast<const float4 *>(row + k + 4);
            r.f[0] = u.x; r.f[1] = u.y; r.f[2] = u.z; r.f[3] = u.w; r.f[4] = v.x; r.f[5] = v.y; r.f[6] = v.z; r.f[7] = v.w;
        } else {
#pragma unroll
            for (int i = 0; i < 8; ++i) r.f[i] = k + i < ci ? row[k + i] : 0.0f;
        }
        return r;
    }
    __device__ static __forceinline__ void parts(const Raw &r, uint4 (&out)[3]) {
        uint32_t b[3][4];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            uint32_t lo[3], hi[3];
            split(r.f[2 * i], lo);
            split(r.f[2 * i + 1], hi);
#pragma unroll
            for (int q = 0; q < 3; ++q) b[q][i] = lo[q] | (hi[q] << 16);
        }
#pragma unroll
        for (int q = 0; q < 3; ++q) out[q] = make_uint4(b[q][0], b[q][1], b[q][2], b[q][3]);
    }
};

__device__ __forceinline__ void copy16(uint32_t dst, const void *src) {
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(dst), "l"(src) : "memory");
}
__device__ __forceinline__ void copy_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int LEFT>
__device__ __forceinline__ void copy_wait() { asm volatile("cp.async.wait_group %0;" ::"n"(LEFT) : "memory"); }
__device__ __forceinline__ uint32_t smem_addr(const void *p) { return (uint32_t)__cvta_generic_to_shared(p); }

// acc += 16 output channels by 128 input channels (the codes wa, wb of a lane,
// over 64) times NT blocks of eight x rows.  xs[n]: this lane's row of block n in the
// first part, channel 8 t of the unit; part_step in bytes.  Lanes whose row
// does not exist read another: an MMA column is its own.  f0, f1: the unit's
// scales of rows g and g + 8.
template <typename X, int NT, int GROUP>
__device__ __forceinline__ void products(uint4 wa, uint4 wb, float (&acc)[NT][4], const uint8_t *const (&xs)[NT], int offset,
                                         int part_step, const float (&f0)[kUnit / GROUP], const float (&f1)[kUnit / GROUP]) {
    constexpr int kHalves = GROUP / 32;  // steps of 32 channels a scale
    float c[NT][4];
#pragma unroll
    for (int h = 0; h < 4; ++h) {
        const uint32_t lo = h == 0 ? wa.x : (h == 1 ? wa.z : (h == 2 ? wb.x : wb.z));
        const uint32_t hi = h == 0 ? wa.y : (h == 1 ? wa.w : (h == 2 ? wb.y : wb.w));
        uint32_t p[4], q[4];
        decode(lo, p);
        decode(hi, q);
#pragma unroll
        for (int n = 0; n < NT; ++n)
#pragma unroll
            for (int r = 0; r < X::kParts; ++r) {
                const uint4 b = *reinterpret_cast<const uint4 *>(xs[n] + offset + r * part_step + h * 64);
                if (h % kHalves == 0 && r == 0) mma16816_first(c[n], p[0], q[0], p[1], q[1], b.x, b.y);
                else mma16816(c[n], p[0], q[0], p[1], q[1], b.x, b.y);
                mma16816(c[n], p[2], q[2], p[3], q[3], b.z, b.w);
            }
        if (h % kHalves == kHalves - 1) {
            const float s0 = f0[h / kHalves], s1 = f1[h / kHalves];
#pragma unroll
            for (int n = 0; n < NT; ++n) {
                acc[n][0] = fmaf(s0, c[n][0], acc[n][0]);
                acc[n][1] = fmaf(s0, c[n][1], acc[n][1]);
                acc[n][2] = fmaf(s1, c[n][2], acc[n][2]);
                acc[n][3] = fmaf(s1, c[n][3], acc[n][3]);
            }
        }
    }
}

// N scales, side by side in shared memory.
template <int N, typename Elem>
__device__ __forceinline__ void load_scales(const uint8_t *p, float (&f)[N]) {
    struct alignas(N * sizeof(Elem)) Group { Elem v[N]; };
    const Group q = *reinterpret_cast<const Group *>(p);
#pragma unroll
    for (int j = 0; j < N; ++j) f[j] = elem_f(q.v[j]);
}

// CTAs of eight warps a SM: as many as their registers allow without spilling.
__host__ __device__ constexpr int few_ctas(int parts, int nt) { return nt * (parts == 3 ? 2 : 1) >= 4 ? 2 : 3; }
// Shared memory of w4_few before x: the warps' sums (two sides), their rings,
// and 16 rows of scales (two sides).
__host__ __device__ inline int few_sums(int warps, int nt) { return 2 * warps * nt * 128 * 4; }
__host__ __device__ inline int few_ring(int warps) { return warps * kAhead * 1024; }
// (a row of scales: whole units, zeros past the last group, and 16 bytes more,
// so that eight rows' same scales lie in different banks)
__host__ __device__ inline int scale_pitch(int units, int group, int es) { return (units * (kUnit / group) * es + 15) / 16 * 16 + 16; }
__host__ __device__ inline int few_scales(int units, int group, int es) { return 16 * scale_pitch(units, group, es); }

template <typename X, int NT, int GROUP, int WARPS>
__global__ void __launch_bounds__(WARPS * 32, WARPS == 8 ? few_ctas(X::kParts, NT) : 1) w4_few_kernel(W4Args a, int vec) {
    using Elem = typename X::Elem;
    constexpr int kThreads = WARPS * 32, kSum = WARPS * NT * 128, kGroups = kUnit / GROUP;
    extern __shared__ __align__(16) uint8_t shm[];
    float *red = reinterpret_cast<float *>(shm);
    const int spitch = scale_pitch(a.units, GROUP, (int)sizeof(Elem)), sside = 16 * spitch;
    uint8_t *scales = shm + few_sums(WARPS, NT) + few_ring(WARPS);
    uint8_t *xs = scales + 2 * sside;                     // [parts][rows] of pitch bytes
    const int pitch = a.units * kUnit * 2 + kPad, part_step = a.rows * pitch;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, g = lane >> 2, t = lane & 3;
    uint4 *ring = reinterpret_cast<uint4 *>(shm + few_sums(WARPS, NT) + warp * (kAhead * 1024)) + lane;
    pdl_trigger();
    pdl_wait();
    const Elem *x = static_cast<const Elem *>(a.x);
    const Elem *sc = static_cast<const Elem *>(a.scales);
    const int per = (a.units - warp + WARPS - 1) / WARPS;  // this warp's units of a tile
    // what is left to ask for, and where the next unit lies
    int left = ((a.tiles - 1 - (int)blockIdx.x) / (int)gridDim.x + 1) * per, fi = per;
    uint32_t fslot = 0;
    const uint32_t ring0 = smem_addr(ring);
    const uint4 *fw = a.w + ((long long)blockIdx.x * a.units + warp) * 64 + lane;
    const long long jump = ((long long)gridDim.x * a.units - (long long)per * WARPS) * 64;  // from a tile's end to the next
    auto ask = [&]() {
        if (left > 0) {
            copy16(ring0 + fslot, fw);
            copy16(ring0 + fslot + 512, fw + 32);
            fw += WARPS * 64;
            --left;
            if (--fi == 0) {
                fi = per;
                fw += jump;
            }
        }
        copy_commit();
        fslot = (fslot + 1024) & (kAhead * 1024 - 1);
    };
    // 16 rows of scales (rows past the last: as they are, for outputs that
    // nobody stores)
    const bool svec = (reinterpret_cast<uintptr_t>(sc) & 15u) == 0 && a.ng * (int)sizeof(Elem) % 16 == 0;
    auto ask_scales = [&](int tile, int side) {
        if (tile >= a.tiles) return;
        const Elem *src = sc + (long long)tile * 16 * a.ng;
        uint8_t *d = scales + side * sside;
        const int rows = min(16, a.co - tile * 16), n = svec ? a.ng * (int)sizeof(Elem) / 16 : a.ng;
        for (int i = threadIdx.x; i < rows * n; i += kThreads) {
            const int r = i / n, e = i - r * n;
            if (svec) copy16(smem_addr(d + r * spitch) + 16 * e, reinterpret_cast<const uint8_t *>(src + (long long)r * a.ng) + 16 * e);
            else reinterpret_cast<Elem *>(d + r * spitch)[e] = src[(long long)r * a.ng + e];
        }
    };
    for (int i = threadIdx.x; i < 32 * (a.units * kGroups - a.ng); i += kThreads)
        reinterpret_cast<Elem *>(scales + (i & 31) * spitch)[a.ng + (i >> 5)] = elem_from<Elem>(0.0f);
    ask_scales(blockIdx.x, 0);
#pragma unroll
    for (int i = 0; i < kAhead - 1; ++i) ask();  // (the first group holds the scales too)
    // x into shared memory, eight channels a thread at a time, four times over
    // before the first is used
    const int eights = a.units * (kUnit / 8), items = a.rows * eights;
    for (int i = threadIdx.x; i < items; i += 4 * kThreads) {
        typename X::Raw raw[4];
#pragma unroll
        for (int q = 0; q < 4; ++q) {
            const int j = i + q * kThreads, m = j / eights;
            if (j < items) raw[q] = X::fetch(x + (long long)m * a.ci, (j - m * eights) * 8, a.ci, vec != 0);
        }
#pragma unroll
        for (int q = 0; q < 4; ++q) {
            const int j = i + q * kThreads, m = j / eights;
            if (j >= items) continue;
            uint4 v[X::kParts];
            X::parts(raw[q], v);
#pragma unroll
            for (int r = 0; r < X::kParts; ++r) *reinterpret_cast<uint4 *>(xs + r * part_step + m * pitch + (j - m * eights) * 16) = v[r];
        }
    }
    copy_wait<kAhead - 2>();
    __syncthreads();
    const uint8_t *xl[NT];
    float acc[NT][4];
#pragma unroll
    for (int n = 0; n < NT; ++n) {
        xl[n] = xs + min(n * 8 + g, a.rows - 1) * pitch + t * 16;
#pragma unroll
        for (int e = 0; e < 4; ++e) acc[n][e] = 0.0f;
    }
    int side = 0;
    uint32_t slot = 0;
    for (int tile = blockIdx.x; tile < a.tiles; tile += gridDim.x, side ^= 1) {
        ask_scales(tile + gridDim.x, side ^ 1);  // (joins the next group; complete before this tile's barrier)
        const uint8_t *sl = scales + side * sside + g * spitch;
        for (int u = warp; u < a.units; u += WARPS) {
            copy_wait<kAhead - 2>();
            const uint4 wa = ring[slot], wb = ring[slot + 32];
            slot = (slot + 64) & (kAhead * 64 - 1);
            float f0[kGroups], f1[kGroups];
            load_scales<kGroups, Elem>(sl + u * (kGroups * (int)sizeof(Elem)), f0);
            load_scales<kGroups, Elem>(sl + 8 * spitch + u * (kGroups * (int)sizeof(Elem)), f1);
            products<X, NT, GROUP>(wa, wb, acc, xl, u * (kUnit * 2), part_step, f0, f1);
            ask();  // into the slot read last time
        }
        // the tile's sums: one barrier a tile, two sides in turn (a side is
        // written again only after the next tile's barrier)
        float *mine = red + side * kSum + warp * (NT * 128);
#pragma unroll
        for (int n = 0; n < NT; ++n) {
            mine[(n * 8 + 2 * t) * 16 + g] = acc[n][0];
            mine[(n * 8 + 2 * t + 1) * 16 + g] = acc[n][1];
            mine[(n * 8 + 2 * t) * 16 + g + 8] = acc[n][2];
            mine[(n * 8 + 2 * t + 1) * 16 + g + 8] = acc[n][3];
#pragma unroll
            for (int e = 0; e < 4; ++e) acc[n][e] = 0.0f;
        }
        if (per < kAhead) {  // the next scales may be in a group still on the way, or in none
            copy_commit();
            copy_wait<0>();
        }
        __syncthreads();
        for (int o = threadIdx.x; o < a.rows * 16; o += kThreads) {
            const int m = o >> 4, co = tile * 16 + (o & 15);
            if (co >= a.co) continue;
            float v = 0.0f;
#pragma unroll
            for (int q = 0; q < WARPS; ++q) v += red[side * kSum + q * (NT * 128) + o];
            v = act_out(fmaf(v, kCodeScale, a.bias ? a.bias[co] : 0.0f), a.act);
            static_cast<Elem *>(a.y)[(long long)m * a.co + co] = elem_from<Elem>(v);
        }
    }
    copy_wait<0>();
}

// WC: co tiles of a CTA; its eight warps take k in turns of WK = 8 / WC units.
__host__ __device__ constexpr int many_smem(int parts, int nt, int wc) {
    const int x = 3 * parts * nt * 8 * (8 / wc * kUnit * 2 + kPad), ring = 8 * kAhead * 1024, sums = 8 * nt * 128 * 4;
    return ring + x > sums ? ring + x : sums;
}
// CTAs a SM that registers are kept for: one with eight blocks of rows (more
// than 128 registers), and with four whose shared memory leaves room for one
// CTA; else two.
// Left to itself the compiler held some to 80 registers for three CTAs: over 136
// sizes of 10 to 64 rows this takes 0.89 of the time (64 rows of 8192x8192 bf16
// 41.7 us against 63.1, 32 of 4096x16384 22.7 against 33.7, 64 of 8192x28672 143
// against 165; the worst, 10 of 8192x28672 in groups of 64, 60.9 against 58.4).
// Two everywhere: 24 of 8192x8192 37.3 against 33.3; one wherever two do not fit:
// 32 of 8192x8192 fp32, groups of 64, 103 against 75.
__host__ __device__ constexpr int many_ctas(int parts, int nt, int wc) {
    return nt >= 8 || (nt >= 4 && 2 * (many_smem(parts, nt, wc) + 1024) > 227 * 1024) ? 1 : 2;
}
template <typename X, int NT, int GROUP, int WC>
__global__ void __launch_bounds__(256, many_ctas(X::kParts, NT, WC)) w4_many_kernel(W4Args a, int vec) {
    using Elem = typename X::Elem;
    constexpr int WK = 8 / WC, kTurn = WK * kUnit, kPitch = kTurn * 2 + kPad, kGroups = kUnit / GROUP;
    constexpr int kPart = NT * 8 * kPitch, kSide = X::kParts * kPart;
    extern __shared__ __align__(16) uint8_t shm[];  // rings, then x [3][parts][8 NT] rows of kPitch bytes; at the end the warps' sums
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, g = lane >> 2, t = lane & 3;
    const int wc = warp % WC, wk = warp / WC;
    uint4 *ring = reinterpret_cast<uint4 *>(shm + warp * (kAhead * 1024)) + lane;
    uint8_t *xs = shm + 8 * kAhead * 1024;
    const int m0 = blockIdx.y * (NT * 8), rows = min(NT * 8, a.rows - m0);
    const int tile = blockIdx.x * WC + wc;
    const int turns = (a.units + WK - 1) / WK;
    pdl_trigger();
    pdl_wait();
    const Elem *x = static_cast<const Elem *>(a.x) + (long long)m0 * a.ci;
    const int r0 = min(tile * 16 + g, a.co - 1), r1 = min(tile * 16 + g + 8, a.co - 1);  // (rows past the last are not stored)
    const Elem *s0 = static_cast<const Elem *>(a.scales) + (long long)r0 * a.ng, *s1 = static_cast<const Elem *>(a.scales) + (long long)r1 * a.ng;
    const uint4 *fw = a.w + ((long long)tile * a.units + wk) * 64 + lane;
    int fu = tile < a.tiles ? wk : a.units, fslot = 0;
    auto ask = [&]() {
        if (fu < a.units) {
            const uint32_t d = smem_addr(ring + fslot * 64);
            copy16(d, fw);
            copy16(d + 512, fw + 32);
            fw += WK * 64;
            fu += WK;
        }
        copy_commit();
        fslot = fslot + 1 == kAhead ? 0 : fslot + 1;
    };
    // A turn's x: copied as it is (cp.async) where it can be, else fetched into
    // registers before the products of the turn at hand and written after them.
    const bool straight = X::kParts == 1 && vec && a.ci % 8 == 0;
    constexpr int kItems = (NT * 8 * (kTurn / 8) + 255) / 256, kHeld = kItems < 4 ? kItems : 4;
    typename X::Raw held[kHeld];
    auto each = [&](int from, int count, auto &&use) {
#pragma unroll
        for (int q = 0; q < count; ++q) {
            const int i = threadIdx.x + (from + q) * 256, m = i / (kTurn / 8);
            if (m < rows) use(q, m, (i % (kTurn / 8)) * 8);
        }
    };
    auto store = [&](int turn, int m, int kk, const typename X::Raw &r) {
        uint4 v[X::kParts];
        X::parts(r, v);
#pragma unroll
        for (int p = 0; p < X::kParts; ++p)
            *reinterpret_cast<uint4 *>(xs + turn % 3 * kSide + p * kPart + m * kPitch + kk * 2) = v[p];
    };
    auto begin = [&](int turn) {
        if (straight) {
            each(0, kItems, [&](int, int m, int kk) {
                const int k = turn * kTurn + kk;
                uint8_t *d = xs + turn % 3 * kSide + m * kPitch + kk * 2;
                if (k < a.ci) copy16(smem_addr(d), x + (long long)m * a.ci + k);
                else *reinterpret_cast<uint4 *>(d) = make_uint4(0u, 0u, 0u, 0u);
            });
        } else {
            each(0, kHeld, [&](int q, int m, int kk) { held[q] = X::fetch(x + (long long)m * a.ci, turn * kTurn + kk, a.ci, vec != 0); });
        }
    };
    auto end = [&](int turn) {
        if (straight) return;
        each(0, kHeld, [&](int q, int m, int kk) { store(turn, m, kk, held[q]); });
        for (int f = kHeld; f < kItems; ++f)
            each(f, 1, [&](int, int m, int kk) { store(turn, m, kk, X::fetch(x + (long long)m * a.ci, turn * kTurn + kk, a.ci, vec != 0)); });
    };
    float acc[NT][4];
    int row[NT];
#pragma unroll
    for (int n = 0; n < NT; ++n) {
        row[n] = min(n * 8 + g, rows - 1) * kPitch + t * 16 + wk * (kUnit * 2);
#pragma unroll
        for (int e = 0; e < 4; ++e) acc[n][e] = 0.0f;
    }
    // x goes two turns ahead, the weights three: x of turn T is in the group
    // before the last when turn T begins
    begin(0);
    end(0);
    ask();
    if (turns > 1) {
        begin(1);
        end(1);
    }
    ask();
    ask();
    int slot = 0;
    float f0[kGroups], f1[kGroups];
    auto scales = [&](int u) {
#pragma unroll
        for (int j = 0; j < kGroups; ++j) {
            const int gi = min(u * kGroups + j, a.ng - 1);
            f0[j] = elem_f(s0[gi]);
            f1[j] = elem_f(s1[gi]);
        }
    };
    scales(wk);
    for (int turn = 0; turn < turns; ++turn) {
        copy_wait<1>();
        __syncthreads();  // ... for every thread, and everyone has left the side that is staged next
        if (turn + 2 < turns) begin(turn + 2);
        const int u = turn * WK + wk;
        float c0[kGroups], c1[kGroups];
#pragma unroll
        for (int j = 0; j < kGroups; ++j) { c0[j] = f0[j]; c1[j] = f1[j]; }
        scales(u + WK);
        const uint4 wa = ring[slot * 64], wb = ring[slot * 64 + 32];
        slot = slot + 1 == kAhead ? 0 : slot + 1;
        if (u < a.units && tile < a.tiles) {
            const uint8_t *xl[NT];
#pragma unroll
            for (int n = 0; n < NT; ++n) xl[n] = xs + turn % 3 * kSide + row[n];
            products<X, NT, GROUP>(wa, wb, acc, xl, 0, kPart, c0, c1);
        }
        if (turn + 2 < turns) end(turn + 2);
        ask();
    }
    copy_wait<0>();
    if constexpr (WK > 1) {  // the turns' sums, in order
        float *red = reinterpret_cast<float *>(shm);  // [8][NT * 128]
        __syncthreads();
#pragma unroll
        for (int n = 0; n < NT; ++n)
#pragma unroll
            for (int e = 0; e < 4; ++e) red[warp * (NT * 128) + (n * 4 + e) * 32 + lane] = acc[n][e];
        __syncthreads();
        if (wk > 0) return;
#pragma unroll
        for (int n = 0; n < NT; ++n)
#pragma unroll
            for (int e = 0; e < 4; ++e)
                for (int q = 1; q < WK; ++q) acc[n][e] += red[(q * WC + wc) * (NT * 128) + (n * 4 + e) * 32 + lane];
    }
    if (tile >= a.tiles) return;
#pragma unroll
    for (int n = 0; n < NT; ++n)
#pragma unroll
        for (int e = 0; e < 4; ++e) {
            const int m = n * 8 + 2 * t + (e & 1), c = tile * 16 + g + (e >> 1) * 8;
            if (m < rows && c < a.co)
                static_cast<Elem *>(a.y)[(long long)(m0 + m) * a.co + c] =
                    elem_from<Elem>(act_out(fmaf(acc[n][e], kCodeScale, a.bias ? a.bias[c] : 0.0f), a.act));
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

// max(a, b), NaN if either is.
__device__ __forceinline__ float max_nan(float a, float b) {
    float r;
    asm("max.NaN.f32 %0, %1, %2;" : "=f"(r) : "f"(a), "f"(b));
    return r;
}

// Codes and scales of a weight row's group, one warp a group: s = max |w| / 7
// rounded to the scales' type, u = clamp(round_half_even(w / s), -8, 7) + 8.
// A NaN or an infinity among the weights is the scale's too, and every code of
// its group is 8: the layer answers 0 times that, NaN.
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
    for (int k = k0 + lane; k < k1; k += 32) top = max_nan(top, fabsf(elem_f(w[row * ci + k])));
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) top = max_nan(top, __shfl_xor_sync(0xffffffffu, top, o));
    const T s = elem_from<T>(top / 7.0f);
    const float sf = elem_f(s);
    if (lane == 0) scales[i] = s;
    for (int k = k0 + 2 * lane; k < k1; k += 64) {
        uint32_t byte = 0;
#pragma unroll
        for (int e = 0; e < 2; ++e) {
            int q = 0;
            if (k + e < k1 && sf > 0.0f && isfinite(sf)) q = max(-8, min(7, __float2int_rn(elem_f(w[row * ci + k + e]) / sf)));
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
template <typename X, int NT, int WC>
const void *many_group(int group) {
    return group == 32 ? (const void *)&w4_many_kernel<X, NT, 32, WC>
                       : (group == 64 ? (const void *)&w4_many_kernel<X, NT, 64, WC> : (const void *)&w4_many_kernel<X, NT, 128, WC>);
}
// (the shapes that a plan can choose: the others' x does not fit, see create)
template <typename X, int NT, int WC>
const void *many_fits(int group) {
    if constexpr (WC == 8 || many_smem(X::kParts, NT, WC) <= kSmemMost) return many_group<X, NT, WC>(group);
    else return nullptr;
}
template <typename X, int NT>
const void *many_wc(const W4Geom &g) {
    return g.wc == 8 ? many_fits<X, NT, 8>(g.group) : (g.wc == 4 ? many_fits<X, NT, 4>(g.group) : many_fits<X, NT, 2>(g.group));
}
template <typename X>
const void *pick(const W4Geom &g) {
    if (g.many) return g.nt == 1 ? many_wc<X, 1>(g) : (g.nt == 2 ? many_wc<X, 2>(g) : (g.nt == 4 ? many_wc<X, 4>(g) : many_wc<X, 8>(g)));
    return g.warps == 8 ? few_nt<X, 8>(g.nt, g.group) : few_nt<X, 16>(g.nt, g.group);
}

// 32-bit channel counts and unit indices, with room to round up.
bool too_large(int32_t c_in, int32_t c_out) {
    return c_in >= (1 << 28) || c_out >= (1 << 30) || (long long)c_in * c_out >= (1ll << 40);
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
    if (too_large(c_in, c_out) || rows >= (1 << 21)) return CONV_ERR_UNSUPPORTED;
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
    const int es = conv_esize(dtype);
    const long long xb = (long long)parts * rows * (g.units * (kUnit * 2) + kPad), sb = 2LL * few_scales(g.units, group, es);
    auto few = [&](int warps) { return xb + sb + few_sums(warps, g.nt) + few_ring(warps); };
    // x whole in shared memory while two CTAs of eight warps or one of sixteen
    // fit a SM, else in turns (fp32 rows, whose splitting is on the way of
    // every turn, only where not even eight warps fit).
    g.warps = few(8) <= 112 * 1024 || few(16) > kFewMost ? 8 : 16;
    g.many = rows > 32 || few(g.warps) > (parts == 3 || g.warps == 16 ? kFewMost : 112 * 1024);
    if (g.many) {
        g.warps = 8;
        auto smem = [&](int nt, int wc) { return many_smem(parts, nt, wc); };
        auto ctas = [&](int nt, int wc) { return (long long)((tiles + wc - 1) / wc) * ((rows + nt * 8 - 1) / (nt * 8)); };
        // until the card is full: fewer output channels a CTA and longer turns,
        // then fewer rows
        g.nt = rows <= 8 ? 1 : (rows <= 16 ? 2 : (rows <= 32 ? 4 : 8));
        g.wc = 8;
        while (ctas(g.nt, g.wc) < p->num_sms) {
            if (g.wc > 2 && smem(g.nt, g.wc / 2) <= kSmemMost) g.wc /= 2;
            else if (g.nt > 1) g.nt /= 2;
            else break;
        }
        g.smem = smem(g.nt, g.wc);
        g.grid = (tiles + g.wc - 1) / g.wc;
    } else {
        g.smem = (int)few(g.warps);
        int ctas = g.warps == 8 ? few_ctas(parts, g.nt) : 1;
        while (ctas > 1 && ctas * (g.smem + 1024) > 227 * 1024) --ctas;
        g.grid = tiles < ctas * p->num_sms ? tiles : ctas * p->num_sms;
    }
    const char *type = dtype == CONV_F32 ? "f32" : "bf16";
    if (g.many)
        snprintf(p->desc, sizeof(p->desc), "w4 %s group=%d x in turns rows=%dx8 warps=%d wc=%d tiles=%d ctas=%dx%d", type, group, g.nt,
                 g.warps, g.wc, tiles, g.grid, (rows + g.nt * 8 - 1) / (g.nt * 8));
    else
        snprintf(p->desc, sizeof(p->desc), "w4 %s group=%d x in shared memory rows=%dx8 warps=%d tiles=%d ctas=%d", type, group, g.nt,
                 g.warps, tiles, g.grid);
    *out_plan = p;
    return CONV_OK;
}

extern "C" int conv_w4_packed_bytes(int32_t c_in, int32_t c_out, size_t *bytes) {
    if (!bytes) return CONV_ERR_NULL_ARG;
    if (c_in < 1 || c_out < 1) return CONV_ERR_INVALID_SHAPE;
    if (too_large(c_in, c_out)) return CONV_ERR_UNSUPPORTED;
    *bytes = (size_t)((c_out + 15) / 16) * ((c_in + kUnit - 1) / kUnit) * 1024;
    return CONV_OK;
}

extern "C" int conv_w4_pack(int32_t c_in, int32_t c_out, const void *codes, void *packed, void *stream) {
    size_t bytes = 0;
    const int rc = conv_w4_packed_bytes(c_in, c_out, &bytes);
    if (rc != CONV_OK) return rc;
    if (!codes || !packed) return CONV_ERR_NULL_ARG;
    if ((uintptr_t)packed & 15u) return CONV_ERR_MISALIGNED;
    if (conv_overlaps(packed, bytes, codes, (size_t)c_out * ((c_in + 1) / 2))) return CONV_ERR_ALIASING;
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
    if (dtype == CONV_I8 || too_large(c_in, c_out)) return CONV_ERR_UNSUPPORTED;
    if (!w || !codes || !scales) return CONV_ERR_NULL_ARG;
    const size_t es = (size_t)conv_esize(dtype);
    if ((uintptr_t)w % es || (uintptr_t)scales % es) return CONV_ERR_MISALIGNED;
    int ng = (c_in + group - 1) / group;
    long long total = (long long)c_out * ng;
    if ((total + 7) / 8 > 0x7fffffffll) return CONV_ERR_UNSUPPORTED;
    const size_t wb = (size_t)c_in * c_out * es, cb = (size_t)c_out * ((c_in + 1) / 2), sb = (size_t)total * es;
    if (conv_overlaps(codes, cb, w, wb) || conv_overlaps(scales, sb, w, wb) || conv_overlaps(codes, cb, scales, sb)) return CONV_ERR_ALIASING;
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
    if (conv_overlaps(y, yb, x, (size_t)rows * ci * es) || conv_overlaps(y, yb, packed, pb) ||
        conv_overlaps(y, yb, scales, (size_t)co * p->w4.ng * es) || conv_overlaps(y, yb, bias, (size_t)co * 4))
        return CONV_ERR_ALIASING;
    const W4Geom &g = p->w4;
    W4Args a = {x, static_cast<const uint4 *>(packed), scales, bias, y, rows, ci, co, g.ng, g.units, p->act, (co + 15) / 16};
    int vec = ci % 8 == 0 && ((uintptr_t)x & 15u) == 0 ? 1 : 0;
    const void *k = p->dtype == CONV_F32 ? pick<XF32>(g) : pick<XBf16>(g);
    if (!k) return CONV_ERR_UNSUPPORTED;
    if (g.smem > 48 * 1024) {
        const int rc = conv_grant_smem_once(k, p->device, g.smem);
        if (rc != CONV_OK) return rc;
    }
    void *args[] = {&a, &vec};
    const dim3 grid((unsigned)g.grid, (unsigned)(g.many ? (rows + g.nt * 8 - 1) / (g.nt * 8) : 1));
    const cudaError_t e = conv_launch(k, grid, dim3(g.warps * 32), args, (size_t)g.smem, (cudaStream_t)stream);
    return e == cudaSuccess ? CONV_OK : CONV_ERR_CUDA;
}
