// What the kernels of the norms around a block share (k_blocknorm.cu, which has
// the formulas, and k_blocknorm_bwd.cu): arguments, how threads cover rows,
// sums over a row, and the norm of one.
#pragma once

#include <cuda_bf16.h>
#include <stdint.h>

#include "conv_internal.h"
#include "epilogue.cuh"
#include "maps.cuh"
#include "tc_ptx.cuh"

namespace bn {

using namespace convk;

constexpr int kMaxC = 8192;        // channels: 512 threads of 16
constexpr int kThreads = 256;      // of a forward CTA whose rows take no more
constexpr int kMostThreads = 512;  // of a row, and of the gradient's CTAs
constexpr int kCluster = 16;       // CTAs of a gradient in one launch, and the sets of rows that each takes at most
constexpr int kClusterSets = 2;
enum { SUM_A, SUM_B, SUM_G2, SUM_B2, SUMS };

struct BnArgs {
    const void *x, *f, *dy, *dz;   // f, dy and dz may be null
    void *o0, *o1;                 // y, z or dx, df; may be null
    long long px, pf, pdy, pdz, p0, p1;  // elements from one pixel to the next
    const float *scale, *gate, *g1, *b1, *g2, *b2;  // each may be null
    float4 *stats;                 // [rows] (m1, r1, m2, r2) (forward: may be null)
    float *part;                   // gradient: [units or CTAs][SUMS][C]
    float *dscale, *dgate, *dg1, *db1, *dg2, *db2;
    float eps, inv_c;
    int rows, HW, C, Cp, N;        // Cp: C in whole fours, of the workspace
    int post, pre;                 // conv_norm_t
    int tpr, slots, full;          // threads of a row, rows side by side; full: every thread has channels, all of them
    int run, S, units;             // rows of a unit, units an image (of all rows without a gate), units in all
    int whole;                     // gradient: a unit is a whole image of a gated map
    int want_b;                    // gradient: B is asked for
    int joined;                    // gradient: the CTAs are one cluster and join their sums themselves
    int last_t, last_v;            // where a row's last value is, of single ones: Lane::t and the vector
};

// Where a thread stands: which row of those side by side, which of the row's
// channels.  Vector v of a thread is number v * tpr + t of its row; pair i
// holds two consecutive channels of a vector (VEC = 1: of two vectors).
template <int VEC, int K>
struct Lane {
    static constexpr int NV = 8 * K / VEC, P = 4 * K;
    int tpr, t, slot, C;
    __device__ __forceinline__ explicit Lane(const BnArgs &a) : tpr(a.tpr), C(a.C) {
        slot = threadIdx.x / tpr;
        t = threadIdx.x - slot * tpr;
    }
    __device__ __forceinline__ int first(int v) const { return (v * tpr + t) * VEC; }
    __device__ __forceinline__ bool on(int v) const { return first(v) < C; }
    // (channels are whole vectors: a vector's are all in the row, or none)
    __device__ __forceinline__ bool has(int i, int h) const { return VEC == 1 ? on(2 * i + h) : on(i / (VEC < 2 ? 1 : VEC / 2)); }
    __device__ __forceinline__ int chan(int i, int h) const {
        if constexpr (VEC == 1) return first(2 * i + h);
        else return first(i / (VEC / 2)) + i % (VEC / 2) * 2 + h;
    }
    // src at the thread's channels (null: `other`), 0 beyond the row's end
    __device__ __forceinline__ void params(float2 (&v)[P], const float *src, float other) const {
        constexpr int W = VEC % 4 == 0 ? 4 : 1;
        if (W == 4 && src && (reinterpret_cast<uintptr_t>(src) & 15) == 0) {
#pragma unroll
            for (int i = 0; i < P; i += 2) {
                const float4 f = has(i, 0) ? *reinterpret_cast<const float4 *>(src + chan(i, 0)) : make_float4(0.0f, 0.0f, 0.0f, 0.0f);
                v[i] = make_float2(f.x, f.y);
                v[i + 1] = make_float2(f.z, f.w);
            }
            return;
        }
#pragma unroll
        for (int i = 0; i < P; ++i) {
            v[i].x = has(i, 0) ? (src ? src[chan(i, 0)] : other) : 0.0f;
            v[i].y = has(i, 1) ? (src ? src[chan(i, 1)] : other) : 0.0f;
        }
    }
};

// Bytes of an element in the ring.  Single bf16 values, which no asynchronous copy
// takes, come as the word that holds them (another two bytes of the same four, which
// are not used).
__host__ __device__ constexpr int ring_element(int es, int vec) { return es * vec < 4 ? 4 : es; }

// A thread's vectors of one row: from its ring of shared memory, to a map, and
// from a map to the ring.  Vectors beyond the row's end stay 0 in the ring.  CUT: of
// single bf16 values, a map starts in the middle of a word or ends in one; the half
// that is not the map's is not read.  (An instance of its own.  Forward beyond 2048
// channels it is 9 to 13 % slower: 4095x8191 117 us, 4096x8191, whose maps are whole
// words, 103; elsewhere up to 4 %.)
template <typename T, int VEC, int K, bool CUT = false>
struct Row {
    using V = Vec<T, VEC>;
    using Raw = typename V::Raw;
    using L = Lane<VEC, K>;
    static constexpr bool kWord = sizeof(Raw) < 4;
    using Slot = typename std::conditional<kWord, uint32_t, Raw>::type;
    static constexpr int NV = L::NV, P = L::P;
    static constexpr int kElement = ring_element(sizeof(T), VEC);
    static constexpr int step = 32;  // of a thread's vectors in the ring: a warp's lie together
    // the thread's first vector in a ring of `rows` rows
    __device__ static __forceinline__ Slot *ring(uint8_t *smem, int rows) {
        return reinterpret_cast<Slot *>(smem) + (threadIdx.x >> 5) * (rows * NV * step) + (threadIdx.x & 31);
    }
    // whether a thread's first value of a row is the high half of its word
    __device__ static __forceinline__ unsigned odd(const T *row) { return kWord ? (unsigned)(reinterpret_cast<uintptr_t>(row) >> 1) & 1u : 0u; }
    __device__ static __forceinline__ void get(const L &l, const Slot *src, unsigned odd, float2 (&f)[P]) {
#pragma unroll
        for (int v = 0; v < NV; ++v) {
            if constexpr (kWord) {
                const float one = __uint_as_float(src[v * step] << ((odd + v * l.tpr) & 1 ? 0 : 16) & 0xffff0000u);
                if (v % 2) f[v / 2].y = one;
                else f[v / 2].x = one;
            } else {
                float2 one[V::kPairs];
                V::unpack(src[v * step], one);
#pragma unroll
                for (int e = 0; e < V::kPairs; ++e) {
                    if constexpr (VEC == 1) {
                        if (v % 2) f[v / 2].y = one[0].x;
                        else f[v / 2].x = one[0].x;
                    } else f[v * V::kPairs + e] = one[e];
                }
            }
        }
    }
    // (row: the address of the thread's first vector)
    __device__ static __forceinline__ void put(const L &l, T *row, const float2 (&f)[P]) {
#pragma unroll
        for (int v = 0; v < NV; ++v) {
            float2 one[V::kPairs];
#pragma unroll
            for (int e = 0; e < V::kPairs; ++e) {
                if constexpr (VEC == 1) one[0].x = v % 2 ? f[v / 2].y : f[v / 2].x;
                else one[e] = f[v * V::kPairs + e];
            }
            if (l.on(v)) *reinterpret_cast<Raw *>(row + v * l.tpr * VEC) = V::pack(one);
        }
    }
    __device__ static __forceinline__ const void *word(const T *p) { return reinterpret_cast<const void *>(reinterpret_cast<uintptr_t>(p) & ~(uintptr_t)3); }
    // row: the address of the thread's first vector.  CUT: channels from `upto` on are
    // left out, and the first one where `late`; a map's ends are asked for apart.
    __device__ static __forceinline__ void ask(const L &l, const T *row, Slot *dst, int upto, bool late) {
#pragma unroll
        for (int v = 0; v < NV; ++v)
            if (CUT ? l.first(v) < upto && !(v == 0 && late) : l.on(v)) {
                const T *at = row + v * l.tpr * VEC;
                copy_async<(int)sizeof(Slot)>(tc::smem_u32(dst + v * step), kWord ? word(at) : at);
            }
    }
    // A map's last value, and its first (alone: the only one).
    __device__ static __forceinline__ void ask_last(const T *at, Slot *dst) { copy_async_part(tc::smem_u32(dst), word(at), odd(at) ? 4 : 2); }
    __device__ static __forceinline__ void ask_first(const T *at, Slot *dst, bool alone) {
        if (odd(at)) *reinterpret_cast<uint32_t *>(dst) = (uint32_t)*reinterpret_cast<const uint16_t *>(at) << 16;
        else copy_async_part(tc::smem_u32(dst), word(at), alone ? 2 : 4);
    }
    // the vectors beyond the row's end in `rows` rows of the ring
    template <int ROWS>
    __device__ static __forceinline__ void blank(const L &l, Slot *dst) {
#pragma unroll
        for (int v = 0; v < NV; ++v)
            if (!l.on(v))
                for (int i = 0; i < ROWS; ++i) dst[(i * NV + v) * step] = Slot{};
    }
    __device__ static __forceinline__ void zero(Slot *dst) {
#pragma unroll
        for (int v = 0; v < NV; ++v) dst[v * step] = Slot{};
    }
};

// Rows of a part of a warp, of a warp, of several; any of these; of two CTAs
// (the gradient's beyond 4096 channels).
enum { ROW_PART, ROW_WARP, ROW_WARPS, ROW_ANY, ROW_PAIR };

// Two sums over the threads of a row, to all of them.  The first exchange
// leaves one sum to each half of the lanes, which halves the exchanges.  Rows of
// more than a warp then meet in one of two sets of shared entries in turn, a pair
// of warps an entry: whoever writes an entry again has passed the barrier of the
// other set, and with it everyone's reading of this one.
constexpr int kMeet = 12;  // entries of a set: an odd number of warps a row leaves halves empty
template <int ROW, bool FEW = true>
struct RowSum {
    int tpr, slot, pairs;
    float4 *buf;  // [2][kMeet] (two sums of a warp, two of the next)
    int flip;
    __device__ __forceinline__ RowSum(int tpr_, int slot_, float4 *b) : tpr(tpr_), slot(slot_), pairs((tpr_ / 32 + 1) / 2), buf(b + slot_ * pairs), flip(0) {
        if (ROW >= ROW_WARPS && tpr > 32 && (tpr / 32) % 2 && threadIdx.x - slot * tpr < 2)  // (ordered by the first barrier)
            reinterpret_cast<float2 *>(buf + (threadIdx.x - slot * tpr) * kMeet + pairs - 1)[1] = make_float2(0.0f, 0.0f);
    }
    __device__ static __forceinline__ float across(float v, int o) { return __shfl_xor_sync(0xffffffffu, v, o); }
    __device__ __forceinline__ float2 operator()(float a, float b) {
        const int lane = threadIdx.x & 31;
        if (ROW == ROW_PART || (ROW == ROW_ANY && tpr < 32)) {
            if (tpr == 1) return make_float2(a, b);
            const int top = tpr >> 1;
            const bool hi = lane & top;
            float v = (hi ? b : a) + across(hi ? a : b, top);
            for (int o = top >> 1; o > 0; o >>= 1) v += across(v, o);
            const float w = across(v, top);
            return hi ? make_float2(w, v) : make_float2(v, w);
        }
        const bool hi = lane & 16;
        float v = (hi ? b : a) + across(hi ? a : b, 16);
#pragma unroll
        for (int o = 8; o > 0; o >>= 1) v += across(v, o);
        if (ROW == ROW_WARPS || (ROW == ROW_ANY && tpr > 32)) {
            float4 *e = buf + flip;
            flip ^= kMeet;
            if ((lane & 15) == 0) reinterpret_cast<float *>(e)[(threadIdx.x - slot * tpr) / 32 * 2 + (lane >> 4)] = v;
            asm volatile("bar.sync %0, %1;" ::"r"(1 + slot), "r"(tpr) : "memory");
            // up to six warps: every thread reads them all (8x40x40x512 bf16 12.5 us
            // forward, 14.0 where lanes read one each and exchange; 4096 channels,
            // sixteen warps, 57 and 54).  FEW false spares registers.
            if (FEW && pairs <= 3) {
                float2 s = make_float2(0.0f, 0.0f);
                for (int i = 0; i < pairs; ++i) {
                    const float4 f = e[i];
                    s = add2(s, add2(make_float2(f.x, f.y), make_float2(f.z, f.w)));
                }
                return s;
            }
            const int k = lane & 15;
            v = k < 2 * pairs ? reinterpret_cast<const float *>(e)[k * 2 + (lane >> 4)] : 0.0f;
#pragma unroll
            for (int o = 8; o > 0; o >>= 1) v += across(v, o);
        }
        const float w = across(v, 16);
        return hi ? make_float2(w, v) : make_float2(v, w);
    }
};

__device__ __forceinline__ float2 both(float v) { return make_float2(v, v); }
template <int P>
__device__ __forceinline__ float total(const float2 (&v)[P]) {
    float2 s = v[0];
#pragma unroll
    for (int i = 1; i < P; ++i) s = add2(s, v[i]);
    return s.x + s.y;
}

// m and r of one norm of RB rows (1 or 2), and the values normalised in place.
template <int VEC, int K, int RB, typename SUM>
__device__ __forceinline__ void normalise(const Lane<VEC, K> &l, SUM &sum, float2 (&v)[RB][4 * K], int kind, const BnArgs &a,
                                          float2 (&mr)[RB]) {
    constexpr int P = 4 * K;
    float2 m = make_float2(0.0f, 0.0f);
    if (kind == CONV_NORM_LAYER) {
        m = mul2(sum(total(v[0]), RB > 1 ? total(v[RB - 1]) : 0.0f), both(a.inv_c));
#pragma unroll
        for (int b = 0; b < RB; ++b)
#pragma unroll
            for (int i = 0; i < P; ++i) v[b][i] = add2(v[b][i], both(b ? -m.y : -m.x));
        if (!a.full)
#pragma unroll
            for (int b = 0; b < RB; ++b)
#pragma unroll
                for (int i = 0; i < P; ++i) {
                    if (!l.has(i, 0)) v[b][i].x = 0.0f;
                    if (!l.has(i, 1)) v[b][i].y = 0.0f;
                }
    }
    float q[RB];
#pragma unroll
    for (int b = 0; b < RB; ++b) {
        float2 s = mul2(v[b][0], v[b][0]);
#pragma unroll
        for (int i = 1; i < P; ++i) s = fma2(v[b][i], v[b][i], s);
        q[b] = s.x + s.y;
    }
    const float2 s = sum(q[0], RB > 1 ? q[RB - 1] : 0.0f);
#pragma unroll
    for (int b = 0; b < RB; ++b) {
        const float r = __frsqrt_rn(fmaf(b ? s.y : s.x, a.inv_c, a.eps));
        mr[b] = make_float2(b ? m.y : m.x, r);
#pragma unroll
        for (int i = 0; i < P; ++i) v[b][i] = mul2(v[b][i], both(r));
    }
}

// scale gate g1 and scale gate b1 at a thread's channels.
template <int VEC, int K>
__device__ __forceinline__ void factors(const Lane<VEC, K> &l, const BnArgs &a, int n, float2 (&q)[4 * K], float2 (&p)[4 * K]) {
    constexpr int P = 4 * K;
    float2 s[P], g[P];
    l.params(s, a.scale, 1.0f);
    l.params(g, a.gate ? a.gate + (long long)n * a.C : nullptr, 1.0f);
    l.params(q, a.g1, 1.0f);
    l.params(p, a.b1, 0.0f);
#pragma unroll
    for (int i = 0; i < P; ++i) {
        const float2 sg = mul2(s[i], g[i]);
        q[i] = mul2(q[i], sg);
        p[i] = mul2(p[i], sg);
    }
}

// Stages of the gradient's ring: what fits beside one another in shared memory,
__host__ __device__ constexpr int bwd_stages() { return 3; }

// ... and of the forward kernel's.
__host__ __device__ constexpr int fwd_stages(int es, int k) { return k == 2 && es == 4 ? 2 : 3; }

// The gradient's kernel for a vector width (cut: as Row's, of single bf16 values) and
// tpr threads a row (or half a row, of a pair of CTAs), and the launch that joins its
// sums.
const void *pick_bwd(conv_dtype_t dt, int vec, bool cut, bool pair, int tpr, bool all);
cudaError_t launch_join(const BnArgs &a, int parts, cudaStream_t st);

}  // namespace bn
