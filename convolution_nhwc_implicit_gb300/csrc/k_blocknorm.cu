// The norms before and after a block, fused with the block's gate, its residual
// scale and the residual add, over NHWC maps: forward and gradient.
//
// With x the residual stream, f the block's output, each pixel a row of C
// channels, and norms of kind layer (mean and deviation), rms (m = 0) or none
// (m = 0, r = 1):
//   u^ = (f - m1) r1        u = g1 u^ + b1
//   y  = x + scale[c] gate[n,c] u
//   y^ = (y - m2) r2        z = g2 y^ + b2
// and, with dy and dz,
//   e  = g2 dz              dY = dy + r2 (e - [layer] mean e - y^ mean(e y^))
//   v  = scale gate g1 dY   df = r1 (v - [layer] mean v - u^ mean(v u^))
//   dx = dY
//   dg2 = sum dz y^         db2 = sum dz
//   A[n,c] = sum_p dY u^    B[n,c] = sum_p dY
//   dgate = scale (g1 A + b1 B)          dscale = sum_n gate (g1 A + b1 B)
//   dg1 = sum_n scale gate A             db1 = sum_n scale gate B
// The gradient forms y again of x and f, which is as many bytes as reading y
// and spares its rounding.  About 20 operations an element forward and 45
// backward against 8 to 24 bytes moved: memory bounds it.
//
// A thread holds 8 K channels of a row and the channels' sums over its rows; a
// row is shared by as many threads as that takes (lanes of a warp, or whole
// warps that meet in shared memory), and a CTA takes several rows side by side.
// All statistics and sums are fp32, in a fixed order: results do not change
// from run to run.
#include <cuda_bf16.h>
#include <math.h>
#include <stdint.h>
#include <stdio.h>

#include <new>

#include "conv_internal.h"
#include "epilogue.cuh"
#include "maps.cuh"
#include "tc_ptx.cuh"

using namespace convk;

namespace {

constexpr int kMaxC = 8192;        // channels: 512 threads of 16
constexpr int kThreads = 256;      // of a forward CTA whose rows take no more
constexpr int kMostThreads = 512;  // of a row, and of the gradient's CTAs
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

// A thread's vectors of one row: from its ring of shared memory, to a map, and
// from a map to the ring.  Vectors beyond the row's end stay 0 in the ring.
template <typename T, int VEC, int K>
struct Row {
    using V = Vec<T, VEC>;
    using Raw = typename V::Raw;
    using L = Lane<VEC, K>;
    static constexpr int NV = L::NV, P = L::P;
    static constexpr int step = 32;  // of a thread's vectors in the ring: a warp's lie together
    // the thread's first vector in a ring of `rows` rows
    __device__ static __forceinline__ Raw *ring(uint8_t *smem, int rows) {
        return reinterpret_cast<Raw *>(smem) + (threadIdx.x >> 5) * (rows * NV * step) + (threadIdx.x & 31);
    }
    __device__ static __forceinline__ void get(const Raw *src, float2 (&f)[P]) {
#pragma unroll
        for (int v = 0; v < NV; ++v) {
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
    __device__ static __forceinline__ void ask(const L &l, const T *row, Raw *dst) {
#pragma unroll
        for (int v = 0; v < NV; ++v)
            if (l.on(v)) copy_vec(dst + v * step, reinterpret_cast<const Raw *>(row + v * l.tpr * VEC));
    }
    // the vectors beyond the row's end in `rows` rows of the ring
    template <int ROWS>
    __device__ static __forceinline__ void blank(const L &l, Raw *dst) {
#pragma unroll
        for (int v = 0; v < NV; ++v)
            if (!l.on(v))
                for (int i = 0; i < ROWS; ++i) dst[(i * NV + v) * step] = Raw{};
    }
    __device__ static __forceinline__ void zero(Raw *dst) {
#pragma unroll
        for (int v = 0; v < NV; ++v) dst[v * step] = Raw{};
    }
};

// Rows of a part of a warp, of a warp, of several; or any of these.
enum { ROW_PART, ROW_WARP, ROW_WARPS, ROW_ANY };

// Two sums over the threads of a row, to all of them.  The first exchange
// leaves one sum to each half of the lanes, which halves the exchanges.  Rows of
// more than a warp then meet in one of two sets of shared entries in turn:
// whoever writes an entry again has passed the barrier of the other set, and
// with it everyone's reading of this one.
template <int ROW>
struct RowSum {
    int tpr, slot;
    float *buf;  // [2][warps][2]
    int flip;
    __device__ __forceinline__ RowSum(int tpr_, int slot_, float *b) : tpr(tpr_), slot(slot_), buf(b), flip(0) {}
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
            float *e = buf + flip;
            flip ^= kMostThreads / 32 * 2;
            if ((lane & 15) == 0) e[(threadIdx.x >> 5) * 2 + (lane >> 4)] = v;
            asm volatile("bar.sync %0, %1;" ::"r"(1 + slot), "r"(tpr) : "memory");
            const int n = tpr >> 5, k = lane & 15;
            v = k < n ? e[(slot * n + k) * 2 + (lane >> 4)] : 0.0f;
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
template <int VEC, int K, int RB, int ROW>
__device__ __forceinline__ void normalise(const Lane<VEC, K> &l, RowSum<ROW> &sum, float2 (&v)[RB][4 * K], int kind, const BnArgs &a,
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

constexpr int kFwdStages = 3;

// y and z of a run of rows, RB at a time.  ANY: the rows of a gated map that a
// CTA takes may be of several images (RB = 1); otherwise a run is of one.
template <typename T, int VEC, int K, int RB>
__global__ void __launch_bounds__(kMostThreads) bn_fwd_kernel(const __grid_constant__ BnArgs a) {
    using R = Row<T, VEC, K>;
    using Raw = typename R::Raw;
    constexpr int P = R::P, D = kFwdStages, LINE = R::NV * R::step, STAGE = 2 * RB * LINE;
    extern __shared__ __align__(16) uint8_t smem[];
    __shared__ float meet[2 * kMostThreads / 32 * 2];
    Raw *ring = R::ring(smem, D * 2 * RB);  // [D][x, f][RB]
    const Lane<VEC, K> l(a);
    RowSum<ROW_ANY> sum(a.tpr, l.slot, meet);
    const int n = RB > 1 ? blockIdx.x / a.S : 0, s0 = RB > 1 ? blockIdx.x - n * a.S : blockIdx.x;
    const int span = RB > 1 && a.S < a.units ? a.HW : a.rows;
    const int r0 = n * span + s0 * a.run, r1 = n * span + min(span, (s0 + 1) * a.run);
    int row = r0 + l.slot, asked = row;
    const bool block = a.f != nullptr;
    const T *x = static_cast<const T *>(a.x) + row * a.px + l.first(0), *f = static_cast<const T *>(a.f) + row * a.pf + l.first(0);
    T *y = static_cast<T *>(a.o0) + row * a.p0 + l.first(0), *z = static_cast<T *>(a.o1) + row * a.p1 + l.first(0);
    const long long sx = a.slots * a.px, sf = a.slots * a.pf, sy = a.slots * a.p0, sz = a.slots * a.p1;
    pdl_trigger();
    if (!a.full) R::template blank<D * 2 * RB>(l, ring);
    pdl_wait();
    const Raw *d = ring;
    Raw *to = ring;
    auto ask = [&] {
#pragma unroll
        for (int b = 0; b < RB; ++b) {
            if (asked < r1) {
                R::ask(l, x, to + b * LINE);
                if (block) R::ask(l, f, to + (RB + b) * LINE);
            }
            asked += a.slots;
            x += sx;
            f += sf;
        }
        copy_commit();
        to = to == ring + (D - 1) * STAGE ? ring : to + STAGE;
    };
#pragma unroll
    for (int i = 0; i < D - 1; ++i) ask();
    float2 q[P], p[P], g2[P], b2[P];
    int image = n;
    const bool by_row = RB == 1 && a.gate;
    if (by_row) image = min(row, a.rows - 1) / a.HW;
    if (block) factors(l, a, image, q, p);
    l.params(g2, a.g2, 1.0f);
    l.params(b2, a.b2, 0.0f);
    for (int base = r0; base < r1; base += a.slots * RB) {
        copy_wait<D - 2>();
        float2 v[RB][P], u[RB][P];
#pragma unroll
        for (int b = 0; b < RB; ++b) {
            R::get(d + b * LINE, v[b]);
            if (block) R::get(d + (RB + b) * LINE, u[b]);
        }
        d = d == ring + (D - 1) * STAGE ? ring : d + STAGE;
        ask();
        float2 one[RB], two[RB];
#pragma unroll
        for (int b = 0; b < RB; ++b) one[b] = two[b] = make_float2(0.0f, 1.0f);
        if (block) {
            if (by_row && row < r1) {
                const int k = row / a.HW;
                if (k != image) factors(l, a, image = k, q, p);
            }
            if (a.post != CONV_NORM_NONE) normalise<VEC, K, RB>(l, sum, u, a.post, a, one);
            if (a.b1)
#pragma unroll
                for (int b = 0; b < RB; ++b)
#pragma unroll
                    for (int i = 0; i < P; ++i) v[b][i] = add2(v[b][i], p[i]);
#pragma unroll
            for (int b = 0; b < RB; ++b)
#pragma unroll
                for (int i = 0; i < P; ++i) v[b][i] = fma2(q[i], u[b][i], v[b][i]);
            if (a.o0)
#pragma unroll
                for (int b = 0; b < RB; ++b)
                    if (row + b * a.slots < r1) R::put(l, y + b * sy, v[b]);
        }
        if (a.o1) {
            normalise<VEC, K, RB>(l, sum, v, a.pre, a, two);
#pragma unroll
            for (int b = 0; b < RB; ++b) {
#pragma unroll
                for (int i = 0; i < P; ++i) v[b][i] = fma2(v[b][i], g2[i], b2[i]);
                if (row + b * a.slots < r1) R::put(l, z + b * sz, v[b]);
            }
        }
        if (a.stats && l.t == 0)
#pragma unroll
            for (int b = 0; b < RB; ++b)
                if (row + b * a.slots < r1) a.stats[row + b * a.slots] = make_float4(one[b].x, one[b].y, two[b].x, two[b].y);
        row += RB * a.slots;
        y += RB * sy;
        z += RB * sz;
    }
    copy_wait<0>();
}

// The sums of the CTA's threads over the rows side by side: take(sum, pair's
// first channel, value), each channel by one thread.  ent: shared, of NS x
// threads x P pairs; free on entry, free again on return.
template <int FIRST, int NS, int VEC, int K, typename F>
__device__ __forceinline__ void combine(const Lane<VEC, K> &l, int slots, const float2 (&acc)[SUMS][4 * K], float2 *ent, F &&take) {
    constexpr int P = 4 * K;
    if (slots == 1) {
#pragma unroll
        for (int s = 0; s < NS; ++s)
#pragma unroll
            for (int i = 0; i < P; ++i) {
                if (l.has(i, 0)) take(FIRST + s, l.chan(i, 0), acc[FIRST + s][i].x);
                if (l.has(i, 1)) take(FIRST + s, l.chan(i, 1), acc[FIRST + s][i].y);
            }
        return;
    }
    __syncthreads();
    const int nt = blockDim.x;
#pragma unroll
    for (int s = 0; s < NS; ++s)
#pragma unroll
        for (int i = 0; i < P; ++i) ent[(s * P + i) * nt + threadIdx.x] = acc[FIRST + s][i];
    __syncthreads();
    // one (sum, pair, thread of a row) at a time, those of a sum next to one another
    for (int k = threadIdx.x; k < NS * P * l.tpr; k += nt) {
        const int at = k / l.tpr, t = k - at * l.tpr;
        const float2 *e = ent + at * nt + t;
        float2 v = e[0];
        for (int r = 1; r < slots; ++r) v = add2(v, e[r * l.tpr]);
        Lane<VEC, K> o = l;
        o.t = t;
        const int s = at / P, i = at - s * P;
        if (o.has(i, 0)) take(FIRST + s, o.chan(i, 0), v.x);
        if (o.has(i, 1)) take(FIRST + s, o.chan(i, 1), v.y);
    }
    __syncthreads();
}

// Stages of the gradient's ring: what fits beside one another in shared memory.
__host__ __device__ constexpr int bwd_stages(int es, int k) { return k == 1 ? 3 : (es == 2 ? 2 : 1); }

// dx and df of the rows of a CTA's units, and the units' channel sums.  ALL: the
// block, dy and dz are given; what is then not asked for is formed all the same,
// which is fewer instructions than asking.
template <typename T, int VEC, int K, int ROW, bool ALL>
__global__ void __launch_bounds__(kMostThreads) bn_bwd_kernel(const __grid_constant__ BnArgs a) {
    using R = Row<T, VEC, K>;
    using Raw = typename R::Raw;
    constexpr int P = R::P, D = bwd_stages(sizeof(T), K), LINE = R::NV * R::step, STAGE = 4 * LINE;
    extern __shared__ __align__(16) uint8_t smem[];
    __shared__ float meet[2 * kMostThreads / 32 * 2];
    const int nt = blockDim.x;
    Raw *ring = R::ring(smem, D * 4);  // [D][x, f, dy, dz]
    const Lane<VEC, K> l(a);
    // statistics [warp][D][rows of a warp], copied by a lane of each row
    const int line = l.tpr < 32 ? l.tpr : 32, lane = threadIdx.x & 31;
    float4 *const seen = reinterpret_cast<float4 *>(smem + (size_t)D * 4 * R::NV * nt * sizeof(Raw)) +
                         (threadIdx.x >> 5) * (D * (32 / line)) + lane / line;
    const bool copies = lane % line == 0;
    float *held = reinterpret_cast<float *>(smem + (size_t)D * 4 * R::NV * nt * sizeof(Raw) + (size_t)D * (nt / line) * 16);  // whole images: gate A, gate B [2][C]
    RowSum<ROW> sum(a.tpr, l.slot, meet);
    const bool block = ALL || a.f, stream = ALL || a.dy, norm = ALL || a.dz;
    const float mean_post = a.post == CONV_NORM_LAYER ? -a.inv_c : 0.0f, mean_pre = a.pre == CONV_NORM_LAYER ? -a.inv_c : 0.0f;
    const long long sx = a.slots * a.px, sf = a.slots * a.pf, sdy = a.slots * a.pdy, sdz = a.slots * a.pdz;
    const long long s0 = a.slots * a.p0, s1 = a.slots * a.p1;
    pdl_trigger();
    if (a.whole)
        for (int c = threadIdx.x; c < 2 * a.C; c += nt) held[c] = 0.0f;
    __syncthreads();
    pdl_wait();
    float2 q[P], p[P], g2[P], acc[SUMS][P];
#pragma unroll
    for (int s = 0; s < SUMS; ++s)
#pragma unroll
        for (int i = 0; i < P; ++i) acc[s][i] = make_float2(0.0f, 0.0f);
    l.params(g2, a.g2, 1.0f);
    if (block && !a.gate) factors(l, a, 0, q, p);
    for (int unit = blockIdx.x; unit < a.units; unit += gridDim.x) {
        const int n = unit / a.S, k0 = unit - n * a.S;
        const int span = a.gate ? a.HW : a.rows;
        const int r0 = n * span + min(span, k0 * a.run), r1 = n * span + min(span, (k0 + 1) * a.run);
        int row = r0 + l.slot, asked = row;
        const T *x = static_cast<const T *>(a.x) + row * a.px + l.first(0), *f = static_cast<const T *>(a.f) + row * a.pf + l.first(0);
        const T *dy = static_cast<const T *>(a.dy) + row * a.pdy + l.first(0), *dz = static_cast<const T *>(a.dz) + row * a.pdz + l.first(0);
        T *dx = static_cast<T *>(a.o0) + row * a.p0 + l.first(0), *df = static_cast<T *>(a.o1) + row * a.p1 + l.first(0);
        if (!a.full) R::template blank<D * 4>(l, ring);  // (the sums were there between units)
        const Raw *d = ring;
        Raw *to = ring;
        const float4 *sd = seen;
        float4 *sto = seen;
        // A row beyond the run counts as zeros.
        auto ask = [&] {
            if (asked < r1) {
                if (copies) copy_async<16>(tc::smem_u32(sto), a.stats + asked);
                R::ask(l, x, to);
                if (block) R::ask(l, f, to + LINE);
                if (stream) R::ask(l, dy, to + 2 * LINE);
                if (norm) R::ask(l, dz, to + 3 * LINE);
            } else {
                if (copies) *sto = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
#pragma unroll
                for (int m = 0; m < 4; ++m) R::zero(to + m * LINE);
            }
            copy_commit();
            asked += a.slots;
            x += sx;
            f += sf;
            dy += sdy;
            dz += sdz;
            const bool last = to == ring + (D - 1) * STAGE;
            to = last ? ring : to + STAGE;
            sto = last ? seen : sto + 32 / line;
        };
#pragma unroll
        for (int i = 0; i < (D > 1 ? D - 1 : 1); ++i) ask();
        if (block && a.gate) factors(l, a, n, q, p);
        for (int base = r0; base < r1; base += a.slots) {
            const bool on = row < r1;
            copy_wait<(D > 1 ? D - 2 : 0)>();
            __syncwarp();
            const float4 st = *sd;
            float2 u[P], y[P], t[P];  // u^, y^, dY
            R::get(d, y);
            if (block) {
                R::get(d + LINE, u);
                const float2 r = both(st.y), c = both(-st.x * st.y);
                if (ALL || a.b1)
#pragma unroll
                    for (int k = 0; k < P; ++k) y[k] = add2(y[k], p[k]);
#pragma unroll
                for (int k = 0; k < P; ++k) {
                    u[k] = fma2(u[k], r, c);
                    y[k] = fma2(q[k], u[k], y[k]);
                }
            }
            if (stream) R::get(d + 2 * LINE, t);
            else
#pragma unroll
                for (int k = 0; k < P; ++k) t[k] = make_float2(0.0f, 0.0f);
            if (norm) {
                float2 e[P], w = make_float2(0.0f, 0.0f), v = w;
                R::get(d + 3 * LINE, e);
                const float2 r = both(st.w), c = both(-st.z * st.w);
                if (ALL || a.db2)
#pragma unroll
                    for (int k = 0; k < P; ++k) acc[SUM_B2][k] = add2(acc[SUM_B2][k], e[k]);
#pragma unroll
                for (int k = 0; k < P; ++k) {
                    y[k] = fma2(y[k], r, c);
                    acc[SUM_G2][k] = fma2(e[k], y[k], acc[SUM_G2][k]);
                    e[k] = mul2(e[k], g2[k]);
                    w = add2(w, e[k]);
                    v = fma2(e[k], y[k], v);
                }
                const float2 s = sum(w.x + w.y, v.x + v.y);
                const float2 my = both(-s.y * a.inv_c * st.w), m = both(s.x * mean_pre * st.w);
#pragma unroll
                for (int k = 0; k < P; ++k) t[k] = fma2(y[k], my, fma2(e[k], r, add2(t[k], m)));
            }
            const bool last = d == ring + (D - 1) * STAGE;
            d = last ? ring : d + STAGE;
            sd = last ? seen : sd + 32 / line;
            if (D > 1) ask();
            if (on) R::put(l, dx, t);
            if (block) {
                // (what the mean's terms leave in a row beyond the run is 0: its sums are)
                if (ALL || a.want_b)
#pragma unroll
                    for (int k = 0; k < P; ++k) acc[SUM_B][k] = add2(acc[SUM_B][k], t[k]);
#pragma unroll
                for (int k = 0; k < P; ++k) {
                    acc[SUM_A][k] = fma2(t[k], u[k], acc[SUM_A][k]);
                    t[k] = mul2(t[k], q[k]);
                }
                if (a.post != CONV_NORM_NONE) {
                    float2 w = make_float2(0.0f, 0.0f), v = w;
#pragma unroll
                    for (int k = 0; k < P; ++k) {
                        w = add2(w, t[k]);
                        v = fma2(t[k], u[k], v);
                    }
                    const float2 s = sum(w.x + w.y, v.x + v.y);
                    const float2 r = both(st.y), mu = both(-s.y * a.inv_c * st.y);
                    const float2 m = both(s.x * mean_post * st.y);
#pragma unroll
                    for (int k = 0; k < P; ++k) t[k] = fma2(u[k], mu, fma2(t[k], r, m));
                }
                if (on) R::put(l, df, t);
            }
            if (D == 1) {
                __syncwarp();
                ask();
            }
            row += a.slots;
            dx += s0;
            df += s1;
        }
        copy_wait<0>();
        float2 *ent = reinterpret_cast<float2 *>(smem);
        if (a.whole) {  // the image's sums are complete
            combine<SUM_A, 2, VEC, K>(l, a.slots, acc, ent, [&](int s, int c, float v) {
                const float gate = a.gate[(long long)n * a.C + c];
                held[s * a.C + c] += gate * v;
                if (a.dgate) {
                    const float k = (a.scale ? a.scale[c] : 1.0f) * (s == SUM_A ? (a.g1 ? a.g1[c] : 1.0f) : (a.b1 ? a.b1[c] : 0.0f)) * v;
                    // (A and B of a channel are two threads': they meet in the CTA's part of the workspace)
                    a.part[((long long)blockIdx.x * SUMS + s) * a.Cp + c] = k;
                }
            });
            if (a.dgate) {
                __syncthreads();
                const float *one = a.part + (long long)blockIdx.x * SUMS * a.Cp;
                for (int c = threadIdx.x; c < a.C; c += nt) a.dgate[(long long)n * a.C + c] = one[c] + one[a.Cp + c];
                __syncthreads();
            }
#pragma unroll
            for (int i = 0; i < P; ++i) acc[SUM_A][i] = acc[SUM_B][i] = make_float2(0.0f, 0.0f);
        } else {
            combine<0, SUMS, VEC, K>(l, a.slots, acc, ent, [&](int s, int c, float v) {
                a.part[((long long)unit * SUMS + s) * a.Cp + c] = v;
            });
        }
    }
    if (a.whole) {
        combine<SUM_G2, 2, VEC, K>(l, a.slots, acc, reinterpret_cast<float2 *>(smem), [&](int s, int c, float v) {
            a.part[((long long)blockIdx.x * SUMS + s) * a.Cp + c] = v;
        });
        __syncthreads();
        for (int c = threadIdx.x; c < a.C; c += nt) {
            float *one = a.part + (long long)blockIdx.x * SUMS * a.Cp + c;
            one[0] = held[c];
            one[a.Cp] = held[a.C + c];
        }
    }
}

// Joins the units' sums: a CTA takes sixteen channels, four a thread, and 128
// units at a time.  Blocks y = 0 sum over all units; those above an image's
// units for its dgate, an image a warp.
constexpr int kJoin = 512, kJoinC = 16;
__device__ __forceinline__ void add4(float4 &s, const float4 &v, float k) {
    s.x = fmaf(k, v.x, s.x);
    s.y = fmaf(k, v.y, s.y);
    s.z = fmaf(k, v.z, s.z);
    s.w = fmaf(k, v.w, s.w);
}
__device__ __forceinline__ float4 sum8(float4 v) {  // over the lanes of one four of channels
#pragma unroll
    for (int o = 4; o < 32; o *= 2) {
        v.x += __shfl_xor_sync(0xffffffffu, v.x, o);
        v.y += __shfl_xor_sync(0xffffffffu, v.y, o);
        v.z += __shfl_xor_sync(0xffffffffu, v.z, o);
        v.w += __shfl_xor_sync(0xffffffffu, v.w, o);
    }
    return v;
}
__global__ void __launch_bounds__(kJoin) bn_join_kernel(const __grid_constant__ BnArgs a, int parts) {
    __shared__ float4 red[SUMS][kJoin / 32][kJoinC / 4];
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, four = lane & 3, group = lane >> 2;
    const int c = blockIdx.x * kJoinC + four * 4;  // (channels are padded to fours in the workspace)
    const bool on = c < a.C;
    pdl_trigger();
    pdl_wait();
    const float4 zero = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
    if (blockIdx.y > 0) {
        const int n = (blockIdx.y - 1) * (kJoin / 32) + warp;
        float4 A = zero, B = zero;
        if (n < a.N && on)
            for (int s = group; s < a.S; s += 8) {
                const float *u = a.part + ((long long)n * a.S + s) * SUMS * a.Cp + c;
                add4(A, *reinterpret_cast<const float4 *>(u + SUM_A * a.Cp), 1.0f);
                add4(B, *reinterpret_cast<const float4 *>(u + SUM_B * a.Cp), 1.0f);
            }
        A = sum8(A);
        B = sum8(B);
        if (n < a.N && group < 4 && c + group < a.C) {
            const int k = c + group;
            const float g1 = a.g1 ? a.g1[k] : 1.0f, b1 = a.b1 ? a.b1[k] : 0.0f;
            const float va = group == 0 ? A.x : (group == 1 ? A.y : (group == 2 ? A.z : A.w));
            const float vb = group == 0 ? B.x : (group == 1 ? B.y : (group == 2 ? B.z : B.w));
            a.dgate[(long long)n * a.C + k] = (a.scale ? a.scale[k] : 1.0f) * (g1 * va + b1 * vb);
        }
        return;
    }
    float4 v[SUMS] = {zero, zero, zero, zero};
    const bool gated = a.gate && !a.whole;
    if (on)
        for (int u = warp * 8 + group; u < parts; u += kJoin / 4) {
            const float4 *one = reinterpret_cast<const float4 *>(a.part + (long long)u * SUMS * a.Cp + c);
            float4 w[SUMS];
#pragma unroll
            for (int s = 0; s < SUMS; ++s) w[s] = one[s * (a.Cp / 4)];
            if (gated) {
                const float *g = a.gate + (long long)(u / a.S) * a.C + c;
                const float4 k = make_float4(g[0], c + 1 < a.C ? g[1] : 0.0f, c + 2 < a.C ? g[2] : 0.0f, c + 3 < a.C ? g[3] : 0.0f);
#pragma unroll
                for (int s = 0; s < SUM_G2; ++s) w[s] = make_float4(k.x * w[s].x, k.y * w[s].y, k.z * w[s].z, k.w * w[s].w);
            }
#pragma unroll
            for (int s = 0; s < SUMS; ++s) add4(v[s], w[s], 1.0f);
        }
#pragma unroll
    for (int s = 0; s < SUMS; ++s) {
        v[s] = sum8(v[s]);
        if (group == 0) red[s][warp][four] = v[s];
    }
    __syncthreads();
    if (warp == 0) {  // a channel a lane, twice
        const int at = lane & 15, k = blockIdx.x * kJoinC + at;
        float t[SUMS];
#pragma unroll
        for (int s = 0; s < SUMS; ++s) {
            t[s] = 0.0f;
            const float *r = reinterpret_cast<const float *>(red[s]) + at;
            for (int w = lane >> 4; w < kJoin / 32; w += 2) t[s] += r[w * kJoinC];
            t[s] += __shfl_xor_sync(0xffffffffu, t[s], 16);
        }
        if (lane < 16 && k < a.C) {
            const float sc = a.scale ? a.scale[k] : 1.0f;
            if (a.dscale) a.dscale[k] = (a.g1 ? a.g1[k] : 1.0f) * t[SUM_A] + (a.b1 ? a.b1[k] : 0.0f) * t[SUM_B];
            if (a.dg1) a.dg1[k] = sc * t[SUM_A];
            if (a.db1) a.db1[k] = sc * t[SUM_B];
            if (a.dg2) a.dg2[k] = t[SUM_G2];
            if (a.db2) a.db2[k] = t[SUM_B2];
        }
    }
}

// ------------------------------------------------------------------ host side
template <typename T, int VEC>
const void *pick_fwd(int k, int rb) {
    if (rb == 2) return (const void *)&bn_fwd_kernel<T, VEC, 1, 2>;
    return k == 1 ? (const void *)&bn_fwd_kernel<T, VEC, 1, 1> : (const void *)&bn_fwd_kernel<T, VEC, 2, 1>;
}
template <typename T, int VEC>
const void *pick_bwd(int k, int tpr, bool all) {
    if (k == 2) return all ? (const void *)&bn_bwd_kernel<T, VEC, 2, ROW_WARPS, true> : (const void *)&bn_bwd_kernel<T, VEC, 2, ROW_WARPS, false>;
    if (!all) return (const void *)&bn_bwd_kernel<T, VEC, 1, ROW_ANY, false>;
    return tpr < 32 ? (const void *)&bn_bwd_kernel<T, VEC, 1, ROW_PART, true>
                    : (tpr == 32 ? (const void *)&bn_bwd_kernel<T, VEC, 1, ROW_WARP, true> : (const void *)&bn_bwd_kernel<T, VEC, 1, ROW_WARPS, true>);
}
// (rb: rows at a time of the forward kernel, 0: the gradient)
const void *pick_kernel(conv_dtype_t dt, int vec, int rb, int k, int tpr, bool all) {
    using B = __nv_bfloat16;
    if (rb) {
        if (dt == CONV_F32) return vec == 4 ? pick_fwd<float, 4>(k, rb) : pick_fwd<float, 1>(k, rb);
        return vec == 8 ? pick_fwd<B, 8>(k, rb) : (vec == 2 ? pick_fwd<B, 2>(k, rb) : pick_fwd<B, 1>(k, rb));
    }
    if (dt == CONV_F32) return vec == 4 ? pick_bwd<float, 4>(k, tpr, all) : pick_bwd<float, 1>(k, tpr, all);
    return vec == 8 ? pick_bwd<B, 8>(k, tpr, all) : (vec == 2 ? pick_bwd<B, 2>(k, tpr, all) : pick_bwd<B, 1>(k, tpr, all));
}

// Channels a vector access takes: the widest that the channel count, every
// map's pitch and every map's address allow (a null map: any).
struct Map { const void *p; long long pitch; };
template <int N>
int vec_for(const conv_plan *p, const Map (&maps)[N]) {
    const int es = conv_esize(p->dtype);
    const int widths[2] = {16 / es, p->dtype == CONV_F32 ? 1 : 2};
    for (int v : widths) {
        bool ok = p->s.c_in % v == 0;
        for (const Map &m : maps) ok = ok && (!m.p || (m.pitch % v == 0 && (uintptr_t)m.p % (uintptr_t)(v * es) == 0));
        if (ok) return v;
    }
    return 1;
}

// Bytes of the ring of a CTA: a thread's 8 k channels of each map and stage.
// (The gradient's holds the sums of rows side by side after its last row:
// rows side by side have k = 1, so that it has 96 elements a thread where the
// sums are SUMS * 8 in fp32.)
static_assert(3 * 4 * 8 * 2 >= SUMS * 8 * 4, "");
size_t ring_bytes(const BnGeom &g, const BnGeom::Part &d, int es) {
    const size_t maps = (size_t)d.threads * 8 * g.k * es;
    if (d.rb) return 2 * kFwdStages * d.rb * maps;
    const int stages = bwd_stages(es, g.k);  // (and a row's statistics)
    return stages * (4 * maps + (size_t)d.threads / (g.tpr < 32 ? g.tpr : 32) * 16);
}

cudaError_t launch(const conv_plan *p, const BnGeom::Part &d, int vec, BnArgs &a, size_t smem, cudaStream_t st) {
    const void *k = pick_kernel(p->dtype, vec, d.rb, p->bn.k, p->bn.tpr, a.f && a.dy && a.dz);
    if (smem > 40 * 1024) {  // (with the kernel's static shared memory: 48 KB are free)
        const int rc = conv_grant_smem_once(k, p->device, (int)smem);
        if (rc != CONV_OK) return cudaErrorInvalidValue;
    }
    a.slots = d.slots; a.run = d.run; a.S = d.S; a.units = d.units; a.whole = d.whole;
    void *args[] = {&a};
    return conv_launch(k, dim3((unsigned)d.grid), dim3((unsigned)d.threads), args, smem, st);
}

int check_map(const conv_plan *p, const void *t, int64_t *pitch) {
    if (!t) return CONV_OK;
    if (*pitch == 0) *pitch = p->s.c_in;
    if (*pitch < p->s.c_in) return CONV_ERR_INVALID_ARG;
    if (*pitch >= (1ll << 31) || (long long)p->s.n * p->s.h * p->s.w * *pitch >= (1ll << 40)) return CONV_ERR_UNSUPPORTED;
    if ((uintptr_t)t % (uintptr_t)conv_esize(p->dtype)) return CONV_ERR_MISALIGNED;
    return CONV_OK;
}

// Whether a buffer that a run writes shares a byte with another that it reads
// or writes.  A written map may be an input map itself (every element is read
// by the thread that writes it, before it does), not otherwise overlap it.
struct Small { const void *p; size_t bytes; };
template <int M, int W, int I, int O>
bool shared(const Map (&in)[M], const Map (&out)[W], const Small (&small_in)[I], const Small (&small_out)[O], long long rows,
            int C, int es) {
    for (int i = 0; i < W; ++i) {
        for (const Map &m : in)
            if (!(m.p == out[i].p && m.pitch == out[i].pitch) && maps_overlap(m.p, m.pitch, out[i].p, out[i].pitch, rows, C, es))
                return true;
        for (int j = 0; j < i; ++j)
            if (maps_overlap(out[j].p, out[j].pitch, out[i].p, out[i].pitch, rows, C, es)) return true;
        for (const Small &s : small_in)
            if (range_overlaps(s.p, s.bytes, out[i].p, out[i].pitch, rows, C, es)) return true;
    }
    for (int i = 0; i < O; ++i) {
        const Small &s = small_out[i];
        for (const Map &m : in)
            if (range_overlaps(s.p, s.bytes, m.p, m.pitch, rows, C, es)) return true;
        for (const Map &m : out)
            if (range_overlaps(s.p, s.bytes, m.p, m.pitch, rows, C, es)) return true;
        for (const Small &t : small_in)
            if (conv_overlaps(s.p, s.bytes, t.p, t.bytes)) return true;
        for (int j = 0; j < i; ++j)
            if (conv_overlaps(s.p, s.bytes, small_out[j].p, small_out[j].bytes)) return true;
    }
    return false;
}
bool bad_f32(const void *t) { return t && ((uintptr_t)t & 3u); }

long long up(long long a, long long b) { return (a + b - 1) / b; }

// All rows in runs of whole sets of rows side by side, one wave of CTAs.
void divide_rows(BnGeom::Part &d, long long rows, long long set, long long wave) {
    long long run = up(up(rows, wave), set) * set;
    if (run < set) run = set;
    d.run = (int)run;
    d.S = d.units = d.grid = (int)up(rows, run);
    d.whole = 0;
}
// Each image in runs of whole sets, as many as fill the CTAs best: a run costs
// its sets and about four more for its start and end.
void divide_images(BnGeom::Part &d, long long N, long long HW, long long set, long long wave) {
    long long best = -1;
    for (long long S = 1; S <= 1024; ++S) {
        const long long sets = up(up(HW, S), set);
        if (S > 1 && up(HW, sets * set) != S) continue;
        const long long cost = up(N * S, wave) * (sets + 4);
        if (best >= 0 && cost >= best) continue;
        best = cost;
        d.S = (int)S;
        d.run = (int)(S == 1 ? HW : sets * set);
    }
    d.units = d.grid = (int)(N * d.S);
    d.whole = 0;
}

// Threads of a row, rows of a CTA, and how the rows are divided.
void plan_geometry(conv_plan *p) {
    BnGeom &g = p->bn;
    const int C = p->s.c_in, es = conv_esize(p->dtype);
    g.k = C <= 8 * kMostThreads ? 1 : 2;
    const int want = (C + 8 * g.k - 1) / (8 * g.k);
    int tpr = 1;
    if (want > 32) tpr = (want + 31) / 32 * 32;
    else while (tpr < want) tpr *= 2;
    g.tpr = tpr;
    g.full = C == tpr * 8 * g.k;
    const long long N = p->s.n, HW = (long long)p->s.h * p->s.w, rows = N * HW;
    p->ws_bytes = p->ws_bwd_bytes = 0;
    if (rows == 0) return;
    auto part = [&](BnGeom::Part &d, int rb, int threads) {
        d.rb = rb;
        d.slots = tpr <= threads ? threads / tpr : 1;
        d.threads = tpr * d.slots;
    };
    // CTAs of one wave: 512 threads a SM, where their rings fit
    auto wave = [&](const BnGeom::Part &d) {
        const long long smem = (220 * 1024) / (long long)(ring_bytes(g, d, es) + 1024), regs = kMostThreads / d.threads;
        const long long n = smem < regs ? smem : regs;
        return (long long)p->num_sms * (n < 1 ? 1 : n);
    };
    // two rows at a time where a CTA takes more than one set of rows
    part(g.fwd, 1, kThreads);
    if (g.k == 1 && rows > (long long)p->num_sms * g.fwd.slots) g.fwd.rb = 2;
    g.fwd_gated = g.fwd;
    divide_rows(g.fwd, rows, (long long)g.fwd.slots * g.fwd.rb, wave(g.fwd));
    if (g.fwd.rb == 2 && HW >= 4LL * g.fwd.slots) divide_images(g.fwd_gated, N, HW, 2LL * g.fwd.slots, wave(g.fwd_gated));
    else {
        g.fwd_gated.rb = 1;
        divide_rows(g.fwd_gated, rows, g.fwd.slots, wave(g.fwd_gated));
    }
    // the gradient in large CTAs: a part of the sums from each
    part(g.bwd, 0, kMostThreads);
    g.bwd_gated = g.bwd;
    const long long w = wave(g.bwd);
    divide_rows(g.bwd, rows, g.bwd.slots, w);
    divide_images(g.bwd_gated, N, HW, g.bwd.slots, w);
    g.bwd_gated.whole = g.bwd_gated.S == 1;
    if (g.bwd_gated.whole && N > w) g.bwd_gated.grid = (int)w;
    const long long parts = g.bwd.grid > g.bwd_gated.grid ? g.bwd.grid : g.bwd_gated.grid;
    p->ws_bwd_bytes = (size_t)parts * SUMS * ((C + 3) / 4 * 4) * 4;
}

}  // namespace

extern "C" int conv_plan_create_blocknorm(int32_t n, int32_t h, int32_t w, int32_t c, conv_norm_t post, conv_norm_t pre,
                                          float eps, conv_dtype_t dtype, conv_plan_t **out_plan) {
    if (!out_plan) return CONV_ERR_NULL_ARG;
    *out_plan = nullptr;
    if (n < 0 || h < 1 || w < 1 || c < 1) return CONV_ERR_INVALID_SHAPE;
    if ((int)dtype < CONV_F32 || (int)dtype > CONV_I8) return CONV_ERR_INVALID_ARG;
    if ((int)post < CONV_NORM_NONE || (int)post > CONV_NORM_RMS || (int)pre < CONV_NORM_NONE || (int)pre > CONV_NORM_RMS)
        return CONV_ERR_INVALID_ARG;
    if (!(eps >= 0.0f) || !isfinite(eps)) return CONV_ERR_INVALID_ARG;
    if (dtype == CONV_I8) return CONV_ERR_UNSUPPORTED;
    // 32-bit pixel indices, a row's channels in one CTA
    if (c > kMaxC || (long long)h * w >= (1ll << 30) || (long long)h * w * n >= (1ll << 30)) return CONV_ERR_UNSUPPORTED;
    conv_plan *p = new (std::nothrow) conv_plan();
    if (!p) return CONV_ERR_OOM;
    p->s = {n, h, w, c, c, 1, 1};
    p->stride = 1; p->groups = 1; p->dtype = dtype; p->oh = h; p->ow = w;
    p->y_c = c; p->up = 1; p->algo = CONV_ALGO_BLOCKNORM;
    p->bn.post = post; p->bn.pre = pre; p->bn.eps = eps;
    const int rc = conv_plan_bind_device(p, false);
    if (rc != CONV_OK) {
        conv_plan_destroy(p);
        return rc;
    }
    plan_geometry(p);
    static const char *const names[] = {"none", "layer", "rms"};
    snprintf(p->desc, sizeof(p->desc), "blocknorm %s post=%s pre=%s threads=%dx%d channels/thread=%d ctas=%d gradient: %d, gated %d in %d",
             dtype == CONV_F32 ? "f32" : "bf16", names[post], names[pre], p->bn.fwd.slots, p->bn.tpr, 8 * p->bn.k, p->bn.fwd.grid,
             p->bn.bwd.grid, p->bn.bwd_gated.units, p->bn.bwd_gated.grid);
    *out_plan = p;
    return CONV_OK;
}

namespace {
BnArgs base_args(const conv_plan *p, const conv_blocknorm_params_t &w, const void *x, int64_t px, const void *f, int64_t pf) {
    BnArgs a = {};
    a.x = x; a.px = px; a.f = f; a.pf = pf;
    a.scale = w.scale; a.gate = w.gate; a.g1 = w.post_gamma; a.b1 = w.post_beta; a.g2 = w.pre_gamma; a.b2 = w.pre_beta;
    a.eps = p->bn.eps; a.inv_c = 1.0f / (float)p->s.c_in;
    a.N = p->s.n; a.HW = p->s.h * p->s.w; a.rows = a.N * a.HW; a.C = p->s.c_in; a.Cp = (a.C + 3) / 4 * 4;
    a.post = p->bn.post; a.pre = p->bn.pre;
    a.tpr = p->bn.tpr; a.full = p->bn.full;
    return a;
}
int check_params(const conv_plan *p, const conv_blocknorm_params_t &w, const void *f) {
    if (!f && (w.scale || w.gate || w.post_gamma || w.post_beta || p->bn.post != CONV_NORM_NONE)) return CONV_ERR_INVALID_ARG;
    if (p->bn.post == CONV_NORM_NONE && (w.post_gamma || w.post_beta)) return CONV_ERR_INVALID_ARG;
    if (p->bn.pre == CONV_NORM_NONE && (w.pre_gamma || w.pre_beta)) return CONV_ERR_INVALID_ARG;
    if (bad_f32(w.scale) || bad_f32(w.gate) || bad_f32(w.post_gamma) || bad_f32(w.post_beta) || bad_f32(w.pre_gamma) ||
        bad_f32(w.pre_beta))
        return CONV_ERR_MISALIGNED;
    return CONV_OK;
}
}  // namespace

extern "C" int conv_run_blocknorm(const conv_plan_t *plan, const void *x, int64_t x_pitch, const void *f, int64_t f_pitch,
                                  const conv_blocknorm_params_t *params, void *y, int64_t y_pitch, void *z, int64_t z_pitch,
                                  float *stats, void *stream) {
    if (!plan) return CONV_ERR_NULL_ARG;
    const conv_plan *p = plan;
    if (p->algo != CONV_ALGO_BLOCKNORM) return CONV_ERR_INVALID_ARG;
    if (p->s.n == 0) return CONV_OK;
    static const conv_blocknorm_params_t kNone = {};
    const conv_blocknorm_params_t &w = params ? *params : kNone;
    const bool norm = p->bn.pre != CONV_NORM_NONE;
    if (!x || (norm && !z) || (!norm && !y)) return CONV_ERR_NULL_ARG;
    if ((!norm && z) || (!f && y)) return CONV_ERR_INVALID_ARG;
    int rc;
    if ((rc = check_params(p, w, f)) != CONV_OK || (rc = check_map(p, x, &x_pitch)) != CONV_OK ||
        (rc = check_map(p, f, &f_pitch)) != CONV_OK || (rc = check_map(p, y, &y_pitch)) != CONV_OK ||
        (rc = check_map(p, z, &z_pitch)) != CONV_OK)
        return rc;
    if ((uintptr_t)stats & 15u) return CONV_ERR_MISALIGNED;
    const int es = conv_esize(p->dtype), C = p->s.c_in;
    const long long rows = (long long)p->s.n * p->s.h * p->s.w;
    const size_t cb = (size_t)C * 4, nb = (size_t)p->s.n * cb;
    const Map in[2] = {{x, x_pitch}, {f, f_pitch}}, out[2] = {{y, y_pitch}, {z, z_pitch}};
    const Small si[6] = {{w.scale, cb}, {w.gate, nb}, {w.post_gamma, cb}, {w.post_beta, cb}, {w.pre_gamma, cb}, {w.pre_beta, cb}};
    const Small so[1] = {{stats, (size_t)rows * 16}};
    if (shared(in, out, si, so, rows, C, es)) return CONV_ERR_ALIASING;
    BnArgs a = base_args(p, w, x, x_pitch, f, f_pitch);
    a.o0 = y; a.p0 = y_pitch; a.o1 = z; a.p1 = z_pitch;
    a.stats = reinterpret_cast<float4 *>(stats);
    const Map all[4] = {in[0], in[1], out[0], out[1]};
    const BnGeom::Part &g = w.gate ? p->bn.fwd_gated : p->bn.fwd;
    return launch(p, g, vec_for(p, all), a, ring_bytes(p->bn, g, es), (cudaStream_t)stream) == cudaSuccess ? CONV_OK : CONV_ERR_CUDA;
}

extern "C" int conv_run_blocknorm_bwd(const conv_plan_t *plan, const void *x, int64_t x_pitch, const void *f, int64_t f_pitch,
                                      const conv_blocknorm_params_t *params, const float *stats, const void *dy,
                                      int64_t dy_pitch, const void *dz, int64_t dz_pitch, void *dx, int64_t dx_pitch,
                                      void *df, int64_t df_pitch, const conv_blocknorm_grads_t *grads, void *workspace,
                                      void *stream) {
    if (!plan) return CONV_ERR_NULL_ARG;
    const conv_plan *p = plan;
    if (p->algo != CONV_ALGO_BLOCKNORM) return CONV_ERR_INVALID_ARG;
    static const conv_blocknorm_params_t kNone = {};
    static const conv_blocknorm_grads_t kNoGrads = {};
    const conv_blocknorm_params_t &w = params ? *params : kNone;
    const conv_blocknorm_grads_t &d = grads ? *grads : kNoGrads;
    cudaStream_t st = (cudaStream_t)stream;
    const int es = conv_esize(p->dtype), C = p->s.c_in;
    const size_t cb = (size_t)C * 4;
    if (bad_f32(d.scale) || bad_f32(d.gate) || bad_f32(d.post_gamma) || bad_f32(d.post_beta) || bad_f32(d.pre_gamma) ||
        bad_f32(d.pre_beta))
        return CONV_ERR_MISALIGNED;
    if ((p->bn.post == CONV_NORM_NONE && (d.post_gamma || d.post_beta)) || (p->bn.pre == CONV_NORM_NONE && (d.pre_gamma || d.pre_beta)))
        return CONV_ERR_INVALID_ARG;
    if (p->s.n == 0) {  // sums over nothing (a gate has no rows)
        float *const sums[5] = {d.scale, d.post_gamma, d.post_beta, d.pre_gamma, d.pre_beta};
        for (float *s : sums)
            if (s && cudaMemsetAsync(s, 0, cb, st) != cudaSuccess) return CONV_ERR_CUDA;
        return CONV_OK;
    }
    const bool norm = p->bn.pre != CONV_NORM_NONE;
    if (!x || !dx || (norm && !dz) || (!norm && !dy) || !stats || (f && !df)) return CONV_ERR_NULL_ARG;
    if ((!norm && dz) || (!f && (df || d.scale || d.gate)) || (d.gate && !w.gate)) return CONV_ERR_INVALID_ARG;
    int rc;
    if ((rc = check_params(p, w, f)) != CONV_OK || (rc = check_map(p, x, &x_pitch)) != CONV_OK ||
        (rc = check_map(p, f, &f_pitch)) != CONV_OK || (rc = check_map(p, dy, &dy_pitch)) != CONV_OK ||
        (rc = check_map(p, dz, &dz_pitch)) != CONV_OK || (rc = check_map(p, dx, &dx_pitch)) != CONV_OK ||
        (rc = check_map(p, df, &df_pitch)) != CONV_OK)
        return rc;
    if (((uintptr_t)stats & 15u) || ((uintptr_t)workspace & 15u)) return CONV_ERR_MISALIGNED;
    if (!workspace) return CONV_ERR_NULL_ARG;
    const long long rows = (long long)p->s.n * p->s.h * p->s.w;
    const size_t nb = (size_t)p->s.n * cb;
    const Map in[4] = {{x, x_pitch}, {f, f_pitch}, {dy, dy_pitch}, {dz, dz_pitch}}, out[2] = {{dx, dx_pitch}, {df, df_pitch}};
    const Small si[7] = {{w.scale, cb}, {w.gate, nb}, {w.post_gamma, cb}, {w.post_beta, cb}, {w.pre_gamma, cb}, {w.pre_beta, cb},
                         {stats, (size_t)rows * 16}};
    const Small so[7] = {{d.scale, cb}, {d.gate, nb}, {d.post_gamma, cb}, {d.post_beta, cb}, {d.pre_gamma, cb}, {d.pre_beta, cb},
                         {workspace, p->ws_bwd_bytes}};
    if (shared(in, out, si, so, rows, C, es)) return CONV_ERR_ALIASING;
    BnArgs a = base_args(p, w, x, x_pitch, f, f_pitch);
    a.dy = dy; a.pdy = dy_pitch; a.dz = dz; a.pdz = dz_pitch;
    a.o0 = dx; a.p0 = dx_pitch; a.o1 = df; a.p1 = df_pitch;
    a.stats = reinterpret_cast<float4 *>(const_cast<float *>(stats));
    a.part = static_cast<float *>(workspace);
    a.dscale = d.scale; a.dgate = d.gate; a.dg1 = d.post_gamma; a.db1 = d.post_beta; a.dg2 = d.pre_gamma; a.db2 = d.pre_beta;
    a.want_b = d.post_beta || (w.post_beta && (d.scale || d.gate));
    const BnGeom::Part &g = w.gate ? p->bn.bwd_gated : p->bn.bwd;
    const Map all[6] = {in[0], in[1], in[2], in[3], out[0], out[1]};
    const size_t smem = ring_bytes(p->bn, g, es) + (g.whole ? 2 * cb : 0);
    if (launch(p, g, vec_for(p, all), a, smem, st) != cudaSuccess) return CONV_ERR_CUDA;
    const bool sums = d.scale || d.post_gamma || d.post_beta || d.pre_gamma || d.pre_beta, images = d.gate && !g.whole;
    if (!sums && !images) return CONV_OK;
    int parts = g.grid;
    void *args[] = {&a, &parts};
    const dim3 grid((unsigned)((C + kJoinC - 1) / kJoinC), 1 + (unsigned)(images ? (a.N + kJoin / 32 - 1) / (kJoin / 32) : 0));
    return conv_launch((const void *)&bn_join_kernel, grid, dim3(kJoin), args, 0, st) == cudaSuccess ? CONV_OK : CONV_ERR_CUDA;
}
