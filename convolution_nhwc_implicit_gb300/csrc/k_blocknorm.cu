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
constexpr int kThreads = 256;      // of a CTA whose rows take no more
constexpr int kMostThreads = 512;  // of a row
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
    int rows, HW, C, N;
    int post, pre;                 // conv_norm_t
    int tpr, slots;                // threads of a row, rows side by side
    int run;                       // rows of a CTA (gradient: of a unit)
    int S, units;                  // gradient: runs an image (of all rows without a gate), runs in all
    int whole;                     // gradient: a unit is a whole image of a gated map
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
    __device__ __forceinline__ int chan(int i, int h) const {
        if constexpr (VEC == 1) return first(2 * i + h);
        else return first(i / (VEC / 2)) + i % (VEC / 2) * 2 + h;
    }
    __device__ __forceinline__ bool has(int i, int h) const { return chan(i, h) < C; }
    // src at the thread's channels (null: `other`), 0 beyond the row's end
    __device__ __forceinline__ void params(float2 (&v)[P], const float *src, float other) const {
#pragma unroll
        for (int i = 0; i < P; ++i) {
            v[i].x = has(i, 0) ? (src ? src[chan(i, 0)] : other) : 0.0f;
            v[i].y = has(i, 1) ? (src ? src[chan(i, 1)] : other) : 0.0f;
        }
    }
};

template <typename T, int VEC, int K>
struct Row {
    using V = Vec<T, VEC>;
    using Raw = typename V::Raw;
    using L = Lane<VEC, K>;
    static constexpr int NV = L::NV, P = L::P;
    // a thread's vectors of one map, `step` apart in shared memory, 0 beyond the row's end
    __device__ static __forceinline__ void get(const L &l, const Raw *src, int step, float2 (&f)[P]) {
#pragma unroll
        for (int v = 0; v < NV; ++v) {
            float2 one[V::kPairs];
            V::unpack(src[v * step], one);
            const bool on = l.on(v);
#pragma unroll
            for (int e = 0; e < V::kPairs; ++e) {
                if (!on) one[e] = make_float2(0.0f, 0.0f);
                if constexpr (VEC == 1) {
                    if (v % 2) f[v / 2].y = one[0].x;
                    else f[v / 2].x = one[0].x;
                } else f[v * V::kPairs + e] = one[e];
            }
        }
    }
    __device__ static __forceinline__ void put(const L &l, T *row, const float2 (&f)[P]) {
#pragma unroll
        for (int v = 0; v < NV; ++v) {
            float2 one[V::kPairs];
#pragma unroll
            for (int e = 0; e < V::kPairs; ++e) {
                if constexpr (VEC == 1) one[0].x = v % 2 ? f[v / 2].y : f[v / 2].x;
                else one[e] = f[v * V::kPairs + e];
            }
            if (l.on(v)) *reinterpret_cast<Raw *>(row + l.first(v)) = V::pack(one);
        }
    }
    __device__ static __forceinline__ void ask(const L &l, const T *row, Raw *dst, int step) {
#pragma unroll
        for (int v = 0; v < NV; ++v)
            if (l.on(v)) copy_vec(dst + v * step, reinterpret_cast<const Raw *>(row + l.first(v)));
    }
};

// Sums over the threads of a row.  Rows of more than a warp meet in one of two
// sets of shared entries in turn: whoever writes an entry again has passed the
// barrier of the other set, and with it everyone's reading of this one.
struct RowSum {
    int tpr, slot;
    float2 *buf;
    int flip;
    __device__ __forceinline__ RowSum(int tpr_, int slot_, float2 *b) : tpr(tpr_), slot(slot_), buf(b), flip(0) {}
    __device__ __forceinline__ float2 operator()(float2 v) {
#pragma unroll
        for (int o = 16; o > 0; o >>= 1)
            if (o < tpr) {
                const float2 w = make_float2(__shfl_xor_sync(0xffffffffu, v.x, o), __shfl_xor_sync(0xffffffffu, v.y, o));
                v = add2(v, w);
            }
        if (tpr > 32) {
            float2 *b = buf + flip;
            flip ^= kMostThreads / 32;
            if ((threadIdx.x & 31) == 0) b[threadIdx.x >> 5] = v;
            asm volatile("bar.sync %0, %1;" ::"r"(1 + slot), "r"(tpr) : "memory");
            const int n = tpr >> 5;
            v = b[slot * n];
            for (int i = 1; i < n; ++i) v = add2(v, b[slot * n + i]);
        }
        return v;
    }
};

__device__ __forceinline__ float2 both(float v) { return make_float2(v, v); }

// m and r of one norm of a row, and the values normalised in place.
template <int VEC, int K>
__device__ __forceinline__ float2 normalise(const Lane<VEC, K> &l, RowSum &sum, float2 (&v)[4 * K], int kind, float inv_c, float eps) {
    constexpr int P = 4 * K;
    float m = 0.0f;
    if (kind == CONV_NORM_LAYER) {
        float2 s = make_float2(0.0f, 0.0f);
#pragma unroll
        for (int i = 0; i < P; ++i) s = add2(s, v[i]);
        m = sum(make_float2(s.x + s.y, 0.0f)).x * inv_c;
#pragma unroll
        for (int i = 0; i < P; ++i) {
            v[i].x = l.has(i, 0) ? v[i].x - m : 0.0f;
            v[i].y = l.has(i, 1) ? v[i].y - m : 0.0f;
        }
    }
    float2 q = make_float2(0.0f, 0.0f);
#pragma unroll
    for (int i = 0; i < P; ++i) q = fma2(v[i], v[i], q);
    const float r = 1.0f / sqrtf(sum(make_float2(q.x + q.y, 0.0f)).x * inv_c + eps);
#pragma unroll
    for (int i = 0; i < P; ++i) v[i] = mul2(v[i], both(r));
    return make_float2(m, r);
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

// y and z of a run of rows.
template <typename T, int VEC, int K>
__global__ void __launch_bounds__(kMostThreads) bn_fwd_kernel(const __grid_constant__ BnArgs a) {
    using R = Row<T, VEC, K>;
    using Raw = typename R::Raw;
    constexpr int P = R::P, NV = R::NV, D = kFwdStages;
    extern __shared__ __align__(16) uint8_t smem[];
    __shared__ float2 meet[2 * kMostThreads / 32];
    const int nt = blockDim.x;
    Raw *ring = reinterpret_cast<Raw *>(smem) + threadIdx.x;  // [D][2][NV][threads]
    const Lane<VEC, K> l(a);
    RowSum sum(a.tpr, l.slot, meet);
    const int r0 = blockIdx.x * a.run, r1 = min(a.rows, r0 + a.run);
    const int iters = (r1 - r0 + a.slots - 1) / a.slots;
    const T *x = static_cast<const T *>(a.x), *f = static_cast<const T *>(a.f);
    pdl_trigger();
    pdl_wait();
    auto ask = [&](int i) {
        const int row = r0 + i * a.slots + l.slot;
        if (row < r1) {
            Raw *d = ring + (i % D) * (2 * NV) * nt;
            R::ask(l, x + row * a.px, d, nt);
            if (f) R::ask(l, f + row * a.pf, d + NV * nt, nt);
        }
        copy_commit();
    };
#pragma unroll
    for (int i = 0; i < D - 1; ++i) ask(i);
    float2 q[P], p[P], g2[P], b2[P];
    int image = a.gate ? -1 : 0;
    if (f && !a.gate) factors(l, a, 0, q, p);
    l.params(g2, a.g2, 1.0f);
    l.params(b2, a.b2, 0.0f);
    for (int i = 0; i < iters; ++i) {
        const int row = r0 + i * a.slots + l.slot;
        const bool on = row < r1;
        copy_wait<D - 2>();
        const Raw *d = ring + (i % D) * (2 * NV) * nt;
        float2 y[P], u[P];
        R::get(l, d, nt, y);
        if (f) R::get(l, d + NV * nt, nt, u);
        ask(i + D - 1);
        float2 one = make_float2(0.0f, 1.0f), two = one;
        if (f) {
            if (a.gate && on) {
                const int n = row / a.HW;
                if (n != image) factors(l, a, image = n, q, p);
            }
            if (a.post != CONV_NORM_NONE) one = normalise<VEC, K>(l, sum, u, a.post, a.inv_c, a.eps);
#pragma unroll
            for (int k = 0; k < P; ++k) y[k] = fma2(q[k], u[k], add2(y[k], p[k]));
            if (a.o0 && on) R::put(l, static_cast<T *>(a.o0) + row * a.p0, y);
        }
        if (a.o1) {
            two = normalise<VEC, K>(l, sum, y, a.pre, a.inv_c, a.eps);
#pragma unroll
            for (int k = 0; k < P; ++k) y[k] = fma2(y[k], g2[k], b2[k]);
            if (on) R::put(l, static_cast<T *>(a.o1) + row * a.p1, y);
        }
        if (a.stats && on && l.t == 0) a.stats[row] = make_float4(one.x, one.y, two.x, two.y);
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

// dx and df of the rows of a CTA's units, and the units' channel sums.
template <typename T, int VEC, int K>
__global__ void __launch_bounds__(K == 1 ? kThreads * 2 : kMostThreads) bn_bwd_kernel(const __grid_constant__ BnArgs a) {
    using R = Row<T, VEC, K>;
    using Raw = typename R::Raw;
    constexpr int P = R::P, NV = R::NV, D = bwd_stages(sizeof(T), K);
    extern __shared__ __align__(16) uint8_t smem[];
    __shared__ float2 meet[2 * kMostThreads / 32];
    const int nt = blockDim.x;
    Raw *ring = reinterpret_cast<Raw *>(smem) + threadIdx.x;  // [D][4][NV][threads]
    float *held = reinterpret_cast<float *>(smem + (size_t)D * 4 * NV * nt * sizeof(Raw));  // whole images: gate A, gate B [2][C]
    const Lane<VEC, K> l(a);
    RowSum sum(a.tpr, l.slot, meet);
    const T *x = static_cast<const T *>(a.x), *f = static_cast<const T *>(a.f);
    const T *dy = static_cast<const T *>(a.dy), *dz = static_cast<const T *>(a.dz);
    pdl_trigger();
    pdl_wait();
    float2 q[P], p[P], g2[P], acc[SUMS][P];
#pragma unroll
    for (int s = 0; s < SUMS; ++s)
#pragma unroll
        for (int i = 0; i < P; ++i) acc[s][i] = make_float2(0.0f, 0.0f);
    l.params(g2, a.g2, 1.0f);
    if (f && !a.gate) factors(l, a, 0, q, p);
    if (a.whole) {
        for (int c = threadIdx.x; c < 2 * a.C; c += nt) held[c] = 0.0f;
        __syncthreads();
    }
    for (int unit = blockIdx.x; unit < a.units; unit += gridDim.x) {
        const int n = unit / a.S, s0 = unit - n * a.S;
        const int span = a.gate ? a.HW : a.rows;
        const int r0 = n * span + min(span, s0 * a.run), r1 = n * span + min(span, (s0 + 1) * a.run);
        const int iters = (r1 - r0 + a.slots - 1) / a.slots;
        auto ask = [&](int i) {
            const int row = r0 + i * a.slots + l.slot;
            if (row < r1) {
                Raw *d = ring + (i % D) * (4 * NV) * nt;
                R::ask(l, x + row * a.px, d, nt);
                if (f) R::ask(l, f + row * a.pf, d + NV * nt, nt);
                if (dy) R::ask(l, dy + row * a.pdy, d + 2 * NV * nt, nt);
                if (dz) R::ask(l, dz + row * a.pdz, d + 3 * NV * nt, nt);
            }
            copy_commit();
        };
#pragma unroll
        for (int i = 0; i < (D > 1 ? D - 1 : 1); ++i) ask(i);
        if (f && a.gate) factors(l, a, n, q, p);
        for (int i = 0; i < iters; ++i) {
            const int row = r0 + i * a.slots + l.slot;
            const bool on = row < r1;
            const float4 st = on ? a.stats[row] : make_float4(0.0f, 0.0f, 0.0f, 0.0f);
            copy_wait<(D > 1 ? D - 2 : 0)>();
            const Raw *d = ring + (i % D) * (4 * NV) * nt;
            float2 u[P], y[P], t[P];  // u^, y^, dY
            R::get(l, d, nt, y);
            if (f) R::get(l, d + NV * nt, nt, u);
            if (dy) R::get(l, d + 2 * NV * nt, nt, t);
            else
#pragma unroll
                for (int k = 0; k < P; ++k) t[k] = make_float2(0.0f, 0.0f);
            if (f)
#pragma unroll
                for (int k = 0; k < P; ++k) {
                    u[k] = mul2(add2(u[k], both(-st.x)), both(st.y));
                    y[k] = fma2(q[k], u[k], add2(y[k], p[k]));
                }
            if (dz) {
                float2 e[P], w = make_float2(0.0f, 0.0f), v = w;
                R::get(l, d + 3 * NV * nt, nt, e);
#pragma unroll
                for (int k = 0; k < P; ++k) {
                    y[k] = mul2(add2(y[k], both(-st.z)), both(st.w));
                    if (on) {
                        acc[SUM_G2][k] = fma2(e[k], y[k], acc[SUM_G2][k]);
                        acc[SUM_B2][k] = add2(acc[SUM_B2][k], e[k]);
                    }
                    e[k] = mul2(e[k], g2[k]);
                    w = add2(w, e[k]);
                    v = fma2(e[k], y[k], v);
                }
                const float2 s = sum(make_float2(w.x + w.y, v.x + v.y));
                const float m = a.pre == CONV_NORM_LAYER ? -s.x * a.inv_c : 0.0f, my = -s.y * a.inv_c;
#pragma unroll
                for (int k = 0; k < P; ++k) t[k] = fma2(fma2(y[k], both(my), add2(e[k], both(m))), both(st.w), t[k]);
            }
            if (D > 1) ask(i + D - 1);
            if (on) R::put(l, static_cast<T *>(a.o0) + row * a.p0, t);
            if (f) {
                if (on)
#pragma unroll
                    for (int k = 0; k < P; ++k) {
                        acc[SUM_A][k] = fma2(t[k], u[k], acc[SUM_A][k]);
                        acc[SUM_B][k] = add2(acc[SUM_B][k], t[k]);
                    }
#pragma unroll
                for (int k = 0; k < P; ++k) t[k] = mul2(t[k], q[k]);
                if (a.post != CONV_NORM_NONE) {
                    float2 w = make_float2(0.0f, 0.0f), v = w;
#pragma unroll
                    for (int k = 0; k < P; ++k) {
                        w = add2(w, t[k]);
                        v = fma2(t[k], u[k], v);
                    }
                    const float2 s = sum(make_float2(w.x + w.y, v.x + v.y));
                    const float m = a.post == CONV_NORM_LAYER ? -s.x * a.inv_c : 0.0f, mu = -s.y * a.inv_c;
#pragma unroll
                    for (int k = 0; k < P; ++k) t[k] = mul2(fma2(u[k], both(mu), add2(t[k], both(m))), both(st.y));
                }
                if (on) R::put(l, static_cast<T *>(a.o1) + row * a.p1, t);
            }
            if (D == 1) ask(i + 1);
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
                    a.part[((long long)blockIdx.x * SUMS + s) * a.C + c] = k;
                }
            });
            if (a.dgate) {
                __syncthreads();
                const float *one = a.part + (long long)blockIdx.x * SUMS * a.C;
                for (int c = threadIdx.x; c < a.C; c += nt) a.dgate[(long long)n * a.C + c] = one[c] + one[a.C + c];
                __syncthreads();
            }
#pragma unroll
            for (int i = 0; i < P; ++i) acc[SUM_A][i] = acc[SUM_B][i] = make_float2(0.0f, 0.0f);
        } else {
            combine<0, SUMS, VEC, K>(l, a.slots, acc, ent, [&](int s, int c, float v) {
                a.part[((long long)unit * SUMS + s) * a.C + c] = v;
            });
        }
    }
    if (a.whole) {
        combine<SUM_G2, 2, VEC, K>(l, a.slots, acc, reinterpret_cast<float2 *>(smem), [&](int s, int c, float v) {
            a.part[((long long)blockIdx.x * SUMS + s) * a.C + c] = v;
        });
        __syncthreads();
        for (int c = threadIdx.x; c < 2 * a.C; c += nt) a.part[(long long)blockIdx.x * SUMS * a.C + c] = held[c];
    }
}

// Joins the units' sums.  A CTA takes eight channels; four units a warp at a
// time.  Blocks y = 0 sum over all units, those above one image a warp.
constexpr int kJoin = 1024;
__global__ void __launch_bounds__(kJoin) bn_join_kernel(const __grid_constant__ BnArgs a, int parts) {
    __shared__ float red[SUMS][8][kJoin / 32];
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, c = blockIdx.x * 8 + (lane & 7), group = lane >> 3;
    pdl_trigger();
    pdl_wait();
    const float scale = a.scale && c < a.C ? a.scale[c] : 1.0f, g1 = a.g1 && c < a.C ? a.g1[c] : 1.0f;
    const float b1 = a.b1 && c < a.C ? a.b1[c] : 0.0f;
    if (blockIdx.y > 0) {  // dgate of one image (its units are the runs of that image)
        const int n = (blockIdx.y - 1) * (kJoin / 32) + warp;
        float A = 0.0f, B = 0.0f;
        if (n < a.N && c < a.C)
            for (int s = group; s < a.S; s += 4) {
                const float *u = a.part + ((long long)n * a.S + s) * SUMS * a.C + c;
                A += u[SUM_A * a.C];
                B += u[SUM_B * a.C];
            }
#pragma unroll
        for (int o = 8; o < 32; o *= 2) {
            A += __shfl_xor_sync(0xffffffffu, A, o);
            B += __shfl_xor_sync(0xffffffffu, B, o);
        }
        if (n < a.N && c < a.C && group == 0) a.dgate[(long long)n * a.C + c] = scale * (g1 * A + b1 * B);
        return;
    }
    float v[SUMS] = {0.0f, 0.0f, 0.0f, 0.0f};
    if (c < a.C)
        for (int u = warp * 4 + group; u < parts; u += kJoin / 8) {
            const float *one = a.part + (long long)u * SUMS * a.C + c;
            const float gate = a.gate && !a.whole ? a.gate[(long long)(u / a.S) * a.C + c] : 1.0f;
            v[SUM_A] += gate * one[SUM_A * a.C];
            v[SUM_B] += gate * one[SUM_B * a.C];
            v[SUM_G2] += one[SUM_G2 * a.C];
            v[SUM_B2] += one[SUM_B2 * a.C];
        }
#pragma unroll
    for (int s = 0; s < SUMS; ++s) {
#pragma unroll
        for (int o = 8; o < 32; o *= 2) v[s] += __shfl_xor_sync(0xffffffffu, v[s], o);
        if (group == 0) red[s][lane & 7][warp] = v[s];
    }
    __syncthreads();
    if (warp < 8) {  // a channel a warp
        const int k = blockIdx.x * 8 + warp;
#pragma unroll
        for (int s = 0; s < SUMS; ++s) v[s] = warp_sum(red[s][warp][lane]);
        if (lane == 0 && k < a.C) {
            const float sc = a.scale ? a.scale[k] : 1.0f;
            if (a.dscale) a.dscale[k] = (a.g1 ? a.g1[k] : 1.0f) * v[SUM_A] + (a.b1 ? a.b1[k] : 0.0f) * v[SUM_B];
            if (a.dg1) a.dg1[k] = sc * v[SUM_A];
            if (a.db1) a.db1[k] = sc * v[SUM_B];
            if (a.dg2) a.dg2[k] = v[SUM_G2];
            if (a.db2) a.db2[k] = v[SUM_B2];
        }
    }
}

// ------------------------------------------------------------------ host side
template <typename T, int VEC>
const void *pick_k(bool bwd, int k) {
    if (bwd) return k == 1 ? (const void *)&bn_bwd_kernel<T, VEC, 1> : (const void *)&bn_bwd_kernel<T, VEC, 2>;
    return k == 1 ? (const void *)&bn_fwd_kernel<T, VEC, 1> : (const void *)&bn_fwd_kernel<T, VEC, 2>;
}
const void *pick_kernel(bool bwd, conv_dtype_t dt, int vec, int k) {
    if (dt == CONV_F32) return vec == 4 ? pick_k<float, 4>(bwd, k) : pick_k<float, 1>(bwd, k);
    return vec == 8 ? pick_k<__nv_bfloat16, 8>(bwd, k)
                    : (vec == 2 ? pick_k<__nv_bfloat16, 2>(bwd, k) : pick_k<__nv_bfloat16, 1>(bwd, k));
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
size_t ring_bytes(const BnGeom &g, int es, bool bwd) {
    return (size_t)(bwd ? 4 * bwd_stages(es, g.k) : 2 * kFwdStages) * g.threads * 8 * g.k * es;
}

cudaError_t launch(const conv_plan *p, bool bwd, int vec, BnArgs &a, int grid, size_t smem, cudaStream_t st) {
    const void *k = pick_kernel(bwd, p->dtype, vec, p->bn.k);
    if (smem > 40 * 1024) {  // (with the kernel's static shared memory: 48 KB are free)
        const int rc = conv_grant_smem_once(k, p->device, (int)smem);
        if (rc != CONV_OK) return cudaErrorInvalidValue;
    }
    void *args[] = {&a};
    return conv_launch(k, dim3((unsigned)grid), dim3((unsigned)p->bn.threads), args, smem, st);
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
    g.slots = tpr <= kThreads ? kThreads / tpr : 1;
    g.threads = g.tpr * g.slots;
    const long long rows = (long long)p->s.n * p->s.h * p->s.w;
    auto per_sm = [&](size_t smem, int most) {
        int n = (int)((size_t)(220 * 1024) / (smem + 1024));
        if (n > most) n = most;
        return n < 1 ? 1 : n;
    };
    const int regs = 512 * 128 / (g.threads * 128);  // CTAs a SM of 128 registers a thread
    const long long fwd = (long long)p->num_sms * per_sm(ring_bytes(g, es, false), regs > 4 ? 4 : regs);
    const long long bwd = (long long)p->num_sms * per_sm(ring_bytes(g, es, true), regs > 2 ? 2 : regs);
    auto up = [](long long a, long long b) { return (a + b - 1) / b; };
    // forward: runs of whole sets of rows side by side, one wave of CTAs
    long long run = up(up(rows, fwd), g.slots) * g.slots;
    if (run < g.slots) run = g.slots;
    g.run = (int)run;
    g.grid = (int)up(rows, run);
    // gradient without a gate: the same over all rows
    run = up(up(rows, bwd), g.slots) * g.slots;
    if (run < g.slots) run = g.slots;
    g.open.run = (int)run;
    g.open.S = g.open.units = g.open.grid = (int)up(rows, run);
    g.open.whole = 0;
    // with one: whole images, or runs of an image where that leaves SMs idle.
    // A run costs its sets of rows and about four more for its start and end.
    const long long N = p->s.n, HW = (long long)p->s.h * p->s.w;
    long long best = -1;
    for (int S = 1; S <= 1024 && N > 0; ++S) {
        const long long sets = up(up(HW, S), g.slots);
        if (S > 1 && up(HW, sets * g.slots) != S) continue;
        const long long cost = up(N * S, bwd) * (sets + 4);
        if (best < 0 || cost < best) {
            best = cost;
            g.gated.S = S;
            g.gated.run = (int)(S == 1 ? HW : sets * g.slots);
        }
    }
    if (N > 0) {
        g.gated.units = (int)(N * g.gated.S);
        g.gated.whole = g.gated.S == 1;
        g.gated.grid = (int)(g.gated.whole && N > bwd ? bwd : g.gated.units);
    }
    const long long parts = g.open.grid > g.gated.grid ? g.open.grid : g.gated.grid;
    p->ws_bytes = 0;
    p->ws_bwd_bytes = (size_t)parts * SUMS * C * 4;
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
             dtype == CONV_F32 ? "f32" : "bf16", names[post], names[pre], p->bn.slots, p->bn.tpr, 8 * p->bn.k, p->bn.grid,
             p->bn.open.grid, p->bn.gated.units, p->bn.gated.grid);
    *out_plan = p;
    return CONV_OK;
}

namespace {
BnArgs base_args(const conv_plan *p, const conv_blocknorm_params_t &w, const void *x, int64_t px, const void *f, int64_t pf) {
    BnArgs a = {};
    a.x = x; a.px = px; a.f = f; a.pf = pf;
    a.scale = w.scale; a.gate = w.gate; a.g1 = w.post_gamma; a.b1 = w.post_beta; a.g2 = w.pre_gamma; a.b2 = w.pre_beta;
    a.eps = p->bn.eps; a.inv_c = 1.0f / (float)p->s.c_in;
    a.N = p->s.n; a.HW = p->s.h * p->s.w; a.rows = a.N * a.HW; a.C = p->s.c_in;
    a.post = p->bn.post; a.pre = p->bn.pre;
    a.tpr = p->bn.tpr; a.slots = p->bn.slots;
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
    a.run = p->bn.run;
    const Map all[4] = {in[0], in[1], out[0], out[1]};
    return launch(p, false, vec_for(p, all), a, p->bn.grid, ring_bytes(p->bn, es, false), (cudaStream_t)stream) == cudaSuccess
               ? CONV_OK : CONV_ERR_CUDA;
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
    const BnGeom::Bwd &g = w.gate ? p->bn.gated : p->bn.open;
    a.run = g.run; a.S = g.S; a.units = g.units; a.whole = g.whole;
    const Map all[6] = {in[0], in[1], in[2], in[3], out[0], out[1]};
    const size_t smem = ring_bytes(p->bn, es, true) + (g.whole ? 2 * cb : 0);
    if (launch(p, true, vec_for(p, all), a, g.grid, smem, st) != cudaSuccess) return CONV_ERR_CUDA;
    const bool sums = d.scale || d.post_gamma || d.post_beta || d.pre_gamma || d.pre_beta, images = d.gate && !g.whole;
    if (!sums && !images) return CONV_OK;
    int parts = g.grid;
    void *args[] = {&a, &parts};
    const dim3 grid((unsigned)((C + 7) / 8), 1 + (unsigned)(images ? (a.N + kJoin / 32 - 1) / (kJoin / 32) : 0));
    return conv_launch((const void *)&bn_join_kernel, grid, dim3(kJoin), args, 0, st) == cudaSuccess ? CONV_OK : CONV_ERR_CUDA;
}
