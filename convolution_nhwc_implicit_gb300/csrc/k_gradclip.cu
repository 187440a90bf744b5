// The global norm of many gradients, and clipping:
//   norm = sqrt(sum g^2)    k = min(1, max_norm / (norm + 1e-6))    out = k g
// over all elements of a list of tensors.  Two operations an element: memory
// bounds it, one reading for the norm and another with the writing.
//
// Two launches: the first sums squares and leaves a sum a CTA in the workspace,
// the second joins these (every CTA for itself, in the same order), and writes.
// The elements of all tensors, one after the other, are divided evenly among
// the CTAs; a CTA's share is cut at tensors' ends and into items of a few
// thousand elements, one of its warps to an item.  The plan holds that table on
// the device; addresses come with each call as kernel parameters.
//
// Measured on a GB300 by graph replay: 1.0 billion bf16 elements 925 us, 6.2 GB in
// its three passes (two readings, one writing) at 6.7 TB/s, of which the norm
// cannot spare one: the 602 us of two would need it before the first reading;
// 0.37 GB that need no clipping 59 us, one pass at 6.2 TB/s; 66 MB 31 us (the
// second reading from L2).  Sets up to 1.5 MB take one launch of one cluster of
// sixteen CTAs, 5.2 us for 0.55 MB where two launches took 5.9: the call then
// costs 11 us on the host instead of 21.
//
// A lane sums the squares of an item in fp32 (up to about 130 terms), and items
// in fp64.  Where a lane's sum would overflow (above 2^100, or not finite) or
// its squares vanish (below 2^-100, but not all zero), the item is read again
// and its elements scaled by a power of two.
#include <cuda_bf16.h>
#include <math.h>
#include <stdint.h>
#include <stdio.h>
#include <string.h>

#include <algorithm>
#include <new>
#include <vector>

#include "conv_internal.h"
#include "epilogue.cuh"
#include "maps.cuh"

using namespace convk;

// Items of one launch: consecutive tensors, as many as its parameters hold.
struct ClipBatch {
    int t0, t1, grid;
    int first;  // of its CTAs' entries in the table of first items
    int part;   // of its CTAs' sums
};
struct ClipGeom {
    std::vector<int64_t> counts;
    std::vector<uint8_t> es;
    std::vector<ClipBatch> batches;
    int parts = 0;
    bool small = false;  // one launch of one cluster
    int past = 0;        // the second reading and the results go past L2
    uint4 *items = nullptr;  // device: (tensor of the batch | fp32 << 31, elements, first element as two words)
    int *first = nullptr;    // after them: [grid + 1] of each batch
};

namespace {

constexpr int kThreads = 512, kWarps = kThreads / 32;
constexpr int kCtas = 2;          // a SM
constexpr int kItem = 4096;       // elements of an item, at most
constexpr int kItemLeast = 256;   // ... and at least, but for a tensor's end: a vector a lane
constexpr int kCluster = 16;      // CTAs of the one-launch form, and the bytes up to which it is taken
constexpr long long kSmall = 1536 * 1024;
// Bytes of a set whose second reading and whose results do not displace what is
// still to be read in L2 (66 MB 34.0 us, 31.5 so; 247 MB 122.4 and 120.6; 2.1 GB,
// of which L2 holds a twentieth, 916 and 926).
constexpr long long kPast = 1ll << 29;
constexpr int kTurn = 1024;       // elements of four vectors a lane, bf16
constexpr int kMostTensors = 1900;  // of a launch: their addresses are kernel parameters (32 KB at most)

template <int M> struct Tensors { const void *p[M]; };

template <typename T> struct Words;  // 16 bytes as fp32 pairs
template <> struct Words<float> : Vec<float, 4> { static constexpr int N = 4; };
template <> struct Words<__nv_bfloat16> : Vec<__nv_bfloat16, 8> { static constexpr int N = 8; };

// A tensor's piece as a warp takes it: up to N - 1 elements before the first
// 16-byte address, whole vectors, and up to N - 1 elements after them.
struct Cut {
    int head, vecs, tail;
    __device__ __forceinline__ Cut(const void *p, int n, int N, int es) {
        head = min(n, (int)((16u - (unsigned)(uintptr_t)p % 16u) % 16u) / es);
        vecs = (n - head) / N;
        tail = n - head - vecs * N;
    }
};

__device__ __forceinline__ uint32_t bits(const uint4 &v) { return (v.x | v.y | v.z | v.w) & 0x7fff7fffu; }
__device__ __forceinline__ uint32_t bits(const float4 &v) {
    return (__float_as_uint(v.x) | __float_as_uint(v.y) | __float_as_uint(v.z) | __float_as_uint(v.w)) & 0x7fffffffu;
}

// A lane's sum of (by g)^2 over its elements of an item; any: whether one is not 0.
template <typename T>
__device__ __forceinline__ float squares(const T *p, int n, float by, bool &any) {
    using W = Words<T>;
    using Raw = typename W::Raw;
    constexpr int U = 4;
    const int lane = threadIdx.x & 31;
    const Cut c(p, n, W::N, sizeof(T));
    float one = lane < c.head ? Elem<T>::to_f(p[lane]) * by : 0.0f;
    float two = lane < c.tail ? Elem<T>::to_f(p[c.head + c.vecs * W::N + lane]) * by : 0.0f;
    uint32_t seen = (one != 0.0f || two != 0.0f) ? 1u : 0u;
    const Raw *v = reinterpret_cast<const Raw *>(p + c.head);
    float2 s[2] = {make_float2(one * one, two * two), make_float2(0.0f, 0.0f)};
    for (int i = lane; i < c.vecs; i += 32 * U) {
        Raw r[U];
#pragma unroll
        for (int u = 0; u < U; ++u) {
            if (i + 32 * u < c.vecs) r[u] = v[i + 32 * u];
            else r[u] = Raw{};
        }
#pragma unroll
        for (int u = 0; u < U; ++u) {
            float2 f[W::kPairs];
            W::unpack(r[u], f);
            seen |= bits(r[u]);
#pragma unroll
            for (int e = 0; e < W::kPairs; ++e) {
                f[e] = mul2(f[e], make_float2(by, by));
                s[e % 2] = fma2(f[e], f[e], s[e % 2]);
            }
        }
    }
    any = seen != 0;
    return (s[0].x + s[0].y) + (s[1].x + s[1].y);
}

template <typename T>
__device__ __forceinline__ double item_sum(const T *p, int n) {
    bool any;
    const float s = squares(p, n, 1.0f, any);
    const bool high = !(s <= 0x1p100f), low = any && s < 0x1p-100f;
    double d = (double)s;
    if (__any_sync(0xffffffffu, high || low)) {
        const float t = squares(p, n, high ? 0x1p-70f : 0x1p100f, any);
        if (high) d = (double)t * 0x1p140;
        else if (low) d = (double)t * 0x1p-200;
    }
    return d;
}

__device__ __forceinline__ double warp_sum64(double v) {
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
    return v;
}
// A warp's sum of squares over items i, i + kWarps, ... before `end`; it is the
// first of them.
template <int M>
__device__ __forceinline__ double sum_items(const Tensors<M> &t, const uint4 *items, int i, int end, uint4 it) {
    double s = 0.0;
    while (i < end) {
        const uint4 now = it;
        i += kWarps;
        if (i < end) it = items[i];
        const long long at = (long long)(((unsigned long long)now.w << 32) | now.z);
        const void *p = t.p[now.x & 0x7fffffffu];
        if (now.x >> 31) s += item_sum(static_cast<const float *>(p) + at, (int)now.y);
        else s += item_sum(static_cast<const __nv_bfloat16 *>(p) + at, (int)now.y);
    }
    return s;
}
// The CTA's sum of its warps' lanes' sums, in the first warp.
__device__ __forceinline__ double cta_sum(double s, double *red) {
    s = warp_sum64(s);
    if ((threadIdx.x & 31) == 0) red[threadIdx.x >> 5] = s;
    __syncthreads();
    return threadIdx.x < 32 ? warp_sum64(threadIdx.x < kWarps ? red[threadIdx.x] : 0.0) : 0.0;
}

template <int M>
__global__ void __launch_bounds__(kThreads, kCtas) clip_norm_kernel(const __grid_constant__ Tensors<M> t, const uint4 *items,
                                                                    const int *first, double *part) {
    __shared__ double red[kWarps];
    pdl_trigger();
    const int end = first[blockIdx.x + 1], i = first[blockIdx.x] + (int)(threadIdx.x >> 5);
    const uint4 it = i < end ? items[i] : make_uint4(0, 0, 0, 0);
    pdl_wait();
    const double s = cta_sum(sum_items(t, items, i, end, it), red);
    if (threadIdx.x == 0) part[blockIdx.x] = s;
}

// past: read and written as data that is not used again soon.
template <typename T>
__device__ __forceinline__ void scale_item(const T *p, T *q, int n, float k, bool past) {
    using W = Words<T>;
    using Raw = typename W::Raw;
    constexpr int U = 4;
    const int lane = threadIdx.x & 31;
    if (((uintptr_t)p ^ (uintptr_t)q) & 15u) {  // vectors of one are no vectors of the other
        for (int i = lane; i < n; i += 32) q[i] = Elem<T>::from_f(Elem<T>::to_f(p[i]) * k);
        return;
    }
    const Cut c(p, n, W::N, sizeof(T));
    const int end = c.head + c.vecs * W::N;
    if (lane < c.head) q[lane] = Elem<T>::from_f(Elem<T>::to_f(p[lane]) * k);
    if (lane < c.tail) q[end + lane] = Elem<T>::from_f(Elem<T>::to_f(p[end + lane]) * k);
    const Raw *v = reinterpret_cast<const Raw *>(p + c.head);
    Raw *o = reinterpret_cast<Raw *>(q + c.head);
    for (int i = lane; i < c.vecs; i += 32 * U) {
        Raw r[U];
#pragma unroll
        for (int u = 0; u < U; ++u)
            if (i + 32 * u < c.vecs) r[u] = past ? __ldcs(v + i + 32 * u) : v[i + 32 * u];
#pragma unroll
        for (int u = 0; u < U; ++u)
            if (i + 32 * u < c.vecs) {
                float2 f[W::kPairs];
                W::unpack(r[u], f);
#pragma unroll
                for (int e = 0; e < W::kPairs; ++e) f[e] = mul2(f[e], make_float2(k, k));
                if (past) __stcs(o + i + 32 * u, W::pack(f));
                else o[i + 32 * u] = W::pack(f);
            }
    }
}

// The root of a sum in fp32: s = m 4^e with m in [1, 4), and the fp32 root r of m
// with a step of Newton's, r + (m - r^2) / 2r, whose difference is taken in fp64:
// off by half a rounding and little more.  (fp64 has a root of its own, some
// forty instructions on a unit that takes sixteen clocks for each: with it and a
// division in every warp the second launch took 12 us where nothing was to be
// clipped.)
__device__ __forceinline__ float root32(double s) {
    const int high = __double2hiint(s), e = (high >> 20) - 1023;
    if (s == 0.0 || e >= 1024) return (float)s;  // (infinite or NaN)
    const double m = __hiloint2double((high & 0xfffff) | (1023 + (e & 1)) << 20, __double2loint(s));
    const float r = sqrtf((float)m), rest = (float)fma(-(double)r, (double)r, m);
    return scalbnf(r + 0.5f * rest / r, (e - (e & 1)) / 2);
}

// k for a norm.
__device__ __forceinline__ float clip_factor(float norm, float max_norm) {
    return isfinite(norm) ? fminf(1.0f, max_norm / (norm + 1e-6f)) : 1.0f;
}
// A warp's items i, i - kWarps, ... down to `start`, times k: from the end, which
// is what is still in L2.  it: the first of them.
template <int M>
__device__ __forceinline__ void scale_items(const Tensors<M> &t, const Tensors<M> &o, const uint4 *items, int i, int start, uint4 it, float k,
                                            bool past) {
    while (i >= start) {
        const uint4 now = it;
        i -= kWarps;
        if (i >= start) it = items[i];
        const long long at = (long long)(((unsigned long long)now.w << 32) | now.z);
        const int j = now.x & 0x7fffffffu;
        if (now.x >> 31) scale_item(static_cast<const float *>(t.p[j]) + at, (float *)o.p[j] + at, (int)now.y, k, past);
        else scale_item(static_cast<const __nv_bfloat16 *>(t.p[j]) + at, (__nv_bfloat16 *)o.p[j] + at, (int)now.y, k, past);
    }
}

// in place: outs are the gradients, which stay as they are where k = 1.
template <int M>
__global__ void __launch_bounds__(kThreads, kCtas) clip_scale_kernel(const __grid_constant__ Tensors<M> t,
                                                                     const __grid_constant__ Tensors<M> o, const uint4 *items,
                                                                     const int *first, const double *part, int parts,
                                                                     float max_norm, float *norm, int in_place, int past) {
    __shared__ float factor;
    pdl_trigger();
    const int start = first[blockIdx.x], i = first[blockIdx.x + 1] - 1 - (int)(threadIdx.x >> 5);
    const uint4 it = i >= start ? items[i] : make_uint4(0, 0, 0, 0);
    pdl_wait();
    if (threadIdx.x < 32) {
        double s = 0.0;
        for (int j = threadIdx.x; j < parts; j += 32) s += part[j];
        const float whole = root32(warp_sum64(s));
        if (threadIdx.x == 0) {
            factor = clip_factor(whole, max_norm);
            if (norm && blockIdx.x == 0) *norm = whole;
        }
    }
    __syncthreads();
    if (in_place && factor == 1.0f) return;
    scale_items(t, o, items, i, start, it, factor, past);
}

// Both of a small set in one launch: one cluster, whose CTAs read each other's
// sums.
template <int M>
__global__ void __launch_bounds__(kThreads, kCtas) clip_small_kernel(const __grid_constant__ Tensors<M> t,
                                                                     const __grid_constant__ Tensors<M> o, const uint4 *items,
                                                                     const int *first, float max_norm, float *norm, int in_place) {
    __shared__ double red[kWarps], mine;
    __shared__ float factor;
    pdl_trigger();
    const int start = first[blockIdx.x], end = first[blockIdx.x + 1], warp = (int)(threadIdx.x >> 5), i = start + warp;
    const int last = end - 1 - warp;
    const uint4 it = i < end ? items[i] : make_uint4(0, 0, 0, 0), back = last >= start ? items[last] : make_uint4(0, 0, 0, 0);
    pdl_wait();
    double s = cta_sum(sum_items(t, items, i, end, it), red);
    if (threadIdx.x == 0) mine = s;
    cluster_arrive();
    cluster_wait();
    if (threadIdx.x < 32) {
        s = 0.0;
        if (threadIdx.x < gridDim.x) {
            const uint32_t at = tc::mapa_shared(tc::smem_u32(&mine), threadIdx.x);
            asm volatile("ld.shared::cluster.f64 %0, [%1];" : "=d"(s) : "r"(at) : "memory");
        }
        const float whole = root32(warp_sum64(s));
        if (threadIdx.x == 0) {
            factor = clip_factor(whole, max_norm);
            if (blockIdx.x == 0) *norm = whole;
        }
    }
    cluster_arrive();  // (no CTA ends while its sum may still be read)
    __syncthreads();
    if (!in_place || factor != 1.0f) scale_items(t, o, items, last, start, back, factor, false);
    cluster_wait();
}

// ------------------------------------------------------------------ host side
struct Run {
    const ClipGeom *g;
    void *const *grads, *const *outs;
    float max_norm, *norm;
    double *part;
    cudaStream_t st;
};

enum { NORM, SCALE, SMALL };
template <int M>
cudaError_t launch(const Run &r, const ClipBatch &b, int which) {
    Tensors<M> t, o;
    for (int i = b.t0; i < b.t1; ++i) {
        t.p[i - b.t0] = r.grads[i];
        o.p[i - b.t0] = r.outs ? r.outs[i] : r.grads[i];
    }
    const uint4 *items = r.g->items;
    const int *first = r.g->first + b.first;
    int parts = r.g->parts, in_place = r.outs == nullptr;
    float max_norm = r.max_norm, *norm = b.part == 0 ? r.norm : nullptr;
    if (which == SMALL) {
        void *args[] = {&t, &o, &items, &first, &max_norm, &norm, &in_place};
        return conv_launch((const void *)&clip_small_kernel<M>, dim3((unsigned)b.grid), dim3(kThreads), args, 0, r.st, b.grid);
    }
    if (which == NORM) {
        double *part = r.part + b.part;
        void *args[] = {&t, &items, &first, &part};
        return conv_launch((const void *)&clip_norm_kernel<M>, dim3((unsigned)b.grid), dim3(kThreads), args, 0, r.st);
    }
    const double *part = r.part;
    int past = r.g->past;
    void *args[] = {&t, &o, &items, &first, &part, &parts, &max_norm, &norm, &in_place, &past};
    return conv_launch((const void *)&clip_scale_kernel<M>, dim3((unsigned)b.grid), dim3(kThreads), args, 0, r.st);
}

const void *small_kernel(int tensors) {
    return tensors <= 32 ? (const void *)&clip_small_kernel<32>
                         : (tensors <= 128 ? (const void *)&clip_small_kernel<128>
                                           : (tensors <= 512 ? (const void *)&clip_small_kernel<512> : (const void *)&clip_small_kernel<kMostTensors>));
}

cudaError_t launch_batch(const Run &r, const ClipBatch &b, int which) {
    const int n = b.t1 - b.t0;
    if (n <= 32) return launch<32>(r, b, which);
    if (n <= 128) return launch<128>(r, b, which);
    return n <= 512 ? launch<512>(r, b, which) : launch<kMostTensors>(r, b, which);
}

// Divides the tensors [b.t0, b.t1) among at most `wave` CTAs.
void divide(const ClipGeom &g, ClipBatch &b, int wave, std::vector<uint4> &items, std::vector<int> &first) {
    long long bytes = 0;
    for (int t = b.t0; t < b.t1; ++t) bytes += (long long)g.counts[t] * g.es[t];
    // at least 4 KB a CTA
    long long grid = std::min<long long>(wave, (bytes + 4095) / 4096);
    if (grid < 1) grid = 1;
    const long long share = ((bytes + grid - 1) / grid + 31) / 32 * 32;
    b.first = (int)first.size();
    first.push_back((int)items.size());
    long long left = share;
    int ctas = 0;
    auto close = [&] {
        first.push_back((int)items.size());
        ++ctas;
        left = share;
    };
    for (int t = b.t0; t < b.t1; ++t) {
        const int es = g.es[t];
        // a warp's elements in one item, in whole turns of its loads where they take several
        const long long per = share / es / kWarps, unit = per > kTurn ? kTurn : kItemLeast;
        const int item = (int)std::max<long long>(kItemLeast, std::min<long long>(kItem, (per + unit - 1) / unit * unit));
        for (long long at = 0; at < g.counts[t];) {
            long long n = std::min<long long>(g.counts[t] - at, item);
            // (a share ends on a whole number of vectors of the tensor)
            if (n * es > left && ctas + 1 < grid) n = std::max<long long>(16, left / es / 16 * 16);
            n = std::min<long long>(n, g.counts[t] - at);
            items.push_back(make_uint4((unsigned)(t - b.t0) | (es == 4 ? 0x80000000u : 0u), (unsigned)n, (unsigned)at,
                                       (unsigned)((unsigned long long)at >> 32)));
            at += n;
            left -= n * es;
            if (left <= 0 && ctas + 1 < grid) close();
        }
    }
    if (first.back() != (int)items.size() || ctas == 0) close();
    b.grid = ctas;
}

// Whether a tensor that the run writes shares a byte with another.  (Each list is
// most often in the order of its addresses already.)
struct Range {
    uintptr_t from, to;
    bool written;
    bool operator<(const Range &o) const { return from < o.from; }
};
bool overlap(std::vector<Range> &in, std::vector<Range> &out) {
    for (std::vector<Range> *r : {&in, &out})
        if (!std::is_sorted(r->begin(), r->end())) std::sort(r->begin(), r->end());
    uintptr_t any = 0, written = 0;  // ends of what came before
    auto a = in.begin(), b = out.begin();
    while (a != in.end() || b != out.end()) {
        const Range &i = b == out.end() || (a != in.end() && *a < *b) ? *a++ : *b++;
        if (i.from < (i.written ? any : written)) return true;
        any = std::max(any, i.to);
        if (i.written) written = std::max(written, i.to);
    }
    return false;
}

}  // namespace

void clip_destroy(ClipGeom *g) {
    if (!g) return;
    if (g->items) cudaFree(g->items);
    delete g;
}
int clip_launches(const ClipGeom *g) { return g->small ? 1 : 2 * (int)g->batches.size(); }

extern "C" int conv_plan_create_gradclip(int32_t tensors, const int64_t *counts, const conv_dtype_t *dtypes,
                                         conv_plan_t **out_plan) {
    if (!out_plan) return CONV_ERR_NULL_ARG;
    *out_plan = nullptr;
    if (tensors < 0) return CONV_ERR_INVALID_SHAPE;
    if (tensors > 0 && (!counts || !dtypes)) return CONV_ERR_NULL_ARG;
    long long total = 0;
    for (int i = 0; i < tensors; ++i) {
        if (counts[i] < 0) return CONV_ERR_INVALID_SHAPE;
        if ((int)dtypes[i] < CONV_F32 || (int)dtypes[i] > CONV_I8) return CONV_ERR_INVALID_ARG;
        if (dtypes[i] == CONV_I8) return CONV_ERR_UNSUPPORTED;
        if (counts[i] >= (1ll << 40) - total) return CONV_ERR_UNSUPPORTED;
        total += counts[i];
    }
    conv_plan *p = new (std::nothrow) conv_plan();
    if (!p) return CONV_ERR_OOM;
    p->s = {1, 1, 1, 1, 1, 1, 1};
    p->algo = CONV_ALGO_GRADCLIP;
    int rc = conv_plan_bind_device(p, false);
    try {
        if (rc == CONV_OK) {
            p->clip = new ClipGeom();
            ClipGeom &g = *p->clip;
            g.counts.assign(counts, counts + tensors);
            for (int i = 0; i < tensors; ++i) g.es.push_back((uint8_t)conv_esize(dtypes[i]));
            std::vector<uint4> items;
            std::vector<int> first;
            long long bytes = 0;
            for (int i = 0; i < tensors; ++i) bytes += counts[i] * g.es[i];
            g.small = bytes <= kSmall && tensors <= kMostTensors && conv_cluster_fits(small_kernel(tensors), p->device, kCluster, kThreads, 0);
            g.past = bytes < kPast;
            int t = 0;
            do {
                ClipBatch b = {t, std::min(tensors, t + kMostTensors), 0, 0, g.parts};
                divide(g, b, g.small ? kCluster : kCtas * p->num_sms, items, first);
                g.parts += b.grid;
                g.batches.push_back(b);
                t = b.t1;
            } while (t < tensors);
            p->ws_bytes = g.small ? 0 : (size_t)g.parts * sizeof(double);
            // one table: the items, then the CTAs' first ones
            const size_t count = items.size();
            items.resize(count + (first.size() + 3) / 4);
            memcpy(items.data() + count, first.data(), first.size() * sizeof(int));
            const size_t table = items.size() * sizeof(uint4);
            if (cudaMalloc(&g.items, table) != cudaSuccess) rc = CONV_ERR_OOM;
            else rc = conv_upload(g.items, items.data(), table);
            g.first = reinterpret_cast<int *>(g.items + count);
            snprintf(p->desc, sizeof(p->desc), "gradclip %d tensors, %lld elements in %zu items, ctas=%d launches=%d", tensors, total,
                     count, g.parts, clip_launches(&g));
        }
    } catch (...) {
        rc = CONV_ERR_OOM;
    }
    if (rc != CONV_OK) {
        conv_plan_destroy(p);
        return rc;
    }
    *out_plan = p;
    return CONV_OK;
}

extern "C" int conv_run_gradclip(const conv_plan_t *plan, void *const *grads, void *const *outs, float max_norm, float *norm,
                                 void *workspace, void *stream) {
    if (!plan) return CONV_ERR_NULL_ARG;
    const conv_plan *p = plan;
    if (p->algo != CONV_ALGO_GRADCLIP) return CONV_ERR_INVALID_ARG;
    const ClipGeom &g = *p->clip;
    const int tensors = (int)g.counts.size();
    if (!(max_norm > 0.0f)) return CONV_ERR_INVALID_ARG;
    if ((tensors > 0 && !grads) || !norm || (p->ws_bytes && !workspace)) return CONV_ERR_NULL_ARG;
    if (((uintptr_t)norm & 3u) || ((uintptr_t)workspace & 15u)) return CONV_ERR_MISALIGNED;
    try {
        std::vector<Range> read, written;
        read.reserve((size_t)tensors);
        written.reserve((size_t)tensors + 2);
        for (int i = 0; i < tensors; ++i) {
            if (g.counts[i] == 0) continue;
            const uintptr_t in = (uintptr_t)grads[i], out = outs ? (uintptr_t)outs[i] : in;
            if (!in || !out) return CONV_ERR_NULL_ARG;
            if ((in | out) % g.es[i]) return CONV_ERR_MISALIGNED;
            const uintptr_t bytes = (uintptr_t)g.counts[i] * g.es[i];
            written.push_back({out, out + bytes, true});
            if (in != out) read.push_back({in, in + bytes, false});
        }
        if (overlap(read, written)) return CONV_ERR_ALIASING;
        const uintptr_t n0 = (uintptr_t)norm, w0 = (uintptr_t)workspace, w1 = w0 + p->ws_bytes;
        for (const std::vector<Range> *list : {&read, &written})
            for (const Range &i : *list)
                if ((i.from < n0 + 4 && n0 < i.to) || (i.from < w1 && w0 < i.to)) return CONV_ERR_ALIASING;
        if (conv_overlaps(norm, 4, workspace, p->ws_bytes)) return CONV_ERR_ALIASING;
    } catch (...) {
        return CONV_ERR_OOM;
    }
    const Run r = {&g, grads, outs, max_norm, norm, static_cast<double *>(workspace), (cudaStream_t)stream};
    if (g.small) return launch_batch(r, g.batches[0], SMALL) == cudaSuccess ? CONV_OK : CONV_ERR_CUDA;
    for (const int which : {NORM, SCALE})
        for (const ClipBatch &b : g.batches)
            if (launch_batch(r, b, which) != cudaSuccess) return CONV_ERR_CUDA;
    return CONV_OK;
}
