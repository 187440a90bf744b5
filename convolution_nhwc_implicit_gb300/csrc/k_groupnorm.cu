// Group norm with an activation over NHWC maps, forward and gradient.
//
// A group is the cg = C/G consecutive channels of one image, m = H*W*cg
// values:
//   mean = sum x / m        var = sum (x - mean)^2 / m     rstd = 1 / sqrt(var + eps)
//   xhat = (x - mean) rstd  z = gamma xhat + beta          y = act(z)
// and, with dz = dy act'(z),
//   dbeta = sum_{n,p} dz    dgamma = sum_{n,p} dz xhat
//   dx = rstd (gamma dz - (s1 + xhat s2) / m),
//        s1 = sum_group gamma dz,  s2 = sum_group gamma dz xhat.
// About 10 operations a value forward and 30 backward against 2 to 8 bytes
// moved: memory bounds it.
//
// Channels last, a group's values lie cg at a time, C apart, so a thread takes
// one VEC-channel vector (16 bytes where sizes and alignment allow) of every
// R-th pixel and keeps its sums PER CHANNEL: any cg works, odd ones and ones
// that end inside a vector, and channels meet their group only when the CTA's
// sums are joined.  A CTA takes a run of whole pixels, one piece of memory.
//
// Variance: a CTA sums (x - K) and (x - K)^2 of each channel about the first
// value K of its own run, and (mean, M2) of channels and runs are joined by
// Chan's update.  K belongs to the values it is subtracted from, so that the
// cancellation in M2 = q - s^2/n is bounded by the run's length times 2^-24
// however far the mean lies from zero.  All statistics are fp32, in a fixed
// order: results do not change from run to run.
//
// Two forms, chosen by sizes (plan_direction; where a CTA would hold more than
// 256 channels, by a call's addresses too), measured on a GB300 by graph replay
// over changing inputs:
//   clusters    a few groups of an image in the shared memory of one to eight
//               CTAs, one launch.  7x7x512 bf16 3.8 us (as two launches 8.8);
//               8x80x80x256 bf16 with Mish 19.9 us (25.5), 2.6 TB/s of its 52
//               MB; without an activation 17.8 us (22.9), of which a median CTA
//               (clock stamps in an instrumented build) takes 6.3 until its run
//               has come and is summed, 4.7 to join and exchange the sums and
//               3.3 to finish and write.
//   two launches  sums, then results, where a run does not fit.
//               16x160x160x128 fp32 with Mish 110 us: the map is read twice,
//               5.7 TB/s over the three passes of HBM, against 62 us for the two
//               that cannot be avoided.  The gradient of 8x80x80x256 bf16 29.9
//               us: a median CTA (stamped before Mish's slope was clamped, 0.4
//               less in all) takes 7.9 at its pixels in the first launch (x and
//               dy at 6.6 TB/s) and 9.4 in the second, which reads them again
//               from L2 and writes dx; the rest is the launches' starts and ends.
// Tried and slower: one cooperative launch whose CTAs wait for one another's
// sums by image (each further pass adds about 16 us: 8x80x80x256 took 35, 51 and
// 82 us in one, two and four; 151 us at best for the fp32 map); the clusters
// reading the fp32 map twice (113 us against 108 as two launches of the time);
// passes of images that fit L2 (127 to 205 us, each pass paying both launches).
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

constexpr int kThreads = 256;
constexpr int kWarps = kThreads / 32;
// CTAs a SM of the two-launch form: three of the forward kernels' 80 registers;
// two of the gradient's 128 for bf16 (eight channels a thread), three for fp32.
constexpr int kCtas = 3;
__host__ __device__ constexpr int grad_ctas(int es) { return es == 2 ? 2 : kCtas; }
constexpr long long kL2Bytes = 100ll << 20;  // maps beyond this do not stay in L2 from one launch to the next
constexpr int kStageRuns = 4096;             // partial results a CTA stages (32 KB)
// Map bytes of a CTA of a cluster: four CTAs a SM, or two where a cluster of
// eight cannot hold its runs otherwise.  (8x80x80x256 bf16 by CTAs a cluster: 6
// 19.6 us, 8 20.0; 5 and 7, whose clusters need a second wave, 26.7 and 24.5.
// 4 need 102 KB a CTA: 19.3 us in a build that allowed it, where 8 took 19.9.
// That one size is all that was measured above 88 KB, up to which the limit is
// not known to be the best.)
constexpr int kResident = 50 * 1024, kResidentMost = 88 * 1024;
constexpr int kMaxC = 8192;  // channels: their sums stay in shared memory (16 bytes each)

struct GnArgs {
    const void *x, *dy;
    void *out;                 // y, or dx
    long long px, pdy, pout;   // elements from one pixel to the next
    const float *gamma, *beta; // [C] or null
    float *mean, *rstd;        // [N][G] (forward: may be null)
    float *dgamma, *dbeta;     // [C] or null
    float2 *part;              // [N][G][S]: (mean, M2), or (sum gamma dz, sum gamma dz xhat)
    float2 *partc;             // [N][S][C]: (sum dz, sum dz xhat)
    int N, HW, C, G, cg;
    int ppx, S;                // a CTA takes a run of ppx pixels; two launches: S runs an image
    // cluster kernels: groups and channels of a CTA, CTAs an image (a run of
    // pixels each)
    int gb, cb, K, ent;    // ent: entries of the threads' sums in shared memory
    float eps;
    int past_l2;               // two launches: the maps are larger than L2
};

// 1/d of a pair from one hardware reciprocal (its unit is the bound of the
// activations): 1 / (d.x d.y), times the other.  d <= 2.4e17, so that the
// product stays finite; a NaN is put back by its caller's product with z.
__device__ __forceinline__ float2 rcp2(float2 d) {
    const float r = rcp_approx(d.x * d.y);
    return mul2(make_float2(r, r), make_float2(d.y, d.x));
}
// log2 e times a pair clamped at 20, where Mish and its derivative have reached
// their limits z and 1 in fp32 (fminf drops a NaN: see rcp2).
__device__ __forceinline__ float2 exponent(float2 z) {
    return mul2(make_float2(fminf(z.x, 20.0f), fminf(z.y, 20.0f)), make_float2(1.4426950408889634f, 1.4426950408889634f));
}
__device__ __forceinline__ float2 exp2_pair(float2 e) { return make_float2(ex2_approx(e.x), ex2_approx(e.y)); }
// act(z) of a pair.  Mish = z t / (t + 2) with n = e^z, t = n (n + 2): it
// cancels nowhere (~5e-7 relative on the hardware's exp2 and reciprocal).
// ReLU passes NaN on.
template <int ACT>
__device__ __forceinline__ float2 act2(float2 z) {
    if constexpr (ACT == ACT_RELU) return make_float2(z.x < 0.0f ? 0.0f : z.x, z.y < 0.0f ? 0.0f : z.y);
    else if constexpr (ACT == ACT_MISH) {
        const float2 two = make_float2(2.0f, 2.0f);
        const float2 n = exp2_pair(exponent(z));
        const float2 t = mul2(n, add2(n, two));
        return mul2(z, mul2(t, rcp2(add2(t, two))));
    } else return z;
}
// act'(z) of a pair: with w = 1 + e^z, r = 1 / (w^2 + 1), Mish' = 1 - 2 r + z 4 e^z w r^2.
// The factor z is the clamped one too (e^z w r^2, 4e-18 where the exponential
// stops, times a huge z would not be 0, from about 1e9 on): the exponent over
// log2 e.  0 z puts a NaN back.
template <int ACT>
__device__ __forceinline__ float2 dact2(float2 z) {
    if constexpr (ACT == ACT_RELU) return make_float2(z.x > 0.0f ? 1.0f : 0.0f, z.y > 0.0f ? 1.0f : 0.0f);
    else if constexpr (ACT == ACT_MISH) {
        const float2 one = make_float2(1.0f, 1.0f), e = exponent(z);
        const float2 n = exp2_pair(e);
        const float2 w = add2(n, one);
        const float2 r = rcp2(fma2(w, w, one));
        const float2 nr = mul2(mul2(n, r), mul2(w, r));
        return fma2(mul2(e, make_float2(2.772588722239781f, 2.772588722239781f)), nr,
                    fma2(r, make_float2(-2.0f, -2.0f), fma2(z, make_float2(0.0f, 0.0f), one)));
    } else return make_float2(1.0f, 1.0f);
}
__device__ __forceinline__ float2 neg2(float2 v) { return make_float2(-v.x, -v.y); }

// How a CTA's threads cover the channel vectors of its pixels: with cvn vectors
// a pixel, R = kThreads / cvn pixels side by side (R = 1 and several rounds
// where a pixel has more vectors than the CTA threads).
struct Cover {
    int cvn, R, r, col;
    bool on;
    __device__ __forceinline__ Cover(int C, int vec) {
        cvn = C / vec;
        if (cvn >= kThreads) {
            R = 1; r = 0; col = threadIdx.x;
            on = true;
        } else {
            R = kThreads / cvn; r = threadIdx.x / cvn; col = threadIdx.x - r * cvn;
            on = r < R;
        }
    }
    // pixels of a run of np that this thread takes
    __device__ __forceinline__ int count(int np) const { return np > r ? (np - r + R - 1) / R : 0; }
};

// A thread's way through its `cnt` vectors of MAPS maps, s[m] elements apart:
// batches of four vectors a map in a ring of shared memory slots of its own (so
// nothing waits for another thread), one batch of two maps or two of one always
// on the way (cp.async): 128 bytes a thread in flight beside its arithmetic,
// which registers could not hold (the sums of 8x80x80x256 took 21.8 us with
// loads into registers, four vectors at a time, and 17.5 us so, caches cold).  Pointers advance by addition: with an index multiplied out
// a vector, the address arithmetic was half of the instructions.  Two-byte
// vectors, which cp.async does not copy, go through registers.
constexpr int kBatch = 4;
__host__ __device__ constexpr int batches(int maps) { return maps == 2 ? 2 : 3; }
template <typename Raw>
__host__ __device__ constexpr int ring_bytes(int maps) { return sizeof(Raw) >= 4 ? kBatch * batches(maps) * kThreads * (int)sizeof(Raw) * maps : 0; }
// The first batches are asked for at construction, so that they are on their
// way while the thread sets up what it will do with them.
template <int MAPS, typename Raw, typename T>
struct Walk {
    const T *src[MAPS];
    long long step[MAPS];
    Raw *base;
    int cnt, left, to;  // vectors, those not yet asked for, the batch slot to fill
    __device__ __forceinline__ void ask() {
        constexpr int kSlot = kThreads * MAPS;
        Raw *d = base + to * (kBatch * kSlot);
#pragma unroll
        for (int u = 0; u < kBatch; ++u)
            if (u < left)
#pragma unroll
                for (int m = 0; m < MAPS; ++m) {
                    copy_vec(d + u * kSlot + m * kThreads, reinterpret_cast<const Raw *>(src[m]));
                    src[m] += step[m];
                }
        left -= kBatch;
        copy_commit();
        if (++to == batches(MAPS)) to = 0;
    }
    __device__ __forceinline__ Walk(uint8_t *ring, const T *const (&from)[MAPS], const long long (&by)[MAPS], int n)
        : base(reinterpret_cast<Raw *>(ring) + threadIdx.x), cnt(n), left(n), to(0) {
#pragma unroll
        for (int m = 0; m < MAPS; ++m) {
            src[m] = from[m];
            step[m] = by[m];
        }
        if constexpr (sizeof(Raw) >= 4)
#pragma unroll
            for (int i = 1; i < batches(MAPS); ++i) ask();
    }
    template <typename F>
    __device__ __forceinline__ void run(F &&use) {
        if constexpr (sizeof(Raw) >= 4) {
            constexpr int kBatches = batches(MAPS), kSlot = kThreads * MAPS;
            int at = 0;
            for (int n = cnt; n > 0; n -= kBatch) {
                copy_wait<kBatches - 2>();
                ask();
                const Raw *d = base + at * (kBatch * kSlot);
#pragma unroll
                for (int u = 0; u < kBatch; ++u)
                    if (u < n) {
                        Raw v[MAPS];
#pragma unroll
                        for (int m = 0; m < MAPS; ++m) v[m] = d[u * kSlot + m * kThreads];
                        use(v);
                    }
                if (++at == kBatches) at = 0;
            }
            copy_wait<0>();
        } else {
            for (; cnt > 0; cnt -= kBatch) {
                Raw v[kBatch][MAPS];
#pragma unroll
                for (int u = 0; u < kBatch; ++u)
                    if (u < cnt)
#pragma unroll
                        for (int m = 0; m < MAPS; ++m) {
                            v[u][m] = *reinterpret_cast<const Raw *>(src[m]);
                            src[m] += step[m];
                        }
#pragma unroll
                for (int u = 0; u < kBatch; ++u)
                    if (u < cnt) use(v[u]);
            }
        }
    }
};

// The threads' pairs of sums, ent[r * C + c], summed over the R rows: channel c
// into chan[c] (which may be ent itself only for R = 1).  L lanes a channel.
// Every thread of the CTA calls it after a barrier; ends without one.
template <typename F>
__device__ __forceinline__ void join_rows(const float2 *ent, int R, int C, F &&done) {
    int L = 1;
    while (L < 32 && L * 2 * C <= kThreads && L < R) L *= 2;
    const int per = kThreads / L, sub = threadIdx.x % L;
    for (int c0 = 0; c0 < C; c0 += per) {
        const int c = c0 + threadIdx.x / L;
        float2 v = make_float2(0.0f, 0.0f);
        if (c < C)
            for (int r = sub; r < R; r += L) v = add2(v, ent[r * C + c]);
        for (int o = L / 2; o > 0; o >>= 1) {
            v.x += __shfl_xor_sync(0xffffffffu, v.x, o);
            v.y += __shfl_xor_sync(0xffffffffu, v.y, o);
        }
        if (c < C && sub == 0) done(c, v);
    }
}

// (mean, M2) of a group from its channels' (mean, M2), each of `cnt` values;
// every lane of the calling warp returns it.
__device__ __forceinline__ float2 join_channels(const float2 *chan, int cg, float cnt, int lane) {
    float sum = 0.0f;
    for (int c = lane; c < cg; c += 32) sum += chan[c].x;
    const float mu = warp_sum(sum) / (float)cg;
    float m2 = 0.0f;
    for (int c = lane; c < cg; c += 32) {
        const float d = chan[c].x - mu;
        m2 += fmaf(cnt * d, d, chan[c].y);
    }
    return make_float2(mu, warp_sum(m2));
}

// A thread's sums of (x - K) and (x - K)^2 over its pixels of one run, K the
// run's first pixel.
template <typename T, int VEC>
struct StatSums {
    using V = Vec<T, VEC>;
    float2 K[V::kPairs], s1[V::kPairs], s2[V::kPairs];
    __device__ __forceinline__ void start(const typename V::Raw &first) {
        V::unpack(first, K);
#pragma unroll
        for (int e = 0; e < V::kPairs; ++e) {
            K[e] = neg2(K[e]);
            s1[e] = s2[e] = make_float2(0.0f, 0.0f);
        }
    }
    __device__ __forceinline__ void take(const typename V::Raw &raw) {
        float2 f[V::kPairs];
        V::unpack(raw, f);
#pragma unroll
        for (int e = 0; e < V::kPairs; ++e) {
            const float2 d = add2(f[e], K[e]);
            s1[e] = add2(s1[e], d);
            s2[e] = fma2(d, d, s2[e]);
        }
    }
    // ent: this thread's row of sums; piv: the channels' K
    __device__ __forceinline__ void put(float2 *ent, float *piv, bool first_row) const {
#pragma unroll
        for (int e = 0; e < VEC; ++e) {
            const float2 a = s1[e / 2], b = s2[e / 2];
            ent[e] = e % 2 ? make_float2(a.y, b.y) : make_float2(a.x, b.x);
            if (first_row) piv[e] = -(e % 2 ? K[e / 2].y : K[e / 2].x);
        }
    }
};
// A channel's (mean, M2) from its sums about K over cnt values.
__device__ __forceinline__ float2 about(float K, float2 s, float cnt) {
    const float d = s.x / cnt;
    return make_float2(K + d, fmaxf(s.y - s.x * d, 0.0f) + 0.0f * s.y);  // (NaN stays NaN)
}

// (mean, M2) of a group over `n` consecutive runs of `len` pixels of `total`
// (the last ones short or empty), run q's from get(q); n <= 8.
template <typename F>
__device__ __forceinline__ float2 join_few(int n, int len, int total, int cg, F &&get) {
    float2 v[8];
    float mu = 0.0f, m2 = 0.0f;
#pragma unroll
    for (int q = 0; q < 8; ++q)
        if (q < n) v[q] = get(q);
#pragma unroll
    for (int q = 0; q < 8; ++q)
        if (q < n) {
            const float c = (float)max(0, min(len, total - q * len));
            if (c > 0.0f) mu = fmaf(c, v[q].x, mu);
        }
    mu /= (float)min(n * len, total);
#pragma unroll
    for (int q = 0; q < 8; ++q)
        if (q < n) {
            const float c = (float)max(0, min(len, total - q * len)) * (float)cg, d = v[q].x - mu;
            if (c > 0.0f) m2 += fmaf(c * d, d, v[q].y);
        }
    return make_float2(mu, m2);
}

// (mean, M2) of each group over one run of pixels.
template <typename T, int VEC>
__global__ void __launch_bounds__(kThreads, 3) gn_stats_kernel(GnArgs a) {
    using V = Vec<T, VEC>;
    using Raw = typename V::Raw;
    extern __shared__ __align__(16) uint8_t ring[];  // the ring, then [C] channels, [R*C] sums, [C] K
    const Cover cv(a.C, VEC);
    float2 *chan = reinterpret_cast<float2 *>(ring + ring_bytes<Raw>(1)), *ent = chan + a.C;
    float *piv = reinterpret_cast<float *>(ent + cv.R * a.C);
    const int n = blockIdx.y, s = blockIdx.x;
    const int p0 = s * a.ppx, np = min(a.ppx, a.HW - p0);
    pdl_trigger();
    pdl_wait();
    const T *x = static_cast<const T *>(a.x) + ((long long)n * a.HW + p0) * a.px;
    if (cv.on) {
        for (int col = cv.col; col < cv.cvn; col += kThreads) {
            const T *xc = x + col * VEC;
            const T *const from[1] = {xc + cv.r * a.px};
            const long long step[1] = {cv.R * a.px};
            Walk<1, Raw, T> walk(ring, from, step, cv.count(np));
            StatSums<T, VEC> st;
            st.start(*reinterpret_cast<const Raw *>(xc));
            walk.run([&](const Raw (&v)[1]) { st.take(v[0]); });
            st.put(ent + cv.r * a.C + col * VEC, piv + col * VEC, cv.r == 0);
        }
    }
    __syncthreads();
    join_rows(ent, cv.R, a.C, [&](int c, float2 v) { chan[c] = about(piv[c], v, (float)np); });
    __syncthreads();
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    for (int g = warp; g < a.G; g += kWarps) {
        const float2 v = join_channels(chan + g * a.cg, a.cg, (float)np, lane);
        if (lane == 0) a.part[((long long)n * a.G + g) * a.S + s] = v;
    }
}

// The [G][S] partial results of image n, in shared memory if they fit: every
// load of the CTA is then in flight together, where group by group each would
// wait for L2.  Asked for here, a copy group of its own; there after
// staged_runs, which leaves the `later` groups committed since on their way.
__device__ __forceinline__ const float2 *stage_runs(const GnArgs &a, int n, float2 *dst) {
    const float2 *src = a.part + (long long)n * a.G * a.S;
    if ((long long)a.G * a.S > kStageRuns) return src;
    const int total = a.G * a.S;
    for (int i = threadIdx.x; i < total; i += kThreads) copy_async<8>(tc::smem_u32(dst + i), src + i);
    copy_commit();
    return dst;
}
template <int LATER>
__device__ __forceinline__ void staged_runs() {
    copy_wait<LATER>();
    __syncthreads();
}

// mean and rstd of a group of m values from the (mean, M2) of its S runs; every
// lane of the calling warp returns them.
__device__ __forceinline__ float2 join_runs(const GnArgs &a, const float2 *p, int lane) {
    const float inv = 1.0f / ((float)a.HW * (float)a.cg);
    float sum = 0.0f;
    for (int s = lane; s < a.S; s += 32) sum += (float)min(a.ppx, a.HW - s * a.ppx) * (float)a.cg * p[s].x;
    const float mu = warp_sum(sum) * inv;
    float m2 = 0.0f;
    for (int s = lane; s < a.S; s += 32) {
        const float2 v = p[s];
        const float d = v.x - mu;
        m2 += v.y + (float)min(a.ppx, a.HW - s * a.ppx) * (float)a.cg * d * d;
    }
    m2 = warp_sum(m2);
    return make_float2(mu, 1.0f / sqrtf(m2 * inv + a.eps));
}

// Stores one vector, as data that is not read again soon if `past`.
template <typename Raw>
__device__ __forceinline__ void put(Raw *p, const Raw &v, bool past) {
    if (past) __stcs(p, v);
    else *p = v;
}

// What a thread's channels need of the forward formula.
template <int VEC, int PAIRS>
__device__ __forceinline__ void set_lane(float2 (&v)[PAIRS], int e, float f) {
    if (e % 2) v[e / 2].y = f; else v[e / 2].x = f;
    if (VEC == 1) v[0].y = 0.0f;
}

// y = act(gamma (x - mean) rstd + beta) over one run of pixels, from its end to
// its start: of maps larger than L2 the statistics left the ends of the runs
// there.  Results of such maps are written past it (a.past_l2), so that they do
// not drive out what is still to be read.
template <typename T, int VEC, int ACT>
__global__ void __launch_bounds__(kThreads, 3) gn_apply_kernel(GnArgs a) {
    using V = Vec<T, VEC>;
    using Raw = typename V::Raw;
    constexpr int P = V::kPairs;
    extern __shared__ __align__(16) uint8_t ring[];  // the ring, then [G] (mean, rstd), [G][S]
    float2 *stat = reinterpret_cast<float2 *>(ring + ring_bytes<Raw>(1));
    const Cover cv(a.C, VEC);
    const int n = (int)(gridDim.y - 1 - blockIdx.y), s = (int)(gridDim.x - 1 - blockIdx.x);
    const int p0 = s * a.ppx, np = min(a.ppx, a.HW - p0);
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    pdl_trigger();
    pdl_wait();
    const T *x = static_cast<const T *>(a.x) + ((long long)n * a.HW + p0) * a.px;
    T *y = static_cast<T *>(a.out) + ((long long)n * a.HW + p0) * a.pout;
    const int cnt = cv.on ? cv.count(np) : 0, end = cv.r + (cnt - 1) * cv.R;  // this thread's last pixel
    const long long step[1] = {-cv.R * a.px};
    auto walk_at = [&](int col) {
        const T *const from[1] = {x + end * a.px + col * VEC};
        return Walk<1, Raw, T>(ring, from, step, cnt);
    };
    const float2 *runs = stage_runs(a, n, stat + a.G);
    Walk<1, Raw, T> walk = walk_at(cv.col);
    staged_runs<sizeof(Raw) >= 4 ? batches(1) - 1 : 0>();
    for (int g = warp; g < a.G; g += kWarps) {
        const float2 st = join_runs(a, runs + (long long)g * a.S, lane);
        if (lane == 0) {
            stat[g] = st;
            if (s == 0) {
                if (a.mean) a.mean[(long long)n * a.G + g] = st.x;
                if (a.rstd) a.rstd[(long long)n * a.G + g] = st.y;
            }
        }
    }
    __syncthreads();
    if (!cv.on) return;
    for (int col = cv.col; col < cv.cvn; col += kThreads) {
        if (col != cv.col) walk = walk_at(col);
        float2 mu[P], sc[P], be[P];  // mu: minus the mean
#pragma unroll
        for (int e = 0; e < VEC; ++e) {
            const int c = col * VEC + e;
            const float2 st = stat[c / a.cg];
            set_lane<VEC>(mu, e, -st.x);
            set_lane<VEC>(sc, e, st.y * (a.gamma ? a.gamma[c] : 1.0f));
            set_lane<VEC>(be, e, a.beta ? a.beta[c] : 0.0f);
        }
        T *o = y + end * a.pout + col * VEC;
        const long long so = cv.R * a.pout;
        walk.run([&](const Raw (&v)[1]) {
            float2 f[P];
            V::unpack(v[0], f);
#pragma unroll
            for (int e = 0; e < P; ++e) f[e] = act2<ACT>(fma2(add2(f[e], mu[e]), sc[e], be[e]));
            put(reinterpret_cast<Raw *>(o), V::pack(f), a.past_l2);
            o -= so;
        });
    }
}

// A thread's per-channel values of the gradient.  With xc = x - mean:
// z = xc sc + be, sc = rstd gamma; dz = dy act'(z); the sums are of dz and
// dz xc (rstd is multiplied in at the end); dx = dz sc - c1 - xc c2 with
// c1 = rstd m1, c2 = rstd^2 m2'.
template <typename T, int VEC, int ACT>
struct GradLane {
    using V = Vec<T, VEC>;
    using Raw = typename V::Raw;
    static constexpr int P = V::kPairs;
    float2 nmu[P], sc[P], be[P];  // nmu: minus the mean
    __device__ __forceinline__ void set(const GnArgs &a, int e, int c, float mean, float rstd) {
        set_lane<VEC>(nmu, e, -mean);
        set_lane<VEC>(sc, e, rstd * (a.gamma ? a.gamma[c] : 1.0f));
        set_lane<VEC>(be, e, a.beta ? a.beta[c] : 0.0f);
    }
    __device__ __forceinline__ void eval(const Raw &rx, const Raw &rd, float2 (&xc)[P], float2 (&dz)[P]) const {
        V::unpack(rx, xc);
        V::unpack(rd, dz);
#pragma unroll
        for (int e = 0; e < P; ++e) {
            xc[e] = add2(xc[e], nmu[e]);
            if (ACT != ACT_NONE) dz[e] = mul2(dz[e], dact2<ACT>(fma2(xc[e], sc[e], be[e])));
        }
    }
    // A += dz, B += dz xc
    __device__ __forceinline__ void sums(const Raw &rx, const Raw &rd, float2 (&A)[P], float2 (&B)[P]) const {
        float2 xc[P], dz[P];
        eval(rx, rd, xc, dz);
#pragma unroll
        for (int e = 0; e < P; ++e) {
            A[e] = add2(A[e], dz[e]);
            B[e] = fma2(dz[e], xc[e], B[e]);
        }
    }
    // dx, nc1 and nc2 the negated c1 and c2
    __device__ __forceinline__ Raw dx(const Raw &rx, const Raw &rd, const float2 (&nc1)[P], const float2 (&nc2)[P]) const {
        float2 xc[P], dz[P];
        eval(rx, rd, xc, dz);
#pragma unroll
        for (int e = 0; e < P; ++e) xc[e] = fma2(xc[e], nc2[e], fma2(dz[e], sc[e], nc1[e]));
        return V::pack(xc);
    }
};
// A group's sums of gamma times its channels'; every lane of the calling warp
// returns it.  c0: the group's first channel.
__device__ __forceinline__ float2 join_gamma(const GnArgs &a, const float2 *chan, int c0, int lane) {
    float2 v = make_float2(0.0f, 0.0f);
    for (int c = lane; c < a.cg; c += 32) {
        const float w = a.gamma ? a.gamma[c0 + c] : 1.0f;
        const float2 u = chan[c];
        v.x = fmaf(w, u.x, v.x);
        v.y = fmaf(w, u.y, v.y);
    }
    return make_float2(warp_sum(v.x), warp_sum(v.y));
}
template <int VEC, int P>
__device__ __forceinline__ void put_sums(float2 *ent, const float2 (&A)[P], const float2 (&B)[P]) {
#pragma unroll
    for (int e = 0; e < VEC; ++e) ent[e] = e % 2 ? make_float2(A[e / 2].y, B[e / 2].y) : make_float2(A[e / 2].x, B[e / 2].x);
}

// Sums of dz and dz xhat per channel, and of gamma times them per group, over
// one run of pixels.
template <typename T, int VEC, int ACT>
__global__ void __launch_bounds__(kThreads, grad_ctas(sizeof(T))) gn_bwd_sums_kernel(GnArgs a) {
    using L = GradLane<T, VEC, ACT>;
    using Raw = typename L::Raw;
    constexpr int P = L::P;
    extern __shared__ __align__(16) uint8_t ring[];  // the ring, then [C] channels, [R*C] sums
    const Cover cv(a.C, VEC);
    float2 *chan = reinterpret_cast<float2 *>(ring + ring_bytes<Raw>(2)), *ent = chan + a.C;
    const int n = blockIdx.y, s = blockIdx.x;
    const int p0 = s * a.ppx, np = min(a.ppx, a.HW - p0);
    pdl_trigger();
    pdl_wait();
    const T *x = static_cast<const T *>(a.x) + ((long long)n * a.HW + p0) * a.px;
    const T *dy = static_cast<const T *>(a.dy) + ((long long)n * a.HW + p0) * a.pdy;
    if (cv.on) {
        for (int col = cv.col; col < cv.cvn; col += kThreads) {
            const T *const from[2] = {x + cv.r * a.px + col * VEC, dy + cv.r * a.pdy + col * VEC};
            const long long step[2] = {cv.R * a.px, cv.R * a.pdy};
            Walk<2, Raw, T> walk(ring, from, step, cv.count(np));
            L ln;
            float2 A[P], B[P];
#pragma unroll
            for (int e = 0; e < VEC; ++e) {
                const int c = col * VEC + e;
                const long long g = (long long)n * a.G + c / a.cg;
                ln.set(a, e, c, a.mean[g], a.rstd[g]);
            }
#pragma unroll
            for (int e = 0; e < P; ++e) A[e] = B[e] = make_float2(0.0f, 0.0f);
            walk.run([&](const Raw (&v)[2]) { ln.sums(v[0], v[1], A, B); });
            put_sums<VEC>(ent + cv.r * a.C + col * VEC, A, B);
        }
    }
    __syncthreads();
    float2 *pc = a.partc + ((long long)n * a.S + s) * a.C;
    join_rows(ent, cv.R, a.C, [&](int c, float2 v) {
        v.y *= a.rstd[(long long)n * a.G + c / a.cg];
        pc[c] = chan[c] = v;
    });
    __syncthreads();
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    for (int g = warp; g < a.G; g += kWarps) {
        const float2 v = join_gamma(a, chan + g * a.cg, g * a.cg, lane);
        if (lane == 0) a.part[((long long)n * a.G + g) * a.S + s] = v;
    }
}

// dgamma and dbeta from `rows` rows of channel sums, 32 channels a CTA.
__device__ __forceinline__ void join_rows_of_channels(const GnArgs &a, long long rows, int block, int blocks, float2 *red) {
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    for (int c0 = block * 32; c0 < a.C; c0 += blocks * 32) {
        const int c = c0 + lane;
        float2 v = make_float2(0.0f, 0.0f);
        if (c < a.C) {
            // (sixteen rows on their way together: this is the launch's tail)
            for (long long r = warp; r < rows; r += 16 * kWarps) {
                float2 t[16];
#pragma unroll
                for (int u = 0; u < 16; ++u)
                    t[u] = r + u * kWarps < rows ? a.partc[(r + u * kWarps) * a.C + c] : make_float2(0.0f, 0.0f);
#pragma unroll
                for (int o = 8; o > 0; o >>= 1)
#pragma unroll
                    for (int u = 0; u < o; ++u) t[u] = add2(t[u], t[u + o]);
                v = add2(v, t[0]);
            }
        }
        red[warp * 32 + lane] = v;
        __syncthreads();
        if (warp == 0 && c < a.C) {
            for (int q = 1; q < kWarps; ++q) v = add2(v, red[q * 32 + lane]);
            if (a.dbeta) a.dbeta[c] = v.x;
            if (a.dgamma) a.dgamma[c] = v.y;
        }
        __syncthreads();
    }
}
// dx over one run of pixels, backwards like y; with `head`, the last grid row
// joins the channels' sums of every image and run into dgamma and dbeta, 32
// channels a CTA (last, so that no run waits for a place on the card).  The row
// is as wide as an image has runs: with one run an image, as in batches of more
// images than the card holds CTAs, one CTA joins all channels (1024x7x7x1024
// bf16 with Mish 711 us, forward and gradient, where its bytes take 61).
template <typename T, int VEC, int ACT>
__global__ void __launch_bounds__(kThreads, grad_ctas(sizeof(T))) gn_bwd_dx_kernel(GnArgs a, int head) {
    using L = GradLane<T, VEC, ACT>;
    using Raw = typename L::Raw;
    constexpr int P = L::P;
    extern __shared__ __align__(16) uint8_t ring[];  // the ring, then [G] minus c1 and c2, [G][S]; or [kWarps][32] sums
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    pdl_trigger();
    pdl_wait();
    if (head && blockIdx.y == gridDim.y - 1) {
        join_rows_of_channels(a, (long long)a.N * a.S, blockIdx.x, gridDim.x, reinterpret_cast<float2 *>(ring));
        return;
    }
    float2 *sum = reinterpret_cast<float2 *>(ring + ring_bytes<Raw>(2));
    const Cover cv(a.C, VEC);
    const int n = a.N - 1 - (int)blockIdx.y, s = (int)(gridDim.x - 1 - blockIdx.x);
    const int p0 = s * a.ppx, np = min(a.ppx, a.HW - p0);
    const T *x = static_cast<const T *>(a.x) + ((long long)n * a.HW + p0) * a.px;
    const T *dy = static_cast<const T *>(a.dy) + ((long long)n * a.HW + p0) * a.pdy;
    T *dx = static_cast<T *>(a.out) + ((long long)n * a.HW + p0) * a.pout;
    const int cnt = cv.on ? cv.count(np) : 0, end = cv.r + (cnt - 1) * cv.R;
    const long long step[2] = {-cv.R * a.px, -cv.R * a.pdy};
    auto walk_at = [&](int col) {
        const T *const from[2] = {x + end * a.px + col * VEC, dy + end * a.pdy + col * VEC};
        return Walk<2, Raw, T>(ring, from, step, cnt);
    };
    const float2 *runs = stage_runs(a, n, sum + a.G);
    Walk<2, Raw, T> walk = walk_at(cv.col);
    L ln;
    auto set = [&](int col) {
#pragma unroll
        for (int e = 0; e < VEC; ++e) {
            const int c = col * VEC + e;
            const long long g = (long long)n * a.G + c / a.cg;
            ln.set(a, e, c, a.mean[g], a.rstd[g]);
        }
    };
    if (cv.on) set(cv.col);
    const float inv = -1.0f / ((float)a.HW * (float)a.cg);
    staged_runs<sizeof(Raw) >= 4 ? batches(2) - 1 : 0>();
    for (int g = warp; g < a.G; g += kWarps) {
        const float2 *p = runs + (long long)g * a.S;
        const float rs = a.rstd[(long long)n * a.G + g];
        float2 v = make_float2(0.0f, 0.0f);
        for (int q = lane; q < a.S; q += 32) v = add2(v, p[q]);
        v.x = warp_sum(v.x);
        v.y = warp_sum(v.y);
        if (lane == 0) sum[g] = make_float2(v.x * inv * rs, v.y * inv * rs * rs);
    }
    __syncthreads();
    if (!cv.on) return;
    for (int col = cv.col; col < cv.cvn; col += kThreads) {
        if (col != cv.col) {
            walk = walk_at(col);
            set(col);
        }
        float2 c1[P], c2[P];
#pragma unroll
        for (int e = 0; e < VEC; ++e) {
            const float2 v = sum[(col * VEC + e) / a.cg];
            set_lane<VEC>(c1, e, v.x);
            set_lane<VEC>(c2, e, v.y);
        }
        T *o = dx + end * a.pout + col * VEC;
        const long long so = cv.R * a.pout;
        walk.run([&](const Raw (&v)[2]) {
            put(reinterpret_cast<Raw *>(o), ln.dx(v[0], v[1], c1, c2), a.past_l2);
            o -= so;
        });
    }
}

// ------------------------------------------------------------- cluster kernels
// One launch where a few groups of an image fit a cluster: its K
// CTAs take gb groups of an image (gradient: of every image), each CTA a run of
// pixels.  Each sums its run, exchanges the groups' sums with the cluster's
// other CTAs (8 bytes a group, through distributed shared memory) and finishes
// its run, which waits in shared memory meanwhile (cp.async, the whole run in
// flight at once; a thread reads back only what it copied itself): every byte
// crosses HBM and L2 once.

// Rows that a CTA's sums leave in shared memory: one a warp where a warp's
// lanes cover whole pixels (folded with shuffles first), else one a thread row.
__host__ __device__ inline bool folds(int cvn) { return cvn <= 32 && (cvn & (cvn - 1)) == 0; }
template <int P>
__device__ __forceinline__ void fold(float2 (&v)[P], int cvn) {
    for (int o = cvn; o < 32; o <<= 1)
#pragma unroll
        for (int e = 0; e < P; ++e) {
            v[e].x += __shfl_xor_sync(0xffffffffu, v[e].x, o);
            v[e].y += __shfl_xor_sync(0xffffffffu, v[e].y, o);
        }
}

template <typename T, int VEC, int ACT>
__global__ void __launch_bounds__(kThreads, 4) gn_cluster_kernel(GnArgs a) {
    using V = Vec<T, VEC>;
    using Raw = typename V::Raw;
    constexpr int P = V::kPairs;
    extern __shared__ __align__(16) uint8_t shm[];
    const int g0 = blockIdx.y * a.gb, gb = min(a.gb, a.G - g0), cb = gb * a.cg, c0 = g0 * a.cg;
    const int n = blockIdx.z, k = blockIdx.x;
    const int p0 = k * a.ppx, np = min(a.ppx, a.HW - p0);
    const Cover cv(cb, VEC);
    const bool fl = folds(cv.cvn);
    const int rows = fl ? kWarps : cv.R;
    float2 *gpart = reinterpret_cast<float2 *>(shm);          // [gb] this CTA's (mean, M2)
    float2 *stat = gpart + a.gb;                              // [gb] (mean, rstd)
    float2 *chan = stat + a.gb;                               // [cb]
    float2 *ent = chan + a.cb;                                // [rows][cb], at most a.ent
    float *piv = reinterpret_cast<float *>(ent + a.ent);      // [cb]
    Raw *data = reinterpret_cast<Raw *>((reinterpret_cast<uintptr_t>(piv + a.cb) + 15) & ~(uintptr_t)15);
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    pdl_trigger();
    pdl_wait();
    const T *x = static_cast<const T *>(a.x) + ((long long)n * a.HW + p0) * a.px + c0 + cv.col * VEC;
    // this thread's vectors lie kThreads (of which R cvn are at work) apart
    Raw *mine = data + threadIdx.x;
    const int cnt = cv.on ? cv.count(np) : 0, step = cv.R * cv.cvn;
    StatSums<T, VEC> st;
    // the run in four parts, each summed as it lands
    const int part = (cnt + 3) / 4;
    const T *from = x + cv.r * a.px;
    const long long sx = cv.R * a.px;
    Raw *to = mine;
    auto load = [&](int q) {
#pragma unroll 4
        for (int i = min(part, cnt - q * part); i > 0; --i, from += sx, to += step) copy_vec(to, reinterpret_cast<const Raw *>(from));
        copy_commit();
    };
    const Raw *at = mine;
    auto take = [&](int q) {
#pragma unroll 4
        for (int i = min(part, cnt - q * part); i > 0; --i, at += step) st.take(*at);
    };
    load(0); load(1); load(2); load(3);
    Raw first = {};
    if (cv.on) first = *reinterpret_cast<const Raw *>(x);
    st.start(first);
    copy_wait<3>(); take(0);
    copy_wait<2>(); take(1);
    copy_wait<1>(); take(2);
    copy_wait<0>(); take(3);
    if (fl) {
        fold(st.s1, cv.cvn);
        fold(st.s2, cv.cvn);
        if (lane < cv.cvn) st.put(ent + warp * cb + cv.col * VEC, piv + cv.col * VEC, warp == 0);
    } else if (cv.on) {
        st.put(ent + cv.r * cb + cv.col * VEC, piv + cv.col * VEC, cv.r == 0);
    }
    __syncthreads();
    join_rows(ent, rows, cb, [&](int c, float2 v) { chan[c] = about(piv[c], v, (float)np); });
    __syncthreads();
    for (int g = warp; g < gb; g += kWarps) {
        const float2 v = join_channels(chan + g * a.cg, a.cg, (float)np, lane);
        if (lane == 0) gpart[g] = v;
    }
    float2 ga[P], be[P];
    if (cv.on)
#pragma unroll
        for (int e = 0; e < VEC; ++e) {
            const int c = c0 + cv.col * VEC + e;
            set_lane<VEC>(ga, e, a.gamma ? a.gamma[c] : 1.0f);
            set_lane<VEC>(be, e, a.beta ? a.beta[c] : 0.0f);
        }
    if (a.K > 1) {
        cluster_arrive();
        cluster_wait();
    } else {
        __syncthreads();
    }
    for (int g = threadIdx.x; g < gb; g += kThreads) {
        const float2 v = a.K > 1 ? join_few(a.K, a.ppx, a.HW, a.cg, [&](int q) { return ld_peer(gpart + g, q); }) : gpart[g];
        const float rstd = 1.0f / sqrtf(v.y / ((float)a.HW * (float)a.cg) + a.eps);
        stat[g] = make_float2(v.x, rstd);
        if (k == 0) {
            if (a.mean) a.mean[(long long)n * a.G + g0 + g] = v.x;
            if (a.rstd) a.rstd[(long long)n * a.G + g0 + g] = rstd;
        }
    }
    __syncthreads();
    if (a.K > 1) cluster_arrive();  // this CTA has read its peers' sums
    if (cv.on) {
        float2 mu[P];
#pragma unroll
        for (int e = 0; e < VEC; ++e) {
            const float2 s = stat[(cv.col * VEC + e) / a.cg];
            set_lane<VEC>(mu, e, -s.x);
            set_lane<VEC>(ga, e, (e % 2 ? ga[e / 2].y : ga[e / 2].x) * s.y);
        }
        T *y = static_cast<T *>(a.out) + ((long long)n * a.HW + p0 + cv.r) * a.pout + c0 + cv.col * VEC;
        const long long so = cv.R * a.pout;
        auto one = [&](const Raw &v) {
            float2 f[P];
            V::unpack(v, f);
#pragma unroll
            for (int e = 0; e < P; ++e) f[e] = act2<ACT>(fma2(add2(f[e], mu[e]), ga[e], be[e]));
            *reinterpret_cast<Raw *>(y) = V::pack(f);
            y += so;
        };
        const Raw *v = mine;
#pragma unroll 4
        for (int i = cnt; i > 0; --i, v += step) one(*v);
    }
    if (a.K > 1) cluster_wait();  // no CTA leaves while its sums may be read
}

// The gradient: a cluster holds K CTAs of every image, so that dgamma and dbeta
// are complete in it.
template <typename T, int VEC, int ACT>
__global__ void __launch_bounds__(kThreads, 3) gn_bwd_cluster_kernel(GnArgs a) {
    using L = GradLane<T, VEC, ACT>;
    using V = Vec<T, VEC>;
    using Raw = typename V::Raw;
    constexpr int P = V::kPairs;
    extern __shared__ __align__(16) uint8_t shm[];
    const int g0 = blockIdx.y * a.gb, gb = min(a.gb, a.G - g0), cb = gb * a.cg, c0 = g0 * a.cg;
    const int n = blockIdx.x / a.K, k = blockIdx.x - n * a.K;  // blockIdx.x: the rank in the cluster
    const int p0 = k * a.ppx, np = min(a.ppx, a.HW - p0);
    const Cover cv(cb, VEC);
    const bool fl = folds(cv.cvn);
    const int rows = fl ? kWarps : cv.R;
    const int size = a.K * a.N;
    float2 *gpart = reinterpret_cast<float2 *>(shm);  // [gb] this CTA's sums of gamma dz, gamma dz xhat
    float2 *sum = gpart + a.gb;                       // [gb] minus c1 and c2 of the image
    float2 *chan = sum + a.gb;                        // [cb] this CTA's sums of dz, dz xhat
    float2 *ent = chan + a.cb;                        // [rows][cb], at most a.ent
    Raw *data = reinterpret_cast<Raw *>((reinterpret_cast<uintptr_t>(ent + a.ent) + 15) & ~(uintptr_t)15);
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    pdl_trigger();
    pdl_wait();
    const T *x = static_cast<const T *>(a.x) + ((long long)n * a.HW + p0) * a.px + c0 + cv.col * VEC;
    const T *dy = static_cast<const T *>(a.dy) + ((long long)n * a.HW + p0) * a.pdy + c0 + cv.col * VEC;
    Raw *mx = data + threadIdx.x, *md = mx + a.ppx * cv.cvn;
    const int cnt = cv.on ? cv.count(np) : 0, step = cv.R * cv.cvn;
    L ln;
    float2 A[P], B[P];
#pragma unroll
    for (int e = 0; e < P; ++e) A[e] = B[e] = make_float2(0.0f, 0.0f);
    const int part = (cnt + 3) / 4;
    const T *fx = x + cv.r * a.px, *fd = dy + cv.r * a.pdy;
    const long long sx = cv.R * a.px, sd = cv.R * a.pdy;
    Raw *to = mx, *td = md;
    auto load = [&](int q) {
#pragma unroll 2
        for (int i = min(part, cnt - q * part); i > 0; --i, fx += sx, fd += sd, to += step, td += step) {
            copy_vec(to, reinterpret_cast<const Raw *>(fx));
            copy_vec(td, reinterpret_cast<const Raw *>(fd));
        }
        copy_commit();
    };
    const Raw *at = mx, *ad = md;
    auto take = [&](int q) {
#pragma unroll 2
        for (int i = min(part, cnt - q * part); i > 0; --i, at += step, ad += step) ln.sums(*at, *ad, A, B);
    };
    load(0); load(1); load(2); load(3);
    if (cv.on)
#pragma unroll
        for (int e = 0; e < VEC; ++e) {
            const int c = c0 + cv.col * VEC + e;
            const long long g = (long long)n * a.G + c / a.cg;
            ln.set(a, e, c, a.mean[g], a.rstd[g]);
        }
    copy_wait<3>(); take(0);
    copy_wait<2>(); take(1);
    copy_wait<1>(); take(2);
    copy_wait<0>(); take(3);
    if (fl) {
        fold(A, cv.cvn);
        fold(B, cv.cvn);
        if (lane < cv.cvn) put_sums<VEC>(ent + warp * cb + cv.col * VEC, A, B);
    } else if (cv.on) {
        put_sums<VEC>(ent + cv.r * cb + cv.col * VEC, A, B);
    }
    __syncthreads();
    join_rows(ent, rows, cb, [&](int c, float2 v) {
        chan[c] = make_float2(v.x, v.y * a.rstd[(long long)n * a.G + g0 + c / a.cg]);
    });
    __syncthreads();
    for (int g = warp; g < gb; g += kWarps) {
        const float2 v = join_gamma(a, chan + g * a.cg, c0 + g * a.cg, lane);
        if (lane == 0) gpart[g] = v;
    }
    if (size > 1) {
        cluster_arrive();
        cluster_wait();
    } else {
        __syncthreads();
    }
    const float inv = -1.0f / ((float)a.HW * (float)a.cg);
    for (int g = threadIdx.x; g < gb; g += kThreads) {
        float2 v = make_float2(0.0f, 0.0f);
        for (int q = 0; q < a.K; ++q) v = add2(v, size > 1 ? ld_peer(gpart + g, n * a.K + q) : gpart[g]);
        const float rs = a.rstd[(long long)n * a.G + g0 + g];
        sum[g] = make_float2(v.x * inv * rs, v.y * inv * rs * rs);
    }
    if ((a.dgamma || a.dbeta) && blockIdx.x == 0)
        for (int c = threadIdx.x; c < cb; c += kThreads) {
            float2 v = make_float2(0.0f, 0.0f);
            for (int q = 0; q < size; ++q) v = add2(v, size > 1 ? ld_peer(chan + c, q) : chan[c]);
            if (a.dbeta) a.dbeta[c0 + c] = v.x;
            if (a.dgamma) a.dgamma[c0 + c] = v.y;
        }
    __syncthreads();
    if (size > 1) cluster_arrive();
    if (cv.on) {
        float2 m1[P], m2[P];
#pragma unroll
        for (int e = 0; e < VEC; ++e) {
            const float2 s = sum[(cv.col * VEC + e) / a.cg];
            set_lane<VEC>(m1, e, s.x);
            set_lane<VEC>(m2, e, s.y);
        }
        T *dx = static_cast<T *>(a.out) + ((long long)n * a.HW + p0 + cv.r) * a.pout + c0 + cv.col * VEC;
        const long long so = cv.R * a.pout;
        auto one = [&](const Raw &v, const Raw &w) {
            *reinterpret_cast<Raw *>(dx) = ln.dx(v, w, m1, m2);
            dx += so;
        };
        const Raw *v = mx, *w = md;
#pragma unroll 2
        for (int i = cnt; i > 0; --i, v += step, w += step) one(*v, *w);
    }
    if (size > 1) cluster_wait();
}

// ------------------------------------------------------------------ host side
enum { K_STATS, K_APPLY, K_SUMS, K_DX, K_CLUSTER, K_CLUSTER_BWD };

template <typename T, int VEC, int ACT>
const void *pick_act(int which) {
    switch (which) {
    case K_STATS: return (const void *)&gn_stats_kernel<T, VEC>;
    case K_APPLY: return (const void *)&gn_apply_kernel<T, VEC, ACT>;
    case K_SUMS: return (const void *)&gn_bwd_sums_kernel<T, VEC, ACT>;
    case K_DX: return (const void *)&gn_bwd_dx_kernel<T, VEC, ACT>;
    case K_CLUSTER: return (const void *)&gn_cluster_kernel<T, VEC, ACT>;
    default: return (const void *)&gn_bwd_cluster_kernel<T, VEC, ACT>;
    }
}
template <typename T, int VEC>
const void *pick(int which, int act) {
    return act == ACT_MISH ? pick_act<T, VEC, ACT_MISH>(which)
                           : (act == ACT_RELU ? pick_act<T, VEC, ACT_RELU>(which) : pick_act<T, VEC, ACT_NONE>(which));
}

const void *pick_kernel(int which, conv_dtype_t dt, int vec, int act) {
    if (dt == CONV_F32) return vec == 4 ? pick<float, 4>(which, act) : pick<float, 1>(which, act);
    return vec == 8 ? pick<__nv_bfloat16, 8>(which, act)
                    : (vec == 2 ? pick<__nv_bfloat16, 2>(which, act) : pick<__nv_bfloat16, 1>(which, act));
}

// Channels a vector access takes: the widest that the channel count, every
// tensor's pitch and every tensor's address allow.
int vec_for(const conv_plan *p, int count, const void *const *ptr, const long long *pitch) {
    const int es = conv_esize(p->dtype);
    const int widths[2] = {16 / es, p->dtype == CONV_F32 ? 1 : 2};
    for (int v : widths) {
        bool ok = p->s.c_in % v == 0;
        for (int i = 0; i < count; ++i) ok = ok && pitch[i] % v == 0 && ((uintptr_t)ptr[i] % (uintptr_t)(v * es)) == 0;
        if (ok) return v;
    }
    return 1;
}

// Rows of pixels a CTA takes side by side (Cover::R) for a vector width.
int rows_for(int C, int vec) { return C / vec >= kThreads ? 1 : kThreads / (C / vec); }

// The buffers of a run besides its maps, and its maps: whether one that it
// writes shares a byte with any other (CTAs read the inputs while others write).
struct Small { const void *p; size_t bytes; };
struct Map { const void *p; long long pitch; };
template <int I, int O, int M>
bool results_overlap(const Small (&in)[I], const Small (&out)[O], const Map (&maps_in)[M], const Map &result, long long rows, int C,
                     int es) {
    for (const Small &i : in)
        if (range_overlaps(i.p, i.bytes, result.p, result.pitch, rows, C, es)) return true;
    for (int k = 0; k < O; ++k) {
        if (range_overlaps(out[k].p, out[k].bytes, result.p, result.pitch, rows, C, es)) return true;
        for (const Map &m : maps_in)
            if (range_overlaps(out[k].p, out[k].bytes, m.p, m.pitch, rows, C, es)) return true;
        for (const Small &i : in)
            if (conv_overlaps(out[k].p, out[k].bytes, i.p, i.bytes)) return true;
        for (int j = 0; j < k; ++j)
            if (conv_overlaps(out[k].p, out[k].bytes, out[j].p, out[j].bytes)) return true;
    }
    return false;
}

int check_map(const conv_plan *p, const void *t, int64_t *pitch) {
    if (!t) return CONV_ERR_NULL_ARG;
    if (*pitch == 0) *pitch = p->s.c_in;
    if (*pitch < p->s.c_in) return CONV_ERR_INVALID_ARG;
    if (*pitch >= (1ll << 31) || (long long)p->s.n * p->s.h * p->s.w * *pitch >= (1ll << 40)) return CONV_ERR_UNSUPPORTED;
    if ((uintptr_t)t % (uintptr_t)conv_esize(p->dtype)) return CONV_ERR_MISALIGNED;
    return CONV_OK;
}
bool bad_f32(const void *t) { return t && ((uintptr_t)t & 3u); }

GnArgs base_args(const conv_plan *p, const GnGeom::Dir &d, const void *x, long long px, void *out, long long pout, void *ws) {
    GnArgs a = {};
    a.x = x; a.px = px; a.out = out; a.pout = pout;
    a.N = p->s.n; a.HW = p->s.h * p->s.w; a.C = p->s.c_in; a.G = p->groups; a.cg = p->s.c_in / p->groups;
    a.S = d.S; a.ppx = d.ppx; a.past_l2 = d.past_l2; a.eps = p->gn.eps;
    a.part = static_cast<float2 *>(ws);
    a.partc = a.part + (long long)a.N * a.S * a.G;
    return a;
}

// The cluster form of a run, and its shared memory.  The last CTA of a map may
// have fewer channels than the others and then more thread rows: the sums'
// entries are the larger of the two counts.
size_t cluster_args(const GnGeom::Dir &d, int vec, int es, int maps, GnArgs &a) {
    a.gb = d.gb; a.cb = d.cb; a.K = d.K; a.ppx = d.cpx;
    auto entries = [&](int cb) { return (folds(cb / vec) ? kWarps : rows_for(cb, vec)) * cb; };
    const int last = (a.G - (a.G - 1) / a.gb * a.gb) * a.cg;
    a.ent = entries(a.cb) > entries(last) ? entries(a.cb) : entries(last);
    return (size_t)2 * a.gb * 8 + (size_t)a.cb * 8 + (size_t)a.ent * 8 + (size_t)a.cb * 4 + 16 +
           (size_t)a.ppx * a.cb * es * maps;
}
bool clustered(const GnGeom::Dir &d, int vec) { return d.K > 0 && d.cb / vec <= kThreads; }

// How one direction runs.  `maps`: input maps it reads (1, or x and dy).
void plan_direction(const conv_plan *p, int maps, GnGeom::Dir &d, size_t &ws) {
    const int es = conv_esize(p->dtype), C = p->s.c_in, G = p->groups, cg = C / G, HW = p->s.h * p->s.w, N = p->s.n;
    const int wide = 16 / es, au = C % wide == 0 ? wide : (C % 2 == 0 && es == 2 ? 2 : 1);  // the widest vector there can be
    // Two launches: runs of pixels, one wave of CTAs, at least four pixels a
    // thread.
    const int R = rows_for(C, au);
    const int ctas = maps > 1 ? grad_ctas(es) : kCtas;
    long long runs = N > 0 ? ((long long)ctas * p->num_sms) / N : 1;
    const long long most = ((long long)HW + 4LL * R - 1) / (4LL * R);
    if (runs > most) runs = most;
    if (runs < 1) runs = 1;
    d.ppx = (int)((HW + runs - 1) / runs);
    d.S = (HW + d.ppx - 1) / d.ppx;
    d.past_l2 = (long long)N * HW * C * es * maps > kL2Bytes;
    ws = (size_t)N * d.S * ((size_t)G + (maps > 1 ? C : 0)) * sizeof(float2);
    // Clusters: the fewest groups of a CTA that fill whole vectors and 64
    // bytes of a pixel (a DRAM burst); the fewest CTAs an image that hold their
    // runs in shared memory, more while SMs are idle and runs stay above 8 KB.
    // The gradient takes this form where one cluster holds every image.
    d.K = 0;
    int gb = 1;
    while (gb < G && ((gb * cg) % au != 0 || gb * cg * es < 64)) ++gb;
    const int cb = gb * cg;
    const bool always = cb <= kThreads;                   // whatever vector a call's addresses allow
    if (!always && cb / au > kThreads) return;
    auto bytes = [&](int k) { return (long long)((HW + k - 1) / k) * cb * es * maps; };
    const int most_k = maps > 1 ? (N > 0 ? 8 / N : 1) : 8;
    if (most_k < 1) return;
    int K = 1;
    while (K < most_k && bytes(K) > kResident) ++K;
    if (bytes(K) > kResidentMost) return;
    const long long blocks = (G + gb - 1) / gb;
    while (K < most_k && blocks * N * K < p->num_sms && bytes(K) > 8 * 1024) ++K;
    d.cpx = (HW + K - 1) / K;
    d.K = (HW + d.cpx - 1) / d.cpx;
    d.gb = gb; d.cb = cb;
    if (blocks > 65535) { d.K = 0; return; }
    if (always) ws = 0;  // (else a call's addresses decide between the forms)
}

// (ring_bytes, for a vector of so many bytes)
size_t ring_size(int bytes, int maps) { return bytes >= 4 ? (size_t)kBatch * batches(maps) * kThreads * bytes * maps : 0; }
// (groups' statistics, and the runs' results where a CTA stages them)
size_t runs_smem(const GnArgs &a) {
    return ((size_t)a.G + ((long long)a.G * a.S <= kStageRuns ? (size_t)a.G * a.S : 0)) * 8;
}

cudaError_t launch(const conv_plan *p, int which, int vec, GnArgs &a, dim3 grid, size_t smem, cudaStream_t st, int cluster = 1,
                   int head = 0) {
    const void *k = pick_kernel(which, p->dtype, vec, p->act);
    if (smem > 48 * 1024) {
        const int rc = conv_grant_smem_once(k, p->device, (int)smem);
        if (rc != CONV_OK) return cudaErrorInvalidValue;
    }
    void *args[] = {&a, &head};  // (only gn_bwd_dx_kernel takes the second)
    return conv_launch(k, grid, dim3(kThreads), args, smem, st, cluster);
}

}  // namespace

extern "C" int conv_plan_create_groupnorm(int32_t n, int32_t h, int32_t w, int32_t c, int32_t groups, float eps,
                                          conv_dtype_t dtype, conv_act_t act, conv_plan_t **out_plan) {
    if (!out_plan) return CONV_ERR_NULL_ARG;
    *out_plan = nullptr;
    if (n < 0 || h < 1 || w < 1 || c < 1 || groups < 1 || c % groups != 0) return CONV_ERR_INVALID_SHAPE;
    if ((int)dtype < CONV_F32 || (int)dtype > CONV_I8) return CONV_ERR_INVALID_ARG;
    if ((int)act < CONV_ACT_NONE || (int)act > CONV_ACT_MISH) return CONV_ERR_INVALID_ARG;
    if (!(eps >= 0.0f) || !isfinite(eps)) return CONV_ERR_INVALID_ARG;
    if (dtype == CONV_I8) return CONV_ERR_UNSUPPORTED;
    // 32-bit pixel indices inside an image, 65535 images a grid, and the
    // channels' sums in shared memory
    if ((long long)h * w >= (1ll << 30) || n > 65534 || c > kMaxC || (long long)n * h * w * c >= (1ll << 40))
        return CONV_ERR_UNSUPPORTED;
    conv_plan *p = new (std::nothrow) conv_plan();
    if (!p) return CONV_ERR_OOM;
    p->s = {n, h, w, c, c, 1, 1};
    p->stride = 1; p->groups = groups; p->dtype = dtype; p->act = act; p->oh = h; p->ow = w;
    p->y_c = c; p->up = 1; p->algo = CONV_ALGO_GROUPNORM;
    p->gn.eps = eps;
    const int rc = conv_plan_bind_device(p, false);
    if (rc != CONV_OK) {
        conv_plan_destroy(p);
        return rc;
    }
    plan_direction(p, 1, p->gn.fwd, p->ws_bytes);
    plan_direction(p, 2, p->gn.bwd, p->ws_bwd_bytes);
    auto say = [](const GnGeom::Dir &d, int images, char *t, size_t n) {
        if (d.K > 0) snprintf(t, n, "clusters of %d, %d groups", d.K * images, d.gb);
        else snprintf(t, n, "%d runs of %d px", d.S, d.ppx);
    };
    char f[64], b[64];
    say(p->gn.fwd, 1, f, sizeof(f));
    say(p->gn.bwd, n, b, sizeof(b));
    snprintf(p->desc, sizeof(p->desc), "groupnorm %s groups=%dx%d forward: %s; gradient: %s", dtype == CONV_F32 ? "f32" : "bf16",
             groups, c / groups, f, b);
    *out_plan = p;
    return CONV_OK;
}

extern "C" int conv_run_groupnorm(const conv_plan_t *plan, const void *x, int64_t x_pitch, const float *gamma,
                                  const float *beta, void *y, int64_t y_pitch, float *mean, float *rstd,
                                  void *workspace, void *stream) {
    if (!plan) return CONV_ERR_NULL_ARG;
    const conv_plan *p = plan;
    if (p->algo != CONV_ALGO_GROUPNORM) return CONV_ERR_INVALID_ARG;
    if (p->s.n == 0) return CONV_OK;
    int rc;
    if ((rc = check_map(p, x, &x_pitch)) != CONV_OK || (rc = check_map(p, y, &y_pitch)) != CONV_OK) return rc;
    if (p->ws_bytes && !workspace) return CONV_ERR_NULL_ARG;
    if (((uintptr_t)workspace & 15u) || bad_f32(gamma) || bad_f32(beta) || bad_f32(mean) || bad_f32(rstd))
        return CONV_ERR_MISALIGNED;
    const int es = conv_esize(p->dtype), C = p->s.c_in;
    const long long rows = (long long)p->s.n * p->s.h * p->s.w;
    const size_t sb = (size_t)p->s.n * p->groups * 4;
    const size_t cb = (size_t)C * 4;
    const Small in[2] = {{gamma, cb}, {beta, cb}}, out[3] = {{mean, sb}, {rstd, sb}, {workspace, p->ws_bytes}};
    const Map maps_in[1] = {{x, x_pitch}};
    if (maps_overlap(x, x_pitch, y, y_pitch, rows, C, es) || results_overlap(in, out, maps_in, {y, y_pitch}, rows, C, es))
        return CONV_ERR_ALIASING;
    const GnGeom::Dir &d = p->gn.fwd;
    GnArgs a = base_args(p, d, x, x_pitch, y, y_pitch, workspace);
    a.gamma = gamma; a.beta = beta; a.mean = mean; a.rstd = rstd;
    const void *ptrs[2] = {x, y};
    const long long pitches[2] = {x_pitch, y_pitch};
    const int vec = vec_for(p, 2, ptrs, pitches);
    const int R = rows_for(C, vec);
    cudaStream_t st = (cudaStream_t)stream;
    if (clustered(d, vec)) {
        const size_t smem = cluster_args(d, vec, es, 1, a);
        const dim3 grid(d.K, (a.G + d.gb - 1) / d.gb, a.N);
        return launch(p, K_CLUSTER, vec, a, grid, smem, st, d.K) == cudaSuccess ? CONV_OK : CONV_ERR_CUDA;
    }
    const dim3 grid(a.S, a.N);
    const size_t ring = ring_size(vec * es, 1);
    cudaError_t e = launch(p, K_STATS, vec, a, grid, ring + ((size_t)R * C + C) * 8 + (size_t)C * 4, st);
    if (e == cudaSuccess) e = launch(p, K_APPLY, vec, a, grid, ring + runs_smem(a), st);
    return e == cudaSuccess ? CONV_OK : CONV_ERR_CUDA;
}

extern "C" int conv_run_groupnorm_bwd(const conv_plan_t *plan, const void *x, int64_t x_pitch, const float *gamma,
                                      const float *beta, const float *mean, const float *rstd, const void *dy,
                                      int64_t dy_pitch, void *dx, int64_t dx_pitch, float *dgamma, float *dbeta,
                                      void *workspace, void *stream) {
    if (!plan) return CONV_ERR_NULL_ARG;
    const conv_plan *p = plan;
    if (p->algo != CONV_ALGO_GROUPNORM) return CONV_ERR_INVALID_ARG;
    cudaStream_t st = (cudaStream_t)stream;
    const int es = conv_esize(p->dtype), C = p->s.c_in;
    if (bad_f32(dgamma) || bad_f32(dbeta)) return CONV_ERR_MISALIGNED;
    if (p->s.n == 0) {  // sums over nothing
        if ((dgamma && cudaMemsetAsync(dgamma, 0, (size_t)C * 4, st) != cudaSuccess) ||
            (dbeta && cudaMemsetAsync(dbeta, 0, (size_t)C * 4, st) != cudaSuccess))
            return CONV_ERR_CUDA;
        return CONV_OK;
    }
    int rc;
    if ((rc = check_map(p, x, &x_pitch)) != CONV_OK || (rc = check_map(p, dy, &dy_pitch)) != CONV_OK ||
        (rc = check_map(p, dx, &dx_pitch)) != CONV_OK)
        return rc;
    if (!mean || !rstd || (p->ws_bwd_bytes && !workspace)) return CONV_ERR_NULL_ARG;
    if (((uintptr_t)workspace & 15u) || bad_f32(gamma) || bad_f32(beta) || bad_f32(mean) || bad_f32(rstd))
        return CONV_ERR_MISALIGNED;
    const long long rows = (long long)p->s.n * p->s.h * p->s.w;
    const size_t sb = (size_t)p->s.n * p->groups * 4, cb = (size_t)C * 4;
    const Small in[4] = {{gamma, cb}, {beta, cb}, {mean, sb}, {rstd, sb}};
    const Small out[3] = {{dgamma, cb}, {dbeta, cb}, {workspace, p->ws_bwd_bytes}};
    const Map maps_in[2] = {{x, x_pitch}, {dy, dy_pitch}};
    if (maps_overlap(x, x_pitch, dx, dx_pitch, rows, C, es) || maps_overlap(dy, dy_pitch, dx, dx_pitch, rows, C, es) ||
        results_overlap(in, out, maps_in, {dx, dx_pitch}, rows, C, es))
        return CONV_ERR_ALIASING;
    const void *maps[3] = {x, dy, dx};
    const GnGeom::Dir &d = p->gn.bwd;
    GnArgs a = base_args(p, d, x, x_pitch, dx, dx_pitch, workspace);
    a.dy = dy; a.pdy = dy_pitch;
    a.gamma = gamma; a.beta = beta; a.mean = const_cast<float *>(mean); a.rstd = const_cast<float *>(rstd);
    a.dgamma = dgamma; a.dbeta = dbeta;
    const long long pitches[3] = {x_pitch, dy_pitch, dx_pitch};
    const int vec = vec_for(p, 3, maps, pitches);
    const int R = rows_for(C, vec);
    if (clustered(d, vec)) {
        const size_t smem = cluster_args(d, vec, es, 2, a);
        const dim3 grid(d.K * a.N, (a.G + d.gb - 1) / d.gb, 1);
        return launch(p, K_CLUSTER_BWD, vec, a, grid, smem, st, d.K * a.N) == cudaSuccess ? CONV_OK : CONV_ERR_CUDA;
    }
    const int head = dgamma || dbeta ? 1 : 0;
    const size_t ring = ring_size(vec * es, 2);
    cudaError_t e = launch(p, K_SUMS, vec, a, dim3(a.S, a.N), ring + ((size_t)R * C + C) * 8, st);
    const size_t need = ring + runs_smem(a), red = (size_t)kWarps * 32 * 8;
    if (e == cudaSuccess) e = launch(p, K_DX, vec, a, dim3(a.S, a.N + head), need > red ? need : red, st, 1, head);
    return e == cudaSuccess ? CONV_OK : CONV_ERR_CUDA;
}
