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
// Variance: each thread sums (x - K) and (x - K)^2 about its own first value K
// and the pieces are joined by Chan's update (count, mean, M2).  K belongs to
// the values it is subtracted from, so the cancellation in M2 = q - s^2/n is
// bounded by the thread's own count (at most a few hundred) times 2^-24
// however far the mean lies from zero.  All statistics are fp32, in a fixed
// order: results do not change from run to run.
#include <cuda_bf16.h>
#include <math.h>
#include <stdint.h>
#include <stdio.h>

#include <new>

#include "conv_internal.h"
#include "epilogue.cuh"

using namespace convk;

namespace {

constexpr int kThreads = 256;
constexpr int kWarps = kThreads / 32;
constexpr int kMaxC = 8192;  // channels: their sums stay in shared memory (16 bytes each)

// VEC consecutive channels of one pixel as fp32.
template <typename T, int VEC> struct Vec;
template <int VEC> struct Vec<float, VEC> {
    static_assert(VEC == 4 || VEC == 1, "");
    using Raw = typename std::conditional<VEC == 4, float4, float>::type;
    __device__ static __forceinline__ void unpack(const Raw &r, float (&f)[VEC]) {
        if constexpr (VEC == 4) { f[0] = r.x; f[1] = r.y; f[2] = r.z; f[3] = r.w; } else f[0] = r;
    }
    __device__ static __forceinline__ Raw pack(const float (&f)[VEC]) {
        if constexpr (VEC == 4) return make_float4(f[0], f[1], f[2], f[3]);
        else return f[0];
    }
};
template <int VEC> struct Vec<__nv_bfloat16, VEC> {
    static_assert(VEC == 8 || VEC == 2 || VEC == 1, "");
    using Raw = typename std::conditional<VEC == 8, uint4,
                                          typename std::conditional<VEC == 2, uint32_t, uint16_t>::type>::type;
    __device__ static __forceinline__ void two(uint32_t v, float &a, float &b) {
        a = __uint_as_float(v << 16);
        b = __uint_as_float(v & 0xffff0000u);
    }
    __device__ static __forceinline__ uint32_t pair(float a, float b) {
        __nv_bfloat162 p = __floats2bfloat162_rn(a, b);
        return *reinterpret_cast<uint32_t *>(&p);
    }
    __device__ static __forceinline__ void unpack(const Raw &r, float (&f)[VEC]) {
        if constexpr (VEC == 8) {
            two(r.x, f[0], f[1]); two(r.y, f[2], f[3]); two(r.z, f[4], f[5]); two(r.w, f[6], f[7]);
        } else if constexpr (VEC == 2) {
            two(r, f[0], f[1]);
        } else {
            f[0] = __uint_as_float((uint32_t)r << 16);
        }
    }
    __device__ static __forceinline__ Raw pack(const float (&f)[VEC]) {
        if constexpr (VEC == 8)
            return make_uint4(pair(f[0], f[1]), pair(f[2], f[3]), pair(f[4], f[5]), pair(f[6], f[7]));
        else if constexpr (VEC == 2) return pair(f[0], f[1]);
        else return __bfloat16_as_ushort(__float2bfloat16_rn(f[0]));
    }
};

struct GnArgs {
    const void *x, *dy;
    void *out;                 // y, or dx
    long long px, pdy, pout;   // elements from one pixel to the next
    const float *gamma, *beta; // [C] or null
    float *mean, *rstd;        // [N][G] (forward: may be null)
    float *dgamma, *dbeta;     // [C] or null
    float2 *part;              // [N][S][G]: (mean, M2), or (sum gamma dz, sum gamma dz xhat)
    float2 *partc;             // [N][S][C]: (sum dz, sum dz xhat)
    int N, HW, C, G, cg, S, ppx;  // S runs of ppx pixels an image
    float eps;
};

// The activation's value and its derivative.  fp32 maps take CUDA's accurate
// expf and division; bf16 ones the fast forms, ~1e-6 relative, far below the
// 2^-9 of their results.  With n = e^z, t = n (n + 2): Mish = z t / (t + 2),
// Mish' = t / (t + 2) + z 4 n (1 + n) / (t + 2)^2, the exponent clamped at 20
// where both have reached their limits z and 1 in fp32.
template <int ACT, bool FAST>
__device__ __forceinline__ float act_val(float z) {
    if constexpr (ACT == ACT_RELU) return z < 0.0f ? 0.0f : z;  // (NaN stays NaN)
    else if constexpr (ACT == ACT_MISH) return FAST ? mish_fast(z) : mish_f32(z);
    else return z;
}
template <int ACT, bool FAST>
__device__ __forceinline__ float act_grad(float z) {
    if constexpr (ACT == ACT_RELU) return z > 0.0f ? 1.0f : 0.0f;
    else if constexpr (ACT == ACT_MISH) {
        const float zc = fminf(z, 20.0f);
        const float n = FAST ? __expf(zc) : expf(zc);
        const float t = n * (n + 2.0f);
        const float r = FAST ? __fdividef(1.0f, t + 2.0f) : 1.0f / (t + 2.0f);
        return r * (t + z * (4.0f * n * (1.0f + n)) * r);
    } else return 1.0f;
}

__device__ __forceinline__ float warp_sum(float v) {
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
    return v;
}

// How a CTA's threads cover a pixel's channel vectors: with cvn vectors a
// pixel, R = kThreads / cvn pixels side by side (R = 1 and several rounds
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
    // pixels of the run of `np` that thread row q takes
    __device__ __forceinline__ int count(int q, int np) const { return np > q ? (np - q + R - 1) / R : 0; }
};

// (mean, M2) of each group over this CTA's run of pixels.
template <typename T, int VEC>
__global__ void __launch_bounds__(kThreads) gn_stats_kernel(GnArgs a) {
    using V = Vec<T, VEC>;
    extern __shared__ float sh[];  // mean[R*C], M2[R*C], then 3 floats a warp
    const Cover cv(a.C, VEC);
    const int entries = cv.R * a.C;
    float *smean = sh, *sm2 = sh + entries, *swarp = sm2 + entries;
    const int n = blockIdx.y, s = blockIdx.x;
    const int p0 = s * a.ppx, np = min(a.ppx, a.HW - p0);
    pdl_trigger();
    pdl_wait();
    const T *x = static_cast<const T *>(a.x) + ((long long)n * a.HW + p0) * a.px;
    if (cv.on) {
        for (int col = cv.col; col < cv.cvn; col += kThreads) {
            const T *xc = x + col * VEC;
            float K[VEC], s1[VEC], s2[VEC];
#pragma unroll
            for (int e = 0; e < VEC; ++e) K[e] = s1[e] = s2[e] = 0.0f;
            if (cv.r < np) V::unpack(*reinterpret_cast<const typename V::Raw *>(xc + cv.r * a.px), K);
            constexpr int U = 4;
            for (int p = cv.r; p < np; p += cv.R * U) {
                typename V::Raw raw[U];
#pragma unroll
                for (int u = 0; u < U; ++u)
                    if (p + u * cv.R < np) raw[u] = *reinterpret_cast<const typename V::Raw *>(xc + (p + u * cv.R) * a.px);
#pragma unroll
                for (int u = 0; u < U; ++u)
                    if (p + u * cv.R < np) {
                        float f[VEC];
                        V::unpack(raw[u], f);
#pragma unroll
                        for (int e = 0; e < VEC; ++e) {
                            const float d = f[e] - K[e];
                            s1[e] += d;
                            s2[e] = fmaf(d, d, s2[e]);
                        }
                    }
            }
            const int cnt = cv.count(cv.r, np);
            const float inv = cnt > 0 ? 1.0f / (float)cnt : 0.0f;
#pragma unroll
            for (int e = 0; e < VEC; ++e) {
                const int i = cv.r * a.C + col * VEC + e;
                const float d = s1[e] * inv;
                smean[i] = K[e] + d;
                sm2[i] = s2[e] - s1[e] * d;
            }
        }
    }
    __syncthreads();
    // Join: wpg warps a group, each an interleaved share of its R * cg
    // entries; then one thread a group over the warps' results.
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    int wpg = 1;
    while (wpg * 2 * a.G <= kWarps) wpg *= 2;
    const int per = cv.R * a.cg;
    for (int g0 = 0; g0 < a.G; g0 += kWarps / wpg) {
        const int g = g0 + warp / wpg, part = warp % wpg;
        if (g < a.G) {
            float cnt = 0.0f, sum = 0.0f;
            for (int i = part * 32 + lane; i < per; i += wpg * 32) {
                const int r = i / a.cg, c = g * a.cg + (i - r * a.cg);
                const float nr = (float)cv.count(r, np);
                cnt += nr;
                if (nr > 0.0f) sum += nr * smean[r * a.C + c];
            }
            cnt = warp_sum(cnt);
            sum = warp_sum(sum);
            const float mu = cnt > 0.0f ? sum / cnt : 0.0f;
            float m2 = 0.0f;
            for (int i = part * 32 + lane; i < per; i += wpg * 32) {
                const int r = i / a.cg, c = g * a.cg + (i - r * a.cg);
                const float nr = (float)cv.count(r, np);
                if (nr > 0.0f) {
                    const float d = smean[r * a.C + c] - mu;
                    m2 += sm2[r * a.C + c] + nr * d * d;
                }
            }
            m2 = warp_sum(m2);
            if (lane == 0) { swarp[warp * 3] = cnt; swarp[warp * 3 + 1] = mu; swarp[warp * 3 + 2] = m2; }
        }
        __syncthreads();
        if (g < a.G && part == 0 && lane == 0) {
            float cnt = 0.0f, sum = 0.0f, m2 = 0.0f;
            for (int q = 0; q < wpg; ++q) { cnt += swarp[(warp + q) * 3]; sum += swarp[(warp + q) * 3] * swarp[(warp + q) * 3 + 1]; }
            const float mu = sum / cnt;
            for (int q = 0; q < wpg; ++q) {
                const float nq = swarp[(warp + q) * 3], d = swarp[(warp + q) * 3 + 1] - mu;
                if (nq > 0.0f) m2 += swarp[(warp + q) * 3 + 2] + nq * d * d;
            }
            a.part[((long long)n * a.S + s) * a.G + g] = make_float2(mu, m2);
        }
        __syncthreads();
    }
}

// mean and rstd of group g of image n from the S runs' (mean, M2); every lane
// of a warp returns them.
__device__ __forceinline__ float2 join_stats(const GnArgs &a, int n, int g, int lane) {
    const float2 *p = a.part + (long long)n * a.S * a.G + g;
    const float inv = 1.0f / ((float)a.HW * (float)a.cg);
    float sum = 0.0f;
    for (int s = lane; s < a.S; s += 32) sum += (float)min(a.ppx, a.HW - s * a.ppx) * (float)a.cg * p[(long long)s * a.G].x;
    const float mu = warp_sum(sum) * inv;
    float m2 = 0.0f;
    for (int s = lane; s < a.S; s += 32) {
        const float2 v = p[(long long)s * a.G];
        const float d = v.x - mu;
        m2 += v.y + (float)min(a.ppx, a.HW - s * a.ppx) * (float)a.cg * d * d;
    }
    m2 = warp_sum(m2);
    return make_float2(mu, 1.0f / sqrtf(m2 * inv + a.eps));
}

// y = act(gamma (x - mean) rstd + beta) over one run of pixels.
template <typename T, int VEC, int ACT>
__global__ void __launch_bounds__(kThreads) gn_apply_kernel(GnArgs a) {
    using V = Vec<T, VEC>;
    constexpr bool kFast = sizeof(T) == 2;
    extern __shared__ float sh[];  // [G] (mean, rstd)
    float2 *stat = reinterpret_cast<float2 *>(sh);
    const Cover cv(a.C, VEC);
    const int n = blockIdx.y, s = blockIdx.x;
    const int p0 = s * a.ppx, np = min(a.ppx, a.HW - p0);
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    pdl_trigger();
    pdl_wait();
    for (int g = warp; g < a.G; g += kWarps) {
        const float2 st = join_stats(a, n, g, lane);
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
    const T *x = static_cast<const T *>(a.x) + ((long long)n * a.HW + p0) * a.px;
    T *y = static_cast<T *>(a.out) + ((long long)n * a.HW + p0) * a.pout;
    for (int col = cv.col; col < cv.cvn; col += kThreads) {
        float mu[VEC], sc[VEC], be[VEC];
#pragma unroll
        for (int e = 0; e < VEC; ++e) {
            const int c = col * VEC + e;
            const float2 st = stat[c / a.cg];
            mu[e] = st.x;
            sc[e] = st.y * (a.gamma ? a.gamma[c] : 1.0f);
            be[e] = a.beta ? a.beta[c] : 0.0f;
        }
        constexpr int U = 4;
        for (int p = cv.r; p < np; p += cv.R * U) {
            typename V::Raw raw[U];
#pragma unroll
            for (int u = 0; u < U; ++u)
                if (p + u * cv.R < np)
                    raw[u] = *reinterpret_cast<const typename V::Raw *>(x + (p + u * cv.R) * a.px + col * VEC);
#pragma unroll
            for (int u = 0; u < U; ++u)
                if (p + u * cv.R < np) {
                    float f[VEC];
                    V::unpack(raw[u], f);
#pragma unroll
                    for (int e = 0; e < VEC; ++e) f[e] = act_val<ACT, kFast>(fmaf(f[e] - mu[e], sc[e], be[e]));
                    *reinterpret_cast<typename V::Raw *>(y + (p + u * cv.R) * a.pout + col * VEC) = V::pack(f);
                }
        }
    }
}

// Sums of dz and dz xhat per channel, and of gamma times them per group, over
// one run of pixels.
template <typename T, int VEC, int ACT>
__global__ void __launch_bounds__(kThreads) gn_bwd_sums_kernel(GnArgs a) {
    using V = Vec<T, VEC>;
    constexpr bool kFast = sizeof(T) == 2;
    extern __shared__ float sh[];  // [R*C] float2, then [C] float2
    const Cover cv(a.C, VEC);
    float2 *ent = reinterpret_cast<float2 *>(sh);
    float2 *chan = ent + cv.R * a.C;
    const int n = blockIdx.y, s = blockIdx.x;
    const int p0 = s * a.ppx, np = min(a.ppx, a.HW - p0);
    pdl_trigger();
    pdl_wait();
    const T *x = static_cast<const T *>(a.x) + ((long long)n * a.HW + p0) * a.px;
    const T *dy = static_cast<const T *>(a.dy) + ((long long)n * a.HW + p0) * a.pdy;
    if (cv.on) {
        for (int col = cv.col; col < cv.cvn; col += kThreads) {
            float mu[VEC], rs[VEC], ga[VEC], be[VEC], A[VEC], B[VEC];
#pragma unroll
            for (int e = 0; e < VEC; ++e) {
                const int c = col * VEC + e;
                const long long g = (long long)n * a.G + c / a.cg;
                mu[e] = a.mean[g];
                rs[e] = a.rstd[g];
                ga[e] = a.gamma ? a.gamma[c] : 1.0f;
                be[e] = a.beta ? a.beta[c] : 0.0f;
                A[e] = B[e] = 0.0f;
            }
            constexpr int U = 2;
            for (int p = cv.r; p < np; p += cv.R * U) {
                typename V::Raw rx[U], rd[U];
#pragma unroll
                for (int u = 0; u < U; ++u)
                    if (p + u * cv.R < np) {
                        rx[u] = *reinterpret_cast<const typename V::Raw *>(x + (p + u * cv.R) * a.px + col * VEC);
                        rd[u] = *reinterpret_cast<const typename V::Raw *>(dy + (p + u * cv.R) * a.pdy + col * VEC);
                    }
#pragma unroll
                for (int u = 0; u < U; ++u)
                    if (p + u * cv.R < np) {
                        float f[VEC], d[VEC];
                        V::unpack(rx[u], f);
                        V::unpack(rd[u], d);
#pragma unroll
                        for (int e = 0; e < VEC; ++e) {
                            const float xh = (f[e] - mu[e]) * rs[e];
                            const float dz = d[e] * act_grad<ACT, kFast>(fmaf(xh, ga[e], be[e]));
                            A[e] += dz;
                            B[e] = fmaf(dz, xh, B[e]);
                        }
                    }
            }
#pragma unroll
            for (int e = 0; e < VEC; ++e) ent[cv.r * a.C + col * VEC + e] = make_float2(A[e], B[e]);
        }
    }
    __syncthreads();
    // channels over the R rows: L lanes a channel
    int L = 1;
    while (L < 32 && L * 2 * a.C <= kThreads) L *= 2;
    const int per = kThreads / L, sub = threadIdx.x % L;
    for (int c0 = 0; c0 < a.C; c0 += per) {
        const int c = c0 + threadIdx.x / L;
        float A = 0.0f, B = 0.0f;
        if (c < a.C)
            for (int r = sub; r < cv.R; r += L) {
                const float2 v = ent[r * a.C + c];
                A += v.x;
                B += v.y;
            }
        for (int o = L / 2; o > 0; o >>= 1) {
            A += __shfl_xor_sync(0xffffffffu, A, o);
            B += __shfl_xor_sync(0xffffffffu, B, o);
        }
        if (c < a.C && sub == 0) {
            a.partc[((long long)n * a.S + s) * a.C + c] = make_float2(A, B);
            const float ga = a.gamma ? a.gamma[c] : 1.0f;
            chan[c] = make_float2(ga * A, ga * B);
        }
    }
    __syncthreads();
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    for (int g = warp; g < a.G; g += kWarps) {
        float A = 0.0f, B = 0.0f;
        for (int c = lane; c < a.cg; c += 32) {
            const float2 v = chan[g * a.cg + c];
            A += v.x;
            B += v.y;
        }
        A = warp_sum(A);
        B = warp_sum(B);
        if (lane == 0) a.part[((long long)n * a.S + s) * a.G + g] = make_float2(A, B);
    }
}

// dx over one run of pixels (grid rows 1..N); grid row 0 joins the channels'
// sums of every image and run into dgamma and dbeta, 32 channels a CTA.
template <typename T, int VEC, int ACT>
__global__ void __launch_bounds__(kThreads) gn_bwd_dx_kernel(GnArgs a) {
    using V = Vec<T, VEC>;
    constexpr bool kFast = sizeof(T) == 2;
    extern __shared__ float sh[];  // [G] (s1, s2) / m, or [kWarps][32] float2
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    pdl_trigger();
    pdl_wait();
    if (blockIdx.y == 0) {
        if (!a.dgamma && !a.dbeta) return;
        float2 *red = reinterpret_cast<float2 *>(sh);
        const long long rows = (long long)a.N * a.S;
        for (int c0 = blockIdx.x * 32; c0 < a.C; c0 += gridDim.x * 32) {
            const int c = c0 + lane;
            float A = 0.0f, B = 0.0f;
            if (c < a.C)
                for (long long r = warp; r < rows; r += kWarps) {
                    const float2 v = a.partc[r * a.C + c];
                    A += v.x;
                    B += v.y;
                }
            red[warp * 32 + lane] = make_float2(A, B);
            __syncthreads();
            if (warp == 0 && c < a.C) {
                for (int q = 1; q < kWarps; ++q) { A += red[q * 32 + lane].x; B += red[q * 32 + lane].y; }
                if (a.dbeta) a.dbeta[c] = A;
                if (a.dgamma) a.dgamma[c] = B;
            }
            __syncthreads();
        }
        return;
    }
    float2 *sum = reinterpret_cast<float2 *>(sh);
    const Cover cv(a.C, VEC);
    const int n = blockIdx.y - 1, s = blockIdx.x;
    const int p0 = s * a.ppx, np = min(a.ppx, a.HW - p0);
    const float inv = 1.0f / ((float)a.HW * (float)a.cg);
    for (int g = warp; g < a.G; g += kWarps) {
        const float2 *p = a.part + (long long)n * a.S * a.G + g;
        float A = 0.0f, B = 0.0f;
        for (int q = lane; q < a.S; q += 32) {
            const float2 v = p[(long long)q * a.G];
            A += v.x;
            B += v.y;
        }
        A = warp_sum(A);
        B = warp_sum(B);
        if (lane == 0) sum[g] = make_float2(A * inv, B * inv);
    }
    __syncthreads();
    if (!cv.on) return;
    const T *x = static_cast<const T *>(a.x) + ((long long)n * a.HW + p0) * a.px;
    const T *dy = static_cast<const T *>(a.dy) + ((long long)n * a.HW + p0) * a.pdy;
    T *dx = static_cast<T *>(a.out) + ((long long)n * a.HW + p0) * a.pout;
    for (int col = cv.col; col < cv.cvn; col += kThreads) {
        float mu[VEC], rs[VEC], ga[VEC], be[VEC], m1[VEC], m2[VEC];
#pragma unroll
        for (int e = 0; e < VEC; ++e) {
            const int c = col * VEC + e, g = c / a.cg;
            mu[e] = a.mean[(long long)n * a.G + g];
            rs[e] = a.rstd[(long long)n * a.G + g];
            ga[e] = a.gamma ? a.gamma[c] : 1.0f;
            be[e] = a.beta ? a.beta[c] : 0.0f;
            m1[e] = sum[g].x;
            m2[e] = sum[g].y;
        }
        constexpr int U = 2;
        for (int p = cv.r; p < np; p += cv.R * U) {
            typename V::Raw rx[U], rd[U];
#pragma unroll
            for (int u = 0; u < U; ++u)
                if (p + u * cv.R < np) {
                    rx[u] = *reinterpret_cast<const typename V::Raw *>(x + (p + u * cv.R) * a.px + col * VEC);
                    rd[u] = *reinterpret_cast<const typename V::Raw *>(dy + (p + u * cv.R) * a.pdy + col * VEC);
                }
#pragma unroll
            for (int u = 0; u < U; ++u)
                if (p + u * cv.R < np) {
                    float f[VEC], d[VEC];
                    V::unpack(rx[u], f);
                    V::unpack(rd[u], d);
#pragma unroll
                    for (int e = 0; e < VEC; ++e) {
                        const float xh = (f[e] - mu[e]) * rs[e];
                        const float dz = d[e] * act_grad<ACT, kFast>(fmaf(xh, ga[e], be[e]));
                        f[e] = rs[e] * (fmaf(ga[e], dz, -m1[e]) - xh * m2[e]);
                    }
                    *reinterpret_cast<typename V::Raw *>(dx + (p + u * cv.R) * a.pout + col * VEC) = V::pack(f);
                }
        }
    }
}

// ------------------------------------------------------------------ host side
enum { K_STATS, K_APPLY, K_SUMS, K_DX };

template <typename T, int VEC>
const void *pick(int which, int act) {
    switch (which) {
    case K_STATS: return (const void *)&gn_stats_kernel<T, VEC>;
    case K_APPLY:
        return act == ACT_MISH ? (const void *)&gn_apply_kernel<T, VEC, ACT_MISH>
                               : (act == ACT_RELU ? (const void *)&gn_apply_kernel<T, VEC, ACT_RELU>
                                                  : (const void *)&gn_apply_kernel<T, VEC, ACT_NONE>);
    case K_SUMS:
        return act == ACT_MISH ? (const void *)&gn_bwd_sums_kernel<T, VEC, ACT_MISH>
                               : (act == ACT_RELU ? (const void *)&gn_bwd_sums_kernel<T, VEC, ACT_RELU>
                                                  : (const void *)&gn_bwd_sums_kernel<T, VEC, ACT_NONE>);
    default:
        return act == ACT_MISH ? (const void *)&gn_bwd_dx_kernel<T, VEC, ACT_MISH>
                               : (act == ACT_RELU ? (const void *)&gn_bwd_dx_kernel<T, VEC, ACT_RELU>
                                                  : (const void *)&gn_bwd_dx_kernel<T, VEC, ACT_NONE>);
    }
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

// Whether two maps of `rows` pixels share an element.  Two channel slices of
// one buffer (the same pitch) interleave without sharing any.
bool maps_overlap(const void *a, long long pa, const void *b, long long pb, long long rows, int C, int es) {
    if (!a || !b || rows <= 0) return false;
    const uintptr_t a0 = (uintptr_t)a, b0 = (uintptr_t)b;
    const uintptr_t na = (uintptr_t)((rows - 1) * pa + C) * es, nb = (uintptr_t)((rows - 1) * pb + C) * es;
    if (!(a0 < b0 + nb && b0 < a0 + na)) return false;
    if (pa != pb) return true;
    const uintptr_t pitch = (uintptr_t)pa * es, d = (b0 > a0 ? b0 - a0 : pitch - (a0 - b0) % pitch) % pitch;
    return d < (uintptr_t)C * es || pitch - d < (uintptr_t)C * es;
}
bool range_overlaps(const void *small, size_t bytes, const void *map, long long pitch, long long rows, int C, int es) {
    if (!small || !map || rows <= 0 || bytes == 0) return false;
    const uintptr_t a0 = (uintptr_t)small, b0 = (uintptr_t)map;
    return a0 < b0 + (uintptr_t)((rows - 1) * pitch + C) * es && b0 < a0 + bytes;
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

GnArgs base_args(const conv_plan *p, const void *x, long long px, void *out, long long pout, void *ws) {
    GnArgs a = {};
    a.x = x; a.px = px; a.out = out; a.pout = pout;
    a.N = p->s.n; a.HW = p->s.h * p->s.w; a.C = p->s.c_in; a.G = p->groups; a.cg = p->s.c_in / p->groups;
    a.S = p->gn.S; a.ppx = p->gn.ppx; a.eps = p->gn.eps;
    a.part = static_cast<float2 *>(ws);
    a.partc = a.part + (long long)a.N * a.S * a.G;
    return a;
}

cudaError_t launch(const conv_plan *p, int which, int vec, GnArgs &a, dim3 grid, size_t smem, cudaStream_t st) {
    const void *k = pick_kernel(which, p->dtype, vec, p->act);
    if (smem > 48 * 1024) {
        const int rc = conv_grant_smem(k, p->device, (int)smem);
        if (rc != CONV_OK) return cudaErrorInvalidValue;
    }
    void *args[] = {&a};
    return conv_launch(k, grid, dim3(kThreads), args, smem, st);
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
    // Runs of pixels: four CTAs a SM over the whole batch, but at least four
    // pixels a thread.
    const int HW = h * w;
    const int R = rows_for(c, c % (16 / conv_esize(dtype)) == 0 ? 16 / conv_esize(dtype) : 1);
    long long S = n > 0 ? (4LL * p->num_sms + n - 1) / n : 1;
    const long long most = ((long long)HW + 4LL * R - 1) / (4LL * R);
    if (S > most) S = most;
    if (S < 1) S = 1;
    p->gn.ppx = (int)((HW + S - 1) / S);
    p->gn.S = (HW + p->gn.ppx - 1) / p->gn.ppx;
    p->ws_bytes = (size_t)n * p->gn.S * ((size_t)groups + c) * sizeof(float2);
    snprintf(p->desc, sizeof(p->desc), "groupnorm %s groups=%d x %d runs=%d x %d px", dtype == CONV_F32 ? "f32" : "bf16",
             groups, c / groups, p->gn.S, p->gn.ppx);
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
    if (maps_overlap(x, x_pitch, y, y_pitch, rows, C, es) || range_overlaps(gamma, (size_t)C * 4, y, y_pitch, rows, C, es) ||
        range_overlaps(beta, (size_t)C * 4, y, y_pitch, rows, C, es) || range_overlaps(mean, sb, y, y_pitch, rows, C, es) ||
        range_overlaps(rstd, sb, y, y_pitch, rows, C, es) || range_overlaps(mean, sb, x, x_pitch, rows, C, es) ||
        range_overlaps(rstd, sb, x, x_pitch, rows, C, es) ||
        range_overlaps(workspace, p->ws_bytes, x, x_pitch, rows, C, es) ||
        range_overlaps(workspace, p->ws_bytes, y, y_pitch, rows, C, es))
        return CONV_ERR_ALIASING;
    GnArgs a = base_args(p, x, x_pitch, y, y_pitch, workspace);
    a.gamma = gamma; a.beta = beta; a.mean = mean; a.rstd = rstd;
    const void *ptrs[2] = {x, y};
    const long long pitches[2] = {x_pitch, y_pitch};
    const int vec = vec_for(p, 2, ptrs, pitches);
    const int R = rows_for(C, vec);
    cudaStream_t st = (cudaStream_t)stream;
    const dim3 grid(a.S, a.N);
    cudaError_t e = launch(p, K_STATS, vec, a, grid, ((size_t)R * C * 2 + 3 * kWarps) * 4, st);
    if (e == cudaSuccess) e = launch(p, K_APPLY, vec, a, grid, (size_t)a.G * 8, st);
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
    if (!mean || !rstd || (p->ws_bytes && !workspace)) return CONV_ERR_NULL_ARG;
    if (((uintptr_t)workspace & 15u) || bad_f32(gamma) || bad_f32(beta) || bad_f32(mean) || bad_f32(rstd))
        return CONV_ERR_MISALIGNED;
    const long long rows = (long long)p->s.n * p->s.h * p->s.w;
    const size_t sb = (size_t)p->s.n * p->groups * 4, cb = (size_t)C * 4;
    const void *in_small[4] = {gamma, beta, mean, rstd};
    const size_t in_bytes[4] = {cb, cb, sb, sb};
    bool bad = maps_overlap(x, x_pitch, dx, dx_pitch, rows, C, es) || maps_overlap(dy, dy_pitch, dx, dx_pitch, rows, C, es);
    for (int i = 0; i < 4; ++i) bad = bad || range_overlaps(in_small[i], in_bytes[i], dx, dx_pitch, rows, C, es);
    const void *maps[3] = {x, dy, dx};
    const int64_t mp[3] = {x_pitch, dy_pitch, dx_pitch};
    for (int i = 0; i < 3; ++i)
        bad = bad || range_overlaps(dgamma, cb, maps[i], mp[i], rows, C, es) ||
              range_overlaps(dbeta, cb, maps[i], mp[i], rows, C, es) ||
              range_overlaps(workspace, p->ws_bytes, maps[i], mp[i], rows, C, es);
    if (bad) return CONV_ERR_ALIASING;
    GnArgs a = base_args(p, x, x_pitch, dx, dx_pitch, workspace);
    a.dy = dy; a.pdy = dy_pitch;
    a.gamma = gamma; a.beta = beta; a.mean = const_cast<float *>(mean); a.rstd = const_cast<float *>(rstd);
    a.dgamma = dgamma; a.dbeta = dbeta;
    const long long pitches[3] = {x_pitch, dy_pitch, dx_pitch};
    const int vec = vec_for(p, 3, maps, pitches);
    const int R = rows_for(C, vec);
    cudaError_t e = launch(p, K_SUMS, vec, a, dim3(a.S, a.N), ((size_t)R * C + C) * 8, st);
    const size_t dxs = (size_t)a.G * 8 > kWarps * 32 * 8 ? (size_t)a.G * 8 : (size_t)kWarps * 32 * 8;
    if (e == cudaSuccess) e = launch(p, K_DX, vec, a, dim3(a.S, a.N + 1), dxs, st);
    return e == cudaSuccess ? CONV_OK : CONV_ERR_CUDA;
}
