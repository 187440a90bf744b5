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
// A CTA's eight warps share 16 output channels, each every eighth run of 128
// input channels; the partial sums meet in shared memory in a fixed order.
#include <cuda_bf16.h>
#include <math.h>
#include <stdint.h>
#include <stdio.h>

#include <new>

#include "conv_internal.h"
#include "epilogue.cuh"

using namespace convk;

namespace {

constexpr int kWarps = 8;
constexpr int kThreads = kWarps * 32;
constexpr int kUnit = 128;       // input channels a warp takes at a time (two tiles)

struct W4Args {
    const void *x;
    const uint4 *w;
    const void *scales;
    const float *bias;
    void *y;
    int rows, ci, co, ng, units, act;
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

// Eight consecutive channels of one x row as MMA operand registers (bf16
// pairs); channels at and past ci, and rows past the last, are zero.
struct XBf16 {
    static constexpr int kParts = 1;
    using Elem = __nv_bfloat16;
    template <bool VEC>
    __device__ static __forceinline__ void load(const Elem *row, int k, int ci, bool on, uint32_t (&b)[1][4]) {
#pragma unroll
        for (int i = 0; i < 4; ++i) b[0][i] = 0u;
        if (!on) return;
        if (VEC) {
            if (k + 8 <= ci) {
                const uint4 v = *reinterpret_cast<const uint4 *>(row + k);
                b[0][0] = v.x; b[0][1] = v.y; b[0][2] = v.z; b[0][3] = v.w;
            }
        } else {
#pragma unroll
            for (int i = 0; i < 8; ++i)
                if (k + i < ci) b[0][i >> 1] |= (uint32_t)__bfloat16_as_ushort(row[k + i]) << (16 * (i & 1));
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
    template <bool VEC>
    __device__ static __forceinline__ void load(const Elem *row, int k, int ci, bool on, uint32_t (&b)[3][4]) {
        float f[8];
#pragma unroll
        for (int i = 0; i < 8; ++i) f[i] = 0.0f;
        if (on) {
            if (VEC) {
                if (k + 8 <= ci) {
                    const float4 u = *reinterpret_cast<const float4 *>(row + k), v = *reinterpret_cast<const float4 *>(row + k + 4);
                    f[0] = u.x; f[1] = u.y; f[2] = u.z; f[3] = u.w; f[4] = v.x; f[5] = v.y; f[6] = v.z; f[7] = v.w;
                }
            } else {
#pragma unroll
                for (int i = 0; i < 8; ++i)
                    if (k + i < ci) f[i] = row[k + i];
            }
        }
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            uint32_t lo[3], hi[3];
            split(f[2 * i], lo);
            split(f[2 * i + 1], hi);
#pragma unroll
            for (int q = 0; q < 3; ++q) b[q][i] = lo[q] | (hi[q] << 16);
        }
    }
};

// NT: blocks of eight x rows.  GROUP: channels a scale (32, 64 or 128).
// XVEC: x rows allow 16-byte loads of whole eights of channels.
template <typename X, int NT, int GROUP, bool XVEC>
__global__ void __launch_bounds__(kThreads) w4_kernel(W4Args a) {
    using Elem = typename X::Elem;
    extern __shared__ float red[];  // [kWarps][16][NT * 8]
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, g = lane >> 2, t = lane & 3;
    const int co0 = blockIdx.x * 16, m0 = blockIdx.y * (NT * 8);
    pdl_trigger();
    pdl_wait();
    const Elem *x = static_cast<const Elem *>(a.x);
    const Elem *sc = static_cast<const Elem *>(a.scales);
    const uint4 *w = a.w + (long long)blockIdx.x * a.units * 64 + lane;
    const bool on0 = co0 + g < a.co, on1 = co0 + g + 8 < a.co;
    const Elem *s0 = sc + (long long)(co0 + g) * a.ng, *s1 = s0 + 8LL * a.ng;

    float acc[NT][4];
#pragma unroll
    for (int n = 0; n < NT; ++n)
#pragma unroll
        for (int e = 0; e < 4; ++e) acc[n][e] = 0.0f;

    constexpr int kHalvesPerGroup = GROUP / 32;
    constexpr int kGroupsPerUnit = 4 / kHalvesPerGroup;
    for (int u = warp; u < a.units; u += kWarps) {
        const uint4 wa = w[(long long)u * 64], wb = w[(long long)u * 64 + 32];
        float f0[kGroupsPerUnit], f1[kGroupsPerUnit];
#pragma unroll
        for (int j = 0; j < kGroupsPerUnit; ++j) {
            const int gi = u * kGroupsPerUnit + j;
            f0[j] = on0 && gi < a.ng ? elem_f(s0[gi]) : 0.0f;
            f1[j] = on1 && gi < a.ng ? elem_f(s1[gi]) : 0.0f;
        }
        float c[NT][4];
#pragma unroll
        for (int h = 0; h < 4; ++h) {
            if (h % kHalvesPerGroup == 0) {
#pragma unroll
                for (int n = 0; n < NT; ++n)
#pragma unroll
                    for (int e = 0; e < 4; ++e) c[n][e] = 0.0f;
            }
            const uint32_t lo = h == 0 ? wa.x : (h == 1 ? wa.z : (h == 2 ? wb.x : wb.z));
            const uint32_t hi = h == 0 ? wa.y : (h == 1 ? wa.w : (h == 2 ? wb.y : wb.w));
            uint32_t p[4], q[4];
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                p[i] = decode(lo, i);
                q[i] = decode(hi, i);
            }
            const int k = u * kUnit + h * 32 + t * 8;
#pragma unroll
            for (int n = 0; n < NT; ++n) {
                const int m = m0 + n * 8 + g;
                uint32_t b[X::kParts][4];
                X::template load<XVEC>(x + (long long)m * a.ci, k, a.ci, m < a.rows, b);
#pragma unroll
                for (int r = 0; r < X::kParts; ++r) {
                    mma16816(c[n], p[0], q[0], p[1], q[1], b[r][0], b[r][1]);
                    mma16816(c[n], p[2], q[2], p[3], q[3], b[r][2], b[r][3]);
                }
            }
            if (h % kHalvesPerGroup == kHalvesPerGroup - 1) {
                const int j = h / kHalvesPerGroup;
#pragma unroll
                for (int n = 0; n < NT; ++n) {
                    acc[n][0] = fmaf(f0[j], c[n][0], acc[n][0]);
                    acc[n][1] = fmaf(f0[j], c[n][1], acc[n][1]);
                    acc[n][2] = fmaf(f1[j], c[n][2], acc[n][2]);
                    acc[n][3] = fmaf(f1[j], c[n][3], acc[n][3]);
                }
            }
        }
    }
    // [warp][x row][16 output channels]
    float *mine = red + warp * (NT * 8 * 16);
#pragma unroll
    for (int n = 0; n < NT; ++n) {
        mine[(n * 8 + 2 * t) * 16 + g] = acc[n][0];
        mine[(n * 8 + 2 * t + 1) * 16 + g] = acc[n][1];
        mine[(n * 8 + 2 * t) * 16 + g + 8] = acc[n][2];
        mine[(n * 8 + 2 * t + 1) * 16 + g + 8] = acc[n][3];
    }
    __syncthreads();
    for (int i = threadIdx.x; i < NT * 8 * 16; i += kThreads) {
        const int m = m0 + (i >> 4), co = co0 + (i & 15);
        if (m >= a.rows || co >= a.co) continue;
        float v = a.bias ? a.bias[co] : 0.0f;
        float s = 0.0f;
#pragma unroll
        for (int q = 0; q < kWarps; ++q) s += red[q * (NT * 8 * 16) + i];
        v = activate(s + v, a.act);
        static_cast<Elem *>(a.y)[(long long)m * a.co + co] = elem_from<Elem>(v);
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
template <typename X, int NT, int GROUP>
const void *pick_vec(bool vec) {
    return vec ? (const void *)&w4_kernel<X, NT, GROUP, true> : (const void *)&w4_kernel<X, NT, GROUP, false>;
}
template <typename X, int NT>
const void *pick_group(int group, bool vec) {
    return group == 32 ? pick_vec<X, NT, 32>(vec) : (group == 64 ? pick_vec<X, NT, 64>(vec) : pick_vec<X, NT, 128>(vec));
}
template <typename X>
const void *pick_nt(int nt, int group, bool vec) {
    switch (nt) {
    case 1: return pick_group<X, 1>(group, vec);
    case 2: return pick_group<X, 2>(group, vec);
    case 4: return pick_group<X, 4>(group, vec);
    default: return pick_group<X, 8>(group, vec);
    }
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
    p->w4.group = group;
    p->w4.ng = (c_in + group - 1) / group;
    p->w4.units = (c_in + kUnit - 1) / kUnit;
    p->w4.nt = rows <= 8 ? 1 : (rows <= 16 ? 2 : (rows <= 32 ? 4 : 8));
    snprintf(p->desc, sizeof(p->desc), "w4 %s group=%d rows/cta=%d tiles=%d", dtype == CONV_F32 ? "f32" : "bf16", group,
             p->w4.nt * 8, (c_out + 15) / 16);
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
    W4Args a = {x, static_cast<const uint4 *>(packed), scales, bias, y, rows, ci, co, p->w4.ng, p->w4.units, p->act};
    const int nt = p->w4.nt;
    const bool vec = ci % 8 == 0 && ((uintptr_t)x & 15u) == 0;
    const void *k = p->dtype == CONV_F32 ? pick_nt<XF32>(nt, p->w4.group, vec) : pick_nt<XBf16>(nt, p->w4.group, vec);
    void *args[] = {&a};
    const cudaError_t e = conv_launch(k, dim3((unsigned)((co + 15) / 16), (unsigned)((rows + nt * 8 - 1) / (nt * 8))),
                                      dim3(kThreads), args, (size_t)kWarps * nt * 8 * 16 * 4, (cudaStream_t)stream);
    return e == cudaSuccess ? CONV_OK : CONV_ERR_CUDA;
}
