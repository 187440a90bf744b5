// NHWC maps as the operators around the layer take them: [rows] pixels of C
// channels, a pitch of elements from one pixel to the next.  Vector access and
// asynchronous copies on the device, overlaps of maps on the host.
#pragma once

#include <cuda_bf16.h>
#include <stdint.h>

#include <type_traits>

#include "tc_ptx.cuh"

namespace convk {

// VEC consecutive channels of one pixel, as fp32 pairs (VEC = 1: the first
// lane of one pair).
template <typename T, int VEC> struct Vec;
template <int VEC> struct Vec<float, VEC> {
    static_assert(VEC == 4 || VEC == 1, "");
    static constexpr int kPairs = (VEC + 1) / 2;
    using Raw = typename std::conditional<VEC == 4, float4, float>::type;
    __device__ static __forceinline__ void unpack(const Raw &r, float2 (&f)[kPairs]) {
        if constexpr (VEC == 4) { f[0] = make_float2(r.x, r.y); f[1] = make_float2(r.z, r.w); }
        else f[0] = make_float2(r, 0.0f);
    }
    __device__ static __forceinline__ Raw pack(const float2 (&f)[kPairs]) {
        if constexpr (VEC == 4) return make_float4(f[0].x, f[0].y, f[1].x, f[1].y);
        else return f[0].x;
    }
};
template <int VEC> struct Vec<__nv_bfloat16, VEC> {
    static_assert(VEC == 8 || VEC == 2 || VEC == 1, "");
    static constexpr int kPairs = (VEC + 1) / 2;
    using Raw = typename std::conditional<VEC == 8, uint4,
                                          typename std::conditional<VEC == 2, uint32_t, uint16_t>::type>::type;
    __device__ static __forceinline__ float2 two(uint32_t v) {
        return make_float2(__uint_as_float(v << 16), __uint_as_float(v & 0xffff0000u));
    }
    __device__ static __forceinline__ uint32_t pair(float2 v) {
        __nv_bfloat162 p = __floats2bfloat162_rn(v.x, v.y);
        return *reinterpret_cast<uint32_t *>(&p);
    }
    __device__ static __forceinline__ void unpack(const Raw &r, float2 (&f)[kPairs]) {
        if constexpr (VEC == 8) { f[0] = two(r.x); f[1] = two(r.y); f[2] = two(r.z); f[3] = two(r.w); }
        else if constexpr (VEC == 2) f[0] = two(r);
        else f[0] = make_float2(__uint_as_float((uint32_t)r << 16), 0.0f);
    }
    __device__ static __forceinline__ Raw pack(const float2 (&f)[kPairs]) {
        if constexpr (VEC == 8) return make_uint4(pair(f[0]), pair(f[1]), pair(f[2]), pair(f[3]));
        else if constexpr (VEC == 2) return pair(f[0]);
        else return __bfloat16_as_ushort(__float2bfloat16_rn(f[0].x));
    }
};

__device__ __forceinline__ float warp_sum(float v) {
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
    return v;
}

template <int BYTES>
__device__ __forceinline__ void copy_async(uint32_t dst, const void *src) {
    if constexpr (BYTES == 16)
        asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(dst), "l"(src) : "memory");
    else
        asm volatile("cp.async.ca.shared.global [%0], [%1], %2;" ::"r"(dst), "l"(src), "n"(BYTES) : "memory");
}
// Four bytes of which the first `bytes` are read and the others become 0.
__device__ __forceinline__ void copy_async_part(uint32_t dst, const void *src, int bytes) {
    asm volatile("cp.async.ca.shared.global [%0], [%1], 4, %2;" ::"r"(dst), "l"(src), "r"(bytes) : "memory");
}
template <int LEFT>
__device__ __forceinline__ void copy_wait() { asm volatile("cp.async.wait_group %0;" ::"n"(LEFT) : "memory"); }
__device__ __forceinline__ void copy_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
// One vector global -> shared (two-byte vectors through a register).
template <typename Raw>
__device__ __forceinline__ void copy_vec(Raw *dst, const Raw *src) {
    if constexpr (sizeof(Raw) >= 4) copy_async<(int)sizeof(Raw)>(tc::smem_u32(dst), src);
    else *dst = *src;
}

// Distributed shared memory: another CTA's copy of a variable of this one's.
__device__ __forceinline__ float2 ld_peer(const float2 *p, uint32_t rank) {
    float2 v;
    asm volatile("ld.shared::cluster.v2.f32 {%0, %1}, [%2];" : "=f"(v.x), "=f"(v.y) : "r"(tc::mapa_shared(tc::smem_u32(p), rank)) : "memory");
    return v;
}
// (every thread of the CTA, warps converged)
__device__ __forceinline__ void cluster_arrive() { __syncwarp(); asm volatile("barrier.cluster.arrive.release.aligned;" ::: "memory"); }
__device__ __forceinline__ void cluster_wait() { __syncwarp(); asm volatile("barrier.cluster.wait.acquire.aligned;" ::: "memory"); }

// Whether two maps of `rows` pixels share an element.  Two channel slices of
// one buffer (the same pitch) interleave without sharing any.
inline bool maps_overlap(const void *a, long long pa, const void *b, long long pb, long long rows, int C, int es) {
    if (!a || !b || rows <= 0) return false;
    const uintptr_t a0 = (uintptr_t)a, b0 = (uintptr_t)b;
    const uintptr_t na = (uintptr_t)((rows - 1) * pa + C) * es, nb = (uintptr_t)((rows - 1) * pb + C) * es;
    if (!(a0 < b0 + nb && b0 < a0 + na)) return false;
    if (pa != pb) return true;
    const uintptr_t pitch = (uintptr_t)pa * es, d = (b0 > a0 ? b0 - a0 : pitch - (a0 - b0) % pitch) % pitch;
    return d < (uintptr_t)C * es || pitch - d < (uintptr_t)C * es;
}
inline bool range_overlaps(const void *small, size_t bytes, const void *map, long long pitch, long long rows, int C, int es) {
    if (!small || !map || rows <= 0 || bytes == 0) return false;
    const uintptr_t a0 = (uintptr_t)small, b0 = (uintptr_t)map;
    return a0 < b0 + (uintptr_t)((rows - 1) * pitch + C) * es && b0 < a0 + bytes;
}

}  // namespace convk
