// mixer_device.cuh -- element types of the sequence-mixer kernels: vectors of
// four or eight values read to and written from fp32 registers.
#pragma once

#include "quat_device.cuh"

namespace qs {

template <typename T>
__device__ __forceinline__ float4 load4(const T *p);
template <>
__device__ __forceinline__ float4 load4<float>(const float *p) {
    return __ldg(reinterpret_cast<const float4 *>(p));
}
template <>
__device__ __forceinline__ float4 load4<__nv_bfloat16>(const __nv_bfloat16 *p) {
    return IoBF16::get(__ldg(reinterpret_cast<const uint2 *>(p)));
}

__device__ __forceinline__ void store4(float *p, const float4 v) { *reinterpret_cast<float4 *>(p) = v; }
__device__ __forceinline__ void store4(__nv_bfloat16 *p, const float4 v) {
    *reinterpret_cast<uint2 *>(p) = IoBF16::put(v);
}

// N quaternions (4 N consecutive values): one 16-byte access for two of bfloat16.
template <int N, typename T>
__device__ __forceinline__ void load_quads(const T *p, float4 *v) {
#pragma unroll
    for (int i = 0; i < N; ++i) v[i] = load4(p + 4 * i);
}
template <>
__device__ __forceinline__ void load_quads<2, __nv_bfloat16>(const __nv_bfloat16 *p, float4 *v) {
    const uint4 r = __ldg(reinterpret_cast<const uint4 *>(p));
    v[0] = IoBF16::get(make_uint2(r.x, r.y));
    v[1] = IoBF16::get(make_uint2(r.z, r.w));
}
template <int N, typename T>
__device__ __forceinline__ void store_quads(T *p, const float4 *v) {
#pragma unroll
    for (int i = 0; i < N; ++i) store4(p + 4 * i, v[i]);
}
template <>
__device__ __forceinline__ void store_quads<2, __nv_bfloat16>(__nv_bfloat16 *p, const float4 *v) {
    const uint2 a = IoBF16::put(v[0]), b = IoBF16::put(v[1]);
    *reinterpret_cast<uint4 *>(p) = make_uint4(a.x, a.y, b.x, b.y);
}

// N quaternions as they are in memory: loads that run ahead are kept so, because a
// conversion right behind a load waits for it.
template <int N, typename T>
struct RawQuads {
    float4 r[N];
    __device__ __forceinline__ void load(const T *p) {
#pragma unroll
        for (int i = 0; i < N; ++i) r[i] = __ldg(reinterpret_cast<const float4 *>(p) + i);
    }
    __device__ __forceinline__ void get(float4 *v) const {
#pragma unroll
        for (int i = 0; i < N; ++i) v[i] = r[i];
    }
};
template <int N>
struct RawQuads<N, __nv_bfloat16> {
    uint2 r[N];
    __device__ __forceinline__ void load(const __nv_bfloat16 *p) {
        if constexpr (N == 2) {
            const uint4 v = __ldg(reinterpret_cast<const uint4 *>(p));
            r[0] = make_uint2(v.x, v.y), r[1] = make_uint2(v.z, v.w);
        } else {
#pragma unroll
            for (int i = 0; i < N; ++i) r[i] = __ldg(reinterpret_cast<const uint2 *>(p) + i);
        }
    }
    __device__ __forceinline__ void get(float4 *v) const {
#pragma unroll
        for (int i = 0; i < N; ++i) v[i] = IoBF16::get(r[i]);
    }
};

__device__ __forceinline__ float to_float(float v) { return v; }
__device__ __forceinline__ float to_float(__nv_bfloat16 v) { return __bfloat162float(v); }
__device__ __forceinline__ float load1(const float *p) { return __ldg(p); }
__device__ __forceinline__ float load1(const __nv_bfloat16 *p) { return __bfloat162float(*p); }
__device__ __forceinline__ void store1(float *p, float v) { *p = v; }
__device__ __forceinline__ void store1(__nv_bfloat16 *p, float v) { *p = __float2bfloat16_rn(v); }

// One value of an array whose element type is known at run time only.
__device__ __forceinline__ float load_any(const void *p, bool bf16, long long i) {
    return bf16 ? __bfloat162float(static_cast<const __nv_bfloat16 *>(p)[i]) : static_cast<const float *>(p)[i];
}
__device__ __forceinline__ void store_any(void *p, bool bf16, long long i, float v) {
    if (bf16) static_cast<__nv_bfloat16 *>(p)[i] = __float2bfloat16_rn(v);
    else static_cast<float *>(p)[i] = v;
}

__device__ __forceinline__ float dot4(const float4 a, const float4 b) {
    return fmaf(a.x, b.x, fmaf(a.y, b.y, fmaf(a.z, b.z, a.w * b.w)));
}

}  // namespace qs
