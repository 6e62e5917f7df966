// Rows of 128 elements by one warp in fp32, lane l with elements 4l .. 4l+3: the
// loads and stores of the bounded-cache attention kernels, and the running softmax of
// the rows that prompt attention computes on CUDA cores.
#pragma once

#include <cmath>
#include <cstdint>
#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include "ptx.cuh"

namespace qsa {

__device__ __forceinline__ float warp_sum(float x) {
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) x += __shfl_xor_sync(FULL_MASK, x, o);
    return x;
}

// Four consecutive elements as fp32, read through L2.
template <typename T>
__device__ __forceinline__ float4 load4(const T *p);
template <>
__device__ __forceinline__ float4 load4<float>(const float *p) {
    return __ldcg(reinterpret_cast<const float4 *>(p));
}
template <>
__device__ __forceinline__ float4 load4<__half>(const __half *p) {
    const uint2 w = __ldcg(reinterpret_cast<const uint2 *>(p));
    const float2 a = __half22float2(*reinterpret_cast<const __half2 *>(&w.x));
    const float2 b = __half22float2(*reinterpret_cast<const __half2 *>(&w.y));
    return make_float4(a.x, a.y, b.x, b.y);
}
template <>
__device__ __forceinline__ float4 load4<__nv_bfloat16>(const __nv_bfloat16 *p) {
    const uint2 w = __ldcg(reinterpret_cast<const uint2 *>(p));
    return make_float4(__uint_as_float(w.x << 16), __uint_as_float(w.x & 0xFFFF0000u), __uint_as_float(w.y << 16),
                       __uint_as_float(w.y & 0xFFFF0000u));
}

template <typename T>
__device__ __forceinline__ void store4(T *p, float4 v);
template <>
__device__ __forceinline__ void store4<float>(float *p, float4 v) {
    *reinterpret_cast<float4 *>(p) = v;
}
template <>
__device__ __forceinline__ void store4<__half>(__half *p, float4 v) {
    __half2 *q = reinterpret_cast<__half2 *>(p);
    q[0] = __floats2half2_rn(v.x, v.y);
    q[1] = __floats2half2_rn(v.z, v.w);
}
template <>
__device__ __forceinline__ void store4<__nv_bfloat16>(__nv_bfloat16 *p, float4 v) {
    __nv_bfloat162 *q = reinterpret_cast<__nv_bfloat162 *>(p);
    q[0] = __floats2bfloat162_rn(v.x, v.y);
    q[1] = __floats2bfloat162_rn(v.z, v.w);
}

// Running softmax of a row in base 2: maximum, sum and this lane's outputs.
struct RowState {
    float m = -INFINITY, l = 0.0f;
    float4 o = make_float4(0.f, 0.f, 0.f, 0.f);
    __device__ __forceinline__ void add(float logit2, float4 v) {
        if (logit2 == -INFINITY) return;
        const float mn = fmaxf(m, logit2);
        const float a = exp2f(m - mn), p = exp2f(logit2 - mn);
        m = mn;
        l = l * a + p;
        o.x = o.x * a + p * v.x;
        o.y = o.y * a + p * v.y;
        o.z = o.z * a + p * v.z;
        o.w = o.w * a + p * v.w;
    }
    __device__ __forceinline__ float4 result() const {
        const float r = l > 0.0f || l != l ? 1.0f / l : 0.0f;
        return make_float4(o.x * r, o.y * r, o.z * r, o.w * r);
    }
};

__device__ __forceinline__ float dot4(float4 a, float4 b) {
    return fmaf(a.x, b.x, fmaf(a.y, b.y, fmaf(a.z, b.z, a.w * b.w)));
}

}  // namespace qsa
