// dtypes.cuh -- the element types of exl3_dtype: conversions to and from fp32
// and 16-byte vector access, shared by the 4-bit and the routing kernels.
#pragma once

#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <stdint.h>

namespace exl3 {

__device__ __forceinline__ float to_f32(__half v) { return __half2float(v); }
__device__ __forceinline__ float to_f32(__nv_bfloat16 v) { return __bfloat162float(v); }
__device__ __forceinline__ float to_f32(float v) { return v; }

// fp32 -> T, one rounding to nearest even.
template <typename T>
__device__ __forceinline__ T from_f32(float v);
template <>
__device__ __forceinline__ __half from_f32<__half>(float v) { return __float2half_rn(v); }
template <>
__device__ __forceinline__ __nv_bfloat16 from_f32<__nv_bfloat16>(float v) { return __float2bfloat16_rn(v); }
template <>
__device__ __forceinline__ float from_f32<float>(float v) { return v; }

// Elements of one 16-byte vector.
template <typename T>
struct Vec {
    static constexpr int N = 16 / (int)sizeof(T);
};

// (By value: a reference to memory let the compiler load each element by itself,
// 8 narrow loads for one wide one.)
template <typename T>
__device__ __forceinline__ void unpack16(uint4 raw, float (&v)[Vec<T>::N])
{
    T e[Vec<T>::N];
    memcpy(e, &raw, 16);
#pragma unroll
    for (int i = 0; i < Vec<T>::N; ++i)
        v[i] = to_f32(e[i]);
}

template <typename T>
__device__ __forceinline__ uint4 pack16(const float (&v)[Vec<T>::N])
{
    T e[Vec<T>::N];
#pragma unroll
    for (int i = 0; i < Vec<T>::N; ++i)
        e[i] = from_f32<T>(v[i]);
    uint4 raw;
    memcpy(&raw, e, 16);
    return raw;
}

}  // namespace exl3
