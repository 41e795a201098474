// token_ops.cuh -- device helpers shared by the token operators' kernels.
#pragma once

#include <cstdint>
#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include "common.cuh"
#include "token.h"

namespace loom {
namespace dev {

__device__ __forceinline__ float to_f32(float v) { return v; }
__device__ __forceinline__ float to_f32(__half v) { return __half2float(v); }
__device__ __forceinline__ float to_f32(__nv_bfloat16 v) { return __bfloat162float(v); }

template <typename E> __device__ __forceinline__ E from_f32(float v);
template <> __device__ __forceinline__ float from_f32<float>(float v) { return v; }
template <> __device__ __forceinline__ __half from_f32<__half>(float v) { return __float2half_rn(v); }
template <> __device__ __forceinline__ __nv_bfloat16 from_f32<__nv_bfloat16>(float v) { return __float2bfloat16_rn(v); }

// 16 bytes of elements.
template <typename E> struct alignas(16) Vec16 {
    static constexpr int N = 16 / (int)sizeof(E);
    E e[N];
};

__device__ __forceinline__ void store_as(void *y, int32_t dtype, int64_t at, float v)
{
    if (dtype == LOOM_F32)
        static_cast<float *>(y)[at] = v;
    else if (dtype == LOOM_F16)
        static_cast<__half *>(y)[at] = __float2half_rn(v);
    else
        static_cast<__nv_bfloat16 *>(y)[at] = __float2bfloat16_rn(v);
}

// The product's epilogue: acc * (sw * sx) + bias, each step one f32 rounding.
__device__ __forceinline__ float dequantized(int32_t acc, float sw, float sx, const float *bias, int64_t row)
{
    const float v = __fmul_rn((float)acc, __fmul_rn(sw, sx));
    return bias ? __fadd_rn(v, __ldg(bias + row)) : v;
}

}  // namespace dev
}  // namespace loom
