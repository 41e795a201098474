// token_ops.cuh -- device helpers shared by the token operators' kernels.
#pragma once

#include <atomic>
#include <cstdint>
#include <cstring>
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

// Raises a kernel's dynamic shared-memory limit to all that a CTA may have, and checks that the
// kernel brings at least `regs` registers a thread: once per device and kernel (`done` holds
// a bit per device).
inline cudaError_t prepare_kernel(const void *kernel, int regs, std::atomic<uint64_t> &done)
{
    int device = 0;
    cudaError_t e = cudaGetDevice(&device);
    if (e != cudaSuccess)
        return e;
    const uint64_t bit = device < 64 ? 1ull << device : 0;
    if (done.load(std::memory_order_acquire) & bit)
        return cudaSuccess;
    cudaFuncAttributes fa;
    e = cudaFuncGetAttributes(&fa, kernel);
    if (e == cudaSuccess && fa.numRegs < regs)
        e = cudaErrorInvalidConfiguration;
    if (e == cudaSuccess)
        e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, 227 * 1024 - (int)fa.sharedSizeBytes);
    if (e == cudaSuccess)
        done.fetch_or(bit, std::memory_order_acq_rel);
    return e;
}

// As launch_with, for a kernel that prepare_kernel has seen.
template <typename... KArgs, typename... Args>
cudaError_t launch_prepared(void (*kernel)(KArgs...), const loom_launch &L, cudaStream_t stream, Args &&...args)
{
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(L.grid[0], L.grid[1], L.grid[2]);
    cfg.blockDim = dim3(L.block[0], L.block[1], L.block[2]);
    cfg.dynamicSmemBytes = L.smem_bytes;
    cfg.stream = stream;
    cudaLaunchAttribute attr[2];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    attr[1].id = cudaLaunchAttributeClusterDimension;
    attr[1].val.clusterDim.x = L.cluster[0];
    attr[1].val.clusterDim.y = attr[1].val.clusterDim.z = 1;
    cfg.attrs = attr;
    cfg.numAttrs = L.cluster[0] > 1 ? 2 : 1;
    return cudaLaunchKernelEx(&cfg, kernel, std::forward<Args>(args)...);
}

}  // namespace loom
