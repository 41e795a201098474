// i4_matvec.cu -- products of a few 8-bit tokens with 4-bit weights that have a scale for each
// group along k, of one matrix or of the experts that each token goes to (sm_103a).
//
//   y[t][r] = sx[t] * sum_g s[r][g] a[t][r][g] + bias[r],  a = sum_{k in g} W[r][k] X[t][k]
//
// A warp takes a row and a pair: a lane every 32nd word of eight weights, whose product with the
// token's bytes is exact in int32, its sum over the lane's words in f32.
#include "token_ops.cuh"

namespace loom {
namespace {

constexpr int I4_WARPS = 8;

__device__ __forceinline__ float load_scale(const void *s, int32_t dtype, int64_t at)
{
    if (dtype == LOOM_F32)
        return static_cast<const float *>(s)[at];
    if (dtype == LOOM_F16)
        return __half2float(static_cast<const __half *>(s)[at]);
    return __bfloat162float(static_cast<const __nv_bfloat16 *>(s)[at]);
}

__global__ void __launch_bounds__(32 * I4_WARPS) i4_matvec_kernel(const I4Params p)
{
    dev::follow_previous_kernel();
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int64_t row = (int64_t)blockIdx.x * I4_WARPS + warp;
    if (row >= p.n)
        return;
    for (int64_t pair = blockIdx.y; pair < p.pairs; pair += gridDim.y) {
        const int e = p.ids ? p.ids[pair] : 0;
        if (e < 0 || e >= p.experts) {
            if (lane == 0) {
                dev::store_as(p.y, p.y_dtype, pair * p.y_stride + row, 0.0f);
                if (e >= p.experts)
                    dev::flag_error(p.error, LOOM_DEVERR_COUNT_RANGE);
            }
            continue;
        }
        const int64_t w_row = (int64_t)e * p.n + row, x_row = pair / p.pairs_per_x;
        const int32_t *w = p.w + w_row * (p.k / 8), *x = reinterpret_cast<const int32_t *>(p.x + x_row * p.k);
        float sum = 0.0f;
        for (int j = lane; j < p.k / 8; j += 32) {
            int32_t a = 0;
            for (int i = 0; i < 8; ++i) {
                const int32_t v = (int32_t)((uint32_t)w[j] << (28 - 4 * i)) >> 28;
                a += v * (int32_t)(int8_t)(x[2 * j + i / 4] >> (8 * (i & 3)));
            }
            sum = fmaf(load_scale(p.scale_w, p.scale_dtype, w_row * p.groups + 8 * j / p.group), (float)a, sum);
        }
        for (int m = 16; m >= 1; m >>= 1)
            sum += __shfl_xor_sync(dev::FULL_MASK, sum, m);
        if (lane == 0) {
            sum *= p.scale_x[x_row];
            dev::store_as(p.y, p.y_dtype, pair * p.y_stride + row, p.bias ? sum + p.bias[w_row] : sum);
        }
    }
}

}  // namespace

void i4_geometry(int64_t pairs, int64_t n, int64_t, int64_t, int64_t, int64_t, loom_launch *out)
{
    *out = loom_launch{};
    out->grid[0] = (uint32_t)((n + I4_WARPS - 1) / I4_WARPS);
    out->grid[1] = (uint32_t)(pairs < 65535 ? pairs : 65535);
    out->grid[2] = out->block[1] = out->block[2] = 1;
    out->block[0] = 32 * I4_WARPS;
    out->cluster[0] = out->cluster[1] = out->cluster[2] = 1;
    out->subgroup_size = 32;
    out->units_per_cta = I4_WARPS;
    out->kernel = LOOM_KERNEL_I4_MATVEC;
}

cudaError_t launch_i4_matvec(const I4Params &p, const loom_launch &L, cudaStream_t stream)
{
    return launch_with(i4_matvec_kernel, L, stream, p);
}

}  // namespace loom
