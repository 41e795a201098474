// token_route.cu -- routing: the experts of each token and their weights from logits, and the
// gradient of those weights (sm_103a).  One warp takes a token, its scores in shared memory.
#include <cfloat>

#include "token_ops.cuh"

namespace loom {
namespace {

constexpr int RT_WARPS = 4;

// +infinity counts as the largest finite f32; NaN (and -infinity) as -infinity.
__device__ __forceinline__ float logit_of(float l) { return isnan(l) ? -INFINITY : fminf(l, FLT_MAX); }

__device__ __forceinline__ double warp_max(double v)
{
    for (int m = 16; m >= 1; m >>= 1)
        v = fmax(v, __shfl_xor_sync(dev::FULL_MASK, v, m));
    return v;
}

__device__ __forceinline__ double warp_sum(double v)
{
    for (int m = 16; m >= 1; m >>= 1)
        v += __shfl_xor_sync(dev::FULL_MASK, v, m);
    return v;
}

// The place of the largest of v[0..n) (the lowest among equals), or -1 where all are -infinity.
__device__ int warp_argmax(const double *v, int n, int lane)
{
    double best = -INFINITY;
    int at = -1;
    for (int i = lane; i < n; i += 32)
        if (v[i] > best) {
            best = v[i];
            at = i;
        }
    for (int m = 16; m >= 1; m >>= 1) {
        const double b = __shfl_xor_sync(dev::FULL_MASK, best, m);
        const int a = __shfl_xor_sync(dev::FULL_MASK, at, m);
        if (b > best || (b == best && (unsigned)a < (unsigned)at)) {
            best = b;
            at = a;
        }
    }
    return at;
}

__device__ __forceinline__ double score_of(int kind, double l, double m, double sum)
{
    return kind == LOOM_SCORE_SIGMOID ? 1.0 / (1.0 + exp(-l)) : exp(l - m) / sum;
}

template <typename E> __global__ void __launch_bounds__(32 * RT_WARPS) route_kernel(const RouteParams p)
{
    extern __shared__ double route_smem[];
    dev::follow_previous_kernel();
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    double *choose = route_smem + (size_t)warp * 2 * p.experts, *group = choose + p.experts;
    for (int64_t t = (int64_t)blockIdx.x * RT_WARPS + warp; t < p.tokens; t += (int64_t)gridDim.x * RT_WARPS) {
        const E *l = static_cast<const E *>(p.logits) + t * p.stride;
        double m = -INFINITY, sum = 0;
        for (int e = lane; e < p.experts; e += 32)
            m = fmax(m, (double)logit_of(dev::to_f32(l[e])));
        m = warp_max(m);
        if (p.score == LOOM_SCORE_SOFTMAX && m > -INFINITY) {
            for (int e = lane; e < p.experts; e += 32)
                sum += exp((double)logit_of(dev::to_f32(l[e])) - m);
            sum = warp_sum(sum);
        }
        for (int e = lane; e < p.experts; e += 32) {
            const float v = logit_of(dev::to_f32(l[e]));
            const float b = p.bias ? logit_of(p.bias[e]) : 0.0f;
            choose[e] = v == -INFINITY || b == -INFINITY ? -INFINITY : score_of(p.score, v, m, sum) + (double)b;
        }
        __syncwarp();
        if (p.groups > 1) {
            const int size = p.experts / p.groups;
            for (int g = lane; g < p.groups; g += 32) {
                double a = -INFINITY, b = -INFINITY;
                for (int i = 0; i < size; ++i) {
                    const double v = choose[g * size + i];
                    b = fmax(b, fmin(a, v));
                    a = fmax(a, v);
                }
                group[g] = p.group_best == 2 && b > -INFINITY ? a + b : a;
            }
            __syncwarp();
            for (int i = 0; i < p.top_groups; ++i) {
                const int g = warp_argmax(group, p.groups, lane);
                __syncwarp();
                if (g >= 0 && lane == 0)
                    group[g] = NAN;        // kept: never the largest again
                __syncwarp();
            }
            for (int e = lane; e < p.experts; e += 32)
                if (!isnan(group[e / size]))
                    choose[e] = -INFINITY;
            __syncwarp();
        }
        int mine = -1;
        for (int i = 0; i < p.top_k; ++i) {
            const int e = warp_argmax(choose, p.experts, lane);
            if (lane == i)
                mine = e;
            __syncwarp();
            if (e >= 0 && lane == 0)
                choose[e] = -INFINITY;
            __syncwarp();
        }
        double w = 0;
        const double v = mine >= 0 ? (double)logit_of(dev::to_f32(l[mine])) : -INFINITY;
        if (p.renormalise && p.score == LOOM_SCORE_SOFTMAX)
            m = warp_max(v);
        const double low = warp_max(v);
        if (mine >= 0) {
            // sigmoids far below zero are exponentials, which may be taken relative to the largest
            const bool far = p.renormalise && p.score == LOOM_SCORE_SIGMOID && low < -600;
            w = far ? exp(v - low) : score_of(p.score, v, m, p.renormalise ? 1.0 : sum);
        }
        if (p.renormalise)
            w /= warp_sum(w);
        if (lane < p.top_k) {
            p.ids[t * p.top_k + lane] = mine;
            p.weights[t * p.top_k + lane] = mine >= 0 ? (float)(w * p.factor) : 0.0f;
            if (mine >= 0 && p.counts)
                atomicAdd(p.counts + mine, 1);
        }
        __syncwarp();
    }
}

template <typename E> __global__ void __launch_bounds__(32 * RT_WARPS) route_grad_kernel(const RouteGradParams p)
{
    extern __shared__ double route_smem[];
    dev::follow_previous_kernel();
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    double *full = route_smem + (size_t)warp * 2 * p.experts;
    for (int64_t t = (int64_t)blockIdx.x * RT_WARPS + warp; t < p.tokens; t += (int64_t)gridDim.x * RT_WARPS) {
        const E *l = static_cast<const E *>(p.logits) + t * p.stride;
        E *d = static_cast<E *>(p.dlogits) + t * p.dstride;
        const bool soft = p.score == LOOM_SCORE_SOFTMAX;
        int e = lane < p.top_k ? p.ids[t * p.top_k + lane] : -1;
        if (e >= p.experts) {
            dev::flag_error(p.error, LOOM_DEVERR_COUNT_RANGE);
            e = -1;
        }
        float v = e >= 0 ? logit_of(dev::to_f32(l[e])) : -INFINITY;
        if (v == -INFINITY)
            e = -1;
        const double g = e >= 0 ? (double)p.factor * p.dweights[t * p.top_k + lane] : 0.0;
        double m = -INFINITY, sum = 0;
        if (p.renormalise) {
            m = warp_max((double)v);
        } else if (soft) {
            for (int i = lane; i < p.experts; i += 32)
                m = fmax(m, (double)logit_of(dev::to_f32(l[i])));
            m = warp_max(m);
            for (int i = lane; i < p.experts; i += 32)
                sum += m > -INFINITY ? exp((double)logit_of(dev::to_f32(l[i])) - m) : 0.0;
            sum = warp_sum(sum);
        }
        // chosen scores; renormalised ones relative to their sum
        const bool far = p.renormalise && !soft && m < -600;
        double s = e < 0 ? 0.0 : far ? exp(v - m) : score_of(p.score, v, m, p.renormalise ? 1.0 : sum), h = g;
        if (p.renormalise) {
            s /= warp_sum(s);                           // now w / factor
            h = g - warp_sum(g * s);                    // h S of the header
        }
        const double common = soft && !p.renormalise ? warp_sum(h * s) : 0.0;
        for (int i = lane; i < p.experts; i += 32)
            full[i] = 0;
        __syncwarp();
        for (int j = 0; j < p.top_k; ++j) {             // an id may come twice
            if (lane == j && e >= 0)
                full[e] += soft ? s * h : s * h * score_of(LOOM_SCORE_SIGMOID, -v, 0, 1);
            __syncwarp();
        }
        for (int i = lane; i < p.experts; i += 32) {
            double out = full[i];
            if (soft && !p.renormalise) {
                const float li = logit_of(dev::to_f32(l[i]));
                if (li > -INFINITY)
                    out -= exp(li - m) / sum * common;
            }
            d[i] = dev::from_f32<E>((float)out);
        }
        __syncwarp();
    }
}

}  // namespace

bool route_geometry(int64_t tokens, int32_t experts, bool backward, int64_t sms, loom_launch *out)
{
    *out = loom_launch{};
    const int64_t ctas = (tokens + RT_WARPS - 1) / RT_WARPS, most = 4 * sms;
    out->grid[0] = (uint32_t)(ctas < most ? ctas : most);
    out->grid[1] = out->grid[2] = out->block[1] = out->block[2] = 1;
    out->block[0] = 32 * RT_WARPS;
    out->cluster[0] = out->cluster[1] = out->cluster[2] = 1;
    out->subgroup_size = 32;
    out->smem_bytes = (uint32_t)(RT_WARPS * 2 * experts * sizeof(double));
    out->units_per_cta = RT_WARPS;
    out->kernel = backward ? LOOM_KERNEL_ROUTE_BACKWARD : LOOM_KERNEL_ROUTE;
    return true;
}

cudaError_t launch_route(const RouteParams &p, int32_t dtype, const loom_launch &L, cudaStream_t stream)
{
    if (dtype == LOOM_F32)
        return launch_with(route_kernel<float>, L, stream, p);
    return dtype == LOOM_F16 ? launch_with(route_kernel<__half>, L, stream, p) : launch_with(route_kernel<__nv_bfloat16>, L, stream, p);
}

cudaError_t launch_route_grad(const RouteGradParams &p, int32_t dtype, const loom_launch &L, cudaStream_t stream)
{
    if (dtype == LOOM_F32)
        return launch_with(route_grad_kernel<float>, L, stream, p);
    return dtype == LOOM_F16 ? launch_with(route_grad_kernel<__half>, L, stream, p)
                             : launch_with(route_grad_kernel<__nv_bfloat16>, L, stream, p);
}

}  // namespace loom
