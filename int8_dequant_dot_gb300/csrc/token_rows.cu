// token_rows.cu -- operators over the rows of an activation matrix (sm_103a):
// tokens to signed bytes, layer norm (forward, forward to signed bytes,
// backward with the gradients of gain and bias).
//
// All are bound by the bytes of the rows, read once and written once.
//  * Forward and quantisation: a row is held in the registers of one CTA (one
//    warp for short rows), so mean, squares about the mean and largest magnitude
//    are taken from registers in turn, each with one reduction, and the row is
//    read once.  Rows beyond 32768 elements are read again for each pass (L2).
//  * Backward: CTAs walk over the rows; a thread keeps the same columns for all
//    of them, so the gain's and bias's gradients grow in its registers, and each
//    CTA leaves one partial sum per column in the workspace.  A second launch adds
//    the partial sums in a fixed order: no atomics, the same bits on every call.
//    Rows wider than 8192 take two passes: the two sums of each row, then blocks
//    of columns.
//  * Loads are as wide as every row's start allows: 16 or 8 bytes, else one element.
#include "token_ops.cuh"

namespace loom {
namespace {

constexpr int ROW_WARP_ROWS = 4;      // rows per CTA where a warp takes a whole row
constexpr float TINY_AMAX = 7.888609052210118e-31f;   // 2^-100

template <typename E, int V> struct alignas(sizeof(E) * V) Pack {
    E e[V];
};

template <typename E, int V> __device__ __forceinline__ void load_f32(const E *p, float (&v)[V])
{
    const Pack<E, V> q = *reinterpret_cast<const Pack<E, V> *>(p);
#pragma unroll
    for (int i = 0; i < V; ++i)
        v[i] = dev::to_f32(q.e[i]);
}

template <typename E, int V> __device__ __forceinline__ void store_f32(E *p, const float (&v)[V])
{
    Pack<E, V> q;
#pragma unroll
    for (int i = 0; i < V; ++i)
        q.e[i] = dev::from_f32<E>(v[i]);
    *reinterpret_cast<Pack<E, V> *>(p) = q;
}

__device__ __forceinline__ float warp_sum(float v)
{
#pragma unroll
    for (int m = 16; m >= 1; m >>= 1)
        v += __shfl_xor_sync(dev::FULL_MASK, v, m);
    return v;
}

// Sum over the CTA (or the warp where WARP); `red` holds one float per warp and is
// not written again before every thread has read it (each reduction has its own).
template <bool WARP> __device__ __forceinline__ float group_sum(float v, float *red)
{
    v = warp_sum(v);
    if (WARP)
        return v;
    const int lane = threadIdx.x & 31, warps = blockDim.x >> 5;
    if (lane == 0)
        red[threadIdx.x >> 5] = v;
    __syncthreads();
    return warp_sum(lane < warps ? red[lane] : 0.0f);
}

template <bool WARP> __device__ __forceinline__ uint32_t group_max(uint32_t v, uint32_t *red)
{
    v = __reduce_max_sync(dev::FULL_MASK, v);
    if (WARP)
        return v;
    const int lane = threadIdx.x & 31, warps = blockDim.x >> 5;
    if (lane == 0)
        red[threadIdx.x >> 5] = v;
    __syncthreads();
    return __reduce_max_sync(dev::FULL_MASK, lane < warps ? red[lane] : 0u);
}

__device__ __forceinline__ uint32_t magnitude_bits(float v) { return __float_as_uint(v) & 0x7fffffffu; }

// The factor of a token's bytes, and its scale, from the bits of its largest magnitude
// (as whole numbers these order like the magnitudes, with NaN above infinity).
__device__ __forceinline__ float byte_factor(uint32_t amax_bits, float &scale, bool &bad)
{
    const float amax = __uint_as_float(amax_bits);
    bad = amax_bits >= 0x7f800000u;
    if (bad || amax < TINY_AMAX) {   // 127 / amax would leave f32 for the smallest
        scale = bad ? __uint_as_float(0x7fc00000u) : 0.0f;
        return 0.0f;
    }
    scale = __fdiv_rn(amax, 127.0f);
    return __fdiv_rn(127.0f, amax);
}

__device__ __forceinline__ int8_t to_byte(float v, float inv, bool bad)
{
    return bad ? (int8_t)0 : (int8_t)__float2int_rn(__fmul_rn(v, inv));
}

__device__ __forceinline__ float reciprocal_deviation(float squares, int32_t width, float eps)
{
    return __fdiv_rn(1.0f, __fsqrt_rn(__fadd_rn(__fdiv_rn(squares, (float)width), eps)));
}

// One row's outputs of V columns starting at c.
template <RowMode M, int V>
__device__ __forceinline__ void normalise(const RowsParams &p, int32_t c, float mean, float rstd, float (&v)[V])
{
    float g[V], b[V];
#pragma unroll
    for (int i = 0; i < V; ++i) {
        g[i] = p.gain ? __ldg(p.gain + c + i) : 1.0f;
        b[i] = p.bias ? __ldg(p.bias + c + i) : 0.0f;
    }
#pragma unroll
    for (int i = 0; i < V; ++i)
        v[i] = (v[i] - mean) * rstd * g[i] + b[i];
}

template <typename E, RowMode M, int V, int EPT, bool WARP>
__global__ void __launch_bounds__(WARP ? 32 * ROW_WARP_ROWS : 1024) rows_kernel(const RowsParams p)
{
    constexpr int NV = EPT / V;
    __shared__ float red[3][32];
    const int group = WARP ? 32 : blockDim.x, t = WARP ? (threadIdx.x & 31) : threadIdx.x;
    const int64_t row = WARP ? (int64_t)blockIdx.x * (blockDim.x >> 5) + (threadIdx.x >> 5) : blockIdx.x;
    dev::follow_previous_kernel();
    if (WARP && row >= p.rows)
        return;
    const E *x = static_cast<const E *>(p.x) + row * p.x_stride;
    float v[NV][V];
#pragma unroll
    for (int j = 0; j < NV; ++j) {
        const int c = (t + j * group) * V;
        if (c < p.width)
            load_f32<E, V>(x + c, v[j]);
        else
#pragma unroll
            for (int i = 0; i < V; ++i)
                v[j][i] = 0.0f;
    }
    if (M != RowMode::Quantize) {
        float s = 0.0f;
#pragma unroll
        for (int j = 0; j < NV; ++j)
#pragma unroll
            for (int i = 0; i < V; ++i)
                s += v[j][i];
        const float mean = __fdiv_rn(group_sum<WARP>(s, red[0]), (float)p.width);
        s = 0.0f;
#pragma unroll
        for (int j = 0; j < NV; ++j)
            if ((t + j * group) * V < p.width)
#pragma unroll
                for (int i = 0; i < V; ++i)
                    s = fmaf(v[j][i] - mean, v[j][i] - mean, s);
        const float rstd = reciprocal_deviation(group_sum<WARP>(s, red[1]), p.width, p.eps);
        if (M == RowMode::Norm && t == 0) {
            if (p.mean)
                p.mean[row] = mean;
            if (p.rstd)
                p.rstd[row] = rstd;
        }
#pragma unroll
        for (int j = 0; j < NV; ++j) {
            const int c = (t + j * group) * V;
            if (c < p.width) {
                normalise<M, V>(p, c, mean, rstd, v[j]);
                if (M == RowMode::Norm)
                    store_f32<E, V>(static_cast<E *>(p.y) + row * p.y_stride + c, v[j]);
            }
        }
    }
    if (M != RowMode::Norm) {
        uint32_t a = 0;
#pragma unroll
        for (int j = 0; j < NV; ++j)
            if ((t + j * group) * V < p.width)
#pragma unroll
                for (int i = 0; i < V; ++i)
                    a = max(a, magnitude_bits(v[j][i]));
        float scale;
        bool bad;
        const float inv = byte_factor(group_max<WARP>(a, reinterpret_cast<uint32_t *>(red[2])), scale, bad);
        if (t == 0) {
            p.scale[row] = scale;
            if (bad)
                dev::flag_error(p.error, LOOM_DEVERR_NONFINITE);
        }
        int8_t *q = p.q + row * p.width;
#pragma unroll
        for (int j = 0; j < NV; ++j) {
            const int c = (t + j * group) * V;
            if (c < p.width) {
                Pack<int8_t, V> o;
#pragma unroll
                for (int i = 0; i < V; ++i)
                    o.e[i] = to_byte(v[j][i], inv, bad);
                *reinterpret_cast<Pack<int8_t, V> *>(q + c) = o;
            }
        }
    }
}

// The same for rows of any length: each pass reads the row again.
template <typename E, RowMode M, int V> __global__ void __launch_bounds__(1024) long_rows_kernel(const RowsParams p)
{
    __shared__ float red[3][32];
    const int64_t row = blockIdx.x;
    dev::follow_previous_kernel();
    const E *x = static_cast<const E *>(p.x) + row * p.x_stride;
    const int32_t c0 = threadIdx.x * V, step = blockDim.x * V;
    float mean = 0.0f, rstd = 1.0f, v[V];
    if (M != RowMode::Quantize) {
        float s = 0.0f;
        for (int64_t c = c0; c < p.width; c += step) {
            load_f32<E, V>(x + c, v);
#pragma unroll
            for (int i = 0; i < V; ++i)
                s += v[i];
        }
        mean = __fdiv_rn(group_sum<false>(s, red[0]), (float)p.width);
        s = 0.0f;
        for (int64_t c = c0; c < p.width; c += step) {
            load_f32<E, V>(x + c, v);
#pragma unroll
            for (int i = 0; i < V; ++i)
                s = fmaf(v[i] - mean, v[i] - mean, s);
        }
        rstd = reciprocal_deviation(group_sum<false>(s, red[1]), p.width, p.eps);
    }
    if (M == RowMode::Norm) {
        if (threadIdx.x == 0) {
            if (p.mean)
                p.mean[row] = mean;
            if (p.rstd)
                p.rstd[row] = rstd;
        }
        for (int64_t c = c0; c < p.width; c += step) {
            load_f32<E, V>(x + c, v);
            normalise<M, V>(p, (int32_t)c, mean, rstd, v);
            store_f32<E, V>(static_cast<E *>(p.y) + row * p.y_stride + c, v);
        }
        return;
    }
    uint32_t a = 0;
    for (int64_t c = c0; c < p.width; c += step) {
        load_f32<E, V>(x + c, v);
        if (M == RowMode::NormI8)
            normalise<M, V>(p, (int32_t)c, mean, rstd, v);
#pragma unroll
        for (int i = 0; i < V; ++i)
            a = max(a, magnitude_bits(v[i]));
    }
    float scale;
    bool bad;
    const float inv = byte_factor(group_max<false>(a, reinterpret_cast<uint32_t *>(red[2])), scale, bad);
    if (threadIdx.x == 0) {
        p.scale[row] = scale;
        if (bad)
            dev::flag_error(p.error, LOOM_DEVERR_NONFINITE);
    }
    for (int64_t c = c0; c < p.width; c += step) {
        load_f32<E, V>(x + c, v);
        if (M == RowMode::NormI8)
            normalise<M, V>(p, (int32_t)c, mean, rstd, v);
        Pack<int8_t, V> o;
#pragma unroll
        for (int i = 0; i < V; ++i)
            o.e[i] = to_byte(v[i], inv, bad);
        *reinterpret_cast<Pack<int8_t, V> *>(p.q + row * p.width + c) = o;
    }
}

constexpr int EPT_SMALL = 16, EPT_LARGE = 32;

template <typename E, RowMode M, int V>
cudaError_t launch_rows_v(const RowsParams &p, const loom_launch &L, cudaStream_t stream)
{
    if (L.kernel == LOOM_KERNEL_NORM_LONG)
        return launch_with(long_rows_kernel<E, M, V>, L, stream, p);
    if (p.width <= 32 * EPT_SMALL)
        return launch_with(rows_kernel<E, M, V, EPT_SMALL, true>, L, stream, p);
    if (p.width <= 1024 * EPT_SMALL)
        return launch_with(rows_kernel<E, M, V, EPT_SMALL, false>, L, stream, p);
    return launch_with(rows_kernel<E, M, V, EPT_LARGE, false>, L, stream, p);
}

template <typename E, int V>
cudaError_t launch_rows_m(const RowsParams &p, RowMode mode, const loom_launch &L, cudaStream_t stream)
{
    switch (mode) {
    case RowMode::Quantize: return launch_rows_v<E, RowMode::Quantize, V>(p, L, stream);
    case RowMode::Norm: return launch_rows_v<E, RowMode::Norm, V>(p, L, stream);
    default: return launch_rows_v<E, RowMode::NormI8, V>(p, L, stream);
    }
}

// ---- backward ------------------------------------------------------------------
// Sums of two values over the CTA (or warp).
template <bool WARP> __device__ __forceinline__ void group_sum2(float &a, float &b, float2 *red)
{
    a = warp_sum(a);
    b = warp_sum(b);
    if (WARP)
        return;
    const int lane = threadIdx.x & 31, warps = blockDim.x >> 5;
    if (lane == 0)
        red[threadIdx.x >> 5] = make_float2(a, b);
    __syncthreads();
    const float2 r = lane < warps ? red[lane] : make_float2(0.0f, 0.0f);
    a = warp_sum(r.x);
    b = warp_sum(r.y);
}

template <typename E, int V, bool WARP> __global__ void __launch_bounds__(1024) norm_grad_kernel(const NormGradParams p)
{
    constexpr int NV = NG_EPT / V;
    extern __shared__ float shared_sums[];          // WARP: [warps][2][width] at the end
    __shared__ float2 red[2][32];
    const int group = WARP ? 32 : blockDim.x, t = WARP ? (threadIdx.x & 31) : threadIdx.x;
    const int per_cta = WARP ? blockDim.x >> 5 : 1, mine = WARP ? threadIdx.x >> 5 : 0;
    float dg[NV][V], db[NV][V], gain[NV][V];
    dev::follow_previous_kernel();
#pragma unroll
    for (int j = 0; j < NV; ++j)
#pragma unroll
        for (int i = 0; i < V; ++i) {
            const int c = (t + j * group) * V + i;
            dg[j][i] = db[j][i] = 0.0f;
            gain[j][i] = c < p.width && p.gain ? __ldg(p.gain + c) : 1.0f;
        }
    int turn = 0;
    for (int64_t row = (int64_t)blockIdx.x * per_cta + mine; row < p.rows; row += (int64_t)gridDim.x * per_cta) {
        const E *x = static_cast<const E *>(p.x) + row * p.x_stride;
        const E *dy = static_cast<const E *>(p.dy) + row * p.dy_stride;
        const float mean = p.mean[row], rstd = p.rstd[row];
        float xh[NV][V], d[NV][V];
#pragma unroll
        for (int j = 0; j < NV; ++j) {
            const int c = (t + j * group) * V;
            if (c < p.width) {
                load_f32<E, V>(x + c, xh[j]);
                load_f32<E, V>(dy + c, d[j]);
            } else {
#pragma unroll
                for (int i = 0; i < V; ++i) {
                    xh[j][i] = mean;
                    d[j][i] = 0.0f;
                }
            }
        }
        float s1 = 0.0f, s2 = 0.0f;
#pragma unroll
        for (int j = 0; j < NV; ++j)
#pragma unroll
            for (int i = 0; i < V; ++i) {
                xh[j][i] = (xh[j][i] - mean) * rstd;
                const float g = d[j][i] * gain[j][i];
                s1 += g;
                s2 = fmaf(g, xh[j][i], s2);
                dg[j][i] = fmaf(d[j][i], xh[j][i], dg[j][i]);
                db[j][i] += d[j][i];
            }
        if (p.dx) {
            group_sum2<WARP>(s1, s2, red[turn]);
            turn ^= 1;
            s1 = __fdiv_rn(s1, (float)p.width);
            s2 = __fdiv_rn(s2, (float)p.width);
            E *dx = static_cast<E *>(p.dx) + row * p.dx_stride;
#pragma unroll
            for (int j = 0; j < NV; ++j) {
                const int c = (t + j * group) * V;
                if (c < p.width) {
#pragma unroll
                    for (int i = 0; i < V; ++i)
                        d[j][i] = rstd * (d[j][i] * gain[j][i] - s1 - xh[j][i] * s2);
                    store_f32<E, V>(dx + c, d[j]);
                }
            }
        }
    }
    if (!p.partial)
        return;
    float *out = p.partial + (int64_t)blockIdx.x * 2 * p.width;
    float *mine_out = WARP ? shared_sums + (int64_t)mine * 2 * p.width : out;
#pragma unroll
    for (int j = 0; j < NV; ++j)
#pragma unroll
        for (int i = 0; i < V; ++i) {
            const int c = (t + j * group) * V + i;
            if (c < p.width) {
                mine_out[c] = dg[j][i];
                mine_out[p.width + c] = db[j][i];
            }
        }
    if (WARP) {
        __syncthreads();
        for (int i = threadIdx.x; i < 2 * p.width; i += blockDim.x) {
            float s = 0.0f;
            for (int w = 0; w < per_cta; ++w)
                s += shared_sums[w * 2 * p.width + i];
            out[i] = s;
        }
    }
}

// Rows wider than the registers of a CTA: the two sums of each row ...
template <typename E, int V> __global__ void __launch_bounds__(1024) long_norm_sums_kernel(const NormGradParams p)
{
    __shared__ float2 red[32];
    const int64_t row = blockIdx.x;
    dev::follow_previous_kernel();
    const E *x = static_cast<const E *>(p.x) + row * p.x_stride;
    const E *dy = static_cast<const E *>(p.dy) + row * p.dy_stride;
    const float mean = p.mean[row], rstd = p.rstd[row];
    float s1 = 0.0f, s2 = 0.0f, xv[V], d[V];
    for (int64_t c = threadIdx.x * V; c < p.width; c += blockDim.x * V) {
        load_f32<E, V>(x + c, xv);
        load_f32<E, V>(dy + c, d);
#pragma unroll
        for (int i = 0; i < V; ++i) {
            const float g = d[i] * (p.gain ? __ldg(p.gain + c + i) : 1.0f);
            s1 += g;
            s2 = fmaf(g, (xv[i] - mean) * rstd, s2);
        }
    }
    group_sum2<false>(s1, s2, red);
    if (threadIdx.x == 0) {
        p.row_sums[2 * row] = __fdiv_rn(s1, (float)p.width);
        p.row_sums[2 * row + 1] = __fdiv_rn(s2, (float)p.width);
    }
}

// ... then a block of columns (blockIdx.y) of a share of the rows (blockIdx.x).
constexpr int NG_LONG_THREADS = 256;
template <typename E, int V>
__global__ void __launch_bounds__(NG_LONG_THREADS) long_norm_grad_kernel(const NormGradParams p)
{
    const int64_t c = ((int64_t)blockIdx.y * NG_LONG_THREADS + threadIdx.x) * V;
    dev::follow_previous_kernel();
    if (c >= p.width)
        return;
    float dg[V], db[V], gain[V];
#pragma unroll
    for (int i = 0; i < V; ++i) {
        dg[i] = db[i] = 0.0f;
        gain[i] = p.gain ? __ldg(p.gain + c + i) : 1.0f;
    }
    for (int64_t row = blockIdx.x; row < p.rows; row += gridDim.x) {
        const float mean = p.mean[row], rstd = p.rstd[row];
        float xv[V], d[V];
        load_f32<E, V>(static_cast<const E *>(p.x) + row * p.x_stride + c, xv);
        load_f32<E, V>(static_cast<const E *>(p.dy) + row * p.dy_stride + c, d);
        const float s1 = p.dx ? p.row_sums[2 * row] : 0.0f, s2 = p.dx ? p.row_sums[2 * row + 1] : 0.0f;
#pragma unroll
        for (int i = 0; i < V; ++i) {
            const float xh = (xv[i] - mean) * rstd;
            dg[i] = fmaf(d[i], xh, dg[i]);
            db[i] += d[i];
            d[i] = rstd * (d[i] * gain[i] - s1 - xh * s2);
        }
        if (p.dx)
            store_f32<E, V>(static_cast<E *>(p.dx) + row * p.dx_stride + c, d);
    }
    if (p.partial) {
        float *out = p.partial + (int64_t)blockIdx.x * 2 * p.width + c;
#pragma unroll
        for (int i = 0; i < V; ++i) {
            out[i] = dg[i];
            out[p.width + i] = db[i];
        }
    }
}

// Partial column sums [parts][2 width] -> dgain, dbias: 32 columns per CTA, eight
// threads per column over interleaved parts, added in a fixed order.
constexpr int NG_SUM_COLS = 32, NG_SUM_GROUPS = 8;
__global__ void __launch_bounds__(NG_SUM_COLS *NG_SUM_GROUPS)
    norm_grad_columns_kernel(const float *partial, int64_t parts, int32_t width, float *dgain, float *dbias)
{
    __shared__ float part[NG_SUM_GROUPS][NG_SUM_COLS];
    const int col = threadIdx.x % NG_SUM_COLS, group = threadIdx.x / NG_SUM_COLS;
    const int64_t c = (int64_t)blockIdx.x * NG_SUM_COLS + col;
    dev::follow_previous_kernel();
    float s = 0.0f;
    if (c < 2 * (int64_t)width)
#pragma unroll 8
        for (int64_t q = group; q < parts; q += NG_SUM_GROUPS)
            s += partial[q * 2 * width + c];
    part[group][col] = s;
    __syncthreads();
    if (group == 0 && c < 2 * (int64_t)width) {
#pragma unroll
        for (int g = 1; g < NG_SUM_GROUPS; ++g)
            s += part[g][col];
        float *out = c < width ? dgain : dbias;
        if (out)
            out[c < width ? c : c - width] = s;
    }
}

template <typename E, int V>
cudaError_t launch_norm_grad_v(const NormGradParams &p, const loom_launch &L, cudaStream_t stream)
{
    if (p.width <= 32 * NG_EPT)
        return launch_with(norm_grad_kernel<E, V, true>, L, stream, p);
    if (p.width <= NG_MAX_WIDTH)
        return launch_with(norm_grad_kernel<E, V, false>, L, stream, p);
    if (p.dx) {
        loom_launch S = L;
        S.grid[0] = (uint32_t)p.rows;
        S.grid[1] = 1;
        S.block[0] = 1024;
        const cudaError_t e = launch_with(long_norm_sums_kernel<E, V>, S, stream, p);
        if (e != cudaSuccess)
            return e;
    }
    loom_launch G = L;
    G.grid[1] = (uint32_t)((p.width / V + NG_LONG_THREADS - 1) / NG_LONG_THREADS);
    return launch_with(long_norm_grad_kernel<E, V>, G, stream, p);
}

}  // namespace

int row_vec(int32_t dtype, int32_t width, const void *const *pointers, const int64_t *strides, int n)
{
    const int64_t size = dtype_bytes(dtype);
    for (int64_t bytes = 16; bytes > size; bytes >>= 1) {
        const int64_t v = bytes / size;
        if (v == 2)   // 4-byte loads of 16-bit pairs, 8-byte loads of f32 pairs: one element instead
            break;
        bool ok = width % v == 0;
        for (int i = 0; i < n && ok; ++i)
            ok = reinterpret_cast<uintptr_t>(pointers[i]) % bytes == 0 && strides[i] % v == 0;
        if (ok)
            return (int)v;
    }
    return 1;
}

bool rows_geometry(int64_t rows, int32_t width, loom_launch *out)
{
    *out = loom_launch{};
    out->grid[1] = out->grid[2] = out->block[1] = out->block[2] = 1;
    out->cluster[0] = out->cluster[1] = out->cluster[2] = 1;
    out->subgroup_size = 32;
    out->kernel = LOOM_KERNEL_NORM_ROWS;
    out->units_per_cta = 1;
    int64_t threads, grid = rows;
    if (width <= 32 * EPT_SMALL) {
        threads = 32 * ROW_WARP_ROWS;
        out->units_per_cta = ROW_WARP_ROWS;
        grid = (rows + ROW_WARP_ROWS - 1) / ROW_WARP_ROWS;
    } else if (width <= 1024 * EPT_LARGE) {
        const int ept = width <= 1024 * EPT_SMALL ? EPT_SMALL : EPT_LARGE;
        threads = ((int64_t)width + 32 * ept - 1) / (32 * ept) * 32;
    } else {
        threads = 1024;
        out->kernel = LOOM_KERNEL_NORM_LONG;
    }
    if (grid > 0x7fffffff)
        return false;
    out->grid[0] = (uint32_t)grid;
    out->block[0] = (uint32_t)threads;
    return true;
}

cudaError_t launch_rows(const RowsParams &p, RowMode mode, int32_t dtype, int vec, const loom_launch &L,
                        cudaStream_t stream)
{
    if (dtype == LOOM_F32)
        return vec == 4 ? launch_rows_m<float, 4>(p, mode, L, stream) : launch_rows_m<float, 1>(p, mode, L, stream);
    if (dtype == LOOM_F16)
        return vec == 8   ? launch_rows_m<__half, 8>(p, mode, L, stream)
               : vec == 4 ? launch_rows_m<__half, 4>(p, mode, L, stream)
                          : launch_rows_m<__half, 1>(p, mode, L, stream);
    return vec == 8   ? launch_rows_m<__nv_bfloat16, 8>(p, mode, L, stream)
           : vec == 4 ? launch_rows_m<__nv_bfloat16, 4>(p, mode, L, stream)
                      : launch_rows_m<__nv_bfloat16, 1>(p, mode, L, stream);
}

bool norm_grad_geometry(int64_t rows, int32_t width, int64_t sms, loom_launch *out, int64_t *parts)
{
    *out = loom_launch{};
    out->grid[1] = out->grid[2] = out->block[1] = out->block[2] = 1;
    out->cluster[0] = out->cluster[1] = out->cluster[2] = 1;
    out->subgroup_size = 32;
    out->kernel = LOOM_KERNEL_NORM_BACKWARD;
    out->units_per_cta = 1;
    int64_t threads, per_sm, grid = rows;
    if (width <= 32 * NG_EPT) {
        threads = 256;
        per_sm = 4;
        out->units_per_cta = 8;
        grid = (rows + 7) / 8;
        out->smem_bytes = (uint32_t)(8 * 2 * width * 4);
    } else if (width <= NG_MAX_WIDTH) {
        threads = ((int64_t)width + 32 * NG_EPT - 1) / (32 * NG_EPT) * 32;
        per_sm = threads >= 512 ? 1024 / threads : threads >= 256 ? 4 : 8;
        per_sm = per_sm < 1 ? 1 : per_sm;
    } else {
        threads = NG_LONG_THREADS;
        per_sm = 1;
    }
    const int64_t most = per_sm * sms;
    grid = grid < most ? grid : most;
    out->grid[0] = (uint32_t)grid;
    out->block[0] = (uint32_t)threads;
    if (parts)
        *parts = grid;
    return true;
}

int64_t norm_grad_workspace_bytes(int64_t rows, int32_t width, int64_t sms)
{
    loom_launch L;
    int64_t parts = 0;
    norm_grad_geometry(rows, width, sms, &L, &parts);
    return (parts * 2 * width + (width > NG_MAX_WIDTH ? 2 * rows : 0)) * 4;
}

cudaError_t launch_norm_grad(const NormGradParams &p, int32_t dtype, int vec, const loom_launch &L, int64_t parts,
                             cudaStream_t stream)
{
    if (p.rows > 0) {
        cudaError_t e;
        if (dtype == LOOM_F32)
            e = vec == 4 ? launch_norm_grad_v<float, 4>(p, L, stream) : launch_norm_grad_v<float, 1>(p, L, stream);
        else if (dtype == LOOM_F16)
            e = vec == 8   ? launch_norm_grad_v<__half, 8>(p, L, stream)
                : vec == 4 ? launch_norm_grad_v<__half, 4>(p, L, stream)
                           : launch_norm_grad_v<__half, 1>(p, L, stream);
        else
            e = vec == 8   ? launch_norm_grad_v<__nv_bfloat16, 8>(p, L, stream)
                : vec == 4 ? launch_norm_grad_v<__nv_bfloat16, 4>(p, L, stream)
                           : launch_norm_grad_v<__nv_bfloat16, 1>(p, L, stream);
        if (e != cudaSuccess)
            return e;
    }
    if (!p.dgain && !p.dbias)
        return cudaSuccess;
    loom_launch S = L;
    S.grid[0] = (uint32_t)((2 * (int64_t)p.width + NG_SUM_COLS - 1) / NG_SUM_COLS);
    S.grid[1] = 1;
    S.block[0] = NG_SUM_COLS * NG_SUM_GROUPS;
    S.smem_bytes = 0;
    return launch_with(norm_grad_columns_kernel, S, stream, (const float *)p.partial, parts, p.width, p.dgain,
                       p.dbias);
}

}  // namespace loom
