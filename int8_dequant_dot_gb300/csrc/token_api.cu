// token_api.cu -- host side of the token operators (loom_token.h): argument
// validation, launch geometry and the extern "C" entry points.
#include <cmath>
#include <cstring>

#include "token.h"

namespace loom {
namespace {

constexpr uint64_t DEFAULT_WAIT_NS = 1000000000ull;   // 1 s per barrier wait
constexpr int64_t MAX_K = 131068;                     // 128 * 128 * k < 2^31 and k % 4 == 0
constexpr int64_t MAX_INT = 0x7fffffff;
constexpr int64_t MM_MAX_ROWS_PER_CTA = 1024;         // dp4a totals: 32 KiB of shared memory

bool misaligned(const void *p, uintptr_t a) { return (reinterpret_cast<uintptr_t>(p) & (a - 1)) != 0; }
bool known(int32_t dtype) { return dtype == LOOM_F32 || dtype == LOOM_F16 || dtype == LOOM_BF16; }
loom_status of_cuda(cudaError_t e) { return e == cudaSuccess ? LOOM_OK : LOOM_ERR_CUDA; }

loom_status sm_count(int64_t *sms)
{
    int dev = 0, n = 0;
    if (cudaGetDevice(&dev) != cudaSuccess ||
        cudaDeviceGetAttribute(&n, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess || n < 1) {
        cudaGetLastError();
        return LOOM_ERR_CUDA;
    }
    *sms = n;
    return LOOM_OK;
}

loom_launch plain_launch(int64_t gx, int64_t gy, uint32_t block, uint32_t kernel, uint32_t units)
{
    loom_launch L;
    std::memset(&L, 0, sizeof(L));
    L.grid[0] = (uint32_t)gx;
    L.grid[1] = (uint32_t)gy;
    L.grid[2] = 1;
    L.block[0] = block;
    L.block[1] = L.block[2] = 1;
    L.cluster[0] = L.cluster[1] = L.cluster[2] = 1;
    L.subgroup_size = 32;
    L.kernel = kernel;
    L.units_per_cta = units;
    return L;
}

// `sms` 0: the current device's.
// `aligned`: both matrices start on 16 bytes (the tensor cores' copies need that).
loom_status matmul_geometry(int64_t tokens, int64_t n, int64_t k, bool aligned, int64_t path, int64_t sms, loom_launch *out,
                            MatmulTcPlan *plan)
{
    if (tokens < 0 || tokens > MAX_INT || n < 0 || n > MAX_INT || k < 0 || k > MAX_K || k % 4)
        return LOOM_ERR_SHAPE;
    if (path < 0 || path > LOOM_PATH_TENSOR || path == LOOM_PATH_STAGED || sms < 0)
        return LOOM_ERR_ARG;
    if (sms == 0) {
        const loom_status st = sm_count(&sms);
        if (st != LOOM_OK)
            return st;
    }
    if (path == LOOM_PATH_TENSOR && !aligned)
        return LOOM_ERR_ALIGN;
    // Measured (us, dp4a / tensor cores)    1024 x 1024   4096 x 4096   32768 x 2048   8192 x 16384
    //   4 tokens                             2.6 / 7.9     4.9 / 10.5   11.7 / 18.0    25.6 / 31.6
    //   8                                    3.1 / 8.0     7.6 / 10.6   21.9 / 18.0    43.2 / 31.4
    //   16                                   4.9 / 8.0    13.3 / 10.4   39.9 / 17.9    83.6 / 31.8
    //   24, 32                 6.8 / 8.0 and 8.5 / 8.0 (256 x 256: 6.0 / 6.5 and 7.5 / 6.3)
    // A pass of dp4a takes about twice what the weights take the tensor cores, which take 5 us
    // more to begin and end.
    const int64_t passes = (tokens + MM_DP4A_PASS - 1) / MM_DP4A_PASS;
    const bool many = tokens > 4 && (tokens > MM_DP4A_MOST || (2 * passes - 1) * n * k > (36ll << 20));
    const bool tensor = path == LOOM_PATH_TENSOR || (path == LOOM_PATH_AUTO && aligned && many);
    if (tensor && k > 0 && n > 0 && tokens > 0 && matmul_tc_plan(tokens, n, k, k % 16 == 0, sms, plan)) {
        *out = plain_launch(plan->grid, 1, (uint32_t)matmul_tc_threads(*plan), LOOM_KERNEL_I8_MATMUL_TENSOR, 128u);
        out->cluster[0] = (uint32_t)(plan->cg * plan->split);
        out->smem_bytes = plan->smem_bytes;
        return LOOM_OK;
    }
    if (path == LOOM_PATH_TENSOR && k > 0 && n > 0 && tokens > 0)
        return LOOM_ERR_ARG;
    const int64_t slots = sms * MM_DP4A_CTAS_PER_SM;
    int64_t per = (n + slots - 1) / slots;
    per = per < 1 ? 1 : per > MM_MAX_ROWS_PER_CTA ? MM_MAX_ROWS_PER_CTA : per;
    *out = plain_launch((n + per - 1) / per, passes < 65535 ? passes : 65535, 256, LOOM_KERNEL_I8_MATMUL_DP4A, (uint32_t)per);
    out->smem_bytes = (uint32_t)(per * matmul_dp4a_tokens(tokens) * 4);
    return LOOM_OK;
}

loom_status rows_shape(int64_t rows, int64_t width)
{
    return rows < 0 || rows > MAX_INT || width < 0 || width > MAX_INT ? LOOM_ERR_SHAPE : LOOM_OK;
}

loom_status bytes_shape(int64_t rows, int64_t k)
{
    return rows < 0 || rows > MAX_INT || k < 0 || k > MAX_K || k % 4 ? LOOM_ERR_SHAPE : LOOM_OK;
}

bool short_stride(int64_t rows, int64_t stride, int64_t width) { return rows > 1 && stride < width; }

// f32 parameters are read 16 bytes at a time beside wide row accesses.
int param_vec(int vec, const void *a, const void *b) { return misaligned(a, 16) || misaligned(b, 16) ? 1 : vec; }

// Offsets of a single row do not depend on its stride.
int64_t used_stride(int64_t rows, int64_t stride) { return rows > 1 ? stride : 0; }

constexpr int64_t I4_MAX_K = 131064, I4_MAX_ROUTES = 64;

loom_status i4_shape(int64_t n, int64_t k, int64_t group)
{
    return n < 0 || n > MAX_INT || k < 0 || k > I4_MAX_K || k % 8 || group < 32 || group > MAX_INT || (group & (group - 1))
               ? LOOM_ERR_SHAPE : LOOM_OK;
}

// Pairs of one launch: of the experts' products (routes > 0) whole tokens, as many as the kernel's lists hold; else tokens,
// as many as leave its sums of 32 bits room.
int64_t i4_part(int64_t pairs, int64_t routes)
{
    const int64_t most = routes > 0 ? I4_MAX_PAIRS / routes * routes : (int64_t)1 << 24;
    return pairs < most ? pairs : most;
}

loom_status i4_call(I4Params p, int64_t x_rows, int64_t y_stride, int32_t routes, cudaStream_t stream)
{
    if (i4_shape(p.n, p.k, p.group) != LOOM_OK || p.pairs < 0 || short_stride(p.pairs, y_stride, p.n))
        return LOOM_ERR_SHAPE;
    if (!known(p.scale_dtype) || !known(p.y_dtype))
        return LOOM_ERR_ARG;
    if (p.pairs == 0 || p.n == 0)
        return LOOM_OK;
    const bool data = p.experts > 0 && p.k > 0;         // (without experts every route is missing)
    if (!p.y || (p.experts > 0 && !p.scale_x) || (data && (!p.w || !p.scale_w || !p.x)) || (routes > 0 && !p.ids))
        return LOOM_ERR_NULL;
    if (misaligned(p.w, 4) || misaligned(p.x, 4) || misaligned(p.scale_w, dtype_bytes(p.scale_dtype)) || misaligned(p.scale_x, 4) ||
        misaligned(p.bias, 4) || misaligned(p.ids, 4) || misaligned(p.error, 4) || misaligned(p.y, dtype_bytes(p.y_dtype)))
        return LOOM_ERR_ALIGN;
    int64_t sms = 0;
    const loom_status counted = sm_count(&sms);
    if (counted != LOOM_OK)
        return counted;
    p.y_stride = used_stride(p.pairs, y_stride);
    p.groups = (p.k + p.group - 1) / p.group;
    const int64_t pairs = p.pairs, part = i4_part(pairs, routes);
    p.pairs_per_x = x_rows == pairs ? 1 : routes;
    const I4Params whole = p;
    for (int64_t at = 0; at < pairs; at += part) {
        p.pairs = (int32_t)(pairs - at < part ? pairs - at : part);
        p.ids = routes > 0 ? whole.ids + at : nullptr;
        p.x = whole.x + at / p.pairs_per_x * p.k;
        p.scale_x = whole.scale_x + at / p.pairs_per_x;
        p.y = static_cast<char *>(whole.y) + at * p.y_stride * dtype_bytes(p.y_dtype);
        loom_launch L;
        i4_geometry(p.pairs, p.n, p.k, p.group, routes > 0 ? (p.experts > 0 ? p.experts : 1) : 0, sms, &L);
        const cudaError_t e = launch_i4_matvec(p, sms, L, stream);
        if (e != cudaSuccess)
            return LOOM_ERR_CUDA;
    }
    return LOOM_OK;
}

loom_status to_bytes(const void *d_x, int32_t dtype, int64_t rows, int32_t width, int64_t x_stride, const float *gain,
                     const float *bias, float eps, RowMode mode, int32_t *q, float *scale, int32_t *error, void *stream)
{
    loom_status st = bytes_shape(rows, width);
    if (st != LOOM_OK || short_stride(rows, x_stride, width))
        return LOOM_ERR_SHAPE;
    if (!known(dtype) || !(eps >= 0.0f))
        return LOOM_ERR_ARG;
    if (rows == 0)
        return LOOM_OK;
    if (!scale || (width > 0 && (!d_x || !q)))
        return LOOM_ERR_NULL;
    if (misaligned(d_x, dtype_bytes(dtype)) || misaligned(q, 4) || misaligned(scale, 4) || misaligned(gain, 4) ||
        misaligned(bias, 4) || misaligned(error, 4))
        return LOOM_ERR_ALIGN;
    int64_t sms = 0;
    const loom_status counted = sm_count(&sms);
    if (counted != LOOM_OK)
        return counted;
    loom_launch L;
    if (!rows_geometry(rows, width, dtype, sms, &L))
        return LOOM_ERR_SHAPE;
    RowsParams p = {};
    p.x = d_x;
    p.rows = rows;
    p.x_stride = used_stride(rows, x_stride);
    p.width = width;
    p.eps = eps;
    p.gain = gain;
    p.bias = bias;
    p.q = reinterpret_cast<int8_t *>(q);
    p.scale = scale;
    p.error = error;
    p.inject_stall = test_stall();
    const void *ptrs[] = {d_x};
    const int64_t strides[] = {p.x_stride};
    // the bytes of a row start 4-byte aligned (width % 4 == 0): packs of at most 4 unless 8 divides the row
    int vec = row_vec(dtype, width, ptrs, strides, 1);
    if (vec == 8 && misaligned(q, 8))
        vec = 4;
    vec = param_vec(vec, gain, bias);
    return of_cuda(launch_rows(p, mode, dtype, vec, L, static_cast<cudaStream_t>(stream)));
}

}  // namespace
}  // namespace loom

using namespace loom;

extern "C" loom_status loom_token_launch_config(int32_t op, const int64_t *w, int32_t n, loom_launch *out)
{
    if (!w || !out)
        return LOOM_ERR_NULL;
    const auto opt = [&](int i, int64_t dflt) { return i < n ? w[i] : dflt; };
    switch (op) {
    case LOOM_OP_QUANTIZE_TOKENS:
    case LOOM_OP_LAYER_NORM: {
        if (n < 3 || !known((int32_t)w[2]))
            return LOOM_ERR_ARG;
        const loom_status st = op == LOOM_OP_LAYER_NORM ? rows_shape(w[0], w[1]) : bytes_shape(w[0], w[1]);
        if (st != LOOM_OK)
            return st;
        int64_t sms = opt(4, 0);
        if (sms < 0)
            return LOOM_ERR_ARG;
        const loom_status known_sms = sms ? LOOM_OK : sm_count(&sms);
        if (known_sms != LOOM_OK)
            return known_sms;
        return rows_geometry(w[0], (int32_t)w[1], (int32_t)w[2], sms, out) ? LOOM_OK : LOOM_ERR_SHAPE;
    }
    case LOOM_OP_I8_MATMUL:
        if (n < 3)
            return LOOM_ERR_ARG;
    {
        MatmulTcPlan plan;
        return matmul_geometry(w[0], w[1], w[2], opt(3, 1) != 0, opt(4, LOOM_PATH_AUTO), opt(5, 0), out, &plan);
    }
    case LOOM_OP_LAYER_NORM_BACKWARD: {
        if (n < 3 || !known((int32_t)w[2]) || opt(4, 0) < 0)
            return LOOM_ERR_ARG;
        loom_status st = rows_shape(w[0], w[1]);
        int64_t sms = opt(4, 0);
        if (st == LOOM_OK && sms == 0)
            st = sm_count(&sms);
        if (st != LOOM_OK)
            return st;
        norm_grad_geometry(w[0], (int32_t)w[1], (int32_t)w[2], sms, out);
        return LOOM_OK;
    }
    case LOOM_OP_SAMPLE_TOKENS: {
        if (n < 3 || !known((int32_t)w[2]) || opt(3, 0) < 0)
            return LOOM_ERR_ARG;
        if (w[0] < 0 || w[0] > MAX_INT || w[1] < 1 || w[1] > MAX_INT)
            return LOOM_ERR_SHAPE;
        if (!sample_geometry(w[0], (int32_t)w[1], 1, out))
            return LOOM_ERR_SHAPE;
        int64_t sms = opt(3, 0);
        const loom_status counted = sms ? LOOM_OK : sm_count(&sms);
        if (counted != LOOM_OK)
            return counted;
        return sample_geometry(w[0], (int32_t)w[1], sms, out) ? LOOM_OK : LOOM_ERR_SHAPE;
    }
    case LOOM_OP_I4_MATVEC: {
        if (n < 4 || opt(6, 0) < 0)
            return LOOM_ERR_ARG;
        const int64_t experts = opt(4, 0), routes = opt(5, 1);
        if (w[0] < 0 || w[0] > MAX_INT || i4_shape(w[1], w[2], w[3]) != LOOM_OK || experts < 0 || experts > I4_MAX_EXPERTS ||
            routes < 0 || routes > I4_MAX_ROUTES || w[0] * routes > MAX_INT)
            return LOOM_ERR_SHAPE;
        int64_t sms = opt(6, 0);
        const loom_status counted = sms ? LOOM_OK : sm_count(&sms);
        if (counted != LOOM_OK)
            return counted;
        i4_geometry(experts ? i4_part(w[0] * routes, routes) : i4_part(w[0], 0), w[1], w[2], w[3], experts, sms, out);
        return LOOM_OK;
    }
    case LOOM_OP_ROUTE_TOKENS:
    case LOOM_OP_ROUTE_TOKENS_BACKWARD: {
        if (n < 2 || opt(2, 0) < 0)
            return LOOM_ERR_ARG;
        if (w[0] < 0 || w[0] > MAX_INT || w[1] < 1 || w[1] > ROUTE_MAX_EXPERTS)
            return LOOM_ERR_SHAPE;
        int64_t sms = opt(2, 0);
        const loom_status counted = sms ? LOOM_OK : sm_count(&sms);
        if (counted != LOOM_OK)
            return counted;
        return route_geometry(w[0], (int32_t)w[1], op == LOOM_OP_ROUTE_TOKENS_BACKWARD, sms, out) ? LOOM_OK : LOOM_ERR_SHAPE;
    }
    case LOOM_OP_ADJUST_LOGITS: {
        const int64_t dtype = opt(4, LOOM_F32), access = opt(5, AL_ALIGNED);
        if (n < 2 || opt(3, 0) < 0 || dtype < 0 || dtype > LOOM_BF16 || access < AL_APART || access > AL_ALIGNED)
            return LOOM_ERR_ARG;
        if (w[0] < 0 || w[0] > MAX_INT || w[1] < 1 || w[1] > AL_MAX_VOCAB)
            return LOOM_ERR_SHAPE;
        int64_t sms = opt(3, 0);
        const loom_status counted = sms ? LOOM_OK : sm_count(&sms);
        if (counted != LOOM_OK)
            return counted;
        return adjust_geometry(w[0], (int32_t)w[1], opt(2, 1) != 0, dtype_bytes((int32_t)dtype), (int)access, sms, out) ? LOOM_OK : LOOM_ERR_SHAPE;
    }
    default: return LOOM_ERR_ARG;
    }
}

extern "C" loom_status loom_quantize_tokens(const void *d_x, int32_t dtype, int64_t tokens, int32_t k, int64_t x_stride,
                                            int32_t *d_q_packed, float *d_scale, int32_t *d_error, void *stream)
{
    return to_bytes(d_x, dtype, tokens, k, x_stride, nullptr, nullptr, 0.0f, RowMode::Quantize, d_q_packed, d_scale,
                    d_error, stream);
}

extern "C" loom_status loom_layer_norm_i8(const void *d_x, int32_t dtype, int64_t rows, int32_t width, int64_t x_stride,
                                          const float *d_gain, const float *d_bias, float eps, int32_t *d_q_packed,
                                          float *d_scale, int32_t *d_error, void *stream)
{
    return to_bytes(d_x, dtype, rows, width, x_stride, d_gain, d_bias, eps, RowMode::NormI8, d_q_packed, d_scale,
                    d_error, stream);
}

extern "C" loom_status loom_i8_matmul_ex(const int32_t *d_w_packed, const float *d_scale_w, int32_t n_rows, int32_t k,
                                         const int32_t *d_x_packed, const float *d_scale_x, int32_t tokens,
                                         const float *d_bias, void *d_y, int32_t y_dtype, int64_t y_stride,
                                         int32_t *d_acc, int32_t *d_error, const loom_tuning *tuning, void *stream)
{
    if (n_rows < 0 || k < 0 || k > MAX_K || k % 4 || tokens < 0 || short_stride(tokens, y_stride, n_rows))
        return LOOM_ERR_SHAPE;
    if (!known(y_dtype))
        return LOOM_ERR_ARG;
    if (tuning && (tuning->path < 0 || tuning->path > LOOM_PATH_TENSOR || tuning->path == LOOM_PATH_STAGED || tuning->wait_ns < 0))
        return LOOM_ERR_ARG;
    if (tokens == 0 || n_rows == 0)
        return LOOM_OK;
    if (!d_scale_w || !d_scale_x || !d_y || (k > 0 && (!d_w_packed || !d_x_packed)))
        return LOOM_ERR_NULL;
    if (misaligned(d_w_packed, 4) || misaligned(d_x_packed, 4) || misaligned(d_scale_w, 4) || misaligned(d_scale_x, 4) ||
        misaligned(d_bias, 4) || misaligned(d_acc, 4) || misaligned(d_error, 4) || misaligned(d_y, dtype_bytes(y_dtype)))
        return LOOM_ERR_ALIGN;
    const bool aligned = !misaligned(d_w_packed, 16) && !misaligned(d_x_packed, 16);
    loom_launch L;
    MatmulTcPlan plan;
    const loom_status st = matmul_geometry(tokens, n_rows, k, aligned, tuning ? tuning->path : LOOM_PATH_AUTO, 0, &L, &plan);
    if (st != LOOM_OK)
        return st;
    MatmulParams p = {};
    p.w = reinterpret_cast<const int8_t *>(d_w_packed);
    p.scale_w = d_scale_w;
    p.x = reinterpret_cast<const int8_t *>(d_x_packed);
    p.scale_x = d_scale_x;
    p.bias = d_bias;
    p.y = d_y;
    p.acc = d_acc;
    p.error = d_error;
    p.y_stride = used_stride(tokens, y_stride);
    p.tokens = tokens;
    p.n = n_rows;
    p.k = k;
    p.y_dtype = y_dtype;
    p.rows_per_cta = (int32_t)L.units_per_cta;
    p.wait_ns = tuning && tuning->wait_ns ? (uint64_t)tuning->wait_ns : DEFAULT_WAIT_NS;
    if (L.kernel == LOOM_KERNEL_I8_MATMUL_TENSOR)
        return of_cuda(launch_matmul_tc(p, plan, k % 16 == 0, static_cast<cudaStream_t>(stream)));
    return of_cuda(launch_matmul_dp4a(p, aligned && k % 16 == 0, L, static_cast<cudaStream_t>(stream)));
}

extern "C" loom_status loom_i8_matmul(const int32_t *d_w_packed, const float *d_scale_w, int32_t n_rows, int32_t k,
                                      const int32_t *d_x_packed, const float *d_scale_x, int32_t tokens,
                                      const float *d_bias, void *d_y, int32_t y_dtype, int64_t y_stride,
                                      int32_t *d_acc, void *stream)
{
    return loom_i8_matmul_ex(d_w_packed, d_scale_w, n_rows, k, d_x_packed, d_scale_x, tokens, d_bias, d_y, y_dtype,
                             y_stride, d_acc, nullptr, nullptr, stream);
}

extern "C" loom_status loom_layer_norm(const void *d_x, int32_t dtype, int64_t rows, int32_t width, int64_t x_stride,
                                       const float *d_gain, const float *d_bias, float eps, void *d_y, int64_t y_stride,
                                       float *d_mean, float *d_rstd, void *stream)
{
    const loom_status st = rows_shape(rows, width);
    if (st != LOOM_OK || short_stride(rows, x_stride, width) || short_stride(rows, y_stride, width))
        return LOOM_ERR_SHAPE;
    if (!known(dtype) || !(eps >= 0.0f))
        return LOOM_ERR_ARG;
    if (rows == 0 || width == 0)
        return LOOM_OK;
    if (!d_x || !d_y)
        return LOOM_ERR_NULL;
    if (misaligned(d_x, dtype_bytes(dtype)) || misaligned(d_y, dtype_bytes(dtype)) || misaligned(d_gain, 4) ||
        misaligned(d_bias, 4) || misaligned(d_mean, 4) || misaligned(d_rstd, 4))
        return LOOM_ERR_ALIGN;
    int64_t sms = 0;
    const loom_status counted = sm_count(&sms);
    if (counted != LOOM_OK)
        return counted;
    loom_launch L;
    if (!rows_geometry(rows, width, dtype, sms, &L))
        return LOOM_ERR_SHAPE;
    RowsParams p = {};
    p.x = d_x;
    p.rows = rows;
    p.x_stride = used_stride(rows, x_stride);
    p.width = width;
    p.eps = eps;
    p.gain = d_gain;
    p.bias = d_bias;
    p.y = d_y;
    p.y_stride = used_stride(rows, y_stride);
    p.mean = d_mean;
    p.rstd = d_rstd;
    p.inject_stall = test_stall();
    const void *ptrs[] = {d_x, d_y};
    const int64_t strides[] = {p.x_stride, p.y_stride};
    return of_cuda(launch_rows(p, RowMode::Norm, dtype, param_vec(row_vec(dtype, width, ptrs, strides, 2), d_gain, d_bias), L,
                               static_cast<cudaStream_t>(stream)));
}

extern "C" loom_status loom_layer_norm_backward_workspace_bytes(int64_t rows, int32_t width, int64_t *bytes)
{
    if (!bytes)
        return LOOM_ERR_NULL;
    loom_status st = rows_shape(rows, width);
    int64_t sms = 0;
    if (st == LOOM_OK)
        st = sm_count(&sms);
    if (st == LOOM_OK)
        *bytes = norm_grad_workspace_bytes(rows, width, sms);
    return st;
}

extern "C" loom_status loom_layer_norm_backward(const void *d_dy, int64_t dy_stride, const void *d_x, int64_t x_stride,
                                                int32_t dtype, int64_t rows, int32_t width, const float *d_gain,
                                                const float *d_mean, const float *d_rstd, void *d_dx, int64_t dx_stride,
                                                float *d_dgain, float *d_dbias, void *d_workspace,
                                                int64_t workspace_bytes, void *stream)
{
    if (rows_shape(rows, width) != LOOM_OK || short_stride(rows, x_stride, width) || short_stride(rows, dy_stride, width) ||
        (d_dx && short_stride(rows, dx_stride, width)))
        return LOOM_ERR_SHAPE;
    if (!known(dtype))
        return LOOM_ERR_ARG;
    const bool columns = d_dgain || d_dbias;
    if (width == 0 || (!columns && (rows == 0 || !d_dx)))
        return LOOM_OK;
    if (rows > 0 && (!d_dy || !d_x || !d_mean || !d_rstd))
        return LOOM_ERR_NULL;
    const uintptr_t size = dtype_bytes(dtype);
    if (misaligned(d_dy, size) || misaligned(d_x, size) || misaligned(d_dx, size) || misaligned(d_gain, 4) ||
        misaligned(d_mean, 4) || misaligned(d_rstd, 4) || misaligned(d_dgain, 4) || misaligned(d_dbias, 4) ||
        misaligned(d_workspace, 16))
        return LOOM_ERR_ALIGN;
    int64_t sms = 0;
    const loom_status st = sm_count(&sms);
    if (st != LOOM_OK)
        return st;
    const bool needs = rows > 0 && columns;
    if (needs && (!d_workspace || workspace_bytes < norm_grad_workspace_bytes(rows, width, sms)))
        return LOOM_ERR_ARG;
    loom_launch L;
    norm_grad_geometry(rows, width, dtype, sms, &L);
    const int64_t parts = norm_grad_parts(rows, width, sms);
    NormGradParams p = {};
    p.dy = d_dy;
    p.x = d_x;
    p.dy_stride = used_stride(rows, dy_stride);
    p.x_stride = used_stride(rows, x_stride);
    p.dx_stride = used_stride(rows, dx_stride);
    p.rows = rows;
    p.width = width;
    p.gain = d_gain;
    p.mean = d_mean;
    p.rstd = d_rstd;
    p.dx = d_dx;
    p.dgain = d_dgain;
    p.dbias = d_dbias;
    p.inject_stall = test_stall();
    if (needs) {
        p.partial = static_cast<float *>(d_workspace);
        p.row_sums = p.partial + parts * 2 * width;
    }
    const void *ptrs[] = {d_dy, d_x, d_dx ? d_dx : d_x};
    const int64_t strides[] = {p.dy_stride, p.x_stride, d_dx ? p.dx_stride : p.x_stride};
    return of_cuda(launch_norm_grad(p, dtype, param_vec(row_vec(dtype, width, ptrs, strides, 3), d_gain, nullptr), L, parts,
                                    static_cast<cudaStream_t>(stream)));
}

extern "C" loom_status loom_sample_tokens(const void *d_logits, int32_t dtype, int64_t rows, int32_t vocab, int64_t stride,
                                          const float *d_temperature, float temperature, const int32_t *d_top_k,
                                          int32_t top_k, const float *d_top_p, float top_p, const float *d_min_p,
                                          float min_p, const float *d_uniform, int32_t *d_token, float *d_logprob,
                                          int32_t *d_error, void *stream)
{
    loom_launch L;
    if (rows < 0 || rows > MAX_INT || vocab < 1 || short_stride(rows, stride, vocab) ||
        !sample_geometry(rows, vocab, 1, &L))
        return LOOM_ERR_SHAPE;
    if (!known(dtype) || (!d_temperature && !(temperature >= 0.0f)) || (!d_top_p && !(top_p >= 0.0f)) ||
        (!d_min_p && !(min_p >= 0.0f)))
        return LOOM_ERR_ARG;
    if (rows == 0)
        return LOOM_OK;
    if (!d_logits || !d_uniform || !d_token)
        return LOOM_ERR_NULL;
    if (misaligned(d_logits, dtype_bytes(dtype)) || misaligned(d_temperature, 4) || misaligned(d_top_k, 4) ||
        misaligned(d_top_p, 4) || misaligned(d_min_p, 4) || misaligned(d_uniform, 4) || misaligned(d_token, 4) ||
        misaligned(d_logprob, 4) || misaligned(d_error, 4))
        return LOOM_ERR_ALIGN;
    int64_t sms = 0;
    const loom_status counted = sm_count(&sms);
    if (counted != LOOM_OK)
        return counted;
    sample_geometry(rows, vocab, sms, &L);
    SampleParams p = {};
    p.logits = d_logits;
    p.rows = rows;
    p.stride = used_stride(rows, stride);
    p.vocab = vocab;
    p.d_temperature = d_temperature;
    p.d_top_k = d_top_k;
    p.d_top_p = d_top_p;
    p.d_min_p = d_min_p;
    p.temperature = temperature;
    p.top_p = top_p;
    p.min_p = min_p;
    p.top_k = top_k;
    p.uniform = d_uniform;
    p.token = d_token;
    p.logprob = d_logprob;
    p.error = d_error;
    return of_cuda(launch_sample(p, dtype, L, static_cast<cudaStream_t>(stream)));
}

extern "C" loom_status loom_i4_matvec(const int32_t *d_w_packed, const void *d_scale_w, int32_t scale_dtype, int32_t n_rows,
                                      int32_t k, int32_t group, const int32_t *d_x_packed, const float *d_scale_x,
                                      int32_t tokens, const float *d_bias, void *d_y, int32_t y_dtype, int64_t y_stride,
                                      void *stream)
{
    I4Params p = {};
    p.w = d_w_packed;
    p.scale_w = d_scale_w;
    p.scale_dtype = scale_dtype;
    p.x = reinterpret_cast<const int8_t *>(d_x_packed);
    p.scale_x = d_scale_x;
    p.bias = d_bias;
    p.y = d_y;
    p.y_dtype = y_dtype;
    p.pairs = tokens;
    p.experts = 1;
    p.n = n_rows;
    p.k = k;
    p.group = group;
    return i4_call(p, tokens, y_stride, 0, static_cast<cudaStream_t>(stream));
}

extern "C" loom_status loom_i4_matvec_routed(const int32_t *d_w_packed, const void *d_scale_w, int32_t scale_dtype,
                                             int32_t experts, int32_t n_rows, int32_t k, int32_t group,
                                             const int32_t *d_x_packed, const float *d_scale_x, int64_t x_rows,
                                             const int32_t *d_ids, int32_t tokens, int32_t routes, const float *d_bias,
                                             void *d_y, int32_t y_dtype, int64_t y_stride, int32_t *d_error, void *stream)
{
    if (tokens < 0 || experts < 0 || experts > I4_MAX_EXPERTS || routes < 0 || routes > I4_MAX_ROUTES ||
        (int64_t)tokens * routes > MAX_INT || (x_rows != tokens && x_rows != (int64_t)tokens * routes))
        return LOOM_ERR_SHAPE;
    I4Params p = {};
    p.w = d_w_packed;
    p.scale_w = d_scale_w;
    p.scale_dtype = scale_dtype;
    p.x = reinterpret_cast<const int8_t *>(d_x_packed);
    p.scale_x = d_scale_x;
    p.bias = d_bias;
    p.ids = d_ids;
    p.y = d_y;
    p.y_dtype = y_dtype;
    p.error = d_error;
    p.pairs = tokens * routes;
    p.experts = experts;
    p.n = n_rows;
    p.k = k;
    p.group = group;
    return i4_call(p, x_rows, y_stride, routes, static_cast<cudaStream_t>(stream));
}

extern "C" loom_status loom_route_tokens(const void *d_logits, int32_t dtype, int64_t tokens, int32_t experts,
                                         int64_t stride, const float *d_bias, int32_t score, int32_t groups,
                                         int32_t top_groups, int32_t group_best, int32_t top_k, int32_t renormalise,
                                         float factor, int32_t *d_ids, float *d_weights, int32_t *d_counts, void *stream)
{
    if (tokens < 0 || tokens > MAX_INT || experts < 1 || experts > ROUTE_MAX_EXPERTS || top_k < 1 || top_k > ROUTE_MAX_TOP ||
        top_k > experts || groups < 1 || experts % groups || top_groups < 1 || top_groups > groups ||
        short_stride(tokens, stride, experts))
        return LOOM_ERR_SHAPE;
    if (!known(dtype) || (score != LOOM_SCORE_SOFTMAX && score != LOOM_SCORE_SIGMOID) || (group_best != 1 && group_best != 2) ||
        !std::isfinite(factor))
        return LOOM_ERR_ARG;
    if (tokens == 0)
        return LOOM_OK;
    if (!d_logits || !d_ids || !d_weights)
        return LOOM_ERR_NULL;
    if (misaligned(d_logits, dtype_bytes(dtype)) || misaligned(d_bias, 4) || misaligned(d_ids, 4) || misaligned(d_weights, 4) ||
        misaligned(d_counts, 4))
        return LOOM_ERR_ALIGN;
    int64_t sms = 0;
    const loom_status counted = sm_count(&sms);
    if (counted != LOOM_OK)
        return counted;
    loom_launch L;
    if (!route_geometry(tokens, experts, false, sms, &L))
        return LOOM_ERR_SHAPE;
    RouteParams p = {};
    p.logits = d_logits;
    p.tokens = tokens;
    p.stride = used_stride(tokens, stride);
    p.experts = experts;
    p.score = score;
    p.groups = top_groups < groups ? groups : 1;        // (all groups: none is left out)
    p.top_groups = top_groups < groups ? top_groups : 1;
    p.group_best = group_best;
    p.top_k = top_k;
    p.renormalise = renormalise != 0;
    p.factor = factor;
    p.bias = d_bias;
    p.ids = d_ids;
    p.weights = d_weights;
    p.counts = d_counts;
    return of_cuda(launch_route(p, dtype, L, static_cast<cudaStream_t>(stream)));
}

extern "C" loom_status loom_route_tokens_backward(const float *d_dweights, const void *d_logits, int32_t dtype,
                                                  int64_t tokens, int32_t experts, int64_t stride, const int32_t *d_ids,
                                                  int32_t score, int32_t top_k, int32_t renormalise, float factor,
                                                  void *d_dlogits, int64_t dlogits_stride, int32_t *d_error, void *stream)
{
    if (tokens < 0 || tokens > MAX_INT || experts < 1 || experts > ROUTE_MAX_EXPERTS || top_k < 1 || top_k > ROUTE_MAX_TOP ||
        top_k > experts || short_stride(tokens, stride, experts) || short_stride(tokens, dlogits_stride, experts) ||
        (d_logits && d_logits == d_dlogits && tokens > 1 && stride != dlogits_stride))
        return LOOM_ERR_SHAPE;
    if (!known(dtype) || (score != LOOM_SCORE_SOFTMAX && score != LOOM_SCORE_SIGMOID) || !std::isfinite(factor))
        return LOOM_ERR_ARG;
    if (tokens == 0)
        return LOOM_OK;
    if (!d_dweights || !d_logits || !d_ids || !d_dlogits)
        return LOOM_ERR_NULL;
    if (misaligned(d_dweights, 4) || misaligned(d_logits, dtype_bytes(dtype)) || misaligned(d_ids, 4) ||
        misaligned(d_dlogits, dtype_bytes(dtype)) || misaligned(d_error, 4))
        return LOOM_ERR_ALIGN;
    int64_t sms = 0;
    const loom_status counted = sm_count(&sms);
    if (counted != LOOM_OK)
        return counted;
    loom_launch L;
    if (!route_geometry(tokens, experts, true, sms, &L))
        return LOOM_ERR_SHAPE;
    RouteGradParams p = {};
    p.dweights = d_dweights;
    p.logits = d_logits;
    p.tokens = tokens;
    p.stride = used_stride(tokens, stride);
    p.dstride = used_stride(tokens, dlogits_stride);
    p.ids = d_ids;
    p.experts = experts;
    p.score = score;
    p.top_k = top_k;
    p.renormalise = renormalise != 0;
    p.factor = factor;
    p.dlogits = d_dlogits;
    p.error = d_error;
    return of_cuda(launch_route_grad(p, dtype, L, static_cast<cudaStream_t>(stream)));
}

extern "C" loom_status loom_adjust_logits(const void *d_logits, int32_t dtype, int64_t rows, int32_t vocab, int64_t stride,
                                          const int32_t *d_history, int32_t history, int64_t history_stride,
                                          const int32_t *d_lengths, const int32_t *d_prompts, const float *d_repetition,
                                          float repetition, const float *d_frequency, float frequency,
                                          const float *d_presence, float presence, const int32_t *d_bias_ids,
                                          const float *d_bias_values, int32_t biases, const int32_t *d_mask, int32_t masks,
                                          const int32_t *d_mask_rows, void *d_y, int64_t y_stride, int32_t *d_error,
                                          void *stream)
{
    if (rows < 0 || rows > MAX_INT || vocab < 1 || vocab > AL_MAX_VOCAB || short_stride(rows, stride, vocab) ||
        short_stride(rows, y_stride, vocab) || history < 0 || history > AL_MAX_HISTORY || biases < 0 || biases > AL_MAX_BIASES ||
        (d_history && short_stride(rows, history_stride, history)) || masks < 0 ||
        (d_mask && !d_mask_rows && masks < rows && masks != 1) ||
        (d_logits && d_logits == d_y && rows > 1 && stride != y_stride))
        return LOOM_ERR_SHAPE;
    if (!known(dtype) || (!d_repetition && !(repetition > 0.0f && std::isfinite(repetition))) ||
        (!d_frequency && !std::isfinite(frequency)) || (!d_presence && !std::isfinite(presence)))
        return LOOM_ERR_ARG;
    if (rows == 0)
        return LOOM_OK;
    if (!d_logits || !d_y || (biases > 0 && !d_bias_ids != !d_bias_values))
        return LOOM_ERR_NULL;
    if (misaligned(d_logits, dtype_bytes(dtype)) || misaligned(d_y, dtype_bytes(dtype)) || misaligned(d_history, 4) ||
        misaligned(d_lengths, 4) || misaligned(d_prompts, 4) || misaligned(d_repetition, 4) || misaligned(d_frequency, 4) ||
        misaligned(d_presence, 4) || misaligned(d_bias_ids, 4) || misaligned(d_bias_values, 4) || misaligned(d_mask, 4) ||
        misaligned(d_mask_rows, 4) || misaligned(d_error, 4))
        return LOOM_ERR_ALIGN;
    int64_t sms = 0;
    const loom_status counted = sm_count(&sms);
    if (counted != LOOM_OK)
        return counted;
    AdjustParams p = {};
    p.logits = d_logits;
    p.rows = rows;
    p.stride = used_stride(rows, stride);
    p.y_stride = used_stride(rows, y_stride);
    p.history_stride = used_stride(rows, history_stride);
    p.vocab = vocab;
    p.tokens = history > 0 ? d_history : nullptr;
    p.history = p.tokens ? history : 0;
    p.lengths = d_lengths;
    p.prompts = d_prompts;
    p.d_repetition = d_repetition;
    p.d_frequency = d_frequency;
    p.d_presence = d_presence;
    p.repetition = repetition;
    p.frequency = frequency;
    p.presence = presence;
    p.bias_ids = biases > 0 ? d_bias_ids : nullptr;
    p.bias_values = d_bias_values;
    p.biases = p.bias_ids ? biases : 0;
    p.mask = masks > 0 ? d_mask : nullptr;
    p.mask_rows = d_mask_rows;
    p.masks = masks;
    p.y = d_y;
    p.error = d_error;
    loom_launch L;
    const int bytes = dtype_bytes(dtype);
    if (!adjust_geometry(rows, vocab, p.tokens || p.bias_ids, bytes, adjust_access(p, bytes), sms, &L))
        return LOOM_ERR_SHAPE;
    return of_cuda(launch_adjust(p, dtype, L, static_cast<cudaStream_t>(stream)));
}
