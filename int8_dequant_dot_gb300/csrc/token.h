// token.h -- parameters and launchers shared between the host layer of the
// token operators (token_api.cu) and their kernels.  Not part of the ABI.
#pragma once

#include <cstdint>
#include <cuda_runtime.h>

#include "../../include/loom_token.h"
#include "internal.h"

namespace loom {

inline int64_t dtype_bytes(int32_t dtype) { return dtype == LOOM_F32 ? 4 : 2; }

// ---- 8-bit matrix product (i8_matmul.cu: dp4a) -----------------------------------
constexpr int MM_DP4A_PASS = 8;       // tokens per pass of the dp4a kernel
constexpr int MM_DP4A_MOST = 24;      // tokens that it takes by itself, of aligned matrices
constexpr int MM_DP4A_CTAS_PER_SM = 2;
// tokens that a dp4a kernel is built for, one pass taking up to as many
inline int matmul_dp4a_tokens(int64_t tokens) { return tokens <= 1 ? 1 : tokens <= 2 ? 2 : tokens <= 4 ? 4 : MM_DP4A_PASS; }

struct MatmulParams {
    const int8_t *w;          // [n][k]
    const float *scale_w;
    const int8_t *x;          // [tokens][k]
    const float *scale_x;
    const float *bias;        // [n] or NULL
    void *y;                  // [tokens][n], rows y_stride elements apart
    int32_t *acc;             // [tokens][n] or NULL
    int32_t *error;
    int64_t y_stride;
    int32_t tokens, n, k, y_dtype;
    int32_t rows_per_cta;     // dp4a kernel
    uint64_t wait_ns;
};
// tensor cores (i8_matmul_tc.cu)
struct MatmulTcPlan {
    int64_t grid;
    int32_t cg;               // CTAs per MMA: 1 (up to 32 tokens) or 2
    int32_t halves;           // 1, or 2 for tiles of more than 128 tokens
    int32_t tile_t;           // tokens per tile, up to 256: a multiple of 32 per half
    int32_t split;            // shares of k, one per CTA (pair) of a cluster
    int32_t tiles_m, tiles_t; // tiles of channels (128 cg each) and of tokens
    int32_t ahead;            // stages of bytes in the copy ring
    uint32_t stage_bytes, ahead_bytes, smem_bytes;
};
int matmul_tc_threads(const MatmulTcPlan &q);
// false: more tokens than one CTA takes on fewer than two SMs
bool matmul_tc_plan(int64_t tokens, int64_t n, int64_t k, bool vec16, int64_t sms, MatmulTcPlan *out);
cudaError_t launch_matmul_tc(const MatmulParams &p, const MatmulTcPlan &q, bool vec16, cudaStream_t stream);
cudaError_t launch_matmul_dp4a(const MatmulParams &p, bool vec16, const loom_launch &L, cudaStream_t stream);

// ---- rows: quantisation and layer norm (token_rows.cu) ----------------------------
enum class RowMode { Quantize = 0, Norm = 1, NormI8 = 2 };
struct RowsParams {
    const void *x;
    int64_t rows, x_stride;
    int32_t width;
    float eps;
    const float *gain, *bias;   // or NULL
    void *y;                    // Norm: rows y_stride apart
    int64_t y_stride;
    float *mean, *rstd;         // Norm: or NULL
    int8_t *q;                  // Quantize, NormI8: [rows][width]
    float *scale;
    int32_t *error;
    int32_t inject_stall;       // test hook: no copies ahead (their waits run out)
};
// `vec` is the number of elements per load: the widest of 16 bytes, 8 bytes and one
// element that every row's start and the width allow (row_vec).
int row_vec(int32_t dtype, int32_t width, const void *const *pointers, const int64_t *strides, int n);
bool rows_geometry(int64_t rows, int32_t width, int32_t dtype, int64_t sms, loom_launch *out);
cudaError_t launch_rows(const RowsParams &p, RowMode mode, int32_t dtype, int vec, const loom_launch &L,
                        cudaStream_t stream);

constexpr int NG_EPT = 8;                 // columns per thread of the backward kernel; twice that ...
constexpr int32_t NG_MAX_WIDTH = 8192;    // ... for rows that need over 256 threads; wider rows take two passes

struct NormGradParams {
    const void *dy, *x;
    int64_t dy_stride, x_stride, dx_stride, rows;
    int32_t width;
    const float *gain;          // or NULL
    const float *mean, *rstd;
    void *dx;                   // or NULL
    float *dgain, *dbias;       // or NULL
    float *partial;             // [parts][2][width] partial column sums (workspace), or NULL
    int32_t inject_stall;       // test hook: no copies ahead (their waits run out)
    float *row_sums;            // [rows][2]: rows wider than NG_MAX_WIDTH (workspace), or NULL where partial is
};
// Geometry of the first launch of a call that wants all gradients, and the number of partial sums per column.
void norm_grad_geometry(int64_t rows, int32_t width, int32_t dtype, int64_t sms, loom_launch *out);
int64_t norm_grad_parts(int64_t rows, int32_t width, int64_t sms);
int64_t norm_grad_workspace_bytes(int64_t rows, int32_t width, int64_t sms);
cudaError_t launch_norm_grad(const NormGradParams &p, int32_t dtype, int vec, const loom_launch &L, int64_t parts,
                             cudaStream_t stream);

// ---- sampling (token_sample.cu) -----------------------------------------------------
struct SampleParams {
    const void *logits;
    int64_t rows, stride;
    int32_t vocab;
    const float *d_temperature;
    const int32_t *d_top_k;
    const float *d_top_p, *d_min_p;   // per row, or NULL for the values below
    float temperature, top_p, min_p;
    int32_t top_k;
    const float *uniform;
    int32_t *token;
    float *logprob;
    int32_t *error;
};
bool sample_geometry(int64_t rows, int32_t vocab, int64_t sms, loom_launch *out);
cudaError_t launch_sample(const SampleParams &p, int32_t dtype, const loom_launch &L, cudaStream_t stream);

}  // namespace loom
