/*
 * loom_token.h -- the token operators of libloom: what stands around the
 * packed-int8 products of a language model on GB300 (sm_103a).
 *
 *  1. tokens to signed bytes with one scale each (loom_quantize_tokens), and
 *     the matrix product of 8-bit tokens and 8-bit weights with a scale for
 *     each token and each channel (loom_i8_matmul), for one token to many;
 *  2. layer norm: forward, forward handing out 8-bit tokens, and backward with
 *     the reduction of the gain's and the bias's gradient;
 *  3. the choice of the next token from logits, with temperature, top-k, top-p
 *     and min-p, from given random numbers.
 *
 * The conventions of loom.h hold: d_ pointers are device memory of the caller,
 * nothing is allocated or kept, work is enqueued on `stream` (a cudaStream_t)
 * in stream order, empty work returns LOOM_OK, and the same inputs give the
 * same bits on every call.  Offsets are 64-bit: rows x stride may pass 2^31.
 * `d_error` (may be NULL) is the optional device error word.
 * Device waits are bounded.  The product's wait_ns (loom_i8_matmul_ex) says what one that runs
 * out does there; the row operators (2. and the quantisation) wait a second at most for the rows
 * that they copy ahead, and then read them, and all that follow, directly: same results.
 */
#ifndef LOOM_TOKEN_H
#define LOOM_TOKEN_H

#include "loom_tuning.h"

#ifdef __cplusplus
extern "C" {
#endif

/* Element types of activations, logits and outputs.  Scales, gains, biases,
 * statistics and their gradients are always f32. */
typedef enum loom_dtype { LOOM_F32 = 0, LOOM_F16 = 1, LOOM_BF16 = 2 } loom_dtype;

/* Further bits of the device error word. */
#define LOOM_DEVERR_NONFINITE 0x4 /* a token held an infinity or NaN: its scale is NaN, its bytes 0 */
#define LOOM_DEVERR_NO_TOKEN 0x8  /* a row of logits held nothing to choose: its token is -1 */

/* Operators of loom_token_launch_config. */
#define LOOM_OP_QUANTIZE_TOKENS 8      /* workload {tokens, k, dtype, aligned (0/1, default 1),
                                          sm_count (0 = the current device)} */
#define LOOM_OP_I8_MATMUL 9            /* workload {tokens, n, k, aligned (0/1, default 1), path
                                          (LOOM_PATH_*, default auto), sm_count (0 = the current device; the
                                          tensor cores want two SMs for more than 32 tokens, else
                                          LOOM_ERR_ARG where they are asked for)} */
#define LOOM_OP_LAYER_NORM 10          /* workload as LOOM_OP_QUANTIZE_TOKENS, {rows, width, ...} */
#define LOOM_OP_LAYER_NORM_BACKWARD 11 /* workload {rows, width, dtype, aligned (0/1, default 1),
                                          sm_count (0 = the current device)}: the first launch of a
                                          call that wants all gradients (beyond 8192 columns: the rows'
                                          sums, one row a CTA) */
#define LOOM_OP_SAMPLE_TOKENS 12       /* workload {rows, vocab, dtype, sm_count (0 = the current device)} */

/* Kernels they select (loom_launch.kernel). */
#define LOOM_KERNEL_I8_MATMUL_DP4A 18   /* few tokens: dp4a, weights streamed once per pass of up to 8 tokens */
#define LOOM_KERNEL_I8_MATMUL_TENSOR 19 /* tcgen05 MMA on exact f16 copies; units_per_cta = channels */
#define LOOM_KERNEL_NORM_ROWS 20        /* a CTA (or warp) holds a row in registers; CTAs walk over the rows */
#define LOOM_KERNEL_NORM_LONG 21        /* rows longer than the registers of a CTA, read again from L2 */
#define LOOM_KERNEL_NORM_BACKWARD 22    /* CTAs over shares of the rows, column sums in registers */
#define LOOM_KERNEL_SAMPLE 24           /* logits to token */

/* As loom_launch_config, for the operators of this header. */
loom_status loom_token_launch_config(int32_t op, const int64_t *workload, int32_t n_workload, loom_launch *out);

/*
 * Tokens to signed bytes.  For token t of d_x (elements of type `dtype`, rows
 * of k elements `x_stride` elements apart), with amax the largest |x[t][i]|:
 *   d_scale[t] = amax / 127
 *   q[t][i]    = rint(x[t][i] * (127 / amax))
 * where the quotients and the product are single f32 roundings and rint takes
 * ties to even, so the result is defined to the bit, |q| <= 127.  A token with
 * amax < 2^-100 (zeros among them) gives q = 0 and scale 0; one that holds an
 * infinity or NaN gives q = 0 and scale NaN, and LOOM_DEVERR_NONFINITE.
 * d_q_packed: int32 [tokens][k/4], signed bytes packed as in loom_i8_dequant_dot.
 * Errors: NULL -> LOOM_ERR_NULL; pointers not aligned to their element (d_q_packed
 * and d_scale: 4 bytes) -> LOOM_ERR_ALIGN; negative sizes, k % 4 != 0, k > 131068,
 * tokens > 2^31 - 1, x_stride < k (with more than one token) -> LOOM_ERR_SHAPE;
 * unknown dtype -> LOOM_ERR_ARG.
 */
loom_status loom_quantize_tokens(const void *d_x, int32_t dtype, int64_t tokens, int32_t k, int64_t x_stride,
                                 int32_t *d_q_packed, float *d_scale, int32_t *d_error, void *stream);

/*
 * Matrix product of 8-bit tokens and 8-bit weights:
 *   acc[t][r] = sum_k W[r][k] * X[t][k]                                  (int32, exact)
 *   y[t][r]   = (float)acc[t][r] * (d_scale_w[r] * d_scale_x[t]) + d_bias[r]
 * each step one f32 rounding, then one rounding to `y_dtype`.
 * d_w_packed: int32 [n_rows][k/4] (rows of W are the output channels);
 * d_x_packed: int32 [tokens][k/4]; d_bias: f32 [n_rows] or NULL (nothing is added);
 * d_y: [tokens][n_rows], rows `y_stride` elements apart; d_acc: int32
 * [tokens][n_rows] contiguous, or NULL.
 * loom_i8_dequant_dot takes the same operands and gives [n_rows][batch]; this
 * call gives each token's outputs together, and reads W once for many tokens.
 * Errors: NULL -> LOOM_ERR_NULL; misaligned pointers (4 bytes; d_y: its element)
 * -> LOOM_ERR_ALIGN; k % 4 != 0, k > 131068, negative sizes, y_stride < n_rows
 * (with more than one token) -> LOOM_ERR_SHAPE; unknown y_dtype -> LOOM_ERR_ARG.
 */
loom_status loom_i8_matmul(const int32_t *d_w_packed, const float *d_scale_w, int32_t n_rows, int32_t k,
                           const int32_t *d_x_packed, const float *d_scale_x, int32_t tokens, const float *d_bias,
                           void *d_y, int32_t y_dtype, int64_t y_stride, int32_t *d_acc, void *stream);

/* loom_i8_matmul with a device error word and tuning (either may be NULL).  Of
 * the tuning, `path` picks the engine (LOOM_PATH_DIRECT: dp4a; LOOM_PATH_TENSOR:
 * tensor cores, which want both matrices to start on 16 bytes, else LOOM_ERR_ALIGN (without
 * that dp4a takes any number of tokens, in eights: 512 tokens of 4096 x 4096 take 366 us for 28);
 * LOOM_PATH_STAGED -> LOOM_ERR_ARG; by default tensor cores where that holds and there are
 * more than 24 tokens, or more than 4 of enough weights to be worth their start) and
 * wait_ns limits each device wait of the tensor-core kernel: one that runs out sets
 * LOOM_DEVERR_TIMEOUT, the affected y are NaN (acc INT32_MIN), and the device stays usable.
 * The engine does not change a result. */
loom_status loom_i8_matmul_ex(const int32_t *d_w_packed, const float *d_scale_w, int32_t n_rows, int32_t k,
                              const int32_t *d_x_packed, const float *d_scale_x, int32_t tokens, const float *d_bias,
                              void *d_y, int32_t y_dtype, int64_t y_stride, int32_t *d_acc, int32_t *d_error,
                              const loom_tuning *tuning, void *stream);

/*
 * Layer norm of rows:
 *   mean = sum x / width,  rstd = 1 / sqrt(sum (x - mean)^2 / width + eps),
 *   y    = (x - mean) * rstd * gain + bias
 * in f32, y rounded once to `dtype`, the type of x and y.  The squares are taken about
 * the mean, so a row far from zero loses what its mean's rounding takes and no more.  Sums are
 * multiplied by a rounded 1 / width and the root is rsqrtf (2 units at most), which every row's
 * chain of steps would wait for longer if they were exact (5 to 20% of a call).  Rows beyond 32768
 * columns add a thread's share, one column in 1024, in one running sum.
 * d_gain, d_bias: f32 [width], NULL for 1 and 0.  d_mean, d_rstd: f32 [rows],
 * what the backward pass needs; either may be NULL.  d_y may be d_x.
 * Errors: NULL x or y -> LOOM_ERR_NULL; misaligned -> LOOM_ERR_ALIGN; negative
 * sizes, a stride below width (with more than one row), rows > 2^31 - 1 ->
 * LOOM_ERR_SHAPE; eps negative or NaN, unknown dtype -> LOOM_ERR_ARG.
 */
loom_status loom_layer_norm(const void *d_x, int32_t dtype, int64_t rows, int32_t width, int64_t x_stride,
                            const float *d_gain, const float *d_bias, float eps, void *d_y, int64_t y_stride,
                            float *d_mean, float *d_rstd, void *stream);

/*
 * Layer norm handing out 8-bit tokens: loom_quantize_tokens of the f32 rows y
 * above, which are never written.  d_q_packed int32 [rows][width/4], d_scale f32
 * [rows].  Errors as for the two, width in the place of k.
 */
loom_status loom_layer_norm_i8(const void *d_x, int32_t dtype, int64_t rows, int32_t width, int64_t x_stride,
                               const float *d_gain, const float *d_bias, float eps, int32_t *d_q_packed,
                               float *d_scale, int32_t *d_error, void *stream);

/*
 * Layer norm backward.  With xhat = (x - mean) * rstd and g = dy * gain:
 *   dx    = rstd * (g - sum(g) / width - xhat * sum(g * xhat) / width)   per row
 *   dgain = sum over rows of dy * xhat,   dbias = sum over rows of dy
 * d_mean, d_rstd: f32 [rows], as the forward pass left them.  d_dx ([rows][width]
 * of `dtype`, may be d_dy or d_x), d_dgain and d_dbias (f32 [width]) may be NULL where
 * they are not wanted; the sums over no rows are zeros.  The column sums are taken in
 * a fixed order: the same inputs give the same bits.
 * d_workspace: caller-owned device memory, 16-byte aligned, of at least the bytes
 * that loom_layer_norm_backward_workspace_bytes gives; not needed (NULL, 0) when
 * neither d_dgain nor d_dbias is wanted.  Calls that may run at the same time
 * must not share one.
 * Errors: NULL dy, x, mean or rstd -> LOOM_ERR_NULL; misaligned -> LOOM_ERR_ALIGN;
 * sizes and strides as for loom_layer_norm -> LOOM_ERR_SHAPE; a missing or short
 * workspace, unknown dtype -> LOOM_ERR_ARG; no usable device -> LOOM_ERR_CUDA.
 */
loom_status loom_layer_norm_backward(const void *d_dy, int64_t dy_stride, const void *d_x, int64_t x_stride,
                                     int32_t dtype, int64_t rows, int32_t width, const float *d_gain,
                                     const float *d_mean, const float *d_rstd, void *d_dx, int64_t dx_stride,
                                     float *d_dgain, float *d_dbias, void *d_workspace, int64_t workspace_bytes,
                                     void *stream);

/* Bytes of that workspace on the current device.  Errors: NULL -> LOOM_ERR_NULL;
 * sizes -> LOOM_ERR_SHAPE; no usable device -> LOOM_ERR_CUDA. */
loom_status loom_layer_norm_backward_workspace_bytes(int64_t rows, int32_t width, int64_t *bytes);

/*
 * The next token of each row of logits l[0..vocab), rows `stride` elements apart.
 * A logit of -infinity or NaN is never chosen.  With m the largest logit, T the
 * temperature and all steps in f32, the logits get whole-number weights
 *   w[i] = floor(exp((l[i] - m) * (1 / T)) * 2^31)          (w = 2^31 where l[i] = m)
 * T = 0 (a device value that is not above zero) is the greedy choice: w = 2^31 for
 * the first of the largest logits alone.  Then, with the tokens in order of
 * falling logit and of rising index among equals:
 *   top-k  the first top_k of them stay (top_k <= 0: all)
 *   top-p  of those, the ones whose predecessors' weights sum to less than top_p
 *          times the sum of them all, and always the first (top_p >= 1: all)
 *   min-p  of those, the ones with w >= min_p * 2^31 (min_p is cut to [0, 1])
 * With `total` the weight that stays, the token is the lowest index whose running
 * sum of kept weights, in index order, exceeds floor(u * total), where u in [0, 1)
 * is d_uniform[row] (values outside are cut); its log probability is
 * log(w / total).  Sums are whole numbers and the products by top_p, min_p and u are
 * taken in 64-bit floating point, so the choice is defined by these lines alone, in
 * whatever order the sums are taken.
 * Each setting is one device value per row (d_...) or, where that is NULL, the
 * host value for every row.
 * d_token int32 [rows]; d_logprob f32 [rows] or NULL.  A row with nothing to choose
 * gives token -1, log probability NaN and LOOM_DEVERR_NO_TOKEN.
 * Errors: NULL logits, uniform or token -> LOOM_ERR_NULL; misaligned ->
 * LOOM_ERR_ALIGN; rows < 0 or > 2^31 - 1, vocab < 1 or > 393216, stride < vocab (with
 * more than one row) -> LOOM_ERR_SHAPE; unknown dtype, a host temperature, top_p or min_p that is
 * negative or NaN -> LOOM_ERR_ARG.
 */
loom_status loom_sample_tokens(const void *d_logits, int32_t dtype, int64_t rows, int32_t vocab, int64_t stride,
                               const float *d_temperature, float temperature, const int32_t *d_top_k, int32_t top_k,
                               const float *d_top_p, float top_p, const float *d_min_p, float min_p,
                               const float *d_uniform, int32_t *d_token, float *d_logprob, int32_t *d_error,
                               void *stream);

#ifdef __cplusplus
}
#endif

#endif /* LOOM_TOKEN_H */
