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
 *     and min-p, from given random numbers, and in front of it penalties for
 *     repeated tokens, biases and grammar masks on the logits (loom_adjust_logits);
 *  4. products of a few 8-bit tokens with 4-bit weights that have a scale for each
 *     group along k (loom_i4_matvec), also with the matrices of the experts that each
 *     token goes to (loom_i4_matvec_routed), and the routing that names those experts
 *     and their weights, as loom_routed_combine takes them (loom_route_tokens, with
 *     the gradient loom_route_tokens_backward).
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
#define LOOM_OP_I4_MATVEC 13           /* workload {tokens, n, k, group, experts (0: one matrix, default), routes
                                          (default 1), sm_count (0 = the current device)}: the first launch */
#define LOOM_OP_ROUTE_TOKENS 14        /* workload {tokens, experts, sm_count (0 = the current device)}; the shared memory is
                                          that of a call with a bias or groups, and counts (others take less) */
#define LOOM_OP_ROUTE_TOKENS_BACKWARD 15 /* the same */
#define LOOM_OP_ADJUST_LOGITS 16       /* workload {rows, vocab, marks (0/1: penalties or biases, default 1), sm_count
                                          (0 = the current device), dtype (default f32), access (2, default: the rows of
                                          logits and y start on 16 bytes; 1: they start alike, elsewhere; 0: not alike)} */

/* Kernels they select (loom_launch.kernel). */
#define LOOM_KERNEL_I8_MATMUL_DP4A 18   /* few tokens: dp4a, weights streamed once per pass of up to 8 tokens */
#define LOOM_KERNEL_I8_MATMUL_TENSOR 19 /* tcgen05 MMA on exact f16 copies; units_per_cta = channels */
#define LOOM_KERNEL_NORM_ROWS 20        /* a CTA (or warp) holds a row in registers; CTAs walk over the rows */
#define LOOM_KERNEL_NORM_LONG 21        /* rows longer than the registers of a CTA, read again from L2 */
#define LOOM_KERNEL_NORM_BACKWARD 22    /* CTAs over shares of the rows, column sums in registers */
#define LOOM_KERNEL_SAMPLE 24           /* logits to token */
#define LOOM_KERNEL_I4_MATVEC 25        /* units_per_cta = rows of weights (of experts: where all are wanted) */
#define LOOM_KERNEL_ROUTE 26            /* logits to experts; units_per_cta = tokens */
#define LOOM_KERNEL_ROUTE_BACKWARD 27   /* units_per_cta = tokens */
#define LOOM_KERNEL_ADJUST 28           /* slices of rows; units_per_cta = tokens of a slice */

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

/*
 * Logits adjusted before a token is chosen: penalties for tokens that were seen, biases,
 * a grammar's mask.  For row r, token i and logit l, each step one f32 rounding, in this order:
 *   seen     (i is among the first lengths[r] tokens of the row's history):
 *            l = l > 0 ? l / repetition : l * repetition
 *   counted  c > 0 times at places [prompts[r], lengths[r]) of it:
 *            l = l - frequency * c (product and difference rounded), then l = l - presence
 *   biased   l = l + value, of the first of the row's bias entries that names i
 *   masked   l = -infinity where the row's mask has bit i clear (whatever l was, NaN too)
 * and one rounding to `dtype`, the type of logits and y.  Logits that no step changes keep their bits.
 * d_history: int32 [rows][history], rows history_stride elements apart, or NULL (nothing was
 * seen); tokens outside [0, vocab) are passed over.  d_lengths: int32 [rows], or NULL (all
 * `history` tokens); a length outside [0, history] is cut and flagged (LOOM_DEVERR_COUNT_RANGE; where there is no history, NULL
 * or of 0 tokens, lengths and prompts are not looked at).
 * d_prompts: int32 [rows], or NULL (0); outside [0, length] it is cut.  Penalties are one device value per row, or,
 * where that is NULL, the host value for every row; a device repetition that is not above zero counts as 1.
 * d_bias_ids int32 and d_bias_values f32 [rows][biases], or NULL; ids outside [0, vocab)
 * (such as the -1 behind a shorter list) are passed over.
 * d_mask: int32 [masks][ceil(vocab / 32)], token i is bit i % 32 of word i / 32, or NULL (as with masks 0: none).
 * d_mask_rows: int32 [rows], the mask of each row, negative for none; `masks` or more counts as none and is
 * flagged.  NULL: row r has mask r, or, where masks is 1, all rows have that one.
 * d_y may be d_logits (rows, type and stride alike); then only what changes is read and written,
 * and a mask's words.
 * Errors: NULL logits or y, one of the bias arrays alone -> LOOM_ERR_NULL; misaligned -> LOOM_ERR_ALIGN;
 * rows < 0 or > 2^31 - 1, vocab < 1 or > 393216, history < 0 or > 1048575, biases < 0 or > 1024,
 * masks < 0, masks < rows without d_mask_rows (and not 1), a stride below its row, or d_y that is d_logits with
 * another stride (with more than one row) -> LOOM_ERR_SHAPE; unknown dtype, a host repetition not above zero or infinite, a host
 * frequency or presence that is not finite -> LOOM_ERR_ARG.
 */
loom_status loom_adjust_logits(const void *d_logits, int32_t dtype, int64_t rows, int32_t vocab, int64_t stride,
                               const int32_t *d_history, int32_t history, int64_t history_stride,
                               const int32_t *d_lengths, const int32_t *d_prompts, const float *d_repetition,
                               float repetition, const float *d_frequency, float frequency, const float *d_presence,
                               float presence, const int32_t *d_bias_ids, const float *d_bias_values, int32_t biases,
                               const int32_t *d_mask, int32_t masks, const int32_t *d_mask_rows, void *d_y,
                               int64_t y_stride, int32_t *d_error, void *stream);

/*
 * Product of a few 8-bit tokens with 4-bit weights that have a scale for each group of `group`
 * neighbours along k (the last group of a row may be shorter):
 *   a[t][r][g] = sum over k in group g of W[r][k] * X[t][k]                       (exact)
 *   y[t][r]    = d_scale_x[t] * sum over g of scale_w[r][g] * a[t][r][g] + d_bias[r]
 * the sum over groups in f32, and one rounding to `y_dtype`.  Its order is fixed by the sizes, by the GPU's number of SMs and,
 * for one or two tokens, by whether all rows of W start on 16 bytes: the same weights elsewhere may give other last bits.
 * d_w_packed: int32 [n_rows][k/8], word j of a row holds elements 8j..8j+7, element 8j+i in
 * bits [4i, 4i+3] as a signed nibble (-8..7).  d_scale_w: [n_rows][ceil(k / group)] of type
 * scale_dtype; scales beyond 2^100 in size overflow.  d_x_packed: int32 [tokens][k/4], d_scale_x f32 [tokens], as
 * loom_quantize_tokens gives them; d_bias f32 [n_rows] or NULL; d_y [tokens][n_rows], rows
 * `y_stride` elements apart.
 * For few tokens: the weights are read once for every 32 of them.
 * Errors: NULL -> LOOM_ERR_NULL; misaligned pointers (4 bytes; scales and d_y: their elements) ->
 * LOOM_ERR_ALIGN; k % 8 != 0, k > 131064, group not a power of two of at least 32, negative
 * sizes, y_stride < n_rows (with more than one token) -> LOOM_ERR_SHAPE; unknown dtypes -> LOOM_ERR_ARG.
 */
loom_status loom_i4_matvec(const int32_t *d_w_packed, const void *d_scale_w, int32_t scale_dtype, int32_t n_rows,
                           int32_t k, int32_t group, const int32_t *d_x_packed, const float *d_scale_x, int32_t tokens,
                           const float *d_bias, void *d_y, int32_t y_dtype, int64_t y_stride, void *stream);

/*
 * The experts' products: for token t and route j, with e = d_ids[t][j] (int32 [tokens][routes]),
 *   y[t * routes + j] = loom_i4_matvec of matrix e and the pair's token,
 * where d_w_packed is [experts][n_rows][k/8], d_scale_w [experts][n_rows][ceil(k / group)] and d_bias
 * [experts][n_rows] or NULL.  x_rows is `tokens` (a token's routes share its row of X) or
 * tokens * routes (each pair has a row of X and a scale of its own, as a second layer wants).  A
 * negative id is a missing route: its row of y is zeros.  An id of `experts` or more is treated so
 * too and flagged (LOOM_DEVERR_COUNT_RANGE).  A launch takes up to 2048 pairs and goes through a matrix once for every 1, 2,
 * 8, 16 or 32 of them that name it.  The width is the same for all: the smallest that is not below one and a half times the
 * average pairs / min(pairs, experts), or 32 (with up to a fourth as many pairs as experts 1; with one expert its
 * pairs are the average).  Experts that far more pairs name than others therefore cost more passes: 64 tokens to 8
 * of 64 experts of 2048 x 4096 take 89 us, with half of the pairs on two experts 150 to 180.
 * y's rows are loom_routed_combine's payload, row t * routes + j of pair (t, j).
 * Errors: as loom_i4_matvec, and experts < 0 or > 1024, routes < 0 or > 64, tokens * routes > 2^31 - 1,
 * x_rows neither of the two -> LOOM_ERR_SHAPE.
 */
loom_status loom_i4_matvec_routed(const int32_t *d_w_packed, const void *d_scale_w, int32_t scale_dtype, int32_t experts,
                                  int32_t n_rows, int32_t k, int32_t group, const int32_t *d_x_packed,
                                  const float *d_scale_x, int64_t x_rows, const int32_t *d_ids, int32_t tokens,
                                  int32_t routes, const float *d_bias, void *d_y, int32_t y_dtype, int64_t y_stride,
                                  int32_t *d_error, void *stream);

/* Scores of loom_route_tokens. */
typedef enum loom_score { LOOM_SCORE_SOFTMAX = 0, LOOM_SCORE_SIGMOID = 1 } loom_score;

/*
 * Routing: the experts of each token and their weights, from logits [tokens][experts], rows
 * `stride` elements apart.  An expert whose logit is -infinity or NaN, or whose bias is, is never
 * chosen (and has no part in a softmax by its logit); +infinity counts as the largest finite f32.
 *   score[e]  = softmax of the token's logits, or 1 / (1 + exp(-logit))
 *   choice    by score[e] + d_bias[e] (f32 [experts], NULL: by the score): with more than one group
 *             (`groups` equal runs of experts), the top_groups groups whose group_best (1 or 2)
 *             best experts have the largest sum stay (a group with fewer counts those it has);
 *             then the top_k best experts of those, falling.  With no bias, or the same for all, experts
 *             (and groups by their best one) have the order of their logits; else sums are compared as
 *             64-bit floating point has them.  Equal ones go to the lower index.
 *   weight    = factor * score, divided by the sum of the chosen scores where `renormalise`
 * d_ids int32 and d_weights f32 [tokens][top_k]; where fewer than top_k can be chosen the rest
 * are -1 and 0, which loom_routed_combine and loom_i4_matvec_routed take as missing routes.
 * d_counts: int32 [experts] or NULL; the number of tokens that go to each expert is added to it (what a
 * bias for balance is set by).
 * Errors: NULL logits, ids or weights -> LOOM_ERR_NULL; misaligned -> LOOM_ERR_ALIGN; tokens < 0 or
 * > 2^31 - 1, experts < 1 or > 1024, top_k < 1, > 32 or > experts, groups < 1 or not a divisor
 * of experts, top_groups < 1 or > groups, stride < experts (with more than one token) -> LOOM_ERR_SHAPE;
 * unknown dtype or score, group_best neither 1 nor 2, factor not finite -> LOOM_ERR_ARG.
 */
loom_status loom_route_tokens(const void *d_logits, int32_t dtype, int64_t tokens, int32_t experts, int64_t stride,
                              const float *d_bias, int32_t score, int32_t groups, int32_t top_groups,
                              int32_t group_best, int32_t top_k, int32_t renormalise, float factor, int32_t *d_ids,
                              float *d_weights, int32_t *d_counts, void *stream);

/*
 * Gradient of those weights to the logits, the choice held fixed: d_dlogits [tokens][experts] of
 * `dtype`, rows dlogits_stride elements apart, from d_dweights f32 [tokens][top_k], the logits and
 * d_ids.  With g[j] = factor * dweight[j], chosen scores s[j] and S their sum:
 *   renormalised   h[j] = (g[j] - sum(g s) / S) / S,  else h[j] = g[j]
 *   softmax        dlogit[e] = score[e] * (sum of h[j] over ids[j] = e  -  sum(h s))
 *   sigmoid        dlogit[e] = score[e] * (1 - score[e]) * (sum of h[j] over ids[j] = e)
 * (renormalised softmax scores are taken among the chosen experts, where sum(h s) is zero).
 * Missing routes (negative ids, or ids of `experts` or more, which are flagged with
 * LOOM_DEVERR_COUNT_RANGE) take no part; an expert that can't be chosen gets 0.  d_dlogits may be d_logits (with its stride).
 * Errors: as loom_route_tokens, and d_dlogits that is d_logits with another stride (with more than one token) ->
 * LOOM_ERR_SHAPE.
 */
loom_status loom_route_tokens_backward(const float *d_dweights, const void *d_logits, int32_t dtype, int64_t tokens,
                                       int32_t experts, int64_t stride, const int32_t *d_ids, int32_t score,
                                       int32_t top_k, int32_t renormalise, float factor, void *d_dlogits,
                                       int64_t dlogits_stride, int32_t *d_error, void *stream);

#ifdef __cplusplus
}
#endif

#endif /* LOOM_TOKEN_H */
