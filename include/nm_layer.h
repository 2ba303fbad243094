/*
 * nm_layer.h -- C ABI of the operators between the sparse products of a decoder
 * layer and at its answer (sm_103a), next to nm_spmv.h and nm_decode.h:
 *   nm_linear          the N:M product with bias, activation (gated too), scale
 *                      and residual in its epilogue, for any number of tokens;
 *   nm_residual_norm   the residual stream's update by a block's output, with the
 *                      norm after that block and the norm before the next;
 *   nm_token_logprobs  log probabilities of given tokens, the entropy and the
 *                      likeliest tokens, from rows of logits.
 *
 * Conventions, status codes and stream behaviour are nm_spmv.h's: the caller
 * owns every buffer, nothing is allocated, calls enqueue on `stream` and
 * return; arguments are checked on the host before anything is launched, among
 * them that what a call writes meets nothing that it reads (NM_ERR_ALIAS; an array
 * counts from its first element to its last, with what lies between its rows, so
 * column blocks of one matrix meet), but for the buffers that a call says may be the
 * same.  Launches use
 * programmatic dependent launch; every kernel waits for the previous one on
 * the stream before it touches any buffer.  No call uses floating-point atomics:
 * the same inputs give the same bits.  These are inference operators: the
 * library has no backward passes.
 */
#ifndef NM_LAYER_H
#define NM_LAYER_H

#include <stddef.h>
#include <stdint.h>

#include "nm_spmv.h"

#ifdef __cplusplus
extern "C" {
#endif

/* ---------------------------------------------------------------------------
 * nm_linear -- Y = residual + scale * act(W X + bias), W in the packed format.
 *   n = rows outputs a token: Y[t][i] = residual[t][i] + scale * act(s_i), where
 *   s_i = sum_c W[i][c] X[t][c] + bias[i]; or, gated, n = rows / 2 (rows even):
 *   Y[t][i] = residual[t][i] + scale * act(s_2i) * s_2i+1, rows interleaved in
 *   (gate, up) pairs as for nm_spmv_swiglu.
 *     NM_ACT_NONE, NM_ACT_RELU, NM_ACT_SILU  t / (1 + e^-t),
 *     NM_ACT_GELU       t * (1 + erf(t / sqrt 2)) / 2,
 *     NM_ACT_GELU_TANH  t * (1 + tanh(sqrt(2 / pi) (t + 0.044715 t^3))) / 2.
 *   values, masks, X, ldx, cols : as for nm_spmm (values 32-byte, X 16-byte
 *       aligned, ldx % 8 == 0, ldx >= cols).
 *   bias     : device fp16 [rows] or NULL;  scale: finite.
 *   residual : device fp16 [tokens][ldres], ldres >= n, or NULL.  It may be Y
 *              itself (the same address and row stride): the sum is in place.
 *   Y        : device fp16 [tokens][ldy], ldy >= n.
 *   workspace: device scratch, 16-byte aligned, of at least
 *              nm_linear_workspace_bytes(rows, cols, tokens) bytes (may be NULL
 *              when that is 0); it needs no initial contents.
 * Sums, bias, activation, scale and residual are fp32, with one rounding to fp16
 * at the end.  1 token runs on nm_spmv's kernels, 2..8 on nm_spmm's, each with its
 * arithmetic, more on a tensor-core kernel of its own (fp16 products, fp32 sums; up
 * to 8 tokens pruned weights are never multiplied; beyond, a non-finite X[t][c]
 * reaches every row of its token).  The summation order is fixed for a shape and
 * device.  The workspace is needed for 1..8 tokens of rows so long that their x tile,
 * or what it leaves for the rows' sums, does not fit a block's shared memory: columns
 * are cut then.  The tensor-core kernel's bounded waits count in nm_wait_timeouts.
 * (For 2:4 matrices and 6..8 tokens nm_spmm24 is the faster product, without an
 * epilogue.)
 * rows == 0 or tokens == 0 is a no-op.  tokens < 2^31, rows < 2^31 and beyond 8
 * tokens ceil(rows / 128) <= 65535, else NM_ERR_SHAPE.
 * ------------------------------------------------------------------------- */
#define NM_ACT_NONE 0
#define NM_ACT_RELU 1
#define NM_ACT_SILU 2
#define NM_ACT_GELU 3
#define NM_ACT_GELU_TANH 4

typedef struct {
    const void *bias;     /* fp16 [rows] or NULL */
    const void *residual; /* fp16 [tokens][ldres] or NULL */
    int64_t ldres;
    int32_t activation;   /* NM_ACT_* */
    int32_t gated;        /* nonzero: rows are (gate, up) pairs */
    float scale;
} nm_epilogue;

size_t nm_linear_workspace_bytes(int64_t rows, int64_t cols, int64_t tokens);
int nm_linear(const void *values, const uint32_t *masks, int64_t rows, int64_t cols, const void *X,
              int64_t ldx, int64_t tokens, const nm_epilogue *epilogue, void *Y, int64_t ldy,
              void *workspace, size_t workspace_bytes, void *stream);

/* nm_linear_stall_selftest -- exercises the bounded waits of nm_linear's tensor-core
 * kernel (a self-test, as those of nm_decode.h): nm_linear with every wait limited to
 * wait_limit_us (1 .. 2,000,000, else NM_ERR_SHAPE), in which the weights of every other
 * block never come (a call of up to 8 tokens runs as usual: its kernels have no waits).
 * The waits run out, or give up after the first that did, are counted in
 * nm_wait_timeouts(), and the kernel returns with Y undefined; the device stays usable.
 * Until nm_wait_timeouts(1) calls of more than 8 tokens leave Y as it is.  Asynchronous;
 * NM_OK once launched. */
int nm_linear_stall_selftest(const void *values, const uint32_t *masks, int64_t rows, int64_t cols,
                             const void *X, int64_t ldx, int64_t tokens,
                             const nm_epilogue *epilogue, void *Y, int64_t ldy, void *workspace,
                             size_t workspace_bytes, int64_t wait_limit_us, void *stream);

/* ---------------------------------------------------------------------------
 * nm_residual_norm -- between two blocks of a layer:
 *     s = residual_scale * residual + scale * gate * post(block)
 *     residual_out = s,   out = pre(s)
 * where post and pre are each NM_NORM_NONE (the value itself),
 *     NM_NORM_RMS    x / sqrt(mean(x^2) + eps) * (offset + weight) + bias,
 *     NM_NORM_LAYER  (x - mean(x)) / sqrt(var(x) + eps) * (offset + weight) + bias
 * over the row (var: the mean squared deviation).
 *   residual : device fp16 (stream_fp32 == 0) or fp32 [tokens][ldr].
 *   block    : device fp16 [tokens][ldb] or NULL: s = residual_scale * residual
 *              (then post, gate and scale are not used).
 *   gate     : device fp16 [tokens][ldg], or one row for all tokens with
 *              ldg == 0; NULL: 1.
 *   weight, bias of a norm: device fp16 (params_fp32 == 0) or fp32 [width];
 *              either may be NULL (weight: 1 in place of offset + weight; bias: 0).
 *   residual_out : as residual, [tokens][lds]; it may be residual itself (the same
 *              address and row stride); NULL: not written.
 *   out      : device fp16 [tokens][ldo]; NULL: pre is not computed.
 * All arithmetic is fp32, out is computed from the unrounded s, and each output
 * is rounded once.  (Squares are fp32 too: an element beyond 2^63 has an infinite
 * one.  Where rows are many, weight, gate and scale are multiplied before the block's
 * values.)  Rows are independent: a non-finite value spoils its row alone.
 * Any strides and alignment of the elements' size; 16-byte aligned rows are
 * fastest.  tokens == 0 is a no-op; tokens < 2^31, width 1 .. 32768, row strides
 * >= width, eps >= 0 and finite; scale, residual_scale and offsets finite, else
 * NM_ERR_SHAPE.  residual_out and out both NULL -> NM_ERR_NULL.
 * ------------------------------------------------------------------------- */
#define NM_NORM_NONE 0
#define NM_NORM_RMS 1
#define NM_NORM_LAYER 2

typedef struct {
    int32_t kind;        /* NM_NORM_* */
    int32_t params_fp32; /* weight and bias are fp32, else fp16 */
    const void *weight, *bias;
    float offset, eps;
} nm_norm;

int nm_residual_norm(const void *residual, int stream_fp32, int64_t ldr, const void *block,
                     int64_t ldb, const nm_norm *post, const void *gate, int64_t ldg, float scale,
                     float residual_scale, void *residual_out, int64_t lds, const nm_norm *pre,
                     void *out, int64_t ldo, int64_t tokens, int64_t width, void *stream);

/* ---------------------------------------------------------------------------
 * nm_token_logprobs -- for every row x of logits, with p = softmax(x / temperature):
 *   logprob[row][j]     : log p at ids[row][j], j < n_ids (-infinity for an id
 *                         outside [0, vocab): no token has it);
 *   entropy[row]        : - sum p log p (0 log 0 = 0);
 *   top_ids[row][j], top_logprob[row][j], j < top: the tokens of the largest
 *                         logits in descending order, the lowest id first among
 *                         equals (-0 equals +0), and their log p.
 * A row without a finite largest logit, or with NaN, has no distribution:
 * logprob, entropy and top_logprob are NaN and top_ids -1.  A logit of -infinity
 * has probability 0; elements behind vocab are never used.
 *   logits  : device [rows][ld_logits], fp16 (logits_fp32 == 0) or fp32, any
 *             alignment of the element's size; ld_logits >= vocab.
 *   ids     : device int32 [rows][ld_ids], ld_ids >= n_ids (NULL: n_ids == 0).
 *   logprob : device fp32 [rows][n_ids];  entropy : device fp32 [rows] or NULL;
 *   top_ids : device int32 [rows][top];  top_logprob : device fp32 [rows][top].
 * Each logit is read once from memory.  Sums are fp32 relative to the row's
 * largest logit and without its own term, which is 1: log p of a token that is
 * nearly certain, and the entropy, keep fp32 accuracy relative to themselves (terms
 * below 2^-126 of the largest count as 0).
 * rows == 0 is a no-op (arrays may be NULL).  rows < 2^31, vocab 1 .. 2^24,
 * n_ids 0 .. 1024, top 0 .. 32 and <= vocab, temperature 2^-20 .. 2^20, else
 * NM_ERR_SHAPE.
 * ------------------------------------------------------------------------- */
int nm_token_logprobs(const void *logits, int logits_fp32, int64_t ld_logits, int64_t rows,
                      int64_t vocab, const int32_t *ids, int64_t ld_ids, int n_ids,
                      float temperature, float *logprob, float *entropy, int top,
                      int32_t *top_ids, float *top_logprob, void *stream);

#ifdef __cplusplus
}
#endif

#endif /* NM_LAYER_H */
