/*
 * nm_decode.h -- C ABI of the operators around the sparse products in a step
 * of speculative decoding (sm_103a), next to nm_spmv.h.
 *
 * A step takes, per sequence, a tree of up to 64 drafted tokens through the
 * decoder layers as one small batch (nm_spmm, nm_spmm24, nm_spmm_prefill).
 * Node 0 of a tree is the last committed token, whose keys and values are not
 * in the cache yet.  Between the products a layer needs
 *   nm_rope_append     rotary positions on the QKV projection's output, and
 *                      the write of its keys and values into a paged cache
 *                      (fp16, or e4m3 / int8 codes with scales);
 *   nm_tree_attention  attention of every node over its sequence's cached
 *                      context and over the nodes its tree mask shows;
 * and after the last layer
 *   nm_tree_verify     accepts or rejects the drafted tokens against the
 *                      target's probabilities from given random numbers.
 * nm_cache_read reads rows of the cache back as fp16 (a prefix handed on to
 * another process or model).
 *
 * The accepted path is committed with nm_rope_append as well: the rows of the
 * QKV output that belong to the path are appended again with their final
 * slots (their positions are the same, so the rows come out bit for bit the
 * same); q_out may be NULL then.
 *
 * Conventions, status codes and stream behaviour are nm_spmv.h's: the caller
 * owns every buffer, nothing is allocated, calls enqueue on `stream` and
 * return; arguments are checked on the host before anything is launched, among
 * them that what a call writes meets nothing that it reads (NM_ERR_ALIAS).
 * Values that lie on the device (slots, page numbers, lengths, parents) are
 * checked by the kernels: an entry out of range is treated as absent, as each
 * call says, and never read or written through.  Launches use programmatic
 * dependent launch; every kernel waits for the previous one on the stream
 * before it touches any buffer.  No call uses floating-point atomics: the
 * same inputs give the same bits.  nm_tree_attention's and nm_tree_verify's
 * kernels wait on barriers of their own with a limit: nm_wait_timeouts
 * (nm_spmv.h) counts the waits that gave up, after which outputs are undefined.
 */
#ifndef NM_DECODE_H
#define NM_DECODE_H

#include <stddef.h>
#include <stdint.h>

#include "nm_spmv.h"

#ifdef __cplusplus
extern "C" {
#endif

/* What a cache holds.  e4m3 (1 sign, 4 exponent, 3 mantissa bits, largest 448)
 * and int8 codes stand for code * scale, one fp32 scale for each row (one
 * token's head_dim values of one head), in k and in v. */
#define NM_CACHE_FP16 0
#define NM_CACHE_E4M3 1
#define NM_CACHE_INT8 2

/* A paged cache of one layer.  Element d of the row at `offset` of page p and
 * head h is at p * page_stride + (h * page_size + offset) * head_dim + d of k
 * (or v), and its scale at p * scale_page_stride + h * page_size + offset.
 * A slot is p * page_size + offset.
 *   k, v      : device, 32-byte aligned.
 *   *_scale   : device fp32, 4-byte aligned; NULL for NM_CACHE_FP16.  Scales are
 *               not negative (nm_rope_append writes none that is).
 *   page_size : a power of two, 8 .. 2^20;  head_dim : 64 or 128;
 *   pages >= 1, kv_heads 1 .. 1024;
 *   page_stride >= kv_heads * page_size * head_dim elements, a multiple of
 *   32 bytes; scale_page_stride >= kv_heads * page_size. */
typedef struct {
    void *k, *v;
    float *k_scale, *v_scale;
    int64_t pages;
    int64_t page_stride;
    int64_t scale_page_stride;
    int32_t kv_heads, page_size, head_dim, type;
} nm_cache;

/* ---------------------------------------------------------------------------
 * nm_rope_inv_freq -- host-only: the angles per position of the rot_dim / 2
 * rotated pairs, base^(-2 i / rot_dim), scaled for contexts longer than the
 * model was trained on:
 *   NM_ROPE_PLAIN  as is;
 *   NM_ROPE_LINEAR divided by `factor` (positions interpolated);
 *   NM_ROPE_BANDED by wavelength 2 pi / f: shorter than orig_ctx / high: as
 *     is; longer than orig_ctx / low: divided by factor; between them the two
 *     mixed linearly in orig_ctx / wavelength (0 < low < high).
 * rot_dim even, 0 .. 1024; base > 0, factor > 0, else NM_ERR_SHAPE.
 * ------------------------------------------------------------------------- */
#define NM_ROPE_PLAIN 0
#define NM_ROPE_LINEAR 1
#define NM_ROPE_BANDED 2
int nm_rope_inv_freq(float *inv_freq, int rot_dim, double base, int scaling, double factor,
                     double low, double high, double orig_ctx);

/* ---------------------------------------------------------------------------
 * nm_rope_append -- rotate the query and key heads of a QKV projection's
 * output, and write its key and value heads into the cache.
 *   qkv       : device fp16 [tokens][ldqkv], 16-byte aligned, ldqkv % 8 == 0;
 *               a row holds q_heads query heads, then kv_heads key heads, then
 *               kv_heads value heads of head_dim each.
 *   positions : device int32 [tokens] (>= 0);  slots : device int64 [tokens].
 *               A slot outside [0, pages * page_size) is not written (q_out
 *               is).  No two tokens may have the same valid slot.
 *   inv_freq  : device fp32 [rot_dim / 2] (NULL when rot_dim == 0); the first
 *               rot_dim elements of a head are rotated by the angle
 *               position * inv_freq[i], the rest pass through.
 *   interleaved: pair i is (2i, 2i + 1) when nonzero, else
 *               (i, i + rot_dim / 2).  (a, b) becomes
 *               m (a cos - b sin), m (b cos + a sin) with m = mscale (1 unless
 *               a long-context scheme scales its attention).
 *   q_out     : device fp16 [tokens][ldq], 16-byte aligned, ldq % 8 == 0; NULL:
 *               the query heads are skipped.
 * Angles, products and the scales' divisions are fp32; the roundings of the
 * position and of the angle are carried along, so that all positions keep fp32
 * accuracy (2^-21 of |a| + |b| where position * inv_freq's rounding is below 2^-7,
 * positions below 131072 times inv_freq of 1; 2^-20 beyond).  A row's
 * scale is max|x| / 448 (e4m3) or / 127 (int8) and its codes are x / scale,
 * to the nearest (ties to even); a row of zeros has scale 0; a row with a
 * non-finite element has scale NaN (it reads back as NaN).  fp16 rows are
 * rounded once (RNE).  qkv must not overlap q_out or the cache.
 * tokens == 0 is a no-op (the tokens' arrays may be NULL then).  tokens < 2^31,
 * q_heads 1 .. 1024, rot_dim even, 0 .. head_dim, else NM_ERR_SHAPE.
 * ------------------------------------------------------------------------- */
int nm_rope_append(const void *qkv, int64_t ldqkv, int64_t tokens, int q_heads,
                   const int32_t *positions, const int64_t *slots, const float *inv_freq,
                   int rot_dim, int interleaved, float mscale, void *q_out, int64_t ldq,
                   const nm_cache *cache, void *stream);

/* ---------------------------------------------------------------------------
 * nm_cache_read -- rows of the cache as fp16 (code * scale, rounded once).
 *   slots : device int64 [rows]; a slot outside the cache reads as zeros.
 *   k_out, v_out : device fp16 [rows][kv_heads][head_dim], 16-byte aligned;
 *           either may be NULL.  rows == 0 is a no-op (slots may be NULL
 *           then); rows < 2^31.
 * ------------------------------------------------------------------------- */
int nm_cache_read(const nm_cache *cache, const int64_t *slots, int64_t rows, void *k_out,
                  void *v_out, void *stream);

/* ---------------------------------------------------------------------------
 * nm_tree_attention -- attention of the drafted nodes of `seqs` sequences over
 * their cached contexts and trees.
 *   q         : device fp16 [tokens][ldq], 16-byte aligned, ldq % 8 == 0; a row
 *               holds q_heads heads of head_dim; q_heads is a multiple of
 *               kv_heads and query head h reads key head
 *               h / (q_heads / kv_heads).
 *   q_start   : device int32 [seqs + 1], ascending: sequence s has the tokens
 *               q_start[s] .. q_start[s+1] - 1 of q, its nodes 0 .. n - 1.
 *               Nodes beyond max_nodes (1 .. 64) or `tokens` are not computed;
 *               an entry below 0 counts as 0, and a sequence that ends before
 *               it begins has no nodes.
 *   block_table: device int32 [seqs][ld_table], table_cols >= 1 entries used;
 *               entry i of sequence s is the page of its positions
 *               i * page_size ..; positions in a page out of range or beyond
 *               the table are absent (seen by no node).
 *   ctx_len   : device int32 [seqs]: positions 0 .. ctx_len - 1 are the
 *               context, seen by every node (a negative one counts as 0);
 *               position ctx_len + j is node j.
 *   tree_mask : device uint64 [tokens], bit j of a node's word: it sees node j
 *               (its own bit included); NULL: node i sees nodes 0 .. i.
 *   scale     : factor of the scores q . k (finite).
 *   out       : device fp16 [tokens][ldo], 16-byte aligned, ldo % 8 == 0.
 *   lse       : device fp32 [tokens][q_heads] or NULL: log of the sum of
 *               exp(score), the joining weight of attention over parts.
 * A node that sees nothing gets zeros and lse -infinity.  Rows of the cache at
 * positions beyond a sequence's last node are never used, whatever they hold;
 * a non-finite key or value row of a node spoils only the nodes that see it,
 * and a non-finite row of the context all nodes of its sequence.
 * Scores, maxima and sums are fp32.  The weights exp(score - max), times the
 * value row's scale where the cache has one, are rounded to fp16 for the tensor
 * cores' product with the values: by at most 2^-11 of a weight, or 2^-33 of the
 * largest so far where that is more.  (A scale below 2^-64 may count as less or
 * as 2^-80: such values are 0 in fp16.)  Products are accumulated in fp32 and out
 * is rounded once.  The split of the positions over the blocks depends on the
 * lengths, and every part is joined in a fixed order.
 *   workspace : device scratch, 16-byte aligned, of at least
 *       nm_tree_attention_workspace_bytes(...) bytes (counters, then partial
 *       sums of rows cut between blocks), ZERO-FILLED before its first use.  The
 *       counters are at its start whatever the call's shape, nothing else is
 *       written there, and every call leaves them zero: later calls of any shape
 *       on the same device, ordered after this one, can use it as it is.
 * seqs == 0 or tokens == 0 is a no-op (all arrays but the cache's may be NULL
 * then); seqs < 65536, tokens < 2^31, q_heads 1 .. 1024, q_heads / kv_heads <= 64.
 * ------------------------------------------------------------------------- */
size_t nm_tree_attention_workspace_bytes(int64_t seqs, int q_heads, int kv_heads, int head_dim,
                                         int max_nodes);
int nm_tree_attention(const void *q, int64_t ldq, int64_t tokens, int q_heads, int64_t seqs,
                      const int32_t *q_start, int max_nodes, const nm_cache *cache,
                      const int32_t *block_table, int64_t ld_table, int64_t table_cols,
                      const int32_t *ctx_len, const uint64_t *tree_mask, float scale, void *out,
                      int64_t ldo, float *lse, void *workspace, size_t workspace_bytes,
                      void *stream);

/* ---------------------------------------------------------------------------
 * nm_tree_verify -- walk each sequence's tree from node 0, accepting drafted
 * tokens so that the tokens kept are distributed as the target's own.
 *   logits  : device [tokens][ld_logits], fp16 (logits_fp32 == 0) or fp32, row
 *             i: the target's logits after node i; 16-byte aligned, ld_logits
 *             a multiple of 8 (fp16) or 4 (fp32) -- any other base or stride is
 *             taken too, read element by element.
 *   draft   : device fp32 [tokens][ld_draft] or NULL; row n: the distribution
 *             that the children of node n were drawn from, independently.
 *             NULL: the children are proposals without probabilities.
 *   ids     : device int32 [tokens], the nodes' tokens (node 0's is not used);
 *   parents : device int32 [tokens], parent of a node among its sequence's
 *             nodes, lower than the node (node 0's is not used).  A node whose
 *             parent or token is out of range is never visited.
 *   node_start: device int32 [seqs + 1] as q_start above, max_nodes 1 .. 64.
 *   accept  : device fp32 [tokens] in [0, 1), used once per node;
 *   race    : device fp32 [seqs][ld_race] > 0, exponentially distributed.
 * At node n, with w = softmax(logits[n] / temperature), n's children are tried
 * in ascending order: child c with token x is accepted if
 * accept[c] * draft[n][x] < w[x] (without draft: accept[c] < w[x]) and the walk
 * goes on at c; otherwise w becomes relu(w - draft[n]) over its sum (without
 * draft: w with w[x] = 0 over its sum), or stays where that sum is not
 * positive.  When no child is accepted the next token is the index of the
 * largest w[i] / race[s][i] (the lowest of equals): a draw from w.
 * temperature == 0: w is 1 at the largest logit (the lowest index of equals)
 * and accept, race and draft are not read (they may be NULL).
 * A row without a finite largest logit, or with NaN: no child is accepted and
 * the token is -1.
 *   path    : device int32 [seqs][max_nodes]: the nodes visited, node 0 first,
 *             then -1;  count : device int32 [seqs]: how many (0 for a sequence
 *             without nodes);  token : device int32 [seqs]: the next token.
 * Sums are fp32 over fixed parts of the vocabulary, added in a fixed order.
 * seqs == 0 is a no-op (all arrays may be NULL then).  With tokens == 0 no
 * sequence has nodes; path, count and token are written, and the nodes' arrays may
 * be NULL.
 * vocab 1 .. 2^24, seqs < 65536, temperature >= 0 and finite.
 * ------------------------------------------------------------------------- */
int nm_tree_verify(const void *logits, int logits_fp32, int64_t ld_logits, int64_t vocab,
                   const float *draft, int64_t ld_draft, const int32_t *ids,
                   const int32_t *parents, const int32_t *node_start, int64_t tokens,
                   int64_t seqs, int max_nodes, const float *accept, const float *race,
                   int64_t ld_race, float temperature, int32_t *path, int32_t *count,
                   int32_t *token, void *stream);

/* ---------------------------------------------------------------------------
 * nm_tree_attention_stall_selftest, nm_tree_verify_stall_selftest -- exercise
 * the bounded waits (self-tests): the calls above with every wait limited to
 * wait_limit_us (1 .. 2,000,000) and an arrival that never comes.  In every other
 * block of the many-row attention kernel the loaders issue nothing (a call that goes to the few-row
 * kernel runs as usual: that one has no waits); of each sequence's blocks in
 * nm_tree_verify the last sends nothing to the first.  The waits run out or give
 * up after the first that did, are counted in nm_wait_timeouts(), and the kernel
 * returns with its outputs undefined (verify: not written); the device stays
 * usable.  Until nm_wait_timeouts(1) these kernels' calls do nothing.
 * Asynchronous; NM_OK once launched.
 * ------------------------------------------------------------------------- */
int nm_tree_attention_stall_selftest(const void *q, int64_t ldq, int64_t tokens, int q_heads,
                                     int64_t seqs, const int32_t *q_start, int max_nodes,
                                     const nm_cache *cache, const int32_t *block_table,
                                     int64_t ld_table, int64_t table_cols, const int32_t *ctx_len,
                                     const uint64_t *tree_mask, float scale, void *out,
                                     int64_t ldo, float *lse, void *workspace,
                                     size_t workspace_bytes, int64_t wait_limit_us, void *stream);
int nm_tree_verify_stall_selftest(const void *logits, int logits_fp32, int64_t ld_logits,
                                  int64_t vocab, const float *draft, int64_t ld_draft,
                                  const int32_t *ids, const int32_t *parents,
                                  const int32_t *node_start, int64_t tokens, int64_t seqs,
                                  int max_nodes, const float *accept, const float *race,
                                  int64_t ld_race, float temperature, int32_t *path,
                                  int32_t *count, int32_t *token, int64_t wait_limit_us,
                                  void *stream);

#ifdef __cplusplus
}
#endif

#endif /* NM_DECODE_H */
