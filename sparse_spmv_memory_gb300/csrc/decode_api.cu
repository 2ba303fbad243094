// decode_api.cu -- the extern "C" boundary of nm_decode.h: argument checks and
// dispatch.
#include <cuda_fp16.h>
#include <cuda_runtime.h>
#include <math.h>
#include <stdint.h>

#include <initializer_list>

#include "../../include/nm_decode.h"
#include "decode.h"
#include "kernels.h"

using namespace nmk;

namespace {

constexpr int64_t kMax31 = (int64_t)1 << 31;

bool aligned(const void* p, uintptr_t a) { return (reinterpret_cast<uintptr_t>(p) & (a - 1)) == 0; }

bool overlap(const void* a, size_t na, const void* b, size_t nb) {
  const uintptr_t a0 = reinterpret_cast<uintptr_t>(a), b0 = reinterpret_cast<uintptr_t>(b);
  return a && b && na && nb && a0 < b0 + nb && b0 < a0 + na;
}

// An array that a call reads, in bytes.
struct Input {
  const void* at;
  size_t bytes;
};

// Whether [b, b + nb) meets any of them.
bool overlaps_any(const void* b, size_t nb, std::initializer_list<Input> inputs) {
  for (const Input& i : inputs)
    if (overlap(b, nb, i.at, i.bytes)) return true;
  return false;
}

// Bytes from the first to the last element of `rows` rows of `width`, `ld` apart.
size_t span(int64_t rows, int64_t ld, int64_t width, size_t size) {
  return rows > 0 ? (size_t)((rows - 1) * ld + width) * size : 0;
}

int code_bytes(int type) { return type == NM_CACHE_FP16 ? 2 : 1; }

int check_cache(const nm_cache* c, CacheView* v) {
  if (!c || !c->k || !c->v) return NM_ERR_NULL;
  if (c->type < NM_CACHE_FP16 || c->type > NM_CACHE_INT8) return NM_ERR_SHAPE;
  const bool scaled = c->type != NM_CACHE_FP16;
  if (scaled && (!c->k_scale || !c->v_scale)) return NM_ERR_NULL;
  const int64_t ps = c->page_size;
  if (ps < 8 || ps > (1 << 20) || (ps & (ps - 1)) || (c->head_dim != 64 && c->head_dim != 128) ||
      c->kv_heads < 1 || c->kv_heads > 1024 || c->pages < 1 || c->pages >= kMax31)
    return NM_ERR_SHAPE;
  const int64_t per_page = c->kv_heads * ps;
  // a page's stride and the cache's last element stay far below 2^63
  if (c->page_stride < per_page * c->head_dim || c->page_stride >= ((int64_t)1 << 38) ||
      (scaled && (c->scale_page_stride < per_page || c->scale_page_stride >= ((int64_t)1 << 38))))
    return NM_ERR_SHAPE;
  if (!aligned(c->k, 32) || !aligned(c->v, 32) || c->page_stride * code_bytes(c->type) % 32 != 0 ||
      (scaled && (!aligned(c->k_scale, 4) || !aligned(c->v_scale, 4))))
    return NM_ERR_ALIGN;
  v->k = static_cast<uint8_t*>(c->k);
  v->v = static_cast<uint8_t*>(c->v);
  v->k_scale = scaled ? c->k_scale : nullptr;
  v->v_scale = scaled ? c->v_scale : nullptr;
  v->pages = c->pages;
  v->page_stride = c->page_stride;
  v->scale_page_stride = c->scale_page_stride;
  v->kv_heads = c->kv_heads;
  v->page_shift = 0;
  while ((1 << v->page_shift) < ps) ++v->page_shift;
  return NM_OK;
}

// Whether [b, b + nb) meets any of the cache's arrays (each taken as one span).
bool overlaps_cache(const nm_cache* c, const void* b, size_t nb) {
  const size_t codes =
      span(c->pages, c->page_stride, (int64_t)c->kv_heads * c->page_size * c->head_dim, code_bytes(c->type));
  const size_t scales = span(c->pages, c->scale_page_stride, (int64_t)c->kv_heads * c->page_size, 4);
  if (overlap(b, nb, c->k, codes) || overlap(b, nb, c->v, codes)) return true;
  return c->type != NM_CACHE_FP16 &&
         (overlap(b, nb, c->k_scale, scales) || overlap(b, nb, c->v_scale, scales));
}

int sm_count(int* sms) {
  DeviceInfo d;
  if (device_info(&d) != cudaSuccess) return NM_ERR_CUDA;
  *sms = d.sms;
  return NM_OK;
}

int status(cudaError_t e) { return e == cudaSuccess ? NM_OK : NM_ERR_CUDA; }

}  // namespace

extern "C" {

int nm_rope_inv_freq(float* inv_freq, int rot_dim, double base, int scaling, double factor,
                     double low, double high, double orig_ctx) {
  if (rot_dim < 0 || rot_dim > 1024 || rot_dim % 2 || !(base > 0) || !(factor > 0) ||
      scaling < NM_ROPE_PLAIN || scaling > NM_ROPE_BANDED ||
      (scaling == NM_ROPE_BANDED && !(low > 0 && high > low && orig_ctx > 0)))
    return NM_ERR_SHAPE;
  if (!inv_freq && rot_dim > 0) return NM_ERR_NULL;
  const double two_pi = 2.0 * acos(-1.0);
  for (int i = 0; i < rot_dim / 2; ++i) {
    const double f = pow(base, -2.0 * i / rot_dim);
    double g = f;
    if (scaling == NM_ROPE_LINEAR) {
      g = f / factor;
    } else if (scaling == NM_ROPE_BANDED) {
      const double turns = orig_ctx * f / two_pi;  // whole turns in the trained context
      double mix = (turns - low) / (high - low);
      mix = mix < 0 ? 0 : mix > 1 ? 1 : mix;
      g = (1 - mix) * f / factor + mix * f;
    }
    inv_freq[i] = (float)g;
  }
  return NM_OK;
}

int nm_rope_append(const void* qkv, int64_t ldqkv, int64_t tokens, int q_heads,
                   const int32_t* positions, const int64_t* slots, const float* inv_freq,
                   int rot_dim, int interleaved, float mscale, void* q_out, int64_t ldq,
                   const nm_cache* cache, void* stream) {
  // (an empty array's address may be NULL: there is nothing to read or write)
  if (tokens != 0 && (!qkv || !positions || !slots || (!inv_freq && rot_dim != 0))) return NM_ERR_NULL;
  AppendParams p;
  const int st = check_cache(cache, &p.c);
  if (st != NM_OK) return st;
  const int64_t width = (int64_t)(q_heads + 2 * cache->kv_heads) * cache->head_dim;
  const int64_t qwidth = (int64_t)q_heads * cache->head_dim;
  if (tokens < 0 || tokens >= kMax31 || q_heads < 1 || q_heads > 1024 || ldqkv < width ||
      ldqkv >= kMax31 || (q_out && (ldq < qwidth || ldq >= kMax31)) || rot_dim < 0 ||
      rot_dim > cache->head_dim || rot_dim % 2)
    return NM_ERR_SHAPE;
  if (!aligned(qkv, 16) || ldqkv % 8 || (q_out && (!aligned(q_out, 16) || ldq % 8)) ||
      !aligned(positions, 4) || !aligned(slots, 8) || !aligned(inv_freq, 4))
    return NM_ERR_ALIGN;
  if (tokens == 0) return NM_OK;
  const size_t in = span(tokens, ldqkv, width, 2), out = span(tokens, ldq, qwidth, 2);
  const size_t pos = (size_t)tokens * 4, sb = (size_t)tokens * 8, fb = (size_t)(rot_dim / 2) * 4;
  if (overlaps_any(q_out, out, {{qkv, in}, {positions, pos}, {slots, sb}, {inv_freq, fb}}) ||
      overlaps_cache(cache, qkv, in) || (q_out && overlaps_cache(cache, q_out, out)) ||
      overlaps_cache(cache, positions, pos) || overlaps_cache(cache, slots, sb) ||
      overlaps_cache(cache, inv_freq, fb))
    return NM_ERR_ALIAS;
  int sms;
  if (sm_count(&sms) != NM_OK) return NM_ERR_CUDA;
  p.qkv = static_cast<const __half*>(qkv);
  p.ldqkv = ldqkv;
  p.tokens = (int)tokens;
  p.q_heads = q_heads;
  p.positions = positions;
  p.slots = slots;
  p.inv_freq = inv_freq;
  p.rot_dim = rot_dim;
  p.interleaved = interleaved;
  p.mscale = mscale;
  p.q_out = static_cast<__half*>(q_out);
  p.ldq = ldq;
  return status(launch_rope_append(p, cache->head_dim, cache->type, sms,
                                   static_cast<cudaStream_t>(stream)));
}

int nm_cache_read(const nm_cache* cache, const int64_t* slots, int64_t rows, void* k_out,
                  void* v_out, void* stream) {
  if (!slots && rows != 0) return NM_ERR_NULL;
  ReadParams p;
  const int st = check_cache(cache, &p.c);
  if (st != NM_OK) return st;
  if (rows < 0 || rows >= kMax31) return NM_ERR_SHAPE;
  if (!aligned(slots, 8) || !aligned(k_out, 16) || !aligned(v_out, 16)) return NM_ERR_ALIGN;
  if (rows == 0 || (!k_out && !v_out)) return NM_OK;
  const size_t out = (size_t)rows * cache->kv_heads * cache->head_dim * 2;
  if (overlap(k_out, out, v_out, out) || overlaps_cache(cache, k_out, k_out ? out : 0) ||
      overlaps_cache(cache, v_out, v_out ? out : 0) || overlap(k_out, out, slots, (size_t)rows * 8) ||
      overlap(v_out, out, slots, (size_t)rows * 8))
    return NM_ERR_ALIAS;
  int sms;
  if (sm_count(&sms) != NM_OK) return NM_ERR_CUDA;
  p.slots = slots;
  p.rows = (int)rows;
  p.k_out = static_cast<__half*>(k_out);
  p.v_out = static_cast<__half*>(v_out);
  return status(launch_cache_read(p, cache->head_dim, cache->type, sms,
                                  static_cast<cudaStream_t>(stream)));
}

static bool attend_shape_ok(int64_t seqs, int q_heads, int kv_heads, int head_dim, int max_nodes) {
  return seqs >= 0 && seqs < 65536 && q_heads >= 1 && q_heads <= 1024 && kv_heads >= 1 &&
         q_heads % kv_heads == 0 && q_heads / kv_heads <= 64 && max_nodes >= 1 &&
         max_nodes <= kMaxNodes && (head_dim == 64 || head_dim == 128);
}

size_t nm_tree_attention_workspace_bytes(int64_t seqs, int q_heads, int kv_heads, int head_dim,
                                         int max_nodes) {
  int sms;
  if (!attend_shape_ok(seqs, q_heads, kv_heads, head_dim, max_nodes) || sm_count(&sms) != NM_OK)
    return 0;
  return attend_workspace_bytes(seqs, q_heads, kv_heads, head_dim, max_nodes, sms);
}

static int tree_attention(const void* q, int64_t ldq, int64_t tokens, int q_heads, int64_t seqs,
                          const int32_t* q_start, int max_nodes, const nm_cache* cache,
                          const int32_t* block_table, int64_t ld_table, int64_t table_cols,
                          const int32_t* ctx_len, const uint64_t* tree_mask, float scale, void* out,
                          int64_t ldo, float* lse, void* workspace, size_t workspace_bytes,
                          void* stream, uint64_t wait_limit_ns, int stall) {
  if (tokens != 0 && seqs != 0 && (!q || !q_start || !block_table || !ctx_len || !out))
    return NM_ERR_NULL;
  AttendParams p;
  const int st = check_cache(cache, &p.c);
  if (st != NM_OK) return st;
  const int64_t width = (int64_t)q_heads * cache->head_dim;
  if (!attend_shape_ok(seqs, q_heads, cache->kv_heads, cache->head_dim, max_nodes) || tokens < 0 ||
      tokens >= kMax31 || ldq < width || ldq >= kMax31 || ldo < width || ldo >= kMax31 ||
      table_cols < 1 || table_cols >= kMax31 || ld_table < (seqs > 1 ? table_cols : 0) ||
      ld_table >= kMax31 || !isfinite(scale))
    return NM_ERR_SHAPE;
  if (!aligned(q, 16) || ldq % 8 || !aligned(out, 16) || ldo % 8 || !aligned(q_start, 4) ||
      !aligned(block_table, 4) || !aligned(ctx_len, 4) || !aligned(tree_mask, 8) ||
      !aligned(lse, 4) || !aligned(workspace, 16))
    return NM_ERR_ALIGN;
  if (seqs == 0 || tokens == 0) return NM_OK;
  const size_t ob = span(tokens, ldo, width, 2), qb = span(tokens, ldq, width, 2);
  const size_t lb = (size_t)tokens * q_heads * 4;
  auto meets_input = [&](const void* at, size_t n) {
    return overlaps_cache(cache, at, n) ||
           overlaps_any(at, n, {{q, qb}, {q_start, (size_t)(seqs + 1) * 4}, {ctx_len, (size_t)seqs * 4},
                                {block_table, span(seqs, ld_table, table_cols, 4)},
                                {tree_mask, (size_t)tokens * 8}});
  };
  if (meets_input(out, ob) || (lse && meets_input(lse, lb)) || overlap(lse, lb, out, ob)) return NM_ERR_ALIAS;
  int sms;
  if (sm_count(&sms) != NM_OK) return NM_ERR_CUDA;
  const size_t need =
      attend_workspace_bytes(seqs, q_heads, cache->kv_heads, cache->head_dim, max_nodes, sms);
  if (need > 0 && (!workspace || workspace_bytes < need)) return NM_ERR_WORKSPACE;
  if (meets_input(workspace, need) || overlap(workspace, need, out, ob) || overlap(workspace, need, lse, lb))
    return NM_ERR_ALIAS;
  p.q = static_cast<const __half*>(q);
  p.ldq = ldq;
  p.tokens = (int)tokens;
  p.q_heads = q_heads;
  p.seqs = (int)seqs;
  p.max_nodes = max_nodes;
  p.q_start = q_start;
  p.table = block_table;
  p.ld_table = ld_table;
  p.table_cols = table_cols;
  p.ctx_len = ctx_len;
  p.tree_mask = tree_mask;
  p.scale = scale;
  p.out = static_cast<__half*>(out);
  p.ldo = ldo;
  p.lse = lse;
  p.workspace = static_cast<uint8_t*>(workspace);
  p.wait_limit_ns = wait_limit_ns;
  p.stall = stall;
  return status(launch_attend(p, cache->head_dim, cache->type, sms,
                              static_cast<cudaStream_t>(stream)));
}

int nm_tree_attention(const void* q, int64_t ldq, int64_t tokens, int q_heads, int64_t seqs,
                      const int32_t* q_start, int max_nodes, const nm_cache* cache,
                      const int32_t* block_table, int64_t ld_table, int64_t table_cols,
                      const int32_t* ctx_len, const uint64_t* tree_mask, float scale, void* out,
                      int64_t ldo, float* lse, void* workspace, size_t workspace_bytes,
                      void* stream) {
  return tree_attention(q, ldq, tokens, q_heads, seqs, q_start, max_nodes, cache, block_table,
                        ld_table, table_cols, ctx_len, tree_mask, scale, out, ldo, lse, workspace,
                        workspace_bytes, stream, kDecodeWaitNs, 0);
}

int nm_tree_attention_stall_selftest(const void* q, int64_t ldq, int64_t tokens, int q_heads,
                                     int64_t seqs, const int32_t* q_start, int max_nodes,
                                     const nm_cache* cache, const int32_t* block_table,
                                     int64_t ld_table, int64_t table_cols, const int32_t* ctx_len,
                                     const uint64_t* tree_mask, float scale, void* out, int64_t ldo,
                                     float* lse, void* workspace, size_t workspace_bytes,
                                     int64_t wait_limit_us, void* stream) {
  if (wait_limit_us < 1 || wait_limit_us > 2000000) return NM_ERR_SHAPE;
  return tree_attention(q, ldq, tokens, q_heads, seqs, q_start, max_nodes, cache, block_table,
                        ld_table, table_cols, ctx_len, tree_mask, scale, out, ldo, lse, workspace,
                        workspace_bytes, stream, (uint64_t)wait_limit_us * 1000u, 1);
}

static int tree_verify(const void* logits, int logits_fp32, int64_t ld_logits, int64_t vocab,
                       const float* draft, int64_t ld_draft, const int32_t* ids,
                       const int32_t* parents, const int32_t* node_start, int64_t tokens,
                       int64_t seqs, int max_nodes, const float* accept, const float* race,
                       int64_t ld_race, float temperature, int32_t* path, int32_t* count,
                       int32_t* token, void* stream, uint64_t wait_limit_ns, int stall) {
  if (seqs != 0 && (!node_start || !path || !count || !token)) return NM_ERR_NULL;
  if (seqs != 0 && tokens != 0 && (!logits || !ids || !parents)) return NM_ERR_NULL;
  if (!(temperature >= 0.0f) || !isfinite(temperature)) return NM_ERR_SHAPE;
  if (seqs != 0 && tokens != 0 && temperature > 0.0f && (!accept || !race)) return NM_ERR_NULL;
  if (vocab < 1 || vocab > (1 << 24) || tokens < 0 || tokens >= kMax31 || seqs < 0 ||
      seqs >= 65536 || max_nodes < 1 || max_nodes > kMaxNodes || ld_logits < vocab ||
      ld_logits >= kMax31 || (temperature > 0.0f && (ld_race < vocab || ld_race >= kMax31)) ||
      (draft && (ld_draft < vocab || ld_draft >= kMax31)))
    return NM_ERR_SHAPE;
  if (!aligned(logits, logits_fp32 ? 4 : 2) || !aligned(draft, 4) || !aligned(ids, 4) ||
      !aligned(parents, 4) || !aligned(node_start, 4) || !aligned(accept, 4) ||
      !aligned(race, 4) || !aligned(path, 4) || !aligned(count, 4) || !aligned(token, 4))
    return NM_ERR_ALIGN;
  if (seqs == 0) return NM_OK;
  const size_t pb = (size_t)seqs * max_nodes * 4, cb = (size_t)seqs * 4;
  const size_t lb = span(tokens, ld_logits, vocab, logits_fp32 ? 4 : 2);
  const bool sampled = temperature > 0.0f;
  const Input written[] = {{path, pb}, {count, cb}, {token, cb}};
  for (const Input& w : written)
    if (overlaps_any(w.at, w.bytes,
                     {{logits, lb}, {ids, (size_t)tokens * 4}, {parents, (size_t)tokens * 4},
                      {node_start, (size_t)(seqs + 1) * 4},
                      {draft, sampled ? span(tokens, ld_draft, vocab, 4) : 0},
                      {accept, sampled ? (size_t)tokens * 4 : 0},
                      {race, sampled ? span(seqs, ld_race, vocab, 4) : 0}}))
      return NM_ERR_ALIAS;
  if (overlap(path, pb, count, cb) || overlap(path, pb, token, cb) || overlap(count, cb, token, cb))
    return NM_ERR_ALIAS;
  int sms;
  if (sm_count(&sms) != NM_OK) return NM_ERR_CUDA;
  VerifyParams p;
  p.logits = logits;
  p.ld_logits = ld_logits;
  p.vocab = (int)vocab;
  p.draft = temperature > 0.0f ? draft : nullptr;
  p.ld_draft = ld_draft;
  p.ids = ids;
  p.parents = parents;
  p.node_start = node_start;
  p.tokens = (int)tokens;
  p.seqs = (int)seqs;
  p.max_nodes = max_nodes;
  p.accept = accept;
  p.race = race;
  p.ld_race = ld_race;
  p.temperature = temperature;
  p.path = path;
  p.count = count;
  p.token = token;
  p.wait_limit_ns = wait_limit_ns;
  p.stall = stall;
  return status(launch_verify(p, logits_fp32, sms, static_cast<cudaStream_t>(stream)));
}

int nm_tree_verify(const void* logits, int logits_fp32, int64_t ld_logits, int64_t vocab,
                   const float* draft, int64_t ld_draft, const int32_t* ids,
                   const int32_t* parents, const int32_t* node_start, int64_t tokens,
                   int64_t seqs, int max_nodes, const float* accept, const float* race,
                   int64_t ld_race, float temperature, int32_t* path, int32_t* count,
                   int32_t* token, void* stream) {
  return tree_verify(logits, logits_fp32, ld_logits, vocab, draft, ld_draft, ids, parents,
                     node_start, tokens, seqs, max_nodes, accept, race, ld_race, temperature, path,
                     count, token, stream, kDecodeWaitNs, 0);
}

int nm_tree_verify_stall_selftest(const void* logits, int logits_fp32, int64_t ld_logits,
                                  int64_t vocab, const float* draft, int64_t ld_draft,
                                  const int32_t* ids, const int32_t* parents,
                                  const int32_t* node_start, int64_t tokens, int64_t seqs,
                                  int max_nodes, const float* accept, const float* race,
                                  int64_t ld_race, float temperature, int32_t* path,
                                  int32_t* count, int32_t* token, int64_t wait_limit_us,
                                  void* stream) {
  if (wait_limit_us < 1 || wait_limit_us > 2000000) return NM_ERR_SHAPE;
  return tree_verify(logits, logits_fp32, ld_logits, vocab, draft, ld_draft, ids, parents,
                     node_start, tokens, seqs, max_nodes, accept, race, ld_race, temperature, path,
                     count, token, stream, (uint64_t)wait_limit_us * 1000u, 1);
}

}  // extern "C"
