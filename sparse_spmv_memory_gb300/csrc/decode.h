// decode.h -- internal launch interface between the C ABI of nm_decode.h
// (decode_api.cu) and its kernels.
#pragma once

#include <cuda_fp16.h>
#include <cuda_runtime.h>
#include <stdint.h>

namespace nmk {

// What a cache holds (the values of NM_CACHE_* in nm_decode.h).
constexpr int kCacheFp16 = 0, kCacheE4m3 = 1, kCacheInt8 = 2;

constexpr int kMaxNodes = 64;  // nodes of a tree: the bits of a mask word
constexpr uint64_t kDecodeWaitNs = 2000000000ull;  // the kernels' waits give up after this

struct CacheView {
  uint8_t *k, *v;           // codes or fp16
  float *k_scale, *v_scale;
  int64_t pages;
  int64_t page_stride;        // elements
  int64_t scale_page_stride;  // rows
  int kv_heads;
  int page_shift;             // log2(page_size)
};

// ---- rotary positions, cache write and read (rope_cache.cu) -----------------
struct AppendParams {
  const __half* qkv;
  int64_t ldqkv;
  int tokens, q_heads;
  const int32_t* positions;
  const int64_t* slots;
  const float* inv_freq;
  int rot_dim, interleaved;
  float mscale;
  __half* q_out;  // may be null
  int64_t ldq;
  CacheView c;
};
cudaError_t launch_rope_append(const AppendParams& p, int head_dim, int type, int sms,
                               cudaStream_t stream);

struct ReadParams {
  CacheView c;
  const int64_t* slots;
  int rows;
  __half *k_out, *v_out;  // either may be null
};
cudaError_t launch_cache_read(const ReadParams& p, int head_dim, int type, int sms,
                              cudaStream_t stream);

// ---- attention over the cache (attend.cu) -------------------------------------
struct AttendParams {
  const __half* q;
  int64_t ldq;
  int tokens, q_heads, seqs, max_nodes;
  const int32_t* q_start;
  CacheView c;
  const int32_t* table;
  int64_t ld_table, table_cols;
  const int32_t* ctx_len;
  const uint64_t* tree_mask;  // null: causal among the nodes
  float scale;
  __half* out;
  int64_t ldo;
  float* lse;  // may be null
  uint8_t* workspace;
  uint64_t wait_limit_ns;  // bound of every wait in the many-row kernel
  int stall;               // self-test: the loaders of every other block issue nothing
};
size_t attend_workspace_bytes(int64_t seqs, int q_heads, int kv_heads, int head_dim, int max_nodes,
                              int sms);
cudaError_t launch_attend(const AttendParams& p, int head_dim, int type, int sms,
                          cudaStream_t stream);

// Many rows per key head (attend_wide.cuh).
template <int TYPE>
cudaError_t launch_attend_wide(const AttendParams& p, int head_dim, int sms, cudaStream_t stream);
// Its bounded waits that gave up since the last reset.
template <int TYPE>
cudaError_t read_attend_wait_timeouts(unsigned long long* count, int reset);

// ---- verification of drafted tokens (verify.cu) --------------------------------
struct VerifyParams {
  const void* logits;
  int64_t ld_logits;
  int vocab;
  const float* draft;  // may be null
  int64_t ld_draft;
  const int32_t *ids, *parents, *node_start;
  int tokens, seqs, max_nodes;
  const float* accept;
  const float* race;
  int64_t ld_race;
  float temperature;
  int32_t *path, *count, *token;
  uint64_t wait_limit_ns;  // bound of every wait
  int stall;               // self-test: a cluster's last block sends nothing to its first
};
cudaError_t launch_verify(const VerifyParams& p, int logits_fp32, int sms, cudaStream_t stream);
cudaError_t read_verify_wait_timeouts(unsigned long long* count, int reset);

}  // namespace nmk
