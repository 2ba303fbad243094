// attend.cu -- attention of drafted nodes over a paged cache
// (nm_tree_attention).
//
// For a node's query q and the rows (k_j, v_j) that it sees,
//   o = sum_j p_j v_j / sum_j p_j,  p_j = exp(scale q.k_j - m),
// with m the largest score so far: a new maximum m' scales what was summed by
// exp(m - m'), so one pass over the cache does, and parts with their own m
// join by the same rule.
#include <cuda_fp16.h>
#include <cuda_fp8.h>
#include <cuda_runtime.h>
#include <stdint.h>

#include "decode.h"
#include "device.cuh"
#include "kernels.h"

namespace nmk {
namespace {

template <int TYPE>
__device__ __forceinline__ float code_value(const uint8_t* base, int64_t at) {
  if (TYPE == kCacheFp16) return __half2float(reinterpret_cast<const __half*>(base)[at]);
  if (TYPE == kCacheInt8) return (float)(int8_t)base[at];
  return __half2float(__half(__nv_cvt_fp8_to_halfraw(base[at], __NV_E4M3)));
}

// One block per token and query head; a warp takes every 8th position, its
// lanes share the head's elements.
template <int D, int TYPE>
__global__ void __launch_bounds__(256) attend_kernel(AttendParams p) {
  constexpr int E = D / 32, NW = 8;
  __shared__ float so[NW][D], sm[NW], sl[NW];
  pdl_launch_dependents();
  pdl_wait_previous();
  const int t = blockIdx.x, hq = blockIdx.y;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  int s = 0;
  while (s < p.seqs && !(p.q_start[s] <= t && t < p.q_start[s + 1])) ++s;
  if (s == p.seqs) return;
  const int first = max(p.q_start[s], 0);
  const int node = t - first;
  const int n = min(min(p.q_start[s + 1], p.tokens) - first, p.max_nodes);
  if (node >= n) return;
  const int ctx = max(p.ctx_len[s], 0);
  const uint64_t seen = p.tree_mask ? p.tree_mask[t] : (2ull << node) - 1ull;
  const int kh = hq / (p.q_heads / p.c.kv_heads);
  float q[E], o[E], m = -INFINITY, l = 0.0f;
#pragma unroll
  for (int e = 0; e < E; ++e) {
    q[e] = __half2float(p.q[(int64_t)t * p.ldq + (int64_t)hq * D + lane + 32 * e]) * p.scale;
    o[e] = 0.0f;
  }
  for (int64_t j = warp; j < (int64_t)ctx + n; j += NW) {
    if (j >= ctx && !((seen >> (j - ctx)) & 1)) continue;
    const int64_t ti = j >> p.c.page_shift;
    if (ti >= p.table_cols) continue;
    const int64_t page = p.table[(int64_t)s * p.ld_table + ti];
    if (page < 0 || page >= p.c.pages) continue;
    const int64_t in_page = ((int64_t)kh << p.c.page_shift) + (j & ((1 << p.c.page_shift) - 1));
    const int64_t at = page * p.c.page_stride + in_page * D;
    const int64_t sat = page * p.c.scale_page_stride + in_page;
    float d = 0.0f;
#pragma unroll
    for (int e = 0; e < E; ++e) d += q[e] * code_value<TYPE>(p.c.k, at + lane + 32 * e);
    d = warp_sum(d);
    if (TYPE != kCacheFp16) d *= p.c.k_scale[sat];
    const float m2 = fmaxf(m, d);
    const float base = m2 == -INFINITY ? 0.0f : m2;
    const float keep = expf(m - base), w = expf(d - base);
    m = m2;
    l = l * keep + w;
    const float wv = TYPE == kCacheFp16 ? w : w * p.c.v_scale[sat];
#pragma unroll
    for (int e = 0; e < E; ++e)
      o[e] = o[e] * keep + wv * code_value<TYPE>(p.c.v, at + lane + 32 * e);
  }
#pragma unroll
  for (int e = 0; e < E; ++e) so[warp][lane + 32 * e] = o[e];
  if (lane == 0) {
    sm[warp] = m;
    sl[warp] = l;
  }
  __syncthreads();
  float M = -INFINITY, tot = 0.0f;
  for (int w = 0; w < NW; ++w) M = fmaxf(M, sm[w]);
  const float base = M == -INFINITY ? 0.0f : M;
  for (int w = 0; w < NW; ++w) tot += sl[w] * expf(sm[w] - base);
  if (threadIdx.x < D) {
    float x = 0.0f;
    for (int w = 0; w < NW; ++w) x += so[w][threadIdx.x] * expf(sm[w] - base);
    const bool none = tot == 0.0f;
    p.out[(int64_t)t * p.ldo + (int64_t)hq * D + threadIdx.x] = __float2half_rn(none ? 0.0f : x / tot);
    if (threadIdx.x == 0 && p.lse) p.lse[(int64_t)t * p.q_heads + hq] = none ? -INFINITY : M + logf(tot);
  }
}

}  // namespace

size_t attend_workspace_bytes(int64_t, int, int, int, int, int) { return 0; }

template <int D, int TYPE>
static cudaError_t attend_one(const AttendParams& p, cudaStream_t stream) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)p.tokens, (unsigned)p.q_heads);
  cfg.blockDim = dim3(256);
  cfg.stream = stream;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, attend_kernel<D, TYPE>, p);
}

cudaError_t launch_attend(const AttendParams& p, int head_dim, int type, int sms,
                          cudaStream_t stream) {
  if (head_dim == 128) {
    if (type == kCacheFp16) return attend_one<128, kCacheFp16>(p, stream);
    if (type == kCacheE4m3) return attend_one<128, kCacheE4m3>(p, stream);
    return attend_one<128, kCacheInt8>(p, stream);
  }
  if (type == kCacheFp16) return attend_one<64, kCacheFp16>(p, stream);
  if (type == kCacheE4m3) return attend_one<64, kCacheE4m3>(p, stream);
  return attend_one<64, kCacheInt8>(p, stream);
}

}  // namespace nmk
