// verify.cu -- the walk down a tree of drafted tokens (nm_tree_verify).
//
// At a node with target p = softmax(logits / T) and draft q, the distribution
// that the r-th child is tried against is w_r, w_0 = p, and a rejection makes
// it relu(w_r - q) over its sum.  Every w_r has the form relu(a p - b q): from
// (a, b) and Z = sum relu(a p - (b + 1) q), the next pair is (a / Z,
// (b + 1) / Z), since relu(relu(x) - q) = relu(x - q) for q >= 0.  So a
// rejection costs one sum over the vocabulary and nothing is written.  Without
// draft probabilities w_r is p without the rejected tokens over what is left
// of its sum.
#include <cuda_fp16.h>
#include <cuda_runtime.h>
#include <stdint.h>

#include "decode.h"
#include "device.cuh"
#include "kernels.h"

namespace nmk {
namespace {

constexpr int kThreads = 1024;

template <typename T>
__device__ __forceinline__ float logit(const T* row, int i);
template <>
__device__ __forceinline__ float logit<__half>(const __half* row, int i) {
  return __half2float(row[i]);
}
template <>
__device__ __forceinline__ float logit<float>(const float* row, int i) {
  return row[i];
}

struct Best {
  float w;
  int i;
};
// The larger weight, the lower index of equals; i < 0: nothing yet.
__device__ __forceinline__ Best better(Best a, Best b) {
  if (a.i < 0) return b;
  if (b.i < 0) return a;
  return (b.w > a.w || (b.w == a.w && b.i < a.i)) ? b : a;
}

__device__ __forceinline__ float block_sum(float v, float* buf) {
  v = warp_sum(v);
  __syncthreads();
  if ((threadIdx.x & 31) == 0) buf[threadIdx.x >> 5] = v;
  __syncthreads();
  float t = 0.0f;
  for (int w = 0; w < kThreads / 32; ++w) t += buf[w];
  return t;
}

__device__ __forceinline__ float block_max(float v, float* buf) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) v = fmaxf(v, __shfl_xor_sync(0xFFFFFFFFu, v, o));
  __syncthreads();
  if ((threadIdx.x & 31) == 0) buf[threadIdx.x >> 5] = v;
  __syncthreads();
  float t = -INFINITY;
  for (int w = 0; w < kThreads / 32; ++w) t = fmaxf(t, buf[w]);
  return t;
}

__device__ __forceinline__ Best block_best(Best v, Best* buf) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) {
    Best other;
    other.w = __shfl_xor_sync(0xFFFFFFFFu, v.w, o);
    other.i = __shfl_xor_sync(0xFFFFFFFFu, v.i, o);
    v = better(v, other);
  }
  __syncthreads();
  if ((threadIdx.x & 31) == 0) buf[threadIdx.x >> 5] = v;
  __syncthreads();
  Best t{0.0f, -1};
  for (int w = 0; w < kThreads / 32; ++w) t = better(t, buf[w]);
  return t;
}

template <typename T>
__global__ void __launch_bounds__(kThreads) verify_kernel(VerifyParams p) {
  __shared__ float buf[kThreads / 32];
  __shared__ Best bbuf[kThreads / 32];
  __shared__ int s_par[kMaxNodes], s_id[kMaxNodes], s_gone[kMaxNodes];
  pdl_launch_dependents();
  pdl_wait_previous();
  const int s = blockIdx.x, V = p.vocab;
  const int first = min(max(p.node_start[s], 0), p.tokens);
  const int n = min(min(p.node_start[s + 1], p.tokens) - first, p.max_nodes);
  int32_t* path = p.path + (int64_t)s * p.max_nodes;
  if (n <= 0) {
    for (int i = threadIdx.x; i < p.max_nodes; i += kThreads) path[i] = -1;
    if (threadIdx.x == 0) p.count[s] = 0, p.token[s] = -1;
    return;
  }
  if (threadIdx.x < n) {
    s_par[threadIdx.x] = threadIdx.x ? p.parents[first + threadIdx.x] : -1;
    s_id[threadIdx.x] = p.ids[first + threadIdx.x];
  }
  __syncthreads();
  const bool greedy = p.temperature == 0.0f;
  const bool drafted = p.draft && !greedy;
  const float inv_t = greedy ? 1.0f : 1.0f / p.temperature;
  int cur = 0, len = 1, token = -1;
  if (threadIdx.x == 0) path[0] = 0;
  for (;;) {
    const T* row = static_cast<const T*>(p.logits) + (int64_t)(first + cur) * p.ld_logits;
    const float* q = drafted ? p.draft + (int64_t)(first + cur) * p.ld_draft : nullptr;
    int next = -1;
    float nan = 0.0f, mx = -INFINITY;
    Best top{0.0f, -1};
    for (int i = threadIdx.x; i < V; i += kThreads) {
      const float x = logit(row, i);
      if (x != x) nan = 1.0f;
      if (x > mx) mx = x, top = Best{x, i};
    }
    mx = block_max(mx, buf);
    const bool bad = block_max(nan, buf) > 0.0f || !(mx > -INFINITY && mx < INFINITY);
    if (bad) break;
    if (greedy) {
      top = block_best(top, bbuf);
      for (int c = cur + 1; c < n && next < 0; ++c)
        if (s_par[c] == cur && s_id[c] == top.i) next = c;
      if (next < 0) {
        token = top.i;
        break;
      }
    } else {
      float sum = 0.0f;
      for (int i = threadIdx.x; i < V; i += kThreads) sum += expf((logit(row, i) - mx) * inv_t);
      const float inv = 1.0f / block_sum(sum, buf);
      auto prob = [&](int i) { return expf((logit(row, i) - mx) * inv_t) * inv; };
      float a = 1.0f, b = 0.0f;  // w = relu(a p - b q)
      float left = 1.0f;         // without draft: sum of p over what is not rejected
      int gone = 0;
      for (int c = cur + 1; c < n; ++c) {
        const int x = s_id[c];
        if (s_par[c] != cur || x < 0 || x >= V) continue;
        const float u = p.accept[first + c], px = prob(x);
        if (drafted) {
          const float qx = q[x];
          if (u * qx < fmaxf(a * px - b * qx, 0.0f)) {
            next = c;
            break;
          }
          float z = 0.0f;
          for (int i = threadIdx.x; i < V; i += kThreads)
            z += fmaxf(a * prob(i) - (b + 1.0f) * q[i], 0.0f);
          z = block_sum(z, buf);
          if (z > 0.0f) {
            a = a / z;
            b = (b + 1.0f) / z;
          }
        } else {
          bool again = false;
          for (int k = 0; k < gone; ++k) again |= s_gone[k] == x;
          if (!again && u * left < px) {
            next = c;
            break;
          }
          if (!again && left - px > 0.0f) {
            __syncthreads();
            if (threadIdx.x == 0) s_gone[gone] = x;
            __syncthreads();
            ++gone;
            left -= px;
          }
        }
      }
      if (next < 0) {
        Best t{0.0f, -1};
        const float* e = p.race + (int64_t)s * p.ld_race;
        for (int i = threadIdx.x; i < V; i += kThreads) {
          float w = prob(i);
          if (drafted) w = fmaxf(a * w - b * q[i], 0.0f);
          for (int k = 0; k < gone; ++k)
            if (s_gone[k] == i) w = 0.0f;
          t = better(t, Best{w > 0.0f ? w / e[i] : 0.0f, i});
        }
        token = block_best(t, bbuf).i;
        break;
      }
    }
    cur = next;
    if (threadIdx.x == 0) path[len] = cur;
    ++len;
  }
  for (int i = len + threadIdx.x; i < p.max_nodes; i += kThreads) path[i] = -1;
  if (threadIdx.x == 0) {
    p.count[s] = len;
    p.token[s] = token;
  }
}

}  // namespace

cudaError_t launch_verify(const VerifyParams& p, int logits_fp32, int, cudaStream_t stream) {
  if (logits_fp32)
    return launch_kernel(verify_kernel<float>, p.seqs, kThreads, 0, stream, kFlagPdl, p);
  return launch_kernel(verify_kernel<__half>, p.seqs, kThreads, 0, stream, kFlagPdl, p);
}

}  // namespace nmk
