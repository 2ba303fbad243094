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
//
// The walk is sequential: what bounds it is the time from one node's row to
// the next decision, not bandwidth, so one cluster of blocks takes a sequence
// and keeps the node's row (and the draft's) in registers, 32 elements a
// thread; every sum over the vocabulary is a warp's shuffles, one store of each
// warp to every block of the cluster, one cluster barrier, and a sum over all
// warps' values that every warp does for itself, in one fixed order, so that all
// blocks take the same decisions without another exchange.  Only the rows of
// visited nodes are read.
#include <cuda_fp16.h>
#include <cuda_runtime.h>
#include <stdint.h>

#include "decode.h"
#include "device.cuh"
#include "kernels.h"

namespace nmk {
namespace {

constexpr int kThreads = 512, kWarps = 16, kMaxCluster = 16;
constexpr int kHeld = 4;  // groups of 8 elements a thread holds
constexpr float kLog2 = 1.4426950408889634f;

__device__ __forceinline__ float exp2_fast(float x) {  // 2^x, 2^-22 relative, 0 for -inf
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}

// Elements 8 g .. 8 g + 7 of a row, `fill` beyond its end.  vec: the row is
// 16-byte aligned.
__device__ __forceinline__ void load8(const float* row, int g, int n, bool vec, float fill, float (&x)[8]) {
  const float* at = row + (int64_t)g * 8;
  if (vec && g * 8 + 8 <= n) {
    const uint4 a = ld_keep_v4(at), b = ld_keep_v4(at + 4);
    const uint32_t w[8] = {a.x, a.y, a.z, a.w, b.x, b.y, b.z, b.w};
#pragma unroll
    for (int i = 0; i < 8; ++i) x[i] = __uint_as_float(w[i]);
  } else {
#pragma unroll
    for (int i = 0; i < 8; ++i) x[i] = g * 8 + i < n ? at[i] : fill;
  }
}

__device__ __forceinline__ void load8(const __half* row, int g, int n, bool vec, float fill, float (&x)[8]) {
  const __half* at = row + (int64_t)g * 8;
  if (vec && g * 8 + 8 <= n) {
    const uint4 a = ld_keep_v4(at);
    const uint32_t w[4] = {a.x, a.y, a.z, a.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const float2 f = half2_bits_to_float2(w[i]);
      x[2 * i] = f.x;
      x[2 * i + 1] = f.y;
    }
  } else {
#pragma unroll
    for (int i = 0; i < 8; ++i) x[i] = g * 8 + i < n ? __half2float(at[i]) : fill;
  }
}

__device__ __forceinline__ float one(const float* row, int i) { return row[i]; }
__device__ __forceinline__ float one(const __half* row, int i) { return __half2float(row[i]); }

// Asks for elements 8 g .. of a row to come to L2 (a thread of every 128 bytes).
template <typename T>
__device__ __forceinline__ void prefetch8(const T* row, int g, int n) {
  constexpr int kSame = 128 / (8 * sizeof(T));
  if ((threadIdx.x & (kSame - 1)) == 0 && g * 8 < n)
    asm volatile("prefetch.global.L2 [%0];" ::"l"(row + (int64_t)g * 8));
}

// A weight and its index; the larger weight wins, the lower index of equals.
// Index -1: none yet; -2: a row that must not be used, wins over all.
struct Best {
  float w;
  int i;
};
__device__ __forceinline__ Best better(Best a, Best b) {
  if (a.i == -2 || b.i == -1) return a;
  if (b.i == -2 || a.i == -1) return b;
  return (b.w > a.w || (b.w == a.w && b.i < a.i)) ? b : a;
}
__device__ __forceinline__ Best warp_best(Best v) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) {
    Best other;
    other.w = __shfl_xor_sync(0xFFFFFFFFu, v.w, o);
    other.i = __shfl_xor_sync(0xFFFFFFFFu, v.i, o);
    v = better(v, other);
  }
  return v;
}
__device__ __forceinline__ float warp_max(float v) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) v = fmaxf(v, __shfl_xor_sync(0xFFFFFFFFu, v, o));
  return v;
}

template <typename T>
__global__ void __launch_bounds__(kThreads, 1) verify_kernel(VerifyParams p, int vec_logits, int vec_draft,
                                                              int vec_race) {
  __shared__ float2 box[2][kMaxCluster * kWarps];  // every warp's value of the last two exchanges
  __shared__ int s_gone[kMaxNodes];
  pdl_launch_dependents();
  pdl_wait_previous();
  uint32_t rank, cl;
  asm("mov.u32 %0, %%cluster_ctarank;" : "=r"(rank));
  asm("mov.u32 %0, %%cluster_nctarank;" : "=r"(cl));
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int s = blockIdx.x / cl, V = p.vocab;
  const int gt = rank * kThreads + threadIdx.x, stride = cl * kThreads;  // groups of this thread
  const int groups = (V + 7) / 8;
  int round = 0;

  // Every warp's value to every block; where all of them are afterwards.
  auto exchange = [&](float a, float b) -> const float2* {
    float2* here = box[round & 1];
    if (lane < (int)cl) {
      uint32_t remote;
      asm("mapa.shared::cluster.u32 %0, %1, %2;"
          : "=r"(remote)
          : "r"(smem_addr(here + rank * kWarps + warp)), "r"(lane));
      asm volatile("st.shared::cluster.v2.f32 [%0], {%1, %2};" ::"r"(remote), "f"(a), "f"(b) : "memory");
    }
    ++round;  // a box is written again two exchanges on, when all have read it
    asm volatile("barrier.cluster.arrive.release.aligned;" ::: "memory");
    asm volatile("barrier.cluster.wait.acquire.aligned;" ::: "memory");
    return here;
  };
  auto sum_of = [&](float v) {
    const float2* all = exchange(warp_sum(v), 0.0f);
    float t = 0.0f;
    for (int i = lane; i < (int)cl * kWarps; i += 32) t += all[i].x;
    return warp_sum(t);
  };
  auto best_of = [&](Best v) {
    v = warp_best(v);
    const float2* all = exchange(v.w, __int_as_float(v.i));
    Best t{0.0f, -1};
    for (int i = lane; i < (int)cl * kWarps; i += 32) t = better(t, Best{all[i].x, __float_as_int(all[i].y)});
    return warp_best(t);
  };

  const int first = min(max(p.node_start[s], 0), p.tokens);
  const int n = min(min(p.node_start[s + 1], p.tokens) - first, p.max_nodes);
  int32_t* path = p.path + (int64_t)s * p.max_nodes;
  const bool writer = rank == 0 && warp == 0;
  int cur = 0, len = 0, token = -1;
  if (n > 0) {
    // lane l has the nodes l and l + 32
    int par[2], id[2];
    float u[2];
#pragma unroll
    for (int k = 0; k < 2; ++k) {
      const int c = lane + 32 * k;
      const bool in = c > 0 && c < n;
      par[k] = in ? p.parents[first + c] : -1;
      id[k] = in ? p.ids[first + c] : -1;
      u[k] = in && p.temperature > 0.0f ? p.accept[first + c] : 0.0f;
      if (par[k] >= c || id[k] < 0 || id[k] >= V) par[k] = -1;  // never visited
    }
    const bool greedy = p.temperature == 0.0f, drafted = p.draft != nullptr;
    const float scale = greedy ? 1.0f : kLog2 / p.temperature;
    // a row on its way to L2: a child's while its parent is still looked at
    auto fetch = [&](int node) {
      const T* r = static_cast<const T*>(p.logits) + (int64_t)(first + node) * p.ld_logits;
#pragma unroll
      for (int k = 0; k < kHeld; ++k) prefetch8(r, gt + k * stride, V);
      if (drafted) {
        const float* d = p.draft + (int64_t)(first + node) * p.ld_draft;
#pragma unroll
        for (int k = 0; k < kHeld; ++k) prefetch8(d, gt + k * stride, V);
      }
    };
    for (;;) {
      if (writer && lane == 0) path[len] = cur;
      ++len;
      const T* row = static_cast<const T*>(p.logits) + (int64_t)(first + cur) * p.ld_logits;
      const float* qrow = drafted ? p.draft + (int64_t)(first + cur) * p.ld_draft : nullptr;
      float x[kHeld][8], q[kHeld][8];
#pragma unroll
      for (int k = 0; k < kHeld; ++k) load8(row, gt + k * stride, V, vec_logits, -INFINITY, x[k]);
      if (drafted) {
#pragma unroll
        for (int k = 0; k < kHeld; ++k) load8(qrow, gt + k * stride, V, vec_draft, 0.0f, q[k]);
      }
      const uint64_t kids = (uint64_t)__ballot_sync(0xFFFFFFFFu, par[0] == cur) |
                            (uint64_t)__ballot_sync(0xFFFFFFFFu, par[1] == cur) << 32;
      if (kids) fetch(__ffsll(kids) - 1);
      if (len == 1 && !greedy) {
        const float* race = p.race + (int64_t)s * p.ld_race;
#pragma unroll
        for (int k = 0; k < kHeld; ++k) prefetch8(race, gt + k * stride, V);
      }
      float kx[2] = {0.0f, 0.0f}, kq[2] = {1.0f, 1.0f};  // the children's logits and draft
      if (!greedy) {
#pragma unroll
        for (int k = 0; k < 2; ++k)
          if (par[k] == cur) {
            kx[k] = one(row, id[k]);
            if (drafted) kq[k] = qrow[id[k]];
          }
      }
      int next = -1;
      if (greedy) {
        Best t{-INFINITY, -1};
        bool bad = false;
        auto look = [&](const float (&v)[8], int g) {
#pragma unroll
          for (int i = 0; i < 8; ++i) {
            bad |= !(v[i] < INFINITY);  // NaN or +infinity
            if (v[i] > t.w) t = Best{v[i], g * 8 + i};  // ascending: the lowest of equals
          }
        };
#pragma unroll
        for (int k = 0; k < kHeld; ++k) look(x[k], gt + k * stride);
        for (int g = gt + kHeld * stride; g < groups; g += stride) {
          load8(row, g, V, vec_logits, -INFINITY, x[0]);
          look(x[0], g);
        }
        if (bad) t.i = -2;
        t = best_of(t);
        if (t.i >= 0) {
          token = t.i;
          const uint64_t hit = kids & ((uint64_t)__ballot_sync(0xFFFFFFFFu, id[0] == token) |
                                       (uint64_t)__ballot_sync(0xFFFFFFFFu, id[1] == token) << 32);
          if (hit) next = __ffsll(hit) - 1;
        }
        if (next < 0) break;
        token = -1;
        cur = next;
        continue;
      }
      // the largest logit and the sum of 2^((x - largest) scale)
      float m = -INFINITY;
#pragma unroll
      for (int k = 0; k < kHeld; ++k)
#pragma unroll
        for (int i = 0; i < 8; ++i) m = fmaxf(m, x[k][i]);
      float y[8];
      for (int g = gt + kHeld * stride; g < groups; g += stride) {
        load8(row, g, V, vec_logits, -INFINITY, y);
#pragma unroll
        for (int i = 0; i < 8; ++i) m = fmaxf(m, y[i]);
      }
      m = warp_max(m);
      const float m0 = m == -INFINITY ? 0.0f : m;
      float sum = 0.0f;
#pragma unroll
      for (int k = 0; k < kHeld; ++k)
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          x[k][i] = exp2_fast((x[k][i] - m0) * scale);
          sum += x[k][i];
        }
      for (int g = gt + kHeld * stride; g < groups; g += stride) {
        load8(row, g, V, vec_logits, -INFINITY, y);
#pragma unroll
        for (int i = 0; i < 8; ++i) sum += exp2_fast((y[i] - m0) * scale);
      }
      const float2* all = exchange(m, warp_sum(sum));
      float M = -INFINITY, S = 0.0f;
      for (int i = lane; i < (int)cl * kWarps; i += 32) M = fmaxf(M, all[i].x);
      M = warp_max(M);
      if (!(M > -INFINITY && M < INFINITY)) break;
      for (int i = lane; i < (int)cl * kWarps; i += 32) S += all[i].y * exp2_fast((all[i].x - M) * scale);
      S = warp_sum(S);
      if (!(S > 0.0f && S < INFINITY)) break;  // a NaN among the logits
      const float inv = 1.0f / S;
      auto prob = [&](float v) { return exp2_fast((v - M) * scale) * inv; };
      const float mine = m == -INFINITY ? 0.0f : exp2_fast((m - M) * scale) * inv;
#pragma unroll
      for (int k = 0; k < kHeld; ++k)
#pragma unroll
        for (int i = 0; i < 8; ++i) x[k][i] *= mine;

      float a = 1.0f, b = 0.0f;  // w = relu(a p - b q)
      float left = 1.0f;         // without draft: the sum of p over what is not rejected
      int gone = 0;
      for (uint64_t rest = kids; rest && next < 0; rest &= rest - 1) {
        const int c = __ffsll(rest) - 1, from = c & 31;
        const int t = __shfl_sync(0xFFFFFFFFu, c < 32 ? id[0] : id[1], from);
        const float uc = __shfl_sync(0xFFFFFFFFu, c < 32 ? u[0] : u[1], from);
        const float pt = prob(__shfl_sync(0xFFFFFFFFu, c < 32 ? kx[0] : kx[1], from));
        const float qt = __shfl_sync(0xFFFFFFFFu, c < 32 ? kq[0] : kq[1], from);
        const uint64_t later = rest & (rest - 1);
        if (drafted) {
          if (uc * qt < fmaxf(a * pt - b * qt, 0.0f)) {
            next = c;
            break;
          }
          if (later) fetch(__ffsll(later) - 1);
          float z = 0.0f;
#pragma unroll
          for (int k = 0; k < kHeld; ++k)
#pragma unroll
            for (int i = 0; i < 8; ++i) z += fmaxf(a * x[k][i] - (b + 1.0f) * q[k][i], 0.0f);
          for (int g = gt + kHeld * stride; g < groups; g += stride) {
            float v[8];
            load8(row, g, V, vec_logits, -INFINITY, y);
            load8(qrow, g, V, vec_draft, 0.0f, v);
#pragma unroll
            for (int i = 0; i < 8; ++i) z += fmaxf(a * prob(y[i]) - (b + 1.0f) * v[i], 0.0f);
          }
          z = sum_of(z);
          if (z > 0.0f) {
            a = a / z;
            b = (b + 1.0f) / z;
          }
        } else {
          bool again = false;
          for (int k = 0; k < gone; ++k) again |= s_gone[k] == t;
          if (!again && uc * left < pt) {
            next = c;
            break;
          }
          if (!again && left - pt > 0.0f) {
            __syncthreads();
            if (threadIdx.x == 0) s_gone[gone] = t;
            __syncthreads();
            ++gone;
            left -= pt;
          }
        }
      }
      if (next >= 0) {
        cur = next;
        continue;
      }
      // no child: the race over w
      Best t{-1.0f, -1};
      const float* race = p.race + (int64_t)s * p.ld_race;
      if (drafted) {
#pragma unroll
        for (int k = 0; k < kHeld; ++k)
#pragma unroll
          for (int i = 0; i < 8; ++i) x[k][i] = fmaxf(a * x[k][i] - b * q[k][i], 0.0f);
      }
#pragma unroll
      for (int k = 0; k < kHeld; ++k) load8(race, gt + k * stride, V, vec_race, 1.0f, q[k]);
      auto run = [&](const float (&w)[8], const float (&e)[8], int g) {
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          float r = w[i] > 0.0f ? __fdividef(w[i], e[i]) : 0.0f;
          for (int k = 0; k < gone; ++k) r = s_gone[k] == g * 8 + i ? 0.0f : r;
          if (r > t.w && g * 8 + i < V) t = Best{r, g * 8 + i};  // ascending: the lowest of equals
        }
      };
#pragma unroll
      for (int k = 0; k < kHeld; ++k) run(x[k], q[k], gt + k * stride);
      for (int g = gt + kHeld * stride; g < groups; g += stride) {
        load8(row, g, V, vec_logits, -INFINITY, x[0]);
        load8(race, g, V, vec_race, 1.0f, q[0]);
        if (drafted) load8(qrow, g, V, vec_draft, 0.0f, y);
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          x[0][i] = prob(x[0][i]);
          if (drafted) x[0][i] = fmaxf(a * x[0][i] - b * y[i], 0.0f);
        }
        run(x[0], q[0], g);
      }
      token = best_of(t).i;
      break;
    }
  }
  if (writer) {
    for (int i = len + lane; i < p.max_nodes; i += 32) path[i] = -1;
    if (lane == 0) {
      p.count[s] = len;
      p.token[s] = token;
    }
  }
  // no block ends while another may still store to its shared memory
  asm volatile("barrier.cluster.arrive.release.aligned;" ::: "memory");
  asm volatile("barrier.cluster.wait.acquire.aligned;" ::: "memory");
}

bool rows_aligned(const void* p, int64_t ld, size_t size) {
  return p && reinterpret_cast<uintptr_t>(p) % 16 == 0 && ld * (int64_t)size % 16 == 0;
}

template <typename T>
cudaError_t verify_one(const VerifyParams& p, int sms, cudaStream_t stream) {
  auto* k = verify_kernel<T>;
  // The fewest blocks whose threads hold a row (a longer vocabulary's rest is
  // read again for every sum); more of them, down to 8 elements a thread, while
  // all sequences' blocks have an SM each: a sum's 2^x then take less of its time.
  int cl = 1;
  while (cl < kMaxCluster && cl * kThreads * kHeld * 8 < p.vocab) cl *= 2;
  while (cl < kMaxCluster && cl * kThreads * 8 < p.vocab && (int64_t)p.seqs * cl * 2 <= sms) cl *= 2;
  if (cl > 8) {
    static int done[64];
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess) return e;
    if (dev >= 64 || !__atomic_load_n(&done[dev], __ATOMIC_ACQUIRE)) {
      e = cudaFuncSetAttribute(k, cudaFuncAttributeNonPortableClusterSizeAllowed, 1);
      if (e != cudaSuccess) return e;
      if (dev < 64) __atomic_store_n(&done[dev], 1, __ATOMIC_RELEASE);
    }
  }
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)(p.seqs * cl));
  cfg.blockDim = dim3(kThreads);
  cfg.stream = stream;
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim.x = cl;
  attr[0].val.clusterDim.y = attr[0].val.clusterDim.z = 1;
  attr[1].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[1].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 2;
  return cudaLaunchKernelEx(&cfg, k, p, (int)rows_aligned(p.logits, p.ld_logits, sizeof(T)),
                            (int)rows_aligned(p.draft, p.ld_draft, 4), (int)rows_aligned(p.race, p.ld_race, 4));
}

}  // namespace

cudaError_t launch_verify(const VerifyParams& p, int logits_fp32, int sms, cudaStream_t stream) {
  return logits_fp32 ? verify_one<float>(p, sms, stream) : verify_one<__half>(p, sms, stream);
}

}  // namespace nmk
