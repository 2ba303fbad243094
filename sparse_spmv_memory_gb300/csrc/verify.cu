// verify.cu -- the walk down a tree of drafted tokens (nm_tree_verify).
//
// At a node with target p = softmax(logits / T) and draft q, the distribution
// that the r-th child is tried against is w_r, w_0 = p, and a rejection makes
// it relu(w_r - q) over its sum.  Every w_r has the form relu(a p - b q): from
// (a, b) and Z = sum relu(a p - (b + 1) q), the next pair is (a / Z,
// (b + 1) / Z), since relu(relu(x) - q) = relu(x - q) for q >= 0.  So a
// rejection costs one sum over the vocabulary and nothing is written.  Without
// draft probabilities w_r is p without the rejected tokens over what is left
// of its sum: a difference while that is a quarter of p at least, whose rounding
// is then 2^-22 of it a rejection, and else summed anew.
//
// The walk is sequential: what bounds it is the time from one node's row to
// the next decision, not bandwidth.  One cluster of blocks takes a sequence;
// a thread keeps its 16 (or 32) elements of the node's row in registers and of
// the draft's in shared memory, so that two blocks fit an SM.  A sum over the
// vocabulary goes through the block's warps, then by one asynchronous store of
// each block to every block of the cluster, and every warp joins the blocks'
// values for itself in one fixed order: all take the same decisions without
// another exchange.  The rows of the child that is to be tried next are fetched
// to L2 meanwhile.
//
// Measured: a node costs 2 us to load and weigh and an exchange 1.1; 5 nodes of
// one sequence over a vocabulary of 128256 take 12 us, 16 sequences of 32 nodes 39
// (17 % of HBM's rate), 32 of 8 without draft over 50257 19.
#include <cuda_fp16.h>
#include <cuda_runtime.h>
#include <stdint.h>

#include "decode.h"
#include "device.cuh"
#include "kernels.h"
#include "tc.cuh"

namespace nmk {
namespace {

constexpr int kThreads = 512, kWarps = 16, kMaxCluster = 16;
// HELD: groups of 8 elements a thread holds.
constexpr int draft_bytes(int held) { return kThreads * held * 8 * 4; }

__device__ __forceinline__ uint4 load16_if(const void* at, bool on) {
  uint4 v;
  asm volatile(
      "{\n\t.reg .pred p;\n\tsetp.ne.u32 p, %5, 0;\n\t"
      "mov.u32 %0, 0;\n\tmov.u32 %1, 0;\n\tmov.u32 %2, 0;\n\tmov.u32 %3, 0;\n\t"
      "@p ld.global.nc.v4.u32 {%0,%1,%2,%3}, [%4];\n\t}"
      : "=&r"(v.x), "=&r"(v.y), "=&r"(v.z), "=&r"(v.w)
      : "l"(at), "r"((uint32_t)on));
  return v;
}

// One element's bits if `on` (0 else), and its value: the bits are asked for
// where a conversion would wait for them.
__device__ __forceinline__ uint32_t bits_if(const float* at, bool on) {
  uint32_t v;
  asm volatile("{\n\t.reg .pred p;\n\tsetp.ne.u32 p, %2, 0;\n\tmov.u32 %0, 0;\n\t@p ld.global.nc.u32 %0, [%1];\n\t}"
               : "=&r"(v)
               : "l"(at), "r"((uint32_t)on));
  return v;
}
__device__ __forceinline__ uint32_t bits_if(const __half* at, bool on) {
  uint16_t v;
  asm volatile("{\n\t.reg .pred p;\n\tsetp.ne.u32 p, %2, 0;\n\tmov.u16 %0, 0;\n\t@p ld.global.nc.u16 %0, [%1];\n\t}"
               : "=&h"(v)
               : "l"(at), "r"((uint32_t)on));
  return v;
}
template <typename T>
__device__ __forceinline__ float value_of(uint32_t bits) {
  return sizeof(T) == 2 ? __half2float(__ushort_as_half((uint16_t)bits)) : __uint_as_float(bits);
}

__device__ __forceinline__ float one(const float* row, int i) { return row[i]; }
__device__ __forceinline__ float one(const __half* row, int i) { return __half2float(row[i]); }

// A thread's groups of 8 elements of a row of n, `fill` beyond its end: group k
// is the row's g0 + k * stride.  The loads are all issued before the first is
// used; vec: the row is 16-byte aligned.
template <int K, typename T>
__device__ __forceinline__ void load_groups(const T* row, int g0, int stride, int n, bool vec, float fill,
                                            float (&x)[K][8]) {
  constexpr int W = sizeof(T) / 2;  // 16-byte words of a group
  if (!vec) {
#pragma unroll
    for (int k = 0; k < K; ++k)
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        const int e = (g0 + k * stride) * 8 + i;
        x[k][i] = e < n ? one(row, e) : fill;
      }
    return;
  }
  uint4 raw[K][W];
#pragma unroll
  for (int k = 0; k < K; ++k) {
    const int g = g0 + k * stride;
#pragma unroll
    for (int w = 0; w < W; ++w)
      raw[k][w] = load16_if(row + (int64_t)g * 8 + w * (16 / sizeof(T)), g * 8 + 8 <= n);
  }
#pragma unroll
  for (int k = 0; k < K; ++k) {
    const int g = g0 + k * stride;
#pragma unroll
    for (int w = 0; w < W; ++w) {
      const uint32_t v[4] = {raw[k][w].x, raw[k][w].y, raw[k][w].z, raw[k][w].w};
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        if (sizeof(T) == 2) {
          const float2 f = half2_bits_to_float2(v[i]);
          x[k][2 * i] = f.x;
          x[k][2 * i + 1] = f.y;
        } else {
          x[k][4 * w + i] = __uint_as_float(v[i]);
        }
      }
    }
    if (g * 8 + 8 > n) {  // the row's end
#pragma unroll
      for (int i = 0; i < 8; ++i) x[k][i] = g * 8 + i < n ? one(row, g * 8 + i) : fill;
    }
  }
}

// Asks for the thread's groups of a row to come to L2.
template <int K, typename T>
__device__ __forceinline__ void prefetch_groups(const T* row, int g0, int stride, int n) {
  constexpr int kSame = 128 / (8 * sizeof(T));  // threads of 128 bytes
  if ((threadIdx.x & (kSame - 1)) == 0) {
#pragma unroll
    for (int k = 0; k < K; ++k)
      if ((g0 + k * stride) * 8 < n)
        asm volatile("prefetch.global.L2 [%0];" ::"l"(row + (int64_t)(g0 + k * stride) * 8));
  }
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
__device__ __forceinline__ float warp_max(float v) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) v = fmaxf(v, __shfl_xor_sync(0xFFFFFFFFu, v, o));
  return v;
}

// Joins the first W lanes' values (in every lane of each W).
template <int W, typename Op>
__device__ __forceinline__ float2 lanes_join(float2 v, Op op) {
#pragma unroll
  for (int o = W / 2; o > 0; o >>= 1) {
    float2 other;
    other.x = __shfl_xor_sync(0xFFFFFFFFu, v.x, o);
    other.y = __shfl_xor_sync(0xFFFFFFFFu, v.y, o);
    v = op(v, other);
  }
  return v;
}

template <typename T, int HELD>
__global__ void __launch_bounds__(kThreads, 2) verify_kernel(VerifyParams p, int vec_logits, int vec_draft,
                                                              int vec_race) {
  extern __shared__ float4 s_q[];                  // the draft's row: [2 HELD][kThreads]
  __shared__ float2 box[2][kMaxCluster];  // the blocks' values of the last two exchanges
  __shared__ float2 warps[kWarps];
  __shared__ uint64_t bar_mem[2];
  uint32_t rank, cl;
  asm("mov.u32 %0, %%cluster_ctarank;" : "=r"(rank));
  asm("mov.u32 %0, %%cluster_nctarank;" : "=r"(cl));
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  pdl_launch_dependents();
  const uint32_t bars = smem_addr(bar_mem);
  if (threadIdx.x == 0) {
    mbar_init(bars, 1);
    mbar_init(bars + 8, 1);
    fence_mbar_init();
  }
  // No wait of the block's gave up, and none of another's before it began.  It is
  // one value for the whole block, so that its warps leave the walk together: a
  // block that leaves keeps its shared memory until the cluster ends, and the
  // others' next wait, for what it does not send any more, has its limit too.
  bool ok = !__syncthreads_or(threadIdx.x == 0 && wait_aborted());
  // every block's barriers are there before another's store can arrive
  asm volatile("barrier.cluster.arrive.release.aligned;" ::: "memory");
  asm volatile("barrier.cluster.wait.acquire.aligned;" ::: "memory");
  pdl_wait_previous();
  const int s = blockIdx.x / cl, V = p.vocab;
  const int gt = rank * kThreads + threadIdx.x, stride = cl * kThreads;  // groups of this thread
  const int groups = (V + 7) / 8;
  const bool more = HELD * stride < groups;  // a longer vocabulary than the cluster holds
  int round = 0;

  // The values of all threads of the cluster, joined (the same in every thread);
  // none: op's neutral value.  A box is written again two exchanges on: a block
  // sends for the next one when all its warps have read this one.
  auto join = [&](float2 v, float2 none, auto op) {
    v = lanes_join<32>(v, op);
    if (lane == 0) warps[warp] = v;
    const int r = round & 1;
    const uint32_t bar = bars + 8u * r;
    __syncthreads();
    if (warp == 0) {
      v = lanes_join<kWarps>(warps[lane & (kWarps - 1)], op);
      if (lane == 0) mbar_arrive_expect_tx(bar, cl * 8);
      if (lane < (int)cl && !(p.stall && rank == cl - 1 && lane == 0)) {
        uint32_t at, rbar;
        asm("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(at) : "r"(smem_addr(&box[r][rank])), "r"(lane));
        asm("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(rbar) : "r"(bar), "r"(lane));
        asm volatile("st.async.shared::cluster.mbarrier::complete_tx::bytes.v2.f32 [%0], {%1, %2}, [%3];" ::"r"(at),
                     "f"(v.x), "f"(v.y), "r"(rbar)
                     : "memory");
      }
    }
    ok = __syncthreads_and(warp != 0 || mbar_wait(bar, (round >> 1) & 1, p.wait_limit_ns));
    ++round;
    return lanes_join<kMaxCluster>((lane & (kMaxCluster - 1)) < (int)cl ? box[r][lane & (kMaxCluster - 1)] : none, op);
  };
  auto sum_of = [&](float v) {
    return join(make_float2(v, 0.0f), make_float2(0.0f, 0.0f),
                [](float2 a, float2 b) { return make_float2(a.x + b.x, 0.0f); }).x;
  };
  auto best_of = [&](Best v) {
    const float2 r = join(make_float2(v.w, __int_as_float(v.i)), make_float2(0.0f, __int_as_float(-1)),
                          [](float2 a, float2 b) {
                            const Best c = better(Best{a.x, __float_as_int(a.y)}, Best{b.x, __float_as_int(b.y)});
                            return make_float2(c.w, __int_as_float(c.i));
                          });
    return Best{r.x, __float_as_int(r.y)};
  };

  const int first = min(max(p.node_start[s], 0), p.tokens);
  const int n = min(min(max(p.node_start[s + 1], 0), p.tokens) - first, p.max_nodes);
  int32_t* path = p.path + (int64_t)s * p.max_nodes;
  const bool writer = rank == 0 && warp == 0;
  const bool greedy = p.temperature == 0.0f, drafted = p.draft != nullptr;
  // (finite at the smallest temperatures too: the largest logit's exponent is 0 times it)
  const float scale = greedy ? 1.0f : fminf(kLog2e / p.temperature, 3.4e38f);
  const float* race = p.race + (int64_t)s * p.ld_race;
  auto row_of = [&](int node) { return static_cast<const T*>(p.logits) + (int64_t)(first + node) * p.ld_logits; };
  auto draft_of = [&](int node) { return p.draft + (int64_t)(first + node) * p.ld_draft; };
  // rows on their way to L2: a child's while its parent is still looked at
  auto fetch = [&](int node) {
    prefetch_groups<HELD>(row_of(node), gt, stride, V);
    if (drafted) prefetch_groups<HELD>(draft_of(node), gt, stride, V);
  };
  // the thread's groups of the draft's row to shared memory (its own slots)
  auto stage_draft = [&](const float* row) {
#pragma unroll
    for (int k = 0; k < HELD; ++k) {
      const int g = gt + k * stride;
#pragma unroll
      for (int w = 0; w < 2; ++w) {
        float4* slot = s_q + (2 * k + w) * kThreads + threadIdx.x;
        if (vec_draft && g * 8 + 8 <= V) {
          asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(smem_addr(slot)),
                       "l"(row + (int64_t)g * 8 + 4 * w)
                       : "memory");
        } else {
          float v[4];
#pragma unroll
          for (int i = 0; i < 4; ++i) v[i] = g * 8 + 4 * w + i < V ? row[(int64_t)g * 8 + 4 * w + i] : 0.0f;
          *slot = make_float4(v[0], v[1], v[2], v[3]);
        }
      }
    }
  };
  auto draft8 = [&](int k, float (&q)[8]) {
    const float4 a = s_q[2 * k * kThreads + threadIdx.x], b = s_q[(2 * k + 1) * kThreads + threadIdx.x];
    q[0] = a.x, q[1] = a.y, q[2] = a.z, q[3] = a.w;
    q[4] = b.x, q[5] = b.y, q[6] = b.z, q[7] = b.w;
  };
  // the rest of a longer vocabulary: f(first element, 8 logits) for each group
  auto rest_of = [&](const T* row, auto f) {
    if (!more) return;
#pragma unroll 1
    for (int g = gt + HELD * stride; g < groups; g += stride) {
      float y[1][8];
      load_groups(row, g, 0, V, vec_logits, -INFINITY, y);
      f(g * 8, y[0]);
    }
  };

  // whether token t is that of one of the nodes `set`
  auto rejected = [&](uint64_t set, int t) {
    for (; set; set &= set - 1)
      if (p.ids[first + __ffsll(set) - 1] == t) return true;
    return false;
  };

  int cur = 0, len = 0, token = -1;
  if (n > 0 && ok) {
    // lane l has the nodes l and l + 32
    int par[2], id[2];
    float u[2];
    bool loaded = false;
    for (;;) {
      if (writer && lane == 0) path[len] = cur;
      ++len;
      const T* row = row_of(cur);
      const float* qrow = drafted ? draft_of(cur) : nullptr;
      if (!loaded) {
        loaded = true;
        fetch(0);
#pragma unroll
        for (int k = 0; k < 2; ++k) {
          const int c = lane + 32 * k;
          const bool in = c > 0 && c < n;
          par[k] = in ? p.parents[first + c] : -1;
          id[k] = in ? p.ids[first + c] : -1;
          u[k] = in && !greedy ? p.accept[first + c] : 0.0f;
          if (par[k] >= c || id[k] < 0 || id[k] >= V) par[k] = -1;  // never visited
        }
        if (!greedy) prefetch_groups<HELD>(race, gt, stride, V);
      }
      // everything that this node needs is asked for before any of it is used
      uint32_t kx[2], kq[2];  // the children's logits and draft
#pragma unroll
      for (int k = 0; k < 2; ++k) {
        const bool on = par[k] == cur && !greedy;
        kx[k] = bits_if(row + (on ? id[k] : 0), on);
        kq[k] = drafted ? bits_if(qrow + (on ? id[k] : 0), on) : 0x3F800000u;  // 1
      }
      float x[HELD][8];
      if (drafted) stage_draft(qrow);
      load_groups(row, gt, stride, V, vec_logits, -INFINITY, x);
      const uint64_t kids = (uint64_t)__ballot_sync(0xFFFFFFFFu, par[0] == cur) |
                            (uint64_t)__ballot_sync(0xFFFFFFFFu, par[1] == cur) << 32;
      if (kids) fetch(__ffsll(kids) - 1);
      int next = -1;
      if (greedy) {
        Best t{-INFINITY, -1};
        bool bad = false;
        auto look = [&](int e, const float (&v)[8]) {
#pragma unroll
          for (int i = 0; i < 8; ++i) {
            bad |= !(v[i] < INFINITY);                 // NaN or +infinity
            if (v[i] > t.w) t = Best{v[i], e + i};  // ascending: the lowest of equals
          }
        };
#pragma unroll
        for (int k = 0; k < HELD; ++k) look((gt + k * stride) * 8, x[k]);
        rest_of(row, look);
        if (bad) t.i = -2;
        t = best_of(t);
        if (!ok) break;
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
      for (int k = 0; k < HELD; ++k)
#pragma unroll
        for (int i = 0; i < 8; ++i) m = fmaxf(m, x[k][i]);
      rest_of(row, [&](int, const float (&v)[8]) {
#pragma unroll
        for (int i = 0; i < 8; ++i) m = fmaxf(m, v[i]);
      });
      m = warp_max(m);
      const float m0 = m == -INFINITY ? 0.0f : m;
      float sum = 0.0f;
#pragma unroll
      for (int k = 0; k < HELD; ++k)
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          x[k][i] = exp2_fast((x[k][i] - m0) * scale);
          sum += x[k][i];
        }
      rest_of(row, [&](int, const float (&v)[8]) {
#pragma unroll
        for (int i = 0; i < 8; ++i) sum += exp2_fast((v[i] - m0) * scale);
      });
      // (m is the warp's already: the sums of its lanes belong to it)
      const float2 ms = join(make_float2(m, sum), make_float2(-INFINITY, 0.0f), [&](float2 a, float2 b) {
        const float t = fmaxf(a.x, b.x), o = t == -INFINITY ? 0.0f : t;
        return make_float2(t, a.y * exp2_fast((a.x - o) * scale) + b.y * exp2_fast((b.x - o) * scale));
      });
      if (!ok) break;
      const float M = ms.x, S = ms.y;
      if (!(M > -INFINITY && M < INFINITY)) break;
      if (!(S > 0.0f && S < INFINITY)) break;  // a NaN among the logits
      const float inv = 1.0f / S;
      auto prob = [&](float v) { return exp2_fast((v - M) * scale) * inv; };
      const float mine = m == -INFINITY ? 0.0f : exp2_fast((m - M) * scale) * inv;
#pragma unroll
      for (int k = 0; k < HELD; ++k)
#pragma unroll
        for (int i = 0; i < 8; ++i) x[k][i] *= mine;
      if (drafted) asm volatile("cp.async.wait_all;" ::: "memory");

      float a = 1.0f, b = 0.0f;  // w = relu(a p - b q)
      float left = 1.0f;         // without draft: the sum of p over what is not rejected
      uint64_t gone = 0;         // ... and the rejected children
      for (uint64_t rest = kids; rest; rest &= rest - 1) {
        const int c = __ffsll(rest) - 1, from = c & 31;
        const int t = __shfl_sync(0xFFFFFFFFu, c < 32 ? id[0] : id[1], from);
        const float uc = __shfl_sync(0xFFFFFFFFu, c < 32 ? u[0] : u[1], from);
        const float pt = prob(value_of<T>(__shfl_sync(0xFFFFFFFFu, c < 32 ? kx[0] : kx[1], from)));
        const float qt = __uint_as_float(__shfl_sync(0xFFFFFFFFu, c < 32 ? kq[0] : kq[1], from));
        const uint64_t later = rest & (rest - 1);
        if (drafted) {
          if (uc * qt < fmaxf(a * pt - b * qt, 0.0f)) {
            next = c;
            break;
          }
          if (later) fetch(__ffsll(later) - 1);
          float z = 0.0f, q[8];
          const float b1 = b + 1.0f;
#pragma unroll
          for (int k = 0; k < HELD; ++k) {
            draft8(k, q);
#pragma unroll
            for (int i = 0; i < 8; ++i) z += fmaxf(a * x[k][i] - b1 * q[i], 0.0f);
          }
          rest_of(row, [&](int e, const float (&v)[8]) {
#pragma unroll
            for (int i = 0; i < 8; ++i)
              if (e + i < V) z += fmaxf(a * prob(v[i]) - b1 * qrow[e + i], 0.0f);
          });
          z = sum_of(z);
          if (!ok) break;
          if (z > 0.0f) {
            a = a / z;
            b = b1 / z;
          }
        } else {
          const bool same = (gone >> lane & 1 && id[0] == t) || (gone >> (lane + 32) & 1 && id[1] == t);
          const bool again = __any_sync(0xFFFFFFFFu, same);
          if (!again && uc * left < pt) {
            next = c;
            break;
          }
          if (later) fetch(__ffsll(later) - 1);
          if (again) continue;  // its weight is 0 already
          float now = left - pt;
          if (now < 0.25f) {
            float z = 0.0f;
#pragma unroll
            for (int k = 0; k < HELD; ++k)
#pragma unroll
              for (int i = 0; i < 8; ++i) z += (gt + k * stride) * 8 + i == t ? 0.0f : x[k][i];
            rest_of(row, [&](int e, const float (&v)[8]) {
#pragma unroll
              for (int i = 0; i < 8; ++i) z += e + i == t || rejected(gone, e + i) ? 0.0f : prob(v[i]);
            });
            now = sum_of(z);
            if (!ok) break;
          }
          if (now > 0.0f) {
            gone |= 1ull << c;
            left = now;
#pragma unroll
            for (int k = 0; k < HELD; ++k)
#pragma unroll
              for (int i = 0; i < 8; ++i)
                if ((gt + k * stride) * 8 + i == t) x[k][i] = 0.0f;
          }
        }
      }
      if (!ok) break;
      if (next >= 0) {
        cur = next;
        continue;
      }
      // no child: the race over w
#pragma unroll
      for (int k = 0; k < HELD; ++k) {
        if (drafted) {
          float q[8];
          draft8(k, q);
#pragma unroll
          for (int i = 0; i < 8; ++i) x[k][i] = fmaxf(a * x[k][i] - b * q[i], 0.0f);
        }
      }
      Best t{-1.0f, -1};
      auto run = [&](int e, const float (&w)[8], const float (&r)[8]) {
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          // (2 units in the last place off at most: less than the weights themselves are)
          const float v = w[i] > 0.0f ? __fdividef(w[i], r[i]) : 0.0f;
          if (v > t.w && e + i < V) t = Best{v, e + i};  // ascending: the lowest of equals
        }
      };
#pragma unroll
      for (int h = 0; h < HELD; h += 2) {
        float r[2][8];
        load_groups(race, gt + h * stride, stride, V, vec_race, 1.0f, r);
        run((gt + h * stride) * 8, x[h], r[0]);
        run((gt + (h + 1) * stride) * 8, x[h + 1], r[1]);
      }
      if (more) {
        for (int g = gt + HELD * stride; g < groups; g += stride) {
          float w[1][8], r[1][8];
          load_groups(row, g, 0, V, vec_logits, -INFINITY, w);
          load_groups(race, g, 0, V, vec_race, 1.0f, r);
#pragma unroll
          for (int i = 0; i < 8; ++i) {
            w[0][i] = prob(w[0][i]);
            if (drafted && g * 8 + i < V) w[0][i] = fmaxf(a * w[0][i] - b * qrow[g * 8 + i], 0.0f);
            if (rejected(gone, g * 8 + i)) w[0][i] = 0.0f;
          }
          run(g * 8, w[0], r[0]);
        }
      }
      token = best_of(t).i;
      break;
    }
  }
  if (writer && ok) {
    for (int i = len + lane; i < p.max_nodes; i += 32) path[i] = -1;
    if (lane == 0) {
      p.count[s] = len;
      p.token[s] = token;
    }
  }
  asm volatile("cp.async.wait_all;" ::: "memory");
  // no block ends while another may still store to its shared memory
  __syncwarp();
  asm volatile("barrier.cluster.arrive.release.aligned;" ::: "memory");
  asm volatile("barrier.cluster.wait.acquire.aligned;" ::: "memory");
  // All stores have been issued.  A block whose waits did not give up has received
  // its own; for another they land within microseconds.
  if (!ok)
    for (int i = 0; i < 50; ++i) __nanosleep(1000);
}

bool rows_aligned(const void* p, int64_t ld, size_t size) {
  return p && reinterpret_cast<uintptr_t>(p) % 16 == 0 && ld * (int64_t)size % 16 == 0;
}

template <typename T, int HELD>
cudaError_t verify_held(const VerifyParams& p, int cl, cudaStream_t stream) {
  auto* k = verify_kernel<T, HELD>;
  static int done[64];
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  if (dev >= 64 || !__atomic_load_n(&done[dev], __ATOMIC_ACQUIRE)) {
    e = cudaFuncSetAttribute(k, cudaFuncAttributeNonPortableClusterSizeAllowed, 1);
    if (e == cudaSuccess)
      e = cudaFuncSetAttribute(k, cudaFuncAttributeMaxDynamicSharedMemorySize, draft_bytes(HELD));
    if (e != cudaSuccess) return e;
    if (dev < 64) __atomic_store_n(&done[dev], 1, __ATOMIC_RELEASE);
  }
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)(p.seqs * cl));
  cfg.blockDim = dim3(kThreads);
  cfg.dynamicSmemBytes = p.draft ? draft_bytes(HELD) : 0;
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

// Blocks of a cluster: enough that their threads hold a row with 16 elements
// each, as long as all sequences' blocks run at the same time (two an SM, and
// some of a cluster's places lost to its borders); else with 32 each in half as
// many.  A vocabulary beyond 16 blocks' threads is read again for every sum.
template <typename T>
cudaError_t verify_one(const VerifyParams& p, int sms, cudaStream_t stream) {
  int cl = 1;
  while (cl < kMaxCluster && cl * kThreads * 16 < p.vocab) cl *= 2;
  const bool two = cl * kThreads * 16 >= p.vocab && (int64_t)p.seqs * cl <= 2 * sms * 7 / 8;
  if (two) return verify_held<T, 2>(p, cl, stream);
  cl = 1;
  while (cl < kMaxCluster && cl * kThreads * 32 < p.vocab) cl *= 2;
  return verify_held<T, 4>(p, cl, stream);
}

}  // namespace

cudaError_t launch_verify(const VerifyParams& p, int logits_fp32, int sms, cudaStream_t stream) {
  return logits_fp32 ? verify_one<float>(p, sms, stream) : verify_one<__half>(p, sms, stream);
}

cudaError_t read_verify_wait_timeouts(unsigned long long* count, int reset) {
  return read_local_wait_timeouts(count, reset);
}

}  // namespace nmk
