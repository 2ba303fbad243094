// logprobs.cu -- log probabilities of given tokens, the entropy and the likeliest
// tokens from rows of logits (nm_token_logprobs).
//
// A row is read once.  With c = log2(e) / T, a thread keeps for its elements a
// reference M, s = sum 2^t and a = sum 2^t t with t = (x - M) c, and the largest
// element with its chunk; M is not the running maximum but a chunk's maximum that is
// only moved when an element would exceed it by 2^64, so that the common path has
// neither a branch nor a rescaling.  Then, in the block:
//  * the k threads with the largest maxima (k = top, at least 1) hold the k largest
//    elements: an element of another thread is below k maxima.  A warp reads those
//    threads' elements again (from L2) and keeps the best 32 in its lanes;
//  * the sums are joined relative to the largest element and without its own term:
//    the thread that holds it has its sums taken again without it.  So with R = Z - 1,
//    log p = (x - max) / T - log1p(R) is accurate where R is tiny.
// Few rows are cut into a cluster's blocks, whose lists and sums the first block joins.
// Elements are taken in chunks of 8 from the 16-byte boundary at or before the row's
// start, so rows of any alignment are read by whole vectors but for their two ends.
#include <cuda_fp16.h>
#include <cuda_runtime.h>
#include <math.h>
#include <stdint.h>

#include <type_traits>

#include "device.cuh"
#include "kernels.h"
#include "layer.h"

namespace nmk {
namespace {

constexpr int kThreads = 512, kWarps = kThreads / 32, kMaxCluster = 16;
constexpr uint32_t kAll = 0xFFFFFFFFu;
constexpr float kFar = -10000.f;  // 2^kFar is 0; keeps 0 * t from being 0 * infinity

__device__ __forceinline__ float max_nan(float a, float b) {
  float r;
  asm("max.NaN.f32 %0, %1, %2;" : "=f"(r) : "f"(a), "f"(b));
  return r;
}

template <typename T>
struct Lowest;
template <>
struct Lowest<__half> {
  static constexpr float value = -65504.f;
};
template <>
struct Lowest<float> {
  static constexpr float value = -3.402823466e38f;
};

// Order of floats as unsigned integers (-0 and +0 equal); above 0 for any number.
__device__ __forceinline__ uint32_t ordered(float x) {
  const uint32_t u = __float_as_uint(x + 0.f);
  return (u & 0x80000000u) ? ~u : (u | 0x80000000u);
}

__device__ __forceinline__ float unordered(uint32_t o) {
  return __uint_as_float((o & 0x80000000u) ? (o & 0x7FFFFFFFu) : ~o);
}

// Larger keys first: a larger value, then a lower index.  0: nothing.
__device__ __forceinline__ uint64_t key_of(float x, uint32_t at) {
  return ((uint64_t)ordered(x) << 32) | (uint32_t)~at;
}

__device__ __forceinline__ uint64_t shfl64(uint64_t v, int src) { return __shfl_sync(kAll, v, src); }

// Descending sort of a bitonic sequence across the lanes.
__device__ __forceinline__ uint64_t merge_lanes(uint64_t v, int lane) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) {
    const uint64_t w = __shfl_xor_sync(kAll, v, o);
    const bool keep_large = (lane & o) == 0;
    v = (keep_large == (v > w)) ? v : w;
  }
  return v;
}

__device__ __forceinline__ uint64_t sort_lanes(uint64_t v, int lane) {
#pragma unroll
  for (int size = 2; size <= 32; size <<= 1)
#pragma unroll
    for (int o = size >> 1; o > 0; o >>= 1) {
      const uint64_t w = __shfl_xor_sync(kAll, v, o);
      const bool descending = (lane & size) == 0 || size == 32;
      const bool keep_large = ((lane & o) == 0) == descending;
      v = (keep_large == (v > w)) ? v : w;
    }
  return v;
}

// The best 32 of two descending lists, descending.
__device__ __forceinline__ uint64_t join_lists(uint64_t a, uint64_t b, int lane) {
  const uint64_t r = shfl64(b, 31 - lane);
  return merge_lanes(a > r ? a : r, lane);
}

// The best 32 of the warps' lists in list[0] (a power of two of them).
__device__ __forceinline__ void join_warps(uint64_t (*list)[32], uint64_t mine, int warp, int lane) {
  list[warp][lane] = mine;
#pragma unroll 1
  for (int half = kWarps / 2; half > 0; half >>= 1) {
    __syncthreads();
    if (warp < half) list[warp][lane] = join_lists(list[warp][lane], list[warp + half][lane], lane);
  }
  __syncthreads();
}

// The row's chunks: chunk c has the elements 8 c - shift .. 8 c - shift + 7.
template <typename T>
struct Row {
  const T* x;
  int shift, vocab, chunks;
  __device__ Row(const T* row, int v) : x(row), vocab(v) {
    shift = (int)((reinterpret_cast<uintptr_t>(row) & 15) / sizeof(T));
    chunks = (int)((vocab + shift + 7) / 8);
  }
  __device__ __forceinline__ bool whole(int c) const {
    return 8 * c >= shift && 8 * c - shift + 8 <= vocab;
  }
};

struct Raw16 {
  uint32_t w[4];
};
struct Raw32 {
  uint32_t w[8];
};

__device__ __forceinline__ void load_chunk(const Row<__half>& r, int c, Raw16& q) {
  const int at = 8 * c - r.shift;
  if (r.whole(c)) {
    const uint4 u = ld_keep_v4(r.x + at);
    q.w[0] = u.x; q.w[1] = u.y; q.w[2] = u.z; q.w[3] = u.w;
  } else {
    const __half none = __ushort_as_half((unsigned short)0xFC00);  // -infinity
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const int a = at + 2 * i, b = a + 1;
      const __half2 h = __halves2half2(a >= 0 && a < r.vocab ? r.x[a] : none,
                                       b >= 0 && b < r.vocab ? r.x[b] : none);
      q.w[i] = *reinterpret_cast<const uint32_t*>(&h);
    }
  }
}

__device__ __forceinline__ void load_chunk(const Row<float>& r, int c, Raw32& q) {
  const int at = 8 * c - r.shift;
  if (r.whole(c)) {
    const uint4 u = ld_keep_v4(r.x + at), v = ld_keep_v4(r.x + at + 4);
    q.w[0] = u.x; q.w[1] = u.y; q.w[2] = u.z; q.w[3] = u.w;
    q.w[4] = v.x; q.w[5] = v.y; q.w[6] = v.z; q.w[7] = v.w;
  } else {
#pragma unroll
    for (int i = 0; i < 8; ++i)
      q.w[i] = at + i >= 0 && at + i < r.vocab ? __float_as_uint(r.x[at + i]) : 0xFF800000u;
  }
}

__device__ __forceinline__ void elements(const Raw16& q, float (&x)[8]) {
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const float2 f = half2_bits_to_float2(q.w[i]);
    x[2 * i] = f.x;
    x[2 * i + 1] = f.y;
  }
}

__device__ __forceinline__ void elements(const Raw32& q, float (&x)[8]) {
#pragma unroll
  for (int i = 0; i < 8; ++i) x[i] = __uint_as_float(q.w[i]);
}

__device__ __forceinline__ float largest(const Raw16& q, const float (&)[8]) {
  const __half2* h = reinterpret_cast<const __half2*>(q.w);
  const __half2 m = __hmax2_nan(__hmax2_nan(h[0], h[1]), __hmax2_nan(h[2], h[3]));
  return __half2float(__hmax_nan(__low2half(m), __high2half(m)));
}

__device__ __forceinline__ float largest(const Raw32&, const float (&x)[8]) {
  float m = x[0];
#pragma unroll
  for (int i = 1; i < 8; ++i) m = max_nan(m, x[i]);
  return m;
}

// References are kept as the exponents subtract them: fp16 rows as fl(M c), so that a
// thread's t = x c - fl(M c) is one fused operation (finite for finite x) and what the
// rounding of M c adds to every t is taken out at the end; fp32 rows as M, with
// t = (x - M) c, since their x c may overflow.
template <typename T>
__device__ __forceinline__ float reference(float x, float c) {
  return sizeof(T) == 2 ? __fmul_rn(x, c) : x;  // (not fused into what uses it)
}

template <typename T>
__device__ __forceinline__ float difference(float x, float ref, float c) {
  return sizeof(T) == 2 ? fmaf(x, c, -ref) : (x - ref) * c;
}

// t of an element, not below kFar; NaN stays.
template <typename T>
__device__ __forceinline__ float exponent(float x, float ref, float c) {
  return max_nan(difference<T>(x, ref, c), kFar);
}

struct Sums {
  float s, a;
};

// The sums with every t moved by d.
__device__ __forceinline__ Sums shifted(Sums v, float d) {
  d = max_nan(d, kFar);
  const float f = exp2_fast(d);
  return {v.s * f, f * fmaf(d, v.s, v.a)};
}

// The sums relative to `to` in place of `from`.
template <typename T>
__device__ __forceinline__ Sums moved(Sums v, float from, float to, float c) {
  return shifted(v, sizeof(T) == 2 ? from - to : (from - to) * c);
}

struct Part {  // what a block found: sums relative to max(its largest, Lowest) without one largest
  float s, a, largest;
};

struct Shared {
  uint64_t list[kWarps][32];       // the warps' best
  uint64_t from[kMaxCluster][32];  // the first block: the blocks' best
  Part part[kMaxCluster];
  float s[kWarps], a[kWarps];
  float owner_s, owner_a;
};

__device__ __forceinline__ uint32_t cluster_rank() {
  uint32_t r;
  asm volatile("mov.u32 %0, %%cluster_ctarank;" : "=r"(r));
  return r;
}

__device__ __forceinline__ void cluster_arrive() {
  asm volatile("barrier.cluster.arrive.release.aligned;" ::: "memory");
}

__device__ __forceinline__ void cluster_wait() {
  asm volatile("barrier.cluster.wait.acquire.aligned;" ::: "memory");
}

__device__ __forceinline__ uint32_t in_first_block(const void* p) {
  uint32_t r;
  asm("mapa.shared::cluster.u32 %0, %1, 0;" : "=r"(r) : "r"(smem_addr(p)));
  return r;
}

template <typename T>
__global__ void __launch_bounds__(kThreads, 2) logprobs_kernel(const LogprobsParams p, int blocks) {
  using Raw = typename std::conditional<sizeof(T) == 2, Raw16, Raw32>::type;
  constexpr int U = sizeof(T) == 2 ? 4 : 2;  // chunks in flight a thread
  __shared__ Shared sh;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int64_t row = blockIdx.x / (unsigned)blocks;
  const int rank = blocks > 1 ? (int)cluster_rank() : 0;
  if (blocks > 1) cluster_arrive();  // the first block's shared memory is there from here on
  pdl_launch_dependents();
  pdl_wait_previous();
  const Row<T> r(static_cast<const T*>(p.logits) + row * p.ld_logits, p.vocab);
  const int c0 = (int)((int64_t)r.chunks * rank / blocks), c1 = (int)((int64_t)r.chunks * (rank + 1) / blocks);
  const float c = kLog2e / p.temperature;
  const int K = p.top > 0 ? p.top : 1;

  // the first ids' logits, for the end
  int id = -1;
  float id_x = 0.f;
  if (rank == 0 && (int)threadIdx.x < p.n_ids) {
    id = p.ids[row * p.ld_ids + threadIdx.x];
    if (id >= 0 && id < p.vocab) id_x = (float)r.x[id];
  }

  float M = -INFINITY, best = -INFINITY;
  int best_chunk = c0 + (int)threadIdx.x;
  Sums v = {0.f, 0.f};
  for (int k = c0 + (int)threadIdx.x; k < c1; k += U * kThreads) {
    Raw q[U];
#pragma unroll
    for (int u = 0; u < U; ++u)
      if (k + u * kThreads < c1) load_chunk(r, k + u * kThreads, q[u]);
#pragma unroll
    for (int u = 0; u < U; ++u) {
      if (k + u * kThreads >= c1) break;
      float x[8];
      elements(q[u], x);
      const float top = largest(q[u], x);
      if (top > best) {
        best = top;
        best_chunk = k + u * kThreads;
      }
      if (!(difference<T>(top, M, c) <= 64.f)) {  // the first chunk, a far larger element, NaN
        const float to = reference<T>(max_nan(top, Lowest<T>::value), c);
        v = moved<T>(v, M, to, c);
        M = to;
      }
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        const float t = exponent<T>(x[i], M, c), e = exp2_fast(t);
        v.s += e;
        v.a = fmaf(e, t, v.a);
      }
    }
  }

  // the threads with the K largest maxima
  const uint64_t mine = c0 + (int)threadIdx.x < c1 ? key_of(best, best_chunk) : 0;
  join_warps(sh.list, sort_lanes(mine, lane), warp, lane);
  const uint64_t head = sh.list[0][0];
  const float top_x = head ? unordered((uint32_t)(head >> 32)) : -INFINITY;
  const float m = reference<T>(fmaxf(top_x, Lowest<T>::value), c);
  Sums w = {0.f, 0.f};
  if (mine != head) w = moved<T>(v, M, m, c);  // the owner's are taken again without its largest
  w.s = warp_sum(w.s);
  w.a = warp_sum(w.a);
  if (lane == 0) {
    sh.s[warp] = w.s;
    sh.a[warp] = w.a;
  }
  const uint32_t least = (uint32_t)(sh.list[0][K - 1] >> 32);
  uint64_t held[2];  // the threads this warp looks at
#pragma unroll
  for (int i = 0; i < 2; ++i) held[i] = warp + i * kWarps < K ? sh.list[0][warp + i * kWarps] : 0;
  __syncthreads();  // the list is used again

  // their elements, the best 32 in the lanes
  uint64_t list = 0;
#pragma unroll 1
  for (int i = 0; i < 2; ++i) {
    if (!held[i]) break;
    const int chunk = (int)~(uint32_t)held[i];
    const bool owner = warp == 0 && i == 0;
    Sums own = {0.f, 0.f};
    const int first = c0 + (chunk - c0) % kThreads;
#pragma unroll 1
    for (int k0 = first; k0 < c1; k0 += 32 * kThreads) {
      const int k = k0 + lane * kThreads;
      float x[8];
      if (k < c1) {
        Raw q;
        load_chunk(r, k, q);
        elements(q, x);
      }
      bool skipped = false;
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        const int at = 8 * k - r.shift + e;
        const bool real = k < c1 && at >= 0 && at < r.vocab;
        if (owner && real) {
          if (k == chunk && !skipped && x[e] == top_x) {
            skipped = true;  // its largest, once
          } else {
            const float t = exponent<T>(x[e], m, c), y = exp2_fast(t);
            own.s += y;
            own.a = fmaf(y, t, own.a);
          }
        }
        const uint64_t key = real ? key_of(x[e], (uint32_t)at) : 0;
        bool wants = real && (uint32_t)(key >> 32) >= least;
        uint64_t last = shfl64(list, K - 1);
        uint32_t who = __ballot_sync(kAll, wants && key > last);
        while (who) {
          const int src = __ffs(who) - 1;
          const uint64_t in = shfl64(key, src);
          const int place = __popc(__ballot_sync(kAll, list > in));
          const uint64_t up = __shfl_up_sync(kAll, list, 1);
          list = lane < place ? list : lane == place ? in : up;
          if (lane == src) wants = false;
          last = shfl64(list, K - 1);
          who = __ballot_sync(kAll, wants && key > last);
        }
      }
    }
    if (owner) {
      own.s = warp_sum(own.s);
      own.a = warp_sum(own.a);
      if (lane == 0) {
        sh.owner_s = own.s;
        sh.owner_a = own.a;
      }
    }
  }
  if (!head && threadIdx.x == 0) sh.owner_s = sh.owner_a = 0.f;
  join_warps(sh.list, list, warp, lane);

  // the block's part, to the first block
  if (blocks > 1) cluster_wait();
  if (warp == 0) {
    const float s = warp_sum(lane < kWarps ? sh.s[lane] : 0.f) + sh.owner_s;
    const float a = warp_sum(lane < kWarps ? sh.a[lane] : 0.f) + sh.owner_a;
    if (blocks == 1) {
      sh.from[0][lane] = sh.list[0][lane];
      if (lane == 0) sh.part[0] = {s, a, top_x};
    } else {
      asm volatile("st.shared::cluster.u64 [%0], %1;" ::"r"(in_first_block(&sh.from[rank][lane])),
                   "l"(sh.list[0][lane]) : "memory");
      const float f = lane == 0 ? s : lane == 1 ? a : top_x;
      if (lane < 3)
        asm volatile("st.shared::cluster.f32 [%0], %1;" ::"r"(in_first_block(&sh.part[rank].s + lane)),
                     "f"(f) : "memory");
    }
  }
  __syncwarp();
  if (blocks > 1) {
    cluster_arrive();
    if (rank != 0) {
      cluster_wait();
      return;
    }
    cluster_wait();
  } else {
    __syncthreads();
  }

  // the first block joins them: every warp for itself
  uint64_t all = sh.from[0][lane];
  int owner = 0;
  for (int b = 1; b < blocks; ++b) {
    if (sh.from[b][0] > sh.from[owner][0]) owner = b;
    all = join_lists(all, sh.from[b][lane], lane);
  }
  const float x_max = sh.part[owner].largest, ref = reference<T>(x_max, c);
  float R = 0.f, A = 0.f;
  for (int b = 0; b < blocks; ++b) {
    const Part q = sh.part[b];
    Sums z = {q.s, q.a};
    if (b != owner && q.largest != -INFINITY) z.s += 1.f;
    z = moved<T>(z, reference<T>(fmaxf(q.largest, Lowest<T>::value), c), ref, c);
    R += z.s;
    A += z.a;
  }
  if (sizeof(T) == 2) {  // t relative to max c itself
    const Sums z = shifted({R, A}, -fmaf(x_max, c, -ref));
    R = z.s;
    A = z.a;
  }
  const bool valid = fabsf(x_max) < INFINITY && R == R;
  const float log_z = log1pf(R);
  for (int j = threadIdx.x; j < p.n_ids; j += kThreads) {
    if (j != (int)threadIdx.x) {
      id = p.ids[row * p.ld_ids + j];
      if (id >= 0 && id < p.vocab) id_x = (float)r.x[id];
    }
    const float lp = id >= 0 && id < p.vocab ? (id_x - x_max) / p.temperature - log_z : -INFINITY;
    p.logprob[row * p.n_ids + j] = valid ? lp : NAN;
  }
  if (threadIdx.x == 0 && p.entropy)
    p.entropy[row] = valid ? log_z - 0.69314718055994531f * (A / (1.f + R)) : NAN;
  if (warp == 0 && lane < p.top) {
    const float x = unordered((uint32_t)(all >> 32));
    p.top_ids[row * p.top + lane] = valid ? (int32_t)~(uint32_t)all : -1;
    p.top_logprob[row * p.top + lane] = valid ? (x - x_max) / p.temperature - log_z : NAN;
  }
}

template <typename T>
cudaError_t launch_t(const LogprobsParams& p, int sms, cudaStream_t stream) {
  // blocks a row: the most that still fit two blocks an SM and have a chunk a thread
  int blocks = 1;
  while (blocks < kMaxCluster && p.rows * blocks * 2 <= 2 * sms && p.vocab >= blocks * 2 * kThreads * 8) blocks *= 2;
  auto* k = logprobs_kernel<T>;
  static int done[64] = {0};
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  if (dev >= 64 || !__atomic_load_n(&done[dev], __ATOMIC_ACQUIRE)) {
    e = cudaFuncSetAttribute(k, cudaFuncAttributeNonPortableClusterSizeAllowed, 1);
    if (e != cudaSuccess) return e;
    if (dev < 64) __atomic_store_n(&done[dev], 1, __ATOMIC_RELEASE);
  }
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)(p.rows * blocks));
  cfg.blockDim = dim3(kThreads);
  cfg.stream = stream;
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  attr[1].id = cudaLaunchAttributeClusterDimension;
  attr[1].val.clusterDim.x = (unsigned)blocks;
  attr[1].val.clusterDim.y = attr[1].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = blocks > 1 ? 2 : 1;
  return cudaLaunchKernelEx(&cfg, k, p, blocks);
}

}  // namespace

cudaError_t launch_logprobs(const LogprobsParams& p, int logits_fp32, int sms, cudaStream_t stream) {
  return logits_fp32 ? launch_t<float>(p, sms, stream) : launch_t<__half>(p, sms, stream);
}

}  // namespace nmk
