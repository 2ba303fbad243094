// logprobs.cu -- log probabilities of given tokens, the entropy and the likeliest
// tokens from rows of logits (nm_token_logprobs).
//
// A row is read once.  With c = log2(e) / T, a thread keeps for its elements a
// reference M, s = sum 2^t and a = sum 2^t t with t = (x - M) c, and its largest
// element with its chunk.  M is not the running maximum: it begins as the largest of
// the warp's first chunks and moves only when an element would exceed it by 2^4, so the
// common path has neither a branch nor a rescaling, and a loses no digits to t > 0.
// Then, in the block:
//  * the k-th largest (k = top, at least 1) of the warps' four largest thread maxima each
//    (in rows too short for k of those, of all threads' maxima: 4096 of 1700, top 32, take
//    64 us, and 315 without a bound, which lists the whole row)
//    is not above the k-th largest element, and the threads whose maximum reaches it
//    hold the k largest elements.  Those threads' chunks are read again (from L2), a
//    chunk a thread; elements that reach it are listed, and an element's place among
//    the listed is the number of larger ones.  (Where the list overflows, as in rows that
//    a grammar left few tokens, the equal elements are taken in the row's order, or the
//    k-th largest is found digit by digit.)
//  * the sums are joined relative to the largest element and without its own term:
//    the thread that holds it has its sums taken again without it.  So with R = Z - 1,
//    log p = (x - max) / T - log1p(R) is accurate where R is tiny.
// Few rows are cut into a cluster's blocks, whose lists and sums the first block joins.
// Memory bounds many rows: 2048 of 128256 (fp16, top 5) take 99 us, 5.3 TB/s, where
// reading them in this order takes 75 to 77 and the sums without the lists 85; 256
// threads and 64 registers let an SM have four rows, so that one's end is another's
// loads.  Few rows are a chain of latencies: 7.0 us for one row of 128256 (16 blocks).
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

constexpr int kThreads = 256, kWarps = kThreads / 32, kMaxCluster = 16;
constexpr int kBlocksPerSM = 4;  // by registers
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

struct Raw16 {
  uint32_t w[4];
};
struct Raw32 {
  uint32_t w[8];
};

// The row's chunks: chunk c has the elements 8 c - shift .. 8 c - shift + 7, of which the
// first and the last may lie outside the row.
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

__device__ __forceinline__ void load_whole(const __half* p, Raw16& q) {
  const uint4 u = ld_keep_v4(p);
  q.w[0] = u.x; q.w[1] = u.y; q.w[2] = u.z; q.w[3] = u.w;
}

__device__ __forceinline__ void load_whole(const float* p, Raw32& q) {
  const uint4 u = ld_keep_v4(p), v = ld_keep_v4(p + 4);
  q.w[0] = u.x; q.w[1] = u.y; q.w[2] = u.z; q.w[3] = u.w;
  q.w[4] = v.x; q.w[5] = v.y; q.w[6] = v.z; q.w[7] = v.w;
}

__device__ __forceinline__ void nothing(Raw16& q) { q.w[0] = q.w[1] = q.w[2] = q.w[3] = 0xFC00FC00u; }

__device__ __forceinline__ void nothing(Raw32& q) {
#pragma unroll
  for (int i = 0; i < 8; ++i) q.w[i] = 0xFF800000u;
}

// A chunk at the row's ends: -infinity outside.
__device__ __forceinline__ void load_end(const Row<__half>& r, int c, Raw16& q) {
  const int at = 8 * c - r.shift;
  const __half none = __ushort_as_half((unsigned short)0xFC00);
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const int a = at + 2 * i, b = a + 1;
    const __half2 h = __halves2half2(a >= 0 && a < r.vocab ? r.x[a] : none,
                                     b >= 0 && b < r.vocab ? r.x[b] : none);
    q.w[i] = *reinterpret_cast<const uint32_t*>(&h);
  }
}

__device__ __forceinline__ void load_end(const Row<float>& r, int c, Raw32& q) {
  const int at = 8 * c - r.shift;
#pragma unroll
  for (int i = 0; i < 8; ++i)
    q.w[i] = at + i >= 0 && at + i < r.vocab ? __float_as_uint(r.x[at + i]) : 0xFF800000u;
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

__device__ __forceinline__ float largest(const Raw16& q) {
  const __half2* h = reinterpret_cast<const __half2*>(q.w);
  const __half2 m = __hmax2_nan(__hmax2_nan(h[0], h[1]), __hmax2_nan(h[2], h[3]));
  return __half2float(__hmax_nan(__low2half(m), __high2half(m)));
}

__device__ __forceinline__ float largest(const Raw32& q) {
  float m = __uint_as_float(q.w[0]);
#pragma unroll
  for (int i = 1; i < 8; ++i) m = max_nan(m, __uint_as_float(q.w[i]));
  return m;
}

// t of an element: the difference first, which is exact or rounded once, as at a small
// temperature x c and M c are far larger than what is left of them (fma(x, c, -fl(M c))
// is off by half a step of M c, beyond any exponent from |M c| = 2^32 on).
__device__ __forceinline__ float difference(float x, float ref, float c) { return (x - ref) * c; }

// The same, not below kFar; NaN stays.
__device__ __forceinline__ float exponent(float x, float ref, float c) {
  return max_nan(difference(x, ref, c), kFar);
}

struct Sums {
  float s, a;
};

// The sums relative to `to` in place of `from`.
__device__ __forceinline__ Sums moved(Sums v, float from, float to, float c) {
  const float d = exponent(from, to, c), f = exp2_fast(d);
  return {v.s * f, f * fmaf(d, v.s, v.a)};
}

// A thread's running sums, of elements 2 i and of elements 2 i + 1.
struct Running {
  float2 s, a;
};

__device__ __forceinline__ float2 pair_of(const Raw16& q, int i) {
  return half2_bits_to_float2(q.w[i]);
}

__device__ __forceinline__ float2 pair_of(const Raw32& q, int i) {
  return make_float2(__uint_as_float(q.w[2 * i]), __uint_as_float(q.w[2 * i + 1]));
}

// A chunk's terms.
template <typename Raw>
__device__ __forceinline__ void add_chunk(Running& v, const Raw& q, float ref, float c) {
  const float2 c2 = make_float2(c, c), r2 = make_float2(-ref, -ref);
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const float2 x = pair_of(q, i);
    float2 t = __fmul2_rn(__fadd2_rn(x, r2), c2);
    t = make_float2(max_nan(t.x, kFar), max_nan(t.y, kFar));
    const float2 e = make_float2(exp2_fast(t.x), exp2_fast(t.y));
    v.s = __fadd2_rn(v.s, e);
    v.a = __ffma2_rn(e, t, v.a);
  }
}

// What a thread keeps.
template <typename T>
struct Kept {
  Running run;
  float M, best;
  int best_chunk;

  // U chunks, k + u * step each.
  template <int U, typename Raw>
  __device__ __forceinline__ void add(const Raw (&q)[U], int k, int step, float c) {
    float all = -INFINITY;
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const float top = largest(q[u]);
      if (top > best) {
        best = top;
        best_chunk = k + u * step;
      }
      all = u == 0 ? top : max_nan(all, top);
    }
    if (!(difference(all, M, c) <= 4.f)) {  // a far larger element, or NaN
      const float to = max_nan(all, Lowest<T>::value);
      const Sums x = moved({run.s.x, run.a.x}, M, to, c), y = moved({run.s.y, run.a.y}, M, to, c);
      run = {make_float2(x.s, y.s), make_float2(x.a, y.a)};
      M = to;
    }
#pragma unroll
    for (int u = 0; u < U; ++u) add_chunk(run, q[u], M, c);
  }
};

struct Part {  // what a block found: sums relative to max(its largest, Lowest) without one largest
  float s, a, largest;
};

constexpr int kListed = 512;  // candidates for the k largest

struct Shared {
  uint64_t top[32];                // the warps' four largest thread maxima each; the first block's
                                   // at the end: the blocks' largest
  uint64_t listed[kListed];
  uint64_t best[kMaxCluster][32];  // the blocks' k largest, descending (the first block's)
  Part part[kMaxCluster];          // (the first block's)
  uint64_t bound, head;
  uint32_t digit[256];
  float s[kWarps], a[kWarps];
  int sums[kWarps];
  uint16_t holder[kThreads];       // threads whose chunks are read again
  int holders, count;
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

// The largest key of the warp.
__device__ __forceinline__ uint64_t warp_largest(uint64_t key) {
  const uint32_t high = __reduce_max_sync(kAll, (uint32_t)(key >> 32));
  const uint32_t low = __reduce_max_sync(kAll, (uint32_t)(key >> 32) == high ? (uint32_t)key : 0u);
  return ((uint64_t)high << 32) | low;
}

// How many of n keys (a multiple of 2; 16-byte aligned) are larger than `key`.
__device__ __forceinline__ int larger(const uint64_t* keys, int n, uint64_t key) {
  int r = 0;
#pragma unroll 4
  for (int i = 0; i < n; i += 2) {
    const ulonglong2 k = *reinterpret_cast<const ulonglong2*>(keys + i);
    r += (k.x > key) + (k.y > key);
  }
  return r;
}

// The chunks of a row that a block takes: c0 .. c1 - 1, of which f0 .. f1 - 1 are whole
// (thread i has f0 + i, f0 + i + kThreads ...) and the others the row's ends.
template <typename T>
struct Range {
  Row<T> r;
  int c0, c1, f0, f1;
  __device__ Range(const LogprobsParams& p, int64_t row, int rank, int log_blocks)
      : r(static_cast<const T*>(p.logits) + row * p.ld_logits, p.vocab) {
    c0 = r.chunks * rank >> log_blocks;  // (2^21 chunks at most, 16 blocks)
    c1 = r.chunks * (rank + 1) >> log_blocks;
    f0 = c0 + (r.whole(c0) ? 0 : 1);
    f1 = c1 - (c1 - 1 >= f0 && !r.whole(c1 - 1) ? 1 : 0);
  }
};

// The K-th largest of 32 keys, one a lane, of which those that are not 0 differ (0 if
// there are fewer), and the largest.  keys: the same in shared memory.
__device__ __forceinline__ void kth_of(const uint64_t* keys, int lane, int K, uint64_t& kth, uint64_t& head) {
  const uint64_t key = keys[lane];
  const int place = larger(keys, 32, key);
  const uint32_t at = __ballot_sync(kAll, place == K - 1 && key != 0);
  const uint64_t found = __shfl_sync(kAll, key, at ? __ffs(at) - 1 : 0);
  kth = at ? found : 0;
  head = __shfl_sync(kAll, key, __ffs(__ballot_sync(kAll, place == 0)) - 1);
}

// The bound from all threads' keys (out of line: inlined it cost other rows 0.1 us).
__device__ __noinline__ void bound_by_threads(Shared& sh, uint64_t key, int owners, int K) {
  const int place = larger(sh.listed, max(owners + 1, 34) & ~1, key);
  if (key != 0 && place == K - 1) sh.bound = key;
  if (key != 0 && place == 0) sh.head = key;
}

// x, lists and sums of one block: see the head of the file.
template <typename T>
__global__ void __launch_bounds__(kThreads, kBlocksPerSM) logprobs_kernel(const LogprobsParams p, int log_blocks) {
  using Raw = typename std::conditional<sizeof(T) == 2, Raw16, Raw32>::type;
  constexpr int U = sizeof(T) == 2 ? 4 : 2;  // chunks a thread works on at a time, and has on their way
  __shared__ __align__(16) Shared sh;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int blocks = 1 << log_blocks, rank = blocks > 1 ? (int)cluster_rank() : 0;
  if (blocks > 1) cluster_arrive();  // the first block's shared memory is there from here on
  pdl_launch_dependents();
  pdl_wait_previous();
  const float c = kLog2e / p.temperature;
  const int K = p.top > 0 ? p.top : 1;
  const int64_t row = blockIdx.x >> log_blocks;
  const Range<T> g(p, row, rank, log_blocks);
  const Row<T>& r = g.r;
  const int c0 = g.c0, c1 = g.c1, f0 = g.f0, f1 = g.f1;

  // the first ids' logits, for the end
  int id = -1;
  float id_x = 0.f;
  if (rank == 0 && (int)threadIdx.x < p.n_ids) {
    id = p.ids[row * p.ld_ids + threadIdx.x];
    if (id >= 0 && id < p.vocab) id_x = (float)r.x[id];
  }

  // the row's ends go to threads 0 and 32
  const bool starts = threadIdx.x == 0 && f0 > c0, ends = threadIdx.x == 32 && f1 < c1;
  const int mine = f0 + (int)threadIdx.x;
  Kept<T> kept;
  kept.run = {make_float2(0.f, 0.f), make_float2(0.f, 0.f)};
  kept.best = -INFINITY;
  kept.best_chunk = starts ? c0 : mine < f1 ? mine : ends ? f1 : -1;  // its first
  {
    // batches that are whole for all of the warp's lanes, two at a time, one on its way
    // while the other is worked on; then what is left
    const T* at = r.x + 8 * mine - r.shift;
    constexpr int kStep = 8 * kThreads;
    const int room = f1 - (mine - lane) - 32 - (U - 1) * kThreads;
    const int full = room < 0 ? 0 : room / (U * kThreads) + 1;
    Raw q[2][U];
    auto load = [&](Raw (&to)[U]) {
#pragma unroll
      for (int u = 0; u < U; ++u) load_whole(at + u * kStep, to[u]);
      at += U * kStep;
    };
    auto load_last = [&](Raw (&to)[U], int k) {
#pragma unroll
      for (int u = 0; u < U; ++u) {
        if (k + u * kThreads < f1)
          load_whole(at + u * kStep, to[u]);
        else
          nothing(to[u]);
      }
    };
    if (full > 0)
      load(q[0]);
    else
      load_last(q[0], mine);
    float top = -INFINITY;  // the warp's reference
#pragma unroll
    for (int u = 0; u < U; ++u) top = fmaxf(top, largest(q[0][u]));
    kept.M = unordered(__reduce_max_sync(kAll, ordered(fmaxf(top, Lowest<T>::value))));
    if (starts) {
      Raw one[1];
      load_end(r, c0, one[0]);
      kept.template add<1>(one, c0, 0, c);
    }
    int k = mine;
    if (full == 0) {
      kept.template add<U>(q[0], k, kThreads, c);
    } else {
      for (int b = 0;;) {
        if (++b < full) load(q[1]); else load_last(q[1], k + U * kThreads);
        kept.template add<U>(q[0], k, kThreads, c);
        k += U * kThreads;
        if (b >= full) {
          kept.template add<U>(q[1], k, kThreads, c);
          break;
        }
        if (++b < full) load(q[0]); else load_last(q[0], k + U * kThreads);
        kept.template add<U>(q[1], k, kThreads, c);
        k += U * kThreads;
        if (b >= full) {
          kept.template add<U>(q[0], k, kThreads, c);
          break;
        }
      }
    }
    if (ends) {
      Raw one[1];
      load_end(r, f1, one[0]);
      kept.template add<1>(one, f1, 0, c);
    }
  }
  const Sums v = {kept.run.s.x + kept.run.s.y, kept.run.a.x + kept.run.a.y};

  // a lower bound of the K-th largest key: the K-th of the warps' four largest, or of all
  // threads' where those are fewer than K (short rows)
  const uint64_t key = kept.best_chunk >= 0 ? key_of(kept.best, (uint32_t)kept.best_chunk) : 0;
  const int owners = f1 - f0;  // threads that have a whole chunk, and possibly 0 and 32
  const bool by_threads = K > 4 * (owners / 32) + min(owners % 32, 4);
  if (by_threads) {
    sh.listed[threadIdx.x] = key;
    if (threadIdx.x == 0) sh.bound = 0;
  } else {
    uint64_t left = key;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const uint64_t top = warp_largest(left);
      if (lane == 0) sh.top[warp * 4 + i] = top;
      if (left == top) left = 0;
    }
  }
  if (threadIdx.x == 0) {
    sh.holders = 1;  // (the first is the owner)
    sh.count = 0;
  }
  const bool spoilt = __syncthreads_or(v.s != v.s);
  if (by_threads) {
    bound_by_threads(sh, key, owners, K);
  } else if (warp == 0) {
    uint64_t kth, head;
    kth_of(sh.top, lane, K, kth, head);
    if (lane == 0) {
      sh.bound = kth;
      sh.head = head;
    }
  }
  __syncthreads();
  const uint64_t bound = sh.bound, head = sh.head;
  const float top_x = head ? unordered((uint32_t)(head >> 32)) : -INFINITY;
  const float m = fmaxf(top_x, Lowest<T>::value);
  // (a row that has no distribution has no list either)
  const bool hopeless = blocks == 1 && (spoilt || !(fabsf(top_x) < INFINITY));
  int count = 0;
  Sums w = {0.f, 0.f};
  if (key != head && key != 0) w = moved(v, kept.M, m, c);  // the owner's are taken again without its largest
  if (!hopeless) {
    // The owner comes first, so that its sums are always added by the same threads; the
    // others come as they come, which decides nothing.
    if (key != 0 && key >= bound)
      sh.holder[key == head ? 0 : atomicAdd(&sh.holders, 1)] = (uint16_t)threadIdx.x;
    __syncthreads();

    // their chunks, one a thread, and the row's ends
    const int each = (f1 - f0 + kThreads - 1) / kThreads, items = sh.holders * each;
    const int owner_chunk = (int)~(uint32_t)head, owner = head ? (int)sh.holder[0] : -1;
    // calls f_chunk(k, x, holder) for the holders' chunks
    auto visit = [&](auto&& f_chunk) {
      for (int i = threadIdx.x; i < items + 2; i += kThreads) {
        const int e = i - items;
        const int holder = e < 0 ? (int)sh.holder[i / each] : 32 * e;
        const int k = e < 0 ? f0 + holder + i % each * kThreads : e == 0 ? c0 : f1;
        if (e < 0 ? k >= f1 : e == 0 ? f0 == c0 : f1 == c1) continue;
        Raw q;
        if (e < 0)
          load_whole(r.x + 8 * k - r.shift, q);
        else
          load_end(r, k, q);
        float x[8];
        elements(q, x);
        f_chunk(k, x, holder);
      }
    };
    auto list = [&](float x, int at) {
      const int to = atomicAdd(&sh.count, 1);
      if (to < kListed) sh.listed[to] = key_of(x, (uint32_t)at);
    };
    const uint32_t least = (uint32_t)(bound >> 32);
    visit([&](int k, const float (&x)[8], int holder) {
      if (holder == owner) {
        bool skipped = false;
#pragma unroll
        for (int e = 0; e < 8; ++e) {
          if (k == owner_chunk && !skipped && x[e] == top_x) {
            skipped = true;  // its largest, once
          } else {
            const float t = exponent(x[e], m, c), y = exp2_fast(t);
            w.s += y;
            w.a = fmaf(y, t, w.a);
          }
        }
      }
      // elements of the bound's value count up to its chunk
      const uint32_t low = (uint32_t)k <= ~(uint32_t)bound ? least : least + 1;
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        const int at = 8 * k - r.shift + e;
        if (ordered(x[e]) >= low && at >= 0 && at < r.vocab) list(x[e], at);
      }
    });
    __syncthreads();
    count = sh.count;
    if (count > kListed) {  // (the same for all threads)
      // Very many elements of the bound's value: those above it, and then the first of
      // its value in the row's order.
      __syncthreads();
      if (threadIdx.x == 0) sh.count = 0;
      __syncthreads();
      visit([&](int k, const float (&x)[8], int) {
#pragma unroll
        for (int e = 0; e < 8; ++e) {
          const int at = 8 * k - r.shift + e;
          if (ordered(x[e]) > least && at >= 0 && at < r.vocab) list(x[e], at);
        }
      });
      __syncthreads();
      count = sh.count;
      if (count > kListed) {
        // Very many above it too (one thread's chunks, say): the K-th largest key digit
        // by digit, then those that reach it.
        uint64_t prefix = 0;
        int left = K;
        for (int shift = 56; shift >= 0; shift -= 8) {
          for (int i = threadIdx.x; i < 256; i += kThreads) sh.digit[i] = 0;
          __syncthreads();
          visit([&](int k, const float (&x)[8], int) {
#pragma unroll
            for (int e = 0; e < 8; ++e) {
              const int at = 8 * k - r.shift + e;
              if (at < 0 || at >= r.vocab) continue;
              const uint64_t y = key_of(x[e], (uint32_t)at);
              if (shift == 56 || (y >> (shift + 8)) == (prefix >> (shift + 8)))
                atomicAdd(&sh.digit[(y >> shift) & 255], 1u);
            }
          });
          __syncthreads();
          int d = 255;
          for (; d > 0 && (int)sh.digit[d] < left; --d) left -= (int)sh.digit[d];
          prefix |= (uint64_t)d << shift;
          __syncthreads();
        }
        if (threadIdx.x == 0) sh.count = 0;
        __syncthreads();
        visit([&](int k, const float (&x)[8], int) {
#pragma unroll
          for (int e = 0; e < 8; ++e) {
            const int at = 8 * k - r.shift + e;
            if (at >= 0 && at < r.vocab && key_of(x[e], (uint32_t)at) >= prefix) list(x[e], at);
          }
        });
        __syncthreads();
        count = sh.count;
      } else {
        for (int base = c0; base < c1 && count < K; base += kThreads) {
          const int k = base + (int)threadIdx.x;
          Raw q;
          if (k >= c1)
            nothing(q);
          else if (k >= f0 && k < f1)
            load_whole(r.x + 8 * k - r.shift, q);
          else
            load_end(r, k, q);
          float x[8];
          elements(q, x);
          uint32_t equal = 0;
#pragma unroll
          for (int e = 0; e < 8; ++e) {
            const int at = 8 * k - r.shift + e;
            if (k < c1 && ordered(x[e]) == least && at >= 0 && at < r.vocab) equal |= 1u << e;
          }
          int before = __popc(equal);  // how many there are in earlier chunks
#pragma unroll
          for (int o = 1; o < 32; o <<= 1) {
            const int n = __shfl_up_sync(kAll, before, o);
            if (lane >= o) before += n;
          }
          if (lane == 31) sh.sums[warp] = before;
          before -= __popc(equal);
          __syncthreads();
          int all = 0;
          for (int i = 0; i < kWarps; ++i) {
            if (i < warp) before += sh.sums[i];
            all += sh.sums[i];
          }
#pragma unroll
          for (int e = 0; e < 8; ++e)
            if (equal >> e & 1) {
              if (count + before < K) sh.listed[count + before] = key_of(x[e], (uint32_t)(8 * k - r.shift + e));
              ++before;
            }
          count = count + all < K ? count + all : K;
          __syncthreads();
        }
      }
    }
  }
  w.s = warp_sum(w.s);
  w.a = warp_sum(w.a);
  if (lane == 0) {
    sh.s[warp] = w.s;
    sh.a[warp] = w.a;
  }
  if ((count & 1) && threadIdx.x == 0) sh.listed[count] = 0;
  __syncwarp();

  // the block's K largest and its part, in the first block's shared memory
  if (blocks > 1) cluster_wait();
  __syncthreads();
  auto best = [&](int i, uint64_t y) {
    if (blocks == 1)
      sh.best[0][i] = y;
    else
      asm volatile("st.shared::cluster.u64 [%0], %1;" ::"r"(in_first_block(&sh.best[rank][i])), "l"(y) : "memory");
  };
  if ((int)threadIdx.x >= count && threadIdx.x < 32) best(threadIdx.x, 0);
  for (int i = threadIdx.x; i < count; i += kThreads) {
    const uint64_t y = sh.listed[i];
    const int place = larger(sh.listed, (count + 1) & ~1, y);
    if (place < 32) best(place, y);
  }
  if (warp == kWarps - 1) {
    const float s = warp_sum(lane < kWarps ? sh.s[lane] : 0.f), a = warp_sum(lane < kWarps ? sh.a[lane] : 0.f);
    if (blocks == 1) {
      if (lane == 0) sh.part[0] = {s, a, top_x};
    } else if (lane < 3) {
      asm volatile("st.shared::cluster.f32 [%0], %1;" ::"r"(in_first_block(&sh.part[rank].s + lane)),
                   "f"(lane == 0 ? s : lane == 1 ? a : top_x) : "memory");
    }
  }
  __syncwarp();
  if (blocks > 1) {
    cluster_arrive();
    cluster_wait();
    if (rank != 0) return;
  } else {
    __syncthreads();
  }

  // the first block joins them: the sums, every warp for itself
  int holds = 0;
  for (int b = 1; b < blocks; ++b)
    if (sh.best[b][0] > sh.best[holds][0]) holds = b;
  const float x_max = sh.part[holds].largest;
  float R = 0.f, A = 0.f;
  for (int b = 0; b < blocks; ++b) {
    const Part q = sh.part[b];
    Sums z = {q.s, q.a};
    if (b != holds && q.largest != -INFINITY) z.s += 1.f;
    z = moved(z, fmaxf(q.largest, Lowest<T>::value), x_max, c);
    R += z.s;
    A += z.a;
  }
  const bool valid = fabsf(x_max) < INFINITY && R == R && !(blocks == 1 && spoilt);
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
  if (p.top == 0) return;
  auto answer = [&](int place, uint64_t y) {
    p.top_ids[row * p.top + place] = valid ? (int32_t)~(uint32_t)y : -1;
    p.top_logprob[row * p.top + place] =
        valid ? (unordered((uint32_t)(y >> 32)) - x_max) / p.temperature - log_z : NAN;
  };
  if (blocks == 1 || !valid) {
    if ((int)threadIdx.x < p.top) answer(threadIdx.x, sh.best[0][threadIdx.x]);
    return;
  }
  // the largest of the blocks' lists: a lower bound again, and the places of those that reach it
  if (warp == 0) {
    const int per = 32 >> log_blocks;
    sh.top[lane] = sh.best[lane / per][lane % per];
    __syncwarp();
    uint64_t kth, unused;
    kth_of(sh.top, lane, K, kth, unused);
    if (lane == 0) {
      sh.bound = kth;
      sh.count = 0;
    }
  }
  __syncthreads();
  for (int i = threadIdx.x; i < blocks * 32; i += kThreads) {
    const uint64_t y = sh.best[i >> 5][i & 31];
    if (y != 0 && y >= sh.bound) sh.listed[atomicAdd(&sh.count, 1)] = y;  // (512 at most)
  }
  __syncthreads();
  count = sh.count;
  if ((count & 1) && threadIdx.x == 0) sh.listed[count] = 0;
  __syncthreads();
  for (int i = threadIdx.x; i < count; i += kThreads) {
    const uint64_t y = sh.listed[i];
    const int place = larger(sh.listed, (count + 1) & ~1, y);
    if (place < p.top) answer(place, y);
  }
}

template <typename T>
cudaError_t launch_t(const LogprobsParams& p, int sms, cudaStream_t stream) {
  // blocks a row: the most that still fit the SMs at once and have a chunk a thread
  int log_blocks = 0;
  while ((1 << log_blocks) < kMaxCluster && p.rows * (2 << log_blocks) <= kBlocksPerSM * sms &&
         p.vocab >= (2 << log_blocks) * kThreads * 8)
    ++log_blocks;
  const int blocks = 1 << log_blocks;
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
  return cudaLaunchKernelEx(&cfg, k, p, log_blocks);
}

}  // namespace

cudaError_t launch_logprobs(const LogprobsParams& p, int logits_fp32, int sms, cudaStream_t stream) {
  return logits_fp32 ? launch_t<float>(p, sms, stream) : launch_t<__half>(p, sms, stream);
}

}  // namespace nmk
