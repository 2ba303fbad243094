// attend.cuh -- what the attention kernels share: the split of the work over
// the blocks, the addresses of cache rows, and the joining of partial sums.
//
// Work split.  An item is a sequence, a key head and a tile of query rows (row
// r of a sequence and key head is node r / G, query head h G + r % G, G query
// heads sharing the key head).  An item's positions are cut into units; the
// units of all items, one after the other, are cut evenly over the blocks
// (lengths are known on the device only, and the longest sequence must not
// decide).  So a block has some items whole, and at its range's two ends parts
// of items.  Where there are at least two blocks an item, an item's last block is
// left short instead, so that no block has two items (a second one costs a block
// its start-up again: 3 to 5 us).  A part is stored as unnormalised sums with their maxima in the
// block's slot, and the block that completes an item's count of parts joins
// them in block order: the result does not depend on which block that is.
#pragma once

#include <cuda_fp16.h>
#include <stdint.h>

#include "decode.h"
#include "device.cuh"

namespace nmk {

constexpr float kLn2 = 0.6931471805599453f;

__device__ __forceinline__ float log2_fast(float x) {
  float y;
  asm("lg2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}

// r / G for query rows (r < 2^13, 1 <= G <= 64) by a multiplication.
struct Heads {
  uint32_t g, inv;
  __device__ __forceinline__ explicit Heads(int heads) : g(heads), inv(0xFFFFFFFFu / heads + 1u) {}
  __device__ __forceinline__ int node(int r) const { return g == 1 ? r : (int)__umulhi(r, inv); }
  __device__ __forceinline__ int head(int r) const { return r - node(r) * (int)g; }
};

// A sequence's rows and positions.
struct SeqInfo {
  int first;    // its first token
  int n;        // nodes
  int64_t ctx;  // context positions
  int64_t len;  // positions that can be seen by some node
};

__device__ __forceinline__ SeqInfo seq_info(const AttendParams& p, int s) {
  SeqInfo i;
  i.first = max(p.q_start[s], 0);
  i.n = max(0, min(min(max(p.q_start[s + 1], 0), p.tokens) - i.first, p.max_nodes));
  i.ctx = max(p.ctx_len[s], 0);
  i.len = min(i.ctx + i.n, p.table_cols << p.c.page_shift);
  return i;
}

struct Span {        // a part of an item that a block has: units u0 .. u1 - 1 of nu
  int s, h, rt;      // sequence, key head, row tile
  int u0, u1, nu;
  int64_t start;     // the item's first unit among all units
  int64_t item;      // its number among all items, counting row tiles to RT_MAX each
};

// a / b for 0 <= a, 0 < b: a 64-bit division is some hundred instructions, and
// in nearly every call both numbers fit 32 bits.
__device__ __forceinline__ int64_t div_units(int64_t a, int64_t b) {
  if ((((uint64_t)a | (uint64_t)b) >> 32) == 0) return (uint32_t)a / (uint32_t)b;
  return a / b;
}

// The block's range of units, and the walk over its items.
//   ROWS: rows of a tile;  UK: positions of a unit;  NT: threads of the block;
//   min_units: units worth a block.
template <int ROWS, int UK, int NT>
struct Schedule {
  int64_t per;         // units of a block (the last one's may be fewer)
  bool padded;         // items begin at multiples of it
  int64_t begin, end;  // this block's
  int64_t at;          // where the walk is
  int64_t s_start;     // first unit of sequence s
  int s;
  int rt_max;

  __device__ __forceinline__ int64_t block_of(int64_t u) const { return div_units(u, per); }
  static __device__ __forceinline__ int units_of(const SeqInfo& i) {
    return (int)((i.len + UK - 1) / UK);
  }
  __device__ __forceinline__ int tiles_of(const AttendParams& p, const SeqInfo& i) const {
    return (i.n * (p.q_heads / p.c.kv_heads) + ROWS - 1) / ROWS;
  }
  __device__ __forceinline__ int64_t seq_units(const AttendParams& p, int i) const {
    if (i >= p.seqs) return 0;
    const SeqInfo q = seq_info(p, i);
    return (int64_t)units_of(q) * tiles_of(p, q) * p.c.kv_heads;
  }
  __device__ __forceinline__ int64_t per_of(int64_t total, int min_units) const {
    return max(div_units(total + gridDim.x - 1, gridDim.x), (int64_t)min_units);
  }
  __device__ __forceinline__ bool take(int64_t total) {
    begin = at = per * blockIdx.x;
    end = min(begin + per, total);
    return begin < end;
  }
  static __device__ __forceinline__ int64_t warp_total(int64_t v) {
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xFFFFFFFFu, v, o);
    return v;
  }

  // All threads of the block; false: nothing to do.
  __device__ __forceinline__ bool init(const AttendParams& p, int min_units) {
    rt_max = (p.max_nodes * (p.q_heads / p.c.kv_heads) + ROWS - 1) / ROWS;
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    padded = false;
    if (p.seqs <= 32) {  // every warp by itself: no barrier
      int nu = 0, items = 0;
      if (lane < p.seqs) {
        const SeqInfo q = seq_info(p, lane);
        nu = units_of(q);
        items = tiles_of(p, q) * p.c.kv_heads;
      }
      const int64_t all = warp_total((int64_t)nu * items), n_items = warp_total(items);
      per = per_of(all, min_units);
      if (2 * n_items <= gridDim.x && all > 0) {
        // the fewest units with which every item has blocks of its own
        auto blocks = [&](int64_t u) { return warp_total((int64_t)items * (int)div_units(nu + u - 1, u)); };
        padded = true;
        if (blocks(per) > gridDim.x) {
          int64_t lo = per + 1, hi = max(lo, div_units(all + gridDim.x - n_items - 1, gridDim.x - n_items));
          while (lo < hi) {
            const int64_t mid = (lo + hi) >> 1;
            if (blocks(mid) <= gridDim.x) hi = mid;
            else lo = mid + 1;
          }
          per = hi;
        }
      }
      const int64_t v = (padded ? div_units(nu + per - 1, per) * per : (int64_t)nu) * items;
      int64_t x = v;
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const int64_t y = __shfl_up_sync(0xFFFFFFFFu, x, o);
        if (lane >= o) x += y;
      }
      if (!take(__shfl_sync(0xFFFFFFFFu, x, 31))) return false;
      const uint32_t mine = __ballot_sync(0xFFFFFFFFu, x > begin);
      s = __ffs(mine) - 1;
      s_start = __shfl_sync(0xFFFFFFFFu, x - v, s);
      return true;
    }
    __shared__ int64_t sums[NT / 32];
    __shared__ int found;
    __shared__ int64_t found_start;
    int64_t mine = 0;
    for (int i = threadIdx.x; i < p.seqs; i += NT) mine += seq_units(p, i);
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) mine += __shfl_xor_sync(0xFFFFFFFFu, mine, o);
    if (lane == 0) sums[warp] = mine;
    __syncthreads();
    int64_t total = 0;
    for (int w = 0; w < NT / 32; ++w) total += sums[w];
    per = per_of(total, min_units);
    if (!take(total)) return false;
    if (warp == 0) {  // the sequence that has unit `begin`
      int64_t before = 0;
      for (int c = 0; c < p.seqs; c += 32) {
        const int64_t v = seq_units(p, c + lane);
        int64_t x = v;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
          const int64_t y = __shfl_up_sync(0xFFFFFFFFu, x, o);
          if (lane >= o) x += y;
        }
        const uint32_t past = __ballot_sync(0xFFFFFFFFu, before + x > begin);
        if (past) {
          if (lane == __ffs(past) - 1) {
            found = c + lane;
            found_start = before + x - v;
          }
          break;
        }
        before += __shfl_sync(0xFFFFFFFFu, x, 31);
      }
    }
    __syncthreads();
    s = found;
    s_start = found_start;
    return true;
  }

  // The next part of an item; false when the range is done.
  __device__ __forceinline__ bool next(const AttendParams& p, Span& w, SeqInfo& q) {
    if (at >= end) return false;
    int nu, tiles;
    int64_t step;  // from an item's first unit to the next one's
    for (;;) {
      q = seq_info(p, s);
      nu = units_of(q);
      tiles = tiles_of(p, q);
      step = padded ? div_units(nu + per - 1, per) * per : nu;
      const int64_t all = step * tiles * p.c.kv_heads;
      if (at < s_start + all) break;
      s_start += all;
      ++s;
    }
    const int in = (int)div_units(at - s_start, step);  // item of the sequence
    w.s = s;
    w.h = in / tiles;
    w.rt = in % tiles;
    w.nu = nu;
    w.start = s_start + in * step;
    w.u0 = (int)(at - w.start);
    w.u1 = (int)min((int64_t)nu, end - w.start);
    w.item = ((int64_t)s * p.c.kv_heads + w.h) * rt_max + w.rt;
    at = padded ? end : w.start + w.u1;
    return true;
  }
};

// Workspace: a counter for each block, of the narrow kernel's parts of the item
// that goes on past the block's range (an item has one block where it begins, a
// block at most one item that it does not end); what a call needs besides; two
// slots per block of ROWS rows x (D sums, maximum, sum of weights).  The counters
// are at the same place whatever the call's shape and kernel, and nothing else is
// ever written there: they are zeros between calls.
__host__ __device__ constexpr size_t attend_counter_bytes(int blocks) { return (size_t)(blocks + 31) / 32 * 128; }
__host__ __device__ constexpr size_t attend_slot_floats(int rows, int d) { return (size_t)rows * (d + 2); }

// The many-row kernel (attend_wide.cuh) by the rows of a sequence and key head:
// 0: 256 rows of an item; 1, 2, 4: 128, 64, 32 rows in so many copies.
__host__ __device__ constexpr int wide_mode(int rows) {
  return rows <= 32 ? 4 : rows <= 64 ? 2 : rows <= 128 ? 1 : 0;
}
__host__ __device__ constexpr int wide_item_rows(int mode) { return mode == 0 ? 256 : 128 / mode; }
// Behind the counters it has 16 bytes for each item: where its parts are.
__host__ __device__ constexpr size_t join_head_bytes(int64_t items) { return (size_t)(items + 7) / 8 * 128; }

// The slot that block b has an item's part in: its first where its range begins
// inside the item (or with it), else its second.
__device__ __forceinline__ int64_t part_slot(int64_t b, int64_t per, int64_t item_start) {
  return b * 2 + (b * per >= item_start ? 0 : 1);
}

// The maximum and the sum of weights of one row over an item's parts, `at(y)` its
// part y's maximum and `lo` floats on its sum: eight parts' loads are issued
// before the first is used (a plain loop waits for each).
template <typename At>
__device__ __forceinline__ float2 join_ml(int parts, int lo, At at) {
  float M = -INFINITY, tot = 0.0f;
  for (int y0 = 0; y0 < parts; y0 += 8) {
    float m[8], l[8];
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      const float* f = at(min(y0 + j, parts - 1));
      m[j] = __ldcg(f);
      l[j] = __ldcg(f + lo);
    }
    float m2 = M;
#pragma unroll
    for (int j = 0; j < 8; ++j) m2 = fmaxf(m2, m[j]);
    const float o = m2 == -INFINITY ? 0.0f : m2;
    tot *= exp2_fast(M - o);
#pragma unroll
    for (int j = 0; j < 8; ++j) tot += y0 + j < parts ? l[j] * exp2_fast(m[j] - o) : 0.0f;
    M = m2;
  }
  return make_float2(M, tot);
}

// Where a head's rows of positions g .. g + 7 (g a multiple of 8) begin: pages
// hold whole groups of 8.  Negative: absent.
struct RowAt {
  int64_t code;   // element
  int64_t scale;
};
template <int D>  // page: the table's entry for them
__device__ __forceinline__ RowAt group_at(const AttendParams& p, int64_t page, int h, int64_t g) {
  RowAt r{-1, -1};
  if (page >= 0 && page < p.c.pages) {
    const int64_t in = ((int64_t)h << p.c.page_shift) + (g & ((1 << p.c.page_shift) - 1));
    r.code = page * p.c.page_stride + in * D;
    r.scale = page * p.c.scale_page_stride + in;
  }
  return r;
}

// Joins an item's parts when this block's is the last of them (all threads;
// the block's own part is stored).  Returns false if another block will.
__device__ __forceinline__ bool last_of_item(int* counter, int parts) {
  __shared__ int last;
  __threadfence();
  __syncthreads();
  if (threadIdx.x == 0) {
    last = atomicAdd(counter, 1) == parts - 1;
    if (last) *counter = 0;  // ready for the next call
  }
  __syncthreads();
  const bool l = last;
  if (l) __threadfence();
  return l;
}

}  // namespace nmk
