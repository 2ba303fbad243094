// attend_wide.cuh -- nm_tree_attention for many query rows per key head: 128
// rows at a time on tcgen05.
//
// A block walks the positions in tiles of 128.  Two streams, each with a score
// tile, sums and running maxima of its own, keep the tensor core and the
// softmax busy at the same time: with more than 128 rows (PAIR) they are two
// row tiles that share every K and V tile, with fewer they take the tiles of
// one row tile in turn and join at the item's end (attend.cu has the rule).
//   loaders  bring K and V tiles into a ring of stages of fp16, 128-byte
//            swizzled rows: TMA boxes of whole pages for an fp16 cache; codes
//            come by bulk copies into a raw ring and are widened by the warps.
//   MMA      one thread: S = Q K^T into TMEM; O += P V with P from TMEM and V
//            as the MN-major operand (its rows are the reduction's).
//   softmax  two warpgroups, a query row per thread: scores from TMEM, weights
//            back over them as fp16.  The maximum that scales a row moves only
//            when a score exceeds it by 2^6.9, so the sums in TMEM are seldom
//            rescaled.  The weight at that maximum is 2^8 to 2^9: none passes 2^15.9, and
//            all are fp16 at its full precision down to 2^-22 of the largest, since
//            many small ones add up.  (2^11 and 2^4: 16 sequences of 32 nodes over
//            8000 positions 110 us for 104, as scores that pass 2^4 are not seldom.)
// With at most 64 (32) rows, the tile's 128 rows are two (four) copies of them,
// and copy c weighs only the c-th half (quarter) of a tile's positions: a warp can
// read no other lanes of TMEM than its own, so without copies half of the softmax
// warps would have nothing to do and the others all of it.  The copies' sums join
// like the streams'.
// With 8-bit caches the product with V takes codes: the weight of position j is
// 2^(s_j + log2 v_j - m), v_j the row's scale, and the sum of weights adds
// w_j / v_j; a key's scale multiplies its score.  So codes enter the MMA
// exactly and a weight is rounded once.
//
// What bounds it (MODE is the number of copies, 0 for PAIR):
//   fp16, up to 128 rows: HBM.  32 rows over 131072 positions 91 us, 5.9 TB/s,
//     with 160 KB in flight an SM; of the rest 10 us are start, end and join.
//   fp16, 256 rows: a stream's chain scores -> softmax -> product.  A tile takes
//     1.6 us (0.77 softmax, 4 x 0.27 MMAs, two streams in turn), 53 % of the tensor
//     pipe; 16 sequences of 32 nodes over 8000 positions 104 us, 0.86 PFLOP/s.
//     Threads that held 32 scores at a time, with a branch between: 116 us (for 98 then).
//   codes: the chain raw tile -> widened stage -> MMA -> free stage, 1.6 to 1.9 us a
//     tile, since two stages of fp16 and six raw tiles fill the shared memory.
//     64 rows over 100000 positions: int8 81.8 us, e4m3 90.8.  One group of ten
//     widening warps in place of two of five: 89.7 and 97.5, with a third stage
//     91.6 and 97.0.
#pragma once

#include <cuda.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>
#include <stdint.h>
#include <string.h>

#include "attend.cuh"
#include "decode.h"
#include "device.cuh"
#include "kernels.h"
#include "tc.cuh"
#include "tmap.h"
#include "widen.cuh"

namespace nmk {
namespace {

constexpr int kRows = 128, kKeys = 128;
constexpr int kSoftWarps = 8, kMmaWarp = 8, kLoadWarp = 9;
constexpr int kMeta = 8;    // tiles of which it is kept which pages are there
constexpr int kScales = 4;  // tiles whose scales are kept
constexpr uint64_t kDrainNs = 100000000ull;  // copies in flight land long before
constexpr int kBad = 16;    // items whose spoilt nodes are kept
constexpr int kCopyPitch = 20;  // floats: 16 columns of a row, and its banks moved on by 20
constexpr float kLift = 9.0f, kGrow = 6.9f;
// 2^-80: a smaller scale counts as this, and no value times it is an fp16 number but
// 0.  (So a weight over its scale is at most 2^95, and 2^31 of them add up.)
constexpr float kTinyScale = 8.271806125530277e-25f;

// A slot of a tile (item) is written again kMeta (kBad) tiles (items) on.  A
// loader is at most NS + RS <= 10 positions of the ring ahead of the MMAs, and
// a tile's softmax is over when its V tile is consumed: 13 positions before
// the slot's next K tile at least; an item takes two positions or more.  Scales
// are written at most NS <= 4 positions ahead, their slot's next K tile 5 after
// the V tile.
template <int D, int TYPE, int MODE>
struct Wide {
  static constexpr bool PAIR = MODE == 0;
  static constexpr int SPLIT = PAIR ? 1 : MODE;
  static constexpr bool F16 = TYPE == kCacheFp16;
  // Loader warps (384 or 640 threads).  8-bit: one fetches, two groups of CW
  // widen the even and the odd positions of the ring; NS and RS are even, so
  // that a slot's barriers are always waited on by the same group.
  static constexpr int LW = F16 ? 3 : 11, CW = 5;
  static constexpr int THREADS = 32 * (kLoadWarp + LW);
  // Registers of a thread: the launch gives every warpgroup (65536 / THREADS,
  // rounded down to 8) of them, the softmax warpgroups take some of the others'.
  static constexpr int REGS = F16 ? 168 : 96, SOFT_REGS = F16 ? 208 : 144, OTHER_REGS = F16 ? 88 : 64;
  static_assert(2 * SOFT_REGS + (THREADS / 128 - 2) * OTHER_REGS <= THREADS / 128 * REGS,
                "the split fits the launch");
  static constexpr int CH = F16 ? kKeys / SPLIT : 32;  // positions a softmax thread holds
  // The product with V begins when half of the weights are there.
  static constexpr int PARTS = CH == kKeys ? 2 : 1;
  static constexpr int QT = PAIR ? 2 : 1;     // row tiles of an item
  static constexpr int IROWS = QT * kRows / SPLIT;  // rows of an item
  static constexpr int TILE = kKeys * D * 2;  // bytes of a stage
  static constexpr int HALF = kKeys * 128;    // 64 elements of every row
  static constexpr int NS = F16 ? (D == 128 ? (PAIR ? 4 : 5) : 8) : (D == 128 ? 2 : 4);
  static constexpr int RS = F16 ? 0 : (D == 128 && PAIR ? 4 : 6);  // raw tiles
  static constexpr int RAW = kKeys * D;
  static constexpr int Q_OFF = 0;
  static constexpr int ST_OFF = Q_OFF + QT * kRows * D * 2;
  static constexpr int RAW_OFF = ST_OFF + NS * TILE;
  static constexpr int SC_OFF = RAW_OFF + RS * RAW;  // 8-bit: k scale', log2 v, 1 / v
  static constexpr int CB_OFF = SC_OFF + (F16 ? 0 : 3 * kScales * kKeys * 4);
  static constexpr int BYTES = CB_OFF + (SPLIT > 1 ? 2 * kRows * kCopyPitch * 4 : 0);  // rows' copies added
  static constexpr int SMEM = BYTES + 1024;   // room to align the base
  static_assert(SMEM <= 227 * 1024 - 4096, "static shared memory needs room too");
  static_assert(NS + RS <= 10 && NS <= 8, "see above");
  static_assert(F16 || (NS % 2 == 0 && RS % 2 == 0 && LW == 1 + 2 * CW), "see above");
};

struct RawTile {
  int v, edge, stop;  // V (else K); has nodes or absent rows; none: the ring has ended
  int left, node0;    // as Tile's below
  uint32_t there;
  int bad, meta;
};

// TMEM columns.
constexpr uint32_t kS0 = 0, kS1 = 128, kO0 = 256, kO1 = 384, kTmemCols = 512;

__device__ __forceinline__ uint32_t half2_of(float a, float b) {
  const __half2 h = __floats2half2_rn(a, b);
  return *reinterpret_cast<const uint32_t*>(&h);
}

template <int N>
__device__ __forceinline__ void regs_up() {
  asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(N));
}
template <int N>
__device__ __forceinline__ void regs_down() {
  asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(N));
}

// Two fp32 operations in one instruction.
__device__ __forceinline__ float2 fma2(float2 a, float2 b, float2 c) {
  float2 d;
  asm("{\n\t.reg .b64 x, y, z, w;\n\t"
      "mov.b64 x, {%2, %3};\n\tmov.b64 y, {%4, %5};\n\tmov.b64 z, {%6, %7};\n\t"
      "fma.rn.f32x2 w, x, y, z;\n\tmov.b64 {%0, %1}, w;\n\t}"
      : "=f"(d.x), "=f"(d.y)
      : "f"(a.x), "f"(a.y), "f"(b.x), "f"(b.y), "f"(c.x), "f"(c.y));
  return d;
}

__device__ __forceinline__ float2 mul2(float2 a, float2 b) {
  float2 d;
  asm("{\n\t.reg .b64 x, y, w;\n\t"
      "mov.b64 x, {%2, %3};\n\tmov.b64 y, {%4, %5};\n\t"
      "mul.rn.f32x2 w, x, y;\n\tmov.b64 {%0, %1}, w;\n\t}"
      : "=f"(d.x), "=f"(d.y)
      : "f"(a.x), "f"(a.y), "f"(b.x), "f"(b.y));
  return d;
}

__device__ __forceinline__ float2 add2(float2 a, float2 b) {
  float2 d;
  asm("{\n\t.reg .b64 x, y, w;\n\t"
      "mov.b64 x, {%2, %3};\n\tmov.b64 y, {%4, %5};\n\t"
      "add.rn.f32x2 w, x, y;\n\tmov.b64 {%0, %1}, w;\n\t}"
      : "=f"(d.x), "=f"(d.y)
      : "f"(a.x), "f"(a.y), "f"(b.x), "f"(b.y));
  return d;
}

__device__ __forceinline__ void sts_v4(uint32_t at, uint32_t a, uint32_t b, uint32_t c, uint32_t d) {
  asm volatile("st.shared.v4.u32 [%0], {%1,%2,%3,%4};" ::"r"(at), "r"(a), "r"(b), "r"(c), "r"(d)
               : "memory");
}

template <int D, int TYPE, int MODE>
__global__ void __launch_bounds__(Wide<D, TYPE, MODE>::THREADS, 1)
    attend_wide_kernel(const __grid_constant__ AttendParams p, const __grid_constant__ CUtensorMap tm_k,
                       const __grid_constant__ CUtensorMap tm_v) {
  using W = Wide<D, TYPE, MODE>;
  constexpr bool F16 = W::F16, PAIR = W::PAIR;
  constexpr int RS = F16 ? 1 : W::RS, SPLIT = W::SPLIT;
  constexpr int RB = F16 ? W::NS : RS;  // barriers of tiles that landed
  constexpr int IROWS = W::IROWS;
  using Sched = Schedule<IROWS, kKeys, W::THREADS>;
  extern __shared__ uint8_t raw_smem[];
  __shared__ uint64_t bar_mem[2 * W::NS + 8 + RB + RS + 2];
  __shared__ uint32_t tmem_slot;
  __shared__ uint32_t there_of[kMeta];
  __shared__ uint32_t bad_of[kBad][2];
  __shared__ float2 s_ml[2][kRows];
  __shared__ float s_inv[2][kRows];
  // 8-bit: what a raw tile is, for the groups that widen it
  __shared__ RawTile raw_of[RS];
  __shared__ int64_t raw_scales[RS][16];  // of its groups of 8 rows
  const uint32_t base = (smem_addr(raw_smem) + 1023u) & ~1023u;
  uint8_t* gbase = raw_smem + (base - smem_addr(raw_smem));
  const uint32_t sQ = base + W::Q_OFF, sT = base + W::ST_OFF;
  float* scales = reinterpret_cast<float*>(gbase + W::SC_OFF);
  const uint32_t bars = smem_addr(bar_mem);
  auto full = [&](int s) { return bars + 8u * s; };
  auto empty = [&](int s) { return bars + 8u * (W::NS + s); };
  auto sfull = [&](int b) { return bars + 8u * (2 * W::NS + b); };      // scores ready
  auto pfull = [&](int b) { return bars + 8u * (2 * W::NS + 2 + b); };  // weights ready
  auto ofull = [&](int b) { return bars + 8u * (2 * W::NS + 4 + b); };  // sums ready
  const uint32_t qfull = bars + 8u * (2 * W::NS + 6), soft = bars + 8u * (2 * W::NS + 7);
  // a raw tile landed; fp16: a stage that the loaders look at before it is full
  auto rfull = [&](int s) { return bars + 8u * (2 * W::NS + 8 + s); };
  auto rfree = [&](int s) { return bars + 8u * (2 * W::NS + 8 + RB + s); };   // 8-bit: ... and read
  auto phalf = [&](int b) { return bars + 8u * (2 * W::NS + 8 + RB + RS + b); };  // PARTS == 2: the first half of the weights

  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  pdl_launch_dependents();
  if (__syncthreads_or(threadIdx.x == 0 && wait_aborted())) {
    pdl_wait_previous();  // what follows on the stream is after the kernels before this one
    return;
  }
  // what touches no caller's memory comes before the wait for the last kernel
  if (warp == 0 && lane == 0) {
    for (int s = 0; s < W::NS; ++s) {
      mbar_init(full(s), F16 ? W::LW : W::CW);
      mbar_init(empty(s), 1);
    }
    for (int s = 0; s < RB; ++s) mbar_init(rfull(s), 1);
    for (int s = 0; s < RS; ++s) mbar_init(rfree(s), W::CW);
    for (int b = 0; b < 2; ++b) {
      mbar_init(sfull(b), 1);
      mbar_init(pfull(b), 4);
      mbar_init(phalf(b), 4);
      mbar_init(ofull(b), 1);
    }
    mbar_init(qfull, PAIR ? kSoftWarps : kSoftWarps / 2);
    mbar_init(soft, kSoftWarps);
    fence_mbar_init();
    if (F16) {
      prefetch_tmap(&tm_k);
      prefetch_tmap(&tm_v);
    }
  }
  if (threadIdx.x < kBad * 2) bad_of[threadIdx.x / 2][threadIdx.x % 2] = 0;
  if (warp == kMmaWarp) {
    tmem_alloc(smem_addr(&tmem_slot), kTmemCols);
    tmem_relinquish();
  }
  tc_fence_before_sync();
  pdl_wait_previous();
  Sched sched;
  const bool work = sched.init(p, 1);
  __syncthreads();
  tc_fence_after_sync();
  const uint32_t tmem = *(volatile uint32_t*)&tmem_slot;
  const int G = p.q_heads / p.c.kv_heads;
  const Heads heads(G);
  const float cs = p.scale * kLog2e;
  auto wait_warp = [&](uint32_t bar, uint32_t par) {
    return __all_sync(0xFFFFFFFFu, mbar_wait(bar, par, p.wait_limit_ns)) != 0;
  };

  if (!work) {
  } else if (warp >= kLoadWarp) {
    // ---- loaders ---------------------------------------------------------------
    regs_down<W::OTHER_REGS>();
    const int lw = warp - kLoadWarp, lt = lw * 32 + lane;
    constexpr int LT = W::LW * 32;
    const int box_shift = min(p.c.page_shift, 7);  // a box: a page's rows, at most a tile's
    const int page_rows = 1 << box_shift, boxes = kKeys >> box_shift;
    // (16 x 8000 positions: 100 us without, 95 with; what else is in L2, the
    // blocks' parts and the code among it, stays there)
    const uint64_t once = l2_evict_first();
    int c = 0;  // positions of the ring so far
    int item_no = 0, tile_no = 0;
    uint32_t looked = 0;  // fp16: parity of each stage's looks so far
    bool ok = !(p.stall && blockIdx.x % 2 == 0);
    struct Tile {      // a tile of an item; lane l has box l
      int page, row;   // the box's page and first row in it (of all heads')
      bool on;         // it is there
      int have;        // boxes that are
      uint32_t there;  // groups of 8 rows that are there
      int left;        // rows before the sequence's end
      bool edge;       // has nodes, or absent rows
      int node0;       // node number of its first row (far below 0: none near)
      int bad, meta;   // slots
    };
    auto note = [&](const Tile& t, bool first) {  // a K tile's slots (one warp)
      if (lane == 0) {
        there_of[t.meta] = t.there;
        if (first)
          bad_of[(item_no + kBad / 2) % kBad][0] = bad_of[(item_no + kBad / 2) % kBad][1] = 0;
      }
    };
    // Clears halves that are not finite in a node's value row and notes the node:
    // an infinity or NaN must not meet a weight of 0.
    auto clean = [&](uint32_t* h, int words, int node, int slot) {
      uint32_t any = 0;
      for (int y = 0; y < words; ++y) {
        const uint32_t b = bad_halves(h[y]);
        any |= b;
        h[y] &= (b & 1u ? 0u : 0xFFFFu) | (b & 2u ? 0u : 0xFFFF0000u);
      }
      if (any) atomicOr(&bad_of[slot][(node >> 5) & 1], 1u << (node & 31));
    };

    // fp16: the ring's next position is K (v false) or V of tile t.
    auto emit16 = [&](bool v, const Tile& t, bool first) {
      const int st = c % W::NS;
      if (c >= W::NS && !wait_warp(empty(st), (c / W::NS - 1) & 1)) return false;
      const uint32_t dst = sT + st * W::TILE;
      if (!v && lw == 0) note(t, first);
      const bool look = v && t.edge;  // absent rows are to be zeros, nodes' rows are looked at
      // The look has a barrier of the stage's own: no warp can be a look of this
      // stage ahead of another, since the stage is not empty again before all have
      // arrived on `full`.
      const uint32_t bar = look ? rfull(st) : full(st);
      if (lw == 0) {
        if (lane == 0 && (t.have || !look)) mbar_arrive_expect_tx(bar, t.have * page_rows * D * 2);
        __syncwarp();
        if (t.on) {
#pragma unroll
          for (int hf = 0; hf < D / 64; ++hf)
            tma_load_3d(dst + hf * W::HALF + lane * page_rows * 128, v ? &tm_v : &tm_k, hf * 64, t.row,
                        t.page, bar, once);
        }
        __syncwarp();
      } else if (!look && lane == 0) {
        mbar_arrive(full(st));
      }
      if (look) {
        if (t.have) {
          if (!wait_warp(bar, (looked >> st) & 1u)) {
            mbar_wait(bar, (looked >> st) & 1u, kDrainNs, false);  // the copies that it is for land
            return false;
          }
          looked ^= 1u << st;
        }
        constexpr int PR = D / 8;
        for (int id = lt; id < kKeys * PR; id += LT) {
          const int r = id / PR, ch = id % PR;
          const bool there = r < t.left && ((t.there >> (r >> 3)) & 1u);
          if (there && t.node0 + r < 0) continue;
          const uint32_t at = dst + (ch >> 3) * W::HALF + r * 128 + (((ch & 7) ^ (r & 7)) << 4);
          uint32_t h[4] = {0, 0, 0, 0};
          if (there) {
            asm volatile("ld.shared.v4.u32 {%0,%1,%2,%3}, [%4];"
                         : "=r"(h[0]), "=r"(h[1]), "=r"(h[2]), "=r"(h[3])
                         : "r"(at));
            clean(h, 4, t.node0 + r, t.bad);
          }
          sts_v4(at, h[0], h[1], h[2], h[3]);
        }
        fence_proxy_async_smem();
        __syncwarp();
        if (lane == 0) mbar_arrive(full(st));
      }
      __syncwarp();
      ++c;
      return true;
    };

    // 8-bit, the fetching warp: the raw ring's next position is K or V of tile t
    // (null: there is none).
    auto fetch8 = [&](bool v, const Tile* t, bool first) {
      const int st = c % RS;
      if (c >= RS && !wait_warp(rfree(st), (c / RS - 1) & 1)) return false;
      ++c;
      if (!t) {
        if (lane == 0) {
          raw_of[st].stop = 1;
          mbar_arrive(rfull(st));
        }
        __syncwarp();
        return true;
      }
      if (!v) note(*t, first);
      if (!v) {  // where the scales of lane l's group of 8 rows are
        const int box = (lane * 8 >> box_shift) & 15, in = (lane * 8) & (page_rows - 1);
        const int page = __shfl_sync(0xFFFFFFFFu, t->page, box), row = __shfl_sync(0xFFFFFFFFu, t->row, box);
        if (lane < 16)
          raw_scales[st][lane] = (t->there >> lane) & 1u ? page * p.c.scale_page_stride + row + in : -1;
      }
      if (lane == 0) raw_of[st] = RawTile{v, t->edge, 0, t->left, t->node0, t->there, t->bad, t->meta};
      __syncwarp();
      if (lane == 0) mbar_arrive_expect_tx(rfull(st), t->have * page_rows * D);
      __syncwarp();
      if (t->on)
        bulk_load(base + W::RAW_OFF + st * W::RAW + lane * page_rows * D,
                  (v ? p.c.v : p.c.k) + t->page * p.c.page_stride + (int64_t)t->row * D, page_rows * D,
                  rfull(st), once);
      __syncwarp();
      return true;
    };
    // 8-bit, a widening group (ct: thread of it): the raw tile of position c to
    // its stage; with a K tile its scales: k scale log2(e), log2 v, 1 / v.
    const int ct = lt - 32 - (lw > W::CW ? W::CW * 32 : 0);
    constexpr int CT = W::CW * 32;
    bool stop = false;
    auto widen8 = [&]() {
      const int st = c % W::NS, rs = c % RS;
      if (!wait_warp(rfull(rs), (c / RS) & 1)) return false;
      const RawTile t = raw_of[rs];
      if (t.stop) {
        stop = true;
        return true;
      }
      const bool v = t.v;
      float sc[2] = {0.0f, 0.0f};  // row ct's k and v scale, in flight while the codes are widened
      if (!v && ct < kKeys) {
        const int64_t at = raw_scales[rs][ct >> 3];
        if (at >= 0 && ct < t.left) {
          sc[0] = p.c.k_scale[at + (ct & 7)];
          sc[1] = p.c.v_scale[at + (ct & 7)];
        }
      }
      if (c >= W::NS && !wait_warp(empty(st), (c / W::NS - 1) & 1)) return false;
      const uint32_t dst = sT + st * W::TILE, src = base + W::RAW_OFF + rs * W::RAW;
      // A thread's pieces: column piece ch of rows r0, r0 + STEP, ...; the swizzle of
      // row r0 + i STEP differs from row r0's by at most the bit that STEP's
      // multiple of 4 turns.
      constexpr int PR = D / 16, STEP = CT / PR;  // pieces of a row
      static_assert(STEP % 4 == 0, "see above");
      const int ch = ct % PR, r0 = ct / PR;
      const uint32_t from = src + ct * 16;
      // Eight threads store 16 bytes at a time, of one row's two halves (D = 128),
      // which are in the same banks: those of the second half take the upper 8
      // codes of their piece first.
      const bool upper = (ch >> 2) != 0;
      const uint32_t to =
          (dst + (ch >> 2) * W::HALF + r0 * 128 + ((((ch & 3) * 2) ^ (r0 & 7)) << 4)) ^ (upper ? 16u : 0u);
      constexpr uint32_t kTurn = STEP % 8 ? 64u : 0u;
      const bool look = v && t.edge;
      constexpr int ALL = (kKeys + STEP - 1) / STEP, B = 4;
#pragma unroll
      for (int i0 = 0; i0 < ALL; i0 += B) {
        uint32_t w[B][4];
#pragma unroll
        for (int i = 0; i < B; ++i)
          if (i0 + i < ALL && r0 + (i0 + i) * STEP < kKeys)
            asm volatile("ld.shared.v4.u32 {%0,%1,%2,%3}, [%4];"
                         : "=r"(w[i][0]), "=r"(w[i][1]), "=r"(w[i][2]), "=r"(w[i][3])
                         : "r"(from + (i0 + i) * CT * 16));
#pragma unroll
        for (int i = 0; i < B; ++i) {
          const int r = r0 + (i0 + i) * STEP;
          if (i0 + i >= ALL || r >= kKeys) continue;
          if (look && !(r < t.left && ((t.there >> (r >> 3)) & 1u))) w[i][0] = w[i][1] = w[i][2] = w[i][3] = 0;
          uint32_t h[8];
#pragma unroll
          for (int k = 0; k < 4; ++k)
            widen4<F16 ? kCacheE4m3 : TYPE>(D == 128 && upper ? w[i][k ^ 2] : w[i][k], h[2 * k], h[2 * k + 1]);
          if (TYPE == kCacheE4m3 && look && t.node0 + r >= 0) clean(h, 8, t.node0 + r, t.bad);
          const uint32_t at = (to + (i0 + i) * STEP * 128) ^ ((i0 + i) & 1 ? kTurn : 0u);
          sts_v4(at, h[0], h[1], h[2], h[3]);
          sts_v4(at ^ 16u, h[4], h[5], h[6], h[7]);
        }
      }
      if (!v && ct < kKeys) {
        const int j = t.node0 + ct;
        float lv = log2f(sc[1]), rv = 1.0f / sc[1];
        if (sc[1] < kTinyScale) lv = -80.0f, rv = 1.0f / kTinyScale;
        if (t.edge && j >= 0 && !(sc[1] < INFINITY)) {  // a node's row whose scale is not finite
          lv = 0.0f, rv = 1.0f;
          atomicOr(&bad_of[t.bad][(j >> 5) & 1], 1u << (j & 31));
        }
        float* f = scales + t.meta % kScales * kKeys + ct;
        f[0] = sc[0] * cs;
        f[kScales * kKeys] = lv;
        f[2 * kScales * kKeys] = rv;
      }
      fence_proxy_async_smem();
      __syncwarp();
      if (lane == 0) {
        mbar_arrive(full(st));
        mbar_arrive(rfree(rs));
      }
      return true;
    };

    // The positions of the ring in order: K0, V0, K1, V1, ... for PAIR, else
    // K0, K1, V0, K2, V1, ..., as the MMA thread takes them.
    if (F16 || lw == 0) {
      Span w;
      SeqInfo si;
      while (ok && sched.next(p, w, si)) {
        const int n = w.u1 - w.u0;
        const int32_t* table = p.table + (int64_t)w.s * p.ld_table;
        auto look_up = [&](int i) {  // the page of the lane's box
          const int64_t pos = (int64_t)(w.u0 + i) * kKeys + (lane << box_shift);
          return i < n && lane < boxes && pos < si.len ? table[pos >> p.c.page_shift] : -1;
        };
        int32_t entry = look_up(0);
        Tile now, last;
        for (int i = 0; i <= n && ok; ++i) {
          if (i < n) {
            const int64_t pos0 = (int64_t)(w.u0 + i) * kKeys;
            now.page = entry;
            now.on = entry >= 0 && entry < p.c.pages;
            now.row = (w.h << p.c.page_shift) +
                      (int)((pos0 + (lane << box_shift)) & ((1 << p.c.page_shift) - 1));
            entry = look_up(i + 1);
            const uint32_t on = __ballot_sync(0xFFFFFFFFu, now.on);
            now.have = __popc(on);
            now.there = __ballot_sync(0xFFFFFFFFu, lane < 16 && ((on >> (lane * 8 >> box_shift)) & 1u));
            now.left = (int)min((int64_t)kKeys, si.len - pos0);
            now.edge = pos0 + kKeys > si.ctx || now.there != 0xFFFFu;
            now.node0 = (int)max(pos0 - si.ctx, (int64_t)-(1 << 20));
            now.bad = item_no % kBad;
            now.meta = tile_no++ % kMeta;
            if constexpr (F16)
              ok = emit16(false, now, i == 0);
            else
              ok = fetch8(false, &now, i == 0);
            if (PAIR) last = now;
          }
          if (ok && (PAIR ? i < n : i > 0)) {
            if constexpr (F16)
              ok = emit16(true, last, false);
            else
              ok = fetch8(true, &last, false);
          }
          if (!PAIR) last = now;
        }
        ++item_no;
      }
      if (!F16)  // a last position for each group
        for (int i = 0; i < 2 && ok; ++i) ok = fetch8(false, nullptr, false);
      // Before the block ends its copies have landed, whatever else failed (an fp16
      // stage's barrier also has the loaders' arrivals, which may be missing then) ...
      constexpr int NC = F16 ? W::NS : RS;
      for (int pos = max(0, c - NC); pos < c; ++pos)
        ok = __all_sync(0xFFFFFFFFu, mbar_wait(F16 ? full(pos % W::NS) : rfull(pos % RS), (pos / NC) & 1,
                                               ok ? kWaitLimitNs : kDrainNs, false)) && ok;
      // ... and every release of a stage has arrived.
      if (F16)
        for (int pos = max(0, c - W::NS); ok && pos < c; ++pos)
          ok = wait_warp(empty(pos % W::NS), (pos / W::NS) & 1);
    } else {
      const int g = lw > W::CW ? 1 : 0;
      for (c = g; ok; c += 2) {
        ok = widen8();
        if (stop) break;
      }
      for (int pos = max(g, c - W::NS); ok && pos < c; pos += 2)
        ok = wait_warp(empty(pos % W::NS), (pos / W::NS) & 1);
    }
    __syncwarp();
  } else if (warp == kMmaWarp) {
    // ---- MMA issuer ----------------------------------------------------------------
    // The warp walks together, one lane issues.
    regs_down<W::OTHER_REGS>();
    constexpr uint32_t id_s = idesc_f16_f32(kRows, kKeys);
    constexpr uint32_t id_o = idesc_f16_f32(kRows, D) | kIdescBMajorMN;
    const bool lead = elect_one();
    const uint32_t q_lo = desc_sw128_lo(sQ, 16), k_lo = desc_sw128_lo(sT, 16),
                   v_lo = desc_sw128_lo(sT, W::HALF);
    int c = 0, items = 0, np[2] = {0, 0};
    bool ok = true;
    Span w;
    SeqInfo si;
    auto ready = [&](int pos) {
      if (!wait_warp(full(pos % W::NS), (pos / W::NS) & 1)) return false;
      tc_fence_after_sync();
      return true;
    };
    auto scores = [&](int pos, int b) {  // stream b, the K tile of ring position pos
      const uint32_t d = tmem + (b ? kS1 : kS0), k = k_lo + pos % W::NS * (W::TILE >> 4);
      const uint32_t q = q_lo + (PAIR && b ? (kRows * D * 2) >> 4 : 0);
      if (lead) {
#pragma unroll
        for (int ks = 0; ks < D / 16; ++ks) {
          const uint32_t off = ((ks >> 2) * W::HALF + (ks & 3) * 32) >> 4;
          mma_f16(d, desc_of(q + off, kDescSw128Hi), desc_of(k + off, kDescSw128Hi), id_s, ks != 0);
        }
        mma_commit(sfull(b));
      }
      __syncwarp();
    };
    auto sums = [&](int pos, int b, bool add) {
      const uint32_t d = tmem + (b ? kO1 : kO0), a = tmem + (b ? kS1 : kS0);
      const uint32_t v = v_lo + pos % W::NS * (W::TILE >> 4);
      constexpr int STEPS = kKeys / 16 / W::PARTS;
#pragma unroll
      for (int part = 0; part < W::PARTS; ++part) {
        if (!wait_warp(part == W::PARTS - 1 ? pfull(b) : phalf(b), np[b] & 1)) return false;
        tc_fence_after_sync();
        if (lead) {
#pragma unroll
          for (int ks = part * STEPS; ks < (part + 1) * STEPS; ++ks)
            mma_f16_ts(d, a + ks * 8, desc_of(v + ks * (2048 >> 4), kDescSw128Hi), id_o,
                       ks != 0 ? 1u : add ? 1u : 0u);
          if (part == W::PARTS - 1) mma_commit(ofull(b));
        }
        __syncwarp();
      }
      ++np[b];
      return true;
    };
    auto release = [&](int pos) {
      if (lead) mma_commit(empty(pos % W::NS));
      __syncwarp();
    };
    while (ok && sched.next(p, w, si)) {
      const int n = w.u1 - w.u0;
      if (!wait_warp(qfull, items & 1)) break;
      ++items;
      const bool two = PAIR && si.n * G - w.rt * IROWS > kRows;
      ok = ready(c);
      if (!ok) break;
      scores(c, 0);
      if (two) scores(c, 1);
      release(c);
      ++c;
      for (int i = 0; i < n; ++i) {
        const bool more = i + 1 < n;
        if (PAIR) {
          const int cv = c, ck = c + 1;
          ok = ready(cv) && sums(cv, 0, i > 0);
          if (ok && more) {
            ok = ready(ck);
            if (ok) scores(ck, 0);
          }
          if (ok && two) ok = sums(cv, 1, i > 0);
          if (!ok) break;
          release(cv);
          if (more) {
            if (two) scores(ck, 1);
            release(ck);
          }
          c += more ? 2 : 1;
        } else {
          if (more) {
            ok = ready(c);
            if (!ok) break;
            scores(c, (i + 1) & 1);
            release(c);
            ++c;
          }
          ok = ready(c) && sums(c, i & 1, i > 1);
          if (!ok) break;
          release(c);
          ++c;
        }
      }
    }
    __syncwarp();
  } else {
    // ---- softmax -------------------------------------------------------------------
    regs_up<W::SOFT_REGS>();
    const int b = warp >> 2, row = (warp & 3) * 32 + lane;
    // the item's (PAIR: the stream's) row, and which of its copies
    const int irow = PAIR ? row : row % IROWS, copy = PAIR ? 0 : row / IROWS;
    const uint32_t tlane = tmem + ((uint32_t)((warp & 3) * 32) << 16);
    const uint32_t tS = tlane + (b ? kS1 : kS0), tO = tlane + (b ? kO1 : kO0);
    const int step = PAIR ? 1 : 2, off0 = PAIR ? 0 : b;  // tiles of this stream
    int tile_no = 0, item_no = 0, ns = 0, no = 0, phase = 0;
    // A score's step in powers of 2 (fp16).  Not 0, so that a masked -infinity stays
    // one; no score is large enough to tell 1e-30 from 0.
    const float step2 = fmaxf(fabsf(cs), 1e-30f);
    auto soft_sync = [&]() {  // all softmax warps
      __syncwarp();
      if (lane == 0) mbar_arrive(soft);
      return wait_warp(soft, phase++ & 1);
    };
    uint8_t* ws = p.workspace + attend_counter_bytes(gridDim.x);
    int4* heads_of_items = reinterpret_cast<int4*>(ws);
    float* slots = reinterpret_cast<float*>(ws + join_head_bytes((int64_t)p.seqs * p.c.kv_heads * sched.rt_max));
    auto give_weights = [&](uint32_t bar) {
      tmem_st_wait();
      tc_fence_before_sync();
      __syncwarp();
      if (lane == 0) mbar_arrive(bar);
    };
    bool ok = true;
    // An item's queries (of this stream's rows), by this warpgroup: asked for when
    // the last product that reads the ones before is done, announced when they
    // are there, so that the next item's scores are computed while this one ends.
    auto ask_q = [&](const Span& w, const SeqInfo& si) {
      const int r0 = w.rt * IROWS + (PAIR ? b * kRows : 0), rows = min(PAIR ? kRows : IROWS, si.n * G - r0);
      const uint32_t q = sQ + (PAIR && b ? kRows * D * 2 : 0);
      const int t0 = threadIdx.x & 127;
#pragma unroll 4
      for (int i = 0; i < kRows * (D / 8) / 128; ++i) {
        const int id = t0 + i * 128, r = id / (D / 8), ch = id % (D / 8), rr = r0 + (PAIR ? r : r % IROWS);
        const bool on = (PAIR ? r : r % IROWS) < rows;
        const __half* src = p.q;
        if (on) src += (int64_t)(si.first + heads.node(rr)) * p.ldq + (w.h * G + heads.head(rr)) * D + ch * 8;
        cp_async_16(q + (ch >> 3) * W::HALF + r * 128 + (((ch & 7) ^ (r & 7)) << 4), src, on ? 16u : 0u);
      }
    };
    auto announce_q = [&]() {
      cp_async_wait_all();
      fence_proxy_async_smem();
      __syncwarp();
      if (lane == 0) mbar_arrive(qfull);
    };
    Span w, w2;
    SeqInfo si, si2;
    bool have = sched.next(p, w, si);
    if (have && (PAIR || b == 0)) {
      ask_q(w, si);
      announce_q();
    }
    for (; ok && have; w = w2, si = si2) {
      const int n = w.u1 - w.u0;
      have = sched.next(p, w2, si2);  // the next item
      const int r0 = w.rt * IROWS + (PAIR ? b * kRows : 0);  // the stream's first row
      const int rows = max(0, min(PAIR ? kRows : IROWS, si.n * G - r0));
      const int rr = r0 + irow, node = heads.node(rr), hq = w.h * G + heads.head(rr);
      const bool mine = irow < rows;
      const uint64_t bits = !mine ? 0ull
                            : p.tree_mask ? p.tree_mask[si.first + node]
                                          : (2ull << node) - 1ull;
      const bool idle = (PAIR ? (warp & 3) * 32 : (warp & 3) * 32 % IROWS) >= rows;  // a warp without rows
      float m = -INFINITY, l = 0.0f;
      const int tiles = PAIR && rows == 0 ? 0 : (n - off0 + step - 1) / step;
      // this stream has the item's last scores (or reads none of its queries)
      const bool asks = have && (PAIR || b == ((n - 1) & 1));
      if (PAIR && asks && tiles == 0) {
        // A stream without rows waits for no scores.  It waits here until both
        // have announced this item's queries: an arrival for the next item before
        // the other stream's would complete this item's phase in its place.
        ask_q(w2, si2);
        ok = wait_warp(qfull, item_no & 1);
      }
      for (int k = 0; k < tiles; ++k) {
        const int i = off0 + k * step;
        ok = wait_warp(sfull(b), ns++ & 1);
        // (the sums up to here were issued before these scores: no further wait,
        // but every phase of a barrier is seen, so that its parity says which)
        if (ok && k > 0) ok = wait_warp(ofull(b), (no + k - 1) & 1);
        if (!ok) break;
        if (asks && k == tiles - 1) ask_q(w2, si2);
        if (!idle) {
          tc_fence_after_sync();
          const int slot = (tile_no + i) % kMeta;
          const int64_t pos0 = (int64_t)(w.u0 + i) * kKeys;
          const uint32_t there = *(volatile uint32_t*)&there_of[slot];
          const bool edge = pos0 + kKeys > si.ctx || there != 0xFFFFu;
          const float4* ksc = reinterpret_cast<const float4*>(scales + slot % kScales * kKeys);
          const float4* lvs = ksc + kScales * kKeys / 4;
          const float4* rvs = lvs + kScales * kKeys / 4;
          // what the row sees of positions 32 y .. of an edge tile
          auto sees = [&](int y) {
            const int64_t f = pos0 - si.ctx + 32 * y;  // node number of the first
            uint32_t x;
            if (f <= -32) x = ~0u;
            else if (f >= 64) x = 0u;
            else if (f >= 0) x = (uint32_t)(bits >> f);
            else x = (uint32_t)((bits << -f) | ((1ull << -f) - 1ull));
            uint32_t g = there >> (4 * y);
            g = (g & 1u ? 0xFFu : 0u) | (g & 2u ? 0xFF00u : 0u) | (g & 4u ? 0xFF0000u : 0u) |
                (g & 8u ? 0xFF000000u : 0u);
            x &= g;
            const int64_t rest = si.len - pos0 - 32 * y;
            if (rest < 32) x &= rest <= 0 ? 0u : (1u << rest) - 1u;
            return x;
          };
          // CH positions at a time, in one reading of the scores: all maxima first,
          // then the weights, which pass through the MUFU at its rate.
          constexpr int CH = W::CH;
          const int y0 = copy * (4 / SPLIT), y1 = y0 + 4 / SPLIT;  // of 32 positions
#pragma unroll 1
          for (int y = y0; y < y1; y += CH / 32) {
            uint32_t v[CH / 32][32];
#pragma unroll
            for (int z = 0; z < CH / 32; ++z) tmem_ld_32(tS + 32 * (y + z), v[z]);
            tmem_ld_wait();
            // exponents in powers of 2 are v step - m
            if (F16) {
              if (cs < 0.0f) {
#pragma unroll
                for (int x = 0; x < CH; ++x) v[x / 32][x % 32] ^= 0x80000000u;
              }
            } else {
#pragma unroll
              for (int x = 0; x < CH; x += 4) {
                const float4 a = ksc[8 * y + x / 4], d = lvs[8 * y + x / 4];
                const float2 e0 = fma2(make_float2(__uint_as_float(v[x / 32][x % 32]), __uint_as_float(v[x / 32][x % 32 + 1])),
                                       make_float2(a.x, a.y), make_float2(d.x, d.y));
                const float2 e1 = fma2(make_float2(__uint_as_float(v[x / 32][x % 32 + 2]), __uint_as_float(v[x / 32][x % 32 + 3])),
                                       make_float2(a.z, a.w), make_float2(d.z, d.w));
                v[x / 32][x % 32] = __float_as_uint(e0.x), v[x / 32][x % 32 + 1] = __float_as_uint(e0.y);
                v[x / 32][x % 32 + 2] = __float_as_uint(e1.x), v[x / 32][x % 32 + 3] = __float_as_uint(e1.y);
              }
            }
            if (edge) {
#pragma unroll
              for (int z = 0; z < CH / 32; ++z) {
                const uint32_t see = sees(y + z);
#pragma unroll
                for (int x = 0; x < 32; ++x)
                  if (!((see >> x) & 1u)) v[z][x] = 0xFF800000u;  // -inf
              }
            }
            float t[4] = {-INFINITY, -INFINITY, -INFINITY, -INFINITY};
#pragma unroll
            for (int x = 0; x < CH; x += 8) {
#pragma unroll
              for (int z = 0; z < 4; ++z)
                t[z] = fmaxf(fmaxf(t[z], __uint_as_float(v[x / 32][x % 32 + z])), __uint_as_float(v[x / 32][x % 32 + z + 4]));
            }
            const float top = fmaxf(fmaxf(t[0], t[1]), fmaxf(t[2], t[3])) * (F16 ? step2 : 1.0f);
            const bool grow = top > m + (kGrow + kLift) || (m == -INFINITY && top > -INFINITY);
            if (__any_sync(0xFFFFFFFFu, grow)) {
              // seldom (but for an item's first positions): the sums so far, and
              // the weights of this tile so far, move to the new maximum.  A maximum
              // is a whole power of 2, so that a weight times `keep` is exact.
              const float next = ceilf(top) - kLift;
              const float keep = !grow ? 1.0f : m == -INFINITY ? 0.0f : exp2_fast(m - next);
              if (k > 0) {
#pragma unroll 1
                for (int d = 0; d < D; d += 16) {
                  uint32_t o[16];
                  tmem_ld_16(tO + d, o);
                  tmem_ld_wait();
#pragma unroll
                  for (int x = 0; x < 16; ++x) o[x] = __float_as_uint(__uint_as_float(o[x]) * keep);
                  tmem_st_16(tO + d, o);
                }
              }
              if (CH < kKeys / SPLIT) {
#pragma unroll 1
                for (int z = y0; z < y; ++z) {
                  uint32_t o[16];
                  tmem_st_wait();
                  tmem_ld_16(tS + 16 * z, o);
                  tmem_ld_wait();
#pragma unroll
                  for (int x = 0; x < 16; ++x) {
                    const float2 f = half2_bits_to_float2(o[x]);
                    o[x] = half2_of(f.x * keep, f.y * keep);
                  }
                  tmem_st_16(tS + 16 * z, o);
                }
              }
              l *= keep;
              if (grow) m = next;
            }
            const float off = m == -INFINITY ? 0.0f : -m;
            float2 sum[2] = {make_float2(0.0f, 0.0f), make_float2(0.0f, 0.0f)};
#pragma unroll
            for (int z = 0; z < CH / 32; ++z) {
              uint32_t h[16];
#pragma unroll
              for (int x = 0; x < 32; x += 4) {
                const uint32_t* u = &v[z][x];
                float2 e0 = make_float2(__uint_as_float(u[0]), __uint_as_float(u[1]));
                float2 e1 = make_float2(__uint_as_float(u[2]), __uint_as_float(u[3]));
                if (F16) {
                  e0 = fma2(e0, make_float2(step2, step2), make_float2(off, off));
                  e1 = fma2(e1, make_float2(step2, step2), make_float2(off, off));
                } else {
                  e0 = add2(e0, make_float2(off, off));
                  e1 = add2(e1, make_float2(off, off));
                }
                e0 = make_float2(exp2_fast(e0.x), exp2_fast(e0.y));
                e1 = make_float2(exp2_fast(e1.x), exp2_fast(e1.y));
                if (F16) {
                  sum[0] = add2(sum[0], e0);
                  sum[1] = add2(sum[1], e1);
                } else {
                  const float4 r = rvs[8 * (y + z) + x / 4];
                  sum[0] = fma2(e0, make_float2(r.x, r.y), sum[0]);
                  sum[1] = fma2(e1, make_float2(r.z, r.w), sum[1]);
                }
                h[x / 2] = half2_of(e0.x, e0.y);
                h[x / 2 + 1] = half2_of(e1.x, e1.y);
              }
              tmem_st_16(tS + 16 * (y + z), h);
              if (W::PARTS == 2 && z == 1) give_weights(phalf(b));
            }
            l += (sum[0].x + sum[0].y) + (sum[1].x + sum[1].y);
          }
          if (SPLIT > 1) {  // no weight on the other copies' positions
            const uint32_t zero[16] = {};
#pragma unroll 1
            for (int y = 0; y < 4; ++y)
              if (y < y0 || y >= y1) tmem_st_16(tS + 16 * y, zero);
          }
        } else if (W::PARTS == 2) {
          give_weights(phalf(b));
        }
        give_weights(pfull(b));
      }
      if (ok && asks) announce_q();
      if (ok && tiles > 0) ok = wait_warp(ofull(b), (no + tiles - 1) & 1);
      no += tiles;
      tile_no += n;
      // ---- the sums: PAIR: each stream has its rows; else the streams join,
      // stream b writing the b-th half of the columns
      float M = m, tot = l, fa = 1.0f, fb = 0.0f;
      const bool both = !PAIR && n > 1;
      if (!PAIR) {
        s_ml[b][row] = make_float2(m, l);
        if (!ok || !soft_sync()) {
          ok = false;
          break;
        }
        // (a stream without tiles has maximum -infinity and sum 0)
        M = -INFINITY;
#pragma unroll
        for (int c = 0; c < SPLIT; ++c)
          M = fmaxf(M, fmaxf(s_ml[0][irow + c * IROWS].x, s_ml[1][irow + c * IROWS].x));
        const float off = M == -INFINITY ? 0.0f : M;
        tot = 0.0f;
#pragma unroll
        for (int c = 0; c < SPLIT; ++c) {
          const float2 A = s_ml[0][irow + c * IROWS], B = s_ml[1][irow + c * IROWS];
          tot += A.y * exp2_fast(A.x - off) + B.y * exp2_fast(B.x - off);
        }
        fa = exp2_fast(s_ml[0][row].x - off);
        fb = both ? exp2_fast(s_ml[1][row].x - off) : 0.0f;
      }
      if (!ok) break;
      tc_fence_after_sync();
      const uint64_t spoilt = *(volatile uint32_t*)&bad_of[item_no % kBad][0] |
                              (uint64_t)*(volatile uint32_t*)&bad_of[item_no % kBad][1] << 32;
      const float poison = bits & spoilt ? __uint_as_float(0x7FC00000u) : 0.0f;
      const bool whole = w.u0 == 0 && w.u1 == w.nu;
      const float inv = tot == 0.0f ? 0.0f : 1.0f / tot;
      float4* slot4 = reinterpret_cast<float4*>(
          slots + part_slot(blockIdx.x, sched.per, w.start) * attend_slot_floats(IROWS, D));
      const int srow = (PAIR ? b * kRows : 0) + irow;  // row of the item
      __half* out = p.out + (int64_t)(si.first + node) * p.ldo + (int64_t)hq * D;
      const int c0 = PAIR ? 0 : b * (D / 2), c1 = PAIR ? D : (b + 1) * (D / 2);
      if (SPLIT > 1) {
        // the copies' sums, 16 columns at a time through shared memory
        float* cb = reinterpret_cast<float*>(gbase + W::CB_OFF) + b * kRows * kCopyPitch;
#pragma unroll 1
        for (int d0 = c0; d0 < c1 && ok; d0 += 16) {
          uint32_t v[16], u[16];
          if (!idle) {
            tmem_ld_16(tlane + kO0 + d0, v);
            if (both) tmem_ld_16(tlane + kO1 + d0, u);
            tmem_ld_wait();
#pragma unroll
            for (int k = 0; k < 16; k += 4) {
              float x[4];
#pragma unroll
              for (int z = 0; z < 4; ++z) {
                x[z] = __uint_as_float(v[k + z]) * fa + poison;
                if (both) x[z] += __uint_as_float(u[k + z]) * fb;
              }
              *reinterpret_cast<float4*>(cb + row * kCopyPitch + k) = make_float4(x[0], x[1], x[2], x[3]);
            }
          }
          if (d0 == c0) s_inv[b][row] = inv;
          ok = soft_sync();
          if (!ok) break;
          for (int id = threadIdx.x & 127; id < rows * 4; id += 128) {
            const int r = id >> 2, c4 = id & 3;
            float4 x = make_float4(0, 0, 0, 0);
#pragma unroll
            for (int c = 0; c < SPLIT; ++c) {
              const float4 t = *reinterpret_cast<const float4*>(cb + (r + c * IROWS) * kCopyPitch + 4 * c4);
              x.x += t.x, x.y += t.y, x.z += t.z, x.w += t.w;
            }
            const int d = d0 + 4 * c4;
            if (whole) {
              const int r2 = r0 + r;
              const float iv = s_inv[b][r];
              *reinterpret_cast<uint2*>(p.out + (int64_t)(si.first + heads.node(r2)) * p.ldo +
                                        (w.h * G + heads.head(r2)) * D + d) =
                  make_uint2(half2_of(x.x * iv, x.y * iv), half2_of(x.z * iv, x.w * iv));
            } else {
              slot4[d / 4 * IROWS + r] = x;
            }
          }
          ok = soft_sync();
        }
        if (!ok) break;
      } else if (!idle) {
#pragma unroll 1
        for (int d0 = c0; d0 < c1; d0 += 32) {
          uint32_t v[32], u[32];
          tmem_ld_32((PAIR ? tO : tlane + kO0) + d0, v);
          if (both) tmem_ld_32(tlane + kO1 + d0, u);
          tmem_ld_wait();
          float x[32];
#pragma unroll
          for (int k = 0; k < 32; ++k) {
            x[k] = __uint_as_float(v[k]) * fa + poison;
            if (both) x[k] += __uint_as_float(u[k]) * fb;
          }
          if (mine && whole) {
#pragma unroll
            for (int k = 0; k < 32; k += 8)
              *reinterpret_cast<uint4*>(out + d0 + k) =
                  make_uint4(half2_of(x[k] * inv, x[k + 1] * inv), half2_of(x[k + 2] * inv, x[k + 3] * inv),
                             half2_of(x[k + 4] * inv, x[k + 5] * inv),
                             half2_of(x[k + 6] * inv, x[k + 7] * inv));
          } else if (mine) {
#pragma unroll
            for (int k = 0; k < 32; k += 4)
              slot4[(d0 + k) / 4 * IROWS + srow] = make_float4(x[k], x[k + 1], x[k + 2], x[k + 3]);
          }
          __syncwarp();
        }
      }
      const bool writes = mine && (PAIR || (b == 0 && copy == 0));
      if (writes && whole && p.lse)
        p.lse[(int64_t)(si.first + node) * p.q_heads + hq] =
            tot == 0.0f ? -INFINITY : (M + log2f(tot)) * kLn2;
      if (writes && !whole) {
        float* f = reinterpret_cast<float*>(slot4) + IROWS * D;
        f[srow] = M;
        f[IROWS + srow] = tot;
      }
      // attend_join_kernel adds an item's parts: where they are
      if (w.u0 == 0 && threadIdx.x == 0) {
        const int64_t b0 = sched.block_of(w.start), b1 = sched.block_of(w.start + w.nu - 1);
        heads_of_items[w.item] = make_int4((int)part_slot(b0, sched.per, w.start), (int)b0, (int)(b1 - b0) + 1, 0);
      }
      ++item_no;
      tc_fence_before_sync();
      if (!PAIR) ok = soft_sync();  // nobody reads the other stream's sums any more
    }
    cp_async_wait_all();  // (queries asked for before a wait gave up)
  }

  // ---- teardown: MMAs that were issued are done before TMEM is freed
  __syncwarp();
  tc_fence_before_sync();
  __syncthreads();
  if (warp == kMmaWarp) {
    __shared__ uint64_t done_mem;
    const uint32_t done = smem_addr(&done_mem);
    if (lane == 0) {
      mbar_init(done, 1);
      fence_mbar_init();
    }
    __syncwarp();
    if (elect_one()) {  // the lane that issued them
      mma_commit(done);
      mbar_wait(done, 0, kWaitLimitNs, false);
    }
    __syncwarp();
    tc_fence_after_sync();
    tmem_dealloc(tmem, kTmemCols);
  }
}

// Adds the parts of the items that several blocks had: a block takes 32 rows and
// 32 C columns of an item, a thread a row and 4 C columns (warps side by side),
// B parts' loads in flight together.  A launch of its own: one block that added
// its item in the kernel above had 10 to 40 us of it.  Whole rows (C = D / 32)
// where the blocks then fill the device, else a quarter (half) of them: 128 items
// of 256 rows take 7 us more with C = 1, 8 of 32 rows 3 us more with C = 4.
template <int D, int IROWS, int C>
__global__ void __launch_bounds__(256) attend_join_kernel(AttendParams p, int rt_max, int blocks) {
  pdl_launch_dependents();
  pdl_wait_previous();
  const int G = p.q_heads / p.c.kv_heads;
  const int item = blockIdx.x, s = item / (p.c.kv_heads * rt_max), h = item / rt_max % p.c.kv_heads,
            rt = item % rt_max;
  const SeqInfo si = seq_info(p, s);
  const int rows = min(IROWS, si.n * G - rt * IROWS);
  const int r = blockIdx.y * 32 + (threadIdx.x & 31), warp = threadIdx.x >> 5;
  if ((int)blockIdx.y * 32 >= rows) return;
  const uint8_t* ws = p.workspace + attend_counter_bytes(blocks);
  const int4 head = reinterpret_cast<const int4*>(ws)[item];
  const int parts = head.z;
  // (an item without an entry, after a wait that gave up, reads in bounds)
  if (parts < 2 || parts > blocks || (uint32_t)head.x >= 2u * blocks || head.y < 0 || head.y > blocks - parts ||
      r >= rows)
    return;
  const float* slots =
      reinterpret_cast<const float*>(ws + join_head_bytes((int64_t)p.seqs * p.c.kv_heads * rt_max));
  const int c0 = ((int)blockIdx.z * 8 + warp) * C;  // the thread's first 16 bytes of a row
  constexpr int B = C == 4 ? 2 : 8;  // parts in flight
  // after the first, an item's part begins its block's range
  auto part = [&](int y) {
    return slots + (size_t)(y == 0 ? head.x : (head.y + y) * 2) * attend_slot_floats(IROWS, D);
  };
  float4 x[C], v[B][C];
  float pm[B];
  auto fetch = [&](int y0) {
#pragma unroll
    for (int j = 0; j < B; ++j) {
      const float* f = part(min(y0 + j, parts - 1));
      pm[j] = __ldcg(f + IROWS * D + r);
#pragma unroll
      for (int k = 0; k < C; ++k) v[j][k] = __ldcg(reinterpret_cast<const float4*>(f) + (c0 + k) * IROWS + r);
    }
  };
  fetch(0);
  const float2 ml = join_ml(parts, IROWS, [&](int y) { return part(y) + IROWS * D + r; });
  const float M = ml.x, tot = ml.y, off = M == -INFINITY ? 0.0f : M;
#pragma unroll
  for (int k = 0; k < C; ++k) x[k] = make_float4(0, 0, 0, 0);
  for (int y0 = 0; y0 < parts; y0 += B) {
    if (y0 > 0) fetch(y0);
#pragma unroll
    for (int j = 0; j < B; ++j) {
      if (y0 + j >= parts) break;
      const float g = exp2_fast(pm[j] - off);
#pragma unroll
      for (int k = 0; k < C; ++k)
        x[k].x += v[j][k].x * g, x[k].y += v[j][k].y * g, x[k].z += v[j][k].z * g, x[k].w += v[j][k].w * g;
    }
  }
  const float inv = tot == 0.0f ? 0.0f : 1.0f / tot;
  const Heads heads(G);
  const int rr = rt * IROWS + r, node = heads.node(rr), hq = h * G + heads.head(rr);
  __half* dst = p.out + (int64_t)(si.first + node) * p.ldo + hq * D + c0 * 4;
  uint2 y[C];
#pragma unroll
  for (int k = 0; k < C; ++k)
    y[k] = make_uint2(half2_of(x[k].x * inv, x[k].y * inv), half2_of(x[k].z * inv, x[k].w * inv));
  if (C == 1) {
    *reinterpret_cast<uint2*>(dst) = y[0];
  } else {
#pragma unroll
    for (int k = 0; k < C; k += 2)
      *reinterpret_cast<uint4*>(dst + 4 * k) = make_uint4(y[k].x, y[k].y, y[k + 1 < C ? k + 1 : k].x, y[k + 1 < C ? k + 1 : k].y);
  }
  if (c0 == 0 && p.lse)
    p.lse[(int64_t)(si.first + node) * p.q_heads + hq] = tot == 0.0f ? -INFINITY : (M + log2f(tot)) * kLn2;
}

// A cache's pages as {head_dim, kv_heads * page_size rows, pages}, in boxes of
// 64 elements and the rows of a page (at most a tile's).
bool encode_pages(CUtensorMap* m, const void* base, const CacheView& c, int head_dim) {
  const int rows = 1 << c.page_shift;
  const cuuint64_t dims[3] = {(cuuint64_t)head_dim, (cuuint64_t)c.kv_heads * rows, (cuuint64_t)c.pages};
  const cuuint64_t strides[2] = {(cuuint64_t)head_dim * 2, (cuuint64_t)c.page_stride * 2};
  const cuuint32_t box[3] = {64, (cuuint32_t)(rows < kKeys ? rows : kKeys), 1};
  return encode_tiled(m, CU_TENSOR_MAP_DATA_TYPE_FLOAT16, base, 3, dims, strides, box,
                      CU_TENSOR_MAP_SWIZZLE_128B);
}

template <int D, int TYPE, int MODE>
cudaError_t wide_one(const AttendParams& p, int sms, cudaStream_t stream) {
  using W = Wide<D, TYPE, MODE>;
  auto* k = attend_wide_kernel<D, TYPE, MODE>;
  static int done[64];
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  if (dev >= 64 || !__atomic_load_n(&done[dev], __ATOMIC_ACQUIRE)) {
    e = cudaFuncSetAttribute(k, cudaFuncAttributeMaxDynamicSharedMemorySize, W::SMEM);
    if (e != cudaSuccess) return e;
    if (dev < 64) __atomic_store_n(&done[dev], 1, __ATOMIC_RELEASE);
  }
  CUtensorMap tk, tv;
  if (TYPE == kCacheFp16) {
    if (!encode_pages(&tk, p.c.k, p.c, D) || !encode_pages(&tv, p.c.v, p.c, D)) return cudaErrorInvalidValue;
  } else {
    memset(&tk, 0, sizeof(tk));
    memset(&tv, 0, sizeof(tv));
  }
  e = launch_kernel(k, sms, W::THREADS, W::SMEM, stream, kFlagPdl, p, tk, tv);
  if (e != cudaSuccess) return e;
  constexpr int IROWS = W::IROWS;
  const int rows = p.max_nodes * (p.q_heads / p.c.kv_heads), rt_max = (rows + IROWS - 1) / IROWS;
  const dim3 grid((unsigned)(p.seqs * p.c.kv_heads * rt_max), (unsigned)((rows < IROWS ? rows : IROWS) + 31) / 32);
  // whole rows of threads where that fills the device, else a quarter (half)
  cudaLaunchConfig_t cfg = {};
  const bool narrow = grid.x * grid.y < (unsigned)sms;
  cfg.gridDim = dim3(grid.x, grid.y, narrow ? D / 32 : 1);
  cfg.blockDim = dim3(256);
  cfg.stream = stream;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return narrow ? cudaLaunchKernelEx(&cfg, attend_join_kernel<D, IROWS, 1>, p, rt_max, sms)
                : cudaLaunchKernelEx(&cfg, attend_join_kernel<D, IROWS, D / 32>, p, rt_max, sms);
}

template <int D, int TYPE>
cudaError_t wide_rows(const AttendParams& p, int sms, cudaStream_t stream) {
  switch (wide_mode(p.max_nodes * (p.q_heads / p.c.kv_heads))) {
    case 4: return wide_one<D, TYPE, 4>(p, sms, stream);
    case 2: return wide_one<D, TYPE, 2>(p, sms, stream);
    case 1: return wide_one<D, TYPE, 1>(p, sms, stream);
    default: return wide_one<D, TYPE, 0>(p, sms, stream);
  }
}

}  // namespace

// One translation unit for each type (attend_wide_*.cu).
template <int TYPE>
cudaError_t launch_attend_wide(const AttendParams& p, int head_dim, int sms, cudaStream_t stream) {
  return head_dim == 128 ? wide_rows<128, TYPE>(p, sms, stream) : wide_rows<64, TYPE>(p, sms, stream);
}

template <int TYPE>
cudaError_t read_attend_wait_timeouts(unsigned long long* count, int reset) {
  return read_local_wait_timeouts(count, reset);
}

}  // namespace nmk
