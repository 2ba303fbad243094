// attend_wide.cu -- nm_tree_attention for many query rows per key head: 128
// rows at a time on tcgen05.
//
// A block has 128 query rows in shared memory and walks the positions in tiles
// of 128.  Two streams take the tiles in turn, each with a score tile, sums and
// running maxima of its own, so that one's softmax runs while the tensor core
// works for the other; they join at the item's end (attend.cu has the rule).
//   loaders  bring K and V tiles into a ring of stages of fp16, 128-byte
//            swizzled rows: cp.async for an fp16 cache; codes go through a raw
//            ring (every thread copies, widens and stores pieces of its own).
//   MMA      one thread: S = Q K^T into TMEM; O += P V with P from TMEM and V
//            as the MN-major operand (its rows are the reduction's).
//   softmax  two warpgroups, a query row per thread: scores from TMEM, weights
//            back over them as fp16.  The maximum that scales a row moves only
//            when a score exceeds it by 2^8 (fp16 weights reach 2^8 then, at the
//            same relative rounding), so the sums in TMEM are seldom rescaled.
// With 8-bit caches the product with V takes codes: the weight of position j is
// 2^(s_j + log2 v_j - m), v_j the row's scale, and the sum of weights adds
// w_j / v_j; a key's scale multiplies its score.  So codes enter the MMA
// exactly and a weight is rounded once.
#include <cuda_fp16.h>
#include <cuda_runtime.h>
#include <stdint.h>

#include "attend.cuh"
#include "decode.h"
#include "device.cuh"
#include "kernels.h"
#include "tc.cuh"
#include "widen.cuh"

namespace nmk {
namespace {

constexpr int kRows = 128, kKeys = 128;
constexpr int kSoftWarps = 8, kMmaWarp = 8, kLoadWarp = 9;
constexpr int kMeta = 8;    // tiles whose scales are kept (see Wide)
constexpr int kBad = 16;    // items whose spoilt nodes are kept
constexpr float kGrow = 8.0f;
constexpr float kTinyScale = 7.888609052210118e-31f;  // 2^-100: a zero scale counts as this

template <int D, int TYPE>
struct Wide {
  static constexpr bool F16 = TYPE == kCacheFp16;
  static constexpr int LW = F16 ? 4 : 8;  // loader warps
  static constexpr int THREADS = 32 * (kLoadWarp + LW);
  static constexpr int TILE = kKeys * D * 2;  // bytes of a stage
  static constexpr int HALF = kKeys * 128;    // 64 elements of every row
  // K and V tiles in the order of their use; at most 8 (a slot of kMeta is
  // written again 8 tiles on, when at least the tile 4 before was consumed)
  static constexpr int NS = F16 ? (D == 128 ? 5 : 8) : (D == 128 ? 3 : 6);
  static constexpr int LAG = 3;               // fp16: positions copied ahead of their announcement
  static constexpr int RS = F16 ? 0 : 4;      // raw tiles in flight
  static constexpr int RAW = kKeys * D;
  static constexpr int Q_OFF = 0;
  static constexpr int ST_OFF = Q_OFF + kRows * D * 2;
  static constexpr int RAW_OFF = ST_OFF + NS * TILE;
  static constexpr int SC_OFF = RAW_OFF + RS * RAW;  // 8-bit: raw k, raw v, k', log2 v, 1 / v
  static constexpr int BYTES = SC_OFF + (F16 ? 0 : 5 * kMeta * kKeys * 4);
  static constexpr int SMEM = BYTES + 1024;   // room to align the base
  static_assert(SMEM <= 227 * 1024 - 4096, "static shared memory needs room too");
  static_assert(NS <= 8 && (!F16 || LAG < NS), "see above");
};

// TMEM columns.
constexpr uint32_t kS0 = 0, kS1 = 128, kO0 = 256, kO1 = 384, kTmemCols = 512;

template <int D, int TYPE>
__global__ void __launch_bounds__(Wide<D, TYPE>::THREADS, 1) attend_wide_kernel(AttendParams p) {
  using W = Wide<D, TYPE>;
  constexpr bool F16 = W::F16;
  using Sched = Schedule<kRows, kKeys, W::THREADS>;
  extern __shared__ uint8_t raw_smem[];
  __shared__ uint64_t bar_mem[2 * W::NS + 8];
  __shared__ uint32_t tmem_slot, s_last;
  __shared__ uint32_t there_of[kMeta];
  __shared__ uint32_t bad_of[kBad][2];
  __shared__ float2 s_ml[2][kRows];
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

  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  pdl_launch_dependents();
  pdl_wait_previous();
  if (__syncthreads_or(threadIdx.x == 0 && wait_aborted())) return;
  Sched sched;
  if (!sched.init(p, 1)) return;

  if (warp == 0 && lane == 0) {
    for (int s = 0; s < W::NS; ++s) {
      mbar_init(full(s), W::LW);
      mbar_init(empty(s), 1);
    }
    for (int b = 0; b < 2; ++b) {
      mbar_init(sfull(b), 1);
      mbar_init(pfull(b), 4);
      mbar_init(ofull(b), 1);
    }
    mbar_init(qfull, kSoftWarps);
    mbar_init(soft, kSoftWarps);
    fence_mbar_init();
  }
  if (threadIdx.x < kBad * 2) bad_of[threadIdx.x / 2][threadIdx.x % 2] = 0;
  if (warp == kMmaWarp) {
    tmem_alloc(smem_addr(&tmem_slot), kTmemCols);
    tmem_relinquish();
  }
  tc_fence_before_sync();
  __syncthreads();
  tc_fence_after_sync();
  const uint32_t tmem = *(volatile uint32_t*)&tmem_slot;
  const int G = p.q_heads / p.c.kv_heads;
  const float cs = fabsf(p.scale) * kLog2e;  // a negative scale's sign goes to the queries
  auto wait_warp = [&](uint32_t bar, uint32_t par) {
    return __all_sync(0xFFFFFFFFu, mbar_wait(bar, par)) != 0;
  };

  if (warp >= kLoadWarp) {
    // ---- loaders ---------------------------------------------------------------
    const int lw = warp - kLoadWarp;
    int c = 0, said = 0;  // positions of the ring issued and announced
    int tile_no = 0, item_no = 0;
    bool ok = true;
    auto announce = [&](int upto) {
      for (; said < upto; ++said) {
        fence_proxy_async_smem();
        __syncwarp();
        if (lane == 0) mbar_arrive(full(said % W::NS));
      }
    };
    auto acquire = [&](int pos) {  // the stage of ring position pos
      if (pos < W::NS) return true;
      return wait_warp(empty(pos % W::NS), (pos / W::NS - 1) & 1);
    };
    struct Raw {  // what a raw tile is (8-bit)
      int v, edge, node0, bad, meta;
    };
    Raw ring[F16 ? 1 : W::RS];

    // 8-bit: widen the pieces that this thread copied for position pos.
    auto convert = [&](int pos, const Raw& t) {
      if (!acquire(pos)) return false;
      const uint32_t dst = sT + (pos % W::NS) * W::TILE;
      const uint32_t src = base + W::RAW_OFF + (pos % (F16 ? 1 : W::RS)) * W::RAW;
      constexpr int PR = D / 16;  // pieces of a row
      const int lt = lw * 32 + lane;
#pragma unroll
      for (int i = 0; i < kKeys * PR / (W::LW * 32); ++i) {
        const int id = lt + i * W::LW * 32, r = id / PR, ch = id % PR;
        uint32_t w[4], h[8];
        asm volatile("ld.shared.v4.u32 {%0,%1,%2,%3}, [%4];"
                     : "=r"(w[0]), "=r"(w[1]), "=r"(w[2]), "=r"(w[3])
                     : "r"(src + id * 16));
#pragma unroll
        for (int k = 0; k < 4; ++k) widen4<F16 ? kCacheE4m3 : TYPE>(w[k], h[2 * k], h[2 * k + 1]);
        if (TYPE == kCacheE4m3 && t.v && t.edge && t.node0 + r >= 0) {
          uint32_t any = 0;
#pragma unroll
          for (int k = 0; k < 8; ++k) {
            const uint32_t b = bad_halves(h[k]);
            any |= b;
            h[k] &= (b & 1u ? 0u : 0xFFFFu) | (b & 2u ? 0u : 0xFFFF0000u);
          }
          if (any) atomicOr(&bad_of[t.bad][((t.node0 + r) >> 5) & 1], 1u << ((t.node0 + r) & 31));
        }
        const uint32_t at = dst + (ch >> 2) * W::HALF + r * 128;
        const uint32_t c0 = (ch & 3) * 2;
#pragma unroll
        for (int k = 0; k < 2; ++k)
          asm volatile("st.shared.v4.u32 [%0], {%1,%2,%3,%4};" ::"r"(at + (((c0 + k) ^ (r & 7)) << 4)),
                       "r"(h[4 * k]), "r"(h[4 * k + 1]), "r"(h[4 * k + 2]), "r"(h[4 * k + 3])
                       : "memory");
      }
      if (!t.v) {  // the tile's scales: k' = k scale log2(e), log2 v, 1 / v
        const int r = lt & (kKeys - 1);
        const float x = scales[(lt < kKeys ? 0 : kMeta * kKeys) + t.meta * kKeys + r];
        if (lt < kKeys) {
          scales[2 * kMeta * kKeys + t.meta * kKeys + r] = x * cs;
        } else {
          float lv = log2f(x), rv = 1.0f / x;
          if (x < kTinyScale) lv = -100.0f, rv = 1.0f / kTinyScale;
          const int j = t.node0 + r;
          if (t.edge && j >= 0 && !(x < INFINITY)) {  // a node's row with a scale that is not finite
            lv = 0.0f, rv = 1.0f;
            atomicOr(&bad_of[t.bad][(j >> 5) & 1], 1u << (j & 31));
          }
          scales[3 * kMeta * kKeys + t.meta * kKeys + r] = lv;
          scales[4 * kMeta * kKeys + t.meta * kKeys + r] = rv;
        }
      }
      return true;
    };

    Span w;
    SeqInfo si;
    while (ok && sched.next(p, w, si)) {
      const int32_t* table = p.table + (int64_t)w.s * p.ld_table;
      const int n = w.u1 - w.u0;
      const int bad_slot = item_no % kBad;
      auto look_up = [&](int i) {  // lane l: the page of the tile's l-th group of 8
        const int64_t pos = (int64_t)(w.u0 + i) * kKeys + 8 * lane;
        return i < n && lane < 16 && pos < si.len ? table[pos >> p.c.page_shift] : -1;
      };
      // Position c of the ring: K (v false) or V of tile i, whose groups of
      // rows begin at `at`.
      auto emit = [&](bool v, int i, const RowAt& at) {
        const int64_t pos0 = (int64_t)(w.u0 + i) * kKeys;
        const bool edge = pos0 + kKeys > si.ctx;
        const int left = (int)min((int64_t)kKeys, si.len - pos0);  // rows that are there
        const uint8_t* from = v ? p.c.v : p.c.k;
        if (F16) {
          if (c >= W::NS && !__all_sync(0xFFFFFFFFu, mbar_test(empty(c % W::NS), (c / W::NS - 1) & 1))) {
            cp_async_wait_group<0>();  // what has landed is announced before this warp waits
            announce(c);
          }
          if (!acquire(c)) return false;
          if (!v && lw == 0 && lane == 0) {
            if (i == 0) bad_of[(item_no + kBad / 2) % kBad][0] = bad_of[(item_no + kBad / 2) % kBad][1] = 0;
          }
          if (!v && lw == 0) {
            const uint32_t there = __ballot_sync(0xFFFFFFFFu, lane < 16 && at.code >= 0) & 0xFFFFu;
            if (lane == 0) there_of[tile_no % kMeta] = there;
          }
          const uint32_t dst = sT + (c % W::NS) * W::TILE;
          constexpr int PR = D / 8, PI = 32 / PR;  // pieces of a row, rows of an instruction
          const bool slow = v && edge;
#pragma unroll 4
          for (int k = 0; k < 32 / PI; ++k) {
            const int r = lw * 32 + k * PI + lane / PR, ch = lane % PR;
            const int64_t code = __shfl_sync(0xFFFFFFFFu, at.code, r >> 3);
            const bool on = code >= 0 && r < left;
            const uint8_t* src = from + ((on ? code : 0) + (r & 7) * D + ch * 8) * 2;
            const uint32_t to = dst + (ch >> 3) * W::HALF + r * 128 + (((ch & 7) ^ (r & 7)) << 4);
            if (!slow) {
              cp_async_16(to, src, on ? 16u : 0u);
            } else {  // value rows of nodes: an infinity or NaN must not meet a weight of 0
              uint4 x = make_uint4(0, 0, 0, 0);
              if (on) x = ld_stream_v4(src);
              uint32_t h[4] = {x.x, x.y, x.z, x.w}, any = 0;
              const int64_t j = pos0 + r - si.ctx;
              if (j >= 0) {
#pragma unroll
                for (int y = 0; y < 4; ++y) {
                  const uint32_t b = bad_halves(h[y]);
                  any |= b;
                  h[y] &= (b & 1u ? 0u : 0xFFFFu) | (b & 2u ? 0u : 0xFFFF0000u);
                }
                if (any) atomicOr(&bad_of[bad_slot][((int)j >> 5) & 1], 1u << ((int)j & 31));
              }
              asm volatile("st.shared.v4.u32 [%0], {%1,%2,%3,%4};" ::"r"(to), "r"(h[0]), "r"(h[1]),
                           "r"(h[2]), "r"(h[3])
                           : "memory");
            }
          }
          cp_async_commit();
          ++c;
          if (c - said > W::LAG) {
            cp_async_wait_group<W::LAG>();
            announce(c - W::LAG);
          }
        } else {
          constexpr int RS = F16 ? 1 : W::RS;
          if (c >= RS) {  // the raw slot's last tile goes first
            cp_async_wait_group<RS - 1>();
            if (!convert(c - RS, ring[c % RS])) return false;
            announce(c - RS + 1);
          }
          if (!v && lw == 0) {
            const uint32_t there = __ballot_sync(0xFFFFFFFFu, lane < 16 && at.code >= 0) & 0xFFFFu;
            if (lane == 0) {
              there_of[tile_no % kMeta] = there;
              if (i == 0)
                bad_of[(item_no + kBad / 2) % kBad][0] = bad_of[(item_no + kBad / 2) % kBad][1] = 0;
            }
          }
          const uint32_t dst = base + W::RAW_OFF + (c % RS) * W::RAW;
          constexpr int PR = D / 16;
          const int lt = lw * 32 + lane;
#pragma unroll
          for (int k = 0; k < kKeys * PR / (W::LW * 32); ++k) {
            const int id = lt + k * W::LW * 32, r = id / PR, ch = id % PR;
            const int64_t code = __shfl_sync(0xFFFFFFFFu, at.code, r >> 3);
            const bool on = code >= 0 && r < left;
            cp_async_16(dst + id * 16, from + (on ? code : 0) + (r & 7) * D + ch * 16, on ? 16u : 0u);
          }
          if (!v) {
            const int r = lt & (kKeys - 1);
            const int64_t sc = __shfl_sync(0xFFFFFFFFu, at.scale, r >> 3);
            const bool on = sc >= 0 && r < left;
            const float* f = (lt < kKeys ? p.c.k_scale : p.c.v_scale) + (on ? sc : 0) + (r & 7);
            cp_async_4(smem_addr(scales + (lt < kKeys ? 0 : kMeta * kKeys) +
                                 (tile_no % kMeta) * kKeys + r),
                       on ? f : p.c.k_scale, on ? 4u : 0u);
          }
          cp_async_commit();
          ring[c % RS] = Raw{v ? 1 : 0, edge ? 1 : 0, (int)max(pos0 - si.ctx, (int64_t)-(1 << 20)),
                             bad_slot, tile_no % kMeta};
          ++c;
        }
        if (!v) ++tile_no;
        return true;
      };
      // K0, K1, V0, K2, V1, ...: the order in which the MMA thread takes them
      int32_t entry = look_up(0);
      RowAt now{-1, -1}, last{-1, -1};
      for (int i = 0; i <= n && ok; ++i) {
        if (i < n) {
          now = group_at<D>(p, entry, w.h, (int64_t)(w.u0 + i) * kKeys + 8 * (lane & 15));
          entry = look_up(i + 1);
          ok = emit(false, i, now);
        }
        if (ok && i > 0) ok = emit(true, i - 1, last);
        last = now;
      }
      ++item_no;
    }
    if (F16) {
      cp_async_wait_group<0>();
      if (ok) announce(c);
    } else {
      constexpr int RS = F16 ? 1 : W::RS;
      cp_async_wait_group<0>();
      for (int pos = max(0, c - RS); ok && pos < c; ++pos) {
        ok = convert(pos, ring[pos % RS]);
        if (ok) announce(pos + 1);
      }
    }
    // every release of a stage has landed before the block ends
    for (int pos = max(0, c - W::NS); ok && pos < c; ++pos) ok = wait_warp(empty(pos % W::NS), (pos / W::NS) & 1);
  } else if (warp == kMmaWarp) {
    // ---- MMA issuer ----------------------------------------------------------------
    if (lane == 0) {
      constexpr uint32_t id_s = idesc_f16_f32(kRows, kKeys);
      constexpr uint32_t id_o = idesc_f16_f32(kRows, D) | kIdescBMajorMN;
      int c = 0, items = 0, np[2] = {0, 0};
      bool ok = true;
      Span w;
      SeqInfo si;
      auto scores = [&](int i) {
        const int st = c % W::NS;
        if (!mbar_wait(full(st), (c / W::NS) & 1)) return false;
        fence_proxy_async_smem();
        tc_fence_after_sync();
        const uint32_t d = tmem + ((i & 1) ? kS1 : kS0), b = sT + st * W::TILE;
#pragma unroll
        for (int ks = 0; ks < D / 16; ++ks) {
          const uint32_t off = (ks >> 2) * W::HALF + (ks & 3) * 32;
          mma_f16(d, smem_desc_sw128(sQ + off, 16), smem_desc_sw128(b + off, 16), id_s, ks != 0);
        }
        mma_commit(empty(st));
        mma_commit(sfull(i & 1));
        ++c;
        return true;
      };
      while (ok && sched.next(p, w, si)) {
        const int n = w.u1 - w.u0;
        if (!mbar_wait(qfull, items & 1)) break;
        fence_proxy_async_smem();
        ++items;
        ok = scores(0);
        for (int i = 0; i < n && ok; ++i) {
          if (i + 1 < n && !scores(i + 1)) {
            ok = false;
            break;
          }
          const int st = c % W::NS, b = i & 1;
          ok = mbar_wait(full(st), (c / W::NS) & 1) && mbar_wait(pfull(b), np[b] & 1);
          if (!ok) break;
          ++np[b];
          fence_proxy_async_smem();
          tc_fence_after_sync();
          const uint32_t d = tmem + (b ? kO1 : kO0), a = tmem + (b ? kS1 : kS0);
#pragma unroll
          for (int ks = 0; ks < kKeys / 16; ++ks)
            mma_f16_ts(d, a + ks * 8, smem_desc_sw128(sT + st * W::TILE + ks * 2048, W::HALF), id_o,
                       i > 1 || ks != 0);
          mma_commit(empty(st));
          mma_commit(ofull(b));
          ++c;
        }
      }
    }
    __syncwarp();
  } else {
    // ---- softmax -------------------------------------------------------------------
    const int b = warp >> 2, row = (warp & 3) * 32 + lane;
    const uint32_t tlane = tmem + ((uint32_t)((warp & 3) * 32) << 16);
    const uint32_t tS = tlane + (b ? kS1 : kS0), tO = tlane + (b ? kO1 : kO0);
    int tile_no = 0, item_no = 0, ns = 0, no = 0, phase = 0;
    auto soft_sync = [&]() {  // all softmax warps
      __syncwarp();
      if (lane == 0) mbar_arrive(soft);
      return wait_warp(soft, phase++ & 1);
    };
    int* counters = reinterpret_cast<int*>(p.workspace);
    float* slots = reinterpret_cast<float*>(
        p.workspace + attend_counter_bytes((int64_t)p.seqs * p.c.kv_heads * sched.rt_max));
    bool ok = true;
    Span w;
    SeqInfo si;
    while (ok && sched.next(p, w, si)) {
      const int n = w.u1 - w.u0;
      const int rows = min(kRows, si.n * G - w.rt * kRows);
      // queries: every score product of the last item is done
      for (int id = threadIdx.x; id < kRows * (D / 8); id += kSoftWarps * 32) {
        const int r = id / (D / 8), ch = id % (D / 8), rr = w.rt * kRows + r;
        uint4 x = make_uint4(0, 0, 0, 0);
        if (r < rows)
          x = *reinterpret_cast<const uint4*>(p.q + (int64_t)(si.first + rr / G) * p.ldq +
                                              (int64_t)(w.h * G + rr % G) * D + ch * 8);
        const uint32_t sg = p.scale < 0.0f ? 0x80008000u : 0u;
        asm volatile("st.shared.v4.u32 [%0], {%1,%2,%3,%4};" ::"r"(
                         sQ + (ch >> 3) * W::HALF + r * 128 + (((ch & 7) ^ (r & 7)) << 4)),
                     "r"(x.x ^ sg), "r"(x.y ^ sg), "r"(x.z ^ sg), "r"(x.w ^ sg)
                     : "memory");
      }
      fence_proxy_async_smem();
      __syncwarp();
      if (lane == 0) mbar_arrive(qfull);

      const int rr = w.rt * kRows + row, node = rr / G;
      const bool mine = row < rows;
      const uint64_t bits = !mine ? 0ull
                            : p.tree_mask ? p.tree_mask[si.first + node]
                                          : (2ull << node) - 1ull;
      const bool idle = (warp & 3) * 32 >= rows;  // a warp without rows
      float m = -INFINITY, l = 0.0f;
      for (int i = b; i < n; i += 2) {
        ok = wait_warp(sfull(b), ns++ & 1);
        // (the sums up to here were issued before these scores: no further wait,
        // but every phase of a barrier is seen, so that its parity says which)
        if (ok && i > b) ok = wait_warp(ofull(b), (no + (i - b) / 2 - 1) & 1);
        if (!ok) break;
        if (!idle) {
          tc_fence_after_sync();
          const int slot = (tile_no + i) % kMeta;
          const int64_t pos0 = (int64_t)(w.u0 + i) * kKeys;
          const uint32_t there = *(volatile uint32_t*)&there_of[slot];
          const bool edge = pos0 + kKeys > si.ctx || there != 0xFFFFu;
          const float* ksc = scales + 2 * kMeta * kKeys + slot * kKeys;
          const float* lvs = ksc + kMeta * kKeys;
          const float* rvs = lvs + kMeta * kKeys;
          // what the row sees of an edge tile: position x of it in bit x
          uint32_t see[4] = {~0u, ~0u, ~0u, ~0u};
          if (edge) {
            const int64_t k0 = pos0 - si.ctx;  // node number of position 0
#pragma unroll
            for (int y = 0; y < 4; ++y) {
              const int64_t f = k0 + 32 * y;
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
              see[y] = x;
            }
          }
          // the exponent of position x of chunk y, in powers of 2
          auto exponent = [&](float s, int y, int x) {
            const float t = F16 ? s * cs : fmaf(s, ksc[32 * y + x], lvs[32 * y + x]);
            return edge && !((see[y] >> x) & 1u) ? -INFINITY : t;
          };
          float top = -INFINITY;
#pragma unroll
          for (int y = 0; y < 4; ++y) {
            uint32_t v[32];
            tmem_ld_32(tS + 32 * y, v);
            tmem_ld_wait();
            if (F16 && !edge) {
              float t = __uint_as_float(v[0]);
#pragma unroll
              for (int x = 1; x < 32; ++x) t = fmaxf(t, __uint_as_float(v[x]));
              top = fmaxf(top, t * cs);
            } else {
#pragma unroll
              for (int x = 0; x < 32; ++x) top = fmaxf(top, exponent(__uint_as_float(v[x]), y, x));
            }
          }
          const bool grow = top > m + kGrow || (m == -INFINITY && top > -INFINITY);
          const float m2 = grow ? top : m;
          if (i > b && __any_sync(0xFFFFFFFFu, grow)) {  // there are sums so far
            const float keep = !grow ? 1.0f : m == -INFINITY ? 0.0f : exp2_fast(m - m2);
#pragma unroll 1
            for (int y = 0; y < D; y += 32) {
              uint32_t v[32];
              tmem_ld_32(tO + y, v);
              tmem_ld_wait();
#pragma unroll
              for (int x = 0; x < 32; ++x) v[x] = __float_as_uint(__uint_as_float(v[x]) * keep);
              tmem_st_32(tO + y, v);
            }
            l *= keep;
          }
          m = m2;
          const float off = m == -INFINITY ? 0.0f : m;
          float sum[2] = {0.0f, 0.0f};
#pragma unroll
          for (int y = 0; y < 4; ++y) {
            uint32_t v[32], h[16];
            tmem_ld_32(tS + 32 * y, v);
            tmem_ld_wait();
#pragma unroll
            for (int x = 0; x < 32; ++x) {
              const float s = __uint_as_float(v[x]);
              const float e = F16 && !edge ? exp2_fast(fmaf(s, cs, -off))
                                           : exp2_fast(exponent(s, y, x) - off);
              if (F16)
                sum[x & 1] += e;
              else
                sum[x & 1] = fmaf(e, rvs[32 * y + x], sum[x & 1]);
              v[x] = __float_as_uint(e);
            }
#pragma unroll
            for (int x = 0; x < 16; ++x) {
              const __half2 t = __floats2half2_rn(__uint_as_float(v[2 * x]), __uint_as_float(v[2 * x + 1]));
              h[x] = *reinterpret_cast<const uint32_t*>(&t);
            }
            tmem_st_16(tS + 16 * y, h);
          }
          l += sum[0] + sum[1];
          tmem_st_wait();
        }
        tc_fence_before_sync();
        __syncwarp();
        if (lane == 0) mbar_arrive(pfull(b));
      }
      const int mine_tiles = (n - b + 1) / 2;
      if (ok && mine_tiles > 0) ok = wait_warp(ofull(b), (no + mine_tiles - 1) & 1);
      no += mine_tiles;
      tile_no += n;
      // ---- the streams join: columns of the first half here, of the second there
      s_ml[b][row] = make_float2(m, l);
      if (!ok || !soft_sync()) {
        ok = false;
        break;
      }
      tc_fence_after_sync();
      const float2 A = s_ml[0][row], B = s_ml[1][row];
      const float M = fmaxf(A.x, B.x), off = M == -INFINITY ? 0.0f : M;
      const float fa = exp2_fast(A.x - off), fb = n > 1 ? exp2_fast(B.x - off) : 0.0f;
      const float tot = A.y * fa + (n > 1 ? B.y * fb : 0.0f);
      const uint64_t spoilt = *(volatile uint32_t*)&bad_of[item_no % kBad][0] |
                              (uint64_t)*(volatile uint32_t*)&bad_of[item_no % kBad][1] << 32;
      const float poison = bits & spoilt ? __uint_as_float(0x7FC00000u) : 0.0f;
      const bool whole = w.u0 == 0 && w.u1 == w.nu;
      const float inv = tot == 0.0f ? 0.0f : 1.0f / tot;
      float4* slot4 = reinterpret_cast<float4*>(
          slots + part_slot(blockIdx.x, sched.per, w.start) * attend_slot_floats(kRows, D));
      __half* out = p.out + (int64_t)(si.first + node) * p.ldo + (int64_t)(w.h * G + rr % G) * D;
      if (!idle) {
#pragma unroll 1
        for (int y = 0; y < D / 2; y += 32) {
          const int d0 = b * (D / 2) + y;
          uint32_t v[32], u[32];
          tmem_ld_32(tlane + kO0 + d0, v);
          if (n > 1) tmem_ld_32(tlane + kO1 + d0, u);
          tmem_ld_wait();
          float x[32];
#pragma unroll
          for (int k = 0; k < 32; ++k) {
            x[k] = __uint_as_float(v[k]) * fa + poison;
            if (n > 1) x[k] += __uint_as_float(u[k]) * fb;
          }
          if (mine && whole) {
#pragma unroll
            for (int k = 0; k < 32; k += 8) {
              uint32_t h[4];
#pragma unroll
              for (int z = 0; z < 4; ++z) {
                const __half2 t = __floats2half2_rn(x[k + 2 * z] * inv, x[k + 2 * z + 1] * inv);
                h[z] = *reinterpret_cast<const uint32_t*>(&t);
              }
              *reinterpret_cast<uint4*>(out + d0 + k) = make_uint4(h[0], h[1], h[2], h[3]);
            }
          } else if (mine) {
#pragma unroll
            for (int k = 0; k < 32; k += 4)
              slot4[(d0 + k) / 4 * kRows + row] = make_float4(x[k], x[k + 1], x[k + 2], x[k + 3]);
          }
          __syncwarp();
        }
      }
      if (mine && b == 0) {
        if (whole) {
          if (p.lse)
            p.lse[(int64_t)(si.first + node) * p.q_heads + w.h * G + rr % G] =
                tot == 0.0f ? -INFINITY : (M + log2f(tot)) * kLn2;
        } else {
          float* f = reinterpret_cast<float*>(slot4) + kRows * D;
          f[row] = M;
          f[kRows + row] = tot;
        }
      }
      ++item_no;
      tc_fence_before_sync();
      if (whole) {
        ok = soft_sync();  // nobody reads TMEM any more
        continue;
      }
      // ---- the blocks join: the last one to store its part adds all of them
      const int64_t b0 = sched.block_of(w.start), b1 = sched.block_of(w.start + w.nu - 1);
      __threadfence();
      ok = soft_sync();
      if (!ok) break;
      if (threadIdx.x == 0) {
        const bool last = atomicAdd(counters + w.item, 1) == (int)(b1 - b0);
        if (last) counters[w.item] = 0;  // ready for the next call
        __threadfence();
        s_last = last;
      }
      ok = soft_sync();
      if (!ok) break;
      if (!*(volatile uint32_t*)&s_last) continue;
      if (mine) {
      __threadfence();
      float M2 = -INFINITY, tot2 = 0.0f;
      for (int64_t y = b0; y <= b1; ++y)
        M2 = fmaxf(M2, __ldcg(slots + part_slot(y, sched.per, w.start) * attend_slot_floats(kRows, D) +
                              kRows * D + row));
      const float off2 = M2 == -INFINITY ? 0.0f : M2;
      for (int64_t y = b0; y <= b1; ++y) {
        const float* f = slots + part_slot(y, sched.per, w.start) * attend_slot_floats(kRows, D) + kRows * D;
        tot2 += __ldcg(f + kRows + row) * exp2_fast(__ldcg(f + row) - off2);
      }
      const float inv2 = tot2 == 0.0f ? 0.0f : 1.0f / tot2;
#pragma unroll 1
      for (int d0 = b * (D / 2); d0 < (b + 1) * (D / 2); d0 += 16) {
        float4 x[4];
#pragma unroll
        for (int k = 0; k < 4; ++k) x[k] = make_float4(0, 0, 0, 0);
#pragma unroll 2
        for (int64_t y = b0; y <= b1; ++y) {
          const float* f = slots + part_slot(y, sched.per, w.start) * attend_slot_floats(kRows, D);
          const float e = exp2_fast(__ldcg(f + kRows * D + row) - off2);
#pragma unroll
          for (int k = 0; k < 4; ++k) {
            const float4 v = __ldcg(reinterpret_cast<const float4*>(f) + (d0 / 4 + k) * kRows + row);
            x[k].x += v.x * e, x[k].y += v.y * e, x[k].z += v.z * e, x[k].w += v.w * e;
          }
        }
#pragma unroll
        for (int k = 0; k < 4; k += 2) {
          const __half2 h0 = __floats2half2_rn(x[k].x * inv2, x[k].y * inv2);
          const __half2 h1 = __floats2half2_rn(x[k].z * inv2, x[k].w * inv2);
          const __half2 h2 = __floats2half2_rn(x[k + 1].x * inv2, x[k + 1].y * inv2);
          const __half2 h3 = __floats2half2_rn(x[k + 1].z * inv2, x[k + 1].w * inv2);
          *reinterpret_cast<uint4*>(out + d0 + 4 * k) =
              make_uint4(*reinterpret_cast<const uint32_t*>(&h0), *reinterpret_cast<const uint32_t*>(&h1),
                         *reinterpret_cast<const uint32_t*>(&h2), *reinterpret_cast<const uint32_t*>(&h3));
        }
      }
      if (b == 0 && p.lse)
        p.lse[(int64_t)(si.first + node) * p.q_heads + w.h * G + rr % G] =
            tot2 == 0.0f ? -INFINITY : (M2 + log2f(tot2)) * kLn2;
      }
      __syncwarp();
    }
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
      mma_commit(done);
      mbar_wait(done, 0, kWaitLimitNs, false);
    }
    __syncwarp();
    tc_fence_after_sync();
    tmem_dealloc(tmem, kTmemCols);
  }
}

template <int D, int TYPE>
cudaError_t wide_one(const AttendParams& p, int sms, cudaStream_t stream) {
  using W = Wide<D, TYPE>;
  auto* k = attend_wide_kernel<D, TYPE>;
  static int done[64];
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  if (dev >= 64 || !__atomic_load_n(&done[dev], __ATOMIC_ACQUIRE)) {
    e = cudaFuncSetAttribute(k, cudaFuncAttributeMaxDynamicSharedMemorySize, W::SMEM);
    if (e != cudaSuccess) return e;
    if (dev < 64) __atomic_store_n(&done[dev], 1, __ATOMIC_RELEASE);
  }
  return launch_kernel(k, sms, W::THREADS, W::SMEM, stream, kFlagPdl, p);
}

}  // namespace

size_t attend_wide_workspace_bytes(int64_t items, int head_dim, int sms) {
  return attend_counter_bytes(items) + (size_t)sms * 2 * attend_slot_floats(kRows, head_dim) * sizeof(float);
}

cudaError_t launch_attend_wide(const AttendParams& p, int head_dim, int type, int sms,
                               cudaStream_t stream) {
  if (head_dim == 128) {
    if (type == kCacheFp16) return wide_one<128, kCacheFp16>(p, sms, stream);
    if (type == kCacheE4m3) return wide_one<128, kCacheE4m3>(p, sms, stream);
    return wide_one<128, kCacheInt8>(p, sms, stream);
  }
  if (type == kCacheFp16) return wide_one<64, kCacheFp16>(p, sms, stream);
  if (type == kCacheE4m3) return wide_one<64, kCacheE4m3>(p, sms, stream);
  return wide_one<64, kCacheInt8>(p, sms, stream);
}

cudaError_t read_attend_wait_timeouts(unsigned long long* count, int reset) {
  cudaError_t e = cudaMemcpyFromSymbol(count, g_wait_timeouts, sizeof(*count));
  if (e != cudaSuccess || !reset) return e;
  const unsigned long long zero = 0;
  const unsigned int clear = 0;
  e = cudaMemcpyToSymbol(g_wait_timeouts, &zero, sizeof(zero));
  if (e == cudaSuccess) e = cudaMemcpyToSymbol(g_wait_abort, &clear, sizeof(clear));
  return e;
}

}  // namespace nmk
