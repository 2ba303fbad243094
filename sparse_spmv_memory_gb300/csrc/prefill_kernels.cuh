// prefill_kernels.cuh -- Y = W X for a prefill-sized batch of tokens, W in the N:M
// bitmask format (compact fp16 values + one 32-bit mask word per 32 input
// columns), on the sm_103a tensor cores.
//
// The operation is the pages' SpMM regime (aimodeling.com article, "The
// Kernel Is the Other Half of the Answer", and news.bitwarelabs.com summary,
// "What's new": prefill is compute-bound, decode is bandwidth-bound).  The
// packed format is the same one nm_spmv streams, so a model keeps one copy of
// its weights for both regimes.
//
// Design (this library's own; the pages give no prefill kernel):
//  * A block owns a tile of BM = 128 rows of W and BN = NB * NMMA tokens; its
//    fp32 accumulator D (128 x BN) lives in tensor memory, row m in TMEM lane
//    m.  K advances one mask word (32 columns) per pipeline stage.
//  * Producer warps, each a short chain of asynchronous copies per stage so
//    that they run side by side: warp 0 loads the token tile of X by TMA
//    (BN x 32 fp16, 64-byte swizzle); warp 2 loads the tile's compact values
//    (128 rows x 16 fp16) by TMA; the mask words come by TMA from a warp of
//    their own, four stages per box on a barrier of the box's own, when the
//    mask pitch allows it, else by cp.async from warp 2.  Values and X
//    complete on the stage's "full" mbarrier.
//  * Warps 3..18 (densify), in DG groups that take alternate stages: expand
//    each row's 16 kept values into the 32 columns of a K-major,
//    64-byte-swizzled fp16 tile in shared memory, the layout the MMA
//    descriptor names.  A lane builds four adjacent columns as two pairs:
//    the rank of a pair's first column among the word's set bits (popc)
//    indexes its value in the compact row; one table-driven prmt places it,
//    its neighbour or zeros.
//  * MMA: one thread (warp 1), or two taking the even and odd stages into two
//    accumulators, issues tcgen05.mma kind::f16 (M = 128, N = NMMA, K = 16;
//    two per stage and N-part) on the densified tile and the X tile, and
//    tcgen05.commit frees the stage when those MMAs are done.
//  * Epilogue (warps 3..18): tcgen05.ld of the accumulator, fp32 -> fp16 RNE,
//    stores to Y[t][r]; or, under a K split across blocks (grid z: each block
//    one slice of the row's mask words), fp32 stores of the slice's sums, which
//    splitk_sum_kernel adds in slice order.
//  * The stage barriers are rings sized so that every parity wait is exact
//    (see Layout).  Every mbarrier wait gives up after kWaitLimitNs (counted
//    in g_wait_timeouts); the roles then skip to teardown, which waits for the
//    copies and MMAs already issued before tensor memory is freed.
#pragma once

#include <cuda.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>
#include <stdint.h>
#include <string.h>

#include "device.cuh"
#include "epilogue.cuh"
#include "kernels.h"
#include "tc.cuh"
#include "tmap.h"

namespace nmk {
namespace tc {

constexpr int BM = 128;                // rows of W per block = TMEM lanes
constexpr int BK = 32;                 // K columns per stage = one mask word
constexpr int ROW_BYTES = BK * 2;      // 64-byte rows of the swizzled tiles
constexpr int A_BYTES = BM * ROW_BYTES;  // densified W tile
constexpr int V_BYTES = BM * 32;       // compact values: 16 fp16 per row
constexpr int M_BYTES = BM * 4;        // one mask word per row (cp.async ring)
constexpr int MW = 4;                  // mask words per TMA box (16 bytes per row)
constexpr int MT_SLOT = BM * MW * 4;   // 2 KiB: the masks of MW consecutive stages
// Densify warps per block (DW, a kernel parameter) follow the producer and
// MMA warps.  16 measured best on GB300: 8 left the per-stage chains
// exposed, 24 lost to the extra shared-memory and issue contention.
// After them: a second MMA issuer (used by the two-issuer variants) and the
// producer of the mask boxes.
constexpr int FIRST_DENSIFY_WARP = 3;
__host__ __device__ constexpr int mma2_warp(int dw) { return FIRST_DENSIFY_WARP + dw; }
__host__ __device__ constexpr int mask_warp(int dw) { return FIRST_DENSIFY_WARP + dw + 1; }
__host__ __device__ constexpr int threads_for(int dw) { return (FIRST_DENSIFY_WARP + dw + 2) * 32; }

constexpr uint32_t tmem_cols_for(int n) {
  return n <= 32 ? 32u : n <= 64 ? 64u : n <= 128 ? 128u : n <= 256 ? 256u : 512u;
}

// MT: masks arrive by TMA, MW stages' worth per box, into MT_SLOTS slots
// (needs the row pitch of the mask array, words * 4 bytes, to be a multiple
// of 16); otherwise by 4-byte cp.async into a per-stage ring.  A slot is
// refilled once every densify warp has released it (a barrier per slot);
// MW * MT_SLOTS >= STAGES + MW - 1 boxes in flight keep the box of every
// stage in the pipeline resident while the densify warps reach it.
// MS: 0, one thread issues every stage's MMAs; 1, two threads take the even
// and odd stages into two accumulators that the epilogue adds.
constexpr int gcd_int(int a, int b) { return b ? gcd_int(b, a % b) : a; }

template <int NMMA, int NB, int STAGES, int DG, int MS, bool MT>
struct Layout {
  static constexpr int BN = NMMA * NB;
  static constexpr int B_BYTES = BN * ROW_BYTES;
  static constexpr int A_OFF = 0;
  static constexpr int B_OFF = A_OFF + STAGES * A_BYTES;
  static constexpr int V_OFF = B_OFF + STAGES * B_BYTES;
  static constexpr int M_OFF = V_OFF + STAGES * V_BYTES;
  static constexpr int MT_SLOTS = (STAGES + MW - 1 + MW - 1) / MW;
  static constexpr int M_REGION = MT ? MT_SLOTS * MT_SLOT : STAGES * M_BYTES;
  // Stage barriers.  A parity wait tells a phase from the one before it only,
  // so it is exact only if the waiter itself saw the barrier's previous phase
  // complete.  The "full" barriers therefore form a ring of lcm(STAGES, DG):
  // all phases of one belong to stages of one densify group, which waits for
  // each.  The "afull" barriers form a ring of 2 * STAGES when two MMA
  // issuers split an odd STAGES, so all phases of one belong to one issuer.
  // The "empty" barriers, one per shared-memory slot, are waited by
  // producers that issue every stage.
  static constexpr int FULL_RING = STAGES * DG / gcd_int(STAGES, DG);
  static constexpr int AFULL_RING = (MS && STAGES % 2) ? 2 * STAGES : STAGES;
  // barriers: full (ring), empty (per slot), afull (ring), accum, mfull,
  // mfree (per mask slot)
  static constexpr int BAR_OFF = M_OFF + M_REGION;
  static constexpr int N_BARS = FULL_RING + STAGES + AFULL_RING + 1 + 2 * MT_SLOTS;
  static constexpr int SLOT_OFF = BAR_OFF + N_BARS * 8;
  static constexpr int BYTES = SLOT_OFF + 16;
  static constexpr int SMEM = BYTES + 1024;  // room to align the base to 1024
  static constexpr uint32_t TMEM_COLS = tmem_cols_for(MS ? 2 * BN : BN);
  static_assert(!MS || 2 * BN <= 512, "two issuers keep two accumulators in tensor memory");
  static_assert(!MT || MW * MT_SLOTS >= STAGES + MW - 1, "mask slot reused too early");
  static_assert(NMMA % 16 == 0 && NMMA >= 16 && NMMA <= 256, "tcgen05 M=128 needs N in 16..256");
  static_assert(BN >= 64 && BN <= 512 && BN % 32 == 0, "epilogue reads 32-column chunks");
  static_assert(B_OFF % 1024 == 0 && (NMMA * ROW_BYTES) % 1024 == 0, "swizzled tiles 1024-aligned");
};

// RPW rows x 32 columns of one stage: lane (h, p) of warp wg builds columns
// 4p .. 4p+3 of rows r_i = wg * RPW + 4 i + h (h = lane / 8, p = lane % 8),
// i < RPW / 4, as two column pairs.  For a pair (2j, 2j+1) of the row's word
// the rank c of column 2j among the set bits indexes its value in the compact
// row; the values of rank c and c + 1 are loaded zero-extended and one prmt,
// its selector looked up from a 4-entry table by the pair's two mask bits,
// places them or zeros.  The shared-memory accesses are issued in three
// batches (mask words, values, stores) so that each batch's latency is paid
// once per stage rather than once per row.
// sMw: this stage's mask word of row 0; mstride: bytes from one row's word
// to the next row's.
template <int RPW>
__device__ __forceinline__ void densify_stage(uint32_t sA, uint32_t sV, uint32_t sMw,
                                              uint32_t mstride, int wg, int lane) {
  static_assert(RPW % 8 == 0, "the swizzle phases below need whole groups of 8 rows");
  constexpr int R = RPW / 4;
  const int h = lane >> 3, p = lane & 7;
  const uint32_t b0 = 4u * p;
  const uint32_t below = (1u << b0) - 1u;       // columns of the word left of 4p
  const uint32_t r_first = (uint32_t)(wg * RPW + h);
  // 64-byte swizzle: 16-byte chunk index ^= (row >> 1) & 3.  Row r_i gives
  // (r_i >> 1) & 3 = (2 i + (h >> 1)) & 3 = (2 i & 3) ^ (h >> 1), since
  // wg * RPW / 2 is a multiple of 4: two lane-constant offsets by i & 1.
  const uint32_t lane_chunk = (uint32_t)((p >> 1) ^ (h >> 1));
  const uint32_t in_chunk = (uint32_t)(p & 1) * 8u;
  const uint32_t off_even = (lane_chunk << 4) + in_chunk;           // i even: phase ^ 0
  const uint32_t off_odd = ((lane_chunk ^ 2u) << 4) + in_chunk;     // i odd:  phase ^ 2
  // prmt selectors by q (bit 0: column 2j kept, bit 1: 2j+1 kept) for the
  // values v (rank c) and w (rank c + 1): q 0 -> 0x3232 (0, 0),
  // 1 -> 0x3210 (v, 0), 2 -> 0x1032 (0, v), 3 -> 0x5410 (v, w).
  constexpr uint32_t kSelLo = 0x32103232u, kSelHi = 0x54101032u;
  uint32_t m[R], nib[R], v[R][4];
#pragma unroll
  for (int i = 0; i < R; ++i) m[i] = lds_u32(sMw + mstride * (r_first + 4 * i));
#pragma unroll
  for (int i = 0; i < R; ++i) {
    const uint32_t r = r_first + 4 * i;
    const uint32_t c = __popc(m[i] & below);            // rank of column 4p
    nib[i] = (m[i] >> b0) & 15u;
    const uint32_t c2 = c + __popc(nib[i] & 3u);         // rank of column 4p + 2
    const uint32_t a0 = sV + 32u * r + 2u * c, a2 = sV + 32u * r + 2u * c2;
    v[i][0] = lds_u16_32(a0);
    v[i][1] = lds_u16_32(a0 + 2u);
    v[i][2] = lds_u16_32(a2);
    v[i][3] = lds_u16_32(a2 + 2u);
  }
#pragma unroll
  for (int i = 0; i < R; ++i) {
    const uint32_t r = r_first + 4 * i;
    const uint32_t lo = prmt(v[i][0], v[i][1], prmt(kSelLo, kSelHi, (nib[i] & 3u) * 0x22u + 0x10u));
    const uint32_t hi = prmt(v[i][2], v[i][3], prmt(kSelLo, kSelHi, (nib[i] >> 2) * 0x22u + 0x10u));
    sts_u64(sA + r * ROW_BYTES + ((i & 1) ? off_odd : off_even), lo, hi);
  }
}

// All threads of the cluster; those that have left count as there.
__device__ __forceinline__ void cluster_sync() {
  __syncwarp();
  asm volatile("barrier.cluster.arrive.release.aligned;" ::: "memory");
  asm volatile("barrier.cluster.wait.acquire.aligned;" ::: "memory");
}

// A shared-memory address of this block in block `rank` of the cluster.
__device__ __forceinline__ uint32_t remote_smem(uint32_t at, uint32_t rank) {
  uint32_t r;
  asm("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(r) : "r"(at), "r"(rank));
  return r;
}

// n <= N outputs of a lane, ldy apart: residual + scale * x.
template <int N>
__device__ __forceinline__ void store_outputs(const Epilogue& e, const float (&x)[N], int n, int64_t t0, int64_t o,
                                              __half* Y, int64_t ldy) {
  __half* y = Y + t0 * ldy + o;
  if (e.residual) {
    const __half* res = e.residual + t0 * e.ldres + o;
#pragma unroll
    for (int i0 = 0; i0 < N; i0 += 16) {
      __half h[16];  // on their way at a time
#pragma unroll
      for (int i = 0; i < 16; ++i)
        if (i0 + i < n) {
          h[i] = *res;
          res += e.ldres;
        }
#pragma unroll
      for (int i = 0; i < 16; ++i)
        if (i0 + i < n) {
          *y = __float2half_rn(fmaf(e.scale, x[i0 + i], __half2float(h[i])));
          y += ldy;
        }
    }
  } else {
#pragma unroll
    for (int i = 0; i < N; ++i)
      if (i < n) {
        *y = __float2half_rn(e.scale * x[i]);
        y += ldy;
      }
  }
}

// The epilogue of nm_linear for n <= 32 tokens (from t0) of the row held by each lane
// of a warp.  Gated: lanes 2i and 2i + 1 hold a gate row and its up row; they trade
// halves, so that the even lane finishes the first 16 tokens and the odd lane the last
// 16, each token's outputs of a warp lying side by side.
__device__ __forceinline__ void linear_store_32(const Epilogue& e, const uint32_t (&v)[32], bool row_ok,
                                                int64_t r, int64_t t0, int n, __half* Y,
                                                int64_t ldy, int lane) {
  const float b = row_ok ? bias_at(e, r) : 0.f;
  if (e.gated) {
    const bool odd = lane & 1;
    float g[16], u[16];
#pragma unroll
    for (int i = 0; i < 16; ++i) {
      const float lo = __uint_as_float(v[i]) + b, hi = __uint_as_float(v[16 + i]) + b;
      const float other = __shfl_xor_sync(0xFFFFFFFFu, odd ? lo : hi, 1);
      g[i] = odd ? other : lo;
      u[i] = odd ? hi : other;
    }
    activate_fast(g, e.act);
#pragma unroll
    for (int i = 0; i < 16; ++i) g[i] *= u[i];
    store_outputs<16>(e, g, row_ok ? n - (odd ? 16 : 0) : 0, t0 + (odd ? 16 : 0), r >> 1, Y, ldy);
  } else {
    float x[32];
#pragma unroll
    for (int i = 0; i < 32; ++i) x[i] = __uint_as_float(v[i]) + b;
    activate_fast(x, e.act);
    store_outputs<32>(e, x, row_ok ? n : 0, t0, r, Y, ldy);
  }
}

// DG: the densify warps form DG groups; group g expands stages g, g + DG,
// ... with 128 / (16 / DG) rows per warp.  Each stage costs a warp a fixed
// chain of barrier waits, fences and arrivals (hundreds of cycles of
// latency) besides its rows, so with DG groups that chain overlaps DG stages.
template <int NMMA, int NB, int STAGES, int G, int DG, int DW, int MS, bool MT, bool EPI>
__global__ void __launch_bounds__(threads_for(DW), 1)
    spmm_tc_kernel(const __grid_constant__ CUtensorMap tm_v, const __grid_constant__ CUtensorMap tm_x,
                   const __grid_constant__ CUtensorMap tm_m, const uint32_t* __restrict__ masks,
                   __half* __restrict__ Y, float* __restrict__ part, int64_t rows, int words,
                   int wslice, int64_t T, int64_t ldy, uint64_t wait_limit_ns, int stall_weights,
                   const Epilogue epi, int tile) {
  using L = Layout<NMMA, NB, STAGES, DG, MS, MT>;
  static_assert(DG == 1 || G == 1, "waiting on every second stage needs one densify group");
  // G = 2 waits on the odd stages' afull barriers only; with an even ring each
  // of those barriers serves odd stages alone, so every parity wait stays exact.
  static_assert(G == 1 || L::AFULL_RING % 2 == 0, "waiting on every second stage needs an even ring");
  static_assert(MS == 0 || G == 1, "each of two issuers waits on each of its stages");
  static_assert(DW % DG == 0 && DW % 4 == 0, "equal densify groups, whole TMEM quadrants");
  static_assert(threads_for(DW) <= 1024, "a block has at most 1024 threads");
  static_assert(DG <= MW, "every densify group must read every mask box, in order");
  constexpr int WPG = DW / DG;             // warps per densify group
  constexpr int RPW = BM / WPG;            // rows per warp and stage
  extern __shared__ uint8_t smem_raw[];
  const uint32_t raw = smem_addr(smem_raw);
  const uint32_t base = (raw + 1023u) & ~1023u;
  const uint32_t sA = base + L::A_OFF, sB = base + L::B_OFF, sV = base + L::V_OFF,
                 sM = base + L::M_OFF, bars = base + L::BAR_OFF, slot = base + L::SLOT_OFF;
  constexpr int FB = L::FULL_RING, AB = L::AFULL_RING;
  // full / afull: by stage kt (rings of FB / AB); empty: by slot kt % STAGES.
  auto full = [&](int kt) { return bars + 8u * (kt % FB); };
  auto full_par = [&](int kt) { return (uint32_t)((kt / FB) & 1); };
  auto empty = [&](int s) { return bars + 8u * (FB + s); };
  auto afull = [&](int kt) { return bars + 8u * (FB + STAGES + kt % AB); };
  auto afull_par = [&](int kt) { return (uint32_t)((kt / AB) & 1); };
  const uint32_t accum = bars + 8u * (FB + STAGES + AB);
  // A mask box serves MW consecutive stages that may belong to different
  // densify groups, so it completes on a barrier of its own.
  auto mfull = [&](int slot) { return bars + 8u * (FB + STAGES + AB + 1 + slot); };
  // ... and is released on one when every densify warp has finished its last
  // stage in the box (the stages of a box may go to different MMA issuers, so
  // no single stage's completion implies that).
  auto mfree = [&](int slot) {
    return bars + 8u * (FB + STAGES + AB + 1 + L::MT_SLOTS + slot);
  };

  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  if (EPI) pdl_launch_dependents();
  // After a wait gave up (this launch or an earlier one not yet reset), the
  // block does nothing: the decision is block-uniform, taken before any
  // barrier, copy or tensor-memory allocation.
  // (A cluster's blocks write each other's shared memory, so none of them leaves before
  // the others: their waits give up at once instead.)
  if (!(EPI && gridDim.z > 1) && __syncthreads_or(threadIdx.x == 0 && wait_aborted())) return;
  const int64_t r0 = (int64_t)blockIdx.y * BM;
  // Tokens of one MMA: NMMA, or (EPI) what the launcher chose.
  const int nmma = EPI ? tile : NMMA;
  const int64_t n0 = (int64_t)blockIdx.x * (EPI ? NB * nmma : L::BN);
  // K split: this block multiplies the mask words w0 .. w0 + nk - 1 (stage
  // kt is word w0 + kt); w0 is a multiple of MW, so mask boxes stay aligned.
  const int w0 = (int)blockIdx.z * wslice;
  const int nk = min(words - w0, wslice);

  if (warp == 0 && lane == 0) {
    for (int k = 0; k < FB; ++k)
      mbar_init(full(k), MT ? 2 : 2 + 32);    // two expect_tx arrivals (+ 32 cp.async arrivals)
    for (int s = 0; s < STAGES; ++s) mbar_init(empty(s), 1);  // tcgen05.commit
    for (int k = 0; k < AB; ++k) mbar_init(afull(k), WPG);    // one arrival per warp of the group
    mbar_init(accum, MS ? 2 : 1);             // final commit of each issuer
    for (int m = 0; m < L::MT_SLOTS; ++m) {
      mbar_init(mfull(m), 1);
      mbar_init(mfree(m), DW);
    }
    fence_mbar_init();
    prefetch_tmap(&tm_v);
    prefetch_tmap(&tm_x);
    if (MT) prefetch_tmap(&tm_m);
  }
  if (warp == 1) {
    tmem_alloc(slot, L::TMEM_COLS);
    tmem_relinquish();
  }
  tc_fence_before_sync();
  __syncthreads();
  tc_fence_after_sync();
  uint32_t tmem_base;
  asm volatile("ld.shared.u32 %0, [%1];" : "=r"(tmem_base) : "r"(slot) : "memory");

  if (EPI) pdl_wait_previous();  // (everything above touches no argument's memory)

  // Teardown must not free shared memory under copies still in flight: a
  // producer waits (bounded) for the stages it issued among the last STAGES
  // of the row -- the final use of each slot, so the phase it waits for is
  // the slot's last.  A producer that stopped early on a timeout issued
  // nothing in the last 2 s worth waiting for.
  auto drain = [&](int last) {
    for (int kt = last; kt >= 0 && kt > nk - 1 - STAGES; --kt)
      mbar_wait(full(kt), full_par(kt), wait_limit_ns, false);
  };

  bool fine = false;  // (densify warps) the accumulator is whole
  if (warp == 0) {
    // ---- X producer: the token tile of each stage -------------------------
    if (lane == 0) {
      int last = -1;
      for (int kt = 0; kt < nk; ++kt) {
        const int s = kt % STAGES, u = kt / STAGES;
        if (u > 0 && !mbar_wait(empty(s), (u - 1) & 1, wait_limit_ns)) break;
        mbar_arrive_expect_tx(full(kt), EPI ? NB * nmma * ROW_BYTES : L::B_BYTES);
#pragma unroll
        for (int j = 0; j < NB; ++j)
          tma_load_2d(sB + s * L::B_BYTES + j * NMMA * ROW_BYTES, &tm_x, (w0 + kt) * BK,
                      (int)(n0 + j * nmma), full(kt));
        last = kt;
      }
      drain(last);
    }
    __syncwarp();
  } else if (warp == 2) {
    // ---- W producer: compact values (and, without MT, mask words) ----------
    // With MT one lane issues the values' TMA (the mask boxes have a warp of
    // their own); without, all lanes also gather the mask words by cp.async,
    // each arriving on the stage barrier when its copies land.
    // stall_weights (self-test only) issues nothing: every consumer's bounded
    // wait then runs out and the block tears down without storing Y.
    if ((!MT || lane == 0) && !stall_weights) {
      int last = -1;
      for (int kt = 0; kt < nk; ++kt) {
        const int s = kt % STAGES, u = kt / STAGES;
        int ok = 1;
        if (u > 0 && lane == 0) ok = mbar_wait(empty(s), (u - 1) & 1, wait_limit_ns);
        if (!MT) ok = __shfl_sync(0xFFFFFFFFu, ok, 0);
        if (!ok) break;
        if (lane == 0) {
          mbar_arrive_expect_tx(full(kt), V_BYTES);
          tma_load_2d(sV + s * V_BYTES, &tm_v, (w0 + kt) * 16, (int)r0, full(kt));
        }
        if (!MT) {
#pragma unroll
          for (int i = 0; i < BM / 32; ++i) {
            const int rr = lane + 32 * i;
            const int64_t gr = r0 + rr;
            const bool in = gr < rows;
            cp_async_4(sM + s * M_BYTES + 4u * rr, masks + (in ? gr : 0) * words + w0 + kt,
                       in ? 4u : 0u);
          }
          cp_async_arrive_noinc(full(kt));
        }
        last = kt;
      }
      if (!MT) cp_async_wait_all();
      if (lane == 0) drain(last);
    }
    __syncwarp();
  } else if (warp == mask_warp(DW)) {
    // ---- mask producer (MT): one box of MW stages' mask words at a time -----
    // A slot is refilled only after every densify warp released it from the
    // slot's previous box.  This warp alone refills, in box order, so the
    // release waited for is always the previous box's.
    if (MT && lane == 0 && !stall_weights) {
      int nbox = 0;
      for (int kt = 0; kt < nk; kt += MW) {
        const int b = kt / MW, ms = b % L::MT_SLOTS;
        if (b >= L::MT_SLOTS &&
            !mbar_wait(mfree(ms), ((b / L::MT_SLOTS) - 1) & 1, wait_limit_ns))
          break;
        mbar_arrive_expect_tx(mfull(ms), MT_SLOT);
        tma_load_2d(sM + ms * MT_SLOT, &tm_m, w0 + kt, (int)r0, mfull(ms));
        nbox = kt / MW + 1;
      }
      const int b0 = nbox > L::MT_SLOTS ? nbox - L::MT_SLOTS : 0;  // boxes still in flight
      for (int b = b0; b < nbox; ++b)
        mbar_wait(mfull(b % L::MT_SLOTS), (b / L::MT_SLOTS) & 1, wait_limit_ns);
    }
    __syncwarp();
  } else if (warp == 1 || warp == mma2_warp(DW)) {
    // ---- MMA issuers ----------------------------------------------------
    // Each waits only on the densify barriers: the densify warps saw the
    // stage's "full" barrier complete (so the TMA-loaded X tile is visible
    // through their release-arrive).  With one densify group (DG == 1) every
    // warp arrives on the stages in order, so G = 2 may wait on every second
    // barrier only (afull(kt + 1) complete implies afull(kt)).  A barrier test,
    // a commit and each tcgen05.mma cost the issuing thread tens to hundreds
    // of cycles, so with MS == 1 two threads share the stages (even / odd,
    // into two accumulators).
    const int role = warp == 1 ? 0 : 1;
    if (lane == 0 && (role == 0 || MS != 0)) {
      const uint32_t idesc = EPI ? idesc_f16_f32(BM, nmma) : idesc_f16_f32(BM, NMMA);
      const int k0 = MS ? role : 0, kstep = MS ? 2 : G;
      const uint32_t dacc = tmem_base + (uint32_t)(MS && role ? L::BN : 0);
      for (int kt = k0; kt < nk; kt += kstep) {
        const int last = MS ? kt : (kt + G - 1 < nk ? kt + G - 1 : nk - 1);
        if (!mbar_wait(afull(last), afull_par(last), wait_limit_ns)) break;
        tc_fence_after_sync();
        for (int k = kt; k <= last; ++k) {
          const int s = k % STAGES;
#pragma unroll
          for (int ks = 0; ks < BK / 16; ++ks) {
            const uint64_t ad = smem_desc_sw64(sA + s * A_BYTES + ks * 32);
#pragma unroll
            for (int j = 0; j < NB; ++j) {
              const uint64_t bd =
                  smem_desc_sw64(sB + s * L::B_BYTES + j * NMMA * ROW_BYTES + ks * 32);
              mma_f16(dacc + (uint32_t)(j * NMMA), ad, bd, idesc, (k != k0) || (ks != 0));
            }
          }
          // Only a slot that a producer refills gets its release: no one
          // waits for the last STAGES stages', and a commit's arrival is not
          // ordered with the accum commit's, so it could land after this
          // block ended, in the barriers of the next block on the SM.
          if (k + STAGES < nk) mma_commit(empty(s));
        }
      }
      mma_commit(accum);  // also after an early exit: completes once issued MMAs finish
    }
    __syncwarp();
  } else {
    // ---- densify, then epilogue -----------------------------------------
    const int dw = warp - FIRST_DENSIFY_WARP;
    const int grp = dw / WPG, wg = dw % WPG;
    bool ok = true;
    int box = -1;  // mask box this warp last waited for
    for (int kt = grp; kt < nk; kt += DG) {
      const int s = kt % STAGES;
      bool got = mbar_wait(full(kt), full_par(kt), wait_limit_ns);
      if (MT && kt / MW != box) {
        // The box's slot is refilled only after every densify warp released
        // it, so the phase this warp sees here is this box's.
        box = kt / MW;
        got = got && mbar_wait(mfull(box % L::MT_SLOTS), (box / L::MT_SLOTS) & 1, wait_limit_ns);
      }
      // The warp decides together, so no lane is left behind at a warp barrier.
      if (!__all_sync(0xFFFFFFFFu, got)) { ok = false; break; }
      const uint32_t sMw = MT ? sM + ((kt / MW) % L::MT_SLOTS) * MT_SLOT + (kt % MW) * 4u
                              : sM + s * M_BYTES;
      densify_stage<RPW>(sA + s * A_BYTES, sV + s * V_BYTES, sMw, MT ? MW * 4u : 4u, wg, lane);
      // Each lane orders its tile writes before the tensor core's reads; the
      // warp barrier then lets one release-arrive publish all 32 lanes' writes
      // (one arrival per warp: 32 arrivals on one barrier word serialise).
      fence_proxy_async_smem();
      __syncwarp();
      if (lane == 0) {
        mbar_arrive(afull(kt));
        // This warp's last stage in the mask box: it has read the box (its
        // loads precede the release-arrive), so the slot may be refilled.
        if (MT && kt + DG >= MW * (kt / MW + 1)) mbar_arrive(mfree((kt / MW) % L::MT_SLOTS));
      }
    }
    if (!mbar_wait(accum, 0, wait_limit_ns)) ok = false;
    tc_fence_after_sync();
    // tcgen05.ld is a warp-wide instruction: the whole warp reads or none does.
    fine = __all_sync(0xFFFFFFFFu, ok);
    if (!EPI && fine) {
      const int quad = warp & 3;              // TMEM lanes 32*quad .. +31
      const int qi = dw >> 2;                 // this warp's index among its quadrant's warps
      constexpr int QW = DW / 4;              // warps per quadrant, striding the columns
      const int64_t r = r0 + 32 * quad + lane;
      const bool row_ok = r < rows;
      const uint32_t tbase = tmem_base + ((uint32_t)(32 * quad) << 16);
#pragma unroll 1
      for (int c0 = qi * 32; c0 < L::BN; c0 += QW * 32) {
        uint32_t v[32];
        tmem_ld_32(tbase + (uint32_t)c0, v);
        tmem_ld_wait();
        if (MS && nk > 1) {  // the odd stages' accumulator (none when nk == 1)
          uint32_t w[32];
          tmem_ld_32(tbase + (uint32_t)(L::BN + c0), w);
          tmem_ld_wait();
#pragma unroll
          for (int i = 0; i < 32; ++i)
            v[i] = __float_as_uint(__uint_as_float(v[i]) + __uint_as_float(w[i]));
        }
        if (row_ok && part) {  // K split: this slice's fp32 sums, [slice][T][rows]
          float* pz = part + (int64_t)blockIdx.z * T * rows + r;
#pragma unroll
          for (int i = 0; i < 32; ++i) {
            const int64_t t = n0 + c0 + i;
            if (t < T) pz[t * rows] = __uint_as_float(v[i]);
          }
        } else if (row_ok) {
#pragma unroll
          for (int i = 0; i < 32; ++i) {
            const int64_t t = n0 + c0 + i;
            if (t < T) Y[t * ldy + r] = __float2half_rn(__uint_as_float(v[i]));
          }
        }
      }
    }
  }

  if constexpr (EPI) {
    // ---- nm_linear's epilogue -------------------------------------------------
    // The accumulator's columns in pieces of 32 (an MMA's tokens may end inside one).
    // Under a K split the blocks of a row tile's slices are a cluster: piece i is
    // finished by block i % slices, to which the others send theirs through
    // distributed shared memory (their rings lie idle by now), and which adds them in
    // slice order: nothing goes through memory, and no second launch.
    const int slices = (int)gridDim.z, me = (int)blockIdx.z;
    const int per = (nmma + 31) / 32, pieces = NB * per;
    const int dw = warp - FIRST_DENSIFY_WARP, quad = warp & 3, qi = dw >> 2;
    const bool mine = warp >= FIRST_DENSIFY_WARP && warp < FIRST_DENSIFY_WARP + DW && fine;
    constexpr int QW = DW / 4;
    const int64_t r = r0 + 32 * quad + lane;
    const uint32_t tbase = tmem_base + ((uint32_t)(32 * quad) << 16);
    auto column = [&](int i) { return i / per * NMMA + i % per * 32; };
    auto sums = [&](int i, uint32_t (&v)[32]) {
      tmem_ld_32(tbase + (uint32_t)column(i), v);
      tmem_ld_wait();
      if (MS && nk > 1) {  // the odd stages' accumulator (none when nk == 1)
        uint32_t w[32];
        tmem_ld_32(tbase + (uint32_t)(L::BN + column(i)), w);
        tmem_ld_wait();
#pragma unroll
        for (int k = 0; k < 32; ++k) v[k] = __float_as_uint(__uint_as_float(v[k]) + __uint_as_float(w[k]));
      }
    };
    // its first token, and how many it has
    auto first = [&](int i) { return n0 + i / per * nmma + i % per * 32; };
    auto count = [&](int i) { return (int)min((int64_t)min(nmma - i % per * 32, 32), T - first(i)); };
    // Where block `from`'s piece i lies in the shared memory of the block that finishes it:
    // [place among the others][its pieces][32 tokens][128 rows] fp32.
    const int share = (pieces + slices - 1) / slices;
    auto inbox = [&](int i, int from) {
      const int to = i % slices, at = (from < to ? from : from - 1) * share + i / slices;
      return base + (uint32_t)(at * (32 * BM * 4) + (32 * quad + lane) * 4);
    };
    if (slices > 1) {
      cluster_sync();  // every block is done with its ring
      if (mine) {
#pragma unroll 1
        for (int i = qi; i < pieces; i += QW) {
          if (i % slices == me || count(i) <= 0) continue;
          uint32_t v[32];
          sums(i, v);
          const uint32_t to = remote_smem(inbox(i, me), (uint32_t)(i % slices));
#pragma unroll
          for (int k = 0; k < 32; ++k)
            asm volatile("st.shared::cluster.u32 [%0], %1;" ::"r"(to + k * (BM * 4)), "r"(v[k]) : "memory");
        }
      }
      cluster_sync();
    }
    if (mine) {
#pragma unroll 1
      for (int i = me + qi * slices; i < pieces; i += QW * slices) {
        const int n = count(i);
        if (n <= 0) continue;
        uint32_t v[32];
        sums(i, v);
        if (slices > 1) {
          float acc[32];
#pragma unroll
          for (int k = 0; k < 32; ++k) acc[k] = 0.f;
          for (int z = 0; z < slices; ++z) {
            if (z == me) {
#pragma unroll
              for (int k = 0; k < 32; ++k) acc[k] += __uint_as_float(v[k]);
            } else {
              const uint32_t from = inbox(i, z);
#pragma unroll
              for (int k = 0; k < 32; ++k) acc[k] += lds_f32(from + k * (BM * 4));
            }
          }
#pragma unroll
          for (int k = 0; k < 32; ++k) v[k] = __float_as_uint(acc[k]);
        }
        linear_store_32(epi, v, r < rows, r, first(i), n, Y, ldy, lane);
      }
    }
  }

  tc_fence_before_sync();
  __syncthreads();
  if (warp == 1) {
    // Tensor memory is freed only after the MMAs that write it have completed:
    // one more bounded (not abortable) wait on the final commit, which a
    // normal run passed already.  An MMA issuer that stopped early committed
    // what it issued, so the barrier still completes.
    mbar_wait(accum, 0, wait_limit_ns, false);
    tc_fence_after_sync();
    tmem_dealloc(tmem_base, L::TMEM_COLS);
  }
}

// ---- host ------------------------------------------------------------------
static bool encode_2d(CUtensorMap* m, const void* ptr, uint64_t inner, uint64_t outer,
                      uint64_t stride_bytes, uint32_t box_inner, uint32_t box_outer,
                      CUtensorMapSwizzle swz,
                      CUtensorMapDataType dtype = CU_TENSOR_MAP_DATA_TYPE_FLOAT16) {
  const cuuint64_t dims[2] = {inner, outer};
  const cuuint64_t strides[1] = {stride_bytes};
  const cuuint32_t box[2] = {box_inner, box_outer};
  return encode_tiled(m, dtype, ptr, 2, dims, strides, box, swz);
}

template <int NMMA, int NB, int STAGES, int G, int DG, int DW, int MS, bool MT, bool EPI>
static cudaError_t launch_tc_mt(const SpmmTcParams& p, cudaStream_t stream) {
  using L = Layout<NMMA, NB, STAGES, DG, MS, MT>;
  CUtensorMap tm_v, tm_x, tm_m;
  memset(&tm_m, 0, sizeof(tm_m));
  const int tile = EPI ? p.tile : NMMA;  // tokens of an MMA
  if (MT && !encode_2d(&tm_m, p.masks, (uint64_t)p.words, (uint64_t)p.rows,
                       (uint64_t)p.words * 4, MW, BM, CU_TENSOR_MAP_SWIZZLE_NONE,
                       CU_TENSOR_MAP_DATA_TYPE_UINT32))
    return cudaErrorInvalidValue;
  if (!encode_2d(&tm_v, p.values, (uint64_t)p.words * 16, (uint64_t)p.rows,
                 (uint64_t)p.words * 32, 16, BM, CU_TENSOR_MAP_SWIZZLE_NONE) ||
      !encode_2d(&tm_x, p.X, (uint64_t)p.words * 32, (uint64_t)p.T, (uint64_t)p.ldx * 2, BK,
                 tile, CU_TENSOR_MAP_SWIZZLE_64B))
    return cudaErrorInvalidValue;
  if (EPI && p.slices > 1) {  // what a block is sent fits its ring
    const int pieces = NB * ((tile + 31) / 32), share = (pieces + p.slices - 1) / p.slices;
    if ((p.slices - 1) * share * 32 * BM * 4 > L::M_OFF) return cudaErrorInvalidValue;
  }
  auto* k = spmm_tc_kernel<NMMA, NB, STAGES, G, DG, DW, MS, MT, EPI>;
  static int attr_done[64] = {0};
  int dev = 0;
  cudaGetDevice(&dev);
  if (dev >= 0 && dev < 64 && !attr_done[dev]) {
    cudaError_t e = cudaFuncSetAttribute(k, cudaFuncAttributeMaxDynamicSharedMemorySize, L::SMEM);
    if (e != cudaSuccess) return e;
    attr_done[dev] = 1;
  }
  const int wslice = p.slices > 1 ? p.wslice : p.words;
  const dim3 grid((unsigned)((p.T + NB * tile - 1) / (NB * tile)), (unsigned)((p.rows + BM - 1) / BM),
                  (unsigned)(p.slices > 1 ? p.slices : 1));
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = grid;
  cfg.blockDim = dim3(threads_for(DW));
  cfg.dynamicSmemBytes = L::SMEM;
  cfg.stream = stream;
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  attr[1].id = cudaLaunchAttributeClusterDimension;
  attr[1].val.clusterDim.x = attr[1].val.clusterDim.y = 1;
  attr[1].val.clusterDim.z = grid.z;
  cfg.attrs = attr;
  cfg.numAttrs = EPI ? (grid.z > 1 ? 2 : 1) : 0;
  const uint64_t limit = p.wait_limit_ns ? p.wait_limit_ns : kWaitLimitNs;
  float* part = p.slices > 1 ? p.part : nullptr;
  return cudaLaunchKernelEx(&cfg, k, tm_v, tm_x, tm_m, p.masks, p.Y, part, p.rows, p.words,
                            wslice, p.T, p.ldy, limit, p.stall_weights, p.epi, tile);
}

// Mask words by TMA when the mask array allows it (16-byte aligned, row pitch
// words * 4 a multiple of 16: every decoder shape), else by cp.async.
template <int NMMA, int NB, int STAGES, int G, int DG, int DW, int MS, bool EPI>
static cudaError_t launch_tc(const SpmmTcParams& p, cudaStream_t stream) {
  const bool mt = p.words % 4 == 0 && (reinterpret_cast<uintptr_t>(p.masks) & 15) == 0;
  return mt ? launch_tc_mt<NMMA, NB, STAGES, G, DG, DW, MS, true, EPI>(p, stream)
            : launch_tc_mt<NMMA, NB, STAGES, G, DG, DW, MS, false, EPI>(p, stream);
}

}  // namespace tc
}  // namespace nmk
