// linear_tc.cu -- nm_linear for more than 8 tokens: Y = residual + scale * act(W X + bias)
// on the sm_103a tensor cores, W in the N:M bitmask format.
//
// As in prefill.cu a block owns 128 rows of W (the MMA's M, TMEM lanes) and a tile of
// tokens (its N), K advances by one mask word a stage, producers load a stage's compact
// values, mask words and token tile by TMA, densify warps expand the weights to a
// swizzled fp16 tile, one or two threads issue the MMAs, and the accumulator stays in
// tensor memory.  What is this kernel's own:
//  * The rings are apart.  A stage's compact values are free again once they are
//    expanded, its expanded tile and its token tile once its MMAs are done, and the token
//    tile is the largest by far (32 KB of 512 tokens; an expanded tile has 8 KB, compact
//    values 4).  One ring of all three has as many stages as token tiles fit, 5 at 512
//    tokens, and a stage then takes a fifth of the way from an empty slot through the
//    loads, the expansion and the MMAs: 441 ns at 512 tokens, and still 375 at 32, with the
//    tensor pipe 53 % busy.  With twelve stages of values, which come from HBM, and the
//    others' rings as long as fits it is 355 and 322.
//  * Few instructions of the threads that feed the rest.  A copy costs its thread 200
//    cycles and more, a wait 100, an MMA 45 and a commit 55, beside densify warps that keep
//    the schedulers half busy.  So values and masks come four stages at a time, two warps
//    load token tiles, and tokens and weights of a stage share a barrier; with the cheaper
//    expansion of expand_32 320 tokens take 285 ns a stage for 330, 128 take 211 for 262.
//  * An MMA has as many tokens as there are (a multiple of 16), not a full tile's.
//  * A K split's blocks are a cluster and trade their sums through distributed shared
//    memory (see the epilogue): no workspace, no second launch.
//  * The epilogue, and launches that overlap the previous kernel's end.
// Every mbarrier wait is bounded as prefill.cu's are (the same limits and counters).
#include <cuda.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>
#include <stdint.h>
#include <string.h>

#include <type_traits>

#include "device.cuh"
#include "epilogue.cuh"
#include "kernels.h"
#include "tc.cuh"
#include "tc_tiles.cuh"

namespace nmk {
namespace tc {
namespace {

constexpr int DW = 16;  // densify warps
__host__ __device__ constexpr int tokens2_warp(int dw) { return mask_warp(dw); }  // the second producer of token tiles
constexpr int lcm_int(int a, int b) { return a / gcd_int(a, b) * b; }

// NMMA: tokens of an MMA at most; NB MMAs a block and K step; S: slots of expanded weights
// and token tiles, a stage each; SV: slots of compact values and mask words, MW stages (a
// box) each; DG densify groups, which take the stages in turn.  Two threads issue
// MMAs: MS 1, the even and the odd stages into two accumulators; MS 2, the two MMAs of
// every K step.  MT: masks come by TMA (the mask array is 16-byte aligned with rows of
// whole boxes), else by cp.async.
//
// Barriers.  A parity wait tells a phase from the one before it only, so it is exact
// only if the waiter saw the barrier's phase before, or the barrier cannot have gone a
// phase further.  fullv, vfree (a box there, and used up): every densify warp has a stage
// in every box.  ready (tokens there and weights expanded; one barrier for one wait of the
// issuers): a ring of an even number of slots, which the producers and issuers of even and
// odd stages share out.  done (MMAs complete), by stage: a token producer waits for all of
// its stages in order; the densify warps of stage kt wait for stage kt - S, and RD being a
// multiple of 2 S, the stage that would complete the same barrier's next phase needs the
// slot that they are about to fill.
template <int NMMA, int NB, int S, int SV, int DG, int MS, bool MT>
struct Shape {
  static constexpr int BN = NMMA * NB;
  static constexpr int B_BYTES = BN * ROW_BYTES;
  static constexpr int V_SLOT = BM * MW * 32;  // rows of 128 bytes, swizzled
  static constexpr int A_OFF = 0;
  static constexpr int B_OFF = A_OFF + S * A_BYTES;
  static constexpr int V_OFF = B_OFF + S * B_BYTES;
  static constexpr int M_OFF = V_OFF + SV * V_SLOT;
  static constexpr int BAR_OFF = M_OFF + SV * MT_SLOT;
  static constexpr int RD = lcm_int(2 * S, DG);
  static constexpr int N_BARS = 2 * SV + S + RD + 1;  // fullv, vfree, ready, done, accum
  static constexpr int SLOT_OFF = BAR_OFF + N_BARS * 8;
  static constexpr int SMEM = SLOT_OFF + 16 + 1024;  // room to align the base to 1024
  static constexpr uint32_t TMEM_COLS = tmem_cols_for(MS == 1 ? 2 * BN : BN);
  static_assert(S % 2 == 0, "even and odd stages have slots of their own");
  static_assert(MS == 1 ? NB == 1 && 2 * BN <= 512 : NB == 2, "what two issuers share");
  static_assert(NMMA % 16 == 0 && NMMA >= 16 && NMMA <= 256, "tcgen05 M=128 needs N in 16..256");
  static_assert(BN <= 512 && B_OFF % 1024 == 0 && (NMMA * ROW_BYTES) % 1024 == 0 && V_OFF % 1024 == 0,
                "swizzled tiles 1024-aligned");
  static_assert(SMEM <= 232448, "a block's shared memory");
  static_assert(DW % DG == 0 && DG <= MW, "every densify group has a stage in every box");
};

// Expands 32 rows of a stage, which is word j of its box: sV rows of 128 bytes, their
// 16-byte chunks at place ^ (row & 7), sM rows of MW mask words, to the stage's swizzled
// tile at sA (chunk ^= (row >> 1) & 3).
//
// Where every byte of the mask words keeps 4 columns (1:2, 2:4, 4:8), which the warp sees
// for itself (bytes: so far), a byte's values are 8 aligned bytes of the compact row, and a
// lane takes a byte, four lanes a row: the nibble's bits spread to the bytes of a word, bit
// i the byte i, times 0x01010100 are the ranks of its columns in it (byte i: how many kept
// ones lie below), times 0x22 plus 0x10 the prmt selector of that value's two bytes; columns
// that are not kept become 0 by a mask.  Else a lane takes a nibble, as two column pairs:
// the rank of a pair's first column, a popcount, finds its values, which one prmt by the
// pair's mask bits places.  That is twice the instructions: 270 ns a stage for 212 at 128
// tokens, 300 for 285 at 320.
__device__ __forceinline__ void expand_32(uint32_t sA, uint32_t sV, uint32_t sM, int j, int row0, int lane,
                                          bool& bytes) {
  if (bytes) {
    const uint32_t m = lds_u32(sM + (uint32_t)(row0 + lane) * (MW * 4u) + 4u * j);
    uint32_t c = m - ((m >> 1) & 0x55555555u);
    c = (c & 0x33333333u) + ((c >> 2) & 0x33333333u);
    c = (c + (c >> 4)) & 0x0F0F0F0Fu;
    bytes = __all_sync(0xFFFFFFFFu, c == 0x04040404u || m == 0u);  // (0: rows behind the last)
  }
  if (bytes) {
    const uint32_t h = lane >> 2, p = lane & 3, r = (uint32_t)row0 + h;  // rows r + 8 i: r & 7 = h
    const uint32_t from = sV + 128u * r + (((2u * j + (p >> 1)) ^ h) << 4) + 8u * (p & 1);
    const uint32_t byte = sM + r * (MW * 4u) + 4u * j + p, to = sA + r * ROW_BYTES + ((p ^ (h >> 1)) << 4);
    uint32_t b[4], v01[4], v23[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      b[i] = lds_u8_32(byte + 8u * MW * 4u * i);
      lds_u64(from + 8u * 128u * i, v01[i], v23[i]);
    }
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const uint32_t lo = ((b[i] & 15u) * 0x00204081u) & 0x01010101u, hi = ((b[i] >> 4) * 0x00204081u) & 0x01010101u;
      const uint32_t s0 = lo * 0x22222200u + 0x10101010u;
      const uint32_t s1 = hi * 0x22222200u + (__popc(b[i] & 15u) * 0x22222222u + 0x10101010u);
      const uint32_t k0 = lo * 0xFFu, k1 = hi * 0xFFu;
      sts_u128(to + 8u * ROW_BYTES * i, prmt(v01[i], v23[i], s0) & prmt(k0, 0u, 0x1100u),
               prmt(v01[i], v23[i], s0 >> 16) & prmt(k0, 0u, 0x3322u),
               prmt(v01[i], v23[i], s1) & prmt(k1, 0u, 0x1100u),
               prmt(v01[i], v23[i], s1 >> 16) & prmt(k1, 0u, 0x3322u));
    }
    return;
  }
  // (the rank after a row's last value is never selected; it reads the next row or the one before)
  const uint32_t h = lane >> 3, p = lane & 7, b0 = 4u * p, below = (1u << b0) - 1u, r = (uint32_t)row0 + h;
  const uint32_t stage = 32u * j;
  // selectors by q (bit 0: the pair's first column kept, bit 1: the second) for the values v
  // (rank c) and w (rank c + 1): 0x3232 (0, 0), 0x3210 (v, 0), 0x1032 (0, v), 0x5410 (v, w)
  constexpr uint32_t kSelLo = 0x32103232u, kSelHi = 0x54101032u;
  uint32_t nib[8], v[8][4];
#pragma unroll
  for (int i = 0; i < 8; ++i) nib[i] = lds_u32(sM + (r + 4u * i) * (MW * 4u) + 4u * j);
#pragma unroll
  for (int i = 0; i < 8; ++i) {  // rows r + 4 i: row & 7 = h + 4 (i & 1)
    const uint32_t at = (sV + 128u * r) | ((h + 4u * (i & 1)) << 4), more = 4u * 128u * i;
    const uint32_t first = stage + 2u * __popc(nib[i] & below);
    nib[i] = (nib[i] >> b0) & 15u;
    const uint32_t second = first + 2u * __popc(nib[i] & 3u);
    v[i][0] = lds_u16_32((first ^ at) + more);
    v[i][1] = lds_u16_32(((first + 2u) ^ at) + more);
    v[i][2] = lds_u16_32((second ^ at) + more);
    v[i][3] = lds_u16_32(((second + 2u) ^ at) + more);
  }
#pragma unroll
  for (int i = 0; i < 8; ++i) {  // (row >> 1) & 3 = (h >> 1) ^ (2 (i & 1))
    const uint32_t lo = prmt(v[i][0], v[i][1], prmt(kSelLo, kSelHi, (nib[i] & 3u) * 0x22u + 0x10u));
    const uint32_t hi = prmt(v[i][2], v[i][3], prmt(kSelLo, kSelHi, (nib[i] >> 2) * 0x22u + 0x10u));
    sts_u64(sA + (r + 4u * i) * ROW_BYTES + (((p >> 1) ^ (h >> 1) ^ (2u * (i & 1))) << 4) + 8u * (p & 1), lo, hi);
  }
}

// Waits of this kernel: mbar_wait with what follows a first test out of line (inlined at
// each of them it is most of the kernel's code, and a block took 1 us longer).
__device__ __noinline__ bool wait_late(uint32_t bar, uint32_t parity, uint64_t limit_ns) {
  return mbar_wait(bar, parity, limit_ns);
}
__device__ __forceinline__ bool wait(uint32_t bar, uint32_t parity, uint64_t limit_ns) {
  return mbar_try_wait(bar, parity) || wait_late(bar, parity, limit_ns);
}

// For copies and MMAs that are on their way: they come, however short the limit of this
// launch and whatever else gave up, so this has the default limit.  But a barrier of both
// tokens and weights also counts the densify warps, which do not come any more once a wait
// has given up: then the copies have a tenth of a second.
constexpr uint64_t kDrainNs = 100000000;
__device__ __noinline__ void landed_late(uint32_t bar, uint32_t parity) {
  const uint64_t t0 = global_timer_ns();
  while (!mbar_try_wait(bar, parity))
    if ((int64_t)(global_timer_ns() - t0) > (int64_t)(wait_aborted() ? kDrainNs : kWaitLimitNs)) {
      atomicAdd(&g_wait_timeouts, 1ull);
      atomicExch(&g_wait_abort, 1u);
      break;
    }
}
__device__ __forceinline__ void landed(uint32_t bar, uint32_t parity) {
  if (!mbar_try_wait(bar, parity)) landed_late(bar, parity);
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

template <int NMMA, int NB, int S, int SV, int DG, int MS, bool MT>
__global__ void __launch_bounds__(threads_for(DW), 1)
    linear_tc_kernel(const __grid_constant__ CUtensorMap tm_v, const __grid_constant__ CUtensorMap tm_x,
                     const __grid_constant__ CUtensorMap tm_m, const uint32_t* __restrict__ masks, __half* Y,
                     int64_t rows, int words, int wslice, int64_t T, int64_t ldy, uint64_t wait_limit_ns,
                     int stall, const Epilogue e, int nmma) {
  using L = Shape<NMMA, NB, S, SV, DG, MS, MT>;
  constexpr int WPG = DW / DG;  // warps per densify group
  constexpr int RPW = BM / WPG;  // rows per warp and stage
  static_assert(RPW % 32 == 0, "expand_32");
  extern __shared__ uint8_t smem_raw[];
  const uint32_t raw = smem_addr(smem_raw);
  const uint32_t base = (raw + 1023u) & ~1023u;
  const uint32_t sA = base + L::A_OFF, sB = base + L::B_OFF, sV = base + L::V_OFF, sM = base + L::M_OFF,
                 bars = base + L::BAR_OFF, slot = base + L::SLOT_OFF;
  auto fullv = [&](int box) { return bars + 8u * (box % SV); };
  auto vfree = [&](int box) { return bars + 8u * (SV + box % SV); };
  auto ready = [&](int kt) { return bars + 8u * (2 * SV + kt % S); };
  auto done = [&](int kt) { return bars + 8u * (2 * SV + S + kt % L::RD); };
  const uint32_t accum = bars + 8u * (2 * SV + S + L::RD);

  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  pdl_launch_dependents();
  // After a wait gave up (this launch or an earlier one not yet reset), the block does
  // nothing: it has no stages, and no sums to send or to store.  It takes the way to the
  // end all the same: a cluster's blocks write each other's shared memory, so none leaves
  // before the others, and what follows on the stream is after the kernels before this
  // one.  (The flag is there once the setup is done: a wait for it first costs 0.5 us.)
  const bool aborted = threadIdx.x == 0 && wait_aborted();
  const int64_t r0 = (int64_t)blockIdx.y * BM;
  const int64_t n0 = (int64_t)blockIdx.x * (NB * nmma);

  if (warp == 0 && lane == 0) {
    for (int k = 0; k < SV; ++k) {
      mbar_init(fullv(k), MT ? 1 : 1 + 32);  // (+ 32 cp.async arrivals)
      mbar_init(vfree(k), DW);
    }
    for (int k = 0; k < S; ++k) mbar_init(ready(k), 1 + WPG);
    for (int k = 0; k < L::RD; ++k) mbar_init(done(k), MS == 2 ? 2 : 1);  // tcgen05.commit
    mbar_init(accum, 2);                                                  // final commit of each issuer
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
  const bool dead = __syncthreads_or(aborted);
  tc_fence_after_sync();
  // K split: this block multiplies the mask words w0 .. w0 + nk - 1 (stage kt is word
  // w0 + kt); w0 is a multiple of MW, so mask boxes stay aligned.
  const int w0 = (int)blockIdx.z * wslice;
  const int nk = dead ? 0 : min(words - w0, wslice);
  uint32_t tmem_base;
  asm volatile("ld.shared.u32 %0, [%1];" : "=r"(tmem_base) : "r"(slot) : "memory");
  pdl_wait_previous();  // (everything above touches no argument's memory)

  // Before it ends, a producer waits (bounded) for its copies among a ring's last: shared
  // memory must not be given up, or written by the cluster, under copies in flight.  Each
  // is the last use of its slot, whose use before it waited for.
  bool fine = false;  // (densify warps) the accumulator is whole
  if (warp == 0 || warp == tokens2_warp(DW)) {
    // ---- token tiles: the even stages, the odd ones --------------------------------
    // (A copy costs its thread 200 cycles and more: one alone would bound a stage.)
    if (lane == 0) {
      int last = -1;
      for (int kt = warp == 0 ? 0 : 1; kt < nk; kt += 2) {
        if (kt >= S && !wait(done(kt - S), ((kt - S) / L::RD) & 1, wait_limit_ns)) break;
        mbar_arrive_expect_tx(ready(kt), NB * nmma * ROW_BYTES);
#pragma unroll
        for (int j = 0; j < NB; ++j)
          tma_load_2d(sB + kt % S * L::B_BYTES + j * NMMA * ROW_BYTES, &tm_x, (w0 + kt) * BK,
                      (int)(n0 + j * nmma), ready(kt));
        last = kt;
      }
      for (int kt = last; kt >= 0 && kt > last - S; kt -= 2) landed(ready(kt), (kt / S) & 1);
    }
    __syncwarp();
  } else if (warp == 2) {
    // ---- compact values and mask words, a box of MW stages at a time ------------------
    // (stall, the self-test's: every other block's issue nothing)
    if ((!MT || lane == 0) && !(stall && (blockIdx.x + blockIdx.y + blockIdx.z) % 2 == 0)) {
      const int boxes = (nk + MW - 1) / MW;
      int last = -1;
      for (int box = 0; box < boxes; ++box) {
        int ok = 1;
        if (box >= SV && lane == 0) ok = wait(vfree(box), (box / SV - 1) & 1, wait_limit_ns);
        if (!MT) ok = __shfl_sync(0xFFFFFFFFu, ok, 0);
        if (!ok) break;
        const int at = box % SV, w = w0 + box * MW;
        if (lane == 0) {
          mbar_arrive_expect_tx(fullv(box), L::V_SLOT + (MT ? MT_SLOT : 0));
          tma_load_2d(sV + at * L::V_SLOT, &tm_v, w * 16, (int)r0, fullv(box));
          if (MT) tma_load_2d(sM + at * MT_SLOT, &tm_m, w, (int)r0, fullv(box));
        }
        if (!MT) {
#pragma unroll
          for (int i = 0; i < BM * MW / 32; ++i) {
            const int e = lane + 32 * i, word = w + e % MW;
            const int64_t gr = r0 + e / MW;
            const bool in = gr < rows && word < words;
            cp_async_4(sM + at * MT_SLOT + 4u * e, masks + (in ? gr * words + word : 0), in ? 4u : 0u);
          }
          cp_async_arrive_noinc(fullv(box));
        }
        last = box;
      }
      if (!MT) cp_async_wait_all();
      if (lane == 0)
        for (int box = last; box >= 0 && box > last - SV; --box)
          landed(fullv(box), (box / SV) & 1);
    }
    __syncwarp();
  } else if (warp == 1 || warp == mma2_warp(DW)) {
    // ---- MMAs ----------------------------------------------------------------------
    // The issuing threads share their schedulers with the densify warps, which keep those
    // two thirds busy: every instruction of a stage costs them several cycles, a barrier
    // test 100 to 200 and an MMA 80, so slots and phases are counted and not divided for,
    // descriptors are sums of 32 bits, and there are two such threads.
    auto issue = [&](auto which) {
      constexpr int role = decltype(which)::value;
      const uint32_t idesc = idesc_f16_f32(BM, nmma);
      const uint64_t a0 = smem_desc_sw64(sA), b0 = smem_desc_sw64(sB + (MS == 2 ? role * NMMA * ROW_BYTES : 0));
      const uint32_t a_high = (uint32_t)(a0 >> 32), b_high = (uint32_t)(b0 >> 32);
      const uint32_t a_low = (uint32_t)a0, b_low = (uint32_t)b0;
      auto desc = [](uint32_t high, uint32_t low) { return ((uint64_t)high << 32) | low; };
      constexpr int kStep = MS == 1 ? 2 : 1;
      constexpr int k0 = MS == 1 ? role : 0;
      const uint32_t dacc = tmem_base + (uint32_t)(role == 0 ? 0 : MS == 1 ? L::BN : NMMA);
      int at = k0, id = k0;  // the slot, and the place in done's ring
      uint32_t phase = 0;
      auto next = [](int& i, int ring) {
        i += kStep;
        const bool around = i >= ring;
        if (around) i -= ring;
        return around ? 1u : 0u;
      };
      bool gave_up = false;
      for (int kt = k0; kt < nk; kt += kStep) {
        if (!__all_sync(0xFFFFFFFFu, wait(ready(0) + 8u * at, phase, wait_limit_ns))) {
          gave_up = true;
          break;
        }
        tc_fence_after_sync();
        const uint32_t al = a_low + (uint32_t)at * (A_BYTES / 16), bl = b_low + (uint32_t)at * (L::B_BYTES / 16);
        if (elect_one()) {
#pragma unroll
          for (int ks = 0; ks < BK / 16; ++ks)
            mma_f16(dacc, desc(a_high, al + ks * 2), desc(b_high, bl + ks * 2), idesc, kt != k0 || ks != 0);
          // Only where someone waits for it: a commit's arrival is not ordered with the
          // accum commit's, so another could land after this block ended, in the barriers
          // of the next block on the SM.
          if (kt + S < nk) mma_commit(done(0) + 8u * id);
        }
        __syncwarp();
        phase ^= next(at, S);
        next(id, L::RD);
      }
      if (elect_one()) mma_commit(accum);  // also after an early exit: completes once issued MMAs finish
      if (gave_up) __nanosleep(200000);    // (arrivals in done that nobody waits for any more land meanwhile)
    };
    if (warp == 1)
      issue(std::integral_constant<int, 0>());
    else
      issue(std::integral_constant<int, 1>());
    __syncwarp();
  } else {
    // ---- expansion of the weights ------------------------------------------------------
    const int dw = warp - FIRST_DENSIFY_WARP, grp = dw / WPG, wg = dw % WPG;
    bool ok = !dead, bytes = true;
    for (int kt = grp; kt < nk; kt += DG) {
      const int box = kt / MW, at = box % SV;
      bool got = wait(fullv(box), (box / SV) & 1, wait_limit_ns);
      if (kt >= S) got = got && wait(done(kt - S), ((kt - S) / L::RD) & 1, wait_limit_ns);
      // The warp decides together, so no lane is left behind at a warp barrier.
      if (!__all_sync(0xFFFFFFFFu, got)) {
        ok = false;
        break;
      }
#pragma unroll
      for (int q = 0; q < RPW; q += 32)
        expand_32(sA + kt % S * A_BYTES, sV + at * L::V_SLOT, sM + at * MT_SLOT, kt % MW, wg * RPW + q, lane, bytes);
      // Each lane orders its tile writes before the tensor core's reads; the warp barrier
      // then lets one release-arrive publish all 32 lanes' writes and the end of their
      // reads of the values and the masks.
      fence_proxy_async_smem();
      __syncwarp();
      if (lane == 0) {
        mbar_arrive(ready(kt));
        if (kt + DG >= MW * (box + 1)) mbar_arrive(vfree(box));  // its last stage in the box
      }
    }
    if (!wait(accum, 0, wait_limit_ns)) ok = false;
    tc_fence_after_sync();
    // tcgen05.ld is a warp-wide instruction: the whole warp reads or none does.
    fine = __all_sync(0xFFFFFFFFu, ok);
  }

  // ---- epilogue --------------------------------------------------------------------------
  // The accumulator's columns in pieces of 32 (an MMA's tokens may end inside one).  Under
  // a K split the blocks of a row tile's slices are a cluster: piece i is finished by block
  // i % slices, to which the others send theirs through distributed shared memory (their
  // rings lie idle by now), and which adds them in slice order: nothing goes through memory,
  // and there is no second launch.
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
    if (MS == 1 && nk > 1) {  // the odd stages' accumulator (none when nk == 1)
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
      linear_store_32(e, v, r < rows, r, first(i), n, Y, ldy, lane);
    }
  }

  tc_fence_before_sync();
  __syncthreads();
  if (warp == 1) {
    // Tensor memory is freed only after the MMAs that write it have completed: one more
    // bounded (not abortable) wait on the final commit, which a normal run passed already.
    landed(accum, 0);
    tc_fence_after_sync();
    tmem_dealloc(tmem_base, L::TMEM_COLS);
  }
}

template <int NMMA, int NB, int S, int SV, int DG, int MS, bool MT>
cudaError_t launch_mt(const SpmmTcParams& p, cudaStream_t stream) {
  using L = Shape<NMMA, NB, S, SV, DG, MS, MT>;
  if (p.tile < 16 || p.tile > NMMA || p.tile % 16) return cudaErrorInvalidValue;
  CUtensorMap tm_v, tm_x, tm_m;
  memset(&tm_m, 0, sizeof(tm_m));
  if (MT && !encode_2d(&tm_m, p.masks, (uint64_t)p.words, (uint64_t)p.rows, (uint64_t)p.words * 4, MW, BM,
                       CU_TENSOR_MAP_SWIZZLE_NONE, CU_TENSOR_MAP_DATA_TYPE_UINT32))
    return cudaErrorInvalidValue;
  if (!encode_2d(&tm_v, p.values, (uint64_t)p.words * 16, (uint64_t)p.rows, (uint64_t)p.words * 32, MW * 16, BM,
                 CU_TENSOR_MAP_SWIZZLE_128B) ||
      !encode_2d(&tm_x, p.X, (uint64_t)p.words * 32, (uint64_t)p.T, (uint64_t)p.ldx * 2, BK, p.tile,
                 CU_TENSOR_MAP_SWIZZLE_64B))
    return cudaErrorInvalidValue;
  if (p.slices > 1) {  // what a block is sent fits its rings
    const int pieces = NB * ((p.tile + 31) / 32), share = (pieces + p.slices - 1) / p.slices;
    if ((p.slices - 1) * share * 32 * BM * 4 > L::BAR_OFF) return cudaErrorInvalidValue;
  }
  auto* k = linear_tc_kernel<NMMA, NB, S, SV, DG, MS, MT>;
  static int done[64] = {0};
  int dev = 0;
  cudaError_t err = cudaGetDevice(&dev);
  if (err != cudaSuccess) return err;
  if (dev >= 64 || !__atomic_load_n(&done[dev], __ATOMIC_ACQUIRE)) {
    err = cudaFuncSetAttribute(k, cudaFuncAttributeMaxDynamicSharedMemorySize, L::SMEM);
    if (err != cudaSuccess) return err;
    if (dev < 64) __atomic_store_n(&done[dev], 1, __ATOMIC_RELEASE);
  }
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)((p.T + NB * p.tile - 1) / (NB * p.tile)), (unsigned)((p.rows + BM - 1) / BM),
                     (unsigned)p.slices);
  cfg.blockDim = dim3(threads_for(DW));
  cfg.dynamicSmemBytes = L::SMEM;
  cfg.stream = stream;
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  attr[1].id = cudaLaunchAttributeClusterDimension;
  attr[1].val.clusterDim.x = attr[1].val.clusterDim.y = 1;
  attr[1].val.clusterDim.z = (unsigned)p.slices;
  cfg.attrs = attr;
  cfg.numAttrs = p.slices > 1 ? 2 : 1;
  return cudaLaunchKernelEx(&cfg, k, tm_v, tm_x, tm_m, p.masks, p.Y, p.rows, p.words,
                            p.slices > 1 ? p.wslice : p.words, p.T, p.ldy, p.wait_limit_ns ? p.wait_limit_ns : kWaitLimitNs,
                            p.stall_weights, p.epi, p.tile);
}

// Mask words by TMA when the mask array allows it (16-byte aligned, row pitch words * 4 a
// multiple of 16: every decoder shape), else by cp.async.
template <int NMMA, int NB, int S, int SV, int DG, int MS>
cudaError_t launch(const SpmmTcParams& p, cudaStream_t stream) {
  const bool mt = p.words % 4 == 0 && (reinterpret_cast<uintptr_t>(p.masks) & 15) == 0;
  return mt ? launch_mt<NMMA, NB, S, SV, DG, MS, true>(p, stream)
            : launch_mt<NMMA, NB, S, SV, DG, MS, false>(p, stream);
}

}  // namespace
}  // namespace tc

// variant: kCands' index
cudaError_t launch_spmm_tc_linear(const SpmmTcParams& p, int variant, cudaStream_t stream) {
  switch (variant) {
    case 0: return tc::launch<256, 2, 4, 3, 4, 2>(p, stream);
    case 1: return tc::launch<256, 1, 6, 4, 4, 1>(p, stream);
    case 2: return tc::launch<128, 1, 8, 5, 4, 1>(p, stream);
    case 3: return tc::launch<160, 2, 6, 3, 4, 2>(p, stream);
    default: return cudaErrorInvalidValue;
  }
}

namespace {

// (variant, MMAs a block, tokens of an MMA at most, ns a stage: base, and by token beyond
// `flat`), measured with 152 row tiles of 8192 columns, 2:4, one block an SM: 296 ns at 128
// tokens to 425 at 512, 220 to 257 (256 tokens), 211, and 245 to 285 (320).  Up to 128
// tokens the expansion of the weights bounds a stage, with two MMAs a stage their issue,
// and at 512 the loads of token tiles (32 KB in 1.3 us, four under way).
struct Cand {
  int variant, mmas, most;
  double ns, by_token;
  int flat;
};
constexpr Cand kCands[] = {{0, 2, 256, 290.0, 0.27, 64}, {1, 1, 256, 222.0, 0.28, 128},
                           {2, 1, 128, 211.0, 0.0, 0}, {3, 2, 160, 245.0, 0.6, 256}};
constexpr double kFixedNs = 4000.0;   // prologue, pipeline fill, teardown
constexpr double kTokenNs = 10.5;     // the epilogue, a token of the tile
constexpr double kClusterNs = 2500.0; // the slices' exchange,
constexpr double kSliceNs = 250.0;    // each of them, and
constexpr double kSentNs = 4.0;       // what a token's share of it takes
// Clusters of 1 .. 8 such blocks that run at once on 152 SMs (cudaOccupancyMaxActiveClusters):
// a cluster's SMs belong to one group of them.
constexpr int kClusters[] = {152, 76, 46, 36, 28, 23, 15, 15};
constexpr int kMaxSlices = 8, kMaxSent = 13;  // pieces of 16 KB that a block's rings can take

}  // namespace

// The least time by a model: waves of blocks x (a slice's stages + fixed costs).  Tokens
// are spread evenly over the blocks that a variant's full tiles would need, and over a
// block's MMAs, in multiples of 16 (300 tokens: two MMAs of 160 for two of 256).
LinearTcPlan linear_tc_plan(int64_t rows, int words, int64_t tokens, int sms) {
  LinearTcPlan best{2, 1, 16};
  double least = 0.0;
  for (const Cand& c : kCands) {
    const int64_t full = (int64_t)c.most * c.mmas, blocks = (tokens + full - 1) / full;
    const int64_t each = (tokens + blocks - 1) / blocks;
    const int tile = (int)(((each + c.mmas - 1) / c.mmas + 15) / 16 * 16);
    const int64_t tiles = (rows + 127) / 128 * ((tokens + tile * c.mmas - 1) / (tile * c.mmas));
    const int all = tile * c.mmas, pieces = c.mmas * ((tile + 31) / 32);
    const double stage = c.ns + c.by_token * (all > c.flat ? all - c.flat : 0);
    for (int z = 1; z <= kMaxSlices; ++z) {
      if (z > 1 && (spmm_tc_slices(words, z) != z || (z - 1) * ((pieces + z - 1) / z) > kMaxSent)) continue;
      const int64_t clusters = (int64_t)kClusters[z - 1] * sms / 152, at_once = (clusters > 0 ? clusters : 1) * z;
      const int64_t waves = (tiles * z + at_once - 1) / at_once;
      const double exchange = z > 1 ? kClusterNs + kSliceNs * z + kSentNs * all : 0.0;
      const double t = waves * (spmm_tc_slice_words(words, z) * stage + kFixedNs + kTokenNs * all / z + exchange);
      if (least == 0.0 || t < least * 0.98) {
        least = t;
        best = {c.variant, z, tile};
      }
    }
  }
  return best;
}

// ---- nm_linear for 1 .. 8 tokens of rows too long for a block's shared memory, whose
// columns are cut: the partial sums that nm_spmm's kernel leaves are added and finished here.  V rows a thread
// (an even number of them where rows come in pairs): V = 4 takes 16-byte loads of the
// partial sums, which need rows % 4 == 0; V = 2 serves any even number of rows, V = 1 the
// rest.
template <int V>
__global__ void __launch_bounds__(256) linear_combine_kernel(const float* __restrict__ part,
                                                             int slices, int64_t tokens,
                                                             int64_t rows, const Epilogue e,
                                                             __half* Y, int64_t ldy) {
  pdl_launch_dependents();
  pdl_wait_previous();
  const int64_t plane = tokens * rows;
  for (int64_t t = blockIdx.y; t < tokens; t += gridDim.y) {
    for (int64_t r = ((int64_t)blockIdx.x * blockDim.x + threadIdx.x) * V; r < rows;
         r += (int64_t)gridDim.x * blockDim.x * V) {
      const float* q = part + t * rows + r;
      float s[V];
#pragma unroll
      for (int i = 0; i < V; ++i) s[i] = 0.f;
#pragma unroll 4
      for (int z = 0; z < slices; ++z) {
        if constexpr (V == 4) {
          const float4 a = *reinterpret_cast<const float4*>(q + z * plane);
          s[0] += a.x; s[1] += a.y; s[2] += a.z; s[3] += a.w;
        } else {
#pragma unroll
          for (int i = 0; i < V; ++i) s[i] += q[z * plane + i];
        }
      }
#pragma unroll
      for (int i = 0; i < V; ++i) s[i] += bias_at(e, r + i);
      if (V > 1 && e.gated) {
#pragma unroll
        for (int i = 0; i + 1 < V; i += 2) {
          const int64_t o = (r + i) / 2;
          Y[t * ldy + o] = __float2half_rn(fmaf(e.scale, activate(s[i], e.act) * s[i + 1], residual_at(e, t, o)));
        }
      } else {
#pragma unroll
        for (int i = 0; i < V; ++i)
          Y[t * ldy + r + i] = __float2half_rn(fmaf(e.scale, activate(s[i], e.act), residual_at(e, t, r + i)));
      }
    }
  }
}

cudaError_t launch_linear_combine(const float* part, int slices, int64_t tokens, int64_t rows,
                                  const Epilogue& epi, __half* Y, int64_t ldy, int sms,
                                  cudaStream_t stream) {
  const int v = rows % 4 == 0 ? 4 : rows % 2 == 0 ? 2 : 1;
  const int64_t bx = (rows + 256 * v - 1) / (256 * v);
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)(bx < 65535 ? bx : 65535), (unsigned)(tokens < 65535 ? tokens : 65535));
  cfg.blockDim = dim3(256);
  cfg.stream = stream;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  auto* k = v == 4 ? linear_combine_kernel<4> : v == 2 ? linear_combine_kernel<2> : linear_combine_kernel<1>;
  return cudaLaunchKernelEx(&cfg, k, part, slices, tokens, rows, epi, Y, ldy);
}

cudaError_t read_linear_wait_timeouts(unsigned long long* count, int reset) {
  return read_local_wait_timeouts(count, reset);
}

}  // namespace nmk
