// densify.cuh -- what the tensor-core products of the N:M format share (prefill.cu,
// linear_tc.cu): tile sizes, the expansion of compact values and mask words into a
// swizzled fp16 tile, and 2-D tensor maps.
#pragma once

#include <cuda.h>
#include <cuda_runtime.h>
#include <stdint.h>

#include "device.cuh"
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

constexpr int gcd_int(int a, int b) { return b ? gcd_int(b, a % b) : a; }


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

static bool encode_2d(CUtensorMap* m, const void* ptr, uint64_t inner, uint64_t outer,
                      uint64_t stride_bytes, uint32_t box_inner, uint32_t box_outer,
                      CUtensorMapSwizzle swz,
                      CUtensorMapDataType dtype = CU_TENSOR_MAP_DATA_TYPE_FLOAT16) {
  const cuuint64_t dims[2] = {inner, outer};
  const cuuint64_t strides[1] = {stride_bytes};
  const cuuint32_t box[2] = {box_inner, box_outer};
  return encode_tiled(m, dtype, ptr, 2, dims, strides, box, swz);
}

}  // namespace tc
}  // namespace nmk
