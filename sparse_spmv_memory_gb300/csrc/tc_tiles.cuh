// tc_tiles.cuh -- what the tensor-core products of the N:M format share (prefill.cu,
// linear_tc.cu): tile sizes, the places of a block's warps, and 2-D tensor maps.
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
