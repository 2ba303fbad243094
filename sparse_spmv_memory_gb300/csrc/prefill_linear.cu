// prefill_linear.cu -- nm_linear's products for more than 8 tokens: nm_spmm_prefill's
// kernel with the epilogue, in the variants that the plans choose from, and the
// combine of nm_spmm's column slices.
#include <cuda_fp16.h>
#include <cuda_runtime.h>
#include <stdint.h>

#include "kernels.h"
#include "prefill_kernels.cuh"

namespace nmk {

cudaError_t launch_spmm_tc_linear(const SpmmTcParams& p, int variant, cudaStream_t stream) {
  switch (variant) {  // as in tc::kVariants (prefill.cu)
    case 1: return tc::launch_tc<256, 1, 7, 1, 2, 16, 1, true>(p, stream);
    case 2: return tc::launch_tc<128, 1, 10, 1, 4, 16, 1, true>(p, stream);
    case 3: return tc::launch_tc<64, 1, 12, 1, 4, 16, 1, true>(p, stream);
    case 4: return tc::launch_tc<256, 2, 5, 1, 4, 16, 0, true>(p, stream);
    default: return cudaErrorInvalidValue;
  }
}

namespace {

// (variant, MMAs a block, tokens of an MMA at most, ns a stage: base, and by token beyond
// `flat`).  Measured with 152 row tiles of 8192 columns, one block an SM, at 16 tokens
// an MMA up to the most: 375 .. 456 ns, 305 .. 340, 259 .. 264, 239; up to there the
// expansion of the weights bounds a stage and beyond the MMAs.
struct Cand {
  int variant, mmas, most;
  double ns, by_token;
  int flat;
};
constexpr Cand kCands[] = {{4, 2, 256, 372.0, 0.42, 256}, {1, 1, 256, 305.0, 0.34, 144},
                           {2, 1, 128, 259.0, 0.04, 0}, {3, 1, 64, 239.0, 0.0, 0}};
constexpr double kFixedNs = 4000.0;   // prologue, pipeline fill, teardown
constexpr double kTokenNs = 16.0;     // the epilogue, a token of the tile
constexpr double kClusterNs = 1200.0; // the slices' exchange, and
constexpr double kSentNs = 6.0;       // what a token's share of it takes
constexpr int kMaxSlices = 8, kMaxSent = 13;  // pieces of 16 KB that a ring can take

}  // namespace

// The least time by a model: waves of blocks x (a slice's stages + fixed costs).  Tokens
// are spread evenly over the blocks that a variant's full tiles would need, and over a
// block's MMAs, in multiples of 16 (300 tokens: two MMAs of 160 for two of 256).
LinearTcPlan linear_tc_plan(int64_t rows, int words, int64_t tokens, int sms) {
  LinearTcPlan best{3, 1, 64};
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
      // clusters of z blocks leave some of a cluster's places empty: whole ones of 16 SMs
      const int64_t at_once = z == 1 ? sms : (int64_t)sms / 16 * (16 / z) * z + sms % 16 / z * z;
      const int64_t waves = (tiles * z + at_once - 1) / at_once;
      const double exchange = z > 1 ? kClusterNs + kSentNs * all : 0.0;
      const double t = waves * (spmm_tc_slice_words(words, z) * stage + kFixedNs + kTokenNs * all / z + exchange);
      if (least == 0.0 || t < least * 0.98) {
        least = t;
        best = {c.variant, z, tile};
      }
    }
  }
  return best;
}

cudaError_t read_linear_wait_timeouts(unsigned long long* count, int reset) {
  return read_local_wait_timeouts(count, reset);
}

// V rows a thread (an even number of them where rows come in pairs): V = 4 takes
// 16-byte loads of the partial sums, which need rows % 4 == 0; V = 2 serves any
// even number of rows, V = 1 the rest.
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

}  // namespace nmk
