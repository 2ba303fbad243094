// prefill_linear.cu -- nm_linear's products for more than 8 tokens: nm_spmm_prefill's
// kernel with the epilogue, in the variants that the plans choose from, and the
// combine of its K split (and of nm_spmm's column slices).
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

// Tokens of one MMA: the tokens spread evenly over the blocks that the variant's full
// tiles would need, and over a block's MMAs, in multiples of 16.  (300 tokens: two of
// 160 in a block for two of 256.)
int linear_tile(int variant, int64_t tokens) {
  constexpr int kMmas[] = {2, 1, 1, 1, 2};
  const int64_t full = spmm_tc_block_tokens(variant), blocks = (tokens + full - 1) / full;
  const int64_t each = (tokens + blocks - 1) / blocks, n = kMmas[variant];
  return (int)(((each + n - 1) / n + 15) / 16 * 16);
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
          Y[t * ldy + o] = __float2half_rn(fmaf(e.scale, activate_fast(s[i], e.act) * s[i + 1], residual_at(e, t, o)));
        }
      } else {
#pragma unroll
        for (int i = 0; i < V; ++i)
          Y[t * ldy + r + i] = __float2half_rn(fmaf(e.scale, activate_fast(s[i], e.act), residual_at(e, t, r + i)));
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
