// norm_rows.cuh -- what the kernels of nm_residual_norm share (residual_norm.cu,
// residual_norm_any.cu): arithmetic on pairs, sums over a row, launches of a row a block.
#pragma once

#include <cuda_fp16.h>
#include <cuda_runtime.h>
#include <stdint.h>

#include "../../include/nm_layer.h"
#include "device.cuh"
#include "kernels.h"
#include "layer.h"

namespace nmk {
namespace {

// Two fp32 values, and arithmetic on both at once.
using Pair = float2;

__device__ __forceinline__ Pair pair(float a, float b) { return make_float2(a, b); }
__device__ __forceinline__ Pair fma2(Pair a, Pair b, Pair c) { return __ffma2_rn(a, b, c); }
__device__ __forceinline__ Pair mul2(Pair a, Pair b) { return __fmul2_rn(a, b); }
__device__ __forceinline__ Pair add2(Pair a, Pair b) { return __fadd2_rn(a, b); }

// Sum over the threads of a row (threadIdx.y's, blockDim.x of them).
struct RowSum {
  float (*part)[32];  // [2][warps of the block]
  int turn = 0;
  __device__ __forceinline__ float operator()(float v) {
    v = warp_sum(v);
    const int warps = blockDim.x >> 5;
    if (warps == 1) return v;
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    float* at = part[turn] + threadIdx.y * warps;
    turn ^= 1;  // the sum after next writes here again, past the next one's barrier
    if (lane == 0) at[warp] = v;
    __syncthreads();
    if (warps <= 8) {
      v = (lane & 7) < warps ? at[lane & 7] : 0.f;
#pragma unroll
      for (int o = 4; o > 0; o >>= 1) v += __shfl_xor_sync(0xFFFFFFFFu, v, o);
      return v;
    }
    if (warps <= 16) {
      v = (lane & 15) < warps ? at[lane & 15] : 0.f;
#pragma unroll
      for (int o = 8; o > 0; o >>= 1) v += __shfl_xor_sync(0xFFFFFFFFu, v, o);
      return v;
    }
    return warp_sum(lane < warps ? at[lane] : 0.f);
  }
};

// A kernel that takes a row on `threads` threads (a multiple of 32).
template <typename K>
cudaError_t launch_rows(K* kernel, const ResidualNormParams& p, int threads, cudaStream_t stream) {
  const int rows = threads >= 256 ? 1 : 256 / threads;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)((p.tokens + rows - 1) / rows));
  cfg.blockDim = dim3((unsigned)threads, (unsigned)rows);
  cfg.stream = stream;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, kernel, p);
}

}  // namespace
}  // namespace nmk
