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

// Sums over the threads of a row (threadIdx.y's, blockDim.x of them), of one value or of
// two at once.
struct RowSum {
  float (*part)[32];  // [4][warps of the block]
  int turn = 0;
  __device__ __forceinline__ float operator()(float v) {
    v = warp_sum(v);
    const int warps = blockDim.x >> 5;
    if (warps == 1) return v;
    const int at = take_turn();
    const int lane = threadIdx.x & 31;
    if (lane == 0) part[at][first() + (threadIdx.x >> 5)] = v;
    __syncthreads();
    return joined(part[at] + first(), warps, lane);
  }
  // (The lanes' halves take a value each after the first exchange: two values cost little
  // more than one.)
  __device__ __forceinline__ Pair operator()(Pair v) {
    const int lane = threadIdx.x & 31, which = lane >> 4;
    float u = halves(v, which);
    const int warps = blockDim.x >> 5;
    if (warps > 1) {
      const int at = take_turn();
      if ((lane & 15) == 0) part[at + which][first() + (threadIdx.x >> 5)] = u;
      __syncthreads();
      if (warps <= 16) {
        const int n = warps <= 8 ? 8 : 16, i = lane & (n - 1);
        u = i < warps ? part[at + which][first() + i] : 0.f;
        if (n == 16) u += __shfl_xor_sync(0xFFFFFFFFu, u, 8);
#pragma unroll
        for (int o = 4; o > 0; o >>= 1) u += __shfl_xor_sync(0xFFFFFFFFu, u, o);
      } else {
        const bool in = lane < warps;
        u = halves(pair(in ? part[at][first() + lane] : 0.f, in ? part[at + 1][first() + lane] : 0.f), which);
      }
    }
    return pair(__shfl_sync(0xFFFFFFFFu, u, 0), __shfl_sync(0xFFFFFFFFu, u, 16));
  }

 private:
  __device__ __forceinline__ int take_turn() {  // the sum after next writes here again, past the next one's barrier
    const int at = turn;
    turn ^= 2;
    return at;
  }
  // The warp's sum of v.x in the lower lanes, of v.y in the upper.
  static __device__ __forceinline__ float halves(Pair v, int which) {
    float u = (which ? v.y : v.x) + __shfl_xor_sync(0xFFFFFFFFu, which ? v.x : v.y, 16);
#pragma unroll
    for (int o = 8; o > 0; o >>= 1) u += __shfl_xor_sync(0xFFFFFFFFu, u, o);
    return u;
  }
  __device__ __forceinline__ int first() const { return threadIdx.y * (blockDim.x >> 5); }
  static __device__ __forceinline__ float joined(const float* at, int warps, int lane) {
    if (warps <= 8) {
      float v = (lane & 7) < warps ? at[lane & 7] : 0.f;
#pragma unroll
      for (int o = 4; o > 0; o >>= 1) v += __shfl_xor_sync(0xFFFFFFFFu, v, o);
      return v;
    }
    if (warps <= 16) {
      float v = (lane & 15) < warps ? at[lane & 15] : 0.f;
#pragma unroll
      for (int o = 8; o > 0; o >>= 1) v += __shfl_xor_sync(0xFFFFFFFFu, v, o);
      return v;
    }
    return warp_sum(lane < warps ? at[lane] : 0.f);
  }
};

// A layer norm's mean as a first sum gives it is off by roundings, |mean| 2^-24 and more,
// which counts where the deviations are not larger (a row of equal elements is normed by
// eps alone).  What it is off by is the mean of what it leaves: the norm is (x - rest) r
// of the elements x about the first mean, both from their sum and their squares' sum.
struct Factor {
  float r, rest;  // (rest 0 but for layer norms)
};

__device__ __forceinline__ Factor layer_factor(Pair sums, float inv_width, float eps) {
  const float rest = sums.x * inv_width, var = fmaf(-rest, rest, sums.y * inv_width);
  return {1.f / sqrtf((var < 0.f ? 0.f : var) + eps), rest};  // (NaN stays)
}

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
