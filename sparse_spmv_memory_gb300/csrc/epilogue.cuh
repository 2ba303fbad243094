// epilogue.cuh -- the epilogue of nm_linear: y = residual + scale * act(sum + bias),
// or with rows in (gate, up) pairs act(gate) * up, all in fp32.
#pragma once

#include <cuda_fp16.h>
#include <stdint.h>

#include "../../include/nm_layer.h"
#include "device.cuh"
#include "kernels.h"

namespace nmk {

__device__ __forceinline__ float activate(float x, int act) {
  switch (act) {  // the same for every thread of a launch
    case NM_ACT_RELU: return x > 0.f ? x : (x != x ? x : 0.f);
    case NM_ACT_SILU: return x / (1.f + expf(-x));
    case NM_ACT_GELU: return 0.5f * x * erfcf(x * -0.70710678118654752f);  // 1 + erf(-5) has no digits left
    case NM_ACT_GELU_TANH:  // (1 + tanh u) / 2 = 1 / (1 + e^-2u)
      return x / (1.f + expf(-1.59576912160573071f * fmaf(0.044715f * x * x, x, x)));
    default: return x;
  }
}

// The same for the tensor-core kernel, whose epilogue nothing overlaps (exact division
// and expf cost a wave of 128 x 512 tiles 9 us of 12): 2^x of the hardware and an
// approximate division, 2^-21 relative beside the 2^-11 of the fp16 result.
__device__ __forceinline__ float activate_fast(float x, int act) {
  switch (act) {
    case NM_ACT_SILU: return __fdividef(x, 1.f + exp2_fast(x * -kLog2e));
    case NM_ACT_GELU_TANH:
      return __fdividef(x, 1.f + exp2_fast((-1.59576912160573071f * kLog2e) * fmaf(0.044715f * x * x, x, x)));
    default: return activate(x, act);
  }
}

__device__ __forceinline__ float bias_at(const Epilogue& e, int64_t row) {
  return e.bias ? __half2float(e.bias[row]) : 0.f;
}

__device__ __forceinline__ float residual_at(const Epilogue& e, int64_t token, int64_t i) {
  return e.residual ? __half2float(e.residual[token * e.ldres + i]) : 0.f;
}

}  // namespace nmk
