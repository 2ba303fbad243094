// epilogue.cuh -- the epilogue of nm_linear: y = residual + scale * act(sum + bias),
// or with rows in (gate, up) pairs act(gate) * up, all in fp32.
#pragma once

#include <cuda_fp16.h>
#include <stdint.h>

#include "../../include/nm_layer.h"
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

__device__ __forceinline__ float bias_at(const Epilogue& e, int64_t row) {
  return e.bias ? __half2float(e.bias[row]) : 0.f;
}

__device__ __forceinline__ float residual_at(const Epilogue& e, int64_t token, int64_t i) {
  return e.residual ? __half2float(e.residual[token * e.ldres + i]) : 0.f;
}

}  // namespace nmk
