// epilogue.cuh -- the epilogue of nm_linear: y = residual + scale * act(sum + bias),
// or with rows in (gate, up) pairs act(gate) * up, all in fp32.
#pragma once

#include <cuda_fp16.h>
#include <stdint.h>

#include "../../include/nm_layer.h"
#include "device.cuh"
#include "kernels.h"

namespace nmk {

// (Not inlined: a copy for each of a thread's outputs overran the instruction cache, which
// cost the tensor-core kernel's epilogue 3 us even where no activation was asked for.)
static __device__ __noinline__ float gelu(float x) {
  return 0.5f * x * erfcf(x * -0.70710678118654752f);  // 1 + erf(-5) has no digits left
}

__device__ __forceinline__ float activate(float x, int act) {
  switch (act) {  // the same for every thread of a launch
    case NM_ACT_RELU: return x > 0.f ? x : (x != x ? x : 0.f);
    case NM_ACT_SILU: return x / (1.f + expf(-x));
    case NM_ACT_GELU: return gelu(x);
    case NM_ACT_GELU_TANH:  // (1 + tanh u) / 2 = 1 / (1 + e^-2u)
      return x / (1.f + expf(-1.59576912160573071f * fmaf(0.044715f * x * x, x, x)));
    default: return x;
  }
}

// The same for N values of the tensor-core kernel, whose epilogue nothing overlaps: 2^x of
// the hardware and an approximate division, 2^-18 relative beside the 2^-11 of the fp16
// result (the argument of 2^x carries 2^-24 of itself).
template <int N>
__device__ __forceinline__ void activate_fast(float (&x)[N], int act) {
  if (act == NM_ACT_NONE) return;
  if (act == NM_ACT_RELU) {
#pragma unroll
    for (int i = 0; i < N; ++i) x[i] = activate(x[i], NM_ACT_RELU);
  } else if (act == NM_ACT_GELU) {
    // The normal distribution's tail q(u) = e^(-u^2 / 2) f(u), u = |x|, with f a polynomial
    // of 1 / (1 + 0.21 u): a least-squares fit of its relative error, reweighted until it
    // was level, 7e-7 for u up to 7 (q is 1e-12 there), 1e-6 with fp32's roundings.
#pragma unroll
    for (int i = 0; i < N; ++i) {
      const float u = fabsf(x[i]), t = __fdividef(1.f, fmaf(0.21f, u, 1.f));
      float f = 0.52884574f;
      f = fmaf(f, t, -0.96879248f);
      f = fmaf(f, t, 1.1535979f);
      f = fmaf(f, t, -0.56957506f);
      f = fmaf(f, t, 0.31265665f);
      f = fmaf(f, t, 0.039669259f);
      f = fmaf(f, t, 0.0035983000f);
      const float q = f * exp2_fast(x[i] * x[i] * (-0.5f * kLog2e));
      x[i] *= x[i] > 0.f ? 1.f - q : q;
    }
  } else {
    const bool silu = act == NM_ACT_SILU;
#pragma unroll
    for (int i = 0; i < N; ++i) {
      const float t = silu ? x[i] * -kLog2e
                           : (-1.59576912160573071f * kLog2e) * fmaf(0.044715f * x[i] * x[i], x[i], x[i]);
      x[i] = __fdividef(x[i], 1.f + exp2_fast(t));
    }
  }
}

__device__ __forceinline__ float bias_at(const Epilogue& e, int64_t row) {
  return e.bias ? __half2float(e.bias[row]) : 0.f;
}

__device__ __forceinline__ float residual_at(const Epilogue& e, int64_t token, int64_t i) {
  return e.residual ? __half2float(e.residual[token * e.ldres + i]) : 0.f;
}

}  // namespace nmk
