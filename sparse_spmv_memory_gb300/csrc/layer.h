// layer.h -- internal launch interface between the C ABI of nm_layer.h
// (layer_api.cu) and its kernels.  Not part of the public ABI.
#pragma once

#include <cuda_fp16.h>
#include <cuda_runtime.h>
#include <stdint.h>

#include "kernels.h"

namespace nmk {

// ---- the residual stream's update and the norms around it (residual_norm.cu) ----
struct NormArgs {
  const void *weight, *bias;  // null: 1, 0
  int kind;                   // NM_NORM_*
  int params_fp32;
  float offset, eps;
};

struct ResidualNormParams {
  const void* residual;  // fp16 or fp32
  int64_t ldr;
  const __half* block;  // null: no update
  int64_t ldb;
  NormArgs post;
  const __half* gate;  // null: 1
  int64_t ldg;
  float scale, residual_scale;
  void* stream_out;  // as residual; null: not written
  int64_t lds;
  NormArgs pre;
  __half* out;  // null: not computed
  int64_t ldo;
  int64_t tokens;
  int width;
  // set by the launcher
  float inv_width = 0.f;
  int own_gate = 0;  // 1: a gate for every token
};
cudaError_t launch_residual_norm(const ResidualNormParams& p, int stream_fp32, const DeviceInfo& d,
                                 cudaStream_t stream);

// rows of any stride and alignment, element by element (residual_norm_any.cu), and
// whether they are taken: widths up to 8192, or 16384 where all rows are of pairs
bool takes_any_rows(const ResidualNormParams& p, int stream_fp32);
cudaError_t launch_any_rows(const ResidualNormParams& p, int stream_fp32, cudaStream_t stream);

// ---- log probabilities of tokens (logprobs.cu) ----------------------------------
struct LogprobsParams {
  const void* logits;
  int64_t ld_logits;
  int64_t rows;
  int vocab;
  const int32_t* ids;
  int64_t ld_ids;
  int n_ids;
  float temperature;
  float* logprob;
  float* entropy;  // may be null
  int top;
  int32_t* top_ids;
  float* top_logprob;
};
cudaError_t launch_logprobs(const LogprobsParams& p, int logits_fp32, int sms, cudaStream_t stream);

}  // namespace nmk
