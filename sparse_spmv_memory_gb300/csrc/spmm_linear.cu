// spmm_linear.cu -- nm_linear's products for 2..8 tokens (and for one token with rows
// too long for nm_spmv): nm_spmm's kernels with the epilogue, in the variants that
// the default plans take.  The gathers of x in shared memory bound them, as nm_spmm:
// 10240 x 8192 at 8 tokens 29.0 us (28.2).
#include "spmm_kernels.cuh"

namespace nmk {

template <int BP>
static cudaError_t launch_bp(const SpmmLinearParams& p, int variant, int grid, cudaStream_t stream, int flags) {
  switch (variant) {
#define NM_SPMM_LINEAR_CASE(i)                                                                   \
  case i:                                                                                        \
    return launch_spmm_t<kSpmmVariants[i][0], kSpmmVariants[i][1], BP, kSpmmVariants[i][2], true>( \
        p, grid, flags, stream);
    NM_SPMM_LINEAR_CASE(0) NM_SPMM_LINEAR_CASE(1) NM_SPMM_LINEAR_CASE(3)
#undef NM_SPMM_LINEAR_CASE
    default: return cudaErrorInvalidValue;
  }
}

cudaError_t launch_spmm_linear(const SpmmLinearParams& p0, const SpmmPlan& plan, int flags,
                               cudaStream_t stream) {
  SpmmLinearParams p = p0;
  p.bps = plan.grid / p.slices;
  // whole pairs in a block where the kernel itself has the epilogue
  const bool by_pairs = p.epi.gated && p.slices == 1;
  const int64_t units = by_pairs ? p.rows / 2 : p.rows;
  p.rows_q = units / p.bps;
  p.rows_r = (int)(units % p.bps);
  p.ystride = (int)((by_pairs ? 2 : 1) * (p.rows_q + 1));
  p.steps_q = p.steps / p.slices;
  p.steps_r = p.steps % p.slices;
  switch (plan.bp) {
    case 2: return launch_bp<2>(p, plan.variant, plan.grid, stream, flags);
    case 4: return launch_bp<4>(p, plan.variant, plan.grid, stream, flags);
    case 6: return launch_bp<6>(p, plan.variant, plan.grid, stream, flags);
    case 8: return launch_bp<8>(p, plan.variant, plan.grid, stream, flags);
    default: return cudaErrorInvalidValue;
  }
}

}  // namespace nmk
