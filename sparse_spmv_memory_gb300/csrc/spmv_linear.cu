// spmv_linear.cu -- nm_linear's one-token products: nm_spmv's kernels with the
// general epilogue, in the variants that the default plans take.  HBM bounds them:
// 57344 x 8192 gated 78 to 80 us (the product alone 77 to 79), 4096 x 4096 with a
// residual 5.4 to 5.9 (4.9: the sums go through shared memory once more).
#include <cuda_fp16.h>
#include <cuda_runtime.h>
#include <stdint.h>

#include "kernels.h"
#include "spmv_kernels.cuh"

namespace nmk {

cudaError_t launch_spmv_linear(const SpmvParams& p, const SpmvPlan& plan, int flags,
                               cudaStream_t stream) {
  switch (plan.variant) {  // as in kSpmvVariants (spmv.cu)
    case 0: return launch_spmv_e<24, 2, 1, 2>(p, plan.grid, flags, stream);
    case 1: return launch_spmv_e<20, 3, 2, 2>(p, plan.grid, flags, stream);
    case 6: return launch_spmv_e<28, 1, 1, 2>(p, plan.grid, flags, stream);
    default: return cudaErrorInvalidValue;
  }
}

}  // namespace nmk
