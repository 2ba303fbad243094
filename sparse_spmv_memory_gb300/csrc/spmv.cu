// spmv.cu -- launches of the batch-one N:M bitmask SpMV (spmv_kernels.cuh).
#include <cuda_fp16.h>
#include <cuda_runtime.h>
#include <stdint.h>

#include "kernels.h"
#include "spmv_kernels.cuh"

namespace nmk {

size_t spmv_smem_bytes(int pitch, int nw) {
  return (size_t)(34 * pitch + 6 * nw) * sizeof(float);  // x tile, pf, pl, rinfo
}

template <int NW, int U, int DEC>
static cudaError_t launch_spmv_t(const SpmvParams& p, int grid, int epi, int flags,
                                 cudaStream_t stream) {
  return epi ? launch_spmv_e<NW, U, DEC, 1>(p, grid, flags, stream)
             : launch_spmv_e<NW, U, DEC, 0>(p, grid, flags, stream);
}

// (warps per block, steps in flight per warp, decode).  Every variant runs
// one resident block per SM.  Sweeps on GB300 over the decode-layer shapes put
// variant 6 ahead below ~33M weight positions (more warps hide the decode's
// latencies when each warp has only a few steps), variant 0 up to ~134M and
// variant 1 above; the others stay for tuning and so the tests cover more
// block shapes.  (Blocks sized for two per SM, one or two launched per SM,
// were slower on every shape.)
static const int kSpmvVariants[][3] = {{24, 2, 1}, {20, 3, 2}, {16, 4, 2}, {24, 2, 2},
                                       {24, 2, 3}, {16, 2, 1}, {28, 1, 1}};

int spmv_variant_count() { return (int)(sizeof(kSpmvVariants) / sizeof(kSpmvVariants[0])); }

int spmv_variant_warps(int variant) {
  return (variant >= 0 && variant < spmv_variant_count()) ? kSpmvVariants[variant][0] : 0;
}

cudaError_t launch_spmv(const SpmvParams& p, const SpmvPlan& plan, int flags,
                        cudaStream_t stream, int epilogue) {
  switch (plan.variant) {
#define NM_SPMV_CASE(i)                                                                 \
  case i:                                                                              \
    return launch_spmv_t<kSpmvVariants[i][0], kSpmvVariants[i][1], kSpmvVariants[i][2]>( \
        p, plan.grid, epilogue, flags, stream);
    NM_SPMV_CASE(0) NM_SPMV_CASE(1) NM_SPMV_CASE(2) NM_SPMV_CASE(3) NM_SPMV_CASE(4)
    NM_SPMV_CASE(5) NM_SPMV_CASE(6)
#undef NM_SPMV_CASE
    default: return cudaErrorInvalidValue;
  }
}

}  // namespace nmk
