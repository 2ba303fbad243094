// attend_wide_fp16.cu -- the many-row attention kernels of fp16 caches.
#include "attend_wide.cuh"

namespace nmk {
template cudaError_t launch_attend_wide<kCacheFp16>(const AttendParams&, int, int, cudaStream_t);
template cudaError_t read_attend_wait_timeouts<kCacheFp16>(unsigned long long*, int);
}  // namespace nmk
