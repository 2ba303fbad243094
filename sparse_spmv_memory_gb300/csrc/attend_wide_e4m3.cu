// attend_wide_e4m3.cu -- the many-row attention kernels of e4m3 caches.
#include "attend_wide.cuh"

namespace nmk {
template cudaError_t launch_attend_wide<kCacheE4m3>(const AttendParams&, int, int, cudaStream_t);
template cudaError_t read_attend_wait_timeouts<kCacheE4m3>(unsigned long long*, int);
}  // namespace nmk
