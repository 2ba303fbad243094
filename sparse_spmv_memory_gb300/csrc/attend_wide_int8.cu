// attend_wide_int8.cu -- the many-row attention kernels of int8 caches.
#include "attend_wide.cuh"

namespace nmk {
template cudaError_t launch_attend_wide<kCacheInt8>(const AttendParams&, int, int, cudaStream_t);
template cudaError_t read_attend_wait_timeouts<kCacheInt8>(unsigned long long*, int);
}  // namespace nmk
