// prefill.cu -- the prefill products' plan, launches and the K split's combine; the
// kernel is in prefill_kernels.cuh.
#include <cuda_fp16.h>
#include <cuda_runtime.h>
#include <stdint.h>

#include "kernels.h"
#include "prefill_kernels.cuh"

namespace nmk {
namespace tc {

// One entry a kernel variant; the stage counts are the deepest that fit 227 KB of
// shared memory (4 for the first 512-token variant, kept as the shallower
// alternative).
struct Variant {
  int nmma, nb, stages, g, dg, dw, ms;
};
constexpr Variant kVariants[] = {{256, 2, 4, 1, 2, 16, 0},  {256, 1, 7, 1, 2, 16, 1},
                                 {128, 1, 10, 1, 4, 16, 1}, {64, 1, 12, 1, 4, 16, 1},
                                 {256, 2, 5, 1, 4, 16, 0}};
constexpr int kVariantCount = sizeof(kVariants) / sizeof(kVariants[0]);

// Y[t][r] = fp16(sum over slices z, in increasing z, of part[z][t][r]): the
// K split's fixed-order combine (one rounding, no atomics).  V = 4: each
// thread takes four consecutive rows (16-byte loads, one 8-byte store), and
// issues the slices' loads four at a time; the additions keep slice order.
__device__ __forceinline__ float4 add4(float4 a, float4 b) {
  return make_float4(a.x + b.x, a.y + b.y, a.z + b.z, a.w + b.w);
}

template <int V>
__global__ void __launch_bounds__(256) splitk_sum_kernel(const float* __restrict__ part,
                                                         int slices, int64_t T, int64_t rows,
                                                         __half* __restrict__ Y, int64_t ldy) {
  const int64_t plane = T * rows;
  for (int64_t t = blockIdx.y; t < T; t += gridDim.y) {
    for (int64_t r = ((int64_t)blockIdx.x * blockDim.x + threadIdx.x) * V; r < rows;
         r += (int64_t)gridDim.x * blockDim.x * V) {
      const float* q = part + t * rows + r;
      if (V == 4) {
        float4 acc = *reinterpret_cast<const float4*>(q);
        int z = 1;
        for (; z + 3 < slices; z += 4) {
          const float4 a = *reinterpret_cast<const float4*>(q + z * plane);
          const float4 b = *reinterpret_cast<const float4*>(q + (z + 1) * plane);
          const float4 c = *reinterpret_cast<const float4*>(q + (z + 2) * plane);
          const float4 d = *reinterpret_cast<const float4*>(q + (z + 3) * plane);
          acc = add4(add4(add4(add4(acc, a), b), c), d);
        }
        for (; z < slices; ++z) acc = add4(acc, *reinterpret_cast<const float4*>(q + z * plane));
        const __half2 lo = __floats2half2_rn(acc.x, acc.y), hi = __floats2half2_rn(acc.z, acc.w);
        uint2 w;
        w.x = *reinterpret_cast<const uint32_t*>(&lo);
        w.y = *reinterpret_cast<const uint32_t*>(&hi);
        *reinterpret_cast<uint2*>(Y + t * ldy + r) = w;
      } else {
        float acc = q[0];
        for (int z = 1; z < slices; ++z) acc += q[z * plane];
        Y[t * ldy + r] = __float2half_rn(acc);
      }
    }
  }
}

static cudaError_t launch_splitk_sum(const SpmmTcParams& p, cudaStream_t stream) {
  // Four rows a thread when every row group of Y is 8-byte aligned (the
  // partial planes then are 16-byte aligned: the workspace is).
  const bool v4 = p.rows % 4 == 0 && p.ldy % 4 == 0 &&
                  (reinterpret_cast<uintptr_t>(p.Y) & 7) == 0;
  const int64_t per_block = v4 ? 1024 : 256;
  const int64_t bx = (p.rows + per_block - 1) / per_block;
  const dim3 grid((unsigned)(bx < 65535 ? bx : 65535), (unsigned)(p.T < 65535 ? p.T : 65535));
  if (v4)
    splitk_sum_kernel<4><<<grid, 256, 0, stream>>>(p.part, p.slices, p.T, p.rows, p.Y, p.ldy);
  else
    splitk_sum_kernel<1><<<grid, 256, 0, stream>>>(p.part, p.slices, p.T, p.rows, p.Y, p.ldy);
  return cudaGetLastError();
}

}  // namespace tc

int spmm_tc_variant_count() { return tc::kVariantCount; }

// Words per K slice when a row of `words` mask words is cut into at most
// `splits` slices: a multiple of four (one mask box), so every slice but the
// last is whole boxes.  The slice count is then ceil(words / slice).
int spmm_tc_slice_words(int words, int splits) {
  if (splits <= 1 || words <= 4) return words;
  const int w = (words + splits - 1) / splits;
  const int r = (w + 3) / 4 * 4;
  return r < words ? r : words;
}

int spmm_tc_slices(int words, int splits) {
  const int w = spmm_tc_slice_words(words, splits);
  return (words + w - 1) / w;
}

size_t spmm_tc_workspace_bytes(int64_t rows, int words, int64_t T, int splits) {
  const int z = spmm_tc_slices(words, splits);
  return z > 1 ? (size_t)z * (size_t)T * (size_t)rows * sizeof(float) : 0;
}

// Time model of a plan (variant, K slices), in ns: waves of blocks x (the
// slice's stages x the variant's time per 32-column stage + a block's fixed
// cost + its output stores: fp16 Y, or fp32 sums when split), plus, when
// split, the combine (a launch and its traffic).  Times per stage measured on
// GB300 over the decoder-layer shapes, one block per SM: 512 tokens 441 (5
// stages), 256 tokens 319 (7), 128 tokens 232 (10), 64 tokens 218 (12).  The
// other constants were fitted to a sweep of every (variant, 1..8 slices) over
// eight decoder matrices (4096..57344 rows, 4096..28672 columns) at 16, 64,
// 256, 512 and 2048 tokens, on which the model picks the fastest plan in
// every case.  A larger token tile does more work per stage; a smaller one,
// or a K split, fills more SMs when rows (or tokens) are few.
namespace {
struct Cand {
  int variant, tokens;
  double ns_per_stage;
};
constexpr Cand kCand[] = {{4, 512, 441.0}, {1, 256, 319.0}, {2, 128, 232.0}, {3, 64, 218.0}};
constexpr double kBlockNs = 3000.0;        // prologue, pipeline fill, teardown
constexpr double kStoreBytesPerNs = 80.0;  // one block's output stores (per SM)
constexpr double kCombineNs = 2500.0;      // the combine kernel's launch and ramp
constexpr double kCombineBytesPerNs = 8000.0;  // partial sums written, read; Y written
constexpr size_t kMaxSplitBytes = (size_t)256 << 20;

double plan_ns(const Cand& c, int64_t rows, int words, int64_t T, int sms, int splits) {
  const int64_t tiles = ((rows + 127) / 128) * ((T + c.tokens - 1) / c.tokens);
  const int z = spmm_tc_slices(words, splits);
  const int64_t waves = (tiles * z + sms - 1) / sms;
  const double out_bytes = (double)c.tokens * 128.0 * (z > 1 ? 4.0 : 2.0);
  double t = (double)waves * (spmm_tc_slice_words(words, splits) * c.ns_per_stage + kBlockNs +
                              out_bytes / kStoreBytesPerNs);
  if (z > 1)
    t += kCombineNs + (double)(4 * z + 4 * z + 2) * (double)T * (double)rows / kCombineBytesPerNs;
  return t;
}
}  // namespace

// The plan of least modelled time.  variant >= 0 fixes the variant; splits
// >= 1 fixes the slice request (1: no split); max_splits bounds the search.
void spmm_tc_default_plan(int64_t rows, int words, int64_t T, int sms, int variant, int splits,
                          int max_splits, int* variant_out, int* splits_out) {
  if (sms < 1) sms = 1;
  int best_v = variant >= 0 ? variant : 3, best_z = 1;
  double best_t = 0.0;
  for (const auto& c : kCand) {
    if (variant >= 0 && c.variant != variant) continue;
    const int lo = splits >= 1 ? splits : 1, hi = splits >= 1 ? splits : max_splits;
    for (int z = lo; z <= hi; ++z) {
      if (z > 1 && (spmm_tc_slices(words, z) != z ||
                    spmm_tc_workspace_bytes(rows, words, T, z) > kMaxSplitBytes))
        continue;
      const double t = plan_ns(c, rows, words, T, sms, z);
      if (best_t == 0.0 || t < best_t * 0.97) {  // prefer the earlier (larger tile, fewer slices)
        best_v = c.variant;
        best_z = z;
        best_t = t;
      }
    }
  }
  if (variant >= 0 && best_t == 0.0) best_z = splits >= 1 ? splits : 1;  // variant 0: not modelled
  *variant_out = best_v;
  *splits_out = best_z;
}

int spmm_tc_default_variant(int64_t rows, int64_t T, int sms) {
  int v, z;
  spmm_tc_default_plan(rows, 32, T, sms, -1, 1, 1, &v, &z);
  return v;
}

int spmm_tc_block_tokens(int variant) {
  return tc::kVariants[variant].nmma * tc::kVariants[variant].nb;
}

static cudaError_t launch_spmm_tc_main(const SpmmTcParams& p, int variant, cudaStream_t stream) {
  switch (variant) {
    case 0: return tc::launch_tc<256, 2, 4, 1, 2, 16, 0, false>(p, stream);
    case 1: return tc::launch_tc<256, 1, 7, 1, 2, 16, 1, false>(p, stream);
    case 2: return tc::launch_tc<128, 1, 10, 1, 4, 16, 1, false>(p, stream);
    case 3: return tc::launch_tc<64, 1, 12, 1, 4, 16, 1, false>(p, stream);
    case 4: return tc::launch_tc<256, 2, 5, 1, 4, 16, 0, false>(p, stream);
    default: return cudaErrorInvalidValue;
  }
}

cudaError_t launch_spmm_tc(const SpmmTcParams& p, int variant, cudaStream_t stream) {
  cudaError_t e = launch_spmm_tc_main(p, variant, stream);
  if (e != cudaSuccess || p.slices <= 1) return e;
  return tc::launch_splitk_sum(p, stream);
}

cudaError_t read_wait_timeouts(unsigned long long* count, int reset) {
  return read_local_wait_timeouts(count, reset);
}

}  // namespace nmk
