// residual_norm.cu -- the residual stream's update by a block's output with the norms
// around it (nm_residual_norm): s = ra r + sc gate post(b), out = pre(s).
//
// A row's elements stay in the registers of its threads from the loads to the
// stores, in fp32, so that every array is read or written once: a row costs
// 2 + 2 bytes an element in and 2 + 2 out (fp16 stream), and the kernel is bound by
// memory.  All of a row's loads are issued before the first sum over the row; a sum
// is a warp butterfly, one shared-memory exchange and another butterfly, and a
// layer norm takes its mean first and then the squares about it.
#include <cuda_fp16.h>
#include <cuda_runtime.h>
#include <stdint.h>

#include "../../include/nm_layer.h"
#include "device.cuh"
#include "kernels.h"
#include "layer.h"

namespace nmk {
namespace {

// V elements at p (16-byte aligned for V = 8) as fp32.
template <int V>
__device__ __forceinline__ void load_elems(const __half* p, float (&x)[V]) {
  if constexpr (V == 8) {
    const uint4 u = *reinterpret_cast<const uint4*>(p);
    const uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const float2 f = half2_bits_to_float2(w[i]);
      x[2 * i] = f.x;
      x[2 * i + 1] = f.y;
    }
  } else {
#pragma unroll
    for (int i = 0; i < V; ++i) x[i] = __half2float(p[i]);
  }
}

template <int V>
__device__ __forceinline__ void load_elems(const float* p, float (&x)[V]) {
  if constexpr (V == 8) {
    const float4 a = *reinterpret_cast<const float4*>(p), b = *reinterpret_cast<const float4*>(p + 4);
    x[0] = a.x; x[1] = a.y; x[2] = a.z; x[3] = a.w;
    x[4] = b.x; x[5] = b.y; x[6] = b.z; x[7] = b.w;
  } else {
#pragma unroll
    for (int i = 0; i < V; ++i) x[i] = p[i];
  }
}

template <int V>
__device__ __forceinline__ void store_elems(__half* p, const float (&x)[V]) {
  if constexpr (V == 8) {
    uint32_t w[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const __half2 h = __floats2half2_rn(x[2 * i], x[2 * i + 1]);
      w[i] = *reinterpret_cast<const uint32_t*>(&h);
    }
    *reinterpret_cast<uint4*>(p) = make_uint4(w[0], w[1], w[2], w[3]);
  } else {
#pragma unroll
    for (int i = 0; i < V; ++i) p[i] = __float2half_rn(x[i]);
  }
}

template <int V>
__device__ __forceinline__ void store_elems(float* p, const float (&x)[V]) {
  if constexpr (V == 8) {
    reinterpret_cast<float4*>(p)[0] = make_float4(x[0], x[1], x[2], x[3]);
    reinterpret_cast<float4*>(p)[1] = make_float4(x[4], x[5], x[6], x[7]);
  } else {
#pragma unroll
    for (int i = 0; i < V; ++i) p[i] = x[i];
  }
}

template <int V>
__device__ __forceinline__ void load_param(const void* p, int fp32, int at, float (&x)[V]) {
  if (fp32)
    load_elems<V>(static_cast<const float*>(p) + at, x);
  else
    load_elems<V>(static_cast<const __half*>(p) + at, x);
}

// Sum over the threads of a row (threadIdx.y's, blockDim.x of them).
struct RowSum {
  float (*part)[32];  // [2][warps of the block]
  int turn = 0;
  __device__ __forceinline__ float operator()(float v) {
    v = warp_sum(v);
    const int warps = blockDim.x >> 5;
    if (warps == 1) return v;
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    float* at = part[turn] + threadIdx.y * warps;
    turn ^= 1;  // the sum after next writes here again, past the next one's barrier
    if (lane == 0) at[warp] = v;
    __syncthreads();
    return warp_sum(lane < warps ? at[lane] : 0.f);
  }
};

// x = norm(x) over the row.
template <int V, int N>
__device__ __forceinline__ void normalise(float (&x)[N][V], const NormArgs& a, int width, RowSum& sum) {
  if (a.kind == NM_NORM_NONE) return;
  const float inv_width = 1.f / (float)width;
  float mean = 0.f;
  if (a.kind == NM_NORM_LAYER) {
    float s = 0.f;
#pragma unroll
    for (int j = 0; j < N; ++j)
#pragma unroll
      for (int i = 0; i < V; ++i) s += x[j][i];
    mean = sum(s) * inv_width;
  }
  float q = 0.f;
#pragma unroll
  for (int j = 0; j < N; ++j) {
    const bool in = ((int)threadIdx.x + j * (int)blockDim.x) * V < width;  // V divides width
#pragma unroll
    for (int i = 0; i < V; ++i) {
      x[j][i] = in ? x[j][i] - mean : 0.f;
      q = fmaf(x[j][i], x[j][i], q);
    }
  }
  const float r = 1.f / sqrtf(sum(q) * inv_width + a.eps);
#pragma unroll
  for (int j = 0; j < N; ++j) {
    const int at = ((int)threadIdx.x + j * (int)blockDim.x) * V;
    if (at >= width) continue;
    float w[V];
    if (a.weight) {
      load_param<V>(a.weight, a.params_fp32, at, w);
#pragma unroll
      for (int i = 0; i < V; ++i) x[j][i] *= r * (a.offset + w[i]);
    } else {
#pragma unroll
      for (int i = 0; i < V; ++i) x[j][i] *= r;
    }
    if (a.bias) {
      load_param<V>(a.bias, a.params_fp32, at, w);
#pragma unroll
      for (int i = 0; i < V; ++i) x[j][i] += w[i];
    }
  }
}

// A row on blockDim.x threads, N groups of V elements each; blockDim.y rows a block.
template <typename S, int V, int N>
__global__ void __launch_bounds__(1024) residual_norm_kernel(const ResidualNormParams p) {
  __shared__ float part[2][32];
  pdl_launch_dependents();
  pdl_wait_previous();
  const int64_t row = (int64_t)blockIdx.x * blockDim.y + threadIdx.y;
  const bool live = row < p.tokens;
  RowSum sum{part};
  float s[N][V], b[N][V];
#pragma unroll
  for (int j = 0; j < N; ++j) {
    const int at = ((int)threadIdx.x + j * (int)blockDim.x) * V;
#pragma unroll
    for (int i = 0; i < V; ++i) s[j][i] = b[j][i] = 0.f;
    if (live && at < p.width) {
      load_elems<V>(static_cast<const S*>(p.residual) + row * p.ldr + at, s[j]);
      if (p.block) load_elems<V>(p.block + row * p.ldb + at, b[j]);
    }
  }
  if (p.block) normalise<V, N>(b, p.post, p.width, sum);
#pragma unroll
  for (int j = 0; j < N; ++j) {
    const int at = ((int)threadIdx.x + j * (int)blockDim.x) * V;
    if (p.block && p.gate && live && at < p.width) {
      float g[V];
      load_elems<V>(p.gate + row * p.ldg + at, g);
#pragma unroll
      for (int i = 0; i < V; ++i) b[j][i] *= g[i];
    }
#pragma unroll
    for (int i = 0; i < V; ++i) {
      s[j][i] *= p.residual_scale;
      if (p.block) s[j][i] = fmaf(p.scale, b[j][i], s[j][i]);
    }
    if (p.stream_out && live && at < p.width)
      store_elems<V>(static_cast<S*>(p.stream_out) + row * p.lds + at, s[j]);
  }
  if (!p.out) return;
  normalise<V, N>(s, p.pre, p.width, sum);
#pragma unroll
  for (int j = 0; j < N; ++j) {
    const int at = ((int)threadIdx.x + j * (int)blockDim.x) * V;
    if (live && at < p.width) store_elems<V>(p.out + row * p.ldo + at, s[j]);
  }
}

bool at16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15) == 0; }

// Whether every row of every array can be taken 8 elements at a time.
bool vectors(const ResidualNormParams& p, int stream_fp32) {
  const int64_t r8 = stream_fp32 ? 4 : 8;  // elements in 16 bytes
  const NormArgs* norms[2] = {&p.post, &p.pre};
  for (const NormArgs* n : norms)
    if (n->kind != NM_NORM_NONE && !(at16(n->weight) && at16(n->bias))) return false;
  return p.width % 8 == 0 && at16(p.residual) && p.ldr % r8 == 0 && at16(p.stream_out) &&
         p.lds % r8 == 0 && at16(p.block) && p.ldb % 8 == 0 && at16(p.gate) && p.ldg % 8 == 0 &&
         at16(p.out) && p.ldo % 8 == 0;
}

template <typename S, int V, int N>
cudaError_t launch_as(const ResidualNormParams& p, int threads, cudaStream_t stream) {
  const int rows = threads >= 256 ? 1 : 256 / threads;
  const int64_t blocks = (p.tokens + rows - 1) / rows;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)blocks);
  cfg.blockDim = dim3((unsigned)threads, (unsigned)rows);
  cfg.stream = stream;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, residual_norm_kernel<S, V, N>, p);
}

template <typename S>
cudaError_t launch_stream(const ResidualNormParams& p, int stream_fp32, cudaStream_t stream) {
  const bool vec = vectors(p, stream_fp32);
  const int groups = vec ? p.width / 8 : p.width;
  const int per = vec ? 4 : 32;  // groups a thread may hold
  int n = 1;
  while ((int64_t)n * 1024 < groups) n *= 2;
  if (n > per) return cudaErrorInvalidValue;
  int threads = ((groups + n - 1) / n + 31) / 32 * 32;
  if (threads < 256)  // whole rows a block: a power of two of warps
    for (int t = 32;; t *= 2)
      if (t >= threads) {
        threads = t;
        break;
      }
  if (vec) {
    switch (n) {
      case 1: return launch_as<S, 8, 1>(p, threads, stream);
      case 2: return launch_as<S, 8, 2>(p, threads, stream);
      default: return launch_as<S, 8, 4>(p, threads, stream);
    }
  }
  switch (n) {
    case 1: return launch_as<S, 1, 1>(p, threads, stream);
    case 2: return launch_as<S, 1, 2>(p, threads, stream);
    case 4: return launch_as<S, 1, 4>(p, threads, stream);
    case 8: return launch_as<S, 1, 8>(p, threads, stream);
    case 16: return launch_as<S, 1, 16>(p, threads, stream);
    default: return launch_as<S, 1, 32>(p, threads, stream);
  }
}

}  // namespace

cudaError_t launch_residual_norm(const ResidualNormParams& p, int stream_fp32, int sms,
                                 cudaStream_t stream) {
  return stream_fp32 ? launch_stream<float>(p, 1, stream) : launch_stream<__half>(p, 0, stream);
}

}  // namespace nmk
