// residual_norm.cu -- the residual stream's update by a block's output with the norms
// around it (nm_residual_norm): s = ra r + sc gate post(b), out = pre(s).
//
// A row's elements stay in the registers of its threads from the loads to the
// stores, so that every array is read or written once: a row costs 2 + 2 bytes an
// element in and 2 + 2 out (fp16 stream), and memory bounds it.  What it costs
// besides is instructions: a sum over the row is a warp butterfly, a shared-memory
// exchange and another butterfly for every thread, so a thread takes 32 elements of
// an fp16 stream (N = 4 groups of 8) where there are rows enough to fill the SMs,
// and 8 where there are few and the time to the result counts.  (4096 rows of 8192
// with 8 elements a thread: 100 us, 58 % of the issue slots.)  A layer norm takes its
// mean first and then the squares about it.
//
// Groups are the 16-byte pieces of the stream's row (8 elements; 32 bytes of an fp32
// stream): a row that starts inside one, or ends inside one, has its ends moved
// element by element and everything else by whole vectors, as has every other array
// whose row starts at the same place in a piece (rows of an odd width, all alike);
// arrays that do not are read and written element by element.
#include <cuda_fp16.h>
#include <cuda_runtime.h>
#include <stdint.h>

#include "../../include/nm_layer.h"
#include "device.cuh"
#include "kernels.h"
#include "layer.h"

namespace nmk {
namespace {

template <typename S>
struct Raw {  // 8 elements as they lie in memory
  uint32_t w[2 * sizeof(S)];
};

__device__ __forceinline__ void widen(const Raw<__half>& q, float (&x)[8]) {
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const float2 f = half2_bits_to_float2(q.w[i]);
    x[2 * i] = f.x;
    x[2 * i + 1] = f.y;
  }
}

__device__ __forceinline__ void widen(const Raw<float>& q, float (&x)[8]) {
#pragma unroll
  for (int i = 0; i < 8; ++i) x[i] = __uint_as_float(q.w[i]);
}

__device__ __forceinline__ Raw<__half> narrow(const float (&x)[8], __half) {
  Raw<__half> q;
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const __half2 h = __floats2half2_rn(x[2 * i], x[2 * i + 1]);
    q.w[i] = *reinterpret_cast<const uint32_t*>(&h);
  }
  return q;
}

__device__ __forceinline__ Raw<float> narrow(const float (&x)[8], float) {
  Raw<float> q;
#pragma unroll
  for (int i = 0; i < 8; ++i) q.w[i] = __float_as_uint(x[i]);
  return q;
}

__device__ __forceinline__ uint32_t bits(__half h) { return __half_as_ushort(h); }

// A row of an array and how its groups are read: group elements at .. at + 7, by
// vectors where the row's pieces are the stream's (vec) and all 8 are in the row.
template <typename S, bool WHOLE>
struct Line {
  S* row;
  bool vec;
  int width;

  __device__ __forceinline__ bool whole(int at) const {
    return WHOLE || (vec && at >= 0 && at + 8 <= width);
  }

  __device__ __forceinline__ Raw<S> load(int at) const {
    Raw<S> q;
    if (whole(at)) {
#pragma unroll
      for (int i = 0; i < (int)sizeof(S) / 2; ++i) {
        const uint4 u = reinterpret_cast<const uint4*>(row + at)[i];
        q.w[4 * i] = u.x;
        q.w[4 * i + 1] = u.y;
        q.w[4 * i + 2] = u.z;
        q.w[4 * i + 3] = u.w;
      }
    } else {
#pragma unroll
      for (int i = 0; i < 2 * (int)sizeof(S); ++i) q.w[i] = 0u;
#pragma unroll
      for (int i = 0; i < 8; ++i)
        if (at + i >= 0 && at + i < width) {
          if constexpr (sizeof(S) == 2)
            q.w[i / 2] |= bits(row[at + i]) << (16 * (i & 1));
          else
            q.w[i] = __float_as_uint(row[at + i]);
        }
    }
    return q;
  }

  __device__ __forceinline__ void store(int at, const float (&x)[8]) const {
    const Raw<S> q = narrow(x, S());
    if (whole(at)) {
#pragma unroll
      for (int i = 0; i < (int)sizeof(S) / 2; ++i)
        reinterpret_cast<uint4*>(row + at)[i] =
            make_uint4(q.w[4 * i], q.w[4 * i + 1], q.w[4 * i + 2], q.w[4 * i + 3]);
    } else {
#pragma unroll
      for (int i = 0; i < 8; ++i)
        if (at + i >= 0 && at + i < width) {
          if constexpr (sizeof(S) == 2)
            row[at + i] = __ushort_as_half((unsigned short)(q.w[i / 2] >> (16 * (i & 1))));
          else
            row[at + i] = __uint_as_float(q.w[i]);
        }
    }
  }
};

// Where in its 8-element piece an address lies, and whether a row whose groups begin
// `shift` elements into a piece can be taken by vectors of 16 bytes.
template <typename S>
__device__ __forceinline__ int place(const void* p) {
  return (int)(reinterpret_cast<uintptr_t>(p) / sizeof(S)) & 7;
}

template <typename S, bool WHOLE>
__device__ __forceinline__ Line<S, WHOLE> line(const void* base, int64_t offset, int shift, int width) {
  S* row = static_cast<S*>(const_cast<void*>(base)) + offset;
  return {row, ((place<S>(row) - shift) & (16 / (int)sizeof(S) - 1)) == 0, width};
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
    if (warps <= 8) {
      v = (lane & 7) < warps ? at[lane & 7] : 0.f;
#pragma unroll
      for (int o = 4; o > 0; o >>= 1) v += __shfl_xor_sync(0xFFFFFFFFu, v, o);
      return v;
    }
    return warp_sum(lane < warps ? at[lane] : 0.f);
  }
};

// x times a norm's weight plus its bias, at a group.
template <bool WHOLE, typename P>
__device__ __forceinline__ void scaled(float (&x)[8], float r, const NormArgs& a, int at, int shift, int width) {
  float w[8];
  if (a.weight) {
    widen(line<P, WHOLE>(a.weight, 0, shift, width).load(at), w);
#pragma unroll
    for (int i = 0; i < 8; ++i) x[i] *= r * (a.offset + w[i]);
  } else {
#pragma unroll
    for (int i = 0; i < 8; ++i) x[i] *= r;
  }
  if (a.bias) {
    widen(line<P, WHOLE>(a.bias, 0, shift, width).load(at), w);
#pragma unroll
    for (int i = 0; i < 8; ++i) x[i] += w[i];
  }
}

// The mean (0 but for a layer norm) and 1 / sqrt(mean square about it + eps) of a
// row; get(j, x) gives group j's elements, whatever outside the row.
template <bool WHOLE, int N, typename Get>
__device__ __forceinline__ float2 moments(const NormArgs& a, int width, int shift, RowSum& sum, Get&& get) {
  const float inv_width = 1.f / (float)width;
  auto outside = [&](int j, int i) {
    const int at = 8 * ((int)threadIdx.x + j * (int)blockDim.x) - shift;
    return WHOLE ? at >= width : at + i < 0 || at + i >= width;
  };
  float mean = 0.f;
  if (a.kind == NM_NORM_LAYER) {
    float s = 0.f;
#pragma unroll
    for (int j = 0; j < N; ++j) {
      float x[8];
      get(j, x);
#pragma unroll
      for (int i = 0; i < 8; ++i) s += outside(j, i) ? 0.f : x[i];
    }
    mean = sum(s) * inv_width;
  }
  float q = 0.f;
#pragma unroll
  for (int j = 0; j < N; ++j) {
    float x[8];
    get(j, x);
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const float d = outside(j, i) ? 0.f : x[i] - mean;
      q = fmaf(d, d, q);
    }
  }
  return {mean, 1.f / sqrtf(sum(q) * inv_width + a.eps)};
}

// A row on blockDim.x threads, N groups a thread; blockDim.y rows a block.  WHOLE: all
// rows of all arrays are whole 16-byte pieces.
template <typename S, int N, bool WHOLE>
__global__ void __launch_bounds__(1024) residual_norm_kernel(const ResidualNormParams p) {
  __shared__ float part[2][32];
  pdl_launch_dependents();
  pdl_wait_previous();
  const int64_t row = (int64_t)blockIdx.x * blockDim.y + threadIdx.y;
  const bool live = row < p.tokens;
  const int width = p.width;
  RowSum sum{part};
  const int shift = WHOLE ? 0 : place<S>(static_cast<const S*>(p.residual) + row * p.ldr);
  auto at = [&](int j) { return 8 * ((int)threadIdx.x + j * (int)blockDim.x) - shift; };
  auto mine = [&](int j) { return live && at(j) < width; };
  const Line<__half, WHOLE> gate = line<__half, WHOLE>(p.gate, row * p.ldg, shift, width);

  Raw<S> r[N];
  Raw<__half> b[N];
#pragma unroll
  for (int j = 0; j < N; ++j) {
    r[j] = Raw<S>{};
    b[j] = Raw<__half>{};
  }
  if (p.block) {
    const Line<__half, WHOLE> from = line<__half, WHOLE>(p.block, row * p.ldb, shift, width);
#pragma unroll
    for (int j = 0; j < N; ++j)
      if (mine(j)) b[j] = from.load(at(j));
  }
  {
    const Line<S, WHOLE> from = line<S, WHOLE>(p.residual, row * p.ldr, shift, width);
#pragma unroll
    for (int j = 0; j < N; ++j)
      if (mine(j)) r[j] = from.load(at(j));
  }
  if (p.block && p.gate && p.ldg != 0) {  // a token's own gate is on its way meanwhile
#pragma unroll
    for (int j = 0; j < N; ++j)
      if (mine(j)) asm volatile("prefetch.global.L2 [%0];" ::"l"(gate.row + max(at(j), 0)));
  }

  float2 post = {0.f, 1.f};
  if (p.block && p.post.kind != NM_NORM_NONE)
    post = moments<WHOLE, N>(p.post, width, shift, sum, [&](int j, float (&x)[8]) { widen(b[j], x); });
  float s[N][8];
  const Line<S, WHOLE> to = line<S, WHOLE>(p.stream_out, row * p.lds, shift, width);
#pragma unroll
  for (int j = 0; j < N; ++j) {
    widen(r[j], s[j]);
#pragma unroll
    for (int i = 0; i < 8; ++i) s[j][i] *= p.residual_scale;
    if (!mine(j)) continue;
    if (p.block) {
      float x[8];
      widen(b[j], x);
      if (p.post.kind != NM_NORM_NONE) {
#pragma unroll
        for (int i = 0; i < 8; ++i) x[i] -= post.x;
        if (p.post.params_fp32)
          scaled<WHOLE, float>(x, post.y, p.post, at(j), shift, width);
        else
          scaled<WHOLE, __half>(x, post.y, p.post, at(j), shift, width);
      }
      if (p.gate) {
        float g[8];
        widen(gate.load(at(j)), g);
#pragma unroll
        for (int i = 0; i < 8; ++i) x[i] *= g[i];
      }
#pragma unroll
      for (int i = 0; i < 8; ++i) s[j][i] = fmaf(p.scale, x[i], s[j][i]);
    }
    if (p.stream_out) to.store(at(j), s[j]);
  }
  if (!p.out) return;

  float2 pre = {0.f, 1.f};
  if (p.pre.kind != NM_NORM_NONE)
    pre = moments<WHOLE, N>(p.pre, width, shift, sum, [&](int j, float (&x)[8]) {
#pragma unroll
      for (int i = 0; i < 8; ++i) x[i] = s[j][i];
    });
  const Line<__half, WHOLE> out = line<__half, WHOLE>(p.out, row * p.ldo, shift, width);
#pragma unroll
  for (int j = 0; j < N; ++j) {
    if (!mine(j)) continue;
    if (p.pre.kind != NM_NORM_NONE) {
#pragma unroll
      for (int i = 0; i < 8; ++i) s[j][i] -= pre.x;
      if (p.pre.params_fp32)
        scaled<WHOLE, float>(s[j], pre.y, p.pre, at(j), shift, width);
      else
        scaled<WHOLE, __half>(s[j], pre.y, p.pre, at(j), shift, width);
    }
    out.store(at(j), s[j]);
  }
}

bool at16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15) == 0; }

// Whether every row of every array is whole 16-byte pieces.
template <typename S>
bool whole_rows(const ResidualNormParams& p) {
  const int64_t r = 16 / sizeof(S);  // elements of the stream in a piece of 16 bytes
  const NormArgs* norms[2] = {&p.post, &p.pre};
  for (const NormArgs* n : norms)
    if (!at16(n->weight) || !at16(n->bias)) return false;
  return p.width % 8 == 0 && at16(p.residual) && p.ldr % r == 0 && at16(p.stream_out) &&
         p.lds % r == 0 && at16(p.block) && p.ldb % 8 == 0 && at16(p.gate) && p.ldg % 8 == 0 &&
         at16(p.out) && p.ldo % 8 == 0;
}

template <typename S, int N, bool WHOLE>
cudaError_t launch_as(const ResidualNormParams& p, int groups, cudaStream_t stream) {
  int threads = ((groups + N - 1) / N + 31) / 32 * 32;
  if (threads < 256) {  // whole rows a block: a power of two of warps each
    int t = 32;
    while (t < threads) t *= 2;
    threads = t;
  }
  const int rows = threads >= 256 ? 1 : 256 / threads;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)((p.tokens + rows - 1) / rows));
  cfg.blockDim = dim3((unsigned)threads, (unsigned)rows);
  cfg.stream = stream;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, residual_norm_kernel<S, N, WHOLE>, p);
}

template <typename S, bool WHOLE>
cudaError_t launch_n(const ResidualNormParams& p, int sms, cudaStream_t stream) {
  const int groups = WHOLE ? p.width / 8 : (p.width + 14) / 8;  // with a start anywhere in a piece
  // the fewest a thread while the rows' threads fit the SMs at once
  const int most = sizeof(S) == 2 ? 4 : 2;
  int n = 1;
  while (n < 4 && ((groups + n - 1) / n > 1024 || (n < most && p.tokens * ((groups + n - 1) / n) > (int64_t)sms * 1024)))
    n *= 2;
  if constexpr (!WHOLE)
    if (groups > 4096) return launch_as<S, 5, WHOLE>(p, groups, stream);  // 32768 and a start inside a piece
  switch (n) {
    case 1: return launch_as<S, 1, WHOLE>(p, groups, stream);
    case 2: return launch_as<S, 2, WHOLE>(p, groups, stream);
    default: return launch_as<S, 4, WHOLE>(p, groups, stream);
  }
}

template <typename S>
cudaError_t launch_stream(const ResidualNormParams& p, int sms, cudaStream_t stream) {
  return whole_rows<S>(p) ? launch_n<S, true>(p, sms, stream) : launch_n<S, false>(p, sms, stream);
}

}  // namespace

cudaError_t launch_residual_norm(const ResidualNormParams& p, int stream_fp32, int sms,
                                 cudaStream_t stream) {
  return stream_fp32 ? launch_stream<float>(p, sms, stream) : launch_stream<__half>(p, sms, stream);
}

}  // namespace nmk
