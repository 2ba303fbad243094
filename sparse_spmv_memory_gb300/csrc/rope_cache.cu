// rope_cache.cu -- rotary positions with the write of keys and values into a
// paged cache (nm_rope_append), and reading its rows back (nm_cache_read).
#include <cuda_fp16.h>
#include <cuda_fp8.h>
#include <cuda_runtime.h>
#include <stdint.h>

#include "decode.h"
#include "device.cuh"
#include "kernels.h"

namespace nmk {
namespace {

__device__ __forceinline__ void unpack8(uint4 u, float (&x)[8]) {
  const uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const float2 f = half2_bits_to_float2(w[i]);
    x[2 * i] = f.x;
    x[2 * i + 1] = f.y;
  }
}

__device__ __forceinline__ uint4 pack8(const float (&x)[8]) {
  uint32_t w[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const __half2 h = __floats2half2_rn(x[2 * i], x[2 * i + 1]);
    w[i] = *reinterpret_cast<const uint32_t*>(&h);
  }
  return make_uint4(w[0], w[1], w[2], w[3]);
}

template <int TYPE>
__device__ __forceinline__ uint2 encode8(const float (&x)[8], float scale) {
  // A row of zeros has scale 0; its codes are 0 / 1.
  const float s = scale > 0.0f ? scale : 1.0f;
  uint32_t b[8];
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    const float y = __fdiv_rn(x[i], s);
    if (TYPE == kCacheE4m3) {
      b[i] = __nv_cvt_float_to_fp8(y, __NV_SATFINITE, __NV_E4M3);
    } else {
      b[i] = (uint32_t)max(-127, min(127, __float2int_rn(y))) & 0xFFu;
    }
  }
  return make_uint2(b[0] | b[1] << 8 | b[2] << 16 | b[3] << 24,
                    b[4] | b[5] << 8 | b[6] << 16 | b[7] << 24);
}

// cos and sin of p * f for a position p, times m.  The product's rounding
// error e (exact by fma) turns the rounded angle's pair by e: at position
// 131071 it reaches 2^-8 of a radian, which would be the largest error by far.
__device__ __forceinline__ void turn_of(float p, float f, float m, float& c, float& s) {
  const float a = __fmul_rn(p, f);
  const float e = __fmaf_rn(p, f, -a);
  float s0, c0;
  sincosf(a, &s0, &c0);
  const float d = 1.0f - 0.5f * e * e;  // |e| <= 2^-7 for p < 2^17: e^4 / 24 is below fp32
  c = m * fmaf(-s0, e, c0 * d);
  s = m * fmaf(c0, e, s0 * d);
}

// A block takes one token and a part of its heads: its first threads put the
// token's cos and sin in shared memory, then groups of D / 8 lanes take a head
// each, 8 elements a lane.
template <int D, int TYPE>
__global__ void __launch_bounds__(256) append_kernel(AppendParams p, int heads_per_block) {
  constexpr int L = D / 8;           // lanes of a head
  __shared__ float sc[D / 2], ss[D / 2];
  pdl_launch_dependents();
  pdl_wait_previous();
  const int t = blockIdx.x;
  const int half = p.rot_dim >> 1;
  const float pos = (float)p.positions[t];
  for (int i = threadIdx.x; i < half; i += blockDim.x) turn_of(pos, p.inv_freq[i], p.mscale, sc[i], ss[i]);
  __syncthreads();
  const int H = p.c.kv_heads;
  const int h_first = p.q_out ? 0 : p.q_heads;
  const int h_end = p.q_heads + 2 * H;
  const int lane = threadIdx.x % L, group = threadIdx.x / L;
  const int64_t slot = p.slots[t];
  const bool keep = slot >= 0 && slot < (p.c.pages << p.c.page_shift);
  const __half* row = p.qkv + (int64_t)t * p.ldqkv;
  const int h0 = h_first + blockIdx.y * heads_per_block;
  const int h1 = min(h0 + heads_per_block, h_end);
  // every group runs the same number of turns: the shuffles need whole warps
  for (int hb = h0; hb < h1; hb += 256 / L) {
    const int h = hb + group;
    const bool on = h < h1 && (h < p.q_heads || keep);
    float x[8];
    uint4 raw = make_uint4(0, 0, 0, 0);
    if (on) raw = ld_keep_v4(row + (int64_t)h * D + lane * 8);
    unpack8(raw, x);
    if (on && h < p.q_heads + H) {
      if (p.interleaved) {
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const int k = lane * 4 + i;
          if (k < half) {
            const float a = x[2 * i], b = x[2 * i + 1];
            x[2 * i] = a * sc[k] - b * ss[k];
            x[2 * i + 1] = b * sc[k] + a * ss[k];
          }
        }
      } else if (lane * 8 < p.rot_dim) {
        float y[8];
        if ((half & 7) == 0) {  // the partners are 8 neighbours too
          const int other = lane * 8 < half ? lane * 8 + half : lane * 8 - half;
          unpack8(ld_keep_v4(row + (int64_t)h * D + other), y);
        } else {
#pragma unroll
          for (int i = 0; i < 8; ++i) {
            const int e = lane * 8 + i;
            y[i] = e < p.rot_dim
                       ? __half2float(row[(int64_t)h * D + (e < half ? e + half : e - half)])
                       : 0.0f;
          }
        }
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          const int e = lane * 8 + i;
          if (e < half)
            x[i] = x[i] * sc[e] - y[i] * ss[e];
          else if (e < p.rot_dim)
            x[i] = x[i] * sc[e - half] + y[i] * ss[e - half];
        }
      }
    }
    // largest magnitude of the row, by its bits: a NaN ranks above infinity
    uint32_t top = 0;
    if (TYPE != kCacheFp16) {
#pragma unroll
      for (int i = 0; i < 8; ++i) top = max(top, __float_as_uint(x[i]) & 0x7FFFFFFFu);
#pragma unroll
      for (int o = L / 2; o > 0; o >>= 1) top = max(top, __shfl_xor_sync(0xFFFFFFFFu, top, o));
    }
    if (!on) continue;
    if (h < p.q_heads) {
      *reinterpret_cast<uint4*>(p.q_out + (int64_t)t * p.ldq + (int64_t)h * D + lane * 8) = pack8(x);
      continue;
    }
    const bool is_v = h >= p.q_heads + H;
    const int kh = h - p.q_heads - (is_v ? H : 0);
    const int64_t page = slot >> p.c.page_shift;
    const int64_t in_page = ((int64_t)kh << p.c.page_shift) + (slot & ((1 << p.c.page_shift) - 1));
    const int64_t at = page * p.c.page_stride + in_page * D + lane * 8;
    uint8_t* dst = is_v ? p.c.v : p.c.k;
    if (TYPE == kCacheFp16) {
      *reinterpret_cast<uint4*>(dst + at * 2) = pack8(x);
    } else {
      const float scale = top >= 0x7F800000u
                              ? __uint_as_float(0x7FC00000u)
                              : __fdiv_rn(__uint_as_float(top), TYPE == kCacheE4m3 ? 448.0f : 127.0f);
      *reinterpret_cast<uint2*>(dst + at) = encode8<TYPE>(x, scale);
      if (lane == 0) (is_v ? p.c.v_scale : p.c.k_scale)[page * p.c.scale_page_stride + in_page] = scale;
    }
  }
}

template <int TYPE>
__device__ __forceinline__ void decode8(const uint8_t* at, float scale, float (&x)[8]) {
  if (TYPE == kCacheFp16) {
    unpack8(ld_stream_v4(at), x);
    return;
  }
  const uint2 u = *reinterpret_cast<const uint2*>(at);
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    const uint32_t b = ((i < 4 ? u.x : u.y) >> (8 * (i & 3))) & 0xFFu;
    if (TYPE == kCacheE4m3) {
      const __half_raw h = __nv_cvt_fp8_to_halfraw((__nv_fp8_storage_t)b, __NV_E4M3);
      x[i] = __half2float(__half(h)) * scale;
    } else {
      x[i] = (float)(int8_t)b * scale;
    }
  }
}

// A thread takes 8 elements of a row.
template <int D, int TYPE>
__global__ void __launch_bounds__(256) read_kernel(ReadParams p) {
  constexpr int L = D / 8;
  pdl_launch_dependents();
  pdl_wait_previous();
  const int64_t n = (int64_t)p.rows * p.c.kv_heads * L;
  const int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x;
  if (i >= n) return;
  const int lane = (int)(i % L);
  const int64_t rh = i / L;
  const int h = (int)(rh % p.c.kv_heads);
  const int64_t slot = p.slots[rh / p.c.kv_heads];
  const bool is_v = blockIdx.y != 0;
  __half* out = is_v ? p.v_out : p.k_out;
  if (!out) return;
  float x[8] = {0, 0, 0, 0, 0, 0, 0, 0};
  if (slot >= 0 && slot < (p.c.pages << p.c.page_shift)) {
    const int64_t page = slot >> p.c.page_shift;
    const int64_t in_page = ((int64_t)h << p.c.page_shift) + (slot & ((1 << p.c.page_shift) - 1));
    const float scale = TYPE == kCacheFp16 ? 1.0f
                                           : (is_v ? p.c.v_scale : p.c.k_scale)
                                                 [page * p.c.scale_page_stride + in_page];
    const int64_t at = page * p.c.page_stride + in_page * D + lane * 8;
    decode8<TYPE>((is_v ? p.c.v : p.c.k) + at * (TYPE == kCacheFp16 ? 2 : 1), scale, x);
  }
  *reinterpret_cast<uint4*>(out + i * 8) = pack8(x);
}

}  // namespace

template <int D, int TYPE>
static cudaError_t append_one(const AppendParams& p, int sms, cudaStream_t stream) {
  const int heads = (p.q_out ? p.q_heads : 0) + 2 * p.c.kv_heads;
  constexpr int kPer = 256 / (D / 8);  // heads a block takes at a time
  // Few tokens: a block per turn of heads; many: a block walks a token's heads.
  const int turns = (heads + kPer - 1) / kPer;
  int parts = turns;
  while (parts > 1 && (int64_t)p.tokens * parts > 8 * sms) parts = (parts + 1) / 2;
  const int per = (turns + parts - 1) / parts * kPer;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)p.tokens, (unsigned)((heads + per - 1) / per));
  cfg.blockDim = dim3(256);
  cfg.stream = stream;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, append_kernel<D, TYPE>, p, per);
}

cudaError_t launch_rope_append(const AppendParams& p, int head_dim, int type, int sms,
                               cudaStream_t stream) {
  if (head_dim == 128) {
    if (type == kCacheFp16) return append_one<128, kCacheFp16>(p, sms, stream);
    if (type == kCacheE4m3) return append_one<128, kCacheE4m3>(p, sms, stream);
    return append_one<128, kCacheInt8>(p, sms, stream);
  }
  if (type == kCacheFp16) return append_one<64, kCacheFp16>(p, sms, stream);
  if (type == kCacheE4m3) return append_one<64, kCacheE4m3>(p, sms, stream);
  return append_one<64, kCacheInt8>(p, sms, stream);
}

template <int D, int TYPE>
static cudaError_t read_one(const ReadParams& p, cudaStream_t stream) {
  const int64_t n = (int64_t)p.rows * p.c.kv_heads * (D / 8);
  const int64_t blocks = (n + 255) / 256;
  if (blocks > 0x7FFFFFFF) return cudaErrorInvalidValue;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)blocks, 2);
  cfg.blockDim = dim3(256);
  cfg.stream = stream;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, read_kernel<D, TYPE>, p);
}

cudaError_t launch_cache_read(const ReadParams& p, int head_dim, int type, cudaStream_t stream) {
  if (head_dim == 128) {
    if (type == kCacheFp16) return read_one<128, kCacheFp16>(p, stream);
    if (type == kCacheE4m3) return read_one<128, kCacheE4m3>(p, stream);
    return read_one<128, kCacheInt8>(p, stream);
  }
  if (type == kCacheFp16) return read_one<64, kCacheFp16>(p, stream);
  if (type == kCacheE4m3) return read_one<64, kCacheE4m3>(p, stream);
  return read_one<64, kCacheInt8>(p, stream);
}

}  // namespace nmk
