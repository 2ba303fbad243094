// rope_cache.cu -- rotary positions with the write of keys and values into a
// paged cache (nm_rope_append), and reading its rows back (nm_cache_read).
#include <cuda_fp16.h>
#include <cuda_fp8.h>
#include <cuda_runtime.h>
#include <stdint.h>

#include "decode.h"
#include "device.cuh"
#include "kernels.h"
#include "widen.cuh"

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

// cos and sin of pos * f, times m.  The product's rounding error e (exact by fma)
// turns the rounded angle's pair by e: at position 131071 and f = 1 it reaches 2^-8
// of a radian, which would be the largest error by far.
__device__ __forceinline__ void turn_of(int pos, float f, float m, float& c, float& s) {
  const float p = (float)pos;
  const float a = __fmul_rn(p, f);
  float e = __fmaf_rn(p, f, -a);
  float s0, c0;
  sincosf(a, &s0, &c0);
  if (fabsf(e) > 0.0078125f || (uint32_t)pos + (1u << 24) > (2u << 24)) {
    // Far positions: e is an angle of its own, and above 2^24 the position's rounding
    // times f joins it.  The sum's two parts: the first turns by its cosine and sine,
    // the second (2^-16 for f of 1) is the new e.
    const float rest = (float)(int)((int64_t)pos - (int64_t)p);
    const float h = __fmul_rn(rest, f), l = __fmaf_rn(rest, f, -h);
    const float t = __fadd_rn(e, h), b = __fsub_rn(t, e);
    e = __fadd_rn(__fadd_rn(__fsub_rn(e, __fsub_rn(t, b)), __fsub_rn(h, b)), l);
    float s1, c1;
    sincosf(t, &s1, &c1);
    const float c2 = c0 * c1 - s0 * s1;
    s0 = s0 * c1 + c0 * s1;
    c0 = c2;
  }
  const float d = 1.0f - 0.5f * e * e;  // |e| <= 2^-7: e^3 / 6 is 2^-23.6, below fp32
  c = m * fmaf(-s0, e, c0 * d);
  s = m * fmaf(c0, e, s0 * d);
}

// A warp takes one token and 32 / (D / 8) heads at a time, 8 elements a lane, up
// to `turns` times.  Its lanes compute the token's cos and sin once, two angles
// each, and hand them round by shuffles; a pair's other half comes from the lane
// that has it.  No shared memory, no barrier, the next turn's load in flight.
// What bounds it: latency for few tokens (one token of 48 heads 1.8 us in a graph),
// for many the issue of angles, shuffles and conversions, 2.5 instructions a clock,
// and the waits between slot, position, frequencies and row (512 tokens of 80 heads
// to e4m3 6.5 us with its inputs in L2, 8.5 from HBM, where its bytes take 3).
template <int D, int TYPE>
__global__ void __launch_bounds__(128) append_kernel(AppendParams p, int turns) {
  constexpr int L = D / 8, HEADS = 32 / L;  // lanes of a head, heads of a turn
  pdl_launch_dependents();
  pdl_wait_previous();
  const int t = blockIdx.x;
  const int lane = threadIdx.x & 31, in = lane % L;
  const int half = p.rot_dim >> 1, H = p.c.kv_heads;
  const int h_end = p.q_heads + 2 * H;
  const int step = HEADS * 4 * gridDim.y;  // heads of a turn of all the token's warps
  const int hw = (p.q_out ? 0 : p.q_heads) + (blockIdx.y * 4 + (threadIdx.x >> 5)) * HEADS;
  if (hw >= h_end) return;  // the whole warp
  const __half* row = p.qkv + (int64_t)t * p.ldqkv;
  auto load = [&](int h) { return h < h_end ? ld_keep_v4(row + h * D + in * 8) : make_uint4(0, 0, 0, 0); };
  uint4 raw = load(hw + lane / L);
  const int64_t slot = p.slots[t];
  const bool keep = slot >= 0 && slot < (p.c.pages << p.c.page_shift);
  const int64_t page = slot >> p.c.page_shift, off = slot & ((1 << p.c.page_shift) - 1);

  // angles 2 lane and 2 lane + 1, and from them the lane's own
  float ac[2] = {1.0f, 1.0f}, as[2] = {0.0f, 0.0f}, c[8], s[8];
  const int pos = p.positions[t];
#pragma unroll
  for (int k = 0; k < 2; ++k)
    if (2 * lane + k < half) turn_of(pos, p.inv_freq[2 * lane + k], p.mscale, ac[k], as[k]);
  const bool vec = (half & 7) == 0, turned = in * 8 < p.rot_dim;
  const bool upper = in * 8 >= half;       // vec: the second of the pairs
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    // the angle of element i (interleaved: of elements 2i, 2i + 1 for i < 4)
    const int e = in * 8 + i;
    const int a = p.interleaved ? in * 4 + (i & 3) : e < half ? e : e - half;
    const float c0 = __shfl_sync(0xFFFFFFFFu, ac[0], (a >> 1) & 31), c1 = __shfl_sync(0xFFFFFFFFu, ac[1], (a >> 1) & 31);
    const float s0 = __shfl_sync(0xFFFFFFFFu, as[0], (a >> 1) & 31), s1 = __shfl_sync(0xFFFFFFFFu, as[1], (a >> 1) & 31);
    c[i] = a & 1 ? c1 : c0;
    s[i] = a & 1 ? s1 : s0;
    if (!p.interleaved && e < half) s[i] = -s[i];  // a cos - b sin, b cos + a sin
  }
  const int other = lane - in + (upper ? in - (half >> 3) : in + (half >> 3));

  for (int k = 0; k < turns; ++k) {
    const int hk = hw + k * step;
    if (hk >= h_end) break;  // the whole warp
    const int h = hk + lane / L;
    const uint4 now = raw;
    if (k + 1 < turns) raw = load(h + step);
    float x[8];
    unpack8(now, x);
    if (hk < p.q_heads + H && half > 0) {  // some of the warp's heads are rotated
      const bool rot = h < p.q_heads + H;
      if (p.interleaved) {
        if (rot) {
#pragma unroll
          for (int i = 0; i < 4; ++i)
            if (in * 4 + i < half) {
              const float a = x[2 * i], b = x[2 * i + 1];
              x[2 * i] = a * c[i] - b * s[i];
              x[2 * i + 1] = b * c[i] + a * s[i];
            }
        }
      } else {
        float y[8];
        if (vec) {
          uint4 q;
          q.x = __shfl_sync(0xFFFFFFFFu, now.x, other & 31);
          q.y = __shfl_sync(0xFFFFFFFFu, now.y, other & 31);
          q.z = __shfl_sync(0xFFFFFFFFu, now.z, other & 31);
          q.w = __shfl_sync(0xFFFFFFFFu, now.w, other & 31);
          unpack8(q, y);
        } else {
#pragma unroll
          for (int i = 0; i < 8; ++i) {
            const int e = in * 8 + i;
            y[i] = rot && e < p.rot_dim ? __half2float(row[h * D + (e < half ? e + half : e - half)]) : 0.0f;
          }
        }
        if (rot && turned) {
#pragma unroll
          for (int i = 0; i < 8; ++i)
            if (in * 8 + i < p.rot_dim) x[i] = x[i] * c[i] + y[i] * s[i];
        }
      }
    }
    // largest magnitude of the row, by its bits: a NaN ranks above infinity
    uint32_t top = 0;
    if (TYPE != kCacheFp16 && hk + HEADS > p.q_heads) {
#pragma unroll
      for (int i = 0; i < 8; ++i) top = max(top, __float_as_uint(x[i]) & 0x7FFFFFFFu);
#pragma unroll
      for (int o = L / 2; o > 0; o >>= 1) top = max(top, __shfl_xor_sync(0xFFFFFFFFu, top, o));
    }
    if (h < p.q_heads) {
      *reinterpret_cast<uint4*>(p.q_out + (int64_t)t * p.ldq + h * D + in * 8) = pack8(x);
    } else if (h < h_end && keep) {
      const bool is_v = h >= p.q_heads + H;
      const int kh = h - p.q_heads - (is_v ? H : 0);
      const int64_t in_page = ((int64_t)kh << p.c.page_shift) + off;
      const int64_t at = page * p.c.page_stride + in_page * D + in * 8;
      uint8_t* dst = is_v ? p.c.v : p.c.k;
      if (TYPE == kCacheFp16) {
        *reinterpret_cast<uint4*>(dst + at * 2) = pack8(x);
      } else {
        const float scale = top >= 0x7F800000u
                                ? __uint_as_float(0x7FC00000u)
                                : __fdiv_rn(__uint_as_float(top), TYPE == kCacheE4m3 ? 448.0f : 127.0f);
        *reinterpret_cast<uint2*>(dst + at) = encode8<TYPE>(x, scale);
        if (in == 0) (is_v ? p.c.v_scale : p.c.k_scale)[page * p.c.scale_page_stride + in_page] = scale;
      }
    }
  }
}

// A warp takes a slot: its rows are one 16-byte piece a lane, 32 lanes at a time
// over the heads, K and V side by side, and both outputs are contiguous.  Bound
// by HBM: 65536 rows of 8 heads from e4m3, a third of the bytes read and two
// written, take 64 us, 6.4 TB/s.
template <int D, int TYPE>
__global__ void __launch_bounds__(256) read_kernel(ReadParams p) {
  constexpr bool F16 = TYPE == kCacheFp16;
  constexpr int E = F16 ? 8 : 16;              // elements of a piece
  constexpr int L = D / E, HEADS = 32 / L;     // lanes of a row, heads at a time
  pdl_launch_dependents();
  pdl_wait_previous();
  const int lane = threadIdx.x & 31, piece = lane % L;
  const int H = p.c.kv_heads;
  const int warps = gridDim.x * 8;
  for (int64_t r = blockIdx.x * 8 + (threadIdx.x >> 5); r < p.rows; r += warps) {
    const int64_t slot = p.slots[r];
    const bool there = slot >= 0 && slot < (p.c.pages << p.c.page_shift);
    const int64_t page = slot >> p.c.page_shift, off = slot & ((1 << p.c.page_shift) - 1);
#pragma unroll 4
    for (int h = lane / L; h < H; h += HEADS) {
      const int64_t in_page = ((int64_t)h << p.c.page_shift) + off;
      const int64_t at = page * p.c.page_stride + in_page * D + piece * E;
      const int64_t sat = page * p.c.scale_page_stride + in_page;
      uint4 raw[2];
      float scale[2];
#pragma unroll
      for (int k = 0; k < 2; ++k) {
        raw[k] = make_uint4(0, 0, 0, 0);
        scale[k] = 0.0f;
        if (there && (k ? p.v_out : p.k_out)) {
          raw[k] = ld_stream_v4((k ? p.c.v : p.c.k) + at * (F16 ? 2 : 1));
          if (!F16) scale[k] = (k ? p.c.v_scale : p.c.k_scale)[sat];
        }
      }
#pragma unroll
      for (int k = 0; k < 2; ++k) {
        __half* out = k ? p.v_out : p.k_out;
        if (!out) continue;
        uint4* dst = reinterpret_cast<uint4*>(out + (r * H + h) * D + piece * E);
        if (F16) {
          __stcs(dst, raw[k]);
        } else {
          const uint32_t w[4] = {raw[k].x, raw[k].y, raw[k].z, raw[k].w};
          uint32_t o[8];
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            uint32_t lo, hi;
            widen4<F16 ? kCacheE4m3 : TYPE>(w[i], lo, hi);
            const float2 a = half2_bits_to_float2(lo), b = half2_bits_to_float2(hi);
            const __half2 x = __floats2half2_rn(a.x * scale[k], a.y * scale[k]);
            const __half2 y = __floats2half2_rn(b.x * scale[k], b.y * scale[k]);
            o[2 * i] = *reinterpret_cast<const uint32_t*>(&x);
            o[2 * i + 1] = *reinterpret_cast<const uint32_t*>(&y);
          }
          __stcs(dst, make_uint4(o[0], o[1], o[2], o[3]));
          __stcs(dst + 1, make_uint4(o[4], o[5], o[6], o[7]));
        }
      }
    }
  }
}

}  // namespace

template <int D, int TYPE>
static cudaError_t append_one(const AppendParams& p, int sms, cudaStream_t stream) {
  const int heads = (p.q_out ? p.q_heads : 0) + 2 * p.c.kv_heads;
  constexpr int kPer = 32 / (D / 8) * 4;  // heads of a block's turn
  // As many turns as leave every SM 44 warps: a turn more spares a warp its angles
  // (some 60 instructions a lane), but one token's heads go side by side.  512
  // tokens of 80 heads: 3 turns 6.4 us, 4 7.4, 5 (24 warps) 9.6, 2 7.0.
  const int all = (heads + kPer - 1) / kPer;
  int64_t turns = ((int64_t)p.tokens * all + 11 * sms / 2) / (11 * sms);
  turns = turns < 1 ? 1 : turns > all ? all : turns;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)p.tokens, (unsigned)((all + turns - 1) / turns));
  cfg.blockDim = dim3(128);
  cfg.stream = stream;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, append_kernel<D, TYPE>, p, (int)turns);
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
static cudaError_t read_one(const ReadParams& p, int sms, cudaStream_t stream) {
  // Several times the blocks that fit at once, so that those that end early make
  // room for others; a long read's warps take several rows each.  65536 rows of 8
  // heads, fp16, e4m3 and int8: 79.8, 63.8 and 62.8 us; 20 blocks an SM 81.9, 64.3
  // and 65.5; 8 83.7, 71.1 and 76.3; 5 92.6, 85.0 and 72.7.
  const int64_t blocks = ((int64_t)p.rows + 7) / 8;
  return launch_kernel(read_kernel<D, TYPE>, (int)(blocks < 32 * sms ? blocks : 32 * sms), 256, 0, stream,
                       kFlagPdl, p);
}

cudaError_t launch_cache_read(const ReadParams& p, int head_dim, int type, int sms,
                              cudaStream_t stream) {
  if (head_dim == 128) {
    if (type == kCacheFp16) return read_one<128, kCacheFp16>(p, sms, stream);
    if (type == kCacheE4m3) return read_one<128, kCacheE4m3>(p, sms, stream);
    return read_one<128, kCacheInt8>(p, sms, stream);
  }
  if (type == kCacheFp16) return read_one<64, kCacheFp16>(p, sms, stream);
  if (type == kCacheE4m3) return read_one<64, kCacheE4m3>(p, sms, stream);
  return read_one<64, kCacheInt8>(p, sms, stream);
}

}  // namespace nmk
