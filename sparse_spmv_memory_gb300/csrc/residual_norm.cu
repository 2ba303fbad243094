// residual_norm.cu -- the residual stream's update by a block's output with the norms
// around it (nm_residual_norm): s = ra r + sc gate post(b), out = pre(s).
//
// A row's elements stay in the registers of its threads from the loads to the
// stores, so that every array is read or written once: a row costs 2 + 2 bytes an
// element in and 2 + 2 out (fp16 stream), and memory bounds it.  What keeps it from
// that is the time from a row's first load to its last store, in which an SM holds few
// rows, and the instructions: so whatever does not depend on a sum over the row (the
// norms' parameters, the gate) is asked for before that sum, and rows bypass L1 so that
// the parameters stay there.  Groups of 8 elements are a thread's unit of work.  A layer
// norm takes its mean first, and then the squares about it and what the mean is off by.
//
// The kernels, by the rows: few rows of whole groups (a row a block, one group a
// thread: the time to the result counts), many of them (blocks that stay), and long rows
// of any width, stride and alignment (shorter ones of these: residual_norm_any.cu).
#include <cuda_fp16.h>
#include <cuda_runtime.h>
#include <stdint.h>

#include "norm_rows.cuh"

namespace nmk {
namespace {

// 16 bytes that are read once: not kept in L1.  (Not read-only loads: the stream may be
// updated where it lies.)
__device__ __forceinline__ uint4 load_once(const void* p) {
  uint4 v;
  asm volatile("ld.global.L1::no_allocate.v4.u32 {%0,%1,%2,%3}, [%4];"
               : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w)
               : "l"(p));
  return v;
}

template <typename S>
struct Raw {  // a group as it lies in memory
  static constexpr int kSlots = sizeof(S) / 2;  // pieces of 16 bytes
  uint32_t w[4 * kSlots];
  __device__ __forceinline__ void read(const S* p) {
#pragma unroll
    for (int i = 0; i < kSlots; ++i) {
      const uint4 u = load_once(reinterpret_cast<const uint4*>(p) + i);
      w[4 * i] = u.x;
      w[4 * i + 1] = u.y;
      w[4 * i + 2] = u.z;
      w[4 * i + 3] = u.w;
    }
  }
};

struct Group {  // 8 elements in fp32
  Pair v[4];
};

__device__ __forceinline__ Group widen(const Raw<__half>& q) {
  Group x;
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const float2 f = half2_bits_to_float2(q.w[i]);
    x.v[i] = pair(f.x, f.y);
  }
  return x;
}

__device__ __forceinline__ Group widen(const Raw<float>& q) {
  Group x;
#pragma unroll
  for (int i = 0; i < 4; ++i) x.v[i] = pair(__uint_as_float(q.w[2 * i]), __uint_as_float(q.w[2 * i + 1]));
  return x;
}

__device__ __forceinline__ Raw<__half> narrow(const Group& x, __half) {
  Raw<__half> q;
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const float2 f = x.v[i];
    const __half2 h = __floats2half2_rn(f.x, f.y);
    q.w[i] = *reinterpret_cast<const uint32_t*>(&h);
  }
  return q;
}

__device__ __forceinline__ Raw<float> narrow(const Group& x, float) {
  Raw<float> q;
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const float2 f = x.v[i];
    q.w[2 * i] = __float_as_uint(f.x);
    q.w[2 * i + 1] = __float_as_uint(f.y);
  }
  return q;
}

__device__ __forceinline__ void times(Group& x, const Group& y) {
#pragma unroll
  for (int i = 0; i < 4; ++i) x.v[i] = mul2(x.v[i], y.v[i]);
}

__device__ __forceinline__ void times(Group& x, float y) {
#pragma unroll
  for (int i = 0; i < 4; ++i) x.v[i] = mul2(x.v[i], pair(y, y));
}

// x - mean (layer norms only, the mean as its sum gives it), and the factor of the norm;
// r = 1 without a norm.  x is 0 outside the row, and zero(j, x) makes it so again.
template <int N, typename Zero>
__device__ __forceinline__ Factor factor(Group (&x)[N], const NormArgs& a, float inv_width, RowSum& sum, Zero&& zero) {
  if (a.kind == NM_NORM_NONE) return {1.f, 0.f};
  auto total = [&]() {
    Pair t = pair(0.f, 0.f);
#pragma unroll
    for (int j = 0; j < N; ++j)
      t = add2(t, add2(add2(x[j].v[0], x[j].v[1]), add2(x[j].v[2], x[j].v[3])));
    return t.x + t.y;
  };
  auto squares = [&]() {
    Pair t = pair(0.f, 0.f);
#pragma unroll
    for (int j = 0; j < N; ++j)
#pragma unroll
      for (int i = 0; i < 4; ++i) t = fma2(x[j].v[i], x[j].v[i], t);
    return t.x + t.y;
  };
  if (a.kind != NM_NORM_LAYER) return {1.f / sqrtf(sum(squares()) * inv_width + a.eps), 0.f};
  const float mean = __fmul_rn(sum(total()), inv_width);  // (equal elements, as a rule: nothing left)
#pragma unroll
  for (int j = 0; j < N; ++j) {
#pragma unroll
    for (int i = 0; i < 4; ++i) x[j].v[i] = add2(x[j].v[i], pair(-mean, -mean));
    zero(j, x[j]);
  }
  return layer_factor(sum(pair(total(), squares())), inv_width, a.eps);
}

// The same with the rest of the mean taken from x (no longer 0 outside the row): r.
template <int N, typename Zero>
__device__ __forceinline__ float centred(Group (&x)[N], const NormArgs& a, float inv_width, RowSum& sum, Zero&& zero) {
  const Factor f = factor<N>(x, a, inv_width, sum, zero);
  if (a.kind == NM_NORM_LAYER) {
#pragma unroll
    for (int j = 0; j < N; ++j)
#pragma unroll
      for (int i = 0; i < 4; ++i) x[j].v[i] = add2(x[j].v[i], pair(-f.rest, -f.rest));
  }
  return f.r;
}

template <int N>
__device__ __forceinline__ float centred(Group (&x)[N], const NormArgs& a, float inv_width, RowSum& sum) {
  return centred<N>(x, a, inv_width, sum, [](int, Group&) {});
}

// For kernels that multiply by r first: x r - rest r in one operation (-0 without a rest,
// which changes nothing).
struct Scale {
  Pair r, shift;
  __device__ __forceinline__ explicit Scale(const Factor& f) {
    const float s = -__fmul_rn(f.rest, f.r);
    r = pair(f.r, f.r);
    shift = pair(s, s);
  }
  __device__ __forceinline__ void operator()(Group& x) const {
#pragma unroll
    for (int i = 0; i < 4; ++i) x.v[i] = fma2(x.v[i], r, shift);
  }
};

// N groups of a norm's parameters, packed where they are fp16.
template <int N>
struct Packed {
  uint4 w[N];
  __device__ __forceinline__ void load(const void* base, int fp32, int at, int step) {
    if (fp32) return;
#pragma unroll
    for (int j = 0; j < N; ++j)
      w[j] = *reinterpret_cast<const uint4*>(static_cast<const __half*>(base) + at + j * step);
  }
  __device__ __forceinline__ Group get(int j, const void* base, int fp32, int at) const {
    if (fp32) {
      const float4* f = reinterpret_cast<const float4*>(static_cast<const float*>(base) + at);
      const float4 a = f[0], b = f[1];
      return {{pair(a.x, a.y), pair(a.z, a.w), pair(b.x, b.y), pair(b.z, b.w)}};
    }
    Raw<__half> q;
    q.w[0] = w[j].x;
    q.w[1] = w[j].y;
    q.w[2] = w[j].z;
    q.w[3] = w[j].w;
    return widen(q);
  }
};

template <typename S>
__device__ __forceinline__ void put(S* to, const Group& x) {
  const Raw<S> q = narrow(x, S());
#pragma unroll
  for (int i = 0; i < Raw<S>::kSlots; ++i)
    reinterpret_cast<uint4*>(to)[i] = make_uint4(q.w[4 * i], q.w[4 * i + 1], q.w[4 * i + 2], q.w[4 * i + 3]);
}

// x times a norm's r (offset + weight), plus its bias, for a group whose parameters were
// asked for before.
template <typename P>
__device__ __forceinline__ void apply(Group& x, float r, const NormArgs& a, const P& weight, const P& bias, int j,
                                      int at) {
  if (a.weight) {
    const Group w = weight.get(j, a.weight, a.params_fp32, at);
    const Pair r2 = pair(r, r), off = pair(r * a.offset, r * a.offset);
#pragma unroll
    for (int i = 0; i < 4; ++i) x.v[i] = mul2(x.v[i], fma2(w.v[i], r2, off));
  } else {
    times(x, r);
  }
  if (a.bias) {
    const Group w = bias.get(j, a.bias, a.params_fp32, at);
#pragma unroll
    for (int i = 0; i < 4; ++i) x.v[i] = add2(x.v[i], w.v[i]);
  }
}

// ---- few rows of whole groups ---------------------------------------------------------
// A row on blockDim.x threads, N groups a thread; blockDim.y rows a block.  One row of
// 4096: 1.9 us, loads and one sum.
template <typename S, int N>
__global__ void __launch_bounds__(1024) residual_norm_few_kernel(const ResidualNormParams p) {
  __shared__ float part[4][32];
  pdl_launch_dependents();
  pdl_wait_previous();
  const int at = 8 * (int)threadIdx.x, step = 8 * (int)blockDim.x;
  const int64_t mine = (int64_t)blockIdx.x * blockDim.y + threadIdx.y;
  const bool live = mine < p.tokens;
  const int64_t row = live ? mine : p.tokens - 1;  // (rows past the end work on the last, and store nothing)
  RowSum sum{part};
  Group s[N];
  Raw<S> r[N];
#pragma unroll
  for (int j = 0; j < N; ++j) r[j].read(static_cast<const S*>(p.residual) + row * p.ldr + at + j * step);
  Packed<N> weight, bias;
  if (p.block) {
    Raw<__half> b[N], g[N];
#pragma unroll
    for (int j = 0; j < N; ++j) b[j].read(p.block + row * p.ldb + at + j * step);
    if (p.post.weight) weight.load(p.post.weight, p.post.params_fp32, at, step);
    if (p.post.bias) bias.load(p.post.bias, p.post.params_fp32, at, step);
    if (p.gate) {
#pragma unroll
      for (int j = 0; j < N; ++j) g[j].read(p.gate + row * p.ldg + at + j * step);
    }
#pragma unroll
    for (int j = 0; j < N; ++j) s[j] = widen(b[j]);
    if (p.post.kind != NM_NORM_NONE) {
      const float q = centred<N>(s, p.post, p.inv_width, sum);
#pragma unroll
      for (int j = 0; j < N; ++j) apply(s[j], q, p.post, weight, bias, j, at + j * step);
    }
    if (p.out && p.pre.weight) weight.load(p.pre.weight, p.pre.params_fp32, at, step);
#pragma unroll
    for (int j = 0; j < N; ++j) {
      if (p.gate) times(s[j], widen(g[j]));
      Group x = widen(r[j]);
      times(x, p.residual_scale);
#pragma unroll
      for (int i = 0; i < 4; ++i) s[j].v[i] = fma2(pair(p.scale, p.scale), s[j].v[i], x.v[i]);
    }
  } else {
    if (p.out && p.pre.weight) weight.load(p.pre.weight, p.pre.params_fp32, at, step);
#pragma unroll
    for (int j = 0; j < N; ++j) {
      s[j] = widen(r[j]);
      times(s[j], p.residual_scale);
    }
  }
  if (p.out && p.pre.bias) bias.load(p.pre.bias, p.pre.params_fp32, at, step);
  if (p.stream_out && live) {
#pragma unroll
    for (int j = 0; j < N; ++j) put(static_cast<S*>(p.stream_out) + row * p.lds + at + j * step, s[j]);
  }
  if (!p.out) return;
  if (p.pre.kind != NM_NORM_NONE) {
    const float q = centred<N>(s, p.pre, p.inv_width, sum);
#pragma unroll
    for (int j = 0; j < N; ++j) apply(s[j], q, p.pre, weight, bias, j, at + j * step);
  }
  if (live) {
#pragma unroll
    for (int j = 0; j < N; ++j) put(p.out + row * p.ldo + at + j * step, s[j]);
  }
}

// ---- many rows of whole groups -------------------------------------------------------
// Blocks that stay and take row after row.  A thread keeps its columns: the norms'
// parameters, the gate that all tokens share and the scale are multiplied once, in
// fp32, and held in registers (P and W, with BIAS also their biases), which leaves a
// row two conversions and about seven operations on both of two elements; and the
// next rows' stream, block and gate are on their way to shared memory meanwhile, each
// thread's own groups to slots of its own (no barrier).  4096 rows of 8192 with both
// norms and a gate: 49 us (5.5 TB/s), with layer norms 82; a block a row, with the
// parameters read for every row, took 55 (RMS norms), half of it issuing instructions and
// half waiting for a row's loads.
__device__ __forceinline__ void copy_async(uint4* to, const void* from) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(smem_addr(to)), "l"(from) : "memory");
}

template <typename S>
__device__ __forceinline__ Raw<S> staged(const uint4* p, int step) {
  Raw<S> q;
#pragma unroll
  for (int i = 0; i < Raw<S>::kSlots; ++i) {
    const uint4 u = p[i * step];
    q.w[4 * i] = u.x;
    q.w[4 * i + 1] = u.y;
    q.w[4 * i + 2] = u.z;
    q.w[4 * i + 3] = u.w;
  }
  return q;
}

// offset + weight (1 without), or a bias (0 without), of the group at `at`.
__device__ __forceinline__ Group parameters(const void* base, int fp32, float offset, float without, int at) {
  if (!base) return {{pair(without, without), pair(without, without), pair(without, without), pair(without, without)}};
  Packed<1> w;
  w.load(base, fp32, at, 0);
  Group x = w.get(0, base, fp32, at);
  const Pair o = pair(offset, offset);
#pragma unroll
  for (int i = 0; i < 4; ++i) x.v[i] = add2(x.v[i], o);
  return x;
}

template <typename S, int N, bool BIAS>
__global__ void __launch_bounds__(1024) residual_norm_many_kernel(const ResidualNormParams p, int stages) {
  __shared__ float part[4][32];
  extern __shared__ uint4 slots[];
  constexpr int kStream = sizeof(S) / 2;  // slots of a group of the stream
  const int threads = blockDim.x * blockDim.y;
  uint4* const own = slots + threadIdx.y * blockDim.x + threadIdx.x;
  const int per_stage = N * (kStream + 1 + p.own_gate);
  auto slot = [&](int stage, int k) { return own + (stage * per_stage + k) * threads; };
  const int at = 8 * (int)threadIdx.x, step = 8 * (int)blockDim.x;
  auto fetch = [&](int64_t row, int stage) {
    if (row < p.tokens) {
#pragma unroll
      for (int j = 0; j < N; ++j) {
        if (p.block) copy_async(slot(stage, j), p.block + row * p.ldb + at + j * step);
        const S* r = static_cast<const S*>(p.residual) + row * p.ldr + at + j * step;
#pragma unroll
        for (int i = 0; i < kStream; ++i)
          copy_async(slot(stage, N + j * kStream + i), r + i * (16 / (int)sizeof(S)));
        if (p.own_gate) copy_async(slot(stage, N * (1 + kStream) + j), p.gate + row * p.ldg + at + j * step);
      }
    }
    asm volatile("cp.async.commit_group;" ::: "memory");
  };
  pdl_launch_dependents();
  pdl_wait_previous();
  int64_t row = (int64_t)blockIdx.x * blockDim.y + threadIdx.y;
  const int64_t next = (int64_t)gridDim.x * blockDim.y;
  for (int i = 0; i < stages - 1; ++i) fetch(row + i * next, i);

  Group P[N], W[N], PB[BIAS ? N : 1], WB[BIAS ? N : 1];
#pragma unroll
  for (int j = 0; j < N; ++j) {
    const int c = at + j * step;
    P[j] = parameters(p.post.weight, p.post.params_fp32, p.post.offset, 1.f, c);
    W[j] = parameters(p.pre.weight, p.pre.params_fp32, p.pre.offset, 1.f, c);
    Group g = parameters(p.own_gate ? nullptr : p.gate, 0, 0.f, 1.f, c);
    times(g, p.scale);
    times(P[j], g);
    if (BIAS) {
      PB[j] = parameters(p.post.bias, p.post.params_fp32, 0.f, 0.f, c);
      WB[j] = parameters(p.pre.bias, p.pre.params_fp32, 0.f, 0.f, c);
      times(PB[j], g);
    }
  }

  RowSum sum{part};
  const Pair keep = pair(p.residual_scale, p.residual_scale);
  int stage = 0, free_stage = stages - 1;
  // (the block's rows go through the barriers together: those past the end too)
  for (int64_t first = (int64_t)blockIdx.x * blockDim.y; first < p.tokens; first += next, row += next) {
    fetch(row + (stages - 1) * next, free_stage);
    if (stages == 4)
      asm volatile("cp.async.wait_group 3;" ::: "memory");
    else if (stages == 3)
      asm volatile("cp.async.wait_group 2;" ::: "memory");
    else
      asm volatile("cp.async.wait_group 1;" ::: "memory");
    const bool live = row < p.tokens;
    Group s[N];
    if (p.block) {
#pragma unroll
      for (int j = 0; j < N; ++j) s[j] = widen(staged<__half>(slot(stage, j), threads));
      const Scale scaled(factor<N>(s, p.post, p.inv_width, sum, [](int, Group&) {}));
#pragma unroll
      for (int j = 0; j < N; ++j) {
        Group x = widen(staged<S>(slot(stage, N + j * kStream), threads));
        scaled(s[j]);
        if (p.own_gate) {
          const Group g = widen(staged<__half>(slot(stage, N * (1 + kStream) + j), threads));
          Group w = P[j];
          times(w, g);
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            x.v[i] = mul2(keep, x.v[i]);
            if (BIAS) x.v[i] = fma2(PB[j].v[i], g.v[i], x.v[i]);
            s[j].v[i] = fma2(s[j].v[i], w.v[i], x.v[i]);
          }
        } else {
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            x.v[i] = BIAS ? fma2(keep, x.v[i], PB[j].v[i]) : mul2(keep, x.v[i]);
            s[j].v[i] = fma2(s[j].v[i], P[j].v[i], x.v[i]);
          }
        }
      }
    } else {
#pragma unroll
      for (int j = 0; j < N; ++j) {
        s[j] = widen(staged<S>(slot(stage, N + j * kStream), threads));
#pragma unroll
        for (int i = 0; i < 4; ++i) s[j].v[i] = mul2(keep, s[j].v[i]);
      }
    }
    if (p.stream_out && live) {
      S* to = static_cast<S*>(p.stream_out) + row * p.lds + at;
#pragma unroll
      for (int j = 0; j < N; ++j) put(to + j * step, s[j]);
    }
    if (p.out) {
      const Scale scaled(factor<N>(s, p.pre, p.inv_width, sum, [](int, Group&) {}));
      __half* to = p.out + row * p.ldo + at;
#pragma unroll
      for (int j = 0; j < N; ++j) {
        scaled(s[j]);
#pragma unroll
        for (int i = 0; i < 4; ++i)
          s[j].v[i] = BIAS ? fma2(s[j].v[i], W[j].v[i], WB[j].v[i]) : mul2(s[j].v[i], W[j].v[i]);
        if (live) put(to + j * step, s[j]);
      }
    }
    free_stage = stage;
    stage = stage + 1 == stages ? 0 : stage + 1;
  }
  asm volatile("cp.async.wait_all;" ::: "memory");
}

// ---- long rows of any kind ------------------------------------------------------------
// Groups are the 16-byte pieces of the stream's row (32 bytes of an fp32 stream), so a
// row may start and end inside one: group j's elements are at(j) .. at(j) + 7, of
// which those in 0 .. width - 1 are the row's.  Every array whose row starts at the
// same place in a piece (rows of an odd width, all alike) is read by whole pieces, the
// ends with what lies beside them as far as it is the array's (the rows before and
// after), and written by whole pieces but for the ends; other arrays element by element.
template <typename S>
__device__ __forceinline__ int place(const void* p) {  // in its group, of an address
  return (int)(reinterpret_cast<uintptr_t>(p) / sizeof(S)) & 7;
}

__device__ __forceinline__ uint32_t bits(__half h) { return __half_as_ushort(h); }

// 0 for the elements of a group outside the row.
__device__ __forceinline__ void trim(Group& x, int at, int width) {
  if (at >= 0 && at + 8 <= width) return;
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    if (at + 2 * i < 0 || at + 2 * i >= width) x.v[i].x = 0.f;
    if (at + 2 * i + 1 < 0 || at + 2 * i + 1 >= width) x.v[i].y = 0.f;
  }
}

template <typename S>
struct Line {  // a row of an array
  S* row;
  int width;
  bool vec;       // its pieces are the stream's, and one lies inside the row
  int low, high;  // the group starts whose pieces are the array's
  int inside;     // one of them

  __device__ __forceinline__ Line(const void* base, int64_t index, int64_t rows, int64_t ld, int shift, int w) {
    row = static_cast<S*>(const_cast<void*>(base)) + index * ld;
    width = w;
    inside = (8 - shift) & 7;
    vec = ((place<S>(row) - shift) & (16 / (int)sizeof(S) - 1)) == 0 && inside + 8 <= w;
    const int64_t before = index * ld, behind = (rows - 1 - index) * ld + w - 8;
    low = before > 8 ? -8 : -(int)before;
    high = behind > w ? w : (int)behind;
  }

  __device__ __forceinline__ Raw<S> gather(int at) const {
    Raw<S> q;
#pragma unroll
    for (int i = 0; i < 4 * Raw<S>::kSlots; ++i) q.w[i] = 0u;
#pragma unroll
    for (int i = 0; i < 8; ++i)
      if (at + i >= 0 && at + i < width) {
        if constexpr (sizeof(S) == 2)
          q.w[i / 2] |= bits(row[at + i]) << (16 * (i & 1));
        else
          q.w[i] = __float_as_uint(row[at + i]);
      }
    return q;
  }

  // N groups; what they hold outside the row is not the row's.
  template <int N, typename At>
  __device__ __forceinline__ void load(Raw<S> (&q)[N], At&& at) const {
    bool odd = !vec;
    if (vec) {
#pragma unroll
      for (int j = 0; j < N; ++j) {
        const bool safe = at(j) >= low && at(j) <= high;
        q[j].read(row + (safe ? at(j) : inside));
        odd |= !safe && at(j) < width;
      }
    }
    if (odd) {
#pragma unroll
      for (int j = 0; j < N; ++j)
        if (!vec || at(j) < low || at(j) > high) q[j] = gather(at(j));
    }
  }

  __device__ __forceinline__ void store(int at, const Group& x) const {
    if (vec && at >= 0 && at + 8 <= width) {
      put(row + at, x);
      return;
    }
    const Raw<S> q = narrow(x, S());
#pragma unroll
    for (int i = 0; i < 8; ++i)
      if (at + i >= 0 && at + i < width) {
        if constexpr (sizeof(S) == 2)
          row[at + i] = __ushort_as_half((unsigned short)(q.w[i / 2] >> (16 * (i & 1))));
        else
          row[at + i] = __uint_as_float(q.w[i]);
      }
  }
};

// N groups of a norm's parameters, widened: the pieces that hold them, and the words
// picked by their place, which is the same for a whole row of the stream.
template <int N>
struct Picked {
  uint32_t w[N][8];

  template <typename At>
  __device__ __forceinline__ void load(const void* base, int fp32, At&& at, int shift, int width) {
    const int lead = (8 - shift) & 7;  // at = 8 k + lead
    const int top = (width - 16) / 8 * 8;
    const bool pieces = (reinterpret_cast<uintptr_t>(base) & 15) == 0 && width >= 16;
    if (pieces) {
#pragma unroll
      for (int j = 0; j < N; ++j) {
        const int from = min(max(at(j) - lead, 0), top);
        if (fp32)
          pick(static_cast<const float*>(base) + from, lead, w[j]);
        else
          pick(static_cast<const __half*>(base) + from, lead, w[j]);
      }
    }
#pragma unroll
    for (int j = 0; j < N; ++j) {
      if ((pieces && at(j) - lead >= 0 && at(j) - lead <= top) || at(j) >= width) continue;
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        const bool in = at(j) + i >= 0 && at(j) + i < width;
        w[j][i] = !in ? 0u
                      : __float_as_uint(fp32 ? static_cast<const float*>(base)[at(j) + i]
                                             : __half2float(static_cast<const __half*>(base)[at(j) + i]));
      }
    }
  }

  // 8 of 16 words (or halves) from `lead` on.
  static __device__ __forceinline__ void pick(const float* p, int lead, uint32_t* w) {
    uint32_t q[16];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const uint4 u = reinterpret_cast<const uint4*>(p)[i];
      q[4 * i] = u.x;
      q[4 * i + 1] = u.y;
      q[4 * i + 2] = u.z;
      q[4 * i + 3] = u.w;
    }
#pragma unroll
    for (int i = 0; i < 12; ++i) q[i] = (lead & 4) ? q[i + 4] : q[i];
#pragma unroll
    for (int i = 0; i < 10; ++i) q[i] = (lead & 2) ? q[i + 2] : q[i];
#pragma unroll
    for (int i = 0; i < 8; ++i) w[i] = (lead & 1) ? q[i + 1] : q[i];
  }

  static __device__ __forceinline__ void pick(const __half* p, int lead, uint32_t* w) {
    uint32_t q[8];
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      const uint4 u = reinterpret_cast<const uint4*>(p)[i];
      q[4 * i] = u.x;
      q[4 * i + 1] = u.y;
      q[4 * i + 2] = u.z;
      q[4 * i + 3] = u.w;
    }
#pragma unroll
    for (int i = 0; i < 6; ++i) q[i] = (lead & 4) ? q[i + 2] : q[i];
#pragma unroll
    for (int i = 0; i < 5; ++i) q[i] = (lead & 2) ? q[i + 1] : q[i];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const float2 f = half2_bits_to_float2(__funnelshift_r(q[i], q[i + 1], (lead & 1) * 16));
      w[2 * i] = __float_as_uint(f.x);
      w[2 * i + 1] = __float_as_uint(f.y);
    }
  }

  __device__ __forceinline__ Group get(int j, const void*, int, int) const {
    Raw<float> q;
#pragma unroll
    for (int i = 0; i < 8; ++i) q.w[i] = w[j][i];
    return widen(q);
  }
};

// A row on blockDim.x threads, N groups a thread; blockDim.y rows a block.  MAX, MIN:
// threads a block at most, and blocks an SM at least (what the registers are cut to).
template <typename S, int N, int MAX, int MIN>
__global__ void __launch_bounds__(MAX, MIN) residual_norm_long_kernel(const ResidualNormParams p) {
  __shared__ float part[4][32];
  pdl_launch_dependents();
  pdl_wait_previous();
  const int64_t mine = (int64_t)blockIdx.x * blockDim.y + threadIdx.y;
  const bool live = mine < p.tokens;
  const int64_t row = live ? mine : p.tokens - 1;  // (rows past the end work on the last, and store nothing)
  const int width = p.width;
  RowSum sum{part};
  const int shift = place<S>(static_cast<const S*>(p.residual) + row * p.ldr);
  const int first = 8 * (int)threadIdx.x - shift, step = 8 * (int)blockDim.x;
  auto at = [&](int j) { return first + j * step; };
  auto zero = [&](int j, Group& x) { trim(x, at(j), width); };

  Group s[N];
  Raw<S> r[N];
  Line<S>(p.residual, row, p.tokens, p.ldr, shift, width).load(r, at);
  Picked<N> weight, bias;
  if (p.block) {
    Raw<__half> b[N];
    const Line<__half> gate(p.gate, p.ldg ? row : 0, p.ldg ? p.tokens : 1, p.ldg, shift, width);
    Line<__half>(p.block, row, p.tokens, p.ldb, shift, width).load(b, at);
    if (p.gate && p.ldg != 0) {  // a token's own gate is on its way to L2 meanwhile
#pragma unroll
      for (int j = 0; j < N; ++j)
        asm volatile("prefetch.global.L2 [%0];" ::"l"(gate.row + min(max(at(j), 0), width - 1)));
    }
    const bool normed = p.post.kind != NM_NORM_NONE;
    if (normed && p.post.weight) weight.load(p.post.weight, p.post.params_fp32, at, shift, width);
#pragma unroll
    for (int j = 0; j < N; ++j) {
      s[j] = widen(b[j]);
      zero(j, s[j]);
    }
    if (normed) {
      const float q = centred<N>(s, p.post, p.inv_width, sum, zero);
      if (p.post.bias) bias.load(p.post.bias, p.post.params_fp32, at, shift, width);
#pragma unroll
      for (int j = 0; j < N; ++j) apply(s[j], q, p.post, weight, bias, j, at(j));
    }
    if (p.gate) {
      gate.load(b, at);
#pragma unroll
      for (int j = 0; j < N; ++j) times(s[j], widen(b[j]));
    }
#pragma unroll
    for (int j = 0; j < N; ++j) {
      Group x = widen(r[j]);
      times(x, p.residual_scale);
#pragma unroll
      for (int i = 0; i < 4; ++i) s[j].v[i] = fma2(pair(p.scale, p.scale), s[j].v[i], x.v[i]);
    }
  } else {
#pragma unroll
    for (int j = 0; j < N; ++j) {
      s[j] = widen(r[j]);
      times(s[j], p.residual_scale);
    }
  }
#pragma unroll
  for (int j = 0; j < N; ++j) zero(j, s[j]);
  if (p.stream_out && live) {
    const Line<S> to(p.stream_out, row, p.tokens, p.lds, shift, width);
#pragma unroll
    for (int j = 0; j < N; ++j) to.store(at(j), s[j]);
  }
  if (!p.out) return;
  if (p.pre.kind != NM_NORM_NONE) {
    if (p.pre.weight) weight.load(p.pre.weight, p.pre.params_fp32, at, shift, width);
    const float q = centred<N>(s, p.pre, p.inv_width, sum, zero);
    if (p.pre.bias) bias.load(p.pre.bias, p.pre.params_fp32, at, shift, width);
#pragma unroll
    for (int j = 0; j < N; ++j) apply(s[j], q, p.pre, weight, bias, j, at(j));
  }
  if (live) {
    const Line<__half> to(p.out, row, p.tokens, p.ldo, shift, width);
#pragma unroll
    for (int j = 0; j < N; ++j) to.store(at(j), s[j]);
  }
}

// ---- launches -----------------------------------------------------------------------
bool at16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15) == 0; }

// Whether every row of every array is whole 16-byte pieces.
template <typename S>
bool whole_rows(const ResidualNormParams& p) {
  const int64_t r = 16 / sizeof(S);  // elements of the stream in a piece of 16 bytes
  const NormArgs* norms[2] = {&p.post, &p.pre};
  for (const NormArgs* n : norms)
    if (!at16(n->weight) || !at16(n->bias)) return false;
  return p.width % 256 == 0 && at16(p.residual) && p.ldr % r == 0 && at16(p.stream_out) &&
         p.lds % r == 0 && at16(p.block) && p.ldb % 8 == 0 && at16(p.gate) && p.ldg % 8 == 0 &&
         at16(p.out) && p.ldo % 8 == 0;
}

template <typename S, int N, int MAX>
cudaError_t launch_long(const ResidualNormParams& p, int groups, cudaStream_t stream) {
  const int threads = ((groups + N - 1) / N + 31) / 32 * 32;
  return launch_rows(residual_norm_long_kernel<S, N, MAX, 1>, p, threads, stream);
}

template <typename S, int N, bool BIAS>
cudaError_t launch_many(const ResidualNormParams& p0, int groups, const DeviceInfo& d, cudaStream_t stream) {
  ResidualNormParams p = p0;
  p.own_gate = p.gate && p.ldg != 0;
  auto* k = residual_norm_many_kernel<S, N, BIAS>;
  static int done[64] = {0};
  cudaError_t e = ensure_max_smem(reinterpret_cast<const void*>(k), done, 64, 1024);
  if (e != cudaSuccess) return e;
  const int threads = groups / N, rows = threads >= 256 ? 1 : 256 / threads;
  const size_t stage = (size_t)threads * rows * 16 * N * (sizeof(S) / 2 + 1 + p.own_gate);
  // as many blocks as 64 registers a thread let an SM have, and as many stages (2 .. 4)
  // as their shared memory then holds
  int blocks = 1024 / (threads * rows), stages;
  for (;; --blocks) {
    stages = (int)((size_t)(d.smem_sm / blocks - 1536) / stage);
    if (stages >= 2 || blocks == 1) break;
  }
  if (stages < 2) return cudaErrorInvalidValue;  // (48 KB a stage at most: never)
  if (stages > 4) stages = 4;
  const int64_t sets = (p.tokens + rows - 1) / rows;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)(sets < (int64_t)d.sms * blocks ? sets : (int64_t)d.sms * blocks));
  cfg.blockDim = dim3((unsigned)threads, (unsigned)rows);
  cfg.dynamicSmemBytes = stage * stages;
  cfg.stream = stream;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, k, p, stages);
}

template <typename S, int N>
cudaError_t launch_many(const ResidualNormParams& p, int groups, const DeviceInfo& d, cudaStream_t stream) {
  const bool bias = (p.post.kind != NM_NORM_NONE && p.post.bias) || (p.pre.kind != NM_NORM_NONE && p.pre.bias);
  return bias ? launch_many<S, N, true>(p, groups, d, stream) : launch_many<S, N, false>(p, groups, d, stream);
}

template <typename S>
cudaError_t launch_stream(const ResidualNormParams& p, const DeviceInfo& d, cudaStream_t stream) {
  if (whole_rows<S>(p)) {
    // a row a block, one group a thread, while the rows' threads fit the SMs at once
    const int groups = p.width / 8;
    if (groups <= 1024 && p.tokens * groups <= (int64_t)d.sms * 1024)
      return launch_rows(residual_norm_few_kernel<S, 1>, p, groups, stream);
    if (groups <= 1024) {
      if (groups % 64 == 0) return launch_many<S, 2>(p, groups, d, stream);
      return launch_many<S, 1>(p, groups, d, stream);
    }
    if (groups <= 2048 && groups % 64 == 0)
      return launch_rows(residual_norm_few_kernel<S, 2>, p, groups / 2, stream);
    if (groups % 128 == 0)
      return launch_rows(residual_norm_few_kernel<S, 4>, p, groups / 4, stream);
  }
  // Other rows element by element up to 8192 accesses of a row, else by shifted groups:
  // 777 rows of 5121 (fp32 stream, layer norms) 22.5 us for 24.8 when it was chosen (25.0
  // now, with the mean corrected), 16384 of 100 5.8 for 17.8; 2000 of 30001 180 for 314.
  if (takes_any_rows(p, sizeof(S) == 4)) return launch_any_rows(p, sizeof(S) == 4, stream);
  const int groups = (p.width + 14) / 8;  // with a start anywhere in a piece
  if (groups <= 2048) return launch_long<S, 4, 512>(p, groups, stream);
  if (groups <= 4096) return launch_long<S, 4, 1024>(p, groups, stream);
  return launch_long<S, 5, 1024>(p, groups, stream);  // 32768 and a start inside a piece
}

}  // namespace

cudaError_t launch_residual_norm(const ResidualNormParams& p0, int stream_fp32, const DeviceInfo& d,
                                 cudaStream_t stream) {
  ResidualNormParams p = p0;
  p.inv_width = 1.f / (float)p.width;
  return stream_fp32 ? launch_stream<float>(p, d, stream) : launch_stream<__half>(p, d, stream);
}

}  // namespace nmk
