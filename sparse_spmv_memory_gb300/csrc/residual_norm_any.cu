// residual_norm_any.cu -- nm_residual_norm for rows of any width, stride and alignment.
//
// A row's elements are dealt to its threads one at a time (V 1), or two where all rows
// begin on even elements (V 2): the accesses of a warp lie side by side wherever the row
// begins, and need no shifting.  What bounds it is issuing instructions, of which an
// odd row takes one for every load and store of 32 elements, so the distance of a
// thread's elements is a constant of the kernel (T) and their addresses are immediate.
// A thread has E pairs in fp32 registers; block, stream, gate and the first parameters
// are asked for before the first sum.  64 registers a thread (40 for pairs): with fewer
// they are spilled.  777 rows of 5121, fp32 stream, layer norms and a gate for each token:
// 25.0 us (2.2 TB/s), three rounds of blocks of 8 us each, loads and four sums one after
// the other; 4096 of 1002, fp16: 8.0 us (4.1 TB/s); 16384 of 100: 5.8.
#include "norm_rows.cuh"

namespace nmk {
namespace {

// Accesses j and j + 1 of a thread to a row, as fp32: elements j T and (j + 1) T from `q`
// on (V 1), or one access of two (V 2, j counts pairs).  `left`: elements from q to the
// row's end.
template <int V, int T>
struct Accesses {
  int left;

  __device__ __forceinline__ bool in(int k, int h) const {  // of pair k, its half
    return V == 2 ? 2 * T * k < left : T * (2 * k + h) < left;
  }
  __device__ __forceinline__ Pair load(const float* q, int k) const {
    if (V == 2) return in(k, 0) ? *reinterpret_cast<const float2*>(q + 2 * T * k) : pair(0.f, 0.f);
    return pair(in(k, 0) ? q[T * 2 * k] : 0.f, in(k, 1) ? q[T * (2 * k + 1)] : 0.f);
  }
  __device__ __forceinline__ uint32_t packed(const __half* q, int k) const {
    if (V == 2) return in(k, 0) ? *reinterpret_cast<const uint32_t*>(q + 2 * T * k) : 0u;
    const unsigned short* u = reinterpret_cast<const unsigned short*>(q);
    const uint32_t a = in(k, 0) ? u[T * 2 * k] : 0u, b = in(k, 1) ? u[T * (2 * k + 1)] : 0u;
    return a | b << 16;
  }
  __device__ __forceinline__ Pair load(const __half* q, int k) const { return half2_bits_to_float2(packed(q, k)); }
  __device__ __forceinline__ void store(float* q, int k, Pair x) const {
    if (V == 2) {
      if (in(k, 0)) *reinterpret_cast<float2*>(q + 2 * T * k) = x;
    } else {
      if (in(k, 0)) q[T * 2 * k] = x.x;
      if (in(k, 1)) q[T * (2 * k + 1)] = x.y;
    }
  }
  __device__ __forceinline__ void store(__half* q, int k, Pair x) const {
    const __half2 h = __floats2half2_rn(x.x, x.y);
    if (V == 2) {
      if (in(k, 0)) *reinterpret_cast<__half2*>(q + 2 * T * k) = h;
    } else {
      if (in(k, 0)) q[T * 2 * k] = __low2half(h);
      if (in(k, 1)) q[T * (2 * k + 1)] = __high2half(h);
    }
  }
};

// E pairs of a norm's parameters, packed where they are fp16.
template <int E>
struct Params {
  uint32_t w[E];
  template <typename A>
  __device__ __forceinline__ void load(const A& acc, const void* base, int fp32, int at) {
    if (fp32) return;
#pragma unroll
    for (int k = 0; k < E; ++k) w[k] = acc.packed(static_cast<const __half*>(base) + at, k);
  }
  template <typename A>
  __device__ __forceinline__ Pair get(const A& acc, const void* base, int fp32, int at, int k) const {
    return fp32 ? acc.load(static_cast<const float*>(base) + at, k) : half2_bits_to_float2(w[k]);
  }
};

// x - mean (layer norms only; no longer 0 outside the row), and 1 / sqrt(mean square +
// eps) of it; 1 without a norm.
template <int E, typename A>
__device__ __forceinline__ float centred(Pair (&x)[E], const A& acc, const NormArgs& a, float inv_width, RowSum& sum) {
  if (a.kind == NM_NORM_NONE) return 1.f;
  auto total = [&]() {
    Pair t = pair(0.f, 0.f);
#pragma unroll
    for (int k = 0; k < E; ++k) t = add2(t, x[k]);
    return t.x + t.y;
  };
  auto squares = [&]() {
    Pair t = pair(0.f, 0.f);
#pragma unroll
    for (int k = 0; k < E; ++k) t = fma2(x[k], x[k], t);
    return t.x + t.y;
  };
  if (a.kind != NM_NORM_LAYER) return 1.f / sqrtf(sum(squares()) * inv_width + a.eps);
  const float mean = __fmul_rn(sum(total()), inv_width);  // (equal elements, as a rule: nothing left)
#pragma unroll
  for (int k = 0; k < E; ++k)
    x[k] = pair(acc.in(k, 0) ? x[k].x - mean : 0.f, acc.in(k, 1) ? x[k].y - mean : 0.f);
  const Factor f = layer_factor(sum(pair(total(), squares())), inv_width, a.eps);
#pragma unroll
  for (int k = 0; k < E; ++k) x[k] = add2(x[k], pair(-f.rest, -f.rest));
  return f.r;
}

// x times a norm's r (offset + weight), plus its bias.
template <int E, typename A>
__device__ __forceinline__ void apply(Pair (&x)[E], float r, const A& acc, const NormArgs& a, const Params<E>& weight,
                                      const Params<E>& bias, int at) {
  const Pair r2 = pair(r, r);
  if (a.weight) {
    const Pair off = pair(r * a.offset, r * a.offset);
#pragma unroll
    for (int k = 0; k < E; ++k) x[k] = mul2(x[k], fma2(weight.get(acc, a.weight, a.params_fp32, at, k), r2, off));
  } else {
#pragma unroll
    for (int k = 0; k < E; ++k) x[k] = mul2(x[k], r2);
  }
  if (a.bias) {
#pragma unroll
    for (int k = 0; k < E; ++k) x[k] = add2(x[k], bias.get(acc, a.bias, a.params_fp32, at, k));
  }
}

constexpr int block_threads(int t) { return t < 256 ? 256 : t; }

// A row on T threads; blockDim.y rows a block.
template <typename S, int V, int T, int E>
__global__ void __launch_bounds__(block_threads(T), (V == 2 ? 1536 : 1024) / block_threads(T))
    residual_norm_any_kernel(const ResidualNormParams p) {
  __shared__ float part[4][32];
  pdl_launch_dependents();
  pdl_wait_previous();
  const int64_t mine = (int64_t)blockIdx.x * blockDim.y + threadIdx.y;
  const bool live = mine < p.tokens;
  const int64_t row = live ? mine : p.tokens - 1;  // (rows past the end work on the last, and store nothing)
  RowSum sum{part};
  const int at = V * (int)threadIdx.x;
  const Accesses<V, T> acc{p.width - at};
  Pair s[E], r[E];
  Params<E> weight, bias;
  const S* const res = static_cast<const S*>(p.residual) + row * p.ldr + at;
  if (p.block) {
    const __half* const b = p.block + row * p.ldb + at;
#pragma unroll
    for (int k = 0; k < E; ++k) s[k] = acc.load(b, k);
#pragma unroll
    for (int k = 0; k < E; ++k) r[k] = acc.load(res, k);
    uint32_t g[E];
    const __half* const gate = p.gate + (p.gate ? row * p.ldg + at : 0);
    if (p.gate) {
#pragma unroll
      for (int k = 0; k < E; ++k) g[k] = acc.packed(gate, k);
    }
    if (p.post.kind != NM_NORM_NONE) {
      if (p.post.weight) weight.load(acc, p.post.weight, p.post.params_fp32, at);
      const float q = centred(s, acc, p.post, p.inv_width, sum);
      if (p.post.bias) bias.load(acc, p.post.bias, p.post.params_fp32, at);
      apply(s, q, acc, p.post, weight, bias, at);
    }
    if (p.gate) {
#pragma unroll
      for (int k = 0; k < E; ++k) s[k] = mul2(s[k], half2_bits_to_float2(g[k]));
    }
    const Pair scale = pair(p.scale, p.scale), keep = pair(p.residual_scale, p.residual_scale);
#pragma unroll
    for (int k = 0; k < E; ++k) s[k] = fma2(scale, s[k], mul2(keep, r[k]));
  } else {
    const Pair keep = pair(p.residual_scale, p.residual_scale);
#pragma unroll
    for (int k = 0; k < E; ++k) s[k] = mul2(keep, acc.load(res, k));
  }
  const bool normed = p.pre.kind != NM_NORM_NONE;
  if (p.out && normed && p.pre.weight) weight.load(acc, p.pre.weight, p.pre.params_fp32, at);
  if (p.stream_out && live) {
    S* const to = static_cast<S*>(p.stream_out) + row * p.lds + at;
#pragma unroll
    for (int k = 0; k < E; ++k) acc.store(to, k, s[k]);
  }
  if (!p.out) return;
  if (normed) {
    if (p.block && (p.post.kind == NM_NORM_LAYER || (p.post.kind == NM_NORM_RMS && p.post.bias))) {
      // (a mean or a bias left the places outside other than 0)
#pragma unroll
      for (int k = 0; k < E; ++k) s[k] = pair(acc.in(k, 0) ? s[k].x : 0.f, acc.in(k, 1) ? s[k].y : 0.f);
    }
    const float q = centred(s, acc, p.pre, p.inv_width, sum);
    if (p.pre.bias) bias.load(acc, p.pre.bias, p.pre.params_fp32, at);
    apply(s, q, acc, p.pre, weight, bias, at);
  }
  if (live) {
    __half* const to = p.out + row * p.ldo + at;
#pragma unroll
    for (int k = 0; k < E; ++k) acc.store(to, k, s[k]);
  }
}

// Whether all rows begin on even elements and have an even number of them.
template <typename S>
bool even_rows(const ResidualNormParams& p) {
  auto even = [](const void* a, size_t size) { return reinterpret_cast<uintptr_t>(a) % (2 * size) == 0; };
  const NormArgs* norms[2] = {&p.post, &p.pre};
  for (const NormArgs* n : norms)
    if (!even(n->weight, n->params_fp32 ? 4 : 2) || !even(n->bias, n->params_fp32 ? 4 : 2)) return false;
  return p.width % 2 == 0 && even(p.residual, sizeof(S)) && p.ldr % 2 == 0 && even(p.stream_out, sizeof(S)) &&
         p.lds % 2 == 0 && even(p.block, 2) && p.ldb % 2 == 0 && even(p.gate, 2) && p.ldg % 2 == 0 && even(p.out, 2) &&
         p.ldo % 2 == 0;
}

// n accesses of a row.
template <typename S, int V>
cudaError_t launch_any(const ResidualNormParams& p, int n, cudaStream_t stream) {
  // V 1: 2 E accesses a thread, V 2: E
  constexpr int P = V == 1 ? 2 : 1;
  auto fits = [&](int threads, int e) { return n <= threads * P * e; };
  if (fits(32, 2)) return launch_rows(residual_norm_any_kernel<S, V, 32, 2>, p, 32, stream);
  if (fits(32, 4)) return launch_rows(residual_norm_any_kernel<S, V, 32, 4>, p, 32, stream);
  if (fits(32, 8)) return launch_rows(residual_norm_any_kernel<S, V, 32, 8>, p, 32, stream);
  if (fits(128, 4)) return launch_rows(residual_norm_any_kernel<S, V, 128, 4>, p, 128, stream);
  if (fits(128, 6)) return launch_rows(residual_norm_any_kernel<S, V, 128, 6>, p, 128, stream);
  if (fits(128, 8)) return launch_rows(residual_norm_any_kernel<S, V, 128, 8>, p, 128, stream);
  if (fits(512, 4)) return launch_rows(residual_norm_any_kernel<S, V, 512, 4>, p, 512, stream);
  if (fits(512, 6)) return launch_rows(residual_norm_any_kernel<S, V, 512, 6>, p, 512, stream);
  if (V == 1 || fits(512, 8)) return launch_rows(residual_norm_any_kernel<S, V, 512, 8>, p, 512, stream);
  return launch_rows(residual_norm_any_kernel<S, 2, 1024, 8>, p, 1024, stream);
}

template <typename S>
cudaError_t launch_stream(const ResidualNormParams& p, cudaStream_t stream) {
  return even_rows<S>(p) ? launch_any<S, 2>(p, p.width / 2, stream) : launch_any<S, 1>(p, p.width, stream);
}

}  // namespace

bool takes_any_rows(const ResidualNormParams& p, int stream_fp32) {
  return p.width <= 8192 || (p.width <= 16384 && (stream_fp32 ? even_rows<float>(p) : even_rows<__half>(p)));
}

cudaError_t launch_any_rows(const ResidualNormParams& p, int stream_fp32, cudaStream_t stream) {
  return stream_fp32 ? launch_stream<float>(p, stream) : launch_stream<__half>(p, stream);
}

}  // namespace nmk
