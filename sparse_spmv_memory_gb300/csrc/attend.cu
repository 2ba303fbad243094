// attend.cu -- attention of drafted nodes over a paged cache
// (nm_tree_attention), for few query rows per key head; attend_wide.cuh has the
// kernel for many.
//
// For a node's query q and the rows (k_j, v_j) that it sees,
//   o = sum_j p_j v_j / sum_j p_j,  p_j = 2^(s_j - m),  s_j = scale log2(e) q.k_j,
// with m the largest score so far: a new maximum m' scales what was summed by
// 2^(m - m'), so one pass over the cache does, and parts with their own m join
// by the same rule.
#include <cuda_fp16.h>
#include <cuda_runtime.h>
#include <stdint.h>

#include "attend.cuh"
#include "decode.h"
#include "device.cuh"
#include "kernels.h"
#include "widen.cuh"

namespace nmk {
namespace {

// ---- loads and conversions -----------------------------------------------------
template <int WORDS>  // 2, 4 or 8 words; zeros where !on
__device__ __forceinline__ void load_words(const uint8_t* at, bool on, uint32_t* r) {
#pragma unroll
  for (int i = 0; i < WORDS; ++i) r[i] = 0;
  if (!on) return;
  if (WORDS == 8) {
    uint32_t v[8];
    ld_stream_v8(reinterpret_cast<const uint32_t*>(at), v);
#pragma unroll
    for (int i = 0; i < 8; ++i) r[i] = v[i];
  } else if (WORDS == 4) {
    const uint4 v = ld_stream_v4(at);
    r[0] = v.x, r[1] = v.y, r[2] = v.z, r[3] = v.w;
  } else {
    asm volatile("ld.global.nc.L1::no_allocate.v2.u32 {%0,%1}, [%2];"
                 : "=r"(r[0]), "=r"(r[1])
                 : "l"(at));
  }
}

__device__ __forceinline__ void mma16816(float (&d)[4], const uint32_t (&a)[4], uint32_t b0,
                                         uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, "
      "{%0,%1,%2,%3};"
      : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
      : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}

__device__ __forceinline__ uint32_t pack_half2(float a, float b) {
  const __half2 h = __floats2half2_rn(a, b);
  return *reinterpret_cast<const uint32_t*>(&h);
}

// ---- the kernel for few rows ------------------------------------------------------
// mma.sync.m16n8k16 with the query rows as A (16 at a time), a head's rows of K
// as B for the scores, and of V as B for the sums.  K and V come from HBM
// straight into the registers the MMA reads them from, 32 bytes a lane: the
// order of a product's k index is free as long as A and B agree, and so is the
// order of the output's columns.  Lane 4g + q
//   - of K holds of row g (per 8 positions) the elements that the k slots of q
//     are given to: any 4 per MMA, so whole 16- to 32-byte pieces of the row;
//   - of V holds of the rows 2q, 2q+1, 2q+8, 2q+9 the piece g of the row: its
//     column t of MMA n-tile t.  Two rows' halves are paired by byte permutes.
// No shared memory, no barrier, until a block's warps join their sums.  A warp
// takes every NW-th unit of the block's part.
//
// What bounds it: the bytes that a warp's registers have in flight, and with codes
// the chain load, widen, product, weight, permute, product, which two or three
// warps a scheduler do not cover (35 % of issue slots, 16 % of the tensor pipe).
// Hence 12 warps of 16 positions for codes (8 rows over 100000 positions, e4m3:
// 69.0 us; 8 warps of 32: 72.4, 10: 73.4, 14: 92.4 and 16: 94.9, which spill),
// and 8 warps for fp16, whose rows take twice the registers.  1 token over 500
// positions: 9.1 us, of which launch, lengths and the table's look-up some 3, the
// loads 1.5, and joining warps, then blocks, 3.
constexpr int kNarrowRows = 16;
constexpr float kLift = 14.0f;

template <int D, int TYPE>
struct Narrow {
  static constexpr bool F16 = TYPE == kCacheFp16;
  static constexpr int NW = F16 ? 8 : 12;       // warps
  static constexpr int NG = 2;                // groups of 8 positions in a unit
  static constexpr int UK = 8 * NG;           // positions of a unit
  static constexpr int KS = D / 16;           // MMA k steps of a score
  static constexpr int NT = D / 8;            // n-tiles of an output row
  static constexpr int KW = D * (F16 ? 2 : 1) / 16;  // words of K a lane holds per group
  static constexpr int VW = D * (F16 ? 2 : 1) / 32;  // words of V a lane holds per row
  // the element of k step ks, MMA slots 2q, 2q+1, 2q+8, 2q+9: four from here
  static __device__ __forceinline__ int k_elem(int ks, int q) {
    return F16 ? (ks >> 2) * 64 + 16 * q + 4 * (ks & 3) : (D / 4) * q + 4 * ks;
  }
};

template <int D, int TYPE>
__global__ void __launch_bounds__(Narrow<D, TYPE>::NW * 32, 1) attend_narrow_kernel(AttendParams p) {
  using N = Narrow<D, TYPE>;
  constexpr bool F16 = N::F16;
  constexpr int ROWS = kNarrowRows, NW = N::NW, NTH = NW * 32, PITCH = D + 4;
  using Sched = Schedule<ROWS, N::UK, NTH>;
  extern __shared__ __align__(16) uint8_t dyn[];
  float* so = reinterpret_cast<float*>(dyn);                     // [NW][ROWS][PITCH]
  __shared__ uint4 sq[N::KS][32];                            // A fragments of the queries
  __shared__ uint64_t smask[ROWS];
  __shared__ float sm[NW][ROWS], sl[NW][ROWS], sf[NW][ROWS];
  __shared__ float row_m[ROWS], row_l[ROWS];
  pdl_launch_dependents();
  pdl_wait_previous();
  Sched sched;
  if (!sched.init(p, NW)) return;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, g = lane >> 2, q = lane & 3;
  const int G = p.q_heads / p.c.kv_heads;
  const Heads heads(G);
  const float cs = p.scale * kLog2e;
  int* counters = reinterpret_cast<int*>(p.workspace);
  float* slots = reinterpret_cast<float*>(p.workspace + attend_counter_bytes(gridDim.x));

  Span w;
  SeqInfo si;
  while (sched.next(p, w, si)) {
    const int rows = min(ROWS, si.n * G - w.rt * ROWS);
    __syncthreads();  // the shared arrays of the last item are free
    for (int i = threadIdx.x; i < N::KS * 32; i += NTH) {
      const int ks = i / 32, ln = i % 32;
      const int e = N::k_elem(ks, ln & 3);
      uint2 v[2];
#pragma unroll
      for (int k = 0; k < 2; ++k) {
        const int r = (ln >> 2) + 8 * k, rr = w.rt * ROWS + r;
        v[k] = make_uint2(0, 0);
        if (r < rows)
          v[k] = *reinterpret_cast<const uint2*>(p.q + (int64_t)(si.first + heads.node(rr)) * p.ldq +
                                                 (w.h * G + heads.head(rr)) * D + e);
      }
      sq[ks][ln] = make_uint4(v[0].x, v[1].x, v[0].y, v[1].y);
    }
    for (int r = threadIdx.x; r < ROWS; r += NTH) {
      const int node = heads.node(w.rt * ROWS + r);
      smask[r] = r >= rows ? 0ull : p.tree_mask ? p.tree_mask[si.first + node] : (2ull << node) - 1ull;
    }
    __syncthreads();

    float o[N::NT][4], m[2], l[2];
#pragma unroll
    for (int t = 0; t < N::NT; ++t)
#pragma unroll
      for (int i = 0; i < 4; ++i) o[t][i] = 0.0f;
    m[0] = m[1] = -INFINITY;
    l[0] = l[1] = 0.0f;
    const int32_t* table = p.table + (int64_t)w.s * p.ld_table;
    uint32_t kr[N::NG][N::KW], vr[N::NG][2][N::VW];
    float ksc[N::NG][2], vsc[N::NG][2];
    RowAt at[N::NG];
    int32_t entry[N::NG];  // table entries of the unit after the one being loaded

    auto look_up = [&](int u) {
#pragma unroll
      for (int c = 0; c < N::NG; ++c) {
        const int64_t pos = (int64_t)u * N::UK + 8 * c;
        entry[c] = u < w.u1 && pos < si.len ? table[pos >> p.c.page_shift] : -1;
      }
    };
    auto find = [&](int u) {
#pragma unroll
      for (int c = 0; c < N::NG; ++c)
        at[c] = group_at<D>(p, entry[c], w.h, (int64_t)u * N::UK + 8 * c);
    };
    auto load_k = [&](int u) {
#pragma unroll
      for (int c = 0; c < N::NG; ++c) {
        const int64_t pos = (int64_t)u * N::UK + 8 * c;
        const bool on = at[c].code >= 0 && pos + g < si.len;
        const uint8_t* base = p.c.k + (at[c].code + g * D) * (F16 ? 2 : 1);
        constexpr int PIECE = N::KW > 8 ? 8 : N::KW;  // words of a load
#pragma unroll
        for (int i = 0; i < N::KW / PIECE; ++i)
          load_words<PIECE>(base + (i * 4 + q) * PIECE * 4, on, &kr[c][i * PIECE]);
        if (!F16) {
#pragma unroll
          for (int i = 0; i < 2; ++i) {
            const bool son = at[c].code >= 0 && pos + 2 * q + i < si.len;
            ksc[c][i] = son ? p.c.k_scale[at[c].scale + 2 * q + i] : 0.0f;
            vsc[c][i] = son ? p.c.v_scale[at[c].scale + 2 * q + i] : 0.0f;
          }
        }
      }
    };
    auto load_v = [&](int u) {
#pragma unroll
      for (int c = 0; c < N::NG; ++c) {
        const int64_t pos = (int64_t)u * N::UK + 8 * c;
#pragma unroll
        for (int i = 0; i < 2; ++i) {
          const int r = 2 * q + i;
          const bool on = at[c].code >= 0 && pos + r < si.len;
          load_words<N::VW>(p.c.v + (at[c].code + r * D) * (F16 ? 2 : 1) + g * N::VW * 4, on, vr[c][i]);
        }
      }
    };

    int u = w.u0 + warp;
    if (u < w.u1) {
      look_up(u);
      find(u);
      load_k(u);
      load_v(u);
      look_up(u + NW);
    }
    for (; u < w.u1; u += NW) {
      const int64_t pos0 = (int64_t)u * N::UK;
      uint32_t there = 0;
#pragma unroll
      for (int c = 0; c < N::NG; ++c) there |= at[c].code >= 0 ? 1u << c : 0u;
      // ---- scores: row g (i = 0, 1) and g + 8 (2, 3) of positions 8c + 2q, + 1
      float s[N::NG][4];
#pragma unroll
      for (int c = 0; c < N::NG; ++c)
#pragma unroll
        for (int i = 0; i < 4; ++i) s[c][i] = 0.0f;
#pragma unroll
      for (int ks = 0; ks < N::KS; ++ks) {
        const uint4 f = sq[ks][lane];
        const uint32_t a[4] = {f.x, f.y, f.z, f.w};
#pragma unroll
        for (int c = 0; c < N::NG; ++c) {
          uint32_t b0, b1;
          if (F16) {
            b0 = kr[c][2 * ks];
            b1 = kr[c][2 * ks + 1];
          } else {
            widen4<TYPE>(kr[c][ks], b0, b1);
          }
          mma16816(s[c], a, b0, b1);
        }
      }
      float vs[N::NG][2], lv[N::NG][2];
#pragma unroll
      for (int c = 0; c < N::NG; ++c)
#pragma unroll
        for (int i = 0; i < 2; ++i) {
          const float f = F16 ? cs : cs * ksc[c][i];
          s[c][i] *= f;
          s[c][2 + i] *= f;
          if (!F16) {
            vs[c][i] = vsc[c][i];
            lv[c][i] = fmaxf(log2_fast(vsc[c][i]), -40.0f);
          }
        }
      if (u + NW < w.u1) {
        find(u + NW);
        load_k(u + NW);
        look_up(u + 2 * NW);
      }
      // ---- masks: the last units have the nodes, or end
      const bool edge = pos0 + N::UK > si.ctx || there != (1u << N::NG) - 1u;
      uint32_t seen[2] = {~0u, ~0u};  // bit 2c + i: row sees position 8c + 2q + i
      if (edge) {
#pragma unroll
        for (int k = 0; k < 2; ++k) {
          const uint64_t bits = smask[g + 8 * k];
          uint32_t see = 0;
#pragma unroll
          for (int c = 0; c < N::NG; ++c)
#pragma unroll
            for (int i = 0; i < 2; ++i) {
              const int64_t pos = pos0 + 8 * c + 2 * q + i, j = pos - si.ctx;
              const bool on =
                  ((there >> c) & 1u) && pos < si.len && (j < 0 || ((bits >> (j & 63)) & 1ull));
              see |= on ? 1u << (2 * c + i) : 0u;
              if (!on) s[c][2 * k + i] = -INFINITY;
            }
          seen[k] = see;
        }
      }
      // ---- weights: the largest is 2^kLift, so that they are fp16 at its full
      // precision down to 2^-28 of it: many small ones add up
      uint32_t a[N::NG / 2][4];
      float keep[2];
      bool grew = false;
#pragma unroll
      for (int k = 0; k < 2; ++k) {
        float top = -INFINITY;
#pragma unroll
        for (int c = 0; c < N::NG; ++c)
#pragma unroll
          for (int i = 0; i < 2; ++i) top = fmaxf(top, F16 ? s[c][2 * k + i] : s[c][2 * k + i] + lv[c][i]);
        top = fmaxf(top, __shfl_xor_sync(0xFFFFFFFFu, top, 1));
        top = fmaxf(top, __shfl_xor_sync(0xFFFFFFFFu, top, 2));
        const float next = fmaxf(m[k], top - kLift);
        keep[k] = m[k] == -INFINITY ? 0.0f : exp2_fast(m[k] - next);
        grew |= next != m[k];
        l[k] *= keep[k];
        m[k] = next;
        const float base = next == -INFINITY ? 0.0f : next;
#pragma unroll
        for (int c = 0; c < N::NG; ++c) {
          float e[2];
#pragma unroll
          for (int i = 0; i < 2; ++i) {
            e[i] = exp2_fast(s[c][2 * k + i] - base);
            l[k] += e[i];
            if (!F16) e[i] = (seen[k] >> (2 * c + i)) & 1u ? e[i] * vs[c][i] : 0.0f;
          }
          a[c / 2][(c & 1) * 2 + k] = pack_half2(e[0], e[1]);
        }
      }
      if (__any_sync(0xFFFFFFFFu, grew)) {
#pragma unroll
        for (int k = 0; k < 2; ++k)
#pragma unroll
          for (int t = 0; t < N::NT; ++t) {
            o[t][2 * k] *= keep[k];
            o[t][2 * k + 1] *= keep[k];
          }
      }
      // ---- sums
      uint32_t bad = 0;  // bit 2c + i: the value row of position 8c + 2q + i is not finite
#pragma unroll
      for (int c2 = 0; c2 < N::NG / 2; ++c2) {
#pragma unroll
        for (int j = 0; j < N::VW; ++j) {
          // b[x][y]: rows (2q, 2q+1) of group 2 c2 + y, columns of n-tile x
          uint32_t b[4][2];
#pragma unroll
          for (int y = 0; y < 2; ++y) {
            const uint32_t r0 = vr[2 * c2 + y][0][j], r1 = vr[2 * c2 + y][1][j];
            if (F16) {
              b[0][y] = byte_perm(r0, r1, 0x5410);
              b[1][y] = byte_perm(r0, r1, 0x7632);
            } else {
              widen4<TYPE>(byte_perm(r0, r1, 0x5140), b[0][y], b[1][y]);
              widen4<TYPE>(byte_perm(r0, r1, 0x7362), b[2][y], b[3][y]);
            }
            if (edge) {
#pragma unroll
              for (int x = 0; x < (F16 ? 2 : 4); ++x) {
                const uint32_t h = bad_halves(b[x][y]);
                if (h) {
                  bad |= h << (2 * (2 * c2 + y));
                  b[x][y] &= (h & 1u ? 0u : 0xFFFFu) | (h & 2u ? 0u : 0xFFFF0000u);
                }
              }
            }
          }
#pragma unroll
          for (int x = 0; x < (F16 ? 2 : 4); ++x)
            mma16816(o[j * (F16 ? 2 : 4) + x], a[c2], b[x][0], b[x][1]);
        }
      }
      if (u + NW < w.u1) load_v(u + NW);
      if (edge) {
        // a value row with an infinity or NaN entered as zeros there, so that
        // only the rows that see it are spoilt
        bad |= __shfl_xor_sync(0xFFFFFFFFu, bad, 4);
        bad |= __shfl_xor_sync(0xFFFFFFFFu, bad, 8);
        bad |= __shfl_xor_sync(0xFFFFFFFFu, bad, 16);
#pragma unroll
        for (int k = 0; k < 2; ++k) {
          uint32_t hit = bad & seen[k];
          hit |= __shfl_xor_sync(0xFFFFFFFFu, hit, 1);
          hit |= __shfl_xor_sync(0xFFFFFFFFu, hit, 2);
          if (hit) {
#pragma unroll
            for (int t = 0; t < N::NT; ++t) o[t][2 * k] = o[t][2 * k + 1] = __uint_as_float(0x7FC00000u);
          }
        }
      }
    }

    // ---- join the warps: every warp's sums, maxima and weights to shared memory
#pragma unroll
    for (int k = 0; k < 2; ++k) {
      float sum = l[k];
      sum += __shfl_xor_sync(0xFFFFFFFFu, sum, 1);
      sum += __shfl_xor_sync(0xFFFFFFFFu, sum, 2);
      const int r = g + 8 * k;
      if (q == 0) {
        sm[warp][r] = m[k];
        sl[warp][r] = sum;
      }
      if (r >= rows) continue;
      float* dst = so + ((size_t)warp * ROWS + r) * PITCH;
      // n-tile t, columns 2q, 2q+1 are elements (D/8) 2q + t and (D/8)(2q+1) + t
#pragma unroll
      for (int t = 0; t < N::NT; ++t) {
        dst[(D / 8) * 2 * q + t] = o[t][2 * k];
        dst[(D / 8) * (2 * q + 1) + t] = o[t][2 * k + 1];
      }
    }
    __syncthreads();
    for (int r = threadIdx.x; r < ROWS; r += NTH) {
      float M = -INFINITY, tot = 0.0f;
      for (int x = 0; x < NW; ++x) M = fmaxf(M, sm[x][r]);
      const float base = M == -INFINITY ? 0.0f : M;
      for (int x = 0; x < NW; ++x) {
        const float f = exp2_fast(sm[x][r] - base);
        sf[x][r] = f;
        tot += sl[x][r] * f;
      }
      row_m[r] = M;
      row_l[r] = tot;
    }
    __syncthreads();
    const bool whole = w.u0 == 0 && w.u1 == w.nu;
    float* slot = slots + part_slot(blockIdx.x, sched.per, w.start) * attend_slot_floats(ROWS, D);
    for (int i = threadIdx.x; i < rows * (D / 4); i += NTH) {
      const int r = i / (D / 4), d = i % (D / 4) * 4;
      float4 x = make_float4(0, 0, 0, 0);
#pragma unroll
      for (int y = 0; y < NW; ++y) {
        const float4 v = *reinterpret_cast<const float4*>(so + ((size_t)y * ROWS + r) * PITCH + d);
        const float f = sf[y][r];
        x.x += v.x * f, x.y += v.y * f, x.z += v.z * f, x.w += v.w * f;
      }
      if (whole) {
        const float inv = row_l[r] == 0.0f ? 0.0f : 1.0f / row_l[r];
        const int rr = w.rt * ROWS + r;
        __half* dst = p.out + (int64_t)(si.first + heads.node(rr)) * p.ldo + (w.h * G + heads.head(rr)) * D + d;
        *reinterpret_cast<uint2*>(dst) =
            make_uint2(pack_half2(x.x * inv, x.y * inv), pack_half2(x.z * inv, x.w * inv));
      } else {
        *reinterpret_cast<float4*>(slot + (size_t)r * D + d) = x;
      }
    }
    for (int r = threadIdx.x; r < rows; r += NTH) {
      if (whole) {
        const int rr = w.rt * ROWS + r;
        if (p.lse)
          p.lse[(int64_t)(si.first + heads.node(rr)) * p.q_heads + w.h * G + heads.head(rr)] =
              row_l[r] == 0.0f ? -INFINITY : (row_m[r] + log2f(row_l[r])) * kLn2;
      } else {
        slot[(size_t)ROWS * D + r] = row_m[r];
        slot[(size_t)ROWS * D + ROWS + r] = row_l[r];
      }
    }
    if (whole) continue;

    // ---- join the blocks: the last one to store its part adds all of them
    const int64_t b0 = sched.block_of(w.start), b1 = sched.block_of(w.start + w.nu - 1);
    const int parts = (int)(b1 - b0 + 1);
    if (!last_of_item(counters + b0, parts)) continue;
    float* factor = so;  // [parts][ROWS]
    auto part = [&](int y) {
      return slots + part_slot(b0 + y, sched.per, w.start) * attend_slot_floats(ROWS, D);
    };
    for (int r = threadIdx.x; r < rows; r += NTH) {
      const float2 ml = join_ml(parts, ROWS, [&](int y) { return part(y) + ROWS * D + r; });
      row_m[r] = ml.x == -INFINITY ? 0.0f : ml.x;
      row_l[r] = ml.y == 0.0f ? 0.0f : 1.0f / ml.y;
      const int rr = w.rt * ROWS + r;
      if (p.lse)
        p.lse[(int64_t)(si.first + heads.node(rr)) * p.q_heads + w.h * G + heads.head(rr)] =
            ml.y == 0.0f ? -INFINITY : (ml.x + log2f(ml.y)) * kLn2;
    }
    __syncthreads();
    for (int i = threadIdx.x; i < parts * rows; i += NTH) {
      const int y = i / rows, r = i % rows;
      factor[y * ROWS + r] = exp2_fast(__ldcg(part(y) + ROWS * D + r) - row_m[r]) * row_l[r];
    }
    __syncthreads();
    for (int i = threadIdx.x; i < rows * (D / 4); i += NTH) {
      const int r = i / (D / 4), d = i % (D / 4) * 4;
      float4 x = make_float4(0, 0, 0, 0);
      for (int y0 = 0; y0 < parts; y0 += 8) {
        float4 v[8];
#pragma unroll
        for (int j = 0; j < 8; ++j)
          v[j] = __ldcg(reinterpret_cast<const float4*>(part(min(y0 + j, parts - 1)) + (size_t)r * D + d));
#pragma unroll
        for (int j = 0; j < 8; ++j) {
          const float f = y0 + j < parts ? factor[(y0 + j) * ROWS + r] : 0.0f;
          x.x += v[j].x * f, x.y += v[j].y * f, x.z += v[j].z * f, x.w += v[j].w * f;
        }
      }
      const int rr = w.rt * ROWS + r;
      *reinterpret_cast<uint2*>(p.out + (int64_t)(si.first + heads.node(rr)) * p.ldo +
                                (w.h * G + heads.head(rr)) * D + d) =
          make_uint2(pack_half2(x.x, x.y), pack_half2(x.z, x.w));
    }
  }
}

template <int D, int TYPE>
cudaError_t launch_narrow(const AttendParams& p, int sms, cudaStream_t stream) {
  constexpr size_t smem = (size_t)Narrow<D, TYPE>::NW * kNarrowRows * (D + 4) * sizeof(float);
  auto* k = attend_narrow_kernel<D, TYPE>;
  static int done[64];
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  if (dev >= 64 || !__atomic_load_n(&done[dev], __ATOMIC_ACQUIRE)) {
    e = cudaFuncSetAttribute(k, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem);
    if (e != cudaSuccess) return e;
    if (dev < 64) __atomic_store_n(&done[dev], 1, __ATOMIC_RELEASE);
  }
  return launch_kernel(k, sms, Narrow<D, TYPE>::NW * 32, smem, stream, kFlagPdl, p);
}

}  // namespace

size_t attend_workspace_bytes(int64_t seqs, int q_heads, int kv_heads, int head_dim, int max_nodes,
                              int sms) {
  // (the narrow kernel's parts are smaller, and it has no heads of items)
  const int rows = max_nodes * (q_heads / kv_heads), wide = wide_item_rows(wide_mode(rows));
  return attend_counter_bytes(sms) + join_head_bytes(seqs * kv_heads * ((rows + wide - 1) / wide)) +
         (size_t)sms * 2 * attend_slot_floats(wide, head_dim) * sizeof(float);
}

// The narrow kernel has 16 rows of an item, so from 17 on it would read K and V
// a second time, or hold two row tiles in registers.  The latter, with 32 rows:
// 103.5, 102 and 105 us (fp16, e4m3, int8) over 100000 positions, and 35.9 us
// (fp16) over 32 sequences of 200, where the wide kernel takes 72.9, 84.6, 75.4
// and 25.5; over one of 500 (fp16) 13.3 and 15.5, the one case that it loses.
// With up to 16 rows the narrow kernel begins and ends 2 to 4 us sooner, but has
// fewer bytes of an fp16 cache in flight than the wide one's ring.  Of 8 rows and
// 8 key heads (narrow, wide): 500 positions 9.3, 13.1 us; 4000 14.3, 16.8; 16000
// 23.1, 25.3; 32000 35.0, 33.6; 100000 82.3, 70.8; 16 sequences of 4000 49.5,
// 46.1; 64 of 1500 79.0, 67.0: even at 64 to 130 MB, taken by what the tables can
// hold, since the lengths are on the device.  Codes: 8 rows over 100000 positions
// 69.3, 84 (e4m3) and 70.4, 72.9 (int8): the wide kernel's widening costs more.
cudaError_t launch_attend(const AttendParams& p, int head_dim, int type, int sms,
                          cudaStream_t stream) {
  const double held = (double)p.seqs * (double)p.table_cols * (double)(1 << p.c.page_shift) * p.c.kv_heads * head_dim * 4;
  if (p.max_nodes * (p.q_heads / p.c.kv_heads) > kNarrowRows || (type == kCacheFp16 && held >= sms * 655360.0))
    return type == kCacheFp16   ? launch_attend_wide<kCacheFp16>(p, head_dim, sms, stream)
           : type == kCacheE4m3 ? launch_attend_wide<kCacheE4m3>(p, head_dim, sms, stream)
                                : launch_attend_wide<kCacheInt8>(p, head_dim, sms, stream);
  if (head_dim == 128) {
    if (type == kCacheFp16) return launch_narrow<128, kCacheFp16>(p, sms, stream);
    if (type == kCacheE4m3) return launch_narrow<128, kCacheE4m3>(p, sms, stream);
    return launch_narrow<128, kCacheInt8>(p, sms, stream);
  }
  if (type == kCacheFp16) return launch_narrow<64, kCacheFp16>(p, sms, stream);
  if (type == kCacheE4m3) return launch_narrow<64, kCacheE4m3>(p, sms, stream);
  return launch_narrow<64, kCacheInt8>(p, sms, stream);
}

}  // namespace nmk
