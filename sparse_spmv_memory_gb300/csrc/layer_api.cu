// layer_api.cu -- the extern "C" boundary of nm_layer.h: argument checks, plans and
// dispatch.
#include <cuda_fp16.h>
#include <cuda_runtime.h>
#include <math.h>
#include <stdint.h>

#include <initializer_list>

#include "../../include/nm_layer.h"
#include "kernels.h"
#include "layer.h"

using namespace nmk;

namespace {

constexpr int64_t kMax31 = (int64_t)1 << 31;

bool aligned(const void* p, uintptr_t a) { return (reinterpret_cast<uintptr_t>(p) & (a - 1)) == 0; }

struct Array {
  const void* at;
  size_t bytes;
};

bool overlap(const Array& a, const Array& b) {
  const uintptr_t a0 = reinterpret_cast<uintptr_t>(a.at), b0 = reinterpret_cast<uintptr_t>(b.at);
  return a.at && b.at && a.bytes && b.bytes && a0 < b0 + b.bytes && b0 < a0 + a.bytes;
}

bool overlaps_any(const Array& a, std::initializer_list<Array> others) {
  for (const Array& o : others)
    if (overlap(a, o)) return true;
  return false;
}

// Bytes from the first to the last element of `rows` rows of `width`, `ld` apart.
size_t span(int64_t rows, int64_t ld, int64_t width, size_t size) {
  return rows > 0 ? (size_t)((rows - 1) * ld + width) * size : 0;
}

int status(cudaError_t e) { return e == cudaSuccess ? NM_OK : NM_ERR_CUDA; }

// ---- nm_linear -------------------------------------------------------------------
// Shared memory that a block's x tile leaves for its rows' fp32 sums, at least: blocks
// whose rows would take more than there is are made smaller (a larger grid), and a
// tile that leaves less is cut into column slices.
constexpr size_t kSumBytes = 8 * 1024;

enum class Path { kSpmv, kSpmm, kPrefill };

struct LinearPlan {
  Path path;
  SpmvPlan spmv;
  SpmvParams vp;
  SpmmPlan spmm;
  SpmmParams mp;
  LinearTcPlan tc;
  int sms;
  size_t workspace;
};

// Blocks of a multiple of the SMs' number whose `width` sums a row fit in `room` bytes.
int grid_for(int64_t rows, int width, size_t room, int sms, int grid) {
  const int64_t most = (int64_t)(room / (sizeof(float) * width)) - 2;  // rows a block may have
  const int64_t want = (rows + most - 1) / most;
  return want <= grid ? grid : (int)((want + sms - 1) / sms * sms);
}

int linear_plan(int64_t rows, int64_t cols, int64_t tokens, int gated, LinearPlan* pl) {
  DeviceInfo d;
  if (device_info(&d) != cudaSuccess) return NM_ERR_CUDA;
  pl->sms = d.sms;
  pl->workspace = 0;
  const int64_t units = gated ? rows / 2 : rows;
  if (tokens == 1) {
    pl->path = Path::kSpmv;
    const int st = make_spmv_plan(rows, cols, -1, 0, &pl->spmv, &pl->vp);
    const size_t tile = st == NM_OK ? spmv_smem_bytes(pl->vp.pitch, pl->spmv.warps) : 0;
    if (st == NM_OK && tile + kSumBytes <= (size_t)d.smem_optin) {
      pl->spmv.grid = grid_for(rows, 1, (size_t)d.smem_optin - tile, d.sms, pl->spmv.grid);
      if (pl->spmv.grid > units) pl->spmv.grid = (int)units;
      return NM_OK;
    }
  }
  if (tokens <= 8) {  // (one token: rows too long for a block's shared memory)
    pl->path = Path::kSpmm;
    int slices = 0;
    for (;;) {
      const int st = make_spmm_plan(rows, cols, (int)tokens, -1, 0, slices, &pl->spmm, &pl->mp);
      if (st != NM_OK) return st;
      if (pl->mp.slices > 1) break;
      const size_t tile = spmm_smem_bytes(pl->mp.pitch, pl->spmm.warps, pl->spmm.bp, 0);
      if (tile + kSumBytes <= (size_t)d.smem_optin) {
        pl->spmm.grid = grid_for(rows, pl->spmm.bp, (size_t)d.smem_optin - tile, d.sms, pl->spmm.grid);
        if (pl->spmm.grid > units) pl->spmm.grid = (int)units;
        return NM_OK;
      }
      slices = 2;
    }
    pl->workspace = spmm_workspace_for(pl->mp);
    return NM_OK;
  }
  if ((rows + 127) / 128 > 65535) return NM_ERR_SHAPE;
  pl->path = Path::kPrefill;
  pl->tc = linear_tc_plan(rows, (int)(cols / 32), tokens, d.sms);
  return NM_OK;
}

bool linear_shape_ok(int64_t rows, int64_t cols, int64_t tokens) {
  return rows >= 0 && rows < kMax31 && cols > 0 && cols < kMax31 && cols % 32 == 0 && tokens >= 0 &&
         tokens < kMax31;
}

// ---- nm_residual_norm ------------------------------------------------------------
int check_norm(const nm_norm* n, NormArgs* a) {
  a->kind = n ? n->kind : NM_NORM_NONE;
  a->weight = a->bias = nullptr;
  a->params_fp32 = 0;
  a->offset = a->eps = 0.f;
  if (a->kind == NM_NORM_NONE) return NM_OK;
  if (a->kind != NM_NORM_RMS && a->kind != NM_NORM_LAYER) return NM_ERR_SHAPE;
  if (!isfinite(n->offset) || !isfinite(n->eps) || n->eps < 0.f) return NM_ERR_SHAPE;
  const uintptr_t size = n->params_fp32 ? 4 : 2;
  if (!aligned(n->weight, size) || !aligned(n->bias, size)) return NM_ERR_ALIGN;
  a->weight = n->weight;
  a->bias = n->bias;
  a->params_fp32 = n->params_fp32 != 0;
  a->offset = n->offset;
  a->eps = n->eps;
  return NM_OK;
}

}  // namespace

extern "C" {

size_t nm_linear_workspace_bytes(int64_t rows, int64_t cols, int64_t tokens) {
  LinearPlan pl;
  if (!linear_shape_ok(rows, cols, tokens) || rows == 0 || tokens == 0 ||
      linear_plan(rows, cols, tokens, 0, &pl) != NM_OK)
    return 0;
  return pl.workspace;
}

// nm_linear with the limit of the tensor-core kernel's waits and the self-test's stall.
static int linear_call(const void* values, const uint32_t* masks, int64_t rows, int64_t cols, const void* X,
                       int64_t ldx, int64_t tokens, const nm_epilogue* epilogue, void* Y, int64_t ldy,
                       void* workspace, size_t workspace_bytes, void* stream, uint64_t wait_limit_ns, int stall) {
  if (!epilogue) return NM_ERR_NULL;
  if (rows != 0 && tokens != 0 && (!values || !masks || !X || !Y)) return NM_ERR_NULL;
  const nm_epilogue& e = *epilogue;
  if (!linear_shape_ok(rows, cols, tokens) || (e.gated && rows % 2)) return NM_ERR_SHAPE;
  const int64_t n = e.gated ? rows / 2 : rows;
  if (ldx < cols || ldx >= kMax31 || ldy < n || ldy >= kMax31 ||
      (e.residual && (e.ldres < n || e.ldres >= kMax31)) || e.activation < NM_ACT_NONE ||
      e.activation > NM_ACT_GELU_TANH || !isfinite(e.scale))
    return NM_ERR_SHAPE;
  if (!aligned(values, 32) || !aligned(masks, 4) || !aligned(X, 16) || ldx % 8 != 0 ||
      !aligned(Y, 2) || !aligned(e.bias, 2) || !aligned(e.residual, 2) || !aligned(workspace, 16))
    return NM_ERR_ALIGN;
  if (rows == 0 || tokens == 0) return NM_OK;
  const Array w{values, (size_t)rows * cols}, m{masks, (size_t)rows * cols / 8},
      x{X, span(tokens, ldx, cols, 2)}, b{e.bias, (size_t)rows * 2},
      res{e.residual, span(tokens, e.ldres, n, 2)}, y{Y, span(tokens, ldy, n, 2)};
  const bool in_place = e.residual == Y && (e.ldres == ldy || tokens == 1);
  if (overlaps_any(y, {w, m, x, b}) || (!in_place && overlap(y, res))) return NM_ERR_ALIAS;
  LinearPlan pl;
  const int st = linear_plan(rows, cols, tokens, e.gated, &pl);
  if (st != NM_OK) return st;
  if (pl.workspace > 0 && (!workspace || workspace_bytes < pl.workspace)) return NM_ERR_WORKSPACE;
  if (overlaps_any({workspace, pl.workspace}, {w, m, x, b, res, y})) return NM_ERR_ALIAS;
  Epilogue epi;
  epi.bias = static_cast<const __half*>(e.bias);
  epi.residual = static_cast<const __half*>(e.residual);
  epi.ldres = e.ldres;
  epi.scale = e.scale;
  epi.act = e.activation;
  epi.gated = e.gated != 0;
  __half* out = static_cast<__half*>(Y);
  float* part = static_cast<float*>(workspace);
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  if (pl.path == Path::kSpmv) {
    SpmvParams& p = pl.vp;
    p.values = static_cast<const uint32_t*>(values);
    p.masks = masks;
    p.x = static_cast<const __half*>(X);
    p.y = out;
    p.early_weights = 0;
    p.epi = epi;
    return status(launch_spmv_linear(p, pl.spmv, kFlagPdl, s));
  }
  if (pl.path == Path::kSpmm) {
    SpmmLinearParams p;
    static_cast<SpmmParams&>(p) = pl.mp;
    p.values = static_cast<const uint32_t*>(values);
    p.masks = masks;
    p.X = static_cast<const __half*>(X);
    p.ldx = ldx;
    p.Y = out;
    p.ldy = ldy;
    p.partial = part;
    p.early_weights = 0;
    p.epi = epi;
    const cudaError_t err = launch_spmm_linear(p, pl.spmm, kFlagPdl, s);
    if (err != cudaSuccess || p.slices == 1) return status(err);
    return status(launch_linear_combine(part, p.slices, tokens, rows, epi, out, ldy, pl.sms, s));
  }
  SpmmTcParams p;
  p.values = values;
  p.masks = masks;
  p.X = X;
  p.ldx = ldx;
  p.Y = out;
  p.ldy = ldy;
  p.rows = rows;
  p.words = (int)(cols / 32);
  p.T = tokens;
  p.slices = spmm_tc_slices(p.words, pl.tc.slices);
  p.wslice = spmm_tc_slice_words(p.words, pl.tc.slices);
  p.epi = epi;
  p.tile = pl.tc.tile;
  p.wait_limit_ns = wait_limit_ns;
  p.stall_weights = stall;
  return status(launch_spmm_tc_linear(p, pl.tc.variant, s));
}

int nm_linear(const void* values, const uint32_t* masks, int64_t rows, int64_t cols, const void* X,
              int64_t ldx, int64_t tokens, const nm_epilogue* epilogue, void* Y, int64_t ldy,
              void* workspace, size_t workspace_bytes, void* stream) {
  return linear_call(values, masks, rows, cols, X, ldx, tokens, epilogue, Y, ldy, workspace, workspace_bytes, stream,
                     0, 0);
}

int nm_linear_stall_selftest(const void* values, const uint32_t* masks, int64_t rows, int64_t cols, const void* X,
                             int64_t ldx, int64_t tokens, const nm_epilogue* epilogue, void* Y, int64_t ldy,
                             void* workspace, size_t workspace_bytes, int64_t wait_limit_us, void* stream) {
  if (wait_limit_us <= 0 || wait_limit_us > 2000000) return NM_ERR_SHAPE;
  return linear_call(values, masks, rows, cols, X, ldx, tokens, epilogue, Y, ldy, workspace, workspace_bytes, stream,
                     (uint64_t)wait_limit_us * 1000u, 1);
}

int nm_residual_norm(const void* residual, int stream_fp32, int64_t ldr, const void* block,
                     int64_t ldb, const nm_norm* post, const void* gate, int64_t ldg, float scale,
                     float residual_scale, void* residual_out, int64_t lds, const nm_norm* pre,
                     void* out, int64_t ldo, int64_t tokens, int64_t width, void* stream) {
  if (tokens != 0 && (!residual || (!residual_out && !out))) return NM_ERR_NULL;
  ResidualNormParams p;
  int st = check_norm(block ? post : nullptr, &p.post);
  if (st == NM_OK) st = check_norm(out ? pre : nullptr, &p.pre);
  if (st != NM_OK) return st;
  const bool gated = block && gate;
  auto bad = [&](bool used, int64_t ld) { return used && (ld < width || ld >= kMax31); };
  if (tokens < 0 || tokens >= kMax31 || width < 1 || width > 32768 || bad(true, ldr) ||
      bad(block, ldb) || bad(gated && ldg != 0, ldg) || bad(residual_out, lds) || bad(out, ldo) ||
      !isfinite(scale) || !isfinite(residual_scale))
    return NM_ERR_SHAPE;
  const size_t es = stream_fp32 ? 4 : 2;
  if (!aligned(residual, es) || !aligned(residual_out, es) || !aligned(block, 2) ||
      !aligned(gate, 2) || !aligned(out, 2))
    return NM_ERR_ALIGN;
  if (tokens == 0) return NM_OK;
  const Array r{residual, span(tokens, ldr, width, es)}, b{block, span(tokens, ldb, width, 2)},
      g{gated ? gate : nullptr, span(ldg ? tokens : 1, ldg, width, 2)},
      so{residual_out, span(tokens, lds, width, es)}, o{out, span(tokens, ldo, width, 2)};
  auto params = [&](const NormArgs& a, const void* at) {
    return Array{at, (size_t)width * (a.params_fp32 ? 4 : 2)};
  };
  const Array pw = params(p.post, p.post.weight), pb = params(p.post, p.post.bias),
              nw = params(p.pre, p.pre.weight), nb = params(p.pre, p.pre.bias);
  const bool in_place = residual_out == residual && (lds == ldr || tokens == 1);
  if (overlaps_any(o, {r, b, g, so, pw, pb, nw, nb}) || overlaps_any(so, {b, g, pw, pb, nw, nb}) ||
      (!in_place && overlap(so, r)))
    return NM_ERR_ALIAS;
  DeviceInfo d;
  if (device_info(&d) != cudaSuccess) return NM_ERR_CUDA;
  p.residual = residual;
  p.ldr = ldr;
  p.block = static_cast<const __half*>(block);
  p.ldb = block ? ldb : 0;
  p.gate = gated ? static_cast<const __half*>(gate) : nullptr;
  p.ldg = gated ? ldg : 0;
  p.scale = scale;
  p.residual_scale = residual_scale;
  p.stream_out = residual_out;
  p.lds = residual_out ? lds : 0;
  p.out = static_cast<__half*>(out);
  p.ldo = out ? ldo : 0;
  p.tokens = tokens;
  p.width = (int)width;
  return status(launch_residual_norm(p, stream_fp32, d, static_cast<cudaStream_t>(stream)));
}

int nm_token_logprobs(const void* logits, int logits_fp32, int64_t ld_logits, int64_t rows,
                      int64_t vocab, const int32_t* ids, int64_t ld_ids, int n_ids,
                      float temperature, float* logprob, float* entropy, int top,
                      int32_t* top_ids, float* top_logprob, void* stream) {
  if (rows != 0 && (!logits || (n_ids > 0 && (!ids || !logprob)) || (top > 0 && (!top_ids || !top_logprob))))
    return NM_ERR_NULL;
  if (rows < 0 || rows >= kMax31 || vocab < 1 || vocab > (1 << 24) || ld_logits < vocab ||
      ld_logits >= kMax31 || n_ids < 0 || n_ids > 1024 ||
      (n_ids > 0 && (ld_ids < n_ids || ld_ids >= kMax31)) || top < 0 || top > 32 || top > vocab ||
      !(temperature >= 0x1p-20f && temperature <= 0x1p20f))
    return NM_ERR_SHAPE;
  if (!aligned(logits, logits_fp32 ? 4 : 2) || !aligned(ids, 4) || !aligned(logprob, 4) ||
      !aligned(entropy, 4) || !aligned(top_ids, 4) || !aligned(top_logprob, 4))
    return NM_ERR_ALIGN;
  if (rows == 0) return NM_OK;
  const Array in[2] = {{logits, span(rows, ld_logits, vocab, logits_fp32 ? 4 : 2)},
                       {n_ids ? ids : nullptr, span(rows, ld_ids, n_ids, 4)}};
  const Array out[4] = {{n_ids ? logprob : nullptr, (size_t)rows * n_ids * 4}, {entropy, (size_t)rows * 4},
                        {top ? top_ids : nullptr, (size_t)rows * top * 4},
                        {top ? top_logprob : nullptr, (size_t)rows * top * 4}};
  for (int i = 0; i < 4; ++i) {
    if (overlaps_any(out[i], {in[0], in[1]})) return NM_ERR_ALIAS;
    for (int j = 0; j < i; ++j)
      if (overlap(out[i], out[j])) return NM_ERR_ALIAS;
  }
  DeviceInfo d;
  if (device_info(&d) != cudaSuccess) return NM_ERR_CUDA;
  LogprobsParams p;
  p.logits = logits;
  p.ld_logits = ld_logits;
  p.rows = rows;
  p.vocab = (int)vocab;
  p.ids = ids;
  p.ld_ids = ld_ids;
  p.n_ids = n_ids;
  p.temperature = temperature;
  p.logprob = logprob;
  p.entropy = entropy;
  p.top = top;
  p.top_ids = top_ids;
  p.top_logprob = top_logprob;
  return status(launch_logprobs(p, logits_fp32, d.sms, static_cast<cudaStream_t>(stream)));
}

}  // extern "C"
