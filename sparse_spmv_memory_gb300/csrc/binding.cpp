// binding.cpp -- the Python side of nm_decode.h and nm_layer.h: tensors to pointers,
// sizes and strides, checked.  The operators of a decoding step run for a few
// microseconds each, about what a handful of attribute reads of a tensor costs
// in Python (a ctypes call of one of them took 25 us and more on the GB300's
// host, this 4), so these calls are marshalled in C++; decode.py and layer.py
// have their signatures and documentation.
#include <ATen/core/Tensor.h>
#include <ATen/ops/empty.h>
#include <ATen/ops/zeros.h>
#include <c10/cuda/CUDAGuard.h>
#include <c10/cuda/CUDAStream.h>
#include <torch/csrc/autograd/python_variable.h>

#include <cmath>
#include <exception>
#include <initializer_list>
#include <stdexcept>
#include <string>

#include "../../include/nm_decode.h"
#include "../../include/nm_layer.h"

namespace {

using at::Tensor;

struct Refused : std::invalid_argument {  // becomes a ValueError
  using std::invalid_argument::invalid_argument;
};
struct Status {  // becomes an NMError
  int code;
  const char* call;
};
struct PythonError {};  // already set

[[noreturn]] void refuse(const std::string& why) { throw Refused(why); }

// The tensors of a call, all on the device of the first.
struct Tensors {
  int device = -1;

  // An argument that is a CUDA tensor, or (optional) None.
  const Tensor* operator()(PyObject* o, const char* what, bool optional = false) {
    if (o == Py_None && optional) return nullptr;
    if (!THPVariable_Check(o)) {
      PyErr_Format(PyExc_TypeError, "%s must be a tensor", what);
      throw PythonError{};
    }
    const Tensor& t = THPVariable_Unpack(o);
    if (!t.is_cuda()) refuse("nm_* calls take CUDA tensors (there is no CPU path)");
    const int on = (int)t.get_device();
    if (device < 0) device = on;
    if (on != device) refuse(std::string(what) + " is on another device than the call's first tensor");
    return &t;
  }
};

template <typename T = void>
T* pointer(const Tensor* t) {
  return t ? static_cast<T*>(t->data_ptr()) : nullptr;
}

int64_t integer(PyObject* o) {
  const long long v = PyLong_AsLongLong(o);
  if (v == -1 && PyErr_Occurred()) throw PythonError{};
  return v;
}

int int32(PyObject* o, const char* what) {
  const int64_t v = integer(o);
  if (v < INT32_MIN || v > INT32_MAX) refuse(std::string(what) + " is out of range");
  return (int)v;
}

double real(PyObject* o) {
  const double v = PyFloat_AsDouble(o);
  if (v == -1.0 && PyErr_Occurred()) throw PythonError{};
  return v;
}

bool truth(PyObject* o) {
  const int v = PyObject_IsTrue(o);
  if (v < 0) throw PythonError{};
  return v != 0;
}

// The tensors' device, and the stream that a call was given (None: that device's
// current one): both are the current ones meanwhile, so that what the call
// allocates, and the zeros of a workspace, are ordered with its kernels.
struct OnStream {
  c10::cuda::CUDAGuard device;
  c10::cuda::OptionalCUDAStreamGuard guard;
  OnStream(PyObject* o, const Tensors& in) : device((c10::DeviceIndex)in.device) {
    if (o == Py_None) return;
    const unsigned long long v = PyLong_AsUnsignedLongLong(o);
    if (v == (unsigned long long)-1 && PyErr_Occurred()) throw PythonError{};
    guard.reset_stream(c10::cuda::getStreamFromExternal(reinterpret_cast<cudaStream_t>(static_cast<uintptr_t>(v)),
                                                        (c10::DeviceIndex)in.device));
  }
  void* stream() const { return c10::cuda::getCurrentCUDAStream().stream(); }
};

// Whether the dimensions from `first` on are laid out densely.
bool dense_from(const Tensor& t, int first) {
  int64_t want = 1;
  for (int d = (int)t.dim() - 1; d >= first; --d) {
    if (t.size(d) != 1 && t.stride(d) != want) return false;
    want *= t.size(d);
  }
  return true;
}

void vector(const Tensor* t, at::ScalarType type, int64_t n, const char* what) {
  if (t && (t->scalar_type() != type || t->numel() != n || !t->is_contiguous()))
    refuse(std::string(what) + " must be a contiguous " + at::toString(type) + " tensor of " +
           std::to_string(n) + " elements");
}

// Elements from one row to the next of a matrix with unit column stride.
int64_t row_stride(const Tensor& t, const char* what) {
  if (t.dim() != 2 || (t.stride(1) != 1 && t.size(1) != 1))
    refuse(std::string(what) + " must be a matrix with unit column stride");
  return t.size(0) > 1 ? t.stride(0) : t.size(1);
}

// The token stride of fp16 [tokens][heads][dim] with dense heads.
int64_t head_stride(const Tensor& t, int64_t tokens, int64_t dim, const char* what) {
  if (t.scalar_type() != at::kHalf || t.dim() != 3 || t.size(0) != tokens || t.size(2) != dim ||
      !dense_from(t, 1))
    refuse(std::string(what) + " must be float16 [tokens][heads][head_dim], contiguous but for the "
                               "token stride");
  return tokens > 1 ? t.stride(0) : t.size(1) * t.size(2);
}

nm_cache cache_of(Tensors& tensor, PyObject* k_, PyObject* v_, PyObject* ks_, PyObject* vs_) {
  const Tensor &k = *tensor(k_, "k_cache"), &v = *tensor(v_, "v_cache");
  const Tensor *ks = tensor(ks_, "k_scale", true), *vs = tensor(vs_, "v_scale", true);
  nm_cache c;
  const at::ScalarType type = k.scalar_type();
  c.type = type == at::kHalf ? NM_CACHE_FP16
           : type == at::kFloat8_e4m3fn ? NM_CACHE_E4M3
           : type == at::kChar ? NM_CACHE_INT8 : -1;
  if (c.type < 0 || v.scalar_type() != type)
    refuse("k_cache and v_cache must both be float16, float8_e4m3fn or int8");
  if (k.dim() != 4 || k.sizes() != v.sizes() || k.strides() != v.strides() || !dense_from(k, 1))
    refuse("k_cache and v_cache must be [pages][kv_heads][page_size][head_dim] of one shape and "
           "stride, contiguous but for the page stride");
  if (k.size(1) > INT32_MAX || k.size(2) > INT32_MAX || k.size(3) > INT32_MAX)
    refuse("k_cache is too large");
  c.scale_page_stride = 0;
  if (c.type != NM_CACHE_FP16) {
    if (!ks || !vs) refuse("an 8-bit cache needs k_scale and v_scale");
    for (const Tensor* s : {ks, vs})
      if (s->scalar_type() != at::kFloat || s->sizes() != k.sizes().slice(0, 3) ||
          s->strides() != ks->strides() || !dense_from(*s, 1))
        refuse("k_scale and v_scale must be float32 [pages][kv_heads][page_size] of one stride, "
               "contiguous but for the page stride");
    c.scale_page_stride = k.size(0) > 1 ? ks->stride(0) : k.size(1) * k.size(2);
  } else if (ks || vs) {
    refuse("a float16 cache takes no scales");
  }
  c.k = pointer(&k);
  c.v = pointer(&v);
  c.k_scale = pointer<float>(ks);
  c.v_scale = pointer<float>(vs);
  c.pages = k.size(0);
  c.page_stride = k.size(0) > 1 ? k.stride(0) : k.size(1) * k.size(2) * k.size(3);
  c.kv_heads = (int32_t)k.size(1);
  c.page_size = (int32_t)k.size(2);
  c.head_dim = (int32_t)k.size(3);
  return c;
}

void check(int code, const char* call) {
  if (code != NM_OK) throw Status{code, call};
}

PyObject* wrapped(const Tensor* given, PyObject* given_o, Tensor& made) {
  if (!given) return THPVariable_Wrap(made);
  Py_INCREF(given_o);
  return given_o;
}

// Several outputs of a call in one allocation, each at a multiple of 256 bytes: an
// allocation costs about a microsecond on the GB300's host, as much as the rest of a
// call's marshalling.  Whoever keeps one output then keeps the memory of all, so from
// kShared bytes on, where the kernel takes as long as the call (5 us) and hides the
// microsecond, each has an allocation of its own.
struct Outputs {
  static constexpr int64_t kShared = 16 << 20;
  Tensor whole;  // (undefined: none)
  at::TensorOptions like;
  int64_t used = 0;

  explicit Outputs(int64_t bytes, const at::TensorOptions& o) : like(o) {
    if (bytes < kShared) whole = at::empty({bytes}, like.dtype(at::kByte));
  }

  static int64_t room(int64_t bytes) { return (bytes + 255) / 256 * 256; }

  Tensor next(at::IntArrayRef sizes, at::ScalarType type) {
    if (!whole.defined()) return at::empty(sizes, like.dtype(type));
    const caffe2::TypeMeta meta = c10::scalarTypeToTypeMeta(type);
    auto impl = c10::make_intrusive<c10::TensorImpl>(c10::Storage(whole.storage()), whole.key_set(), meta);
    impl->set_storage_offset(used / (int64_t)meta.itemsize());
    impl->set_sizes_contiguous(sizes);
    int64_t n = (int64_t)meta.itemsize();
    for (int64_t d : sizes) n *= d;
    used += room(n);
    return Tensor(std::move(impl));
  }
};

PyObject* tuple_of(std::initializer_list<PyObject*> items) {
  PyObject* t = PyTuple_New((Py_ssize_t)items.size());
  Py_ssize_t i = 0;
  for (PyObject* o : items) {
    if (t && o)
      PyTuple_SET_ITEM(t, i++, o);
    else
      Py_XDECREF(o);
  }
  if (t && i != (Py_ssize_t)items.size()) {
    Py_DECREF(t);
    return nullptr;
  }
  return t;
}

// (qkv, k_cache, v_cache, positions, slots, inv_freq, q_heads, k_scale, v_scale,
//  interleaved, mscale, q, want_q, stream)
PyObject* rope_append(PyObject* const* a) {
  Tensors tensor;
  const nm_cache c = cache_of(tensor, a[1], a[2], a[7], a[8]);
  const Tensor &qkv = *tensor(a[0], "qkv"), &pos = *tensor(a[3], "positions"),
               &slots = *tensor(a[4], "slots"), &freq = *tensor(a[5], "inv_freq");
  const int64_t q_heads = integer(a[6]);
  if (qkv.scalar_type() != at::kHalf || qkv.dim() != 2 ||
      qkv.size(1) != (q_heads + 2 * c.kv_heads) * c.head_dim)
    refuse("qkv must be float16 [tokens][(q_heads + 2 kv_heads) * head_dim]");
  const int64_t tokens = qkv.size(0);
  vector(&pos, at::kInt, tokens, "positions");
  vector(&slots, at::kLong, tokens, "slots");
  vector(&freq, at::kFloat, freq.numel(), "inv_freq");
  const Tensor* q = tensor(a[11], "q", true);
  const bool want = q || truth(a[12]);
  Tensor made;
  const OnStream on(a[13], tensor);
  if (want && !q) made = at::empty({tokens, q_heads, c.head_dim}, qkv.options());
  const Tensor* out = q ? q : want ? &made : nullptr;
  if (out && out->dim() == 3 && out->size(1) != q_heads) refuse("q must have q_heads heads");
  check(nm_rope_append(pointer(&qkv), row_stride(qkv, "qkv"), tokens, (int)q_heads,
                       pointer<int32_t>(&pos), pointer<int64_t>(&slots), pointer<float>(&freq),
                       (int)std::min<int64_t>(2 * freq.numel(), 1 << 20), truth(a[9]) ? 1 : 0,
                       (float)real(a[10]), pointer(out),
                       out ? head_stride(*out, tokens, c.head_dim, "q") : 0, &c, on.stream()),
        "nm_rope_append");
  if (!out) Py_RETURN_NONE;
  return wrapped(q, a[11], made);
}

// (k_cache, v_cache, slots, k_scale, v_scale, k, v, stream)
PyObject* cache_read(PyObject* const* a) {
  Tensors tensor;
  const nm_cache c = cache_of(tensor, a[0], a[1], a[3], a[4]);
  const Tensor& slots = *tensor(a[2], "slots");
  const int64_t rows = slots.numel();
  vector(&slots, at::kLong, rows, "slots");
  const Tensor *k = tensor(a[5], "k", true), *v = tensor(a[6], "v", true);
  for (const Tensor* t : {k, v})
    if (t && (t->scalar_type() != at::kHalf || t->sizes() != at::IntArrayRef({rows, c.kv_heads, c.head_dim}) ||
              !t->is_contiguous()))
      refuse("k and v must be contiguous float16 [rows][kv_heads][head_dim]");
  Tensor mk, mv;
  const auto half = slots.options().dtype(at::kHalf);
  const OnStream on(a[7], tensor);
  if (!k) mk = at::empty({rows, c.kv_heads, c.head_dim}, half);
  if (!v) mv = at::empty({rows, c.kv_heads, c.head_dim}, half);
  check(nm_cache_read(&c, pointer<int64_t>(&slots), rows, pointer(k ? k : &mk), pointer(v ? v : &mv),
                      on.stream()),
        "nm_cache_read");
  return tuple_of({wrapped(k, a[5], mk), wrapped(v, a[6], mv)});
}

// (q, k_cache, v_cache, block_table, ctx_len, q_start, max_nodes, tree_mask,
//  k_scale, v_scale, scale, out, lse, workspace, stream)
PyObject* tree_attention(PyObject* const* a) {
  Tensors tensor;
  const nm_cache c = cache_of(tensor, a[1], a[2], a[8], a[9]);
  const Tensor &q = *tensor(a[0], "q"), &table = *tensor(a[3], "block_table"),
               &ctx = *tensor(a[4], "ctx_len"), &start = *tensor(a[5], "q_start");
  const Tensor *mask = tensor(a[7], "tree_mask", true), *out = tensor(a[11], "out", true),
               *lse = tensor(a[12], "lse", true), *ws = tensor(a[13], "workspace", true);
  const int max_nodes = int32(a[6], "max_nodes");
  if (q.dim() != 3) refuse("q must be float16 [tokens][q_heads][head_dim]");
  const int64_t tokens = q.size(0), q_heads = q.size(1), seqs = ctx.numel();
  const int64_t ldq = head_stride(q, tokens, c.head_dim, "q");
  vector(&ctx, at::kInt, seqs, "ctx_len");
  vector(&start, at::kInt, seqs + 1, "q_start");
  vector(mask, at::kLong, tokens, "tree_mask");
  if (table.scalar_type() != at::kInt || table.dim() != 2 || table.size(0) != seqs)
    refuse("block_table must be int32 [seqs][entries]");
  if (q_heads > INT32_MAX) refuse("q is too large");
  Tensor mo, ml, mw;
  const OnStream on(a[14], tensor);
  if (!out) mo = at::empty({tokens, q_heads, c.head_dim}, q.options());
  const Tensor& o = out ? *out : mo;
  const int64_t ldo = head_stride(o, tokens, c.head_dim, "out");
  if (o.size(1) != q_heads) refuse("out must have as many heads as q");
  if (!lse) ml = at::empty({tokens, q_heads}, q.options().dtype(at::kFloat));
  const Tensor& l = lse ? *lse : ml;
  vector(&l, at::kFloat, tokens * q_heads, "lse");
  if (!ws) {
    const size_t need = nm_tree_attention_workspace_bytes(seqs, (int)q_heads, c.kv_heads, c.head_dim, max_nodes);
    mw = at::zeros({(int64_t)need}, q.options().dtype(at::kByte));
  } else if (!ws->is_contiguous()) {
    refuse("workspace must be contiguous");
  }
  const Tensor& work = ws ? *ws : mw;
  check(nm_tree_attention(pointer(&q), ldq, tokens, (int)q_heads, seqs, pointer<int32_t>(&start), max_nodes,
                          &c, pointer<int32_t>(&table), row_stride(table, "block_table"), table.size(1),
                          pointer<int32_t>(&ctx), pointer<uint64_t>(mask),
                          a[10] == Py_None ? 1.0f / std::sqrt((float)c.head_dim) : (float)real(a[10]),
                          pointer(&o), ldo, pointer<float>(&l), pointer(&work), work.nbytes(),
                          on.stream()),
        "nm_tree_attention");
  return tuple_of({wrapped(out, a[11], mo), wrapped(lse, a[12], ml)});
}

// (logits, tokens, parents, node_start, max_nodes, draft, accept, race,
//  temperature, path, count, token, stream)
PyObject* tree_verify(PyObject* const* a) {
  Tensors tensor;
  const Tensor &logits = *tensor(a[0], "logits"), &ids = *tensor(a[1], "tokens"),
               &parents = *tensor(a[2], "parents"), &start = *tensor(a[3], "node_start");
  const Tensor *draft = tensor(a[5], "draft", true), *accept = tensor(a[6], "accept", true),
               *race = tensor(a[7], "race", true), *path = tensor(a[9], "path", true),
               *count = tensor(a[10], "count", true), *token = tensor(a[11], "token", true);
  const int max_nodes = int32(a[4], "max_nodes");
  const bool fp32 = logits.scalar_type() == at::kFloat;
  if (!fp32 && logits.scalar_type() != at::kHalf) refuse("logits must be float16 or float32");
  const int64_t ld = row_stride(logits, "logits"), n = logits.size(0), vocab = logits.size(1);
  const int64_t seqs = start.numel() - 1;
  vector(&ids, at::kInt, n, "tokens");
  vector(&parents, at::kInt, n, "parents");
  if (seqs < 0) refuse("node_start must have an element more than there are sequences");
  vector(&start, at::kInt, seqs + 1, "node_start");
  vector(accept, at::kFloat, n, "accept");
  auto rows = [&](const Tensor* t, int64_t want, const char* what) -> int64_t {
    if (!t) return 0;
    if (t->scalar_type() != at::kFloat || t->dim() != 2 || t->size(0) != want || t->size(1) != vocab)
      refuse(std::string(what) + " must be float32 [" + std::to_string(want) + "][vocab]");
    return row_stride(*t, what);
  };
  const int64_t ldd = rows(draft, n, "draft"), ldr = rows(race, seqs, "race");
  const auto i32 = logits.options().dtype(at::kInt);
  Tensor mp, mc, mt;
  const OnStream on(a[12], tensor);
  // (the call refuses any other number of nodes, and nothing is allocated for it)
  if (!path) mp = at::empty({seqs, std::min(std::max(1, max_nodes), 64)}, i32);
  if (!count) mc = at::empty({seqs}, i32);
  if (!token) mt = at::empty({seqs}, i32);
  vector(path, at::kInt, seqs * max_nodes, "path");
  vector(count, at::kInt, seqs, "count");
  vector(token, at::kInt, seqs, "token");
  check(nm_tree_verify(pointer(&logits), fp32 ? 1 : 0, ld, vocab, pointer<float>(draft), ldd,
                       pointer<int32_t>(&ids), pointer<int32_t>(&parents), pointer<int32_t>(&start), n,
                       seqs, max_nodes, pointer<float>(accept), pointer<float>(race), ldr,
                       (float)real(a[8]), pointer<int32_t>(path ? path : &mp),
                       pointer<int32_t>(count ? count : &mc), pointer<int32_t>(token ? token : &mt),
                       on.stream()),
        "nm_tree_verify");
  return tuple_of({wrapped(path, a[9], mp), wrapped(count, a[10], mc), wrapped(token, a[11], mt)});
}

// A float16 matrix of rows x cols with unit column stride; its row stride.
int64_t half_rows(const Tensor& t, int64_t rows, int64_t cols, const char* what) {
  if (t.scalar_type() != at::kHalf || t.dim() != 2 || t.size(0) != rows || t.size(1) != cols)
    refuse(std::string(what) + " must be float16 [" + std::to_string(rows) + "][" + std::to_string(cols) + "]");
  return row_stride(t, what);
}

// (values, masks, X, bias, activation, gated, scale, residual, Y, workspace, stream, cols)
PyObject* linear(PyObject* const* a) {
  Tensors tensor;
  const Tensor &values = *tensor(a[0], "values"), &masks = *tensor(a[1], "masks"), &x = *tensor(a[2], "X");
  const Tensor *bias = tensor(a[3], "bias", true), *residual = tensor(a[7], "residual", true),
               *y = tensor(a[8], "Y", true), *ws = tensor(a[9], "workspace", true);
  if (x.scalar_type() != at::kHalf || x.dim() != 2) refuse("X must be float16 [tokens][cols]");
  const int64_t tokens = x.size(0), cols = a[11] == Py_None ? x.size(1) : integer(a[11]);
  if (cols < 1 || cols > x.size(1)) refuse("cols must be 1 .. the width of X");
  if (masks.scalar_type() != at::kInt || masks.dim() != 2 || !masks.is_contiguous() ||
      masks.size(1) * 32 != cols)
    refuse("masks must be contiguous int32 [rows][cols / 32]");
  const int64_t rows = masks.size(0);
  if (values.scalar_type() != at::kHalf || !values.is_contiguous() || values.numel() != rows * (cols / 2))
    refuse("values must be contiguous float16 [rows][cols / 2]");
  nm_epilogue e;
  e.activation = int32(a[4], "activation");
  e.gated = truth(a[5]) ? 1 : 0;
  if (e.gated && rows % 2) refuse("a gated product needs an even number of rows");
  const int64_t n = e.gated ? rows / 2 : rows;
  vector(bias, at::kHalf, rows, "bias");
  e.bias = pointer(bias);
  e.residual = pointer(residual);
  e.ldres = residual ? half_rows(*residual, tokens, n, "residual") : 0;
  e.scale = (float)real(a[6]);
  Tensor my, mw;
  const OnStream on(a[10], tensor);
  if (!y) my = at::empty({tokens, n}, x.options());
  const Tensor& out = y ? *y : my;
  const int64_t ldy = half_rows(out, tokens, n, "Y");
  if (!ws) {
    const size_t need = nm_linear_workspace_bytes(rows, cols, tokens);
    if (need) mw = at::empty({(int64_t)need}, x.options().dtype(at::kByte));
  } else if (!ws->is_contiguous()) {
    refuse("workspace must be contiguous");
  }
  check(nm_linear(pointer(&values), pointer<uint32_t>(&masks), rows, cols, pointer(&x),
                  tokens > 1 ? row_stride(x, "X") : (row_stride(x, "X") + 7) / 8 * 8, tokens, &e,
                  pointer(&out), ldy, ws ? pointer(ws) : mw.defined() ? mw.data_ptr() : nullptr,
                  ws ? ws->nbytes() : mw.defined() ? mw.nbytes() : 0, on.stream()),
        "nm_linear");
  return wrapped(y, a[8], my);
}

// A norm's weight and bias: float16 or float32 alike, [width] each.
nm_norm norm_of(Tensors& tensor, PyObject* kind, PyObject* weight_, PyObject* bias_, int64_t width,
                float offset, float eps, const char* what) {
  const Tensor *w = tensor(weight_, what, true), *b = tensor(bias_, what, true);
  nm_norm n;
  n.kind = int32(kind, what);
  if (n.kind == NM_NORM_NONE && (w || b)) refuse(std::string("a weight or bias needs its ") + what);
  n.offset = offset;
  n.eps = eps;
  const at::ScalarType type = w ? w->scalar_type() : b ? b->scalar_type() : at::kHalf;
  if (type != at::kHalf && type != at::kFloat)
    refuse(std::string("the weight and bias of ") + what + " must be float16 or float32");
  n.params_fp32 = type == at::kFloat;
  vector(w, type, width, what);
  vector(b, type, width, what);
  n.weight = pointer(w);
  n.bias = pointer(b);
  return n;
}

// (residual, block, norm, weight, bias, post_norm, post_weight, post_bias, gate, scale,
//  residual_scale, weight_offset, eps, residual_out, out, stream)
PyObject* residual_norm(PyObject* const* a) {
  Tensors tensor;
  const Tensor& r = *tensor(a[0], "residual");
  const Tensor *block = tensor(a[1], "block", true), *gate = tensor(a[8], "gate", true),
               *given_r = tensor(a[13], "residual_out", true), *given_o = tensor(a[14], "out", true);
  const bool fp32 = r.scalar_type() == at::kFloat;
  if ((!fp32 && r.scalar_type() != at::kHalf) || r.dim() != 2)
    refuse("residual must be float16 or float32 [tokens][width]");
  const int64_t tokens = r.size(0), width = r.size(1);
  const float offset = (float)real(a[11]), eps = (float)real(a[12]);
  const nm_norm pre = norm_of(tensor, a[2], a[3], a[4], width, offset, eps, "norm");
  const nm_norm post = norm_of(tensor, a[5], a[6], a[7], width, offset, eps, "post_norm");
  const double scale = real(a[9]), residual_scale = real(a[10]);
  if (!block && (gate || post.kind != NM_NORM_NONE)) refuse("a gate or a norm after the block needs the block");
  const int64_t ldr = row_stride(r, "residual");
  const int64_t ldb = block ? half_rows(*block, tokens, width, "block") : 0;
  int64_t ldg = 0;
  if (gate) {
    if (gate->dim() < 2 || gate->size(0) != tokens || tokens == 1)
      vector(gate, at::kHalf, width, "gate");  // one for all tokens
    else
      ldg = half_rows(*gate, tokens, width, "gate");
  }
  if (pre.kind == NM_NORM_NONE && given_o) refuse("out needs a norm");
  Tensor mr, mo;
  const OnStream on(a[15], tensor);
  // without a block and a factor the stream stays what it is
  const bool same = !block && residual_scale == 1.0 && !given_r;
  const bool make_r = !given_r && !same, make_o = pre.kind != NM_NORM_NONE && !given_o;
  if (make_r && make_o) {
    const int64_t n = tokens * width;
    Outputs both(Outputs::room(n * (fp32 ? 4 : 2)) + n * 2, r.options());
    mr = both.next({tokens, width}, r.scalar_type());
    mo = both.next({tokens, width}, at::kHalf);
  } else if (make_r) {
    mr = at::empty({tokens, width}, r.options());
  } else if (make_o) {
    mo = at::empty({tokens, width}, r.options().dtype(at::kHalf));
  }
  const Tensor* to = given_r ? given_r : same ? nullptr : &mr;
  const Tensor* o = given_o ? given_o : mo.defined() ? &mo : nullptr;
  if (to && (to->scalar_type() != r.scalar_type() || to->sizes() != r.sizes()))
    refuse("residual_out must be of residual's type and shape");
  if (to || o)
    check(nm_residual_norm(pointer(&r), fp32 ? 1 : 0, ldr, pointer(block), ldb, &post, pointer(gate), ldg,
                           (float)scale, (float)residual_scale, pointer(to),
                           to ? row_stride(*to, "residual_out") : 0, &pre, pointer(o),
                           o ? half_rows(*o, tokens, width, "out") : 0, tokens, width, on.stream()),
          "nm_residual_norm");
  PyObject* first = o ? wrapped(given_o, a[14], mo) : Py_NewRef(Py_None);
  return tuple_of({first, same ? Py_NewRef(a[0]) : wrapped(given_r, a[13], mr)});
}

// (logits, tokens, top, temperature, logprob, entropy, top_ids, top_logprob, stream)
PyObject* token_logprobs(PyObject* const* a) {
  Tensors tensor;
  const Tensor& logits = *tensor(a[0], "logits");
  const Tensor *ids = tensor(a[1], "tokens", true), *lp = tensor(a[4], "logprob", true),
               *entropy = tensor(a[5], "entropy", true), *top_ids = tensor(a[6], "top_ids", true),
               *top_lp = tensor(a[7], "top_logprob", true);
  const bool fp32 = logits.scalar_type() == at::kFloat;
  if (!fp32 && logits.scalar_type() != at::kHalf) refuse("logits must be float16 or float32");
  const int64_t ld = row_stride(logits, "logits"), rows = logits.size(0), vocab = logits.size(1);
  const int top = int32(a[2], "top");
  if (ids && (ids->scalar_type() != at::kInt || ids->dim() < 1 || ids->dim() > 2 || ids->size(0) != rows))
    refuse("tokens must be int32 [rows] or [rows][n]");
  const bool flat = ids && ids->dim() == 1;
  const int64_t n = !ids ? 0 : flat ? 1 : ids->size(1);
  if (n > INT32_MAX) refuse("tokens is too large");
  const int64_t ld_ids = !ids ? 0 : flat ? (rows > 1 ? ids->stride(0) : 1) : n ? row_stride(*ids, "tokens") : 0;
  const auto f32 = logits.options().dtype(at::kFloat);
  Tensor ml, me, mi, mt;
  const OnStream on(a[8], tensor);
  // (the call refuses any other number, and nothing is allocated for it)
  const int64_t k = std::min(std::max(0, top), 32);
  if (!lp || !entropy || !top_ids || !top_lp) {
    const auto room = [](bool given, int64_t words) { return given ? 0 : Outputs::room(4 * words); };
    Outputs made(room(lp, rows * n) + room(entropy, rows) + room(top_ids, rows * k) + room(top_lp, rows * k), f32);
    if (!lp) ml = flat ? made.next({rows}, at::kFloat) : made.next({rows, n}, at::kFloat);
    if (!entropy) me = made.next({rows}, at::kFloat);
    if (!top_ids) mi = made.next({rows, k}, at::kInt);
    if (!top_lp) mt = made.next({rows, k}, at::kFloat);
  }
  vector(lp, at::kFloat, rows * n, "logprob");
  vector(entropy, at::kFloat, rows, "entropy");
  vector(top_ids, at::kInt, rows * k, "top_ids");
  vector(top_lp, at::kFloat, rows * k, "top_logprob");
  check(nm_token_logprobs(pointer(&logits), fp32 ? 1 : 0, ld, rows, vocab, pointer<int32_t>(ids), ld_ids, (int)n,
                          (float)real(a[3]), pointer<float>(lp ? lp : &ml), pointer<float>(entropy ? entropy : &me),
                          top, pointer<int32_t>(top_ids ? top_ids : &mi), pointer<float>(top_lp ? top_lp : &mt),
                          on.stream()),
        "nm_token_logprobs");
  return tuple_of({wrapped(lp, a[4], ml), wrapped(entropy, a[5], me), wrapped(top_ids, a[6], mi),
                   wrapped(top_lp, a[7], mt)});
}

// Runs a call, with whatever it throws turned into a Python exception.
template <PyObject* (*CALL)(PyObject* const*), int ARGS>
PyObject* entry(PyObject*, PyObject* const* args, Py_ssize_t n) {
  if (n != ARGS) {
    PyErr_Format(PyExc_TypeError, "expected %d arguments, got %zd", ARGS, n);
    return nullptr;
  }
  try {
    return CALL(args);
  } catch (const PythonError&) {
  } catch (const Status& s) {
    PyObject* nm = PyImport_ImportModule("sparse_spmv_memory_gb300");
    PyObject* type = nm ? PyObject_GetAttrString(nm, "NMError") : nullptr;
    PyObject* e = type ? PyObject_CallFunction(type, "is", s.code, s.call) : nullptr;
    if (e) PyErr_SetObject(type, e);
    Py_XDECREF(e);
    Py_XDECREF(type);
    Py_XDECREF(nm);
  } catch (const Refused& e) {
    PyErr_SetString(PyExc_ValueError, e.what());
  } catch (const std::exception& e) {
    PyErr_SetString(PyExc_RuntimeError, e.what());
  }
  return nullptr;
}

PyMethodDef kMethods[] = {
    {"rope_append", reinterpret_cast<PyCFunction>(reinterpret_cast<void*>(&entry<rope_append, 14>)),
     METH_FASTCALL, nullptr},
    {"cache_read", reinterpret_cast<PyCFunction>(reinterpret_cast<void*>(&entry<cache_read, 8>)),
     METH_FASTCALL, nullptr},
    {"tree_attention", reinterpret_cast<PyCFunction>(reinterpret_cast<void*>(&entry<tree_attention, 15>)),
     METH_FASTCALL, nullptr},
    {"tree_verify", reinterpret_cast<PyCFunction>(reinterpret_cast<void*>(&entry<tree_verify, 13>)),
     METH_FASTCALL, nullptr},
    {"linear", reinterpret_cast<PyCFunction>(reinterpret_cast<void*>(&entry<linear, 12>)),
     METH_FASTCALL, nullptr},
    {"residual_norm", reinterpret_cast<PyCFunction>(reinterpret_cast<void*>(&entry<residual_norm, 16>)),
     METH_FASTCALL, nullptr},
    {"token_logprobs", reinterpret_cast<PyCFunction>(reinterpret_cast<void*>(&entry<token_logprobs, 9>)),
     METH_FASTCALL, nullptr},
    {nullptr, nullptr, 0, nullptr}};

PyModuleDef kModule = {PyModuleDef_HEAD_INIT, "_decode_ext", nullptr, -1, kMethods,
                       nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__decode_ext(void) { return PyModule_Create(&kModule); }
