// The binding of the norms, the paged cache and the chunk attention: checks that
// the tensors of a call fit together, allocates what the caller did not give, and
// calls the library (include/sparse_attn.h). paged.py has the signatures and their
// documentation and passes everything on by position.
//
// These calls are made once per layer and decode step, where the kernels take 2 to 7
// us: the same checks and conversions in Python and ctypes took 12 to 17 us of host
// time a call (27 the backward of the norm), more than the kernel that they start;
// here it is 4 to 7 (13). No streams: text goes through std::string alone.
#include <Python.h>

#include <algorithm>
#include <optional>
#include <string>
#include <vector>

#include <ATen/core/Tensor.h>
#include <ATen/ops/empty.h>
#include <ATen/ops/zeros.h>
#include <c10/cuda/CUDAGuard.h>
#include <c10/cuda/CUDAStream.h>
#include <torch/csrc/Dtype.h>
#include <torch/csrc/Exceptions.h>
#include <torch/csrc/autograd/python_variable.h>
#include <torch/csrc/utils/object_ptr.h>

#include "sparse_attn.h"

namespace {

using at::IntArrayRef;
using at::ScalarType;
using at::Tensor;

// The library's entry points, in the library that the package has loaded, and the
// package's check of a status, which raises.
struct {
  decltype(&sparse_attn_qk_norm_workspace_size) workspace_size;
  decltype(&sparse_attn_qk_norm_rope) norm;
  decltype(&sparse_attn_qk_norm_rope_bwd) norm_bwd;
  decltype(&sparse_attn_cache_append) append;
  decltype(&sparse_attn_cache_read) read;
  decltype(&sparse_attn_chunk) chunk;
  PyObject* check;
} g = {};

[[noreturn]] void raise(PyObject* type, const std::string& why) {
  PyErr_SetString(type, why.c_str());
  throw python_error();
}
[[noreturn]] void refuse(const std::string& why) { raise(PyExc_ValueError, why); }
[[noreturn]] void refuse_type(const std::string& why) { raise(PyExc_TypeError, why); }

// ---- arguments, in order -------------------------------------------------------
class Args {
 public:
  Args(PyObject* const* a, Py_ssize_t n, Py_ssize_t want) : a_(a) {
    if (n != want) refuse_type("wrong number of arguments");
  }
  PyObject* object() { return *a_++; }
  const Tensor& tensor(const char* name) { return unpack(object(), name); }
  // nullptr for None
  const Tensor* optional(const char* name) {
    PyObject* o = object();
    return o == Py_None ? nullptr : &unpack(o, name);
  }
  double number() {
    const double x = PyFloat_AsDouble(object());
    if (x == -1.0 && PyErr_Occurred()) throw python_error();
    return x;
  }
  bool truth() {
    const int x = PyObject_IsTrue(object());
    if (x < 0) throw python_error();
    return x;
  }
  // The C int nearest to an integer, which means the same (a window past every row)
  // or is refused like it; *cut: whether it is another number.
  static int32_t int32(PyObject* o, bool* cut = nullptr) {
    PyObject* i = PyNumber_Index(o);
    if (!i) throw python_error();
    int over = 0;
    const long long x = PyLong_AsLongLongAndOverflow(i, &over);
    Py_DECREF(i);
    if (over == 0 && x == -1 && PyErr_Occurred()) throw python_error();
    const long long y = over ? (over > 0 ? INT32_MAX : INT32_MIN)
                             : std::max<long long>(INT32_MIN, std::min<long long>(x, INT32_MAX));
    if (cut) *cut = over || x != y;
    return (int32_t)y;
  }
  int32_t int32() { return int32(object()); }

 private:
  static const Tensor& unpack(PyObject* o, const char* name) {
    if (!THPVariable_Check(o)) refuse_type(std::string(name) + " must be a tensor");
    return THPVariable_Unpack(o);
  }
  PyObject* const* a_;
};

int32_t size32(int64_t n) {
  if (n > INT32_MAX) refuse("every size must fit 32 bits");
  return (int32_t)n;
}

// The device of the call's first tensor, which becomes the current one, and the
// stream: that device's current one, or `stream`, which then becomes it.
class Place {
 public:
  Place(const Tensor& t, PyObject* stream) : index((int)t.get_device()) {
    if (!t.is_cuda()) refuse("the tensors must be on a CUDA device");
    device_.emplace(t.device());
    if (stream != Py_None) {
      const int64_t id = field(stream, "stream_id"), at = field(stream, "device_index");
      const int64_t type = field(stream, "device_type");
      if (at != index || type != (int64_t)c10::DeviceType::CUDA)
        refuse("stream must be on cuda:" + std::to_string(index));
      stream_.emplace(c10::Stream::unpack3(id, (c10::DeviceIndex)at, c10::DeviceType::CUDA));
    }
  }
  void* stream() const { return c10::cuda::getCurrentCUDAStream((c10::DeviceIndex)index).stream(); }
  const int index;

 private:
  static int64_t field(PyObject* o, const char* name) {
    PyObject* x = PyObject_GetAttrString(o, name);
    if (!x) throw python_error();
    const long long y = PyLong_AsLongLong(x);
    Py_DECREF(x);
    if (y == -1 && PyErr_Occurred()) throw python_error();
    return y;
  }
  std::optional<c10::cuda::CUDAGuard> device_;
  std::optional<c10::cuda::CUDAStreamGuard> stream_;
};

std::string described(ScalarType type, IntArrayRef shape, const Place& at) {
  std::string s = std::string(c10::toString(type)) + " tensor of shape [";
  for (size_t i = 0; i < shape.size(); ++i) s += (i ? ", " : "") + std::to_string(shape[i]);
  return s + "] on cuda:" + std::to_string(at.index);
}
bool fits(const Tensor& t, IntArrayRef shape, ScalarType type, const Place& at) {
  return t.scalar_type() == type && t.sizes() == shape && t.is_cuda() &&
         t.get_device() == at.index;
}
void whole(const char* name, const Tensor& t, IntArrayRef shape, ScalarType type,
           const Place& at) {
  if (!fits(t, shape, type, at) || !t.is_contiguous())
    refuse(std::string(name) + " must be a contiguous " + described(type, shape, at));
}
// Rows whose elements are contiguous; strides of 0 where there is one.
void rows(const char* name, const Tensor& t, IntArrayRef shape, ScalarType type, const Place& at,
          int64_t* strides) {
  if (!fits(t, shape, type, at) || t.strides().back() != 1)
    refuse(std::string(name) + " must be a " + described(type, shape, at) +
           " with contiguous rows");
  for (size_t i = 0; i + 1 < shape.size(); ++i) strides[i] = shape[i] > 1 ? t.strides()[i] : 0;
}
sa_head_strides head_rows(const char* name, const Tensor& t, IntArrayRef shape, ScalarType type,
                          const Place& at) {
  int64_t s[4];
  rows(name, t, shape, type, at, s);
  return {s[0], s[1], s[2], s[3]};
}
sa_row_strides token_rows(const char* name, const Tensor& t, IntArrayRef shape, ScalarType type,
                          const Place& at) {
  int64_t s[3];
  rows(name, t, shape, type, at, s);
  return {s[0], s[1], s[2]};
}

bool overlap(const Tensor& a, const Tensor& b) {
  if (a.numel() == 0 || b.numel() == 0) return false;
  auto span = [](const Tensor& t, const char*& from, const char*& to) {
    int64_t last = 0;
    for (int64_t i = 0; i < t.dim(); ++i) last += (t.size(i) - 1) * t.stride(i);
    from = static_cast<const char*>(t.const_data_ptr());
    to = from + (last + 1) * (int64_t)t.element_size();
  };
  const char *a0, *a1, *b0, *b1;
  span(a, a0, a1);
  span(b, b0, b1);
  return a0 < b1 && b0 < a1;
}
// out is `own` (contiguous) or shares no memory with it, and none with the others.
void apart(const char* name, const Tensor& out, const Tensor* own,
           std::initializer_list<const Tensor*> others) {
  if (own && overlap(out, *own) &&
      (out.const_data_ptr() != own->const_data_ptr() || !own->is_contiguous()))
    refuse(std::string(name) + " overlaps its input");
  for (const Tensor* o : others)
    if (o && overlap(out, *o)) refuse(std::string(name) + " overlaps another tensor of the call");
}
Tensor empty(const Tensor& like) { return at::empty(like.sizes(), like.options()); }
// `out`, checked, or a new contiguous tensor like `like`.
Tensor output(const char* name, const Tensor* out, const Tensor& like, const Place& at,
              std::initializer_list<const Tensor*> others) {
  if (!out) return empty(like);
  whole(name, *out, like.sizes(), like.scalar_type(), at);
  apart(name, *out, &like, others);
  return *out;
}

template <typename T = void>
const T* in(const Tensor* t) {
  return t ? static_cast<const T*>(t->const_data_ptr()) : nullptr;
}
template <typename T = void>
T* out_of(const Tensor& t) {
  return t.defined() ? static_cast<T*>(t.mutable_data_ptr()) : nullptr;
}

bool both(const char* what, const Tensor* a, const Tensor* b) {
  if (!a != !b) refuse(std::string(what) + ": both or neither");
  return a != nullptr;
}
sa_dtype row_type(ScalarType t) {
  if (t != at::kFloat && t != at::kBFloat16)
    refuse_type(std::string("unsupported dtype ") + c10::toString(t));
  return t == at::kFloat ? SA_DTYPE_F32 : SA_DTYPE_BF16;
}

// The library call without the interpreter's lock, and its status. (f may throw: a
// tensor without storage has no address to give.)
struct Unlocked {
  PyThreadState* const state = PyEval_SaveThread();
  ~Unlocked() { PyEval_RestoreThread(state); }
};
template <typename F>
void call(const char* name, F f) {
  const sa_status status = [&] {
    const Unlocked here;
    return f();
  }();
  if (status == SA_OK) return;
  PyObject* r = PyObject_CallFunction(g.check, "si", name, (int)status);
  Py_XDECREF(r);
  throw python_error();
}
PyObject* wrap(const Tensor& t) {
  if (t.defined()) return THPVariable_Wrap(t);
  Py_RETURN_NONE;
}
PyObject* wrapped(std::initializer_list<Tensor> all) {
  PyObject* r = PyTuple_New((Py_ssize_t)all.size());
  if (!r) throw python_error();
  Py_ssize_t i = 0;
  for (const Tensor& t : all) PyTuple_SET_ITEM(r, i++, wrap(t));
  return r;
}

// ---- norms of queries and keys -----------------------------------------------------
struct Norm {
  const Tensor &q, &k;
  const Tensor *qw, *kw;
  sa_qk_norm_params p;
  sa_head_strides qs, ks;
};
// q, k, weights, eps, rotate, rope_base, pos0
Norm norm_args(Args& a, const Tensor& q, const Place& at) {
  Norm n{q, a.tensor("k"), nullptr, nullptr, {}, {}, {}};
  n.qw = a.optional("q_weight");
  n.kw = a.optional("k_weight");
  if (q.dim() != 5 || n.k.dim() != 5) refuse("q and k must be [L, B, H, T, D]");
  n.p.dtype = row_type(q.scalar_type());
  n.p.eps = (float)a.number();
  n.p.rotate = a.truth();
  n.p.rope_base = (float)a.number();
  n.p.pos0 = a.int32();
  const IntArrayRef s = q.sizes();
  n.p.L = size32(s[0]); n.p.B = size32(s[1]); n.p.Hq = size32(s[2]); n.p.T = size32(s[3]);
  n.p.D = size32(s[4]);
  n.p.Hkv = size32(n.k.size(2));
  n.qs = head_rows("q", q, s, q.scalar_type(), at);
  n.ks = head_rows("k", n.k, {s[0], s[1], n.k.size(2), s[3], s[4]}, q.scalar_type(), at);
  if (both("q_weight and k_weight", n.qw, n.kw)) {
    whole("q_weight", *n.qw, {s[0], s[4]}, at::kFloat, at);
    whole("k_weight", *n.kw, {s[0], s[4]}, at::kFloat, at);
  } else if (!n.p.rotate) {
    refuse("without weights there is only the rotation");
  }
  return n;
}

PyObject* qk_norm_rope(PyObject*, PyObject* const* args, Py_ssize_t count) {
  HANDLE_TH_ERRORS
  Args a(args, count, 11);
  PyObject* stream = a.object();
  const Tensor& q = a.tensor("q");
  const Place at(q, stream);
  const Norm n = norm_args(a, q, at);
  const Tensor *q_out = a.optional("q_out"), *k_out = a.optional("k_out");
  const Tensor qo = output("q_out", q_out, q, at, {&n.k, n.qw, n.kw, k_out});
  const Tensor ko = output("k_out", k_out, n.k, at, {&q, n.qw, n.kw});
  call("sparse_attn_qk_norm_rope", [&] {
    return g.norm(&n.p, in(&q), &n.qs, in(&n.k), &n.ks, in<float>(n.qw), in<float>(n.kw),
                  out_of(qo), out_of(ko), at.stream());
  });
  return wrapped({qo, ko});
  END_HANDLE_TH_ERRORS
}

PyObject* qk_norm_rope_bwd(PyObject*, PyObject* const* args, Py_ssize_t count) {
  HANDLE_TH_ERRORS
  Args a(args, count, 16);
  PyObject* stream = a.object();
  const Tensor& q = a.tensor("q");
  const Place at(q, stream);
  const Norm n = norm_args(a, q, at);
  const Tensor &dq_out = a.tensor("dq_out"), &dk_out = a.tensor("dk_out");
  const Tensor *dq_ = a.optional("dq"), *dk_ = a.optional("dk");
  const Tensor *dqw_ = a.optional("dq_weight"), *dkw_ = a.optional("dk_weight");
  const Tensor* given = a.optional("workspace");
  const sa_head_strides dqs = head_rows("dq_out", dq_out, q.sizes(), q.scalar_type(), at);
  const sa_head_strides dks = head_rows("dk_out", dk_out, n.k.sizes(), q.scalar_type(), at);
  const Tensor dq = output("dq", dq_, dq_out, at, {&q, &n.k, &dk_out, n.qw, n.kw, dk_});
  const Tensor dk = output("dk", dk_, dk_out, at, {&q, &n.k, &dq_out, n.qw, n.kw});
  Tensor dqw, dkw, ws;
  if (n.qw) {
    dqw = output("dq_weight", dqw_, *n.qw, at, {&q, &n.k, &dq_out, &dk_out, &dq, &dk, dkw_});
    dkw = output("dk_weight", dkw_, *n.kw, at, {&q, &n.k, &dq_out, &dk_out, &dq, &dk});
    if (!given) {
      ws = at::empty({(int64_t)g.workspace_size(&n.p)}, q.options().dtype(at::kByte));
    } else {
      if (!given->is_cuda() || given->get_device() != at.index || !given->is_contiguous())
        refuse("workspace must be a contiguous buffer on cuda:" + std::to_string(at.index));
      apart("workspace", *given, nullptr,
            {&q, &n.k, &dq_out, &dk_out, n.qw, n.kw, &dq, &dk, &dqw, &dkw});
      ws = *given;
    }
  } else if (dqw_ || dkw_) {
    refuse("no weights, no gradients of them");
  }
  call("sparse_attn_qk_norm_rope_bwd", [&] {
    return g.norm_bwd(&n.p, in(&q), &n.qs, in(&n.k), &n.ks, in<float>(n.qw), in<float>(n.kw),
                      in(&dq_out), &dqs, in(&dk_out), &dks, out_of(dq), out_of(dk),
                      out_of<float>(dqw), out_of<float>(dkw), out_of(ws),
                      ws.defined() ? ws.nbytes() : 0, at.stream());
  });
  return wrapped({dq, dk, dqw, dkw});
  END_HANDLE_TH_ERRORS
}

// ---- paged cache --------------------------------------------------------------------
struct Cache {
  const Tensor &k, &v;
  const Tensor *k_scale, *v_scale;
  static Cache of(PyObject* o) {      // a PagedCache
    if (!PyTuple_Check(o) || PyTuple_GET_SIZE(o) != 4) refuse_type("cache must be a PagedCache");
    PyObject* items[4];
    for (int i = 0; i < 4; ++i) items[i] = PyTuple_GET_ITEM(o, i);
    Args a(items, 4, 4);
    const Tensor &k = a.tensor("cache.k"), &v = a.tensor("cache.v");
    const Tensor* ks = a.optional("cache.k_scale");
    return {k, v, ks, a.optional("cache.v_scale")};
  }
  // Refuses a tensor that shares memory with the pages or their scales.
  void apart_from(const char* name, const Tensor& t) const {
    for (const Tensor* x : {&k, &v, k_scale, v_scale})
      if (x && overlap(t, *x)) refuse(std::string(name) + " overlaps the cache");
  }
};
struct Paged {
  sa_paged_params p;
  sa_pages c;
};
// L < 0: the cache's own; hq < 0: the cache's heads
Paged paged_args(const Cache& c, const Tensor& table, ScalarType dtype, int64_t L, int64_t N,
                 int64_t hq, const Place& at) {
  if (c.k.dim() != 5) refuse("cache.k must be [L, n_pages, Hkv, page_size, D]");
  const IntArrayRef s = c.k.sizes();
  const ScalarType held = c.k.scalar_type();
  const bool q8 = held == at::kFloat8_e4m3fn;
  if ((dtype != at::kFloat && dtype != at::kBFloat16) || (!q8 && held != dtype))
    refuse_type(std::string("rows of ") + c10::toString(dtype) + " and a cache of " +
                c10::toString(held));
  const int64_t shape[5] = {L < 0 ? s[0] : L, s[1], s[2], s[3], s[4]};
  whole("cache.k", c.k, shape, held, at);
  whole("cache.v", c.v, shape, held, at);
  if (q8) {
    if (!c.k_scale || !c.v_scale) refuse("float8_e4m3fn pages need k_scale and v_scale");
    whole("cache.k_scale", *c.k_scale, IntArrayRef(shape, 4), at::kFloat, at);
    whole("cache.v_scale", *c.v_scale, IntArrayRef(shape, 4), at::kFloat, at);
  } else if (c.k_scale || c.v_scale) {
    refuse("scales belong to float8_e4m3fn pages only");
  }
  if (table.dim() != 2) refuse("page_table must be [B, max_pages]");
  whole("page_table", table, table.sizes(), at::kInt, at);
  Paged x;
  x.p = {size32(shape[0]), size32(N), size32(table.size(0)), size32(hq < 0 ? s[2] : hq),
         size32(s[2]), size32(s[4]), size32(s[1]), size32(s[3]), size32(table.size(1)),
         row_type(dtype), q8 ? SA_CACHE_E4M3 : SA_CACHE_PLAIN};
  x.c = {c.k.mutable_data_ptr(), c.v.mutable_data_ptr(),
         const_cast<float*>(in<float>(c.k_scale)), const_cast<float*>(in<float>(c.v_scale)),
         in<int32_t>(&table)};
  return x;
}
void sequences(const Tensor& cu, const Tensor& cached, int64_t B, const Place& at) {
  whole("cu_q", cu, {B + 1}, at::kInt, at);
  whole("cached", cached, {B}, at::kInt, at);
}

PyObject* cache_append(PyObject*, PyObject* const* args, Py_ssize_t count) {
  HANDLE_TH_ERRORS
  Args a(args, count, 13);
  PyObject* stream = a.object();
  const Tensor& q = a.tensor("q");
  const Place at(q, stream);
  const Tensor &k = a.tensor("k"), &v = a.tensor("v");
  const Cache cache = Cache::of(a.object());
  const Tensor &table = a.tensor("page_table"), &cu = a.tensor("cu_q");
  const Tensor& cached = a.tensor("cached");
  const Tensor *qw = a.optional("q_weight"), *kw = a.optional("k_weight");
  const float eps = (float)a.number(), base = (float)a.number();
  const Tensor* given = a.optional("q_out");
  if (q.dim() != 4 || k.dim() != 4) refuse("q, k and v must be [L, N, heads, D]");
  const ScalarType type = q.scalar_type();
  const int64_t L = q.size(0), N = q.size(1), D = q.size(3);
  const Paged x = paged_args(cache, table, type, L, N, q.size(2), at);
  const int64_t kv[4] = {L, N, x.p.Hkv, x.p.D};
  const sa_row_strides qs = token_rows("q", q, {L, N, q.size(2), x.p.D}, type, at);
  const sa_row_strides ks = token_rows("k", k, kv, type, at);
  const sa_row_strides vs = token_rows("v", v, kv, type, at);
  sequences(cu, cached, x.p.B, at);
  if (both("q_weight and k_weight", qw, kw)) {
    whole("q_weight", *qw, {L, D}, at::kFloat, at);
    whole("k_weight", *kw, {L, D}, at::kFloat, at);
  }
  Tensor out;
  if (!given) {
    out = empty(q);
  } else {
    whole("q_out", *given, q.sizes(), type, at);
    apart("q_out", *given, nullptr, {&q, &k, &v, qw, kw, &table, &cu, &cached});
    cache.apart_from("q_out", *given);
    out = *given;
  }
  // (the pages are written: nothing else of the call may lie in them)
  apart("cache.k", cache.k, nullptr, {&cache.v, cache.k_scale, cache.v_scale});
  apart("cache.v", cache.v, nullptr, {cache.k_scale, cache.v_scale});
  if (cache.k_scale) apart("cache.k_scale", *cache.k_scale, nullptr, {cache.v_scale});
  for (const Tensor* t : {&q, &k, &v, qw, kw, &table, &cu, &cached})
    if (t) cache.apart_from("an input", *t);
  call("sparse_attn_cache_append", [&] {
    return g.append(&x.p, &x.c, in<int32_t>(&cu), in<int32_t>(&cached), in(&q), &qs, in(&k), &ks,
                    in(&v), &vs, in<float>(qw), in<float>(kw), eps, base, out_of(out),
                    at.stream());
  });
  return wrap(out);
  END_HANDLE_TH_ERRORS
}

PyObject* cache_read(PyObject*, PyObject* const* args, Py_ssize_t count) {
  HANDLE_TH_ERRORS
  Args a(args, count, 8);
  PyObject* stream = a.object();
  const Cache cache = Cache::of(a.object());
  const Place at(cache.k, stream);
  const Tensor &table = a.tensor("page_table"), &lengths = a.tensor("lengths");
  PyObject *asked = a.object(), *kind = a.object();
  const Tensor *k_out = a.optional("k_out"), *v_out = a.optional("v_out");
  both("k_out and v_out", k_out, v_out);
  ScalarType type = cache.k.scalar_type();
  if (kind != Py_None) {
    if (!THPDtype_Check(kind)) refuse_type("dtype must be a torch.dtype");
    type = reinterpret_cast<THPDtype*>(kind)->scalar_type;
  } else if (k_out) {
    type = k_out->scalar_type();
  } else if (type == at::kFloat8_e4m3fn) {
    type = at::kBFloat16;
  }
  const Paged x = paged_args(cache, table, type, -1, 0, -1, at);
  whole("lengths", lengths, {x.p.B}, at::kInt, at);
  const int64_t rows = asked != Py_None ? Args::int32(asked)
                       : k_out          ? (k_out->dim() == 5 ? k_out->size(3) : -1)
                                        : (int64_t)x.p.max_pages * x.p.page_size;
  if (rows < 0) refuse("k_out and v_out must be [L, B, Hkv, rows, D], rows at least 0");
  const int64_t shape[5] = {x.p.L, x.p.B, x.p.Hkv, rows, x.p.D};
  Tensor k, v;
  if (k_out) {
    whole("k_out", *k_out, shape, type, at);
    whole("v_out", *v_out, shape, type, at);
    apart("v_out", *v_out, nullptr, {k_out});
    for (const Tensor* t : {k_out, v_out}) {
      cache.apart_from(t == k_out ? "k_out" : "v_out", *t);
      apart(t == k_out ? "k_out" : "v_out", *t, nullptr, {&table, &lengths});
    }
    k = *k_out;
    v = *v_out;
  } else {
    k = at::zeros(shape, cache.k.options().dtype(type));
    v = at::zeros(shape, cache.k.options().dtype(type));
  }
  const int32_t n = size32(rows);
  call("sparse_attn_cache_read", [&] {
    return g.read(&x.p, &x.c, in<int32_t>(&lengths), n, out_of(k), out_of(v), at.stream());
  });
  return wrapped({k, v});
  END_HANDLE_TH_ERRORS
}

PyObject* chunk_attn(PyObject*, PyObject* const* args, Py_ssize_t count) {
  HANDLE_TH_ERRORS
  Args a(args, count, 15);
  PyObject* stream = a.object();
  const Tensor& q = a.tensor("q");
  const Place at(q, stream);
  const Cache cache = Cache::of(a.object());
  const Tensor &table = a.tensor("page_table"), &cu = a.tensor("cu_q");
  const Tensor &cached = a.tensor("cached"), &alpha = a.tensor("alpha");
  const int32_t window = a.int32();
  PyObject* list = a.object();
  const int32_t sinks = a.int32();
  const float scale = (float)a.number();
  const Tensor* beta = a.optional("beta");
  const Tensor *out_ = a.optional("out"), *lse_ = a.optional("lse");
  const bool want_lse = a.truth();
  if (q.dim() != 4) refuse("q must be [L, N, Hq, D]");
  const ScalarType type = q.scalar_type();
  const int64_t L = q.size(0), N = q.size(1), Hq = q.size(2);
  const Paged x = paged_args(cache, table, type, L, N, Hq, at);
  const sa_row_strides qs = token_rows("q", q, {L, N, Hq, x.p.D}, type, at);
  sequences(cu, cached, x.p.B, at);
  whole("alpha", alpha, {L}, at::kFloat, at);
  if (beta) whole("beta", *beta, {L, N, Hq}, at::kFloat, at);
  std::vector<int32_t> offsets;
  PyObject* items = PySequence_Fast(list, "offsets must be a sequence");
  if (!items) throw python_error();
  const THPObjectPtr held(items);
  for (Py_ssize_t i = 0; i < PySequence_Fast_GET_SIZE(items); ++i) {
    bool cut = false;
    offsets.push_back(Args::int32(PySequence_Fast_GET_ITEM(items, i), &cut));
    if (cut) refuse("offsets must fit 32 bits");
  }
  Tensor out, lse;
  if (!out_) {
    out = empty(q);
  } else {
    whole("out", *out_, q.sizes(), type, at);
    apart("out", *out_, nullptr, {&q, &table, &cu, &cached, &alpha, beta, lse_});
    cache.apart_from("out", *out_);
    out = *out_;
  }
  if (lse_) {
    whole("lse", *lse_, {L, N, Hq}, at::kFloat, at);
    apart("lse", *lse_, nullptr, {&q, &table, &cu, &cached, &alpha, beta});
    cache.apart_from("lse", *lse_);
    lse = *lse_;
  } else if (want_lse) {
    lse = at::empty({L, N, Hq}, alpha.options());
  }
  call("sparse_attn_chunk", [&] {
    return g.chunk(&x.p, &x.c, in<int32_t>(&cu), in<int32_t>(&cached), in(&q), &qs,
                   in<float>(&alpha), in<float>(beta), window, (int32_t)offsets.size(),
                   offsets.data(), sinks, scale, out_of(out), out_of<float>(lse), at.stream());
  });
  return wrapped({out, lse});
  END_HANDLE_TH_ERRORS
}

// bind(check, six addresses in the order of g)
PyObject* bind(PyObject*, PyObject* const* args, Py_ssize_t count) {
  HANDLE_TH_ERRORS
  Args a(args, count, 7);
  PyObject* check = a.object();
  void* at[6];
  for (void*& p : at) {
    p = PyLong_AsVoidPtr(a.object());
    if (!p) {
      if (PyErr_Occurred()) throw python_error();
      refuse("an entry point is missing");
    }
  }
  g.workspace_size = reinterpret_cast<decltype(g.workspace_size)>(at[0]);
  g.norm = reinterpret_cast<decltype(g.norm)>(at[1]);
  g.norm_bwd = reinterpret_cast<decltype(g.norm_bwd)>(at[2]);
  g.append = reinterpret_cast<decltype(g.append)>(at[3]);
  g.read = reinterpret_cast<decltype(g.read)>(at[4]);
  g.chunk = reinterpret_cast<decltype(g.chunk)>(at[5]);
  Py_INCREF(check);
  Py_XSETREF(g.check, check);
  Py_RETURN_NONE;
  END_HANDLE_TH_ERRORS
}

using Fast = PyObject* (*)(PyObject*, PyObject* const*, Py_ssize_t);
PyMethodDef method(const char* name, Fast f) {
  return {name, reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(f)), METH_FASTCALL,
          nullptr};
}
PyMethodDef methods[] = {method("bind", bind),
                         method("qk_norm_rope", qk_norm_rope),
                         method("qk_norm_rope_bwd", qk_norm_rope_bwd),
                         method("cache_append", cache_append),
                         method("cache_read", cache_read),
                         method("chunk_attn", chunk_attn),
                         {nullptr, nullptr, 0, nullptr}};
PyModuleDef module = {PyModuleDef_HEAD_INIT, "_binding", nullptr, -1, methods,
                      nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__binding() { return PyModule_Create(&module); }
