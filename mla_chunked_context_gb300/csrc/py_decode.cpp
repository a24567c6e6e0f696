// The decode calls' Python binding: the checks of their tensors and the calls
// into the library.  A CPython module rather than ctypes, because these calls
// are made once a layer and token, where the host's time counts: checking and
// marshalling append's 17 arguments takes 7.6 us in Python through ctypes.
// Each function returns the library's code; a tensor that does not fit raises
// ValueError before anything is enqueued.
#include <c10/cuda/CUDAFunctions.h>
#include <c10/cuda/CUDAStream.h>
#include <torch/csrc/Dtype.h>
#include <torch/csrc/autograd/python_variable.h>

#include <initializer_list>
#include <sstream>
#include <stdexcept>
#include <string>
#include <vector>

#include "mla_chunked_context.h"

namespace {

using at::ScalarType;
using Shape = std::initializer_list<int64_t>;

// A Python exception is set already.
struct PythonError {};

PyObject *attr(PyObject *o, PyObject *name) {
  PyObject *v = PyObject_GetAttr(o, name);
  if (!v) throw PythonError();
  return v;  // a new reference
}

bool truth(PyObject *o) {
  const int v = PyObject_IsTrue(o);
  if (v < 0) throw PythonError();
  return v != 0;
}

int32_t narrow(int64_t v, const char *where, const char *name) {
  if (v < INT32_MIN || v > INT32_MAX)
    throw std::invalid_argument(std::string(where) + ": " + name + " has too many elements");
  return int32_t(v);
}

struct Names {
  PyObject *field[8];
  PyObject *cuda_stream;
} names;

// The Dims object's fields, and the storage type.
struct Dims {
  mla_dims_t c{};
  ScalarType type = ScalarType::Undefined;
  int64_t H, L, P, Dn, Dv, bs;
  explicit Dims(PyObject *o) {
    int64_t v[6];
    for (int i = 0; i < 6; ++i) {
      PyObject *f = attr(o, names.field[i]);
      v[i] = PyLong_AsLongLong(f);
      Py_DECREF(f);
      if (v[i] == -1 && PyErr_Occurred()) throw PythonError();
      if (v[i] < INT32_MIN || v[i] > INT32_MAX) throw std::invalid_argument("Dims: out of range");
    }
    PyObject *f = attr(o, names.field[6]);
    const double scale = PyFloat_AsDouble(f);
    Py_DECREF(f);
    if (scale == -1.0 && PyErr_Occurred()) throw PythonError();
    f = attr(o, names.field[7]);
    if (THPDtype_Check(f)) type = reinterpret_cast<THPDtype *>(f)->scalar_type;
    Py_DECREF(f);
    H = v[0], L = v[1], P = v[2], Dn = v[3], Dv = v[4], bs = v[5];
    c.num_heads = int32_t(H);
    c.kv_lora_rank = int32_t(L);
    c.qk_rope_dim = int32_t(P);
    c.qk_nope_dim = int32_t(Dn);
    c.v_dim = int32_t(Dv);
    c.block_size = int32_t(bs);
    c.softmax_scale = float(scale);
    if (type == ScalarType::BFloat16)
      c.dtype = MLA_DTYPE_BF16;
    else if (type == ScalarType::Float)
      c.dtype = MLA_DTYPE_F32;
    else if (type == ScalarType::Half)
      c.dtype = MLA_DTYPE_F16;
    else
      throw std::invalid_argument("unsupported dtype");
  }
};

// Checks the tensors of one call.
class Call {
 public:
  explicit Call(const char *where) : where_(where) {}

  const at::Tensor &tensor(const char *name, PyObject *o) const {
    if (!THPVariable_Check(o))
      throw std::invalid_argument(std::string(where_) + ": " + name + " has to be a tensor");
    return THPVariable_Unpack(o);
  }
  int64_t size(const char *name, PyObject *o, int dim, int dims) const {
    const at::Tensor &t = tensor(name, o);
    if (t.dim() != dims) {
      std::ostringstream s;
      s << where_ << ": " << name << " has to have " << dims << " dimensions, got " << t.dim();
      throw std::invalid_argument(s.str());
    }
    return t.size(dim);
  }
  // On the current device, where the C calls work.
  void on_device(const char *name, const at::Tensor &t) {
    if (t.is_cuda()) {
      if (device_ < 0) device_ = c10::cuda::current_device();
      if (t.get_device() == device_) return;
    }
    std::ostringstream s;
    s << where_ << ": " << name << " is on " << t.device() << ", the current device is ";
    if (c10::cuda::device_count() > 0)
      s << "cuda:" << int(c10::cuda::current_device());
    else
      s << "none";
    throw std::invalid_argument(s.str());
  }
  // Contiguous, of that type and shape; nullptr for None.
  void *take(const char *name, PyObject *o, ScalarType type, Shape shape) {
    if (o == Py_None) return nullptr;
    const at::Tensor &t = tensor(name, o);
    on_device(name, t);
    if (t.scalar_type() != type || t.sizes() != c10::IntArrayRef(shape) || !t.is_contiguous()) {
      std::ostringstream s;
      s << where_ << ": " << name << " has to be contiguous " << c10::IntArrayRef(shape) << " "
        << type << ", got " << t.sizes() << " " << t.scalar_type()
        << (t.is_contiguous() ? "" : ", not contiguous");
      throw std::invalid_argument(s.str());
    }
    return t.data_ptr();
  }
  template <typename T>
  T *take(const char *name, PyObject *o, ScalarType type, Shape shape) {
    return static_cast<T *>(take(name, o, type, shape));
  }
  // The stream given, or the current one.
  void *stream(PyObject *o) {
    if (o == Py_None) {
      if (device_ < 0) device_ = c10::cuda::current_device();
      return c10::cuda::getCurrentCUDAStream(device_).stream();
    }
    PyObject *v = attr(o, names.cuda_stream);
    void *s = PyLong_AsVoidPtr(v);
    Py_DECREF(v);
    if (!s && PyErr_Occurred()) throw PythonError();
    return s;
  }
  [[noreturn]] void refuse(const std::string &what) const {
    throw std::invalid_argument(std::string(where_) + ": " + what);
  }

 private:
  const char *where_;
  c10::DeviceIndex device_ = -1;
};

template <typename F>
int unlocked(F call) {
  int rc;
  Py_BEGIN_ALLOW_THREADS;
  rc = call();
  Py_END_ALLOW_THREADS;
  return rc;
}

std::string type_name(ScalarType t) {
  std::ostringstream s;
  s << t;
  return s.str();
}

constexpr ScalarType I32 = ScalarType::Int, F32 = ScalarType::Float, I64 = ScalarType::Long;

// dims, kv_a, query_start_loc, seq_lens, rope_table, kv_cache, block_table,
// norm_weight, norm_eps, positions, interleaved, new_latent, q, q_pe_out,
// dev_status, stream
int append(PyObject *const *a) {
  const char *w = "mla_append_latent";
  const Dims d(a[0]);
  Call c(w);
  const int64_t T = c.size("kv_a", a[1], 0, 2), R = c.size("seq_lens", a[3], 0, 1);
  const int64_t blocks = c.size("kv_cache", a[5], 0, 3), stride = c.size("block_table", a[6], 1, 2);
  const int64_t n_pos = a[4] == Py_None ? 0 : c.size("rope_table", a[4], 0, 2);
  const int64_t LP = d.L + d.P;
  const at::Tensor &kv_a = c.tensor("kv_a", a[1]);
  const int64_t ld = T > 1 ? kv_a.stride(0) : LP;
  if (kv_a.scalar_type() != d.type || kv_a.size(1) != LP || kv_a.stride(1) != 1 || ld < LP)
    c.refuse("kv_a has to be [T, " + std::to_string(LP) + "] " + type_name(d.type) +
             " with contiguous rows");
  const auto *qsl = c.take<int32_t>("query_start_loc", a[2], I32, {R + 1});
  const auto *lens = c.take<int32_t>("seq_lens", a[3], I32, {R});
  const auto *table = c.take<int32_t>("block_table", a[6], I32, {R, stride});
  void *cache = c.take("kv_cache", a[5], d.type, {blocks, d.bs, LP});
  const void *norm = c.take("norm_weight", a[7], d.type, {d.L});
  const double eps = PyFloat_AsDouble(a[8]);
  if (eps == -1.0 && PyErr_Occurred()) throw PythonError();
  const auto *pos = c.take<int32_t>("positions", a[9], I32, {T});
  const bool interleaved = truth(a[10]);
  const auto *rope = c.take<float>("rope_table", a[4], F32, {n_pos, d.P});
  void *latent = c.take("new_latent", a[11], d.type, {T, LP});
  const void *q = c.take("q", a[12], d.type, {T, d.H, d.Dn + d.P});
  auto *status = c.take<int32_t>("dev_status", a[14], I32, {1});
  c.on_device("kv_a", kv_a);
  void *pe = nullptr;
  int64_t pe_ld = d.P;
  if (a[13] != Py_None) {
    const at::Tensor &t = c.tensor("q_pe_out", a[13]);
    const Shape want = {T, d.H, d.P};
    c.on_device("q_pe_out", t);
    bool good = t.scalar_type() == d.type && t.sizes() == c10::IntArrayRef(want);
    if (good) {
      pe_ld = d.H > 1 ? t.stride(1) : T > 1 ? t.stride(0) : d.P;
      good = (d.P <= 1 || t.stride(2) == 1) && (T <= 1 || t.stride(0) == d.H * pe_ld);
    }
    if (!good) {
      std::ostringstream s;
      s << "q_pe_out has to be a " << c10::IntArrayRef(want) << " " << d.type
        << " view of evenly spaced rows";
      c.refuse(s.str());
    }
    pe = t.data_ptr();
  }
  if (d.P == 0 && a[12] != Py_None && a[13] != Py_None) q = pe = nullptr;  // nothing to rotate
  const int32_t t32 = narrow(T, w, "kv_a"), r32 = narrow(R, w, "seq_lens"),
                p32 = narrow(n_pos, w, "rope_table"), b32 = narrow(blocks, w, "kv_cache"),
                s32 = narrow(stride, w, "block_table");
  const void *x = kv_a.data_ptr();
  void *s = c.stream(a[15]);
  return unlocked([&] {
    return mla_append_latent(&d.c, x, ld, norm, float(eps), t32, r32, qsl, lens, pos, rope, p32,
                             interleaved, cache, b32, table, s32, latent, q, pe, pe_ld, status, s);
  });
}

// dims, q, w_kv_b, q_latent, rope_columns, stream
int absorb(PyObject *const *a) {
  const char *w = "mla_absorb_query";
  const Dims d(a[0]);
  Call c(w);
  const int64_t T = c.size("q", a[1], 0, 3);
  const void *q = c.take("q", a[1], d.type, {T, d.H, d.Dn + d.P});
  const void *kv_b = c.take("w_kv_b", a[2], d.type, {d.H * (d.Dn + d.Dv), d.L});
  void *out = c.take("q_latent", a[3], d.type, {T, d.H, d.L + d.P});
  const bool rope = truth(a[4]);
  const int32_t t32 = narrow(T, w, "q");
  void *s = c.stream(a[5]);
  return unlocked([&] { return mla_absorb_query(&d.c, q, t32, kv_b, rope, out, s); });
}

// dims, o_latent, w_kv_b, out, stream
int expand(PyObject *const *a) {
  const char *w = "mla_expand_output";
  const Dims d(a[0]);
  Call c(w);
  const int64_t T = c.size("o_latent", a[1], 0, 3);
  const void *o = c.take("o_latent", a[1], d.type, {T, d.H, d.L});
  const void *kv_b = c.take("w_kv_b", a[2], d.type, {d.H * (d.Dn + d.Dv), d.L});
  void *out = c.take("out", a[3], d.type, {T, d.H, d.Dv});
  const int32_t t32 = narrow(T, w, "o_latent");
  void *s = c.stream(a[4]);
  return unlocked([&] { return mla_expand_output(&d.c, o, t32, kv_b, out, s); });
}

// dims, causal, query_start_loc, seq_lens, q_latent, kv_cache, block_table,
// workspace, o_latent, lse, dev_status, stream
int attend(PyObject *const *a) {
  const char *w = "mla_latent_attn";
  const Dims d(a[0]);
  Call c(w);
  const int64_t T = c.size("q_latent", a[4], 0, 3), R = c.size("seq_lens", a[3], 0, 1);
  const int64_t blocks = c.size("kv_cache", a[5], 0, 3), stride = c.size("block_table", a[6], 1, 2);
  const int64_t LP = d.L + d.P;
  const int64_t ws_bytes = a[7] == Py_None ? 0 : c.tensor("workspace", a[7]).numel();
  const bool causal = truth(a[1]);
  const void *q = c.take("q_latent", a[4], d.type, {T, d.H, LP});
  const auto *qsl = c.take<int32_t>("query_start_loc", a[2], I32, {R + 1});
  const auto *lens = c.take<int32_t>("seq_lens", a[3], I32, {R});
  const auto *table = c.take<int32_t>("block_table", a[6], I32, {R, stride});
  const void *cache = c.take("kv_cache", a[5], d.type, {blocks, d.bs, LP});
  void *ws = c.take("workspace", a[7], ScalarType::Byte, {ws_bytes});
  void *o = c.take("o_latent", a[8], d.type, {T, d.H, d.L});
  auto *lse = c.take<float>("lse", a[9], F32, {d.H, T});
  auto *status = c.take<int32_t>("dev_status", a[10], I32, {1});
  const int32_t t32 = narrow(T, w, "q_latent"), r32 = narrow(R, w, "seq_lens"),
                b32 = narrow(blocks, w, "kv_cache"), s32 = narrow(stride, w, "block_table");
  void *s = c.stream(a[11]);
  return unlocked([&] {
    return mla_latent_attn(&d.c, causal, r32, qsl, lens, t32, q, cache, b32, table, s32, ws,
                           size_t(ws_bytes), o, lse, status, s);
  });
}

// parents, query_start_loc, seq_lens, tree_mask, positions, dev_status, stream
int layout(PyObject *const *a) {
  const char *w = "mla_tree_layout";
  Call c(w);
  const int64_t T = c.size("parents", a[0], 0, 1), R = c.size("seq_lens", a[2], 0, 1);
  const int64_t words = c.size("tree_mask", a[3], 1, 2);
  const auto *parents = c.take<int32_t>("parents", a[0], I32, {T});
  const auto *qsl = c.take<int32_t>("query_start_loc", a[1], I32, {R + 1});
  const auto *lens = c.take<int32_t>("seq_lens", a[2], I32, {R});
  auto *mask = c.take<uint64_t>("tree_mask", a[3], I64, {T, words});
  auto *positions = c.take<int32_t>("positions", a[4], I32, {T});
  auto *status = c.take<int32_t>("dev_status", a[5], I32, {1});
  const int32_t t32 = narrow(T, w, "parents"), r32 = narrow(R, w, "seq_lens"),
                w32 = narrow(words, w, "tree_mask");
  void *s = c.stream(a[6]);
  return unlocked([&] {
    return mla_tree_layout(t32, r32, qsl, lens, parents, w32, mask, positions, status, s);
  });
}

// dims, query_start_loc, seq_lens, tree_mask, q_latent, kv_cache, block_table,
// workspace, o_latent, lse, dev_status, stream
int tree_attend(PyObject *const *a) {
  const char *w = "mla_tree_attn";
  const Dims d(a[0]);
  Call c(w);
  const int64_t T = c.size("q_latent", a[4], 0, 3), R = c.size("seq_lens", a[2], 0, 1);
  const int64_t blocks = c.size("kv_cache", a[5], 0, 3), stride = c.size("block_table", a[6], 1, 2);
  const int64_t words = c.size("tree_mask", a[3], 1, 2);
  const int64_t LP = d.L + d.P;
  const int64_t ws_bytes = a[7] == Py_None ? 0 : c.tensor("workspace", a[7]).numel();
  const void *q = c.take("q_latent", a[4], d.type, {T, d.H, LP});
  const auto *qsl = c.take<int32_t>("query_start_loc", a[1], I32, {R + 1});
  const auto *lens = c.take<int32_t>("seq_lens", a[2], I32, {R});
  const auto *mask = c.take<uint64_t>("tree_mask", a[3], I64, {T, words});
  const auto *table = c.take<int32_t>("block_table", a[6], I32, {R, stride});
  const void *cache = c.take("kv_cache", a[5], d.type, {blocks, d.bs, LP});
  void *ws = c.take("workspace", a[7], ScalarType::Byte, {ws_bytes});
  void *o = c.take("o_latent", a[8], d.type, {T, d.H, d.L});
  auto *lse = c.take<float>("lse", a[9], F32, {d.H, T});
  auto *status = c.take<int32_t>("dev_status", a[10], I32, {1});
  const int32_t t32 = narrow(T, w, "q_latent"), r32 = narrow(R, w, "seq_lens"),
                b32 = narrow(blocks, w, "kv_cache"), s32 = narrow(stride, w, "block_table"),
                w32 = narrow(words, w, "tree_mask");
  void *s = c.stream(a[11]);
  return unlocked([&] {
    return mla_tree_attn(&d.c, r32, qsl, lens, mask, w32, t32, q, cache, b32, table, s32, ws,
                         size_t(ws_bytes), o, lse, status, s);
  });
}

// target, draft, tokens, parents, query_start_loc, uniform, uniform_next, path,
// num_kept, next_tokens, dev_status, stream
int verify(PyObject *const *a) {
  const char *w = "mla_verify_tree";
  Call c(w);
  const int64_t T = c.size("target", a[0], 0, 2), V = c.size("target", a[0], 1, 2);
  const int64_t R = c.size("path", a[7], 0, 2), deep = c.size("path", a[7], 1, 2);
  const at::Tensor &target = c.tensor("target", a[0]);
  const ScalarType type = target.scalar_type();
  int32_t dtype = MLA_DTYPE_F32;
  if (type == ScalarType::BFloat16)
    dtype = MLA_DTYPE_BF16;
  else if (type != F32)
    c.refuse("target has to be float32 or bfloat16, got " + type_name(type));
  int64_t ld[2] = {V, V};
  const void *rows[2] = {nullptr, nullptr};
  for (int i = 0; i < 2; ++i) {
    if (i == 1 && a[1] == Py_None) break;
    const char *name = i ? "draft" : "target";
    const at::Tensor &t = c.tensor(name, a[i]);
    c.on_device(name, t);
    if (T > 1 && t.dim() == 2) ld[i] = t.stride(0);
    if (t.scalar_type() != type || t.dim() != 2 || t.size(0) != T || t.size(1) != V ||
        (V > 1 && t.stride(1) != 1) || ld[i] < V)
      c.refuse(std::string(name) + " has to be [" + std::to_string(T) + ", " + std::to_string(V) +
               "] " + type_name(type) + " with contiguous rows");
    rows[i] = t.data_ptr();
  }
  const auto *tokens = c.take<int32_t>("tokens", a[2], I32, {T});
  const auto *parents = c.take<int32_t>("parents", a[3], I32, {T});
  const auto *qsl = c.take<int32_t>("query_start_loc", a[4], I32, {R + 1});
  const auto *u = c.take<float>("uniform", a[5], F32, {T});
  const auto *u_next = c.take<float>("uniform_next", a[6], F32, {R});
  if ((a[5] == Py_None) != (a[6] == Py_None)) c.refuse("uniform and uniform_next go together");
  auto *path = c.take<int32_t>("path", a[7], I32, {R, deep});
  auto *kept = c.take<int32_t>("num_kept", a[8], I32, {R});
  auto *next = c.take<int32_t>("next_tokens", a[9], I32, {R});
  auto *status = c.take<int32_t>("dev_status", a[10], I32, {1});
  const int32_t t32 = narrow(T, w, "target"), v32 = narrow(V, w, "target"),
                r32 = narrow(R, w, "path"), p32 = narrow(deep, w, "path");
  void *s = c.stream(a[11]);
  return unlocked([&] {
    return mla_verify_tree(dtype, t32, r32, v32, rows[0], ld[0], rows[1], ld[1], tokens, parents,
                           qsl, u, u_next, path, p32, kept, next, status, s);
  });
}

// dims, path, num_kept, query_start_loc, seq_lens, kv_caches, block_table,
// new_seq_lens, num_tokens, dev_status, stream
int commit(PyObject *const *a) {
  const char *w = "mla_commit_tree";
  const Dims d(a[0]);
  Call c(w);
  const int64_t R = c.size("path", a[1], 0, 2), deep = c.size("path", a[1], 1, 2);
  const int64_t stride = c.size("block_table", a[6], 1, 2), LP = d.L + d.P;
  const auto *path = c.take<int32_t>("path", a[1], I32, {R, deep});
  const auto *kept = c.take<int32_t>("num_kept", a[2], I32, {R});
  const auto *qsl = c.take<int32_t>("query_start_loc", a[3], I32, {R + 1});
  const auto *lens = c.take<int32_t>("seq_lens", a[4], I32, {R});
  const auto *table = c.take<int32_t>("block_table", a[6], I32, {R, stride});
  std::vector<void *> caches;
  int64_t blocks = 0;
  auto layer = [&](PyObject *o) {
    if (caches.empty()) blocks = c.size("kv_caches", o, 0, 3);
    void *p = c.take("kv_caches", o, d.type, {blocks, d.bs, LP});
    if (!p && blocks > 0) c.refuse("kv_caches has to be tensors");
    caches.push_back(p);
  };
  if (PyList_Check(a[5]) || PyTuple_Check(a[5])) {
    const Py_ssize_t n = PySequence_Fast_GET_SIZE(a[5]);
    for (Py_ssize_t i = 0; i < n; ++i) layer(PySequence_Fast_GET_ITEM(a[5], i));
  } else {
    layer(a[5]);
  }
  if (blocks == 0) caches.clear();  // nothing to move
  auto *new_lens = c.take<int32_t>("new_seq_lens", a[7], I32, {R});
  int64_t T = INT32_MAX;
  if (a[8] != Py_None) {
    T = PyLong_AsLongLong(a[8]);
    if (T == -1 && PyErr_Occurred()) throw PythonError();
  }
  auto *status = c.take<int32_t>("dev_status", a[9], I32, {1});
  const int32_t t32 = narrow(T, w, "num_tokens"), r32 = narrow(R, w, "path"),
                p32 = narrow(deep, w, "path"), b32 = narrow(blocks, w, "kv_caches"),
                s32 = narrow(stride, w, "block_table"),
                l32 = narrow(int64_t(caches.size()), w, "kv_caches");
  void *s = c.stream(a[10]);
  return unlocked([&] {
    return mla_commit_tree(&d.c, r32, t32, path, p32, kept, qsl, lens, caches.data(), l32, b32,
                           table, s32, new_lens, status, s);
  });
}

// No C++ exception leaves the module.
template <int (*F)(PyObject *const *), int N>
PyObject *entry(PyObject *, PyObject *const *args, Py_ssize_t n) {
  if (n != N) return PyErr_Format(PyExc_TypeError, "%d arguments expected, got %zd", N, n);
  try {
    return PyLong_FromLong(F(args));
  } catch (const PythonError &) {
  } catch (const std::invalid_argument &e) {
    PyErr_SetString(PyExc_ValueError, e.what());
  } catch (const std::exception &e) {
    PyErr_SetString(PyExc_RuntimeError, e.what());
  }
  return nullptr;
}

template <typename F>
PyCFunction fast(F f) {
  return reinterpret_cast<PyCFunction>(reinterpret_cast<void *>(f));
}

PyMethodDef methods[] = {
    {"append", fast(entry<append, 16>), METH_FASTCALL, nullptr},
    {"absorb", fast(entry<absorb, 6>), METH_FASTCALL, nullptr},
    {"expand", fast(entry<expand, 5>), METH_FASTCALL, nullptr},
    {"attend", fast(entry<attend, 12>), METH_FASTCALL, nullptr},
    {"layout", fast(entry<layout, 7>), METH_FASTCALL, nullptr},
    {"tree_attend", fast(entry<tree_attend, 12>), METH_FASTCALL, nullptr},
    {"verify", fast(entry<verify, 12>), METH_FASTCALL, nullptr},
    {"commit", fast(entry<commit, 11>), METH_FASTCALL, nullptr},
    {nullptr, nullptr, 0, nullptr}};

PyModuleDef module = {PyModuleDef_HEAD_INIT, "_decode", nullptr, -1, methods,
                      nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__decode() {
  const char *fields[8] = {"num_heads", "kv_lora_rank", "qk_rope_dim", "qk_nope_dim",
                           "v_dim", "block_size", "softmax_scale", "dtype"};
  for (int i = 0; i < 8; ++i)
    if (!(names.field[i] = PyUnicode_InternFromString(fields[i]))) return nullptr;
  if (!(names.cuda_stream = PyUnicode_InternFromString("cuda_stream"))) return nullptr;
  PyObject *m = PyModule_Create(&module);
  if (m && PyModule_AddStringConstant(m, "built_for", MLA_BUILT_FOR)) Py_CLEAR(m);
  return m;
}
