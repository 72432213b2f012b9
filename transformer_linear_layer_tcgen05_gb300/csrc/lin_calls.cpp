// lin_calls.cpp -- the short calls' way from Python tensors to the C ABI: the
// extension module _lin_calls, whose functions check their tensors (type,
// device, shape, strides), fill in the shape structures of include/lin.h and
// call the library, whose addresses lin.py binds once. A call of attention or
// of the norms and rotation takes 3 to 10 us on the GPU where it is short, and
// the same checks written in Python took 8 to 18 us of host time before the
// launch; here they take under one.
//
// Marshalling only: the library makes its own checks of addresses, overlaps
// and extents behind these.
#include <Python.h>

#include <c10/cuda/CUDAStream.h>
#include <torch/csrc/autograd/python_variable.h>
#include <torch/version.h>

#include <cmath>
#include <exception>
#include <initializer_list>
#include <string>

#include "lin.h"

namespace {

// Addresses of the library's functions, in the order of kNames.
const char* const kNames[] = {"lin_attention", "lin_attention_backward", "lin_qk_norm_rope",
                              "lin_qk_norm_rope_backward", "lin_distill_topk"};
void* g_address[5];

template <typename F>
F* bound(int i) {
  return reinterpret_cast<F*>(g_address[i]);
}

// An error that is already set as the Python exception.
struct Raised {};

[[noreturn]] void raise(PyObject* type, const std::string& text) {
  PyErr_SetString(type, text.c_str());
  throw Raised();
}

std::string list_of(c10::IntArrayRef sizes) {
  std::string s = "[";
  for (size_t i = 0; i < sizes.size(); ++i) s += (i ? ", " : "") + std::to_string(sizes[i]);
  return s + "]";
}

const at::Tensor* tensor(PyObject* o) {
  return THPVariable_Check(o) ? &THPVariable_Unpack(o) : nullptr;
}

// [tokens, heads, dim] CUDA tensors of one 16-bit type, the last dimension
// contiguous; views of a packed buffer are fine.
struct Heads {
  bool first = true;
  at::ScalarType type = at::kHalf;

  const at::Tensor& take(PyObject* o, const char* name, lin_heads* out) {
    const at::Tensor* t = tensor(o);
    if (!t || !t->is_cuda() || t->dim() != 3)
      raise(PyExc_TypeError, std::string(name) + " must be a CUDA tensor [tokens, heads, dim]");
    if (first) type = t->scalar_type();
    first = false;
    if (t->scalar_type() != type || (type != at::kHalf && type != at::kBFloat16))
      raise(PyExc_TypeError, std::string(name) + " must be float16 or bfloat16, all of one type");
    if (t->stride(2) != 1 && t->size(2) > 1)
      raise(PyExc_ValueError, std::string(name) + ": the entries of a head must be contiguous");
    *out = lin_heads{t->data_ptr(), t->stride(0), t->stride(1)};
    return *t;
  }
  int32_t dtype() const { return type == at::kBFloat16 ? LIN_BFLOAT16 : LIN_BINARY16; }
};

void same_shape(const at::Tensor& t, const char* name, const at::Tensor& like) {
  if (t.sizes() != like.sizes())
    raise(PyExc_ValueError, std::string(name) + " must be " + list_of(like.sizes()));
}

// A contiguous CUDA tensor of the given type and shape.
template <typename T>
T* flat(PyObject* o, const char* name, at::ScalarType type, c10::IntArrayRef shape) {
  const at::Tensor* t = tensor(o);
  if (!t || t->scalar_type() != type || !t->is_cuda() || !t->is_contiguous() || t->sizes() != shape)
    raise(PyExc_TypeError, std::string(name) + " must be a contiguous " +
                               (type == at::kInt ? "torch.int32" : "torch.float32") +
                               " CUDA tensor " + list_of(shape));
  return static_cast<T*>(t->data_ptr());
}
float* f32(PyObject* o, const char* name, c10::IntArrayRef shape) {
  return flat<float>(o, name, at::kFloat, shape);
}

// A float32 CUDA matrix with contiguous rows, any row stride.
const at::Tensor& f32_rows(PyObject* o, const char* name) {
  const at::Tensor* t = tensor(o);
  if (!t || t->scalar_type() != at::kFloat || !t->is_cuda() || t->dim() != 2)
    raise(PyExc_TypeError, std::string(name) + " must be a float32 CUDA matrix");
  if (t->size(1) > 1 && t->stride(1) != 1)
    raise(PyExc_ValueError, std::string(name) + " must have contiguous rows");
  return *t;
}

int64_t integer(PyObject* o, const char* name) {
  if (o == Py_None) raise(PyExc_ValueError, std::string(name) + " is missing");
  const long long v = PyLong_AsLongLong(o);
  if (v == -1 && PyErr_Occurred()) throw Raised();
  return v;
}
double number(PyObject* o) {
  const double v = PyFloat_AsDouble(o);
  if (v == -1.0 && PyErr_Occurred()) throw Raised();
  return v;
}
bool truth(PyObject* o) {
  const int v = PyObject_IsTrue(o);
  if (v < 0) throw Raised();
  return v != 0;
}

// None: torch's current stream; a number: the handle itself.
lin_stream_t stream_of(PyObject* o) {
  if (o == Py_None)
    return reinterpret_cast<lin_stream_t>(c10::cuda::getCurrentCUDAStream().stream());
  return reinterpret_cast<lin_stream_t>(static_cast<intptr_t>(integer(o, "stream")));
}

// The offsets of packed sequences and their longest lengths.
void sequences(lin_attention_shape* s, PyObject* cu_q, PyObject* cu_k, PyObject* max_q,
               PyObject* max_k) {
  s->sequences = 1;
  s->max_q = s->tokens_q;
  s->max_k = s->tokens_k;
  s->cu_q = s->cu_k = nullptr;
  if (cu_q == Py_None && cu_k == Py_None) return;
  if (cu_q == Py_None || cu_k == Py_None) raise(PyExc_ValueError, "cu_q and cu_k go together");
  if (max_q == Py_None || max_k == Py_None)
    raise(PyExc_ValueError, "packed sequences need max_q and max_k");
  auto offsets = [&](PyObject* o, const char* name) -> const at::Tensor& {
    const at::Tensor* t = tensor(o);
    if (!t || t->scalar_type() != at::kInt || !t->is_cuda() || !t->is_contiguous() ||
        t->dim() != 1 || t->numel() < 1)
      raise(PyExc_TypeError, std::string(name) + " must be a contiguous torch.int32 CUDA tensor");
    return *t;
  };
  const at::Tensor &q = offsets(cu_q, "cu_q"), &k = offsets(cu_k, "cu_k");
  if (q.numel() != k.numel())
    raise(PyExc_ValueError, "cu_q and cu_k must have the same number of entries");
  s->sequences = k.numel() - 1;
  s->cu_q = static_cast<const int32_t*>(q.data_ptr());
  s->cu_k = static_cast<const int32_t*>(k.data_ptr());
  s->max_q = integer(max_q, "max_q");
  s->max_k = integer(max_k, "max_k");
}

lin_attention_shape attention_shape(const Heads& h, const at::Tensor& q, const at::Tensor& k,
                                    const at::Tensor& v, PyObject* const* how) {
  if (k.size(2) != q.size(2) || v.sizes() != k.sizes())
    raise(PyExc_ValueError, "shape mismatch: Q" + list_of(q.sizes()) + " K" + list_of(k.sizes()) +
                                " V" + list_of(v.sizes()));
  lin_attention_shape s{};
  s.dtype = h.dtype();
  s.tokens_q = q.size(0);
  s.heads_q = q.size(1);
  s.dim = q.size(2);
  s.tokens_k = k.size(0);
  s.heads_kv = k.size(1);
  sequences(&s, how[0], how[1], how[2], how[3]);
  s.causal = truth(how[4]) ? 1 : 0;
  s.scale = how[5] == Py_None ? (float)(1.0 / std::sqrt((double)s.dim)) : (float)number(how[5]);
  return s;
}

// The status that `body` (a call's checks and the call) gives, as a Python
// number; its errors as Python exceptions.
template <typename Body>
PyObject* guarded(Py_ssize_t n, Py_ssize_t want, Body&& body) {
  if (n != want) {
    PyErr_Format(PyExc_TypeError, "%zd arguments, not %zd", want, n);
    return nullptr;
  }
  try {
    return PyLong_FromLong((long)body());
  } catch (const Raised&) {
    return nullptr;
  } catch (const std::exception& e) {
    PyErr_SetString(PyExc_RuntimeError, e.what());
    return nullptr;
  }
}
// The library's function without the interpreter's lock.
template <typename F, typename... A>
lin_status unlocked(F* f, A... a) {
  lin_status st;
  Py_BEGIN_ALLOW_THREADS
  st = f(a...);
  Py_END_ALLOW_THREADS
  return st;
}

// Q, K, V, O, LSE, cu_q, cu_k, max_q, max_k, causal, scale, stream
PyObject* attention(PyObject*, PyObject* const* a, Py_ssize_t n) {
  return guarded(n, 12, [&] {
    Heads h;
    lin_heads q, k, v, o;
    const at::Tensor &tq = h.take(a[0], "Q", &q), &tk = h.take(a[1], "K", &k),
                     &tv = h.take(a[2], "V", &v), &to = h.take(a[3], "O", &o);
    const lin_attention_shape s = attention_shape(h, tq, tk, tv, a + 5);
    same_shape(to, "O", tq);
    float* lse = f32(a[4], "LSE", {s.heads_q, s.tokens_q});
    return unlocked(bound<decltype(lin_attention)>(0), &s, &q, &k, &v, &o, lse, stream_of(a[11]));
  });
}

// Q, K, V, O, LSE, dO, dQ, dK, dV, cu_q, cu_k, max_q, max_k, causal, scale, stream
PyObject* attention_backward(PyObject*, PyObject* const* a, Py_ssize_t n) {
  return guarded(n, 16, [&] {
    Heads h;
    lin_heads q, k, v, o, dout, dq, dk, dv;
    const at::Tensor &tq = h.take(a[0], "Q", &q), &tk = h.take(a[1], "K", &k),
                     &tv = h.take(a[2], "V", &v), &to = h.take(a[3], "O", &o),
                     &tdo = h.take(a[5], "dO", &dout), &tdq = h.take(a[6], "dQ", &dq),
                     &tdk = h.take(a[7], "dK", &dk), &tdv = h.take(a[8], "dV", &dv);
    const lin_attention_shape s = attention_shape(h, tq, tk, tv, a + 9);
    same_shape(to, "O", tq);
    same_shape(tdo, "dO", tq);
    same_shape(tdq, "dQ", tq);
    same_shape(tdk, "dK", tk);
    same_shape(tdv, "dV", tk);
    const float* lse = f32(a[4], "LSE", {s.heads_q, s.tokens_q});
    return unlocked(bound<decltype(lin_attention_backward)>(1), &s, &q, &k, &v, &o, lse, &dout,
                    &dq, &dk, &dv, stream_of(a[15]));
  });
}

// X, wq, wk, COS, SIN, positions, Q, K, V, eps, interleaved
struct RopeArgs {
  lin_qk_norm_rope_shape s{};
  lin_heads q, k, v;
  const float *x, *wq, *wk, *cos = nullptr, *sin = nullptr;
  const int32_t* positions = nullptr;
  c10::IntArrayRef x_sizes;

  RopeArgs(PyObject* const* a, const char* const (&names)[3]) {
    Heads h;
    const at::Tensor &tq = h.take(a[6], names[0], &q), &tk = h.take(a[7], names[1], &k),
                     &tv = h.take(a[8], names[2], &v);
    s.dtype = h.dtype();
    s.tokens = tq.size(0);
    s.heads_q = tq.size(1);
    s.dim = tq.size(2);
    s.heads_kv = tk.size(1);
    const at::Tensor* tx = tensor(a[0]);
    if (!tx || tx->scalar_type() != at::kFloat || !tx->is_cuda())
      raise(PyExc_TypeError, "X must be a float32 CUDA tensor");
    if (tx->dim() != 2 || !tx->is_contiguous())
      raise(PyExc_ValueError, "X must be a contiguous 2-D tensor");
    if (tk.size(0) != s.tokens || tk.size(2) != s.dim || tv.sizes() != tk.sizes() ||
        tx->size(0) != s.tokens || tx->size(1) != (s.heads_q + 2 * s.heads_kv) * s.dim)
      raise(PyExc_ValueError, "shape mismatch: X" + list_of(tx->sizes()) + " " + names[0] +
                                  list_of(tq.sizes()) + " " + names[1] + list_of(tk.sizes()) + " " +
                                  names[2] + list_of(tv.sizes()));
    x = static_cast<const float*>(tx->data_ptr());
    x_sizes = tx->sizes();
    if (a[3] != Py_None || a[4] != Py_None) {
      const at::Tensor* tc = tensor(a[3]);
      if (!tc || tc->scalar_type() != at::kFloat || !tc->is_cuda())
        raise(PyExc_TypeError, "COS must be a float32 CUDA tensor");
      if (tc->dim() != 2 || !tc->is_contiguous())
        raise(PyExc_ValueError, "COS must be a contiguous 2-D tensor");
      cos = static_cast<const float*>(tc->data_ptr());
      sin = f32(a[4], "SIN", tc->sizes());
      s.table_rows = tc->size(0);
      s.rot = 2 * tc->size(1);
    }
    if (a[5] != Py_None) positions = flat<int32_t>(a[5], "positions", at::kInt, {s.tokens});
    wq = f32(a[1], "wq", {s.dim});
    wk = f32(a[2], "wk", {s.dim});
    s.eps = (float)number(a[9]);
    s.interleaved = truth(a[10]) ? 1 : 0;
  }
};

// RopeArgs', stream
PyObject* qk_norm_rope(PyObject*, PyObject* const* a, Py_ssize_t n) {
  return guarded(n, 12, [&] {
    const RopeArgs r(a, {"Q", "K", "V"});
    return unlocked(bound<decltype(lin_qk_norm_rope)>(2), &r.s, r.x, r.wq, r.wk, r.cos, r.sin,
                    r.positions, &r.q, &r.k, &r.v, stream_of(a[11]));
  });
}

// RopeArgs', dX, dwq, dwk, stream
PyObject* qk_norm_rope_backward(PyObject*, PyObject* const* a, Py_ssize_t n) {
  return guarded(n, 15, [&] {
    const RopeArgs r(a, {"dQ", "dK", "dV"});
    float* dx = f32(a[11], "dX", r.x_sizes);
    float* dwq = f32(a[12], "dwq", {r.s.dim});
    float* dwk = f32(a[13], "dwk", {r.s.dim});
    return unlocked(bound<decltype(lin_qk_norm_rope_backward)>(3), &r.s, r.x, r.wq, r.wk, r.cos,
                    r.sin, r.positions, &r.q, &r.k, &r.v, dx, dwq, dwk, stream_of(a[14]));
  });
}

// LOGITS, ids, teacher, DLOGITS, losses, loss_sum, temperature, inv_norm, stream
PyObject* distill_topk(PyObject*, PyObject* const* a, Py_ssize_t n) {
  return guarded(n, 9, [&] {
    const at::Tensor& z = f32_rows(a[0], "logits");
    const int64_t M = z.size(0), V = z.size(1);
    const at::Tensor* ti = tensor(a[1]);
    const int64_t K = ti && ti->dim() == 2 ? ti->size(1) : 0;
    const int32_t* ids = flat<int32_t>(a[1], "ids", at::kInt, {M, K});
    float* dz = nullptr;
    int64_t ldd = 0;
    if (a[3] != Py_None) {
      const at::Tensor& d = f32_rows(a[3], "dlogits");
      same_shape(d, "dlogits", z);
      dz = static_cast<float*>(d.data_ptr());
      ldd = d.stride(0);
    }
    const float* teacher = f32(a[2], "teacher", {M, K});
    float* losses = f32(a[4], "losses", {M});
    float* loss_sum = f32(a[5], "loss_sum", {1});
    return unlocked(bound<decltype(lin_distill_topk)>(4), static_cast<const float*>(z.data_ptr()),
                    z.stride(0), ids, teacher, dz, ldd, losses, loss_sum, M, V, K,
                    (float)number(a[6]), (float)number(a[7]), stream_of(a[8]));
  });
}

// {name: address} of the library's functions: all of them, or none is taken.
PyObject* bind(PyObject*, PyObject* addresses) {
  void* got[5];
  for (int i = 0; i < 5; ++i) {
    PyObject* v = PyMapping_GetItemString(addresses, kNames[i]);
    if (!v) return nullptr;
    got[i] = PyLong_AsVoidPtr(v);
    Py_DECREF(v);
    if (!got[i]) {
      if (!PyErr_Occurred()) PyErr_SetString(PyExc_ValueError, kNames[i]);
      return nullptr;
    }
  }
  for (int i = 0; i < 5; ++i) g_address[i] = got[i];
  Py_RETURN_NONE;
}

template <typename F>
PyCFunction as_method(F f) {
  return reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(f));
}

PyMethodDef kMethods[] = {
    {"bind", bind, METH_O, nullptr},
    {"attention", as_method(attention), METH_FASTCALL, nullptr},
    {"attention_backward", as_method(attention_backward), METH_FASTCALL, nullptr},
    {"qk_norm_rope", as_method(qk_norm_rope), METH_FASTCALL, nullptr},
    {"qk_norm_rope_backward", as_method(qk_norm_rope_backward), METH_FASTCALL, nullptr},
    {"distill_topk", as_method(distill_topk), METH_FASTCALL, nullptr},
    {nullptr, nullptr, 0, nullptr}};

PyModuleDef kModule = {PyModuleDef_HEAD_INIT, "_lin_calls", nullptr, -1, kMethods,
                       nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__lin_calls() {
  PyObject* m = PyModule_Create(&kModule);
  // (whose classes and ABI the module was compiled against)
  if (m && PyModule_AddStringConstant(m, "torch_version", TORCH_VERSION) < 0) {
    Py_DECREF(m);
    return nullptr;
  }
  return m;
}
