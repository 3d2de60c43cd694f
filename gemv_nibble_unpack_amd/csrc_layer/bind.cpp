// Python marshalling of the decoder-layer and MXFP4 operators: checks torch
// tensors, allocates outputs that the caller left out, and calls the C entry
// points of include/gemv_nibble_unpack_layer.h and gemv_nibble_unpack_mx.h (the
// latter in ../csrc_mx/bind_mx.hpp). No arithmetic happens here.
//
// These calls carry up to ten tensors each and their kernels take a few
// microseconds for a single token, so the marshalling decides what a decode
// step costs: read attribute by attribute from Python, a call's checks and
// allocations took 12 us (attention) to 15 us (norm, append) on the host;
// reading the tensors in C++ leaves mostly the launch itself.
//
// Host code only, built against torch's C++ headers.

#define PY_SSIZE_T_CLEAN
#include <Python.h>

#include <ATen/core/Tensor.h>
#include <ATen/hip/EmptyTensor.h>
#include <c10/core/DeviceGuard.h>
#include <c10/hip/HIPFunctions.h>
#include <c10/hip/HIPStream.h>
#include <torch/csrc/autograd/python_variable.h>

#include "gemv_nibble_unpack_layer.h"
#include "gemv_nibble_unpack_mx.h"

namespace {

using at::ScalarType;
using at::Tensor;

struct Refuse {                 // a ValueError
  const char* why;
};

const Tensor& tensor(PyObject* o, const char* why) {
  if (!THPVariable_Check(o)) throw Refuse{why};
  return THPVariable_Unpack(o);
}
// dense device tensor, or nullptr for None
const Tensor* optional(PyObject* o, const char* why) {
  return o == Py_None ? nullptr : &tensor(o, why);
}
// `t` beside `first`, the tensor whose device the call runs on
void beside(const Tensor& t, const Tensor& first) {
  if (!t.is_cuda()) throw Refuse{"expected a device tensor"};
  if (t.device() != first.device()) throw Refuse{"all tensors must be on one device"};
}
void dense(const Tensor& t, const Tensor& first) {
  beside(t, first);
  if (!t.is_contiguous()) throw Refuse{"expected a contiguous tensor"};
}
void* ptr(const Tensor* t) { return t ? t->data_ptr() : nullptr; }

long integer(PyObject* o) {
  const long v = PyLong_AsLong(o);
  if (v == -1 && PyErr_Occurred()) throw Refuse{nullptr};
  return v;
}
int integer32(PyObject* o) {
  const long v = integer(o);
  if (v != (int)v) throw Refuse{"an integer argument is out of range"};
  return (int)v;
}
double real(PyObject* o) {
  const double v = PyFloat_AsDouble(o);
  if (v == -1.0 && PyErr_Occurred()) throw Refuse{nullptr};
  return v;
}
// Makes the tensors' device the current one for a launch, where it is another
// (asking first costs 0.1 us of a call's host time, a plain device guard 0.2)
struct OnDevice {
  c10::OptionalDeviceGuard guard;
  explicit OnDevice(const Tensor& t) {
    if (c10::hip::current_device() != t.get_device()) guard.reset_device(t.device());
  }
};
// None: torch's current stream on the tensors' device; else a raw stream
hipStream_t stream_of(PyObject* o, const Tensor& t) {
  if (o == Py_None) return c10::hip::getCurrentHIPStream(t.get_device()).stream();
  return (hipStream_t)PyLong_AsVoidPtr(o);
}
Tensor fresh(c10::IntArrayRef size, ScalarType dt, const Tensor& like) {
  return Tensor(at::detail::empty_cuda(size, dt, like.device(), c10::nullopt));
}
int in_dtype(const Tensor& t, const char* why) {
  if (t.scalar_type() == ScalarType::Half) return W4_IN_F16;
  if (t.scalar_type() == ScalarType::Float) return W4_IN_F32;
  throw Refuse{why};
}
int narrow(int64_t v) {
  if (v != (int)v) throw Refuse{"a size is out of range"};
  return (int)v;
}

struct Cache {
  const Tensor &k, &v, &ks, &vs;
  int pages, page, kind;
};
Cache cache(PyObject* const* a, int64_t kv_heads, int64_t dim, const Tensor& first) {
  Cache c{tensor(a[0], "the cache must be four tensors"), tensor(a[1], "the cache must be four tensors"),
          tensor(a[2], "the cache must be four tensors"), tensor(a[3], "the cache must be four tensors"),
          0, 0, 0};
  const auto dt = c.k.scalar_type();
  if (c.v.scalar_type() != dt || (dt != ScalarType::Char && dt != ScalarType::Byte))
    throw Refuse{"cache codes must be int8 (INT8) or uint8 (E4M3), keys and values alike"};
  c.kind = dt == ScalarType::Char ? W4_Q_I8 : W4_Q_F8;
  const auto s = c.k.sizes(), t = c.v.sizes();
  if (s.size() != 4 || t.size() != 4 || s[1] != kv_heads || s[3] != kv8_padded_dim((int)dim) ||
      t[0] != s[0] || t[1] != s[1] || t[2] != s[3] || t[3] != s[2])
    throw Refuse{"cache shapes do not match the heads: keys [pages, heads, page, DP], values "
                 "[pages, heads, DP, page]"};
  for (const Tensor* x : {&c.ks, &c.vs})
    if (x->dim() != 2 || x->size(0) != s[0] || x->size(1) != s[1] ||
        x->scalar_type() != ScalarType::Float)
      throw Refuse{"cache scales must be float32 [pages, heads]"};
  for (const Tensor* x : {&c.k, &c.v, &c.ks, &c.vs}) dense(*x, first);
  c.pages = narrow(s[0]);
  c.page = narrow(s[2]);
  return c;
}

struct Batch {
  const Tensor &table, &len;
  const Tensor* indptr;
  int batch, cols;
};
Batch batch(PyObject* table, PyObject* len, PyObject* indptr, const Tensor& first) {
  Batch b{tensor(table, "page_table must be a tensor"), tensor(len, "kv_len must be a tensor"),
          optional(indptr, "q_indptr must be a tensor or None"), 0, 0};
  const auto I = ScalarType::Int;
  if (b.len.dim() != 1 || b.len.scalar_type() != I || b.table.scalar_type() != I ||
      (b.indptr && (b.indptr->scalar_type() != I || b.indptr->dim() != 1 ||
                    b.indptr->size(0) != b.len.size(0) + 1)))
    throw Refuse{"page_table, kv_len [batch] and q_indptr [batch + 1] must be int32"};
  if (b.table.dim() != 2 || b.table.size(0) != b.len.size(0))
    throw Refuse{"page_table must be [batch, columns]"};
  dense(b.table, first), dense(b.len, first);
  if (b.indptr) dense(*b.indptr, first);
  b.batch = narrow(b.len.size(0));
  b.cols = narrow(b.table.size(1));
  return b;
}
// elements between tokens of [tokens, heads, dim] whose heads are dense
int64_t token_stride(const Tensor& t, const Tensor& first) {
  if (t.dim() != 3 || !t.is_cuda() || t.stride(2) != 1 ||
      (t.stride(1) != t.size(2) && t.size(1) > 1))
    throw Refuse{"q, k and v must be device tensors [tokens, heads, dim] with dense heads"};
  beside(t, first);
  const int64_t row = t.size(1) * t.size(2);
  return t.size(0) > 1 ? t.stride(0) : row;
}

template <typename F>
PyObject* guarded(F f) {
  try {
    return f();
  } catch (const Refuse& r) {
    if (!PyErr_Occurred()) PyErr_SetString(PyExc_ValueError, r.why);
  } catch (const std::exception& e) {        // out of memory, mostly
    PyErr_SetString(PyExc_RuntimeError, e.what());
  }
  return nullptr;
}
bool count(Py_ssize_t n, Py_ssize_t want) {
  if (n == want) return true;
  PyErr_Format(PyExc_TypeError, "expected %zd arguments, got %zd", want, n);
  return false;
}

// x, weight, residual, eps, q_dtype, residual_out, codes, scales, stream
//   -> (codes, scales, sum), or the status of a refused call
PyObject* norm(PyObject*, PyObject* const* a, Py_ssize_t n) {
  if (!count(n, 9)) return nullptr;
  return guarded([&]() -> PyObject* {
    const Tensor& x = tensor(a[0], "x must be a tensor");
    const Tensor& w = tensor(a[1], "weight must be a tensor");
    const Tensor* r = optional(a[2], "residual must be a tensor or None");
    const Tensor* ro = optional(a[5], "residual_out must be a tensor or None");
    const Tensor* co = optional(a[6], "out must be tensors");
    const Tensor* so = optional(a[7], "out must be tensors");
    dense(x, x);
    if (x.dim() != 2) throw Refuse{"x must be [M, K]"};
    const int dt = in_dtype(x, "x must be float16 or float32");
    dense(w, x);
    if (w.scalar_type() != x.scalar_type() || w.numel() != x.size(1))
      throw Refuse{"weight must be [K] of x's type"};
    for (const Tensor* t : {r, ro})
      if (t) {
        dense(*t, x);
        if (t->scalar_type() != x.scalar_type() || t->sizes() != x.sizes())
          throw Refuse{"residual and residual_out must have x's shape and type"};
      }
    const int kind = integer32(a[4]);
    const int M = narrow(x.size(0)), K = narrow(x.size(1));
    Tensor sum, codes, scales;
    if (ro) sum = *ro;
    else if (r) sum = fresh(x.sizes(), x.scalar_type(), x);
    if (co) {
      dense(*co, x);
      if (co->sizes() != x.sizes() || co->element_size() != 1)
        throw Refuse{"out's codes must be one byte each, of x's shape"};
      codes = *co;
    } else {
      codes = fresh(x.sizes(), kind == W4_Q_I8 ? ScalarType::Char : ScalarType::Byte, x);
    }
    if (so) {
      dense(*so, x);
      if (so->scalar_type() != ScalarType::Float || so->numel() != M)
        throw Refuse{"out's scales must be float32 [M]"};
      scales = *so;
    } else {
      scales = fresh({M}, ScalarType::Float, x);
    }
    const OnDevice device(x);
    const int st = add_rmsnorm_q8(x.data_ptr(), ptr(r), w.data_ptr(), dt, M, K, (float)real(a[3]),
                                  kind, sum.defined() ? sum.data_ptr() : nullptr, codes.data_ptr(),
                                  (float*)scales.data_ptr(), stream_of(a[8], x));
    if (st != W4_OK) return PyLong_FromLong(st);
    PyObject* out = PyTuple_New(3);
    if (!out) return nullptr;
    auto give = [&](int i, PyObject* given, const Tensor& t) {
      if (given) Py_INCREF(given);
      PyTuple_SET_ITEM(out, i, given ? given : THPVariable_Wrap(t));
    };
    give(0, co ? a[6] : nullptr, codes);
    give(1, so ? a[7] : nullptr, scales);
    give(2, ro ? a[5] : sum.defined() ? nullptr : a[0], sum);
    return out;
  });
}

// q, k, v, k_cache, v_cache, k_scale, v_scale, page_table, kv_len, q_indptr, max_q, rope,
// style, q_out, stream -> q_out (None without q), or a status
PyObject* append(PyObject*, PyObject* const* a, Py_ssize_t n) {
  if (!count(n, 15)) return nullptr;
  return guarded([&]() -> PyObject* {
    const Tensor* q = optional(a[0], "q must be a tensor or None");
    const Tensor& k = tensor(a[1], "k must be a tensor");
    const Tensor& v = tensor(a[2], "v must be a tensor");
    const int64_t ks = token_stride(k, k), vs = token_stride(v, k);
    const int dt = in_dtype(k, "q, k and v must be float16 or float32");
    if (v.sizes() != k.sizes() || v.scalar_type() != k.scalar_type())
      throw Refuse{"k and v must have one shape and type"};
    const int T = narrow(k.size(0)), heads = narrow(k.size(1)), dim = narrow(k.size(2));
    const Cache c = cache(a + 3, heads, dim, k);
    const Batch b = batch(a[7], a[8], a[9], k);
    int q_heads = heads;
    int64_t qs = 0;
    Tensor made;
    const Tensor* qo = nullptr;
    if (q) {
      qs = token_stride(*q, k);
      if (q->size(0) != T || q->size(2) != dim || q->scalar_type() != k.scalar_type())
        throw Refuse{"q must be [tokens, q_heads, dim] of k's type"};
      q_heads = narrow(q->size(1));
      qo = optional(a[13], "q_out must be a tensor or None");
      if (qo) {
        dense(*qo, k);
        if (qo->sizes() != q->sizes() || qo->scalar_type() != ScalarType::Half)
          throw Refuse{"q_out must be a dense float16 device tensor of q's shape"};
      } else {
        made = fresh(q->sizes(), ScalarType::Half, *q);
        qo = &made;
      }
    }
    const Tensor* rope = optional(a[11], "rope must be a tensor or None");
    if (rope) {
      dense(*rope, k);
      if (rope->dim() != 2 || rope->scalar_type() != ScalarType::Float)
        throw Refuse{"rope must be float32 [positions, rot_dim]"};
    }
    const OnDevice device(k);
    const int st = rope_append_kv8(
        ptr(q), k.data_ptr(), v.data_ptr(), dt, qs, ks, vs, (const float*)ptr(rope),
        rope ? narrow(rope->size(0)) : 0, rope ? narrow(rope->size(1)) : 0, integer32(a[12]),
        (const int32_t*)ptr(b.indptr), (const int32_t*)b.len.data_ptr(),
        (const int32_t*)b.table.data_ptr(), b.batch, T, integer32(a[10]), b.cols, q_heads, heads,
        dim, c.page, c.pages, c.kind, c.k.data_ptr(), c.v.data_ptr(), (float*)c.ks.data_ptr(),
        (float*)c.vs.data_ptr(), (uint16_t*)ptr(qo), stream_of(a[14], k));
    if (st != W4_OK) return PyLong_FromLong(st);
    if (qo && !made.defined()) return Py_NewRef(a[13]);
    if (qo) return THPVariable_Wrap(made);
    Py_RETURN_NONE;
  });
}

// q, k_cache, v_cache, k_scale, v_scale, page_table, kv_len, max_kv, q_indptr, max_q, scale, lse,
// workspace, out, stream -> out, or a status
PyObject* attn(PyObject*, PyObject* const* a, Py_ssize_t n) {
  if (!count(n, 15)) return nullptr;
  return guarded([&]() -> PyObject* {
    const Tensor& q = tensor(a[0], "q must be a tensor");
    const int64_t qs = token_stride(q, q);
    if (q.scalar_type() != ScalarType::Half) throw Refuse{"q must be float16"};
    const int T = narrow(q.size(0)), heads = narrow(q.size(1)), dim = narrow(q.size(2));
    const Tensor& k = tensor(a[1], "the cache must be four tensors");
    const int kv_heads = k.dim() == 4 ? narrow(k.size(1)) : 0;
    const Cache c = cache(a + 1, kv_heads, dim, q);
    const Batch b = batch(a[5], a[6], a[8], q);
    const Tensor* lse = optional(a[11], "lse must be a tensor or None");
    if (lse) {
      dense(*lse, q);
      if (lse->scalar_type() != ScalarType::Float || lse->dim() != 2 || lse->size(0) != T ||
          lse->size(1) != heads)
        throw Refuse{"lse must be float32 [tokens, q_heads]"};
    }
    const Tensor* ws = optional(a[12], "workspace must be a tensor or None");
    if (ws) dense(*ws, q);
    const Tensor* o = optional(a[13], "out must be a tensor or None");
    Tensor made;
    if (o) {
      dense(*o, q);
      if (o->sizes() != q.sizes() || o->scalar_type() != ScalarType::Half)
        throw Refuse{"out must be a dense float16 device tensor of q's shape"};
    } else {
      made = fresh(q.sizes(), ScalarType::Half, q);
      o = &made;
    }
    const float scale = a[10] == Py_None ? (float)(1.0 / std::sqrt((double)dim)) : (float)real(a[10]);
    const OnDevice device(q);
    const int st = paged_attn_kv8(
        (const uint16_t*)q.data_ptr(), qs, c.k.data_ptr(), c.v.data_ptr(),
        (const float*)c.ks.data_ptr(), (const float*)c.vs.data_ptr(), (const int32_t*)ptr(b.indptr),
        (const int32_t*)b.len.data_ptr(), (const int32_t*)b.table.data_ptr(), b.batch, T,
        integer32(a[9]), integer32(a[7]), b.cols, heads, kv_heads, dim, c.page, c.pages, c.kind, scale,
        (uint16_t*)o->data_ptr(), (float*)ptr(lse), ptr(ws), ws ? ws->nbytes() : 0,
        stream_of(a[14], q));
    if (st != W4_OK) return PyLong_FromLong(st);
    return made.defined() ? THPVariable_Wrap(made) : Py_NewRef(a[13]);
  });
}

#include "../csrc_mx/bind_mx.hpp"

PyMethodDef methods[] = {
    {"quantize_mx4", (PyCFunction)(void (*)())mx_quantize, METH_FASTCALL, nullptr},
    {"dequantize_mx4", (PyCFunction)(void (*)())mx_dequantize, METH_FASTCALL, nullptr},
    {"mx4_gemm", (PyCFunction)(void (*)())mx_product, METH_FASTCALL, nullptr},
    {"moe_mx4", (PyCFunction)(void (*)())mx_moe, METH_FASTCALL, nullptr},
    {"add_rmsnorm_q8", (PyCFunction)(void (*)())norm, METH_FASTCALL, nullptr},
    {"rope_append_kv8", (PyCFunction)(void (*)())append, METH_FASTCALL, nullptr},
    {"paged_attn_kv8", (PyCFunction)(void (*)())attn, METH_FASTCALL, nullptr},
    {nullptr, nullptr, 0, nullptr}};

PyModuleDef module = {PyModuleDef_HEAD_INIT, "_layer_bind", nullptr, -1, methods,
                      nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__layer_bind() { return PyModule_Create(&module); }
