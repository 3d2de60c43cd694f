// Marshalling of the MXFP4 operators; included by ../csrc_layer/bind.cpp inside
// its namespace, behind the helpers that both use.

// codes uint8 [R, K/2] and scales uint8 [R, K/32] beside `first`; returns K
int mx_rows_of(const Tensor& codes, const Tensor& scales, const Tensor& first) {
  dense(codes, first), dense(scales, first);
  if (codes.dim() != 2 || scales.dim() != 2 || codes.scalar_type() != ScalarType::Byte ||
      scales.scalar_type() != ScalarType::Byte || codes.size(0) != scales.size(0) ||
      codes.size(1) != 16 * scales.size(1))
    throw Refuse{"MXFP4 rows are uint8 codes [rows, K / 2] and uint8 scales [rows, K / 32]"};
  return narrow(2 * codes.size(1));
}
PyObject* mx_pair(PyObject* ga, const Tensor& a, PyObject* gb, const Tensor& b) {
  PyObject* out = PyTuple_New(2);
  if (!out) return nullptr;
  PyTuple_SET_ITEM(out, 0, ga ? Py_NewRef(ga) : THPVariable_Wrap(a));
  PyTuple_SET_ITEM(out, 1, gb ? Py_NewRef(gb) : THPVariable_Wrap(b));
  return out;
}

// x, codes, scales, stream -> (codes, scales), or the status of a refused call
PyObject* mx_quantize(PyObject*, PyObject* const* a, Py_ssize_t n) {
  if (!count(n, 4)) return nullptr;
  return guarded([&]() -> PyObject* {
    const Tensor& x = tensor(a[0], "x must be a tensor");
    dense(x, x);
    if (x.dim() != 2) throw Refuse{"x must be [rows, K]"};
    const int dt = in_dtype(x, "x must be float16 or float32");
    const int rows = narrow(x.size(0)), K = narrow(x.size(1));
    if (K % 32) return PyLong_FromLong(W4_ERR_SHAPE);
    const Tensor* co = optional(a[1], "out must be tensors");
    const Tensor* so = optional(a[2], "out must be tensors");
    const Tensor codes = co ? *co : fresh({rows, K / 2}, ScalarType::Byte, x);
    const Tensor scales = so ? *so : fresh({rows, K / 32}, ScalarType::Byte, x);
    if (mx_rows_of(codes, scales, x) != K || codes.size(0) != rows)
      throw Refuse{"out must be codes [rows, K / 2] and scales [rows, K / 32] of x's sizes"};
    const OnDevice device(x);
    const int st = quantize_mx4(x.data_ptr(), dt, rows, K, (uint8_t*)codes.data_ptr(),
                                (uint8_t*)scales.data_ptr(), stream_of(a[3], x));
    if (st != W4_OK) return PyLong_FromLong(st);
    return mx_pair(co ? a[1] : nullptr, codes, so ? a[2] : nullptr, scales);
  });
}

// codes, scales, whether float32, out, stream -> out, or a status
PyObject* mx_dequantize(PyObject*, PyObject* const* a, Py_ssize_t n) {
  if (!count(n, 5)) return nullptr;
  return guarded([&]() -> PyObject* {
    const Tensor& c = tensor(a[0], "codes must be a tensor");
    const Tensor& s = tensor(a[1], "scales must be a tensor");
    const int K = mx_rows_of(c, s, c), rows = narrow(c.size(0));
    const bool full = integer(a[2]) != 0;
    const ScalarType dt = full ? ScalarType::Float : ScalarType::Half;
    const Tensor* o = optional(a[3], "out must be a tensor or None");
    Tensor made;
    if (o) {
      dense(*o, c);
      if (o->scalar_type() != dt || o->dim() != 2 || o->size(0) != rows || o->size(1) != K)
        throw Refuse{"out must be [rows, K] of the asked type"};
    } else {
      made = fresh({rows, K}, dt, c);
      o = &made;
    }
    const OnDevice device(c);
    const int st = dequantize_mx4((const uint8_t*)c.data_ptr(), (const uint8_t*)s.data_ptr(), rows, K,
                                  full ? W4_OUT_F32 : W4_OUT_F16, o->data_ptr(), stream_of(a[4], c));
    if (st != W4_OK) return PyLong_FromLong(st);
    return made.defined() ? THPVariable_Wrap(made) : Py_NewRef(a[3]);
  });
}

// op, A, scales of A, Wp, N, bias, out_dtype, workspace, C, stream -> C, or a status
PyObject* mx_product(PyObject*, PyObject* const* a, Py_ssize_t n) {
  if (!count(n, 10)) return nullptr;
  return guarded([&]() -> PyObject* {
    const int op = integer32(a[0]), N = integer32(a[4]), out = integer32(a[6]);
    const Tensor& A = tensor(a[1], "A must be a tensor");
    dense(A, A);
    if (A.dim() != 2) throw Refuse{"A must be [M, K], its 4-bit codes [M, K / 2]"};
    const Tensor* s = optional(a[2], "the scales of A must be a tensor");
    if (op != W4_MX_A16 && !s) throw Refuse{"the scales of A must be a tensor"};
    const int M = narrow(A.size(0));
    int K = narrow(A.size(1));
    if (op == W4_MX_A16) {
      if (A.scalar_type() != ScalarType::Half) throw Refuse{"A must be float16"};
    } else if (op == W4_MX_A8) {
      dense(*s, A);
      if (A.scalar_type() != ScalarType::Byte && A.scalar_type() != ScalarType::Float8_e4m3fn)
        throw Refuse{"A must be E4M3 codes (uint8)"};
      if (s->scalar_type() != ScalarType::Float || s->numel() != M)
        throw Refuse{"a_scale must be float32 [M]"};
    } else {
      K = mx_rows_of(A, *s, A);
    }
    const Tensor& W = tensor(a[3], "Wp must be a tensor");
    dense(W, A);
    const size_t need = prepack_mx4_bytes(N, K);
    if (need == 0) return PyLong_FromLong(W4_ERR_SHAPE);
    if (W.nbytes() < need) throw Refuse{"Wp is not prepack_mx4's of an [N, K] matrix"};
    const Tensor* bias = optional(a[5], "bias must be a tensor or None");
    if (bias) {
      dense(*bias, A);
      if (bias->scalar_type() != ScalarType::Half || bias->numel() != N)
        throw Refuse{"bias must be float16 [N]"};
    }
    if (out != W4_OUT_F16 && out != W4_OUT_F32) return PyLong_FromLong(W4_ERR_ARG);
    const ScalarType dt = out == W4_OUT_F16 ? ScalarType::Half : ScalarType::Float;
    const Tensor* ws = optional(a[7], "workspace must be a tensor or None");
    if (ws) dense(*ws, A);
    const Tensor* C = optional(a[8], "C must be a tensor or None");
    Tensor made;
    if (C) {
      dense(*C, A);
      if (C->scalar_type() != dt || C->dim() != 2 || C->size(0) != M || C->size(1) != N)
        throw Refuse{"C must be [M, N] of the asked type"};
    } else {
      made = fresh({M, N}, dt, A);
      C = &made;
    }
    const OnDevice device(A);
    const hipStream_t stream = stream_of(a[9], A);
    void* wp = ptr(ws);
    const size_t wb = ws ? ws->nbytes() : 0;
    const uint8_t* w = (const uint8_t*)W.data_ptr();
    const uint16_t* b = (const uint16_t*)ptr(bias);
    const int st =
        op == W4_MX_A16
            ? mx4a16_gemm((const uint16_t*)A.data_ptr(), w, b, C->data_ptr(), out, M, N, K, wp, wb, stream)
        : op == W4_MX_A8
            ? mx4a8_gemm((const uint8_t*)A.data_ptr(), (const float*)s->data_ptr(), w, b, C->data_ptr(),
                         out, M, N, K, wp, wb, stream)
            : mx4a4_gemm((const uint8_t*)A.data_ptr(), (const uint8_t*)s->data_ptr(), w, b,
                         C->data_ptr(), out, M, N, K, wp, wb, stream);
    if (st != W4_OK) return PyLong_FromLong(st);
    return made.defined() ? THPVariable_Wrap(made) : Py_NewRef(a[8]);
  });
}

// x, logits, top_k, w_gate_up, w_down, inner, act, renormalize, workspace, out, stream -> out, or a
// status
PyObject* mx_moe(PyObject*, PyObject* const* a, Py_ssize_t n) {
  if (!count(n, 11)) return nullptr;
  return guarded([&]() -> PyObject* {
    const Tensor& x = tensor(a[0], "x must be a tensor");
    const Tensor& l = tensor(a[1], "logits must be a tensor");
    const Tensor& w1 = tensor(a[3], "w_gate_up must be a tensor");
    const Tensor& w2 = tensor(a[4], "w_down must be a tensor");
    dense(x, x), dense(l, x), dense(w1, x), dense(w2, x);
    if (x.dim() != 2 || x.scalar_type() != ScalarType::Half) throw Refuse{"x must be float16 [tokens, hidden]"};
    if (l.dim() != 2 || l.size(0) != x.size(0)) throw Refuse{"logits must be [tokens, experts]"};
    const int dt = in_dtype(l, "logits must be float16 or float32");
    const int T = narrow(x.size(0)), H = narrow(x.size(1)), E = narrow(l.size(1)), top = integer32(a[2]),
              I = integer32(a[5]);
    if (E < 1 || E > W4_MOE_MAX_EXPERTS || I < 32 || I > W4_MAX_K || H < 32 || H > W4_MAX_K)
      return PyLong_FromLong(W4_ERR_SHAPE);
    const size_t n1 = prepack_mx4_bytes(2 * E * I, H), n2 = prepack_mx4_bytes(E * H, I);
    if (n1 == 0 || n2 == 0) return PyLong_FromLong(W4_ERR_SHAPE);
    if (w1.nbytes() < n1 || w2.nbytes() < n2)
      throw Refuse{"weights are not prepack_mx4's of [experts * 2 * inner, hidden] and [experts * hidden, inner]"};
    const Tensor* ws = optional(a[8], "workspace must be a tensor or None");
    if (ws) dense(*ws, x);
    const Tensor* o = optional(a[9], "out must be a tensor or None");
    Tensor made;
    if (o) {
      dense(*o, x);
      if (o->sizes() != x.sizes() || o->scalar_type() != ScalarType::Half)
        throw Refuse{"out must be a dense float16 device tensor of x's shape"};
    } else {
      made = fresh(x.sizes(), ScalarType::Half, x);
      o = &made;
    }
    const OnDevice device(x);
    const int st = moe_mx4((const uint16_t*)x.data_ptr(), l.data_ptr(), dt, T, H, I, E, top,
                           integer32(a[7]), integer32(a[6]), (const uint8_t*)w1.data_ptr(),
                           (const uint8_t*)w2.data_ptr(), (uint16_t*)o->data_ptr(), ptr(ws),
                           ws ? ws->nbytes() : 0, stream_of(a[10], x));
    if (st != W4_OK) return PyLong_FromLong(st);
    return made.defined() ? THPVariable_Wrap(made) : Py_NewRef(a[9]);
  });
}
