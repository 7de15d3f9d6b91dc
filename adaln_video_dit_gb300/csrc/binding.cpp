// Argument marshalling of every call but the AdaLN's, as a CPython
// extension (_binding): the checks, output allocation and struct building that
// _lib.py's functions of the same names need.
//
// A small call's cost is its host code: one token through the norm and rotation
// keeps the GPU busy for 2.6 us, while the same marshalling in Python with ctypes
// took 20 us of host time.  Tensors are read through their Python
// attributes, so this holds no torch header and fits any torch of the
// interpreter's.  The library's entry points are passed in by address (setup).
//
// Every function returns NULL with a Python exception set on a refusal: TypeError
// for a dtype, ValueError for a shape, layout or device, AdalnError for what the
// library refuses.
#define PY_SSIZE_T_CLEAN
#include <Python.h>

#include "../../include/adaln.h"

namespace {

// An owned reference.
struct Ref {
  PyObject* p;
  explicit Ref(PyObject* o = nullptr) : p(o) {}
  ~Ref() { Py_XDECREF(p); }
  Ref(const Ref&) = delete;
  Ref& operator=(const Ref&) = delete;
  void set(PyObject* o) {
    Py_XDECREF(p);
    p = o;
  }
  PyObject* take() {
    PyObject* o = p;
    p = nullptr;
    return o;
  }
  explicit operator bool() const { return p != nullptr; }
};

// ----- what setup() fills --------------------------------------------------------

PyObject *g_empty, *g_empty_like, *g_raw_stream, *g_error;  // callables
PyObject *g_bf16, *g_f32, *g_i32, *g_i64, *g_u8;            // dtypes (singletons)
PyObject *n_get_device, *n_shape, *n_dtype, *n_data_ptr, *n_stride, *n_is_contiguous, *n_device,
    *n_numel, *n_cuda_stream;
PyObject* g_kw_dtype_device;

decltype(&adaln_qk_rope_fwd) f_qk_fwd;
decltype(&adaln_qk_rope_bwd) f_qk_bwd;
decltype(&adaln_qk_rope_bwd_workspace_size) f_qk_ws;
decltype(&adaln_ffn_fwd) f_ffn_fwd;
decltype(&adaln_ffn_bwd) f_ffn_bwd;
decltype(&adaln_ffn_saved_size) f_ffn_saved;
decltype(&adaln_ffn_workspace_size) f_ffn_ws;
decltype(&adaln_dropout_fwd) f_drop_fwd;
decltype(&adaln_dropout_bwd) f_drop_bwd;
decltype(&adaln_dropout_bwd_workspace_size) f_drop_ws;
decltype(&adaln_route_rows) f_route_rows;
decltype(&adaln_route_workspace_size) f_route_ws;
decltype(&adaln_route) f_route;
decltype(&adaln_expert_sort_fwd) f_sort_fwd;
decltype(&adaln_expert_sort_bwd) f_sort_bwd;
decltype(&adaln_expert_combine_fwd) f_combine_fwd;
decltype(&adaln_expert_combine_bwd) f_combine_bwd;
decltype(&adaln_experts_ffn_saved_size) f_experts_saved;
decltype(&adaln_experts_ffn_workspace_size) f_experts_ws;
decltype(&adaln_experts_ffn_fwd) f_experts_fwd;
decltype(&adaln_experts_ffn_bwd) f_experts_bwd;

// ----- reading tensors --------------------------------------------------------------

struct Tensor {
  void* ptr = nullptr;
  int64_t shape[3] = {}, stride[3] = {};
  int ndim = 0;
  long dev = -1;
  PyObject* dtype = nullptr;  // a singleton, borrowed
};

PyObject* call0(PyObject* o, PyObject* name) { return PyObject_CallMethodNoArgs(o, name); }

bool as_int(PyObject* o, int64_t* out) {  // steals o
  Ref r(o);
  if (!r) return false;
  *out = PyLong_AsLongLong(o);
  return !(*out == -1 && PyErr_Occurred());
}

bool tuple_of(PyObject* t, int64_t (&out)[3]) {
  for (Py_ssize_t i = 0; i < PyTuple_GET_SIZE(t); ++i) {
    out[i] = PyLong_AsLongLong(PyTuple_GET_ITEM(t, i));
    if (out[i] == -1 && PyErr_Occurred()) return false;
  }
  return true;
}

// Device, shape (at most 3 dimensions), dtype and pointer; strides if asked.
bool read(PyObject* t, const char* name, Tensor* x, bool strides) {
  int64_t v;
  if (!as_int(call0(t, n_get_device), &v)) return false;
  x->dev = (long)v;
  if (x->dev < 0) {
    PyErr_Format(PyExc_ValueError, "%s must be a CUDA tensor", name);
    return false;
  }
  Ref shape(PyObject_GetAttr(t, n_shape));
  if (!shape) return false;
  if (!PyTuple_Check(shape.p) || PyTuple_GET_SIZE(shape.p) > 3) {
    PyErr_Format(PyExc_ValueError, "%s has too many dimensions", name);
    return false;
  }
  x->ndim = (int)PyTuple_GET_SIZE(shape.p);
  if (!tuple_of(shape.p, x->shape)) return false;
  Ref dtype(PyObject_GetAttr(t, n_dtype));
  if (!dtype) return false;
  x->dtype = dtype.p;
  if (strides) {
    Ref st(call0(t, n_stride));
    if (!st) return false;
    if (!PyTuple_Check(st.p) || PyTuple_GET_SIZE(st.p) != x->ndim || !tuple_of(st.p, x->stride)) {
      if (!PyErr_Occurred()) PyErr_Format(PyExc_ValueError, "%s has no strides", name);
      return false;
    }
  }
  if (!as_int(call0(t, n_data_ptr), &v)) return false;
  x->ptr = (void*)(intptr_t)v;
  return true;
}

bool contiguous(PyObject* t, const char* name) {
  Ref c(call0(t, n_is_contiguous));
  if (!c) return false;
  if (c.p == Py_True) return true;
  PyErr_Format(PyExc_ValueError, "%s must be contiguous", name);
  return false;
}

bool on_device(const Tensor& x, const char* name, long dev) {
  if (x.dev == dev) return true;
  PyErr_Format(PyExc_ValueError, "%s must be on cuda:%ld, not cuda:%ld", name, dev, x.dev);
  return false;
}

bool of_dtype(const Tensor& x, const char* name, PyObject* dtype) {
  if (x.dtype == dtype) return true;
  PyErr_Format(PyExc_TypeError, "%s must be %R, got %R", name, dtype, x.dtype);
  return false;
}

bool of_shape(const Tensor& x, const char* name, int ndim, int64_t a, int64_t b = 0, int64_t c = 0) {
  const int64_t want[3] = {a, b, c};
  bool same = x.ndim == ndim;
  for (int i = 0; i < ndim && same; ++i) same = x.shape[i] == want[i];
  if (same) return true;
  if (ndim == 1)
    PyErr_Format(PyExc_ValueError, "%s must have shape (%lld,)", name, (long long)a);
  else if (ndim == 2)
    PyErr_Format(PyExc_ValueError, "%s must have shape (%lld, %lld)", name, (long long)a, (long long)b);
  else
    PyErr_Format(PyExc_ValueError, "%s must have shape (%lld, %lld, %lld)", name, (long long)a,
                 (long long)b, (long long)c);
  return false;
}

int dtype_code(PyObject* dtype) {
  if (dtype == g_bf16) return ADALN_BF16;
  if (dtype == g_f32) return ADALN_F32;
  PyErr_Format(PyExc_TypeError, "libadaln supports bfloat16 and float32, not %R", dtype);
  return -1;
}

PyObject* new_tensor(PyObject* shape, PyObject* dtype, PyObject* device) {
  PyObject* args[3] = {shape, dtype, device};
  return PyObject_Vectorcall(g_empty, args, 1, g_kw_dtype_device);
}
PyObject* new_bytes(size_t n, PyObject* device) {
  Ref size(PyLong_FromSize_t(n < 16 ? 16 : n));
  return size ? new_tensor(size.p, g_u8, device) : nullptr;
}

// The pointer of a new tensor.
bool pointer(PyObject* t, void** out) {
  int64_t v;
  if (!as_int(call0(t, n_data_ptr), &v)) return false;
  *out = (void*)(intptr_t)v;
  return true;
}

// A given uint8 buffer's pointer and size.
bool buffer(PyObject* t, const char* name, long dev, void** p, size_t* n) {
  Tensor x;
  int64_t v;
  if (!read(t, name, &x, false) || !on_device(x, name, dev) || !of_dtype(x, name, g_u8) ||
      !contiguous(t, name) || !as_int(call0(t, n_numel), &v))
    return false;
  *p = x.ptr;
  *n = (size_t)v;
  return true;
}

bool stream_of(PyObject* stream, long dev, void** out) {
  int64_t v;
  if (stream == Py_None) {
    Ref index(PyLong_FromLong(dev));
    if (!index || !as_int(PyObject_CallOneArg(g_raw_stream, index.p), &v)) return false;
  } else if (!as_int(PyObject_GetAttr(stream, n_cuda_stream), &v)) {
    return false;
  }
  *out = (void*)(intptr_t)v;
  return true;
}

PyObject* refused(int rc, const char* what) {
  Ref e(PyObject_CallFunction(g_error, "is", rc, what));
  if (e) PyErr_SetObject(g_error, e.p);
  return nullptr;
}

bool none(PyObject* o) { return o == Py_None; }

// ----- rotary positions and norm --------------------------------------------------------

// A [T, heads, dh] tensor (any strides, dh contiguous), `like` another's shape,
// dtype and device where given.
bool heads_of(PyObject* t, const char* name, const Tensor* like, Tensor* x, adaln_heads_t* h) {
  if (!read(t, name, x, true)) return false;
  if (x->ndim != 3) {
    PyErr_Format(PyExc_ValueError, "%s must be [T, heads, dh]", name);
    return false;
  }
  if (like && (!of_shape(*x, name, 3, like->shape[0], like->shape[1], like->shape[2]) ||
               !of_dtype(*x, name, like->dtype) || !on_device(*x, name, like->dev)))
    return false;
  if (x->stride[2] != 1 && x->shape[2] != 1) {
    PyErr_Format(PyExc_ValueError, "%s: the elements of a head must be contiguous", name);
    return false;
  }
  *h = adaln_heads_t{x->ptr, x->stride[0], x->stride[1]};
  return true;
}

// The keys beside the queries: the same tokens, head width, dtype and device.
bool beside(PyObject* t, const char* name, const Tensor& q, Tensor* x, adaln_heads_t* h) {
  if (!heads_of(t, name, nullptr, x, h)) return false;
  if (x->shape[0] != q.shape[0] || x->shape[2] != q.shape[2]) {
    PyErr_SetString(PyExc_ValueError, "queries and keys must agree in tokens and head width");
    return false;
  }
  return of_dtype(*x, name, q.dtype) && on_device(*x, name, q.dev);
}

// An output like `like` (whose tensor is `src`): checked, or allocated.
bool heads_out(PyObject* given, const char* name, const Tensor& like, PyObject* src, PyObject* device,
               Ref* out, adaln_heads_t* h) {
  if (!none(given)) {
    Tensor x;
    if (!heads_of(given, name, &like, &x, h)) return false;
    Py_INCREF(given);
    out->set(given);
    return true;
  }
  Ref shape(PyObject_GetAttr(src, n_shape));
  if (!shape) return false;
  out->set(new_tensor(shape.p, like.dtype, device));
  if (!*out || !pointer(out->p, &h->ptr)) return false;
  h->token_stride = like.shape[1] * like.shape[2];
  h->head_stride = like.shape[2];
  return true;
}

bool rope_of(PyObject* table, PyObject* pos, PyObject* pairs, int interleaved, const Tensor& q,
             adaln_rope_t* r) {
  Tensor t, p;
  if (!read(table, "table", &t, false) || !read(pos, "pos", &p, false) ||
      !on_device(t, "table", q.dev) || !on_device(p, "pos", q.dev))
    return false;
  if (t.dtype != g_f32 || p.dtype != g_i32) {
    PyErr_SetString(PyExc_ValueError, "table must be float32 and pos int32");
    return false;
  }
  if (!contiguous(table, "table") || !contiguous(pos, "pos")) return false;
  Ref seq(PySequence_Fast(pairs, "axis_pairs must be a sequence"));
  if (!seq) return false;
  const Py_ssize_t axes = PySequence_Fast_GET_SIZE(seq.p);
  if (axes < 1 || axes > ADALN_MAX_ROPE_AXES) {
    PyErr_Format(PyExc_ValueError, "axis_pairs must hold 1 to %d counts >= 0", ADALN_MAX_ROPE_AXES);
    return false;
  }
  *r = adaln_rope_t{};
  int64_t P = 0;
  for (Py_ssize_t i = 0; i < axes; ++i) {
    const long n = PyLong_AsLong(PySequence_Fast_GET_ITEM(seq.p, i));
    if (n == -1 && PyErr_Occurred()) return false;
    if (n < 0 || n > ADALN_MAX_HEAD_DIM) {
      PyErr_Format(PyExc_ValueError, "axis_pairs must hold 1 to %d counts >= 0", ADALN_MAX_ROPE_AXES);
      return false;
    }
    r->pairs[i] = (int32_t)n;
    P += n;
  }
  if (t.ndim != 3 || t.shape[1] != P || t.shape[2] != 2 || t.shape[0] > INT32_MAX) {
    PyErr_Format(PyExc_ValueError, "table must have shape [rows, %lld, 2]", (long long)P);
    return false;
  }
  if (!of_shape(p, "pos", 2, q.shape[0], axes)) return false;
  r->table = static_cast<const float*>(t.ptr);
  r->pos = static_cast<const int32_t*>(p.ptr);
  r->rows = (int32_t)t.shape[0];
  r->axes = (int32_t)axes;
  r->interleaved = interleaved;
  return true;
}

bool weight_of(PyObject* w, const char* name, const Tensor& q, const void** out) {
  *out = nullptr;
  if (none(w)) return true;
  Tensor x;
  if (!read(w, name, &x, false) || !on_device(x, name, q.dev) || !contiguous(w, name) ||
      !of_dtype(x, name, q.dtype) || !of_shape(x, name, 1, q.shape[2]))
    return false;
  *out = x.ptr;
  return true;
}

// An fp32 [dh] gradient: checked, or allocated.
bool gradient(PyObject* given, const char* name, const Tensor& q, PyObject* device, Ref* out,
              float** p) {
  void* v = nullptr;
  if (none(given)) {
    Ref n(PyLong_FromLongLong(q.shape[2]));
    if (!n) return false;
    out->set(new_tensor(n.p, g_f32, device));
    if (!*out || !pointer(out->p, &v)) return false;
  } else {
    Tensor x;
    if (!read(given, name, &x, false) || !on_device(x, name, q.dev) || !contiguous(given, name) ||
        !of_dtype(x, name, g_f32) || !of_shape(x, name, 1, q.shape[2]))
      return false;
    Py_INCREF(given);
    out->set(given);
    v = x.ptr;
  }
  *p = static_cast<float*>(v);
  return true;
}

bool sizes_fit(const Tensor& q, const Tensor& k) {
  if (q.shape[1] <= INT32_MAX && q.shape[2] <= INT32_MAX && k.shape[1] <= INT32_MAX) return true;
  PyErr_SetString(PyExc_ValueError, "too many heads, or too wide");
  return false;
}

bool flag(PyObject* o, int* out) { return (*out = PyObject_IsTrue(o)) >= 0; }
bool number(PyObject* o, float* out) {
  const double v = PyFloat_AsDouble(o);
  *out = (float)v;
  return !(v == -1.0 && PyErr_Occurred());
}

PyObject* pair_or(Ref& a, Ref& b) {  // (a, b), None for a missing one
  return PyTuple_Pack(2, a ? a.p : Py_None, b ? b.p : Py_None);
}

// qk_rope_fwd(q, k, table, pos, axis_pairs, interleaved, norm, wq, wk, eps, q_out,
//             k_out, stream) -> (q_out, k_out)
PyObject* qk_rope_fwd(PyObject*, PyObject* const* a, Py_ssize_t n) {
  if (n != 13) {
    PyErr_SetString(PyExc_TypeError, "13 arguments");
    return nullptr;
  }
  Tensor q, k;
  adaln_heads_t qh, kh, qo, ko;
  adaln_rope_t rope;
  int interleaved, norm;
  const void *wq, *wk;
  float eps;
  void* stream;
  const bool keys = !none(a[1]);
  if (!heads_of(a[0], "q", nullptr, &q, &qh) || (keys && !beside(a[1], "k", q, &k, &kh)) ||
      !sizes_fit(q, k) || !flag(a[5], &interleaved) || !flag(a[6], &norm) ||
      !rope_of(a[2], a[3], a[4], interleaved, q, &rope) || !weight_of(a[7], "wq", q, &wq) ||
      !weight_of(a[8], "wk", q, &wk) || !number(a[9], &eps))
    return nullptr;
  const int code = dtype_code(q.dtype);
  if (code < 0) return nullptr;
  Ref device(PyObject_GetAttr(a[0], n_device)), out_q, out_k;
  if (!device || !heads_out(a[10], "q_out", q, a[0], device.p, &out_q, &qo) ||
      (keys && !heads_out(a[11], "k_out", k, a[1], device.p, &out_k, &ko)) ||
      !stream_of(a[12], q.dev, &stream))
    return nullptr;
  int rc;
  Py_BEGIN_ALLOW_THREADS;
  rc = f_qk_fwd(&qh, keys ? &kh : nullptr, q.shape[0], (int32_t)q.shape[1],
                keys ? (int32_t)k.shape[1] : 0, (int32_t)q.shape[2], (adaln_dtype_t)code, &rope, norm,
                wq, wk, eps, &qo, keys ? &ko : nullptr, stream);
  Py_END_ALLOW_THREADS;
  if (rc != ADALN_OK) return refused(rc, "adaln_qk_rope_fwd");
  return pair_or(out_q, out_k);
}

// qk_rope_bwd(dq_out, dk_out, table, pos, axis_pairs, interleaved, norm, q, k, wq,
//             wk, eps, dq, dk, dwq, dwk, workspace, stream) -> (dq, dk, dwq, dwk)
PyObject* qk_rope_bwd(PyObject*, PyObject* const* a, Py_ssize_t n) {
  if (n != 18) {
    PyErr_SetString(PyExc_TypeError, "18 arguments");
    return nullptr;
  }
  Tensor dqo, dko, q, k;
  adaln_heads_t dqoh, dkoh, qh, kh, dqh, dkh;
  adaln_rope_t rope;
  int interleaved, norm;
  const void *wq, *wk;
  float eps, *dwq = nullptr, *dwk = nullptr;
  void *stream, *ws = nullptr;
  size_t bytes = 0;
  const bool keys = !none(a[1]);
  if (!heads_of(a[0], "dq_out", nullptr, &dqo, &dqoh) ||
      (keys && !beside(a[1], "dk_out", dqo, &dko, &dkoh)) || !sizes_fit(dqo, dko) ||
      !flag(a[5], &interleaved) || !flag(a[6], &norm) ||
      !rope_of(a[2], a[3], a[4], interleaved, dqo, &rope) || !weight_of(a[9], "wq", dqo, &wq) ||
      !weight_of(a[10], "wk", dqo, &wk) || !number(a[11], &eps))
    return nullptr;
  const int code = dtype_code(dqo.dtype);
  if (code < 0) return nullptr;
  const int32_t hq = (int32_t)dqo.shape[1], hk = keys ? (int32_t)dko.shape[1] : 0;
  const int32_t dh = (int32_t)dqo.shape[2];
  Ref device(PyObject_GetAttr(a[0], n_device)), out_q, out_k, out_wq, out_wk, work;
  if (!device) return nullptr;
  if (norm) {
    if (none(a[7]) || none(a[8]) == keys) {
      PyErr_SetString(PyExc_ValueError, "the norm's backward needs the forward's q (and k)");
      return nullptr;
    }
    if (!heads_of(a[7], "q", &dqo, &q, &qh) || (keys && !heads_of(a[8], "k", &dko, &k, &kh)) ||
        !gradient(a[14], "dwq", dqo, device.p, &out_wq, &dwq) ||
        (keys && !gradient(a[15], "dwk", dqo, device.p, &out_wk, &dwk)))
      return nullptr;
    if (none(a[16])) {
      const int rc = f_qk_ws(dqo.shape[0], hq, hk, dh, (adaln_dtype_t)code, &bytes);
      if (rc != ADALN_OK) return refused(rc, "adaln_qk_rope_bwd_workspace_size");
      if (bytes < 16) bytes = 16;
      work.set(new_bytes(bytes, device.p));
      if (!work || !pointer(work.p, &ws)) return nullptr;
    } else if (!buffer(a[16], "workspace", dqo.dev, &ws, &bytes)) {
      return nullptr;
    }
  }
  if (!heads_out(a[12], "dq", dqo, a[0], device.p, &out_q, &dqh) ||
      (keys && !heads_out(a[13], "dk", dko, a[1], device.p, &out_k, &dkh)) ||
      !stream_of(a[17], dqo.dev, &stream))
    return nullptr;
  int rc;
  Py_BEGIN_ALLOW_THREADS;
  rc = f_qk_bwd(&dqoh, keys ? &dkoh : nullptr, norm ? &qh : nullptr, norm && keys ? &kh : nullptr,
                dqo.shape[0], hq, hk, dh, (adaln_dtype_t)code, &rope, norm, wq, wk, eps, &dqh,
                keys ? &dkh : nullptr, dwq, dwk, ws, bytes, stream);
  Py_END_ALLOW_THREADS;
  if (rc != ADALN_OK) return refused(rc, "adaln_qk_rope_bwd");
  return PyTuple_Pack(4, out_q.p, out_k ? out_k.p : Py_None, out_wq ? out_wq.p : Py_None,
                      out_wk ? out_wk.p : Py_None);
}

// ----- gated feed-forward block -----------------------------------------------------------

bool matrix(PyObject* t, const char* name, int64_t rows, int64_t cols, PyObject* dtype, long dev,
            void** out) {
  Tensor x;
  if (!read(t, name, &x, false) || !on_device(x, name, dev) || !contiguous(t, name) ||
      !of_dtype(x, name, dtype) || !of_shape(x, name, 2, rows, cols))
    return false;
  *out = x.ptr;
  return true;
}

bool matrix_out(PyObject* given, const char* name, PyObject* like, int64_t rows, int64_t cols,
                PyObject* dtype, long dev, Ref* out, void** p) {
  if (none(given)) {
    out->set(PyObject_CallOneArg(g_empty_like, like));
    return *out && pointer(out->p, p);
  }
  if (!matrix(given, name, rows, cols, dtype, dev, p)) return false;
  Py_INCREF(given);
  out->set(given);
  return true;
}

struct Ffn {
  int64_t T, D, F;
  long dev;
  PyObject* dtype;
  int code;
  void *x, *wg, *wu, *wd;
};

bool ffn_args(PyObject* x, PyObject* wg, PyObject* wu, PyObject* wd, Ffn* f) {
  Tensor t, g;
  if (!read(x, "x", &t, false) || !contiguous(x, "x") || !read(wg, "wg", &g, false)) return false;
  if (t.ndim != 2 || g.ndim != 2) {
    PyErr_SetString(PyExc_ValueError, "x must be [T, D] and wg [F, D]");
    return false;
  }
  f->T = t.shape[0], f->D = t.shape[1], f->F = g.shape[0];
  f->dev = t.dev, f->dtype = t.dtype, f->x = t.ptr;
  if (!matrix(wg, "wg", f->F, f->D, t.dtype, t.dev, &f->wg) ||
      !matrix(wu, "wu", f->F, f->D, t.dtype, t.dev, &f->wu) ||
      !matrix(wd, "wd", f->D, f->F, t.dtype, t.dev, &f->wd))
    return false;
  f->code = dtype_code(t.dtype);
  if (f->code < 0) return false;
  if (f->D > INT32_MAX || f->F > INT32_MAX) {
    PyErr_SetString(PyExc_ValueError, "D or F too large");
    return false;
  }
  return true;
}

bool ffn_workspace(PyObject* given, const Ffn& f, bool backward, PyObject* device, Ref* work,
                   void** p, size_t* bytes) {
  if (!none(given)) return buffer(given, "workspace", f.dev, p, bytes);
  const int rc = f_ffn_ws(f.T, (int32_t)f.D, (int32_t)f.F, (adaln_dtype_t)f.code,
                          backward ? nullptr : bytes, backward ? bytes : nullptr);
  if (rc != ADALN_OK) {
    refused(rc, "adaln_ffn_workspace_size");
    return false;
  }
  if (*bytes < 16) *bytes = 16;
  work->set(new_bytes(*bytes, device));
  return *work && pointer(work->p, p);
}

// The saved buffer's least size; a given one is checked against it.
bool ffn_saved(PyObject* given, const Ffn& f, size_t* need, void** p) {
  const int rc = f_ffn_saved(f.T, (int32_t)f.D, (int32_t)f.F, (adaln_dtype_t)f.code, need);
  if (rc != ADALN_OK) {
    refused(rc, "adaln_ffn_saved_size");
    return false;
  }
  if (none(given)) return true;
  size_t have = 0;
  if (!buffer(given, "saved", f.dev, p, &have)) return false;
  if (have >= *need) return true;
  PyErr_Format(PyExc_ValueError, "saved holds %zu bytes, %zu are needed", have, *need);
  return false;
}

// ffn_fwd(x, wg, wu, wd, act, save, y, saved, workspace, stream) -> (y, saved)
PyObject* ffn_fwd(PyObject*, PyObject* const* a, Py_ssize_t n) {
  if (n != 10) {
    PyErr_SetString(PyExc_TypeError, "10 arguments");
    return nullptr;
  }
  Ffn f;
  int save;
  if (!ffn_args(a[0], a[1], a[2], a[3], &f) || !flag(a[5], &save)) return nullptr;
  const long act = PyLong_AsLong(a[4]);
  if (act == -1 && PyErr_Occurred()) return nullptr;
  Ref device(PyObject_GetAttr(a[0], n_device)), y, saved, work;
  void *yp, *sp = nullptr, *ws, *stream;
  size_t need = 0, bytes = 0;
  if (!device || !matrix_out(a[6], "y", a[0], f.T, f.D, f.dtype, f.dev, &y, &yp)) return nullptr;
  if (save || !none(a[7])) {
    if (!ffn_saved(a[7], f, &need, &sp)) return nullptr;
    if (none(a[7])) {
      saved.set(new_bytes(need, device.p));
      if (!saved || !pointer(saved.p, &sp)) return nullptr;
    } else {
      Py_INCREF(a[7]);
      saved.set(a[7]);
    }
  }
  if (!ffn_workspace(a[8], f, false, device.p, &work, &ws, &bytes) || !stream_of(a[9], f.dev, &stream))
    return nullptr;
  int rc;
  Py_BEGIN_ALLOW_THREADS;
  rc = f_ffn_fwd(f.x, f.wg, f.wu, f.wd, f.T, (int32_t)f.D, (int32_t)f.F, (adaln_dtype_t)f.code,
                 (adaln_act_t)act, yp, sp, ws, bytes, stream);
  Py_END_ALLOW_THREADS;
  if (rc != ADALN_OK) return refused(rc, "adaln_ffn_fwd");
  return pair_or(y, saved);
}

// ffn_bwd(dy, x, wg, wu, wd, saved, act, dx, dwg, dwu, dwd, workspace, stream)
//   -> (dx, dwg, dwu, dwd)
PyObject* ffn_bwd(PyObject*, PyObject* const* a, Py_ssize_t n) {
  if (n != 13) {
    PyErr_SetString(PyExc_TypeError, "13 arguments");
    return nullptr;
  }
  Ffn f;
  void *dy, *sp = nullptr, *dxp, *dgp, *dup, *ddp, *ws, *stream;
  size_t need = 0, bytes = 0;
  if (!ffn_args(a[1], a[2], a[3], a[4], &f) ||
      !matrix(a[0], "dy", f.T, f.D, f.dtype, f.dev, &dy))
    return nullptr;
  if (none(a[5])) {
    PyErr_SetString(PyExc_ValueError, "the backward needs what the forward saved");
    return nullptr;
  }
  const long act = PyLong_AsLong(a[6]);
  if (act == -1 && PyErr_Occurred()) return nullptr;
  Ref device(PyObject_GetAttr(a[1], n_device)), dx, dwg, dwu, dwd, work;
  if (!device || !ffn_saved(a[5], f, &need, &sp) ||
      !matrix_out(a[7], "dx", a[1], f.T, f.D, f.dtype, f.dev, &dx, &dxp) ||
      !matrix_out(a[8], "dwg", a[2], f.F, f.D, f.dtype, f.dev, &dwg, &dgp) ||
      !matrix_out(a[9], "dwu", a[3], f.F, f.D, f.dtype, f.dev, &dwu, &dup) ||
      !matrix_out(a[10], "dwd", a[4], f.D, f.F, f.dtype, f.dev, &dwd, &ddp) ||
      !ffn_workspace(a[11], f, true, device.p, &work, &ws, &bytes) ||
      !stream_of(a[12], f.dev, &stream))
    return nullptr;
  int rc;
  Py_BEGIN_ALLOW_THREADS;
  rc = f_ffn_bwd(dy, f.x, f.wg, f.wu, f.wd, sp, f.T, (int32_t)f.D, (int32_t)f.F,
                 (adaln_dtype_t)f.code, (adaln_act_t)act, dxp, dgp, dup, ddp, ws, bytes, stream);
  Py_END_ALLOW_THREADS;
  if (rc != ADALN_OK) return refused(rc, "adaln_ffn_bwd");
  return PyTuple_Pack(4, dx.p, dwg.p, dwu.p, dwd.p);
}

// ----- dropout, gate and residual ------------------------------------------------------------

// Where the mask comes from: None, (seed, offset), or an int64 [2] tensor of them.
bool rng_of(PyObject* o, long dev, adaln_rng_t* r, bool* given) {
  *r = adaln_rng_t{};
  *given = !none(o);
  if (!*given) return true;
  if (PyTuple_Check(o)) {
    if (PyTuple_GET_SIZE(o) != 2) {
      PyErr_SetString(PyExc_ValueError, "rng must be (seed, offset) or an int64 tensor of the two");
      return false;
    }
    uint64_t* to[2] = {&r->seed, &r->offset};
    for (int i = 0; i < 2; ++i) {  // any 64-bit integer, signed or not
      *to[i] = PyLong_AsUnsignedLongLongMask(PyTuple_GET_ITEM(o, i));
      if (*to[i] == (uint64_t)-1 && PyErr_Occurred()) return false;
    }
    return true;
  }
  Tensor x;
  if (!read(o, "rng", &x, false) || !on_device(x, "rng", dev) || !of_dtype(x, "rng", g_i64) ||
      !of_shape(x, "rng", 1, 2) || !contiguous(o, "rng"))
    return false;
  r->state = static_cast<const int64_t*>(x.ptr);
  return true;
}

struct Drop {
  int64_t T, D, nseg = 1;
  long dev;
  PyObject* dtype;
  int code;
  double p;
  adaln_rng_t rng;
  bool drawn;
  void *h, *gate = nullptr;
  const int32_t* seg = nullptr;
};

// h (or dy), p, rng, gate and seg_id.
bool drop_args(PyObject* h, const char* name, PyObject* p, PyObject* rng, PyObject* gate, PyObject* seg,
               Drop* d) {
  Tensor t;
  if (!read(h, name, &t, false) || !contiguous(h, name)) return false;
  if (t.ndim != 2 || t.shape[1] > INT32_MAX) {
    PyErr_Format(PyExc_ValueError, "%s must be [T, D]", name);
    return false;
  }
  d->T = t.shape[0], d->D = t.shape[1], d->dev = t.dev, d->dtype = t.dtype, d->h = t.ptr;
  if ((d->code = dtype_code(t.dtype)) < 0) return false;
  d->p = PyFloat_AsDouble(p);
  if (d->p == -1.0 && PyErr_Occurred()) return false;
  if (!rng_of(rng, t.dev, &d->rng, &d->drawn)) return false;
  if (none(gate) != none(seg)) {
    PyErr_SetString(PyExc_ValueError, "a gate and seg_id belong together");
    return false;
  }
  if (none(gate)) return true;
  Tensor g, s;
  if (!read(gate, "gate", &g, false) || !on_device(g, "gate", d->dev) || !contiguous(gate, "gate") ||
      !of_dtype(g, "gate", d->dtype) || !read(seg, "seg_id", &s, false) ||
      !on_device(s, "seg_id", d->dev) || !contiguous(seg, "seg_id") || !of_dtype(s, "seg_id", g_i32) ||
      !of_shape(s, "seg_id", 1, d->T))
    return false;
  if (g.ndim != 2 || g.shape[1] != d->D || g.shape[0] > INT32_MAX) {
    PyErr_Format(PyExc_ValueError, "gate must have shape [nseg, %lld]", (long long)d->D);
    return false;
  }
  d->nseg = g.shape[0], d->gate = g.ptr, d->seg = static_cast<const int32_t*>(s.ptr);
  return true;
}

// dropout_fwd(h, p, rng, x, gate, seg_id, y, stream) -> y
PyObject* dropout_fwd(PyObject*, PyObject* const* a, Py_ssize_t n) {
  if (n != 8) {
    PyErr_SetString(PyExc_TypeError, "8 arguments");
    return nullptr;
  }
  Drop d;
  Ref y;
  void *x = nullptr, *yp, *stream;
  if (!drop_args(a[0], "h", a[1], a[2], a[4], a[5], &d) ||
      (!none(a[3]) && !matrix(a[3], "x", d.T, d.D, d.dtype, d.dev, &x)) ||
      !matrix_out(a[6], "y", a[0], d.T, d.D, d.dtype, d.dev, &y, &yp) || !stream_of(a[7], d.dev, &stream))
    return nullptr;
  int rc;
  Py_BEGIN_ALLOW_THREADS;
  rc = f_drop_fwd(d.h, x, d.gate, d.seg, d.T, (int32_t)d.D, (int32_t)d.nseg, (adaln_dtype_t)d.code, d.p,
                  d.drawn ? &d.rng : nullptr, yp, stream);
  Py_END_ALLOW_THREADS;
  if (rc != ADALN_OK) return refused(rc, "adaln_dropout_fwd");
  return y.take();
}

// dropout_bwd(dy, p, rng, h, gate, seg_id, dh, dgate, workspace, stream) -> (dh, dgate)
PyObject* dropout_bwd(PyObject*, PyObject* const* a, Py_ssize_t n) {
  if (n != 10) {
    PyErr_SetString(PyExc_TypeError, "10 arguments");
    return nullptr;
  }
  Drop d;
  Ref dh, dgate, work, device(PyObject_GetAttr(a[0], n_device));
  void *h = nullptr, *dhp, *sum = nullptr, *ws = nullptr, *stream;
  size_t bytes = 0;
  if (!device || !drop_args(a[0], "dy", a[1], a[2], a[4], a[5], &d) ||
      (!none(a[3]) && !matrix(a[3], "h", d.T, d.D, d.dtype, d.dev, &h)) ||
      !matrix_out(a[6], "dh", a[0], d.T, d.D, d.dtype, d.dev, &dh, &dhp))
    return nullptr;
  if (!none(a[3]) && none(a[4])) {
    PyErr_SetString(PyExc_ValueError, "h is for the gradient of a gate, and there is none");
    return nullptr;
  }
  if (!none(a[3])) {
    if (none(a[7])) {
      Ref shape(Py_BuildValue("LL", (long long)d.nseg, (long long)d.D));
      if (!shape) return nullptr;
      dgate.set(new_tensor(shape.p, g_f32, device.p));
      if (!dgate || !pointer(dgate.p, &sum)) return nullptr;
    } else {
      if (!matrix(a[7], "dgate", d.nseg, d.D, g_f32, d.dev, &sum)) return nullptr;
      Py_INCREF(a[7]);
      dgate.set(a[7]);
    }
    if (none(a[8])) {
      const int rc = f_drop_ws(d.T, (int32_t)d.D, (int32_t)d.nseg, (adaln_dtype_t)d.code, &bytes);
      if (rc != ADALN_OK) return refused(rc, "adaln_dropout_bwd_workspace_size");
      work.set(new_bytes(bytes, device.p));
      if (!work || !pointer(work.p, &ws)) return nullptr;
    } else if (!buffer(a[8], "workspace", d.dev, &ws, &bytes)) {
      return nullptr;
    }
  }
  if (!stream_of(a[9], d.dev, &stream)) return nullptr;
  int rc;
  Py_BEGIN_ALLOW_THREADS;
  rc = f_drop_bwd(d.h, h, d.gate, d.seg, d.T, (int32_t)d.D, (int32_t)d.nseg, (adaln_dtype_t)d.code, d.p,
                  d.drawn ? &d.rng : nullptr, dhp, static_cast<float*>(sum), ws, bytes, stream);
  Py_END_ALLOW_THREADS;
  if (rc != ADALN_OK) return refused(rc, "adaln_dropout_bwd");
  return pair_or(dh, dgate);
}

// ----- tokens by expert and back ----------------------------------------------------------------

// A contiguous tensor of this dtype and shape: checked and taken, or allocated.
bool array_out(PyObject* given, const char* name, int ndim, int64_t rows, int64_t cols, PyObject* dtype,
               PyObject* device, long dev, Ref* out, void** p) {
  if (none(given)) {
    Ref shape(ndim == 1 ? Py_BuildValue("(L)", (long long)rows)
                        : Py_BuildValue("(LL)", (long long)rows, (long long)cols));
    if (!shape) return false;
    out->set(new_tensor(shape.p, dtype, device));
    return *out && pointer(out->p, p);
  }
  Tensor x;
  if (!read(given, name, &x, false) || !on_device(x, name, dev) || !contiguous(given, name) ||
      !of_dtype(x, name, dtype) || !of_shape(x, name, ndim, rows, cols))
    return false;
  Py_INCREF(given);
  out->set(given);
  *p = x.ptr;
  return true;
}

bool positive(PyObject* o, const char* name, int32_t* out) {
  const long v = PyLong_AsLong(o);
  if (v == -1 && PyErr_Occurred()) return false;
  *out = v < 1 || v > INT32_MAX ? 0 : (int32_t)v;  // (0 is refused by the library)
  return true;
}

// route(expert, E, align, row, starts, counts, workspace, stream)
//   -> (row, starts, counts, rows)
PyObject* route(PyObject*, PyObject* const* a, Py_ssize_t n) {
  if (n != 8) {
    PyErr_SetString(PyExc_TypeError, "8 arguments");
    return nullptr;
  }
  Tensor x;
  int32_t E, align;
  if (!read(a[0], "expert", &x, false) || !of_dtype(x, "expert", g_i32) || !contiguous(a[0], "expert") ||
      !positive(a[1], "E", &E) || !positive(a[2], "align", &align))
    return nullptr;
  if (x.ndim != 2) {
    PyErr_SetString(PyExc_ValueError, "expert must be [T, k]");
    return nullptr;
  }
  const int64_t T = x.shape[0];
  const int32_t k = x.shape[1] > INT32_MAX ? 0 : (int32_t)x.shape[1];
  int64_t rows = 0;
  size_t bytes = 0;
  int rc = f_route_rows(T, k, E, align, &rows);
  if (rc == ADALN_OK) rc = f_route_ws(T, k, E, &bytes);
  if (rc != ADALN_OK) return refused(rc, "adaln_route");
  Ref device(PyObject_GetAttr(a[0], n_device)), row, starts, counts, work;
  void *row_p, *starts_p, *counts_p, *ws = nullptr, *stream;
  if (!device || !array_out(a[3], "row", 2, T, k, g_i32, device.p, x.dev, &row, &row_p) ||
      !array_out(a[4], "starts", 1, (int64_t)E + 1, 0, g_i32, device.p, x.dev, &starts, &starts_p) ||
      !array_out(a[5], "counts", 1, E, 0, g_i32, device.p, x.dev, &counts, &counts_p))
    return nullptr;
  if (!none(a[6])) {
    if (!buffer(a[6], "workspace", x.dev, &ws, &bytes)) return nullptr;
  } else if (bytes > 0) {
    work.set(new_bytes(bytes, device.p));
    if (!work || !pointer(work.p, &ws)) return nullptr;
  }
  if (!stream_of(a[7], x.dev, &stream)) return nullptr;
  Py_BEGIN_ALLOW_THREADS;
  rc = f_route(static_cast<const int32_t*>(x.ptr), T, k, E, align, static_cast<int32_t*>(row_p),
               static_cast<int32_t*>(starts_p), static_cast<int32_t*>(counts_p), ws, bytes, stream);
  Py_END_ALLOW_THREADS;
  if (rc != ADALN_OK) return refused(rc, "adaln_route");
  Ref size(PyLong_FromLongLong(rows));
  return size ? PyTuple_Pack(4, row.p, starts.p, counts.p, size.p) : nullptr;
}

struct Routed {
  int64_t T, rows;
  int32_t k, E, align;
  const int32_t *row, *starts, *counts;
};

// (row, starts, counts, rows, align), on device `dev`.
bool route_of(PyObject* o, long dev, Routed* r) {
  if (!PyTuple_Check(o) || PyTuple_GET_SIZE(o) != 5) {
    PyErr_SetString(PyExc_TypeError, "a route, as adaln_route returns it, is needed");
    return false;
  }
  Tensor row, starts, counts;
  Tensor* const t[3] = {&row, &starts, &counts};
  const char* const names[3] = {"row", "starts", "counts"};
  for (int i = 0; i < 3; ++i) {
    PyObject* const x = PyTuple_GET_ITEM(o, i);
    if (!read(x, names[i], t[i], false) || !on_device(*t[i], names[i], dev) || !contiguous(x, names[i]) ||
        !of_dtype(*t[i], names[i], g_i32))
      return false;
  }
  if (row.ndim != 2 || counts.ndim != 1 || row.shape[1] > INT32_MAX || counts.shape[0] > INT32_MAX) {
    PyErr_SetString(PyExc_ValueError, "row must be [T, k] and counts [E]");
    return false;
  }
  if (!of_shape(starts, "starts", 1, counts.shape[0] + 1)) return false;
  r->rows = PyLong_AsLongLong(PyTuple_GET_ITEM(o, 3));
  if (r->rows == -1 && PyErr_Occurred()) return false;
  if (!positive(PyTuple_GET_ITEM(o, 4), "align", &r->align)) return false;
  r->T = row.shape[0], r->k = (int32_t)row.shape[1], r->E = (int32_t)counts.shape[0];
  r->row = static_cast<const int32_t*>(row.ptr);
  r->starts = static_cast<const int32_t*>(starts.ptr);
  r->counts = static_cast<const int32_t*>(counts.ptr);
  return true;
}

struct Copied {
  Tensor x;
  int32_t D;
  int code;
  Routed r;
};

// x [T, D], or [rows, D] where `sorted`, and its route.
bool copy_args(PyObject* x, const char* name, bool sorted, PyObject* route, Copied* c) {
  if (!read(x, name, &c->x, false) || !contiguous(x, name) || !route_of(route, c->x.dev, &c->r)) return false;
  if (c->x.ndim != 2 || c->x.shape[1] > INT32_MAX) {
    PyErr_Format(PyExc_ValueError, "%s must be [%s, D]", name, sorted ? "rows" : "T");
    return false;
  }
  c->D = (int32_t)c->x.shape[1];
  return of_shape(c->x, name, 2, sorted ? c->r.rows : c->r.T, c->D) &&
         (c->code = dtype_code(c->x.dtype)) >= 0;
}
bool weights_of(PyObject* w, const Copied& c, const float** out) {
  void* p;
  if (!matrix(w, "weight", c.r.T, c.r.k, g_f32, c.x.dev, &p)) return false;
  *out = static_cast<const float*>(p);
  return true;
}

// expert_sort_fwd(x, route, xs, stream) -> xs
PyObject* expert_sort_fwd(PyObject*, PyObject* const* a, Py_ssize_t n) {
  if (n != 4) {
    PyErr_SetString(PyExc_TypeError, "4 arguments");
    return nullptr;
  }
  Copied c;
  void *to, *stream;
  if (!copy_args(a[0], "x", false, a[1], &c)) return nullptr;
  Ref out, device(PyObject_GetAttr(a[0], n_device));
  if (!device || !array_out(a[2], "xs", 2, c.r.rows, c.D, c.x.dtype, device.p, c.x.dev, &out, &to) ||
      !stream_of(a[3], c.x.dev, &stream))
    return nullptr;
  int rc;
  Py_BEGIN_ALLOW_THREADS;
  rc = f_sort_fwd(c.x.ptr, c.r.row, c.r.starts, c.r.counts, c.r.T, c.r.k, c.r.E, c.r.align, c.D,
                  (adaln_dtype_t)c.code, c.r.rows, to, stream);
  Py_END_ALLOW_THREADS;
  return rc != ADALN_OK ? refused(rc, "adaln_expert_sort_fwd") : out.take();
}

// expert_sort_bwd(dxs, route, dx, stream) -> dx
PyObject* expert_sort_bwd(PyObject*, PyObject* const* a, Py_ssize_t n) {
  if (n != 4) {
    PyErr_SetString(PyExc_TypeError, "4 arguments");
    return nullptr;
  }
  Copied c;
  void *to, *stream;
  if (!copy_args(a[0], "dxs", true, a[1], &c)) return nullptr;
  Ref out, device(PyObject_GetAttr(a[0], n_device));
  if (!device || !array_out(a[2], "dx", 2, c.r.T, c.D, c.x.dtype, device.p, c.x.dev, &out, &to) ||
      !stream_of(a[3], c.x.dev, &stream))
    return nullptr;
  int rc;
  Py_BEGIN_ALLOW_THREADS;
  rc = f_sort_bwd(c.x.ptr, c.r.row, c.r.T, c.r.k, c.D, (adaln_dtype_t)c.code, c.r.rows, to, stream);
  Py_END_ALLOW_THREADS;
  return rc != ADALN_OK ? refused(rc, "adaln_expert_sort_bwd") : out.take();
}

// expert_combine_fwd(ys, weight, route, y, stream) -> y
PyObject* expert_combine_fwd(PyObject*, PyObject* const* a, Py_ssize_t n) {
  if (n != 5) {
    PyErr_SetString(PyExc_TypeError, "5 arguments");
    return nullptr;
  }
  Copied c;
  const float* weight;
  void *to, *stream;
  if (!copy_args(a[0], "ys", true, a[2], &c) || !weights_of(a[1], c, &weight)) return nullptr;
  Ref out, device(PyObject_GetAttr(a[0], n_device));
  if (!device || !array_out(a[3], "y", 2, c.r.T, c.D, c.x.dtype, device.p, c.x.dev, &out, &to) ||
      !stream_of(a[4], c.x.dev, &stream))
    return nullptr;
  int rc;
  Py_BEGIN_ALLOW_THREADS;
  rc = f_combine_fwd(c.x.ptr, weight, c.r.row, c.r.T, c.r.k, c.D, (adaln_dtype_t)c.code, c.r.rows, to,
                     stream);
  Py_END_ALLOW_THREADS;
  return rc != ADALN_OK ? refused(rc, "adaln_expert_combine_fwd") : out.take();
}

// expert_combine_bwd(dy, ys, weight, route, dys, dweight, stream) -> (dys, dweight)
PyObject* expert_combine_bwd(PyObject*, PyObject* const* a, Py_ssize_t n) {
  if (n != 7) {
    PyErr_SetString(PyExc_TypeError, "7 arguments");
    return nullptr;
  }
  Copied c;
  const float* weight;
  void *ys, *to, *dw, *stream;
  if (!copy_args(a[0], "dy", false, a[3], &c) || !weights_of(a[2], c, &weight) ||
      !matrix(a[1], "ys", c.r.rows, c.D, c.x.dtype, c.x.dev, &ys))
    return nullptr;
  Ref dys, dweight, device(PyObject_GetAttr(a[0], n_device));
  if (!device || !array_out(a[4], "dys", 2, c.r.rows, c.D, c.x.dtype, device.p, c.x.dev, &dys, &to) ||
      !array_out(a[5], "dweight", 2, c.r.T, c.r.k, g_f32, device.p, c.x.dev, &dweight, &dw) ||
      !stream_of(a[6], c.x.dev, &stream))
    return nullptr;
  int rc;
  Py_BEGIN_ALLOW_THREADS;
  rc = f_combine_bwd(c.x.ptr, ys, weight, c.r.row, c.r.starts, c.r.counts, c.r.T, c.r.k, c.r.E, c.r.align,
                     c.D, (adaln_dtype_t)c.code, c.r.rows, to, static_cast<float*>(dw), stream);
  Py_END_ALLOW_THREADS;
  return rc != ADALN_OK ? refused(rc, "adaln_expert_combine_bwd") : pair_or(dys, dweight);
}

// ----- the experts' feed-forward ------------------------------------------------------------------

// A contiguous [E, rows, cols] tensor.
bool matrices(PyObject* t, const char* name, int64_t E, int64_t rows, int64_t cols, PyObject* dtype,
              long dev, void** out) {
  Tensor x;
  if (!read(t, name, &x, false) || !on_device(x, name, dev) || !contiguous(t, name) ||
      !of_dtype(x, name, dtype) || !of_shape(x, name, 3, E, rows, cols))
    return false;
  *out = x.ptr;
  return true;
}
bool matrices_out(PyObject* given, const char* name, PyObject* like, int64_t E, int64_t rows, int64_t cols,
                  PyObject* dtype, long dev, Ref* out, void** p) {
  if (none(given)) {
    out->set(PyObject_CallOneArg(g_empty_like, like));
    return *out && pointer(out->p, p);
  }
  if (!matrices(given, name, E, rows, cols, dtype, dev, p)) return false;
  Py_INCREF(given);
  out->set(given);
  return true;
}

struct Experts {
  int64_t rows, E, D, F;
  long dev;
  PyObject* dtype;
  int code;
  void *xs, *wg, *wu, *wd;
  const int32_t* starts;
};

bool experts_args(PyObject* xs, PyObject* wg, PyObject* wu, PyObject* wd, PyObject* starts, Experts* f) {
  Tensor t, g, s;
  if (!read(xs, "xs", &t, false) || !contiguous(xs, "xs") || !read(wg, "wg", &g, false)) return false;
  if (t.ndim != 2 || g.ndim != 3) {
    PyErr_SetString(PyExc_ValueError, "xs must be [rows, D] and wg [E, F, D]");
    return false;
  }
  f->rows = t.shape[0], f->D = t.shape[1], f->E = g.shape[0], f->F = g.shape[1];
  f->dev = t.dev, f->dtype = t.dtype, f->xs = t.ptr;
  if (!matrices(wg, "wg", f->E, f->F, f->D, t.dtype, t.dev, &f->wg) ||
      !matrices(wu, "wu", f->E, f->F, f->D, t.dtype, t.dev, &f->wu) ||
      !matrices(wd, "wd", f->E, f->D, f->F, t.dtype, t.dev, &f->wd) || !read(starts, "starts", &s, false) ||
      !on_device(s, "starts", t.dev) || !contiguous(starts, "starts") || !of_dtype(s, "starts", g_i32) ||
      !of_shape(s, "starts", 1, f->E + 1))
    return false;
  f->starts = static_cast<const int32_t*>(s.ptr);
  f->code = dtype_code(t.dtype);
  if (f->code < 0) return false;
  if (f->E > INT32_MAX || f->D > INT32_MAX || f->F > INT32_MAX) {
    PyErr_SetString(PyExc_ValueError, "E, D or F too large");
    return false;
  }
  return true;
}

bool experts_workspace(PyObject* given, const Experts& f, bool backward, PyObject* device, Ref* work,
                       void** p, size_t* bytes) {
  if (!none(given)) return buffer(given, "workspace", f.dev, p, bytes);
  const int rc = f_experts_ws(f.rows, (int32_t)f.E, (int32_t)f.D, (int32_t)f.F, (adaln_dtype_t)f.code,
                              backward ? nullptr : bytes, backward ? bytes : nullptr);
  if (rc != ADALN_OK) {
    refused(rc, "adaln_experts_ffn_workspace_size");
    return false;
  }
  if (*bytes < 16) *bytes = 16;
  work->set(new_bytes(*bytes, device));
  return *work && pointer(work->p, p);
}

bool experts_saved(PyObject* given, const Experts& f, size_t* need, void** p) {
  const int rc = f_experts_saved(f.rows, (int32_t)f.E, (int32_t)f.D, (int32_t)f.F, (adaln_dtype_t)f.code, need);
  if (rc != ADALN_OK) {
    refused(rc, "adaln_experts_ffn_saved_size");
    return false;
  }
  if (none(given)) return true;
  size_t have = 0;
  if (!buffer(given, "saved", f.dev, p, &have)) return false;
  if (have >= *need) return true;
  PyErr_Format(PyExc_ValueError, "saved holds %zu bytes, %zu are needed", have, *need);
  return false;
}

// experts_ffn_fwd(xs, wg, wu, wd, starts, act, save, ys, saved, workspace, stream)
//   -> (ys, saved)
PyObject* experts_ffn_fwd(PyObject*, PyObject* const* a, Py_ssize_t n) {
  if (n != 11) {
    PyErr_SetString(PyExc_TypeError, "11 arguments");
    return nullptr;
  }
  Experts f;
  int save;
  if (!experts_args(a[0], a[1], a[2], a[3], a[4], &f) || !flag(a[6], &save)) return nullptr;
  const long act = PyLong_AsLong(a[5]);
  if (act == -1 && PyErr_Occurred()) return nullptr;
  Ref device(PyObject_GetAttr(a[0], n_device)), ys, saved, work;
  void *yp, *sp = nullptr, *ws, *stream;
  size_t need = 0, bytes = 0;
  if (!device || !matrix_out(a[7], "ys", a[0], f.rows, f.D, f.dtype, f.dev, &ys, &yp)) return nullptr;
  if (save || !none(a[8])) {
    if (!experts_saved(a[8], f, &need, &sp)) return nullptr;
    if (none(a[8])) {
      saved.set(new_bytes(need, device.p));
      if (!saved || !pointer(saved.p, &sp)) return nullptr;
    } else {
      Py_INCREF(a[8]);
      saved.set(a[8]);
    }
  }
  if (!experts_workspace(a[9], f, false, device.p, &work, &ws, &bytes) ||
      !stream_of(a[10], f.dev, &stream))
    return nullptr;
  int rc;
  Py_BEGIN_ALLOW_THREADS;
  rc = f_experts_fwd(f.xs, f.wg, f.wu, f.wd, f.starts, f.rows, (int32_t)f.E, (int32_t)f.D, (int32_t)f.F,
                     (adaln_dtype_t)f.code, (adaln_act_t)act, yp, sp, ws, bytes, stream);
  Py_END_ALLOW_THREADS;
  if (rc != ADALN_OK) return refused(rc, "adaln_experts_ffn_fwd");
  return pair_or(ys, saved);
}

// experts_ffn_bwd(dys, xs, wg, wu, wd, starts, saved, act, dxs, dwg, dwu, dwd, workspace,
//                 stream) -> (dxs, dwg, dwu, dwd)
PyObject* experts_ffn_bwd(PyObject*, PyObject* const* a, Py_ssize_t n) {
  if (n != 14) {
    PyErr_SetString(PyExc_TypeError, "14 arguments");
    return nullptr;
  }
  Experts f;
  void *dys, *sp = nullptr, *dxp, *dgp, *dup, *ddp, *ws, *stream;
  size_t need = 0, bytes = 0;
  if (!experts_args(a[1], a[2], a[3], a[4], a[5], &f) ||
      !matrix(a[0], "dys", f.rows, f.D, f.dtype, f.dev, &dys))
    return nullptr;
  if (none(a[6])) {
    PyErr_SetString(PyExc_ValueError, "the backward needs what the forward saved");
    return nullptr;
  }
  const long act = PyLong_AsLong(a[7]);
  if (act == -1 && PyErr_Occurred()) return nullptr;
  Ref device(PyObject_GetAttr(a[1], n_device)), dxs, dwg, dwu, dwd, work;
  if (!device || !experts_saved(a[6], f, &need, &sp) ||
      !matrix_out(a[8], "dxs", a[1], f.rows, f.D, f.dtype, f.dev, &dxs, &dxp) ||
      !matrices_out(a[9], "dwg", a[2], f.E, f.F, f.D, f.dtype, f.dev, &dwg, &dgp) ||
      !matrices_out(a[10], "dwu", a[3], f.E, f.F, f.D, f.dtype, f.dev, &dwu, &dup) ||
      !matrices_out(a[11], "dwd", a[4], f.E, f.D, f.F, f.dtype, f.dev, &dwd, &ddp) ||
      !experts_workspace(a[12], f, true, device.p, &work, &ws, &bytes) ||
      !stream_of(a[13], f.dev, &stream))
    return nullptr;
  int rc;
  Py_BEGIN_ALLOW_THREADS;
  rc = f_experts_bwd(dys, f.xs, f.wg, f.wu, f.wd, f.starts, sp, f.rows, (int32_t)f.E, (int32_t)f.D,
                     (int32_t)f.F, (adaln_dtype_t)f.code, (adaln_act_t)act, dxp, dgp, dup, ddp, ws, bytes,
                     stream);
  Py_END_ALLOW_THREADS;
  if (rc != ADALN_OK) return refused(rc, "adaln_experts_ffn_bwd");
  return PyTuple_Pack(4, dxs.p, dwg.p, dwu.p, dwd.p);
}

// ----- module --------------------------------------------------------------------------------

template <class F>
bool entry(PyObject* addresses, const char* name, F* out) {
  PyObject* v = PyDict_GetItemString(addresses, name);  // borrowed
  if (!v) {
    PyErr_Format(PyExc_KeyError, "%s", name);
    return false;
  }
  void* p = PyLong_AsVoidPtr(v);
  if (!p && PyErr_Occurred()) return false;
  *out = reinterpret_cast<F>(p);
  return true;
}

// setup(torch, raw_stream, error, {name: address})
PyObject* setup(PyObject*, PyObject* const* a, Py_ssize_t n) {
  if (n != 4 || !PyDict_Check(a[3])) {
    PyErr_SetString(PyExc_TypeError, "setup(torch, raw_stream, error, addresses)");
    return nullptr;
  }
  struct {
    PyObject** to;
    const char* name;
  } const attrs[] = {{&g_empty, "empty"}, {&g_empty_like, "empty_like"}, {&g_bf16, "bfloat16"},
                     {&g_f32, "float32"}, {&g_i32, "int32"},             {&g_i64, "int64"},
                     {&g_u8, "uint8"}},
      names[] = {{&n_get_device, "get_device"}, {&n_shape, "shape"},
                 {&n_dtype, "dtype"},           {&n_data_ptr, "data_ptr"},
                 {&n_stride, "stride"},         {&n_is_contiguous, "is_contiguous"},
                 {&n_device, "device"},         {&n_numel, "numel"},
                 {&n_cuda_stream, "cuda_stream"}};
  for (const auto& x : attrs)
    if (!(*x.to = PyObject_GetAttrString(a[0], x.name))) return nullptr;
  for (const auto& x : names)
    if (!(*x.to = PyUnicode_InternFromString(x.name))) return nullptr;
  if (!(g_kw_dtype_device = Py_BuildValue("(ss)", "dtype", "device"))) return nullptr;
  Py_INCREF(a[1]);
  g_raw_stream = a[1];
  Py_INCREF(a[2]);
  g_error = a[2];
  if (!entry(a[3], "adaln_qk_rope_fwd", &f_qk_fwd) || !entry(a[3], "adaln_qk_rope_bwd", &f_qk_bwd) ||
      !entry(a[3], "adaln_qk_rope_bwd_workspace_size", &f_qk_ws) ||
      !entry(a[3], "adaln_ffn_fwd", &f_ffn_fwd) || !entry(a[3], "adaln_ffn_bwd", &f_ffn_bwd) ||
      !entry(a[3], "adaln_ffn_saved_size", &f_ffn_saved) ||
      !entry(a[3], "adaln_ffn_workspace_size", &f_ffn_ws) ||
      !entry(a[3], "adaln_dropout_fwd", &f_drop_fwd) || !entry(a[3], "adaln_dropout_bwd", &f_drop_bwd) ||
      !entry(a[3], "adaln_dropout_bwd_workspace_size", &f_drop_ws) ||
      !entry(a[3], "adaln_route_rows", &f_route_rows) ||
      !entry(a[3], "adaln_route_workspace_size", &f_route_ws) || !entry(a[3], "adaln_route", &f_route) ||
      !entry(a[3], "adaln_expert_sort_fwd", &f_sort_fwd) ||
      !entry(a[3], "adaln_expert_sort_bwd", &f_sort_bwd) ||
      !entry(a[3], "adaln_expert_combine_fwd", &f_combine_fwd) ||
      !entry(a[3], "adaln_expert_combine_bwd", &f_combine_bwd) ||
      !entry(a[3], "adaln_experts_ffn_saved_size", &f_experts_saved) ||
      !entry(a[3], "adaln_experts_ffn_workspace_size", &f_experts_ws) ||
      !entry(a[3], "adaln_experts_ffn_fwd", &f_experts_fwd) ||
      !entry(a[3], "adaln_experts_ffn_bwd", &f_experts_bwd))
    return nullptr;
  Py_RETURN_NONE;
}

PyMethodDef methods[] = {
    {"setup", (PyCFunction)(void (*)(void))setup, METH_FASTCALL, nullptr},
    {"qk_rope_fwd", (PyCFunction)(void (*)(void))qk_rope_fwd, METH_FASTCALL, nullptr},
    {"qk_rope_bwd", (PyCFunction)(void (*)(void))qk_rope_bwd, METH_FASTCALL, nullptr},
    {"ffn_fwd", (PyCFunction)(void (*)(void))ffn_fwd, METH_FASTCALL, nullptr},
    {"ffn_bwd", (PyCFunction)(void (*)(void))ffn_bwd, METH_FASTCALL, nullptr},
    {"dropout_fwd", (PyCFunction)(void (*)(void))dropout_fwd, METH_FASTCALL, nullptr},
    {"dropout_bwd", (PyCFunction)(void (*)(void))dropout_bwd, METH_FASTCALL, nullptr},
    {"route", (PyCFunction)(void (*)(void))route, METH_FASTCALL, nullptr},
    {"expert_sort_fwd", (PyCFunction)(void (*)(void))expert_sort_fwd, METH_FASTCALL, nullptr},
    {"expert_sort_bwd", (PyCFunction)(void (*)(void))expert_sort_bwd, METH_FASTCALL, nullptr},
    {"expert_combine_fwd", (PyCFunction)(void (*)(void))expert_combine_fwd, METH_FASTCALL, nullptr},
    {"expert_combine_bwd", (PyCFunction)(void (*)(void))expert_combine_bwd, METH_FASTCALL, nullptr},
    {"experts_ffn_fwd", (PyCFunction)(void (*)(void))experts_ffn_fwd, METH_FASTCALL, nullptr},
    {"experts_ffn_bwd", (PyCFunction)(void (*)(void))experts_ffn_bwd, METH_FASTCALL, nullptr},
    {nullptr, nullptr, 0, nullptr}};

PyModuleDef module = {PyModuleDef_HEAD_INIT, "_binding",
                      "Argument marshalling of every call but the AdaLN's.", -1, methods,
                      nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__binding(void) { return PyModule_Create(&module); }
