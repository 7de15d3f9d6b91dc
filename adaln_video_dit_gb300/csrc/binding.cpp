// Argument marshalling of the rotary and feed-forward calls, as a CPython
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
PyObject *g_bf16, *g_f32, *g_i32, *g_u8;                    // dtypes (singletons)
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
                     {&g_f32, "float32"}, {&g_i32, "int32"},             {&g_u8, "uint8"}},
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
      !entry(a[3], "adaln_ffn_workspace_size", &f_ffn_ws))
    return nullptr;
  Py_RETURN_NONE;
}

PyMethodDef methods[] = {
    {"setup", (PyCFunction)(void (*)(void))setup, METH_FASTCALL, nullptr},
    {"qk_rope_fwd", (PyCFunction)(void (*)(void))qk_rope_fwd, METH_FASTCALL, nullptr},
    {"qk_rope_bwd", (PyCFunction)(void (*)(void))qk_rope_bwd, METH_FASTCALL, nullptr},
    {"ffn_fwd", (PyCFunction)(void (*)(void))ffn_fwd, METH_FASTCALL, nullptr},
    {"ffn_bwd", (PyCFunction)(void (*)(void))ffn_bwd, METH_FASTCALL, nullptr},
    {nullptr, nullptr, 0, nullptr}};

PyModuleDef module = {PyModuleDef_HEAD_INIT, "_binding",
                      "Argument marshalling of the rotary and feed-forward calls.", -1, methods,
                      nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__binding(void) { return PyModule_Create(&module); }
