/* Argument marshalling of the decode and scoring calls for Python, in C.
 *
 * These calls take a few microseconds on the GPU, and reading the properties
 * of seven to ten tensors in Python and passing two dozen arguments by ctypes
 * takes longer than that.  Each function here makes the same checks as the
 * binding's Python path (dtype, shape, device, contiguity), calls the C ABI
 * and returns its status.  Anything it does not recognise as a good call
 * (a wrong shape, a CPU tensor, an object that is no tensor) returns None, and
 * the Python path then says what is wrong: nothing is refused here, and
 * nothing passes that the Python path would refuse.
 */
#define PY_SSIZE_T_CLEAN
#include <Python.h>

#include <stdint.h>

#include "coda.h"

enum { F32 = CODA_F32, BF16 = CODA_BF16, E4M3 = CODA_E4M3, I32 = 3, UNKNOWN = 4 };

static PyObject *s_dtype, *s_shape, *s_get_device, *s_is_contiguous, *s_data_ptr, *s_stride;
static PyObject *t_f32, *t_bf16, *t_e4m3, *t_u8, *t_i32, *f_device, *f_stream;
static __typeof__(&coda_paged_append) p_append;
static __typeof__(&coda_paged_attention) p_attention;
static __typeof__(&coda_paged_attention_workspace_bytes) p_workspace;
static __typeof__(&coda_logprobs) p_logprobs;
static __typeof__(&coda_logprobs_backward) p_backward;

/* A tensor's data: a missing one (None) has ptr NULL and here = 0. */
typedef struct {
  void* ptr;
  const void* dtype; /* the dtype object, for comparing only */
  int here, type, nd;
  int64_t shape[4], numel;
} View;

/* Reads tensor t on device dev; 0 if it is not one that the fast path takes.
 * dense: it has to be contiguous. */
static int view(PyObject* t, View* v, long dev, int dense) {
  v->ptr = NULL;
  v->here = 0;
  v->numel = 0;
  if (t == Py_None) return 1;
  PyObject* d = PyObject_GetAttr(t, s_dtype);
  if (!d) return 0;
  v->type = d == t_f32 ? F32 : d == t_bf16 ? BF16 : d == t_e4m3 || d == t_u8 ? E4M3 : d == t_i32 ? I32 : UNKNOWN;
  v->dtype = d;
  Py_DECREF(d);
  if (v->type == UNKNOWN) return 0;
  PyObject* s = PyObject_GetAttr(t, s_shape);
  if (!s) return 0;
  int ok = PyTuple_Check(s) && PyTuple_GET_SIZE(s) <= 4;
  v->nd = ok ? (int)PyTuple_GET_SIZE(s) : 0;
  v->numel = 1;
  for (int i = 0; i < v->nd; ++i) {
    v->shape[i] = PyLong_AsLongLong(PyTuple_GET_ITEM(s, i));
    v->numel *= v->shape[i];
  }
  Py_DECREF(s);
  if (!ok) return 0;
  PyObject* r = PyObject_CallMethodNoArgs(t, s_get_device);
  if (!r) return 0;
  ok = PyLong_AsLong(r) == dev;
  Py_DECREF(r);
  if (!ok) return 0;
  if (dense) {
    r = PyObject_CallMethodNoArgs(t, s_is_contiguous);
    if (!r) return 0;
    ok = r == Py_True;
    Py_DECREF(r);
    if (!ok) return 0;
  }
  r = PyObject_CallMethodNoArgs(t, s_data_ptr);
  if (!r) return 0;
  v->ptr = (void*)(uintptr_t)PyLong_AsUnsignedLongLong(r);
  Py_DECREF(r);
  v->here = 1;
  return !PyErr_Occurred();
}

/* Whether a view is a tensor of this type and shape (or, nd < 0, one element or more). */
static int is(const View* v, int type, int nd, int64_t a, int64_t b, int64_t c) {
  if (!v->here || v->type != type) return 0;
  if (nd < 0) return v->numel > 0;
  return v->nd == nd && v->shape[0] == a && (nd < 2 || v->shape[1] == b) && (nd < 3 || v->shape[2] == c);
}
static int is_or_none(const View* v, int type, int nd, int64_t a, int64_t b, int64_t c) {
  return !v->here || is(v, type, nd, a, b, c);
}

/* The row stride of a tensor whose rows are dense; -1 if they are not. */
static int64_t row_stride(PyObject* t, const View* v) {
  PyObject* s = PyObject_CallMethodNoArgs(t, s_stride);
  if (!s) return -1;
  int64_t inner = 1, ld = -1;
  int ok = PyTuple_Check(s) && PyTuple_GET_SIZE(s) == v->nd;
  for (int i = v->nd - 1; ok && i > 0; --i) {
    if (v->shape[i] != 1 && PyLong_AsLongLong(PyTuple_GET_ITEM(s, i)) != inner) ok = 0;
    inner *= v->shape[i];
  }
  if (ok) ld = v->shape[0] > 1 ? PyLong_AsLongLong(PyTuple_GET_ITEM(s, 0)) : inner;
  Py_DECREF(s);
  return ld;
}

/* The current device; -2 on an error. */
static long current_device(void) {
  PyObject* r = PyObject_CallNoArgs(f_device);
  if (!r) return -2;
  const long dev = PyLong_AsLong(r);
  Py_DECREF(r);
  return dev;
}

/* `stream` as an address: None is the device's current stream. */
static int stream_of(PyObject* stream, long dev, cudaStream_t* out) {
  PyObject* r;
  if (stream == Py_None) {
    PyObject* d = PyLong_FromLong(dev);
    if (!d) return 0;
    r = PyObject_CallOneArg(f_stream, d);
    Py_DECREF(d);
    if (!r) return 0;
  } else {
    r = Py_NewRef(stream);
  }
  *out = (cudaStream_t)(uintptr_t)PyLong_AsUnsignedLongLong(r);
  Py_DECREF(r);
  return !PyErr_Occurred();
}

static PyObject* not_taken(void) {
  PyErr_Clear();
  Py_RETURN_NONE;
}

static int caches(const View* k, const View* v, int type) {
  return k->here && k->nd == 4 && v->here && v->nd == 4 && v->dtype == k->dtype &&
         (k->type == type || (type == BF16 && k->type == E4M3)) && v->shape[0] == k->shape[0] &&
         v->shape[1] == k->shape[1] && v->shape[2] == k->shape[2] && v->shape[3] == k->shape[3];
}

/* (Z, positions, row_seq, page_table, Q, k_cache, v_cache, scale_k, scale_v, q_heads, base, stream) */
static PyObject* paged_append(PyObject* self, PyObject* const* a, Py_ssize_t n) {
  (void)self;
  if (n != 12) return not_taken();
  const long dev = current_device();
  View Z, pos, seq, tab, Q, K, V, sk, sv;
  cudaStream_t st;
  if (dev < 0 || !view(a[0], &Z, dev, 1) || !view(a[1], &pos, dev, 1) || !view(a[2], &seq, dev, 1) ||
      !view(a[3], &tab, dev, 1) || !view(a[4], &Q, dev, 1) || !view(a[5], &K, dev, 1) || !view(a[6], &V, dev, 1) ||
      !view(a[7], &sk, dev, 1) || !view(a[8], &sv, dev, 1))
    return not_taken();
  const int64_t hq = PyLong_AsLongLong(a[9]);
  const double base = PyFloat_AsDouble(a[10]);
  if (!stream_of(a[11], dev, &st) || PyErr_Occurred() || !Z.here || (Z.type != F32 && Z.type != BF16) || Z.nd != 2 ||
      !caches(&K, &V, Z.type))
    return not_taken();
  const int64_t M = Z.shape[0], pages = K.shape[0], hkv = K.shape[1], page = K.shape[2], d = K.shape[3];
  if (Z.shape[1] != (hq + 2 * hkv) * d || !is(&pos, I32, 1, M, 0, 0) || !is_or_none(&seq, I32, 1, M, 0, 0) ||
      !tab.here || tab.type != I32 || tab.nd != 2 || !is_or_none(&Q, Z.type, 3, M, hq, d) ||
      !is_or_none(&sk, F32, -1, 0, 0, 0) || !is_or_none(&sv, F32, -1, 0, 0, 0))
    return not_taken();
  coda_status s;
  Py_BEGIN_ALLOW_THREADS
  s = p_append(Z.ptr, pos.ptr, seq.ptr, tab.ptr, Q.ptr, K.ptr, V.ptr, M, tab.shape[0], tab.shape[1], hq, hkv, d, pages,
               page, base, (coda_dtype)Z.type, (coda_dtype)K.type, sk.ptr, sv.ptr, st);
  Py_END_ALLOW_THREADS
  return PyLong_FromLong(s);
}

/* (Q, k_cache, v_cache, page_table, lengths, workspace, row_seq, scale, O, lse, scale_k, scale_v, stream) */
static PyObject* paged_attention(PyObject* self, PyObject* const* a, Py_ssize_t n) {
  (void)self;
  if (n != 13) return not_taken();
  const long dev = current_device();
  View Q, K, V, tab, len, ws, seq, O, lse, sk, sv;
  cudaStream_t st;
  if (dev < 0 || !view(a[0], &Q, dev, 0) || !view(a[1], &K, dev, 1) || !view(a[2], &V, dev, 1) ||
      !view(a[3], &tab, dev, 1) || !view(a[4], &len, dev, 1) || !view(a[5], &ws, dev, 1) ||
      !view(a[6], &seq, dev, 1) || !view(a[8], &O, dev, 1) || !view(a[9], &lse, dev, 1) ||
      !view(a[10], &sk, dev, 1) || !view(a[11], &sv, dev, 1))
    return not_taken();
  const double scale = PyFloat_AsDouble(a[7]);
  if (!stream_of(a[12], dev, &st) || PyErr_Occurred() || !Q.here || (Q.type != F32 && Q.type != BF16) || Q.nd != 3 ||
      !caches(&K, &V, Q.type))
    return not_taken();
  const int64_t M = Q.shape[0], hq = Q.shape[1], d = Q.shape[2], hkv = K.shape[1], ldq = row_stride(a[0], &Q);
  const int64_t size = ws.here ? ws.numel * (ws.type == E4M3 ? 1 : ws.type == BF16 ? 2 : 4) : -1;
  if (ldq < 0 || K.shape[3] != d || !tab.here || tab.type != I32 || tab.nd != 2 || !is(&len, I32, 1, M, 0, 0) ||
      !is_or_none(&seq, I32, 1, M, 0, 0) || !is(&O, Q.type, 2, M, hq * d, 0) || !is_or_none(&lse, F32, 2, M, hq, 0) ||
      !is_or_none(&sk, F32, -1, 0, 0, 0) || !is_or_none(&sv, F32, -1, 0, 0, 0) || size < p_workspace(hq, hkv, d))
    return not_taken();
  coda_status s;
  Py_BEGIN_ALLOW_THREADS
  s = p_attention(Q.ptr, ldq, K.ptr, V.ptr, tab.ptr, len.ptr, seq.ptr, O.ptr, lse.ptr, M, tab.shape[0], tab.shape[1],
                  hq, hkv, d, K.shape[0], K.shape[2], (float)scale, (coda_dtype)Q.type, (coda_dtype)K.type, sk.ptr,
                  sv.ptr, ws.ptr, st);
  Py_END_ALLOW_THREADS
  return PyLong_FromLong(s);
}

/* Row stride of logits [M, V]: of a single row, whole 16 bytes. */
static int64_t logits_stride(PyObject* t, const View* v) {
  const int64_t step = v->type == F32 ? 4 : 8, ld = row_stride(t, v);
  return ld < 0 ? -1 : v->shape[0] > 1 ? ld : (v->shape[1] + step - 1) / step * step;
}

/* (logits, targets, top, logp, entropy, lse, top_logp, top_ids, stream) */
static PyObject* logprobs(PyObject* self, PyObject* const* a, Py_ssize_t n) {
  (void)self;
  if (n != 9) return not_taken();
  const long dev = current_device();
  View x, t, lp, ent, lse, tl, ti;
  cudaStream_t st;
  if (dev < 0 || !view(a[0], &x, dev, 0) || !view(a[1], &t, dev, 1) || !view(a[3], &lp, dev, 1) ||
      !view(a[4], &ent, dev, 1) || !view(a[5], &lse, dev, 1) || !view(a[6], &tl, dev, 1) || !view(a[7], &ti, dev, 1))
    return not_taken();
  const int64_t top = PyLong_AsLongLong(a[2]);
  if (!stream_of(a[8], dev, &st) || PyErr_Occurred() || !x.here || (x.type != F32 && x.type != BF16) || x.nd != 2)
    return not_taken();
  const int64_t M = x.shape[0], V = x.shape[1], ld = logits_stride(a[0], &x);
  if (ld < 0 || !is(&t, I32, 1, M, 0, 0) || !is(&lp, F32, 1, M, 0, 0) || !is(&ent, F32, 1, M, 0, 0) ||
      !is(&lse, F32, 1, M, 0, 0) || (top > 0 && (!is(&tl, F32, 2, M, top, 0) || !is(&ti, I32, 2, M, top, 0))))
    return not_taken();
  coda_status s;
  Py_BEGIN_ALLOW_THREADS
  s = p_logprobs(x.ptr, ld, t.ptr, lp.ptr, ent.ptr, lse.ptr, tl.ptr, ti.ptr, M, V, top, (coda_dtype)x.type, st);
  Py_END_ALLOW_THREADS
  return PyLong_FromLong(s);
}

/* (logits, targets, lse, entropy, dlogp, dentropy, dlogits, stream) */
static PyObject* logprobs_backward(PyObject* self, PyObject* const* a, Py_ssize_t n) {
  (void)self;
  if (n != 8) return not_taken();
  const long dev = current_device();
  View x, t, lse, ent, dl, dh, dx;
  cudaStream_t st;
  if (dev < 0 || !view(a[0], &x, dev, 0) || !view(a[1], &t, dev, 1) || !view(a[2], &lse, dev, 1) ||
      !view(a[3], &ent, dev, 1) || !view(a[4], &dl, dev, 1) || !view(a[5], &dh, dev, 1) || !view(a[6], &dx, dev, 0))
    return not_taken();
  if (!stream_of(a[7], dev, &st) || !x.here || (x.type != F32 && x.type != BF16) || x.nd != 2) return not_taken();
  const int64_t M = x.shape[0], V = x.shape[1];
  if (!is(&dx, x.type, 2, M, V, 0) || !is(&t, I32, 1, M, 0, 0) || !is(&lse, F32, 1, M, 0, 0) ||
      !is_or_none(&ent, F32, 1, M, 0, 0) || !is_or_none(&dl, F32, 1, M, 0, 0) || !is_or_none(&dh, F32, 1, M, 0, 0))
    return not_taken();
  const int64_t ld = logits_stride(a[0], &x), ldd = logits_stride(a[6], &dx);
  if (ld < 0 || ldd < 0) return not_taken();
  coda_status s;
  Py_BEGIN_ALLOW_THREADS
  s = p_backward(x.ptr, ld, t.ptr, lse.ptr, ent.ptr, dl.ptr, dh.ptr, dx.ptr, ldd, M, V, (coda_dtype)x.type, st);
  Py_END_ALLOW_THREADS
  return PyLong_FromLong(s);
}

/* (float32, bfloat16, float8_e4m3fn, uint8, int32, current_device, current_raw_stream, and the addresses of the five
 * C ABI functions in the order of their pointers above): once, before any call. */
static PyObject* init(PyObject* self, PyObject* const* a, Py_ssize_t n) {
  (void)self;
  if (n != 12) {
    PyErr_SetString(PyExc_TypeError, "init takes 12 arguments");
    return NULL;
  }
  PyObject** const objects[] = {&t_f32, &t_bf16, &t_e4m3, &t_u8, &t_i32, &f_device, &f_stream};
  for (int i = 0; i < 7; ++i) Py_XSETREF(*objects[i], Py_NewRef(a[i]));
  uintptr_t f[5];
  for (int i = 0; i < 5; ++i) f[i] = (uintptr_t)PyLong_AsUnsignedLongLong(a[7 + i]);
  if (PyErr_Occurred()) return NULL;
  p_append = (__typeof__(p_append))f[0];
  p_attention = (__typeof__(p_attention))f[1];
  p_workspace = (__typeof__(p_workspace))f[2];
  p_logprobs = (__typeof__(p_logprobs))f[3];
  p_backward = (__typeof__(p_backward))f[4];
  Py_RETURN_NONE;
}

static PyMethodDef methods[] = {
    {"init", (PyCFunction)(void (*)(void))init, METH_FASTCALL, NULL},
    {"paged_append", (PyCFunction)(void (*)(void))paged_append, METH_FASTCALL, NULL},
    {"paged_attention", (PyCFunction)(void (*)(void))paged_attention, METH_FASTCALL, NULL},
    {"logprobs", (PyCFunction)(void (*)(void))logprobs, METH_FASTCALL, NULL},
    {"logprobs_backward", (PyCFunction)(void (*)(void))logprobs_backward, METH_FASTCALL, NULL},
    {NULL, NULL, 0, NULL}};

static struct PyModuleDef module = {PyModuleDef_HEAD_INIT, "_coda_marshal", NULL, -1, methods, NULL, NULL, NULL, NULL};

PyMODINIT_FUNC PyInit__coda_marshal(void) {
  const char* const names[] = {"dtype", "shape", "get_device", "is_contiguous", "data_ptr", "stride"};
  PyObject** const slots[] = {&s_dtype, &s_shape, &s_get_device, &s_is_contiguous, &s_data_ptr, &s_stride};
  for (int i = 0; i < 6; ++i)
    if (!(*slots[i] = PyUnicode_InternFromString(names[i]))) return NULL;
  return PyModule_Create(&module);
}
