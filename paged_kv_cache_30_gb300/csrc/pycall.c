/* pycall.c -- the binding of the 8-bit cache, window, rotation and page calls, on the CPython C API.
 *
 * It does what a ctypes call does (tensors to pkv_tensor descriptors, the current stream, an
 * exception for a negative status) in compiled code: these calls come many times a step and take
 * the device a few microseconds each, and the interpreted form took the host 12 us a call, this
 * one about half.  bind() receives the library's entry points, so the library is loaded in one
 * place, in the package. */
#define PY_SSIZE_T_CLEAN
#include <Python.h>

#include "../../include/pkv.h"

typedef int (*attn8_fn)(const pkv_tensor*, const pkv_tensor*, const pkv_tensor*, const pkv_tensor*,
                        const pkv_tensor*, const pkv_tensor*, int, int, float, int,
                        const pkv_tensor*, const pkv_tensor*, void*);
typedef int (*window_fn)(const pkv_tensor*, const pkv_tensor*, const pkv_tensor*,
                         const pkv_tensor*, const pkv_tensor*, int, int, float, int,
                         const pkv_tensor*, const pkv_tensor*, void*);
typedef int (*append_fn)(const pkv_tensor*, const pkv_tensor*, const pkv_tensor*,
                         const pkv_tensor*, const pkv_tensor*, const pkv_tensor*,
                         const pkv_tensor*, int, void*);
typedef int (*fork_fn)(const pkv_tensor*, const pkv_tensor*, const pkv_tensor*, const pkv_tensor*,
                       const pkv_tensor*, int, const pkv_tensor*, const pkv_tensor*, void*);
typedef int (*rows_fn)(const pkv_tensor*, const pkv_tensor*, const pkv_tensor*, const pkv_tensor*,
                       const pkv_tensor*, int, void*);
typedef int (*trim_fn)(const pkv_tensor*, const pkv_tensor*, const pkv_tensor*, int, int, int, void*);
typedef int (*compact_fn)(const pkv_tensor*, const pkv_tensor*, const pkv_tensor*, int,
                          const pkv_tensor*, const pkv_tensor*, const pkv_tensor*, void*);
typedef int (*copy_fn)(const pkv_tensor* const*, int, const pkv_tensor*, const pkv_tensor*, void*);
typedef int (*rope_fn)(const pkv_tensor*, const pkv_tensor*, const pkv_tensor*, const pkv_tensor*,
                       float, const pkv_tensor*, const pkv_tensor*, float, int, const pkv_tensor*,
                       const pkv_tensor*, void*);
typedef int (*rope_append_fn)(const pkv_tensor*, const pkv_tensor*, const pkv_tensor*,
                              const pkv_tensor*, const pkv_tensor*, float, const pkv_tensor*,
                              const pkv_tensor*, float, int, const pkv_tensor*, const pkv_tensor*,
                              const pkv_tensor*, const pkv_tensor*, int, const pkv_tensor*, void*);
typedef int (*prefix8_fn)(const pkv_tensor*, const pkv_tensor*, const pkv_tensor*,
                          const pkv_tensor*, const pkv_tensor*, const pkv_tensor*,
                          const pkv_tensor*, const pkv_tensor*, float, int, const pkv_tensor*,
                          const pkv_tensor*, void*);
typedef int (*prefix_fn)(const pkv_tensor*, const pkv_tensor*, const pkv_tensor*, const pkv_tensor*,
                         const pkv_tensor*, const pkv_tensor*, const pkv_tensor*, float, int,
                         const pkv_tensor*, const pkv_tensor*, void*);
typedef const char* (*text_fn)(void);

enum { ATTN8, WINDOW, APPEND, FORK, RELEASE, RESERVE, COMPACT, COPY, TRIM, ROPE, ROPE_APPEND,
       PREFIX8, PREFIX, LAST_ERROR, NUM_FNS };
enum { MAX_TENSORS = 66 }; /* 64 page tensors and two lists */

static void* fns[NUM_FNS];
static PyObject *dtypes[5], *raw_stream, *error_type; /* dtypes[code] */
static PyObject *n_data_ptr, *n_shape, *n_stride, *n_dtype, *n_get_device, *n_cuda_stream;

static int fail(int code, const char* message) {
  PyObject* e = PyObject_CallFunction(error_type, "is", code, message);
  if (e) {
    PyErr_SetObject(error_type, e);
    Py_DECREF(e);
  }
  return -1;
}

/* The status of a call: None, or the exception. */
static PyObject* status(int rc) {
  if (rc >= 0) Py_RETURN_NONE;
  fail(rc, ((text_fn)fns[LAST_ERROR])());
  return NULL;
}

static int int64s(PyObject* t, int64_t* out, int n) {
  if (!PyTuple_Check(t) || PyTuple_GET_SIZE(t) != n) {
    PyErr_SetString(PyExc_TypeError, "a tensor's shape and stride are tuples");
    return -1;
  }
  for (int i = 0; i < n; ++i) {
    out[i] = PyLong_AsLongLong(PyTuple_GET_ITEM(t, i));
    if (out[i] == -1 && PyErr_Occurred()) return -1;
  }
  return 0;
}

/* Descriptor of a torch tensor; None is NULL in *slot. */
static int describe(PyObject* t, pkv_tensor* d, const pkv_tensor** slot) {
  *slot = NULL;
  if (t == Py_None) return 0;
  memset(d, 0, sizeof *d);
  PyObject* v = PyObject_GetAttr(t, n_dtype);
  if (!v) return -1;
  for (int i = 1; i < 5; ++i)
    if (v == dtypes[i]) d->dtype = i;
  Py_DECREF(v);
  if (!d->dtype) return fail(PKV_ERR_INVALID_ARG, "unsupported tensor dtype");
  if (!(v = PyObject_GetAttr(t, n_shape))) return -1;
  const Py_ssize_t n = PyTuple_Check(v) ? PyTuple_GET_SIZE(v) : 0;
  int rc = n > 5 ? fail(PKV_ERR_INVALID_ARG, "tensors of more than 5 dims are not supported")
                 : int64s(v, d->shape, (int)n);
  Py_DECREF(v);
  if (rc) return -1;
  d->ndim = (int32_t)n;
  if (!(v = PyObject_CallMethodNoArgs(t, n_stride))) return -1;
  rc = int64s(v, d->stride, (int)n);
  Py_DECREF(v);
  if (rc) return -1;
  if (!(v = PyObject_CallMethodNoArgs(t, n_data_ptr))) return -1;
  d->data = PyLong_AsVoidPtr(v);
  Py_DECREF(v);
  if (!d->data && PyErr_Occurred()) return -1;
  *slot = d;
  return 0;
}

/* A stream argument: None is torch's current stream of the tensor's device. */
static int stream_of(PyObject* s, PyObject* tensor, void** out) {
  PyObject* v;
  if (s == Py_None) {
    PyObject* index = PyObject_CallMethodNoArgs(tensor, n_get_device);
    if (!index) return -1;
    if (PyLong_AsLong(index) < 0) {
      Py_DECREF(index);
      return PyErr_Occurred() ? -1 : fail(PKV_ERR_INVALID_ARG, "a tensor is not on a CUDA device");
    }
    v = PyObject_CallOneArg(raw_stream, index);
    Py_DECREF(index);
  } else if (PyLong_Check(s)) {
    v = Py_NewRef(s);
  } else {
    v = PyObject_GetAttr(s, n_cuda_stream);
  }
  if (!v) return -1;
  *out = PyLong_AsVoidPtr(v);
  Py_DECREF(v);
  return !*out && PyErr_Occurred() ? -1 : 0;
}

/* int(x or 0), within the range of a C int */
static int int_of(PyObject* x, int* out) {
  if (x == Py_None) {
    *out = 0;
    return 0;
  }
  PyObject* v = PyNumber_Long(x);
  if (!v) return -1;
  const long n = PyLong_AsLong(v);
  Py_DECREF(v);
  if (n == -1 && PyErr_Occurred()) return -1;
  if (n != (int)n) return fail(PKV_ERR_INVALID_ARG, "an integer argument exceeds 32 bits");
  *out = (int)n;
  return 0;
}

static int float_of(PyObject* x, float* out) {
  const double v = PyFloat_AsDouble(x);
  if (v == -1.0 && PyErr_Occurred()) return -1;
  *out = (float)v;
  return 0;
}

static int count_args(Py_ssize_t got, Py_ssize_t want) {
  if (!fns[0]) {
    PyErr_SetString(PyExc_RuntimeError, "the library is not loaded");
    return -1;
  }
  if (got == want) return 0;
  PyErr_Format(PyExc_TypeError, "%zd arguments, not %zd", want, got);
  return -1;
}

/* Positions of a call's tensors among its arguments. */
static int describe_all(PyObject* const* a, const int* at, int n, pkv_tensor* d,
                        const pkv_tensor** p) {
  for (int i = 0; i < n; ++i)
    if (describe(a[at[i]], d + i, p + i)) return -1;
  return 0;
}

#define CALL(expr)                \
  int rc;                         \
  Py_BEGIN_ALLOW_THREADS rc = (expr); \
  Py_END_ALLOW_THREADS return status(rc)

/* q, kv_cache, kv_scale, block_table, seq_lens, sinks, window, first_tokens, scale, page_size,
 * out, lse, stream */
static PyObject* attn8(PyObject* self, PyObject* const* a, Py_ssize_t n) {
  static const int at[8] = {0, 1, 2, 3, 4, 5, 10, 11};
  pkv_tensor d[8];
  const pkv_tensor* p[8];
  int window, first, page;
  float scale;
  void* s;
  if (count_args(n, 13) || describe_all(a, at, 8, d, p) || int_of(a[6], &window) ||
      int_of(a[7], &first) || float_of(a[8], &scale) || int_of(a[9], &page) ||
      stream_of(a[12], a[0], &s))
    return NULL;
  CALL(((attn8_fn)fns[ATTN8])(p[0], p[1], p[2], p[3], p[4], p[5], window, first, scale, page, p[6],
                              p[7], s));
}

/* q, kv_cache, block_table, seq_lens, sinks, window, first_tokens, scale, page_size, out, lse,
 * stream */
static PyObject* window_attn(PyObject* self, PyObject* const* a, Py_ssize_t n) {
  static const int at[7] = {0, 1, 2, 3, 4, 9, 10};
  pkv_tensor d[7];
  const pkv_tensor* p[7];
  int window, first, page;
  float scale;
  void* s;
  if (count_args(n, 12) || describe_all(a, at, 7, d, p) || int_of(a[5], &window) ||
      int_of(a[6], &first) || float_of(a[7], &scale) || int_of(a[8], &page) ||
      stream_of(a[11], a[0], &s))
    return NULL;
  CALL(((window_fn)fns[WINDOW])(p[0], p[1], p[2], p[3], p[4], window, first, scale, page, p[5],
                                p[6], s));
}

/* q, kv_cache, kv_scale, block_table, seq_lens, cu_groups, shared_lens, sinks, scale, page_size,
 * out, lse, stream */
static PyObject* prefix8(PyObject* self, PyObject* const* a, Py_ssize_t n) {
  static const int at[10] = {0, 1, 2, 3, 4, 5, 6, 7, 10, 11};
  pkv_tensor d[10];
  const pkv_tensor* p[10];
  int page;
  float scale;
  void* s;
  if (count_args(n, 13) || describe_all(a, at, 10, d, p) || float_of(a[8], &scale) ||
      int_of(a[9], &page) || stream_of(a[12], a[0], &s))
    return NULL;
  CALL(((prefix8_fn)fns[PREFIX8])(p[0], p[1], p[2], p[3], p[4], p[5], p[6], p[7], scale, page, p[8],
                                  p[9], s));
}

/* q, kv_cache, block_table, seq_lens, cu_groups, shared_lens, sinks, scale, page_size, out, lse,
 * stream */
static PyObject* prefix(PyObject* self, PyObject* const* a, Py_ssize_t n) {
  static const int at[9] = {0, 1, 2, 3, 4, 5, 6, 9, 10};
  pkv_tensor d[9];
  const pkv_tensor* p[9];
  int page;
  float scale;
  void* s;
  if (count_args(n, 12) || describe_all(a, at, 9, d, p) || float_of(a[7], &scale) ||
      int_of(a[8], &page) || stream_of(a[11], a[0], &s))
    return NULL;
  CALL(((prefix_fn)fns[PREFIX])(p[0], p[1], p[2], p[3], p[4], p[5], p[6], scale, page, p[7], p[8], s));
}

/* k, v, kv_cache, kv_scale, block_table, seq_lens, cu_tokens, page_size, stream */
static PyObject* append(PyObject* self, PyObject* const* a, Py_ssize_t n) {
  static const int at[7] = {0, 1, 2, 3, 4, 5, 6};
  pkv_tensor d[7];
  const pkv_tensor* p[7];
  int page;
  void* s;
  if (count_args(n, 9) || describe_all(a, at, 7, d, p) || int_of(a[7], &page) ||
      stream_of(a[8], a[0], &s))
    return NULL;
  CALL(((append_fn)fns[APPEND])(p[0], p[1], p[2], p[3], p[4], p[5], p[6], page, s));
}

/* block_table, seq_lens, page_refs, parents, children, page_size, copy_src, copy_dst, stream */
static PyObject* fork_rows(PyObject* self, PyObject* const* a, Py_ssize_t n) {
  static const int at[7] = {0, 1, 2, 3, 4, 6, 7};
  pkv_tensor d[7];
  const pkv_tensor* p[7];
  int page;
  void* s;
  if (count_args(n, 9) || describe_all(a, at, 7, d, p) || int_of(a[5], &page) ||
      stream_of(a[8], a[0], &s))
    return NULL;
  CALL(((fork_fn)fns[FORK])(p[0], p[1], p[2], p[3], p[4], page, p[5], p[6], s));
}

/* block_table, seq_lens, page_refs, rows, lens, page_size, stream */
static PyObject* rows_call(void* fn, PyObject* const* a, Py_ssize_t n) {
  static const int at[5] = {0, 1, 2, 3, 4};
  pkv_tensor d[5];
  const pkv_tensor* p[5];
  int page;
  void* s;
  if (count_args(n, 7) || describe_all(a, at, 5, d, p) || int_of(a[5], &page) ||
      stream_of(a[6], a[0], &s))
    return NULL;
  CALL(((rows_fn)fn)(p[0], p[1], p[2], p[3], p[4], page, s));
}
static PyObject* release(PyObject* self, PyObject* const* a, Py_ssize_t n) {
  return rows_call(fns[RELEASE], a, n);
}
static PyObject* reserve(PyObject* self, PyObject* const* a, Py_ssize_t n) {
  return rows_call(fns[RESERVE], a, n);
}

/* block_table, seq_lens, page_refs, page_size, window, first_tokens, stream */
static PyObject* trim(PyObject* self, PyObject* const* a, Py_ssize_t n) {
  static const int at[3] = {0, 1, 2};
  pkv_tensor d[3];
  const pkv_tensor* p[3];
  int page, window, first;
  void* s;
  if (count_args(n, 7) || describe_all(a, at, 3, d, p) || int_of(a[3], &page) ||
      int_of(a[4], &window) || int_of(a[5], &first) || stream_of(a[6], a[2], &s))
    return NULL;
  CALL(((trim_fn)fns[TRIM])(p[0], p[1], p[2], page, window, first, s));
}

/* block_table, seq_lens, page_refs, page_size, copy_src, copy_dst, num_moves, stream */
static PyObject* compact(PyObject* self, PyObject* const* a, Py_ssize_t n) {
  static const int at[6] = {0, 1, 2, 4, 5, 6};
  pkv_tensor d[6];
  const pkv_tensor* p[6];
  int page;
  void* s;
  if (count_args(n, 8) || describe_all(a, at, 6, d, p) || int_of(a[3], &page) ||
      stream_of(a[7], a[2], &s))
    return NULL;
  CALL(((compact_fn)fns[COMPACT])(p[0], p[1], p[2], page, p[3], p[4], p[5], s));
}

/* pages (a list or tuple of tensors), copy_src, copy_dst, stream */
static PyObject* copy(PyObject* self, PyObject* const* a, Py_ssize_t n) {
  pkv_tensor d[MAX_TENSORS];
  const pkv_tensor* p[MAX_TENSORS];
  void* s;
  if (count_args(n, 4)) return NULL;
  PyObject* pages = PySequence_Tuple(a[0]); /* holds the tensors until the call is made */
  if (!pages) return NULL;
  const Py_ssize_t k = PyTuple_GET_SIZE(pages);
  int bad = 0, rc = 0;
  if (k < 1 || k > MAX_TENSORS - 2)
    bad = fail(PKV_ERR_INVALID_ARG, "pages_copy takes 1 to 64 page tensors");
  for (Py_ssize_t i = 0; !bad && i < k; ++i) {
    PyObject* t = PyTuple_GET_ITEM(pages, i);
    bad = t == Py_None ? fail(PKV_ERR_INVALID_ARG, "a page tensor is None")
                       : describe(t, d + 2 + i, p + 2 + i);
  }
  bad = bad || describe(a[1], d, p) || describe(a[2], d + 1, p + 1) ||
        stream_of(a[3], PyTuple_GET_ITEM(pages, 0), &s);
  if (!bad) {
    Py_BEGIN_ALLOW_THREADS rc = ((copy_fn)fns[COPY])(p + 2, (int)k, p[0], p[1], s);
    Py_END_ALLOW_THREADS
  }
  Py_DECREF(pages);
  return bad ? NULL : status(rc);
}

/* q, k, q_weight, k_weight, eps, positions, rope, rope_factor, interleaved, q_out, k_out, stream */
static PyObject* rope(PyObject* self, PyObject* const* a, Py_ssize_t n) {
  static const int at[8] = {0, 1, 2, 3, 5, 6, 9, 10};
  pkv_tensor d[8];
  const pkv_tensor* p[8];
  int pairs;
  float eps, factor;
  void* s;
  if (count_args(n, 12) || describe_all(a, at, 8, d, p) || float_of(a[4], &eps) ||
      float_of(a[7], &factor) || int_of(a[8], &pairs) || stream_of(a[11], a[0], &s))
    return NULL;
  CALL(((rope_fn)fns[ROPE])(p[0], p[1], p[2], p[3], eps, p[4], p[5], factor, pairs, p[6], p[7], s));
}

/* q, k, v, q_weight, k_weight, eps, positions, rope, rope_factor, interleaved, kv_cache,
 * block_table, seq_lens, cu_tokens, page_size, q_out, stream */
static PyObject* rope_append(PyObject* self, PyObject* const* a, Py_ssize_t n) {
  static const int at[12] = {0, 1, 2, 3, 4, 6, 7, 10, 11, 12, 13, 15};
  pkv_tensor d[12];
  const pkv_tensor* p[12];
  int pairs, page;
  float eps, factor;
  void* s;
  if (count_args(n, 17) || describe_all(a, at, 12, d, p) || float_of(a[5], &eps) ||
      float_of(a[8], &factor) || int_of(a[9], &pairs) || int_of(a[14], &page) ||
      stream_of(a[16], a[0], &s))
    return NULL;
  CALL(((rope_append_fn)fns[ROPE_APPEND])(p[0], p[1], p[2], p[3], p[4], eps, p[5], p[6], factor,
                                          pairs, p[7], p[8], p[9], p[10], page, p[11], s));
}

/* bind(addresses in the order of the enum, torch dtypes of codes 1..4, current stream of a
 * device index, exception type) */
static PyObject* bind(PyObject* self, PyObject* args) {
  PyObject *addresses, *types, *stream, *error;
  if (!PyArg_ParseTuple(args, "O!O!OO", &PyTuple_Type, &addresses, &PyTuple_Type, &types, &stream,
                        &error))
    return NULL;
  if (PyTuple_GET_SIZE(addresses) != NUM_FNS || PyTuple_GET_SIZE(types) != 4) {
    PyErr_SetString(PyExc_ValueError, "bind: wrong number of entry points or dtypes");
    return NULL;
  }
  for (int i = 0; i < NUM_FNS; ++i) {
    fns[i] = PyLong_AsVoidPtr(PyTuple_GET_ITEM(addresses, i));
    if (!fns[i]) {
      fns[0] = NULL;
      if (!PyErr_Occurred()) PyErr_SetString(PyExc_ValueError, "bind: a NULL entry point");
      return NULL;
    }
  }
  for (int i = 0; i < 4; ++i) Py_XSETREF(dtypes[i + 1], Py_NewRef(PyTuple_GET_ITEM(types, i)));
  Py_XSETREF(raw_stream, Py_NewRef(stream));
  Py_XSETREF(error_type, Py_NewRef(error));
  Py_RETURN_NONE;
}

#define METHOD(name, fn) {name, (PyCFunction)(void (*)(void))fn, METH_FASTCALL, NULL}
static PyMethodDef methods[] = {
    {"bind", bind, METH_VARARGS, NULL},
    METHOD("paged_decode_attn_fp8", attn8),
    METHOD("paged_window_attn", window_attn),
    METHOD("gqa_kv_append_fp8", append),
    METHOD("pages_fork", fork_rows),
    METHOD("pages_release", release),
    METHOD("pages_reserve", reserve),
    METHOD("pages_compact", compact),
    METHOD("pages_copy", copy),
    METHOD("pages_trim", trim),
    METHOD("paged_prefix_attn_fp8", prefix8),
    METHOD("paged_prefix_attn", prefix),
    METHOD("qk_norm_rope", rope),
    METHOD("gqa_rope_append", rope_append),
    {NULL, NULL, 0, NULL}};

static struct PyModuleDef module = {PyModuleDef_HEAD_INIT, "_pkvcall", NULL, -1, methods};

PyMODINIT_FUNC PyInit__pkvcall(void) {
  n_data_ptr = PyUnicode_InternFromString("data_ptr");
  n_shape = PyUnicode_InternFromString("shape");
  n_stride = PyUnicode_InternFromString("stride");
  n_dtype = PyUnicode_InternFromString("dtype");
  n_get_device = PyUnicode_InternFromString("get_device");
  n_cuda_stream = PyUnicode_InternFromString("cuda_stream");
  if (!n_data_ptr || !n_shape || !n_stride || !n_dtype || !n_get_device || !n_cuda_stream) return NULL;
  return PyModule_Create(&module);
}
