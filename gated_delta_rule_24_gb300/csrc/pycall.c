// The Python side of the operators whose smallest calls take a few microseconds on the GPU:
// reads the tensors' descriptors and calls the C entry point, which is bound by address.  One token's norm
// and rotation (eight tensors, outputs given) then takes the host 5.6 us, launch included, where it took
// 10.7 with ctypes and struct.
#define PY_SSIZE_T_CLEAN
#include <Python.h>
#include <string.h>

#include "gdn.h"

typedef gdn_status_t (*rope_fn)(const gdn_tensor_t*, const gdn_tensor_t*, const gdn_tensor_t*, const gdn_tensor_t*, float, float,
                                const gdn_tensor_t*, const gdn_tensor_t*, int, const gdn_tensor_t*, const gdn_tensor_t*,
                                cudaStream_t);
typedef gdn_status_t (*prefill_fn)(const gdn_tensor_t*, const gdn_tensor_t*, const gdn_tensor_t*, const gdn_tensor_t*, float,
                                   const gdn_tensor_t*, const gdn_tensor_t*, const gdn_tensor_t*, const gdn_tensor_t*, int,
                                   const gdn_tensor_t*, cudaStream_t);
typedef gdn_status_t (*step_fn)(const gdn_tensor_t*, const gdn_tensor_t*, const gdn_tensor_t*, const gdn_tensor_t*, float,
                                const gdn_tensor_t*, const gdn_tensor_t*, const gdn_tensor_t*, cudaStream_t);
typedef gdn_status_t (*axes_fn)(const gdn_tensor_t*, const gdn_tensor_t*, const gdn_tensor_t*, const gdn_tensor_t*, float, float,
                                const gdn_tensor_t*, const gdn_tensor_t*, const int32_t*, int, int, const gdn_tensor_t*,
                                const gdn_tensor_t*, cudaStream_t);
typedef gdn_status_t (*append_fn)(const gdn_tensor_t*, const gdn_tensor_t*, const gdn_tensor_t*, const gdn_tensor_t*,
                                  const gdn_tensor_t*, float, float, int, const gdn_tensor_t*, const gdn_tensor_t*, const int32_t*,
                                  int, int, const gdn_tensor_t*, const gdn_tensor_t*, const gdn_tensor_t*, const gdn_tensor_t*,
                                  cudaStream_t);
typedef gdn_status_t (*attend_fn)(const gdn_tensor_t*, const gdn_tensor_t*, const gdn_tensor_t*, const gdn_tensor_t*,
                                  const gdn_tensor_t*, float, const gdn_tensor_t*, int64_t, const gdn_tensor_t*, const gdn_tensor_t*,
                                  cudaStream_t);
static rope_fn f_rope;
static prefill_fn f_prefill;
static step_fn f_step;
static axes_fn f_axes;
static append_fn f_append;
static attend_fn f_attend;
static PyObject *n_shape, *n_stride, *n_dtype, *n_data_ptr, *n_is_cuda;
static PyObject* dtypes;  // {torch dtype: its code}
static PyObject* on_host; // called with a tensor that is not the GPU's: raises where that is an error (or None: never asked)

#define MOST 12
typedef struct {
  gdn_tensor_t room[MOST];
  const gdn_tensor_t* at[MOST];
} descriptors;

// At most four sizes or strides out of a tuple; -1 with an exception set.
static int read_tuple(PyObject* t, int64_t* to) {
  const Py_ssize_t n = PyTuple_GET_SIZE(t);
  for (Py_ssize_t i = 0; i < n && i < 4; ++i) {
    to[i] = PyLong_AsLongLong(PyTuple_GET_ITEM(t, i));
    if (to[i] == -1 && PyErr_Occurred()) return -1;
  }
  return (int)n;
}

static int describe(PyObject* t, gdn_tensor_t* d) {
  memset(d, 0, sizeof(*d));
  PyObject* x = PyObject_GetAttr(t, n_shape);
  if (!x) return -1;
  int n = PyTuple_Check(x) ? read_tuple(x, d->shape) : -1;
  Py_DECREF(x);
  if (n > 4) PyErr_SetString(PyExc_ValueError, "at most 4 dims");
  if (n < 0 && !PyErr_Occurred()) PyErr_SetString(PyExc_TypeError, "a tensor is wanted");
  if (n < 0 || n > 4) return -1;
  d->ndim = n;
  x = PyObject_GetAttr(t, n_dtype);
  if (!x) return -1;
  PyObject* code = PyDict_GetItemWithError(dtypes, x);
  if (!code && !PyErr_Occurred()) PyErr_Format(PyExc_TypeError, "unsupported dtype %S", x);
  Py_DECREF(x);
  if (!code) return -1;
  d->dtype = (gdn_dtype_t)PyLong_AsLong(code);
  x = PyObject_CallMethodNoArgs(t, n_stride);
  if (!x) return -1;
  n = PyTuple_Check(x) ? read_tuple(x, d->stride) : -1;
  Py_DECREF(x);
  if (n != d->ndim) {
    if (!PyErr_Occurred()) PyErr_SetString(PyExc_TypeError, "a tensor is wanted");
    return -1;
  }
  x = PyObject_CallMethodNoArgs(t, n_data_ptr);
  if (!x) return -1;
  d->data = PyLong_AsVoidPtr(x);
  Py_DECREF(x);
  return PyErr_Occurred() ? -1 : 0;
}

// 0 where the GPU may read the tensor; -1 with an exception set.
static int check_place(PyObject* t) {
  if (on_host == Py_None) return 0;
  PyObject* x = PyObject_GetAttr(t, n_is_cuda);
  if (!x) return -1;
  Py_DECREF(x);
  if (x == Py_True) return 0;
  x = PyObject_CallOneArg(on_host, t);
  Py_XDECREF(x);
  return x ? 0 : -1;
}

static int describe_all(descriptors* d, PyObject* const* t, int first, int n) {
  for (int i = first; i < first + n; ++i) {
    d->at[i] = t[i - first] == Py_None ? NULL : &d->room[i];
    if (d->at[i] && (describe(t[i - first], &d->room[i]) || check_place(t[i - first]))) return -1;
  }
  return 0;
}
// A gate of one dimension is one decay for each head: the rows of q with a stride of 0.
static void gate_rows(descriptors* d) {
  if (!d->at[0] || !d->at[3] || d->at[3]->ndim != 1) return;
  gdn_tensor_t* g = &d->room[3];
  g->ndim = 2;
  g->shape[1] = g->shape[0];
  g->stride[1] = g->stride[0];
  g->shape[0] = d->at[0]->shape[0];
  g->stride[0] = 0;
}
static int wants(Py_ssize_t n, Py_ssize_t want, const void* fn) {
  if (n != want) PyErr_Format(PyExc_TypeError, "%zd arguments are wanted, got %zd", want, n);
  else if (!fn) PyErr_SetString(PyExc_RuntimeError, "the library is not bound");
  return n == want && fn ? 0 : -1;
}

#define MOST_PAIRS 64
// The axes of the pairs, a sequence of integers; -1 with an exception set.
static int read_axes(PyObject* o, int32_t* to) {
  PyObject* f = PySequence_Fast(o, "pair_axes is a sequence of integers");
  if (!f) return -1;
  const Py_ssize_t n = PySequence_Fast_GET_SIZE(f);
  if (n > MOST_PAIRS) PyErr_Format(PyExc_ValueError, "at most %d pair_axes", MOST_PAIRS);
  for (Py_ssize_t i = 0; i < n && !PyErr_Occurred(); ++i) {
    const long x = PyLong_AsLong(PySequence_Fast_GET_ITEM(f, i));
    to[i] = x < -1 || x > 127 ? -1 : (int32_t)x;   // no axis either way
  }
  Py_DECREF(f);
  return PyErr_Occurred() ? -1 : (int)n;
}

// The arguments are those of the C functions, in their order (without num_pairs: it is the length of pair_axes); then,
// for the prefill and the step, whether a gate may be [H].
static PyObject* qk_norm_rope(PyObject* self, PyObject* const* a, Py_ssize_t n) {
  descriptors d;
  if (wants(n, 12, f_rope) || describe_all(&d, a, 0, 4) || describe_all(&d, a + 6, 4, 2) || describe_all(&d, a + 9, 6, 2)) return NULL;
  const float offset = (float)PyFloat_AsDouble(a[4]), eps = (float)PyFloat_AsDouble(a[5]);
  const int interleaved = PyObject_IsTrue(a[8]);
  cudaStream_t stream = (cudaStream_t)PyLong_AsVoidPtr(a[11]);
  if (PyErr_Occurred()) return NULL;
  gdn_status_t st;
  Py_BEGIN_ALLOW_THREADS
  st = f_rope(d.at[0], d.at[1], d.at[2], d.at[3], offset, eps, d.at[4], d.at[5], interleaved, d.at[6], d.at[7], stream);
  Py_END_ALLOW_THREADS
  return PyLong_FromLong((long)st);
}

static PyObject* decay_prefill(PyObject* self, PyObject* const* a, Py_ssize_t n) {
  descriptors d;
  if (wants(n, 13, f_prefill) || describe_all(&d, a, 0, 4) || describe_all(&d, a + 5, 4, 4) || describe_all(&d, a + 10, 8, 1)) return NULL;
  if (a[12] == Py_True) gate_rows(&d);
  const float scale = (float)PyFloat_AsDouble(a[4]);
  const int invariant = PyObject_IsTrue(a[9]);
  cudaStream_t stream = (cudaStream_t)PyLong_AsVoidPtr(a[11]);
  if (PyErr_Occurred()) return NULL;
  gdn_status_t st;
  Py_BEGIN_ALLOW_THREADS
  st = f_prefill(d.at[0], d.at[1], d.at[2], d.at[3], scale, d.at[4], d.at[5], d.at[6], d.at[7], invariant, d.at[8], stream);
  Py_END_ALLOW_THREADS
  return PyLong_FromLong((long)st);
}

static PyObject* decay_step(PyObject* self, PyObject* const* a, Py_ssize_t n) {
  descriptors d;
  if (wants(n, 10, f_step) || describe_all(&d, a, 0, 4) || describe_all(&d, a + 5, 4, 3)) return NULL;
  if (a[9] == Py_True) gate_rows(&d);
  const float scale = (float)PyFloat_AsDouble(a[4]);
  cudaStream_t stream = (cudaStream_t)PyLong_AsVoidPtr(a[8]);
  if (PyErr_Occurred()) return NULL;
  gdn_status_t st;
  Py_BEGIN_ALLOW_THREADS
  st = f_step(d.at[0], d.at[1], d.at[2], d.at[3], scale, d.at[4], d.at[5], d.at[6], stream);
  Py_END_ALLOW_THREADS
  return PyLong_FromLong((long)st);
}

static PyObject* qk_norm_rope_axes(PyObject* self, PyObject* const* a, Py_ssize_t n) {
  descriptors d;
  int32_t axes[MOST_PAIRS];
  if (wants(n, 13, f_axes) || describe_all(&d, a, 0, 4) || describe_all(&d, a + 6, 4, 2) || describe_all(&d, a + 10, 6, 2)) return NULL;
  const float offset = (float)PyFloat_AsDouble(a[4]), eps = (float)PyFloat_AsDouble(a[5]);
  const int pairs = read_axes(a[8], axes), interleaved = PyObject_IsTrue(a[9]);
  cudaStream_t stream = (cudaStream_t)PyLong_AsVoidPtr(a[12]);
  if (PyErr_Occurred()) return NULL;
  gdn_status_t st;
  Py_BEGIN_ALLOW_THREADS
  st = f_axes(d.at[0], d.at[1], d.at[2], d.at[3], offset, eps, d.at[4], d.at[5], axes, pairs, interleaved, d.at[6], d.at[7], stream);
  Py_END_ALLOW_THREADS
  return PyLong_FromLong((long)st);
}

static PyObject* norm_rope_append(PyObject* self, PyObject* const* a, Py_ssize_t n) {
  descriptors d;
  int32_t axes[MOST_PAIRS];
  if (wants(n, 17, f_append) || describe_all(&d, a, 0, 5) || describe_all(&d, a + 8, 5, 2) || describe_all(&d, a + 12, 7, 4)) return NULL;
  const float offset = (float)PyFloat_AsDouble(a[5]), eps = (float)PyFloat_AsDouble(a[6]);
  const int norm = PyObject_IsTrue(a[7]), pairs = a[10] == Py_None ? 0 : read_axes(a[10], axes), interleaved = PyObject_IsTrue(a[11]);
  cudaStream_t stream = (cudaStream_t)PyLong_AsVoidPtr(a[16]);
  if (PyErr_Occurred()) return NULL;
  gdn_status_t st;
  Py_BEGIN_ALLOW_THREADS
  st = f_append(d.at[0], d.at[1], d.at[2], d.at[3], d.at[4], offset, eps, norm, d.at[5], d.at[6], a[10] == Py_None ? NULL : axes, pairs,
                interleaved, d.at[7], d.at[8], d.at[9], d.at[10], stream);
  Py_END_ALLOW_THREADS
  return PyLong_FromLong((long)st);
}

static PyObject* paged_attention_step(PyObject* self, PyObject* const* a, Py_ssize_t n) {
  descriptors d;
  if (wants(n, 11, f_attend) || describe_all(&d, a, 0, 5) || describe_all(&d, a + 6, 5, 1) || describe_all(&d, a + 8, 6, 2)) return NULL;
  const float scale = (float)PyFloat_AsDouble(a[5]);
  const int64_t prefix = PyLong_AsLongLong(a[7]);
  cudaStream_t stream = (cudaStream_t)PyLong_AsVoidPtr(a[10]);
  if (PyErr_Occurred()) return NULL;
  gdn_status_t st;
  Py_BEGIN_ALLOW_THREADS
  st = f_attend(d.at[0], d.at[1], d.at[2], d.at[3], d.at[4], scale, d.at[5], prefix, d.at[6], d.at[7], stream);
  Py_END_ALLOW_THREADS
  return PyLong_FromLong((long)st);
}

// fill(*tensors): addresses of their descriptors, good until the thread's next call (tests compare them).
static PyObject* fill(PyObject* self, PyObject* const* a, Py_ssize_t n) {
  static _Thread_local descriptors d;
  if (n > MOST) return PyErr_Format(PyExc_ValueError, "at most %d tensors", MOST);
  for (Py_ssize_t i = 0; i < n; ++i) {
    d.at[i] = a[i] == Py_None ? NULL : &d.room[i];
    if (d.at[i] && describe(a[i], &d.room[i])) return NULL;
  }
  PyObject* out = PyList_New(n);
  for (Py_ssize_t i = 0; out && i < n; ++i) {
    PyObject* x = d.at[i] ? PyLong_FromVoidPtr((void*)d.at[i]) : Py_NewRef(Py_None);
    if (!x) { Py_DECREF(out); return NULL; }
    PyList_SET_ITEM(out, i, x);
  }
  return out;
}

// bind({dtype: code}, on_host, then the functions by address): gdn_qk_norm_rope, gdn_decay_prefill, gdn_decay_step,
// gdn_qk_norm_rope_axes, gdn_norm_rope_append, gdn_paged_attention_step.
static PyObject* bind(PyObject* self, PyObject* args) {
  PyObject *d, *host, *f[6];
  if (!PyArg_ParseTuple(args, "O!OOOOOOO", &PyDict_Type, &d, &host, &f[0], &f[1], &f[2], &f[3], &f[4], &f[5])) return NULL;
  f_rope = (rope_fn)PyLong_AsVoidPtr(f[0]);
  f_prefill = (prefill_fn)PyLong_AsVoidPtr(f[1]);
  f_step = (step_fn)PyLong_AsVoidPtr(f[2]);
  f_axes = (axes_fn)PyLong_AsVoidPtr(f[3]);
  f_append = (append_fn)PyLong_AsVoidPtr(f[4]);
  f_attend = (attend_fn)PyLong_AsVoidPtr(f[5]);
  Py_XSETREF(dtypes, Py_NewRef(d));
  Py_XSETREF(on_host, Py_NewRef(host));
  if (PyErr_Occurred()) return NULL;
  Py_RETURN_NONE;
}

static PyMethodDef methods[] = {{"qk_norm_rope", (PyCFunction)(void (*)(void))qk_norm_rope, METH_FASTCALL, NULL},
                                {"decay_prefill", (PyCFunction)(void (*)(void))decay_prefill, METH_FASTCALL, NULL},
                                {"decay_step", (PyCFunction)(void (*)(void))decay_step, METH_FASTCALL, NULL},
                                {"qk_norm_rope_axes", (PyCFunction)(void (*)(void))qk_norm_rope_axes, METH_FASTCALL, NULL},
                                {"norm_rope_append", (PyCFunction)(void (*)(void))norm_rope_append, METH_FASTCALL, NULL},
                                {"paged_attention_step", (PyCFunction)(void (*)(void))paged_attention_step, METH_FASTCALL, NULL},
                                {"fill", (PyCFunction)(void (*)(void))fill, METH_FASTCALL, NULL},
                                {"bind", bind, METH_VARARGS, NULL},
                                {NULL, NULL, 0, NULL}};
static struct PyModuleDef module = {PyModuleDef_HEAD_INIT, "gdn_pycall", NULL, -1, methods, NULL, NULL, NULL, NULL};
PyMODINIT_FUNC PyInit_gdn_pycall(void) {
  n_shape = PyUnicode_InternFromString("shape");
  n_stride = PyUnicode_InternFromString("stride");
  n_dtype = PyUnicode_InternFromString("dtype");
  n_data_ptr = PyUnicode_InternFromString("data_ptr");
  n_is_cuda = PyUnicode_InternFromString("is_cuda");
  dtypes = PyDict_New();
  on_host = Py_NewRef(Py_None);
  if (!n_shape || !n_stride || !n_dtype || !n_data_ptr || !n_is_cuda || !dtypes) return NULL;
  return PyModule_Create(&module);
}
