// The Python side of the operators whose smallest calls take a few microseconds on the GPU: reads the tensors
// without a Python object for each of their properties, allocates results where it is asked to, and calls the C entry point, which
// is bound by address.  Between two launches every Python-level step costs more than it does by itself (the driver's code
// has taken the caches): an append of one token with a new result takes the host 12.8 us with descriptors read from attributes and
// results from torch.empty_like, 6.4 here.
#include <ATen/ATen.h>
#include <c10/cuda/CUDAFunctions.h>
#include <c10/cuda/CUDAStream.h>
#include <torch/csrc/autograd/python_variable.h>

#include <exception>

#include "gdn.h"

namespace {

decltype(&gdn_qk_norm_rope) f_rope;
decltype(&gdn_decay_prefill) f_prefill;
decltype(&gdn_decay_step) f_step;
decltype(&gdn_qk_norm_rope_axes) f_axes;
decltype(&gdn_norm_rope_append) f_append;
decltype(&gdn_paged_attention_step) f_attend;
PyObject* not_here;  // called with a tensor that the current GPU may not read or write: raises where that is an error (or None: never asked)

constexpr int kMost = 12;
struct Descriptors {
  gdn_tensor_t room[kMost];
  const gdn_tensor_t* at[kMost];
  int device = -2;  // the current one, once asked
};

// What stands for a Python exception that is set.
struct Raised {};

const at::Tensor& tensor_of(PyObject* o) {
  if (!THPVariable_Check(o)) {
    PyErr_Format(PyExc_AttributeError, "'%s' object has no attribute 'shape': a tensor is wanted", Py_TYPE(o)->tp_name);
    throw Raised();
  }
  return THPVariable_Unpack(o);
}

void describe(const at::Tensor& t, gdn_tensor_t* d) {
  switch (t.scalar_type()) {
    case at::kFloat: d->dtype = GDN_F32; break;
    case at::kBFloat16: d->dtype = GDN_BF16; break;
    case at::kHalf: d->dtype = GDN_F16; break;
    case at::kInt: d->dtype = GDN_I32; break;
    case at::kLong: d->dtype = GDN_I64; break;
    default:
      PyErr_Format(PyExc_TypeError, "unsupported dtype %s", c10::toString(t.scalar_type()));
      throw Raised();
  }
  const auto sizes = t.sizes(), strides = t.strides();
  if (sizes.size() > 4) {
    PyErr_SetString(PyExc_ValueError, "at most 4 dims");
    throw Raised();
  }
  d->ndim = (int32_t)sizes.size();
  for (size_t i = 0; i < 4; ++i) {
    d->shape[i] = i < sizes.size() ? sizes[i] : 0;
    d->stride[i] = i < sizes.size() ? strides[i] : 0;
  }
  d->data = t.data_ptr();
}

// Asks about a tensor, an argument or a new result, that the current GPU may not read or write.
void ask(Descriptors& d, const at::Tensor& x) {
  if (not_here == Py_None) return;
  if (x.is_cuda()) {
    if (d.device == -2) d.device = c10::cuda::current_device();
    if (x.get_device() == d.device) return;
  }
  PyObject* o = THPVariable_Wrap(x);
  PyObject* r = o ? PyObject_CallOneArg(not_here, o) : nullptr;
  Py_XDECREF(o);
  if (!r) throw Raised();
  Py_DECREF(r);
}
// Descriptors first .. first + n - 1 of the tensors t[0 .. n - 1], none for None.
void describe_all(Descriptors& d, PyObject* const* t, int first, int n) {
  for (int i = first; i < first + n; ++i) {
    d.at[i] = nullptr;
    if (t[i - first] == Py_None) continue;
    const at::Tensor& x = tensor_of(t[i - first]);
    describe(x, &d.room[i]);
    d.at[i] = &d.room[i];
    ask(d, x);
  }
}
// A gate of one dimension is one decay for each head: the rows of q with a stride of 0.
void gate_rows(Descriptors& d) {
  if (!d.at[0] || !d.at[3] || d.at[3]->ndim != 1) return;
  gdn_tensor_t* g = &d.room[3];
  g->ndim = 2;
  g->shape[1] = g->shape[0];
  g->stride[1] = g->stride[0];
  g->shape[0] = d.at[0]->shape[0];
  g->stride[0] = 0;
}
void wants(Py_ssize_t n, Py_ssize_t want, bool bound) {
  if (n == want && bound) return;
  if (n != want) PyErr_Format(PyExc_TypeError, "%zd arguments are wanted, got %zd", want, n);
  else PyErr_SetString(PyExc_RuntimeError, "the library is not bound");
  throw Raised();
}
double real(PyObject* o) {
  const double x = PyFloat_AsDouble(o);
  if (x == -1.0 && PyErr_Occurred()) throw Raised();
  return x;
}
bool truth(PyObject* o) {
  const int x = PyObject_IsTrue(o);
  if (x < 0) throw Raised();
  return x != 0;
}
int64_t integer(PyObject* o) {
  const long long x = PyLong_AsLongLong(o);
  if (x == -1 && PyErr_Occurred()) throw Raised();
  return x;
}
cudaStream_t stream_of(PyObject* o) {
  void* x = PyLong_AsVoidPtr(o);
  if (!x && PyErr_Occurred()) throw Raised();
  return static_cast<cudaStream_t>(x);
}
cudaStream_t current_stream() { return c10::cuda::getCurrentCUDAStream().stream(); }

// The axes of the pairs, a sequence of integers or None.
struct Axes {
  static constexpr int kMostPairs = 64;
  int32_t at[kMostPairs];
  int n = 0;
  bool none;
  explicit Axes(PyObject* o) : none(o == Py_None) {
    if (none) return;
    PyObject* f = PySequence_Fast(o, "pair_axes is a sequence of integers");
    if (!f) throw Raised();
    const Py_ssize_t count = PySequence_Fast_GET_SIZE(f);
    if (count > kMostPairs) PyErr_Format(PyExc_ValueError, "at most %d pair_axes", kMostPairs);
    for (Py_ssize_t i = 0; i < count && !PyErr_Occurred(); ++i) {
      const long long x = PyLong_AsLongLong(PySequence_Fast_GET_ITEM(f, i));
      at[i] = x < 0 || x > 127 ? -1 : (int32_t)x;   // no axis either way
    }
    Py_DECREF(f);
    if (PyErr_Occurred()) throw Raised();
    n = (int)count;
  }
  const int32_t* data() const { return none ? nullptr : at; }
};

// The call itself, without the interpreter's lock.
template <typename Call>
gdn_status_t apart(Call call) {
  gdn_status_t st;
  Py_BEGIN_ALLOW_THREADS
  st = call();
  Py_END_ALLOW_THREADS
  return st;
}
PyObject* status(gdn_status_t st) { return PyLong_FromLong((long)st); }
// Two objects (references given away) as a tuple, None in the place of none.
PyObject* two(PyObject* a, PyObject* b) {
  if (!b) b = Py_NewRef(Py_None);
  PyObject* t = a ? PyTuple_New(2) : nullptr;
  if (!t) {
    Py_XDECREF(a);
    Py_DECREF(b);
    return nullptr;
  }
  PyTuple_SET_ITEM(t, 0, a);
  PyTuple_SET_ITEM(t, 1, b);
  return t;
}
at::Tensor like(const at::Tensor& q, bool rows = false) {  // rows: contiguous whatever the order of q in memory
  return rows ? at::empty(q.sizes(), q.options().requires_grad(false)) : at::empty_like(q, q.options().requires_grad(false));
}
// A result made after an argument that is allowed in pinned memory would lie in ordinary host memory.
void describe_new(Descriptors& d, int i, const at::Tensor& t) {
  describe(t, &d.room[i]);
  d.at[i] = &d.room[i];
  ask(d, t);
}

// A function of the module: what it throws becomes a Python exception.
template <PyObject* (*kBody)(PyObject* const*, Py_ssize_t)>
PyObject* guarded(PyObject*, PyObject* const* a, Py_ssize_t n) {
  try {
    return kBody(a, n);
  } catch (const Raised&) {
  } catch (const std::exception& e) {
    PyErr_SetString(PyExc_RuntimeError, e.what());
  } catch (...) {
    PyErr_SetString(PyExc_RuntimeError, "an exception of no kind");
  }
  return nullptr;
}

// The arguments are those of the C functions, in their order (without num_pairs: it is the length of pair_axes); then,
// for the prefill and the step, whether a gate may be [H].  They return the status.
PyObject* qk_norm_rope(PyObject* const* a, Py_ssize_t n) {
  wants(n, 12, f_rope);
  Descriptors d;
  describe_all(d, a, 0, 4);
  describe_all(d, a + 6, 4, 2);
  describe_all(d, a + 9, 6, 2);
  const float offset = (float)real(a[4]), eps = (float)real(a[5]);
  const bool interleaved = truth(a[8]);
  cudaStream_t stream = stream_of(a[11]);
  return status(apart([&] { return f_rope(d.at[0], d.at[1], d.at[2], d.at[3], offset, eps, d.at[4], d.at[5], interleaved, d.at[6], d.at[7], stream); }));
}

PyObject* decay_prefill(PyObject* const* a, Py_ssize_t n) {
  wants(n, 13, f_prefill);
  Descriptors d;
  describe_all(d, a, 0, 4);
  describe_all(d, a + 5, 4, 4);
  describe_all(d, a + 10, 8, 1);
  if (a[12] == Py_True) gate_rows(d);
  const float scale = (float)real(a[4]);
  const bool invariant = truth(a[9]);
  cudaStream_t stream = stream_of(a[11]);
  return status(apart([&] { return f_prefill(d.at[0], d.at[1], d.at[2], d.at[3], scale, d.at[4], d.at[5], d.at[6], d.at[7], invariant, d.at[8], stream); }));
}

PyObject* decay_step(PyObject* const* a, Py_ssize_t n) {
  wants(n, 10, f_step);
  Descriptors d;
  describe_all(d, a, 0, 4);
  describe_all(d, a + 5, 4, 3);
  if (a[9] == Py_True) gate_rows(d);
  const float scale = (float)real(a[4]);
  cudaStream_t stream = stream_of(a[8]);
  return status(apart([&] { return f_step(d.at[0], d.at[1], d.at[2], d.at[3], scale, d.at[4], d.at[5], d.at[6], stream); }));
}

PyObject* qk_norm_rope_axes(PyObject* const* a, Py_ssize_t n) {
  wants(n, 13, f_axes);
  Descriptors d;
  describe_all(d, a, 0, 4);
  describe_all(d, a + 6, 4, 2);
  describe_all(d, a + 10, 6, 2);
  const float offset = (float)real(a[4]), eps = (float)real(a[5]);
  const Axes axes(a[8]);
  const bool interleaved = truth(a[9]);
  cudaStream_t stream = stream_of(a[12]);
  return status(apart([&] { return f_axes(d.at[0], d.at[1], d.at[2], d.at[3], offset, eps, d.at[4], d.at[5], axes.data(), axes.n, interleaved, d.at[6], d.at[7], stream); }));
}

PyObject* norm_rope_append(PyObject* const* a, Py_ssize_t n) {
  wants(n, 17, f_append);
  Descriptors d;
  describe_all(d, a, 0, 5);
  describe_all(d, a + 8, 5, 2);
  describe_all(d, a + 12, 7, 4);
  const float offset = (float)real(a[5]), eps = (float)real(a[6]);
  const bool norm = truth(a[7]), interleaved = truth(a[11]);
  const Axes axes(a[10]);
  cudaStream_t stream = stream_of(a[16]);
  return status(apart([&] {
    return f_append(d.at[0], d.at[1], d.at[2], d.at[3], d.at[4], offset, eps, norm, d.at[5], d.at[6], axes.data(), axes.n, interleaved,
                    d.at[7], d.at[8], d.at[9], d.at[10], stream);
  }));
}

PyObject* paged_attention_step(PyObject* const* a, Py_ssize_t n) {
  wants(n, 11, f_attend);
  Descriptors d;
  describe_all(d, a, 0, 5);
  describe_all(d, a + 6, 5, 1);
  describe_all(d, a + 8, 6, 2);
  const float scale = (float)real(a[5]);
  const int64_t prefix = integer(a[7]);
  cudaStream_t stream = stream_of(a[10]);
  return status(apart([&] { return f_attend(d.at[0], d.at[1], d.at[2], d.at[3], d.at[4], scale, d.at[5], prefix, d.at[6], d.at[7], stream); }));
}

// The same on the current stream with new results: they return those, or the status where it is not 0.

// q, k, q_weight, k_weight, weight_offset, eps, cos_sin, positions, pair_axes or None, interleaved -> (q_out, k_out)
PyObject* new_qk_norm_rope(PyObject* const* a, Py_ssize_t n) {
  wants(n, 10, f_rope && f_axes);
  Descriptors d;
  describe_all(d, a, 0, 4);
  describe_all(d, a + 6, 4, 2);
  const float offset = (float)real(a[4]), eps = (float)real(a[5]);
  const Axes axes(a[8]);
  const bool interleaved = truth(a[9]);
  at::Tensor q = like(tensor_of(a[0])), k;
  describe_new(d, 6, q);
  d.at[7] = nullptr;
  if (d.at[1]) {
    k = like(tensor_of(a[1]));
    describe_new(d, 7, k);
  }
  cudaStream_t stream = current_stream();
  const gdn_status_t st = apart([&] {
    return axes.none ? f_rope(d.at[0], d.at[1], d.at[2], d.at[3], offset, eps, d.at[4], d.at[5], interleaved, d.at[6], d.at[7], stream)
                     : f_axes(d.at[0], d.at[1], d.at[2], d.at[3], offset, eps, d.at[4], d.at[5], axes.data(), axes.n, interleaved, d.at[6], d.at[7], stream);
  });
  if (st != GDN_OK) return status(st);
  return two(THPVariable_Wrap(q), d.at[1] ? THPVariable_Wrap(k) : nullptr);
}

// q, k, v, q_weight, k_weight, weight_offset, eps, norm, cos_sin, positions, pair_axes or None, interleaved, slots, k_cache, v_cache -> q_out
PyObject* new_norm_rope_append(PyObject* const* a, Py_ssize_t n) {
  wants(n, 15, f_append);
  Descriptors d;
  describe_all(d, a, 0, 5);
  describe_all(d, a + 8, 5, 2);
  describe_all(d, a + 12, 7, 3);
  const float offset = (float)real(a[5]), eps = (float)real(a[6]);
  const bool norm = truth(a[7]), interleaved = truth(a[11]);
  const Axes axes(a[10]);
  const at::Tensor q = like(tensor_of(a[0]));
  describe_new(d, 10, q);
  cudaStream_t stream = current_stream();
  const gdn_status_t st = apart([&] {
    return f_append(d.at[0], d.at[1], d.at[2], d.at[3], d.at[4], offset, eps, norm, d.at[5], d.at[6], axes.data(), axes.n, interleaved,
                    d.at[7], d.at[10], d.at[8], d.at[9], stream);
  });
  return st != GDN_OK ? status(st) : THPVariable_Wrap(q);
}

// q, k_cache, v_cache, page_table, lengths, scale, prefix_pages, prefix_length, whether with lse -> output, or (output, lse)
PyObject* new_paged_attention_step(PyObject* const* a, Py_ssize_t n) {
  wants(n, 9, f_attend);
  Descriptors d;
  describe_all(d, a, 0, 5);
  describe_all(d, a + 6, 5, 1);
  const float scale = (float)real(a[5]);
  const int64_t prefix = integer(a[7]);
  const bool with_lse = truth(a[8]);
  const at::Tensor& q = tensor_of(a[0]);
  const at::Tensor out = like(q, true);
  at::Tensor lse;
  describe_new(d, 6, out);
  d.at[7] = nullptr;
  if (with_lse && q.dim() >= 2) {
    lse = at::empty(q.sizes().slice(0, 2), q.options().dtype(at::kFloat).requires_grad(false));
    describe_new(d, 7, lse);
  }
  cudaStream_t stream = current_stream();
  const gdn_status_t st = apart([&] { return f_attend(d.at[0], d.at[1], d.at[2], d.at[3], d.at[4], scale, d.at[5], prefix, d.at[6], d.at[7], stream); });
  if (st != GDN_OK) return status(st);
  return with_lse ? two(THPVariable_Wrap(out), THPVariable_Wrap(lse)) : THPVariable_Wrap(out);
}

// fill(*tensors): addresses of their descriptors, good until the thread's next call (tests compare them).
PyObject* fill(PyObject* const* a, Py_ssize_t n) {
  static thread_local Descriptors d;
  if (n > kMost) {
    PyErr_Format(PyExc_ValueError, "at most %d tensors", kMost);
    throw Raised();
  }
  for (Py_ssize_t i = 0; i < n; ++i) {
    d.at[i] = a[i] == Py_None ? nullptr : &d.room[i];
    if (d.at[i]) describe(tensor_of(a[i]), &d.room[i]);
  }
  PyObject* out = PyList_New(n);
  for (Py_ssize_t i = 0; out && i < n; ++i) {
    PyObject* x = d.at[i] ? PyLong_FromVoidPtr((void*)d.at[i]) : Py_NewRef(Py_None);
    if (!x) {
      Py_DECREF(out);
      return nullptr;
    }
    PyList_SET_ITEM(out, i, x);
  }
  return out;
}

// bind(not_here, then the functions by address): gdn_qk_norm_rope, gdn_decay_prefill, gdn_decay_step, gdn_qk_norm_rope_axes,
// gdn_norm_rope_append, gdn_paged_attention_step.
PyObject* bind(PyObject* const* a, Py_ssize_t n) {
  wants(n, 7, true);
  void* f[6];
  for (int i = 0; i < 6; ++i) {
    f[i] = PyLong_AsVoidPtr(a[1 + i]);
    if (!f[i] && PyErr_Occurred()) throw Raised();
  }
  f_rope = reinterpret_cast<decltype(f_rope)>(f[0]);
  f_prefill = reinterpret_cast<decltype(f_prefill)>(f[1]);
  f_step = reinterpret_cast<decltype(f_step)>(f[2]);
  f_axes = reinterpret_cast<decltype(f_axes)>(f[3]);
  f_append = reinterpret_cast<decltype(f_append)>(f[4]);
  f_attend = reinterpret_cast<decltype(f_attend)>(f[5]);
  Py_XSETREF(not_here, Py_NewRef(a[0]));
  Py_RETURN_NONE;
}

#define GDN_METHOD(name) {#name, reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(&guarded<name>)), METH_FASTCALL, nullptr}
PyMethodDef methods[] = {GDN_METHOD(qk_norm_rope), GDN_METHOD(decay_prefill), GDN_METHOD(decay_step), GDN_METHOD(qk_norm_rope_axes),
                         GDN_METHOD(norm_rope_append), GDN_METHOD(paged_attention_step), GDN_METHOD(new_qk_norm_rope),
                         GDN_METHOD(new_norm_rope_append), GDN_METHOD(new_paged_attention_step), GDN_METHOD(fill), GDN_METHOD(bind),
                         {nullptr, nullptr, 0, nullptr}};
PyModuleDef module = {PyModuleDef_HEAD_INIT, "gdn_pycall", nullptr, -1, methods, nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit_gdn_pycall(void) {
  not_here = Py_NewRef(Py_None);
  PyObject* m = PyModule_Create(&module);
  // the torch and the Python whose objects are read here, for the binding to compare before it makes a call
  if (m && PyModule_AddStringConstant(m, "made_for", GDN_MADE_FOR) < 0) Py_CLEAR(m);
  return m;
}
