// CPython side of the binding's small calls: tensor checks and the call itself.
//
// A small call's time is the host's. The cache write of 64 tokens (a kernel of 3.7 us, eleven tensors, 32
// arguments) takes 14.3 us on the Grace host through Python and ctypes, 9.8 with a tensor's
// attributes asked for here through the object protocol, 6.5 with them read from the tensor; 2.1 of
// that is the launch.
// A torch tensor is read through PyTorch's own headers; any other object that has a tensor's methods, and
// whatever the quick look does not find in order, goes through the object protocol, which also
// words the errors.
#define PY_SSIZE_T_CLEAN
#include <torch/csrc/Dtype.h>
#include <torch/csrc/autograd/python_variable.h>
#include <torch/version.h>

#include <climits>
#include <cstdint>

#include "pkv_attn.h"

static PyObject *s_get_device, *s_is_contiguous, *s_dtype, *s_shape, *s_data_ptr;

// The tensor behind a Python object if it is one on CUDA device `dev`, of that type and shape (None:
// any); null where it is not, or where this look cannot tell.
static const at::Tensor* look(PyObject* t, long dev, PyObject* dtype, PyObject* shape) {
  if (!THPVariable_Check(t)) return nullptr;
  const at::Tensor& x = THPVariable_Unpack(t);
  if (!x.defined() || !x.has_storage() || !x.is_cuda() || x.get_device() != dev) return nullptr;
  if (dtype != Py_None &&
      (!THPDtype_Check(dtype) || reinterpret_cast<THPDtype*>(dtype)->scalar_type != x.scalar_type()))
    return nullptr;
  if (shape != Py_None) {
    if (!PyTuple_Check(shape) || PyTuple_GET_SIZE(shape) != x.dim()) return nullptr;
    const c10::IntArrayRef sizes = x.sizes();
    for (Py_ssize_t i = 0; i < PyTuple_GET_SIZE(shape); ++i) {
      const long long v = PyLong_AsLongLong(PyTuple_GET_ITEM(shape, i));
      if (v == -1 && PyErr_Occurred()) PyErr_Clear();
      if (v != sizes[i]) return nullptr;
    }
  }
  return &x;
}

// need(tensor, name, device, dtype | None, shape | None) -> address of its data.
// The tensor has to be a contiguous CUDA tensor on that device, of that type and shape.
static PyObject* need(PyObject* self, PyObject* const* a, Py_ssize_t n) {
  (void)self;
  if (n != 5) return PyErr_Format(PyExc_TypeError, "need() takes 5 arguments, got %zd", n);
  PyObject *t = a[0], *r;
  const long want = PyLong_AsLong(a[2]);
  if (want == -1 && PyErr_Occurred()) return NULL;
  try {
    const at::Tensor* x = look(t, want, a[3], a[4]);
    if (x && x->is_contiguous()) return PyLong_FromVoidPtr(x->data_ptr());
  } catch (const std::exception&) {  // a tensor without memory of its own: the protocol says what is wrong
  }
  r = PyObject_CallMethodNoArgs(t, s_get_device);
  if (!r) return NULL;
  const long dev = PyLong_AsLong(r);
  Py_DECREF(r);
  if (dev == -1) {
    if (PyErr_Occurred()) return NULL;
    return PyErr_Format(PyExc_ValueError, "%U must be a CUDA tensor", a[1]);
  }
  if (dev != want)
    return PyErr_Format(PyExc_ValueError, "%U is on cuda:%ld, the current device is cuda:%ld", a[1], dev, want);
  r = PyObject_CallMethodNoArgs(t, s_is_contiguous);
  if (!r) return NULL;
  const int contiguous = r == Py_True;
  Py_DECREF(r);
  if (!contiguous) return PyErr_Format(PyExc_ValueError, "%U must be contiguous", a[1]);
  if (a[3] != Py_None) {
    r = PyObject_GetAttr(t, s_dtype);
    if (!r) return NULL;
    if (r != a[3]) {
      PyErr_Format(PyExc_ValueError, "%U must be %S, got %S", a[1], a[3], r);
      Py_DECREF(r);
      return NULL;
    }
    Py_DECREF(r);
  }
  if (a[4] != Py_None) {
    r = PyObject_GetAttr(t, s_shape);
    if (!r) return NULL;
    const int same = PyObject_RichCompareBool(r, a[4], Py_EQ);
    if (same != 1) {
      if (same == 0) {
        PyObject* got = PySequence_Tuple(r);
        if (got) PyErr_Format(PyExc_ValueError, "%U has shape %R, expected %R", a[1], got, a[4]);
        Py_XDECREF(got);
      }
      Py_DECREF(r);
      return NULL;
    }
    Py_DECREF(r);
  }
  return PyObject_CallMethodNoArgs(t, s_data_ptr);
}

// rows(tensor, device, dtype, (B, C, H, D)) -> (address of its data, elements from one token to the next),
// where each token's heads lie contiguously at one distance per token; None where that does not hold.
static PyObject* rows(PyObject* self, PyObject* const* a, Py_ssize_t n) {
  (void)self;
  if (n != 4) return PyErr_Format(PyExc_TypeError, "rows() takes 4 arguments, got %zd", n);
  const long dev = PyLong_AsLong(a[1]);
  if (dev == -1 && PyErr_Occurred()) return NULL;
  try {
    const at::Tensor* x = look(a[0], dev, a[2], a[3]);
    if (x && x->dim() == 4) {
      const int64_t B = x->size(0), C = x->size(1), H = x->size(2), D = x->size(3);
      const int64_t sb = x->stride(0), sc = x->stride(1);
      if ((x->stride(3) == 1 || D == 1) && (x->stride(2) == D || H == 1) && (sb == C * sc || B == 1 || C == 1))
        return Py_BuildValue("(NL)", PyLong_FromVoidPtr(x->data_ptr()), (long long)(C > 1 ? sc : B > 1 ? sb : H * D));
    }
  } catch (const std::exception&) {
  }
  Py_RETURN_NONE;
}

// Raw arguments: addresses (int or None), integers and floats, as many as the call takes.
static int raw(PyObject* const* a, Py_ssize_t n, Py_ssize_t want, const char* name) {
  if (n != want) {
    PyErr_Format(PyExc_TypeError, "%s() takes %zd arguments, got %zd", name, want, n);
    return 0;
  }
  for (Py_ssize_t i = 0; i < n; ++i) {
    if (a[i] == Py_None || PyFloat_Check(a[i])) continue;
    if (!PyLong_Check(a[i])) {
      PyErr_Format(PyExc_TypeError, "%s() argument %zd is a %s", name, i, Py_TYPE(a[i])->tp_name);
      return 0;
    }
    if (PyLong_AsLongLong(a[i]) == -1 && PyErr_Occurred()) return 0;
  }
  return 1;
}
static void* ptr_of(PyObject* o) { return PyLong_Check(o) ? (void*)(intptr_t)PyLong_AsLongLong(o) : NULL; }
// A size past 32 bits must not wrap into a valid one: INT_MIN is refused by every call.
static int int_of(PyObject* o) {
  if (!PyLong_Check(o)) return INT_MIN;
  const long long v = PyLong_AsLongLong(o);
  return v < INT_MIN || v > INT_MAX ? INT_MIN : (int)v;
}
static float float_of(PyObject* o) {
  return PyFloat_Check(o) ? (float)PyFloat_AS_DOUBLE(o) : PyLong_Check(o) ? (float)PyLong_AsLongLong(o) : 0.0f;
}

#define PTR(i) address{ptr_of(a[i])}
#define INT(i) int_of(a[i])
#define I64(i) (PyLong_Check(a[i]) ? (int64_t)PyLong_AsLongLong(a[i]) : INT64_MIN)
#define FLT(i) float_of(a[i])
// A wrapper takes the arguments with the interpreter lock held and makes the call without it (a
// launch can wait for room in the stream).
struct address {  // becomes a pointer of the type that the call takes
  void* at;
  template <class T>
  operator T*() const {
    return static_cast<T*>(at);
  }
};
struct args {
  address p[16];
  int64_t l[3];
  float f[2];
  int i[12];
};
#define ENTER(name, count)                                                              \
  static PyObject* py_##name(PyObject* self, PyObject* const* a, Py_ssize_t n) {        \
    (void)self;                                                                         \
    args x = {};                                                                         \
    int status;                                                                         \
    if (!raw(a, n, count, #name)) return NULL;
#define CALL(expression)                 \
  Py_BEGIN_ALLOW_THREADS                 \
  status = expression;                   \
  Py_END_ALLOW_THREADS                   \
  return PyLong_FromLong(status);        \
  }

ENTER(attn_qk_norm_rope_append, 32)
  for (int k = 0; k < 3; ++k) x.p[k] = PTR(k), x.l[k] = I64(3 + k);
  x.p[3] = PTR(6), x.p[4] = PTR(7), x.f[0] = FLT(8), x.p[5] = PTR(9), x.i[0] = INT(10), x.i[1] = INT(11);
  x.p[6] = PTR(12), x.i[2] = INT(13);
  for (int k = 0; k < 7; ++k) x.p[7 + k] = PTR(14 + k);
  for (int k = 0; k < 9; ++k) x.i[3 + k] = INT(21 + k);
  x.p[14] = PTR(30), x.p[15] = PTR(31);
CALL((attn_qk_norm_rope_append(x.p[0], x.p[1], x.p[2], x.l[0], x.l[1], x.l[2], x.p[3], x.p[4], x.f[0], x.p[5], x.i[0],
                               x.i[1], x.p[6], x.i[2], x.p[7], x.p[8], x.p[9], x.p[10], x.p[11], x.p[12], x.p[13],
                               x.i[3], x.i[4], x.i[5], x.i[6], x.i[7], x.i[8], x.i[9], x.i[10], x.i[11], x.p[14],
                               x.p[15])))

ENTER(attn_decode_paged_weights, 24)
  for (int k = 0; k < 9; ++k) x.p[k] = PTR(k);
  for (int k = 0; k < 7; ++k) x.i[k] = INT(9 + k);
  x.f[0] = FLT(16), x.f[1] = FLT(17), x.i[7] = INT(18), x.i[8] = INT(19), x.p[9] = PTR(20);
  const int64_t bytes = I64(21);
  x.p[10] = PTR(22), x.p[11] = PTR(23);
CALL((attn_decode_paged_weights(x.p[0], x.p[1], x.p[2], x.p[3], x.p[4], x.p[5], x.p[6], x.p[7], x.p[8], x.i[0],
                                x.i[1], x.i[2], x.i[3], x.i[4], x.i[5], x.i[6], x.f[0], x.f[1], x.i[7], x.i[8],
                                x.p[9], bytes < 0 ? 0 : (size_t)bytes, x.p[10], x.p[11])))

ENTER(attn_chunk_weights, 22)
  for (int k = 0; k < 8; ++k) x.p[k] = PTR(k);
  for (int k = 0; k < 9; ++k) x.i[k] = INT(8 + k);
  x.f[0] = FLT(17), x.f[1] = FLT(18), x.i[9] = INT(19), x.p[8] = PTR(20), x.p[9] = PTR(21);
CALL((attn_chunk_weights(x.p[0], x.p[1], x.p[2], x.p[3], x.p[4], x.p[5], x.p[6], x.p[7], x.i[0], x.i[1], x.i[2],
                         x.i[3], x.i[4], x.i[5], x.i[6], x.i[7], x.i[8], x.f[0], x.f[1], x.i[9], x.p[8], x.p[9])))

ENTER(attn_cache_evict, 22)
  for (int k = 0; k < 9; ++k) x.p[k] = PTR(k);
  for (int k = 0; k < 11; ++k) x.i[k] = INT(9 + k);
  x.p[9] = PTR(20), x.p[10] = PTR(21);
CALL((attn_cache_evict(x.p[0], x.p[1], x.p[2], x.p[3], x.p[4], x.p[5], x.p[6], x.p[7], x.p[8], x.i[0], x.i[1], x.i[2],
                       x.i[3], x.i[4], x.i[5], x.i[6], x.i[7], x.i[8], x.i[9], x.i[10], x.p[9], x.p[10])))

ENTER(attn_linear, 12)
  for (int k = 0; k < 5; ++k) x.p[k] = PTR(k), x.i[k] = INT(5 + k);
  x.p[5] = PTR(10), x.p[6] = PTR(11);
CALL((attn_linear(x.p[0], x.p[1], x.p[2], x.p[3], x.p[4], x.i[0], x.i[1], x.i[2], x.i[3], x.i[4], x.p[5], x.p[6])))

#define METHOD(name, f) {name, (PyCFunction)(void (*)(void))f, METH_FASTCALL, NULL}
static PyMethodDef methods[] = {
    METHOD("need", need),
    METHOD("rows", rows),
    METHOD("attn_qk_norm_rope_append", py_attn_qk_norm_rope_append),
    METHOD("attn_decode_paged_weights", py_attn_decode_paged_weights),
    METHOD("attn_chunk_weights", py_attn_chunk_weights),
    METHOD("attn_cache_evict", py_attn_cache_evict),
    METHOD("attn_linear", py_attn_linear),
    {NULL, NULL, 0, NULL},
};
static struct PyModuleDef module = {PyModuleDef_HEAD_INIT, "_pycall", NULL, -1, methods, NULL, NULL, NULL, NULL};

PyMODINIT_FUNC PyInit__pycall(void) {
  s_get_device = PyUnicode_InternFromString("get_device");
  s_is_contiguous = PyUnicode_InternFromString("is_contiguous");
  s_dtype = PyUnicode_InternFromString("dtype");
  s_shape = PyUnicode_InternFromString("shape");
  s_data_ptr = PyUnicode_InternFromString("data_ptr");
  if (!s_get_device || !s_is_contiguous || !s_dtype || !s_shape || !s_data_ptr) return NULL;
  PyObject* m = PyModule_Create(&module);
  // whose headers this was compiled with: a tensor's layout is the version's
  if (m && PyModule_AddStringConstant(m, "torch_version", TORCH_VERSION)) Py_CLEAR(m);
  return m;
}
