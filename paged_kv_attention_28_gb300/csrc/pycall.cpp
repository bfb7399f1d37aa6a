// CPython side of the binding's small calls: the checks of their tensors and the call itself.
//
// A small call's time is the host's. The cache write of 64 tokens (a kernel of 3.7 us, eleven tensors, 32
// arguments) takes 14.3 us on the Grace host through Python and ctypes, 9.8 with a tensor's
// attributes asked for here through the object protocol, 3.4 with the whole call here and its tensors
// read through PyTorch's headers; 2.1 of that is the launch.
#define PY_SSIZE_T_CLEAN
#include <c10/cuda/CUDAFunctions.h>
#include <c10/cuda/CUDAStream.h>
#include <torch/csrc/Dtype.h>
#include <torch/csrc/DynamicTypes.h>
#include <torch/csrc/autograd/python_variable.h>
#include <torch/version.h>

#include <algorithm>
#include <climits>
#include <cstdint>

#include "pkv_attn.h"

static PyObject *s_get_device, *s_is_contiguous, *s_dtype, *s_shape, *s_data_ptr, *s_cuda_stream;

// need(tensor, name, device, dtype | None, shape | None) -> address of its data.
// The tensor has to be a contiguous CUDA tensor on that device, of that type and shape. Asks it through
// the object protocol: for what address() below does not find in order, and in its words.
static PyObject* need(PyObject* self, PyObject* const* a, Py_ssize_t n) {
  (void)self;
  if (n != 5) return PyErr_Format(PyExc_TypeError, "need() takes 5 arguments, got %zd", n);
  PyObject *t = a[0], *r;
  const long want = PyLong_AsLong(a[2]);
  if (want == -1 && PyErr_Occurred()) return NULL;
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

namespace {

struct Raised {};  // a Python exception is set

template <class... T>
[[noreturn]] void raise(PyObject* type, const char* format, T... values) {
  PyErr_Format(type, format, values...);
  throw Raised{};
}

using c10::ScalarType;
constexpr ScalarType kAny = ScalarType::Undefined, kI32 = ScalarType::Int, kF32 = ScalarType::Float;

struct Shape {
  int dims;  // -1: any shape
  int64_t size[4];
};
constexpr Shape kAnyShape{-1, {}};
template <class... T>
Shape shape(T... v) {
  return {(int)sizeof...(v), {(int64_t)v...}};
}

const at::Tensor& tensor(PyObject* t, const char* name, int dims) {
  if (!THPVariable_Check(t)) raise(PyExc_TypeError, "%s must be a tensor, not %s", name, Py_TYPE(t)->tp_name);
  const at::Tensor& x = THPVariable_Unpack(t);
  if (x.dim() != dims) raise(PyExc_ValueError, "%s must have %d dimensions, has %lld", name, dims, (long long)x.dim());
  return x;
}

// The current device, where every tensor of a call has to be (-2 for a host tensor: no device).
long device_of(const at::Tensor& x) { return x.is_cuda() ? c10::cuda::current_device() : -2; }

bool is_at(const at::Tensor& x, long dev, ScalarType type) {
  return x.has_storage() && x.is_cuda() && x.get_device() == dev && (type == kAny || x.scalar_type() == type);
}

// The address of a contiguous tensor's data on that device, of that type and shape.
void* address(PyObject* t, const char* name, long dev, ScalarType type, const Shape& want) {
  if (THPVariable_Check(t)) {
    const at::Tensor& x = THPVariable_Unpack(t);
    if (is_at(x, dev, type) && x.is_contiguous() &&
        (want.dims < 0 || (x.dim() == want.dims && std::equal(x.sizes().begin(), x.sizes().end(), want.size))))
      return x.data_ptr();
  }
  PyObject* a[5] = {t, PyUnicode_FromString(name), PyLong_FromLong(dev), Py_None, Py_None};
  if (type != kAny) a[3] = reinterpret_cast<PyObject*>(torch::getTHPDtype(type));  // (lives as long as PyTorch)
  if (want.dims >= 0) {
    a[4] = PyTuple_New(want.dims);
    for (int i = 0; a[4] && i < want.dims; ++i) PyTuple_SET_ITEM(a[4], i, PyLong_FromLongLong(want.size[i]));
  }
  PyObject* r = a[1] && a[2] && a[4] ? need(nullptr, a, 5) : nullptr;
  Py_XDECREF(a[1]);
  Py_XDECREF(a[2]);
  if (want.dims >= 0) Py_XDECREF(a[4]);
  if (!r) throw Raised{};
  void* p = PyLong_AsVoidPtr(r);
  Py_DECREF(r);
  return p;
}

void* address_or_null(PyObject* t, const char* name, long dev, ScalarType type, const Shape& want) {
  return t == Py_None ? nullptr : address(t, name, dev, type, want);
}

struct Rows {
  void* at;
  int64_t step;  // elements from one token to the next
};

// [B, C, H, D] whose head rows are contiguous per token, at one distance per token.
Rows token_rows(PyObject* t, const char* name, long dev, ScalarType type, int64_t B, int64_t C, int64_t H, int64_t D) {
  const at::Tensor& x = tensor(t, name, 4);
  if (!is_at(x, dev, kAny))
    raise(PyExc_ValueError, "%s must be a CUDA tensor on the current device, is on %s", name, x.device().str().c_str());
  if (x.scalar_type() != type)
    raise(PyExc_ValueError, "%s must be %s, is %s", name, c10::toString(type), c10::toString(x.scalar_type()));
  if (x.size(0) != B || x.size(1) != C || x.size(2) != H || x.size(3) != D)
    raise(PyExc_ValueError, "%s has shape (%lld, %lld, %lld, %lld), expected (%lld, %lld, %lld, %lld)", name,
          (long long)x.size(0), (long long)x.size(1), (long long)x.size(2), (long long)x.size(3), (long long)B,
          (long long)C, (long long)H, (long long)D);
  const int64_t sb = x.stride(0), sc = x.stride(1);
  if (!((x.stride(3) == 1 || D == 1) && (x.stride(2) == D || H == 1) && (sb == C * sc || B == 1 || C == 1)))
    raise(PyExc_ValueError, "%s must hold each token's heads contiguously at one stride per token, has strides "
          "(%lld, %lld, %lld, %lld)", name, (long long)sb, (long long)sc, (long long)x.stride(2), (long long)x.stride(3));
  return {x.data_ptr(), C > 1 ? sc : B > 1 ? sb : H * D};
}

int dtype_of(const at::Tensor& x) {
  if (x.scalar_type() == kF32) return PKV_F32;
  if (x.scalar_type() == ScalarType::BFloat16) return PKV_BF16;
  raise(PyExc_TypeError, "unsupported dtype %s", c10::toString(x.scalar_type()));
}

// A size past 32 bits must not wrap into a valid one: INT_MIN is refused by every call.
int narrow(int64_t v) { return v < INT_MIN || v > INT_MAX ? INT_MIN : (int)v; }

int64_t integer(PyObject* o) {
  if (!PyLong_Check(o)) {
    PyObject* i = PyNumber_Long(o);
    if (!i) throw Raised{};
    const long long v = PyLong_AsLongLong(i);
    Py_DECREF(i);
    if (v == -1 && PyErr_Occurred()) throw Raised{};
    return v;
  }
  const long long v = PyLong_AsLongLong(o);
  if (v == -1 && PyErr_Occurred()) throw Raised{};
  return v;
}

float number(PyObject* o) {
  const double v = PyFloat_AsDouble(o);
  if (v == -1.0 && PyErr_Occurred()) throw Raised{};
  return (float)v;
}

bool truth(PyObject* o) {
  const int v = PyObject_IsTrue(o);
  if (v < 0) throw Raised{};
  return v;
}

// The handle of a torch stream, or of the device's current one. Asked for after the tensors' checks.
void* stream_of(PyObject* o, long dev) {
  if (o == Py_None) return c10::cuda::getCurrentCUDAStream((c10::DeviceIndex)dev).stream();
  PyObject* h = PyObject_GetAttr(o, s_cuda_stream);
  if (!h) throw Raised{};
  void* p = PyLong_AsVoidPtr(h);
  Py_DECREF(h);
  if (!p && PyErr_Occurred()) throw Raised{};
  return p;
}

int32_t* flag_of(PyObject* o, long dev) {
  return static_cast<int32_t*>(address_or_null(o, "err_flag", dev, kI32, kAnyShape));
}

struct Unlocked {  // a launch can wait for room in the stream: without the interpreter lock
  PyThreadState* state = PyEval_SaveThread();
  ~Unlocked() { PyEval_RestoreThread(state); }
};

// The pages of a pool [num_pages, n_kv_heads, page_size, head_dim].
struct Pool {
  int64_t pages, heads, page, d;
  Shape shape;
};
Pool pool_of(PyObject* t, const char* name) {
  const at::Tensor& x = tensor(t, name, 4);
  return {x.size(0), x.size(1), x.size(2), x.size(3), {4, {x.size(0), x.size(1), x.size(2), x.size(3)}}};
}
void same_head_dim(const Pool& p, int64_t d) {
  if (p.d != d) raise(PyExc_ValueError, "k_pages has head_dim %lld, q has %lld", (long long)p.d, (long long)d);
}

template <class T>
T* as(void* p) {
  return static_cast<T*>(p);
}

int append(PyObject* const* a) {
  const at::Tensor& q = tensor(a[0], "q", 4);
  const int64_t B = q.size(0), C = q.size(1), Hq = q.size(2), D = q.size(3);
  const Pool pool = pool_of(a[3], "k_pages");
  same_head_dim(pool, D);
  const long dev = device_of(q);
  const ScalarType type = q.scalar_type();
  const Rows rq = token_rows(a[0], "q", dev, type, B, C, Hq, D), rk = token_rows(a[1], "k", dev, type, B, C, pool.heads, D),
             rv = token_rows(a[2], "v", dev, type, B, C, pool.heads, D);
  void* kp = address(a[3], "k_pages", dev, type, kAnyShape);
  void* vp = address(a[4], "v_pages", dev, type, pool.shape);
  const int64_t blocks = tensor(a[5], "block_table", 2).size(1);
  const auto* table = as<int32_t>(address(a[5], "block_table", dev, kI32, shape(B, blocks)));
  const auto* prefix = as<int32_t>(address(a[6], "prefix_lens", dev, kI32, shape(B)));
  const auto* chunk = as<int32_t>(address_or_null(a[7], "chunk_lens", dev, kI32, shape(B)));
  int64_t axes = 1;
  const int32_t* positions = nullptr;
  if (a[8] != Py_None) {
    if (THPVariable_Check(a[8]) && THPVariable_Unpack(a[8]).dim() == 3) {
      axes = THPVariable_Unpack(a[8]).size(0);
      positions = as<int32_t>(address(a[8], "positions", dev, kI32, shape(axes, B, C)));
    } else {
      positions = as<int32_t>(address(a[8], "positions", dev, kI32, shape(B, C)));
    }
  }
  int64_t pairs = 0;
  const float* freq = nullptr;
  if (a[9] != Py_None) {
    pairs = tensor(a[9], "inv_freq", 1).size(0);
    freq = as<float>(address(a[9], "inv_freq", dev, kF32, shape(pairs)));
  }
  const auto* axis = as<int32_t>(address_or_null(a[10], "pair_axis", dev, kI32, shape(pairs)));
  void* qn = address_or_null(a[11], "q_norm", dev, type, shape(D));
  void* kn = address_or_null(a[12], "k_norm", dev, type, shape(D));
  const float eps = number(a[13]);
  const int interleaved = truth(a[14]);
  void* out = address(a[15], "out", dev, type, shape(B, C, Hq, D));
  int32_t* err = flag_of(a[16], dev);
  const int dt = dtype_of(q);
  void* stream = stream_of(a[17], dev);
  Unlocked u;
  return attn_qk_norm_rope_append(rq.at, rk.at, rv.at, rq.step, rk.step, rv.step, qn, kn, eps, freq, narrow(2 * pairs),
                                  interleaved, positions, narrow(axes), axis, table, prefix, chunk, out, kp, vp, narrow(B),
                                  narrow(C), narrow(blocks), narrow(pool.pages), narrow(Hq), narrow(pool.heads), narrow(D),
                                  narrow(pool.page), dt, err, stream);
}

int decode_weights(PyObject* const* a) {
  const at::Tensor& q = tensor(a[0], "q", 3);
  const int64_t B = q.size(0), Hq = q.size(1), D = q.size(2);
  const Pool pool = pool_of(a[1], "k_pages");
  same_head_dim(pool, D);
  const long dev = device_of(q);
  const ScalarType type = q.scalar_type();
  void* qp = address(a[0], "q", dev, kAny, kAnyShape);
  void* kp = address(a[1], "k_pages", dev, type, kAnyShape);
  void* vp = address(a[2], "v_pages", dev, type, pool.shape);
  const int64_t blocks = tensor(a[3], "block_table", 2).size(1);
  const auto* table = as<int32_t>(address(a[3], "block_table", dev, kI32, shape(B, blocks)));
  const auto* lens = as<int32_t>(address(a[4], "kv_lens", dev, kI32, shape(B)));
  const Shape sums = shape(B, pool.heads, blocks * pool.page);
  const auto* in = as<float>(address(a[5], "weight_sums", dev, kF32, sums));
  auto* to = as<float>(address(a[6], "sums_out", dev, kF32, sums));
  const float scale = number(a[7]), decay = number(a[8]);
  const int splits = narrow(integer(a[9]));
  void* out = address(a[10], "out", dev, type, shape(B, Hq, D));
  auto* lse = as<float>(address(a[11], "lse", dev, kF32, shape(B, Hq)));
  void* ws = address_or_null(a[12], "workspace", dev, kAny, kAnyShape);
  const size_t bytes = ws ? THPVariable_Unpack(a[12]).nbytes() : 0;
  int32_t* err = flag_of(a[13], dev);
  const int dt = dtype_of(q);
  void* stream = stream_of(a[14], dev);
  Unlocked u;
  return attn_decode_paged_weights(qp, kp, vp, table, lens, out, lse, in, to, narrow(B), narrow(blocks), narrow(pool.pages),
                                   narrow(Hq), narrow(pool.heads), narrow(D), narrow(pool.page), scale, decay, splits, dt,
                                   ws, bytes, err, stream);
}

int chunk_weights(PyObject* const* a) {
  const at::Tensor& q = tensor(a[0], "q", 4);
  const int64_t B = q.size(0), C = q.size(1), Hq = q.size(2), D = q.size(3);
  const Pool pool = pool_of(a[1], "k_pages");
  same_head_dim(pool, D);
  const long dev = device_of(q);
  void* qp = address(a[0], "q", dev, kAny, kAnyShape);
  void* kp = address(a[1], "k_pages", dev, q.scalar_type(), kAnyShape);
  const int64_t blocks = tensor(a[2], "block_table", 2).size(1);
  const auto* table = as<int32_t>(address(a[2], "block_table", dev, kI32, shape(B, blocks)));
  const auto* prefix = as<int32_t>(address(a[3], "prefix_lens", dev, kI32, shape(B)));
  const auto* chunk = as<int32_t>(address_or_null(a[4], "chunk_lens", dev, kI32, shape(B)));
  const auto* lse = as<float>(address(a[5], "lse", dev, kF32, shape(B, Hq, C)));
  const Shape sums = shape(B, pool.heads, blocks * pool.page);
  const auto* in = as<float>(address(a[6], "weight_sums", dev, kF32, sums));
  auto* to = as<float>(address(a[7], "sums_out", dev, kF32, sums));
  const float scale = number(a[8]), decay = number(a[9]);
  const int window = narrow(integer(a[10]));
  int32_t* err = flag_of(a[11], dev);
  const int dt = dtype_of(q);
  void* stream = stream_of(a[12], dev);
  Unlocked u;
  return attn_chunk_weights(qp, kp, table, prefix, chunk, lse, in, to, narrow(B), narrow(C), window, narrow(blocks),
                            narrow(pool.pages), narrow(Hq), narrow(pool.heads), narrow(D), narrow(pool.page), scale, decay,
                            dt, err, stream);
}

int evict(PyObject* const* a) {
  const Pool pool = pool_of(a[0], "k_pages");
  const at::Tensor& k = THPVariable_Unpack(a[0]);
  const long dev = device_of(k);
  const ScalarType type = k.scalar_type();
  void* kp = address(a[0], "k_pages", dev, kAny, kAnyShape);
  void* vp = address(a[1], "v_pages", dev, type, pool.shape);
  const at::Tensor& table_t = tensor(a[2], "block_table", 2);
  const int64_t B = table_t.size(0), blocks = table_t.size(1), new_blocks = tensor(a[5], "new_block_table", 2).size(1);
  const int64_t budget = integer(a[9]), sink = integer(a[10]), recent = integer(a[11]);
  const auto* table = as<int32_t>(address(a[2], "block_table", dev, kI32, kAnyShape));
  const auto* lens = as<int32_t>(address(a[3], "kv_lens", dev, kI32, shape(B)));
  const auto* sums = as<float>(address(a[4], "weight_sums", dev, kF32, shape(B, pool.heads, blocks * pool.page)));
  const auto* new_table = as<int32_t>(address(a[5], "new_block_table", dev, kI32, shape(B, new_blocks)));
  auto* kept = as<int32_t>(address(a[6], "kept", dev, kI32, shape(B, pool.heads, std::max<int64_t>(budget, 0))));
  auto* new_lens = as<int32_t>(address(a[7], "new_lens", dev, kI32, shape(B)));
  auto* new_sums = as<float>(address(a[8], "new_sums", dev, kF32, shape(B, pool.heads, new_blocks * pool.page)));
  int32_t* err = flag_of(a[12], dev);
  const int dt = dtype_of(k);
  void* stream = stream_of(a[13], dev);
  Unlocked u;
  return attn_cache_evict(kp, vp, table, lens, sums, new_table, kept, new_lens, new_sums, narrow(B), narrow(blocks),
                          narrow(new_blocks), narrow(pool.pages), narrow(pool.heads), narrow(pool.d), narrow(pool.page),
                          narrow(budget), narrow(sink), narrow(recent), dt, err, stream);
}

int linear(PyObject* const* a) {
  const at::Tensor& x = tensor(a[0], "x", 2);
  const int64_t m = x.size(0), k = x.size(1), n = tensor(a[1], "w", 2).size(0);
  const long dev = device_of(x);
  const ScalarType type = x.scalar_type();
  void* xp = address(a[0], "x", dev, kAny, kAnyShape);
  void* w = address(a[1], "w", dev, type, shape(n, k));
  void* bias = address_or_null(a[2], "bias", dev, type, shape(n));
  void* residual = address_or_null(a[3], "residual", dev, type, shape(m, n));
  void* out = address(a[4], "out", dev, type, shape(m, n));
  const int act = narrow(integer(a[5]));
  int32_t* err = flag_of(a[6], dev);
  const int dt = dtype_of(x);
  void* stream = stream_of(a[7], dev);
  Unlocked u;
  return attn_linear(xp, w, bias, residual, out, narrow(m), narrow(n), narrow(k), act, dt, err, stream);
}

// A call of N positional arguments; the status of the C call, or the exception that was raised.
template <int (*F)(PyObject* const*), int N>
PyObject* entry(PyObject*, PyObject* const* a, Py_ssize_t n) {
  if (n != N) return PyErr_Format(PyExc_TypeError, "takes %d arguments, got %zd", N, n);
  try {
    return PyLong_FromLong(F(a));
  } catch (const Raised&) {
  } catch (const std::exception& e) {
    PyErr_SetString(PyExc_RuntimeError, e.what());
  }
  return nullptr;
}

}  // namespace

#define METHOD(name, f) {name, (PyCFunction)(void (*)(void))f, METH_FASTCALL, NULL}
static PyMethodDef methods[] = {
    METHOD("need", need),
    METHOD("qk_norm_rope_append", (entry<append, 18>)),
    METHOD("decode_paged_weights", (entry<decode_weights, 15>)),
    METHOD("chunk_weights", (entry<chunk_weights, 13>)),
    METHOD("cache_evict", (entry<evict, 14>)),
    METHOD("linear", (entry<linear, 8>)),
    {NULL, NULL, 0, NULL},
};
static struct PyModuleDef module = {PyModuleDef_HEAD_INIT, "_pycall", NULL, -1, methods, NULL, NULL, NULL, NULL};

PyMODINIT_FUNC PyInit__pycall(void) {
  s_get_device = PyUnicode_InternFromString("get_device");
  s_is_contiguous = PyUnicode_InternFromString("is_contiguous");
  s_dtype = PyUnicode_InternFromString("dtype");
  s_shape = PyUnicode_InternFromString("shape");
  s_data_ptr = PyUnicode_InternFromString("data_ptr");
  s_cuda_stream = PyUnicode_InternFromString("cuda_stream");
  if (!s_cuda_stream || !s_get_device || !s_is_contiguous || !s_dtype || !s_shape || !s_data_ptr) return NULL;
  PyObject* m = PyModule_Create(&module);
  // whose headers this was compiled with: a tensor's layout is the version's
  if (m && PyModule_AddStringConstant(m, "torch_version", TORCH_VERSION)) Py_CLEAR(m);
  return m;
}
