// _hlocall: the marshalling of the layer entry points (hlo_rms_norm, hlo_rms_norm_backward, hlo_dropout, hlo_rotary,
// hlo_logits_process) as a CPython extension. A serving step makes hundreds of these calls on a few
// kilobytes each, where building the descriptors in Python costs more than the kernel (measured on the
// GPU's host for one token's norm: 11 us a call through ctypes, of which the launch is about 2); here the
// tensors' own fields are read. Every function takes its operands by position and returns the hlo_status;
// nothing is kept between calls.
#define PY_SSIZE_T_CLEAN
#include <Python.h>

#include <ATen/core/Tensor.h>
#include <c10/cuda/CUDAStream.h>
#include <torch/csrc/autograd/python_variable.h>

#include <cstdarg>
#include <cstring>
#include <exception>
#include <initializer_list>

#include "hlo_fusion.h"

namespace {

PyObject *s_ptr, *s_addr;
PyObject* g_view_type;    // DeviceView
PyObject* g_error;        // HloError
PyObject* g_dropout_type; // Dropout
PyObject* g_quant_type;   // Quant

int g_device;  // the current device once a call has read a tensor, -1 before; under the interpreter's lock, as all reading is

// One argument: a tensor, a DeviceView or None.
struct Operand {
  hlo_view v;
  void* p = nullptr;
  bool given = false;
  bool words = false;  // a tensor of 64-bit whole numbers, which no view of the library has
  const hlo_view* view() const { return given ? &v : nullptr; }
};

// Raises HloError(HLO_ERR_INVALID_ARG, message).
bool refuse(const char* format, ...) {
  va_list ap;
  va_start(ap, format);
  PyObject* text = PyUnicode_FromFormatV(format, ap);
  va_end(ap);
  PyObject* e = text ? PyObject_CallFunction(g_error, "iO", (int)HLO_ERR_INVALID_ARG, text) : nullptr;
  if (e) PyErr_SetObject(g_error, e);
  Py_XDECREF(e);
  Py_XDECREF(text);
  return false;
}

bool address(PyObject* o, void** p) {
  *p = PyLong_AsVoidPtr(o);
  return *p || !PyErr_Occurred();
}

int32_t type_of(at::ScalarType t) {
  switch (t) {
    case at::kFloat: return HLO_F32;
    case at::kBFloat16: return HLO_BF16;
    case at::kHalf: return HLO_F16;
    case at::kChar: return HLO_S8;
    case at::kInt: return HLO_S32;
    case at::kFloat8_e4m3fn: return HLO_F8E4M3FN;
    default: return -1;
  }
}

bool read(PyObject* t, Operand* o) {
  if (t == Py_None) return true;
  o->given = true;
  if (THPVariable_Check(t)) {
    try {
      const at::Tensor& x = THPVariable_Unpack(t);
      if (!x.is_cuda()) return refuse("a tensor on the GPU is wanted");
      if (g_device < 0) g_device = c10::cuda::current_device();
      if (x.get_device() != g_device)
        return refuse("a tensor is on cuda:%d, and the current device is cuda:%d", (int)x.get_device(), (int)g_device);
      if (x.is_neg()) return refuse("a tensor that negates its memory's values when it is read");
      const auto sizes = x.sizes(), strides = x.strides();
      o->v.rank = (int32_t)x.dim();  // a rank that is too high is the library's to refuse
      o->v.dtype = type_of(x.scalar_type());
      o->words = x.scalar_type() == at::kLong || x.scalar_type() == at::kUInt64;
      for (int64_t d = 0; d < x.dim() && d < HLO_MAX_RANK; ++d) {
        o->v.dims[d] = sizes[d];
        o->v.strides[d] = strides[d];
      }
      o->p = x.data_ptr();
      return true;
    } catch (const std::exception& e) {  // a tensor without storage or strides
      return refuse("%s", e.what());
    }
  }
  if ((PyObject*)Py_TYPE(t) != g_view_type) {
    PyErr_SetString(PyExc_TypeError, "a tensor or a DeviceView is wanted");
    return false;
  }
  PyObject *a = PyObject_GetAttr(t, s_addr), *p = a ? PyObject_GetAttr(t, s_ptr) : nullptr;
  void* view = nullptr;
  const bool ok = a && p && address(a, &view) && address(p, &o->p);
  if (ok) std::memcpy(&o->v, view, sizeof o->v);
  Py_XDECREF(a);
  Py_XDECREF(p);
  return ok;
}

// A contiguous vector of `count` elements (count < 0: any number, stored), an address, or None. *dtype: the wanted type,
// -1 and then set to that of the tensor, which has to be one of the library's, or kWords for 64-bit whole numbers.
constexpr int32_t kWords = -2;
bool read_vector(PyObject* t, int64_t* count, int32_t* dtype, const char* what, void** p) {
  *p = nullptr;
  if (t == Py_None) return true;
  if (PyLong_Check(t)) return address(t, p);
  Operand o;
  if (!read(t, &o)) return false;
  int64_t n = 1;
  bool dense = o.v.rank <= HLO_MAX_RANK;
  for (int d = o.v.rank - 1; dense && d >= 0; --d) {
    dense = o.v.dims[d] == 1 || o.v.strides[d] == n;
    n *= o.v.dims[d];
  }
  if ((!dense && n != 0) || (*count >= 0 && n != *count) || (*dtype >= 0 && o.v.dtype != *dtype) || (*dtype == kWords) != o.words) {
    if (*count < 0) return refuse("%s: a contiguous vector of the right type is wanted", what);
    return refuse("%s: a contiguous vector of %lld elements of the right type is wanted", what, (long long)*count);
  }
  if (o.v.dtype < 0 && !o.words) return refuse("%s: element type not supported", what);
  *count = n;
  *dtype = o.v.dtype;
  *p = o.p;
  return true;
}

bool read_vector(PyObject* t, int64_t count, int32_t dtype, const char* what, void** p) {
  return read_vector(t, &count, &dtype, what, p);
}

// Scratch memory: a contiguous tensor of any type, whose size counts (or fewer bytes of it), or an address with its size.
bool read_scratch(PyObject* t, PyObject* size, void** p, size_t* bytes) {
  *p = nullptr;
  *bytes = 0;
  if (size != Py_None) {
    *bytes = PyLong_AsSize_t(size);
    if (PyErr_Occurred()) return false;
  }
  if (t == Py_None) return true;
  if (PyLong_Check(t)) return address(t, p);
  if (!THPVariable_Check(t)) {
    PyErr_SetString(PyExc_TypeError, "a tensor or an address is wanted");
    return false;
  }
  Operand o;
  if (!read(t, &o)) return false;
  const at::Tensor& x = THPVariable_Unpack(t);
  if (!x.is_contiguous()) return refuse("workspace: a contiguous tensor is wanted");
  if (size != Py_None && *bytes > x.nbytes()) return refuse("workspace: %zu bytes, but the tensor has %zu", *bytes, (size_t)x.nbytes());
  if (size == Py_None) *bytes = x.nbytes();
  *p = o.p;
  return true;
}

// The ctypes structure of that type behind `o` (or NULL for None); its memory outlives the call, since the caller holds it.
template <typename T>
bool read_struct(PyObject* o, PyObject* type, T** out) {
  *out = nullptr;
  if (o == Py_None) return true;
  const int is = PyObject_IsInstance(o, type);
  if (is <= 0) {
    if (is == 0) PyErr_Format(PyExc_TypeError, "a %s is wanted", reinterpret_cast<PyTypeObject*>(type)->tp_name);
    return false;
  }
  Py_buffer b;
  if (PyObject_GetBuffer(o, &b, PyBUF_SIMPLE) != 0) return false;
  const bool ok = b.len == (Py_ssize_t)sizeof(T);
  *out = static_cast<T*>(b.buf);
  PyBuffer_Release(&b);
  if (!ok) PyErr_SetString(PyExc_TypeError, "a parameter structure has the wrong size");
  return ok;
}

// A stream's handle, or None for torch's current stream.
bool read_stream(PyObject* o, void** stream) {
  if (o != Py_None) return address(o, stream);
  try {
    *stream = c10::cuda::getCurrentCUDAStream().stream();
    return true;
  } catch (const std::exception& e) {  // no device
    PyErr_SetString(PyExc_RuntimeError, e.what());
    return false;
  }
}

// The first step of every call.
bool count_is(Py_ssize_t n, Py_ssize_t want) {
  g_device = -1;
  if (n == want) return true;
  PyErr_Format(PyExc_TypeError, "%zd arguments, %zd are wanted", n, want);
  return false;
}

int64_t rows_of(const hlo_view& v) {
  int64_t r = 1;
  for (int d = 0; d + 1 < v.rank && d < HLO_MAX_RANK; ++d) r *= v.dims[d];
  return r;
}
int64_t last_of(const hlo_view& v) { return v.rank > 0 && v.rank <= HLO_MAX_RANK ? v.dims[v.rank - 1] : 0; }

// The status; after a call that ran, its output tensors' versions have moved on, so that autograd notices a saved tensor
// that was overwritten.
PyObject* status(hlo_status s, std::initializer_list<PyObject*> outputs) {
  if (s == HLO_OK) {
    for (PyObject* t : outputs) {
      if (!THPVariable_Check(t)) continue;
      const at::Tensor& x = THPVariable_Unpack(t);
      if (!x.is_inference()) x.unsafeGetTensorImpl()->bump_version();
    }
  }
  return PyLong_FromLong((long)s);
}

#define CALL(expr, ...)                        \
  hlo_status st;                               \
  Py_BEGIN_ALLOW_THREADS;                      \
  st = (expr);                                 \
  Py_END_ALLOW_THREADS;                        \
  return status(st, {__VA_ARGS__})

// x, out, weight, weight_dtype, residual, sum, rstd, eps, weight_offset, dropout, scales, out_q, stream
PyObject* rms_norm(PyObject*, PyObject* const* a, Py_ssize_t n) {
  if (!count_is(n, 13)) return nullptr;
  Operand x, out, res, sum;
  if (!read(a[0], &x) || !read(a[1], &out) || !read(a[4], &res) || !read(a[5], &sum)) return nullptr;
  const int64_t rows = x.given ? rows_of(x.v) : 0;
  int64_t cols = x.given ? last_of(x.v) : 0;
  int32_t wdt = -1;
  void *w, *rstd, *scales, *stream;
  hlo_dropout_params* drop;
  hlo_quant* q;
  if (!read_vector(a[2], &cols, &wdt, "weight", &w) || !read_vector(a[6], rows, HLO_F32, "rstd", &rstd) ||
      !read_vector(a[10], rows, HLO_F32, "scales", &scales) || !read_struct(a[9], g_dropout_type, &drop) || !read_struct(a[11], g_quant_type, &q) ||
      !read_stream(a[12], &stream))
    return nullptr;
  if (wdt < 0) wdt = (int32_t)PyLong_AsLong(a[3]);
  const double eps = PyFloat_AsDouble(a[7]), off = PyFloat_AsDouble(a[8]);
  if (PyErr_Occurred()) return nullptr;
  CALL(hlo_rms_norm(x.view(), x.p, res.view(), res.p, drop, w, wdt, off, eps, sum.view(), sum.p, out.view(), out.p,
                    static_cast<float*>(scales), q, static_cast<float*>(rstd), stream),
       a[1], a[5], a[6], a[10]);
}

// dy, h, rstd, dh, weight, weight_dtype, dsum, dx, dropout, dweight, workspace, workspace_bytes, weight_offset, stream
PyObject* rms_norm_backward(PyObject*, PyObject* const* a, Py_ssize_t n) {
  if (!count_is(n, 14)) return nullptr;
  Operand dy, h, dh, ds, dx;
  if (!read(a[0], &dy) || !read(a[1], &h) || !read(a[3], &dh) || !read(a[6], &ds) || !read(a[7], &dx)) return nullptr;
  const int64_t rows = h.given ? rows_of(h.v) : 0;
  int64_t cols = h.given ? last_of(h.v) : 0;
  const int64_t width = cols;
  int32_t wdt = -1;
  void *w, *rstd, *dw, *ws, *stream;
  size_t bytes;
  hlo_dropout_params* drop;
  if (!read_vector(a[4], &cols, &wdt, "weight", &w) || !read_vector(a[2], rows, HLO_F32, "rstd", &rstd) ||
      !read_vector(a[9], width, HLO_F32, "dweight", &dw) || !read_struct(a[8], g_dropout_type, &drop) || !read_scratch(a[10], a[11], &ws, &bytes) ||
      !read_stream(a[13], &stream))
    return nullptr;
  if (wdt < 0) wdt = (int32_t)PyLong_AsLong(a[5]);
  const double off = PyFloat_AsDouble(a[12]);
  if (PyErr_Occurred()) return nullptr;
  CALL(hlo_rms_norm_backward(dy.view(), dy.p, h.view(), h.p, static_cast<float*>(rstd), w, wdt, off, ds.view(), ds.p, drop, dh.view(),
                             dh.p, dx.view(), dx.p, static_cast<float*>(dw), ws, bytes, stream),
       a[3], a[7], a[9], a[10]);
}

// x, out, dropout, residual, stream
PyObject* dropout(PyObject*, PyObject* const* a, Py_ssize_t n) {
  if (!count_is(n, 5)) return nullptr;
  Operand x, out, res;
  hlo_dropout_params* drop;
  void* stream;
  if (!read(a[0], &x) || !read(a[1], &out) || !read(a[3], &res) || !read_struct(a[2], g_dropout_type, &drop) || !read_stream(a[4], &stream)) return nullptr;
  CALL(hlo_dropout(x.view(), x.p, res.view(), res.p, drop, out.view(), out.p, stream), a[1]);
}

// x, out, positions, turns, n_pairs (None: turns' count, the most that is taken), k, k_out, interleaved, scale, inverse, stream
PyObject* rotary(PyObject*, PyObject* const* a, Py_ssize_t n) {
  if (!count_is(n, 11)) return nullptr;
  Operand x, out, pos, k, kout;
  if (!read(a[0], &x) || !read(a[1], &out) || !read(a[2], &pos) || !read(a[5], &k) || !read(a[6], &kout)) return nullptr;
  int64_t pairs = -1;
  int32_t words = kWords;
  void *turns, *stream;
  if (!read_vector(a[3], &pairs, &words, "turns", &turns) || !read_stream(a[10], &stream)) return nullptr;
  if (a[4] != Py_None) {
    const int64_t wanted = PyLong_AsLongLong(a[4]);
    if (PyErr_Occurred()) return nullptr;
    if (pairs >= 0 && wanted > pairs) {  // an address has no count
      refuse("rotary: %lld pairs, but turns has %lld", (long long)wanted, (long long)pairs);
      return nullptr;
    }
    pairs = wanted;
  }
  const double scale = PyFloat_AsDouble(a[8]);
  const int inter = PyObject_IsTrue(a[7]), inverse = PyObject_IsTrue(a[9]);
  if (PyErr_Occurred()) return nullptr;
  if (pairs > INT32_MAX) pairs = INT32_MAX;
  if (pairs < -1) pairs = -1;  // refused
  CALL(hlo_rotary(x.view(), x.p, out.view(), out.p, k.view(), k.p, kout.view(), kout.p, pos.view(), static_cast<int32_t*>(pos.p),
                  static_cast<uint64_t*>(turns), (int32_t)pairs, inter, inverse, scale, stream),
       a[1], a[6]);
}

// A row of n dimensions serves every row of the batch.
void repeat_row(Operand* o, int64_t batch) {
  if (!o->given || o->v.rank != 1) return;
  o->v.rank = 2;
  o->v.dims[1] = o->v.dims[0];
  o->v.strides[1] = o->v.strides[0];
  o->v.dims[0] = batch;
  o->v.strides[0] = 0;
}

// logits, out, bias, history, lengths, prompt_lengths, repetition, frequency, presence, mask, token, stream
PyObject* logits_process(PyObject*, PyObject* const* a, Py_ssize_t n) {
  if (!count_is(n, 12)) return nullptr;
  Operand x, out, bias, hist, mask;
  if (!read(a[0], &x) || !read(a[1], &out) || !read(a[2], &bias) || !read(a[3], &hist) || !read(a[9], &mask)) return nullptr;
  const int64_t b = x.given && x.v.rank > 0 ? x.v.dims[0] : 0;
  repeat_row(&bias, b);
  repeat_row(&mask, b);
  void *len, *prompt, *rep, *freq, *pres, *token, *stream;
  if (!read_vector(a[4], b, HLO_S32, "lengths", &len) || !read_vector(a[5], b, HLO_S32, "prompt_lengths", &prompt) ||
      !read_vector(a[6], b, HLO_F32, "repetition", &rep) || !read_vector(a[7], b, HLO_F32, "frequency", &freq) ||
      !read_vector(a[8], b, HLO_F32, "presence", &pres) || !read_vector(a[10], b, HLO_S32, "token", &token) ||
      !read_stream(a[11], &stream))
    return nullptr;
  CALL(hlo_logits_process(x.view(), x.p, bias.view(), static_cast<float*>(bias.p), hist.view(), static_cast<int32_t*>(hist.p),
                          static_cast<int32_t*>(len), static_cast<int32_t*>(prompt), static_cast<float*>(rep),
                          static_cast<float*>(freq), static_cast<float*>(pres), mask.view(), static_cast<int32_t*>(mask.p), out.view(),
                          out.p, static_cast<int32_t*>(token), stream),
       a[1], a[10]);
}

// DeviceView, HloError, Dropout and Quant
PyObject* setup(PyObject*, PyObject* const* a, Py_ssize_t n) {
  if (!count_is(n, 4)) return nullptr;
  for (int i = 0; i < 4; ++i) Py_INCREF(a[i]);
  Py_XSETREF(g_view_type, a[0]);
  Py_XSETREF(g_error, a[1]);
  Py_XSETREF(g_dropout_type, a[2]);
  Py_XSETREF(g_quant_type, a[3]);
  Py_RETURN_NONE;
}

PyMethodDef methods[] = {{"setup", (PyCFunction)(void (*)(void))setup, METH_FASTCALL, nullptr},
                         {"rms_norm", (PyCFunction)(void (*)(void))rms_norm, METH_FASTCALL, nullptr},
                         {"rms_norm_backward", (PyCFunction)(void (*)(void))rms_norm_backward, METH_FASTCALL, nullptr},
                         {"dropout", (PyCFunction)(void (*)(void))dropout, METH_FASTCALL, nullptr},
                         {"rotary", (PyCFunction)(void (*)(void))rotary, METH_FASTCALL, nullptr},
                         {"logits_process", (PyCFunction)(void (*)(void))logits_process, METH_FASTCALL, nullptr},
                         {nullptr, nullptr, 0, nullptr}};
PyModuleDef module = {PyModuleDef_HEAD_INIT, "_hlocall", nullptr, -1, methods, nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__hlocall() {
  s_ptr = PyUnicode_InternFromString("ptr");
  s_addr = PyUnicode_InternFromString("addr");
  return PyModule_Create(&module);
}
