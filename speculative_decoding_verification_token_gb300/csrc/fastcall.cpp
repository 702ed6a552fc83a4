// fastcall.cpp -- argument marshalling of the short calls for Python (module _fastcall).
//
// A call that runs for a few microseconds on the GPU must not spend ten on its arguments: reading a
// tensor's device, type, shape, strides and pointer from Python costs about 0.7 us a tensor, and
// spec_process_logits takes up to 19.  These functions do what the binding's Python checks do and
// call the same C entry points (whose addresses bind() gets).  They return the sv_status, or -1 if
// any argument is not what a plain call passes: the Python path then finds out what it is and says
// so.  64 x 5 tokens appended: 8.3 us of host time a call in Python, 3.6 of them the ctypes call and
// the launch.
#define PY_SSIZE_T_CLEAN
#include <Python.h>
#include <c10/cuda/CUDAFunctions.h>
#include <c10/cuda/CUDAStream.h>
#include <torch/csrc/autograd/python_variable.h>

#include "specverify.h"

namespace {

decltype(&spec_history_append) g_history;
decltype(&spec_process_logits) g_process;
decltype(&spec_quantize_fp4) g_quantize;
decltype(&spec_project_fp4) g_project;

// What is known of a call so far: its device, and whether every argument was a plain one.
struct Call {
  int dev = -1;
  bool ok = true;

  const at::Tensor* tensor(PyObject* o, at::ScalarType type) {
    if (!THPVariable_Check(o)) return refuse();
    const at::Tensor& t = THPVariable_Unpack(o);
    if (!t.is_cuda() || t.scalar_type() != type || t.layout() != at::kStrided) return refuse();
    if (dev < 0) {
      if (t.get_device() != c10::cuda::current_device()) return refuse();
      dev = t.get_device();
    }
    return t.get_device() == dev ? &t : refuse();
  }
  const at::Tensor* refuse() {
    ok = false;
    return nullptr;
  }
  // a contiguous [n] (n < 0: any length); None is a null pointer
  template <typename T>
  T* vec(PyObject* o, at::ScalarType type, int64_t n, int64_t* length = nullptr) {
    if (o == Py_None) return nullptr;
    const at::Tensor* t = tensor(o, type);
    if (!t || !t->is_contiguous() || (n >= 0 && (t->dim() != 1 || t->size(0) != n))) {
      ok = false;
      return nullptr;
    }
    if (length) *length = t->numel();
    return static_cast<T*>(t->data_ptr());
  }
  // a 2-D tensor with unit column stride; a single row's stride says nothing
  template <typename T>
  T* mat(PyObject* o, at::ScalarType type, int64_t* rows, int64_t* cols, int64_t* ld) {
    const at::Tensor* t = tensor(o, type);
    if (!t || t->dim() != 2 || (t->size(1) > 1 && t->stride(1) != 1)) {
      ok = false;
      *rows = *cols = *ld = 0;
      return nullptr;
    }
    *rows = t->size(0);
    *cols = t->size(1);
    *ld = t->size(0) > 1 ? t->stride(0) : (std::max(t->stride(0), t->size(1)) + 7) / 8 * 8;
    return static_cast<T*>(t->data_ptr());
  }
  int64_t num(PyObject* o) {
    const int64_t v = PyLong_AsLongLong(o);
    if (v == -1 && PyErr_Occurred()) {
      PyErr_Clear();
      ok = false;
    }
    return v;
  }
  int32_t num32(PyObject* o) {
    const int64_t v = num(o);
    if (v < INT32_MIN || v > INT32_MAX) ok = false;
    return static_cast<int32_t>(v);
  }
  int32_t flag(PyObject* o) {
    const int v = PyObject_IsTrue(o);
    if (v < 0) {
      PyErr_Clear();
      ok = false;
    }
    return v;
  }
  // a torch stream, or None for the current one
  void* stream(PyObject* o) {
    if (o == Py_None) return ok ? c10::cuda::getCurrentCUDAStream(dev).stream() : nullptr;
    PyObject* number = PyObject_GetAttrString(o, "cuda_stream");
    if (!number) {
      PyErr_Clear();
      ok = false;
      return nullptr;
    }
    void* s = reinterpret_cast<void*>(num(number));
    Py_DECREF(number);
    return s;
  }
};

PyObject* answer(long code) { return PyLong_FromLong(code); }

struct History {
  int32_t* counts = nullptr;
  uint32_t *prompt = nullptr, *output = nullptr;
  int64_t n_slots = 0, V = 0, ldc = 0, ldb = 0;
};

History history(Call& c, PyObject* counts, PyObject* prompt, PyObject* output) {
  History h;
  int64_t rows, cols, ld;
  h.counts = c.mat<int32_t>(counts, at::kInt, &h.n_slots, &h.V, &h.ldc);
  h.prompt = c.mat<uint32_t>(prompt, at::kInt, &rows, &cols, &h.ldb);
  c.ok = c.ok && rows == h.n_slots && cols >= (h.V + 31) / 32;
  h.output = c.mat<uint32_t>(output, at::kInt, &rows, &cols, &ld);
  c.ok = c.ok && rows == h.n_slots && cols >= (h.V + 31) / 32 &&
         (ld == h.ldb || h.n_slots == 1) && h.n_slots <= INT32_MAX;
  return h;
}

// Runs `body` (which fills in the call and returns a code) without letting an exception through.
template <typename F>
PyObject* guarded(F&& body) {
  try {
    return answer(body());
  } catch (...) {
    if (PyErr_Occurred()) PyErr_Clear();
    return answer(-1);
  }
}

// tokens, counts, prompt_bits, output_bits, slots, lens, prompt, reset, status, stream
PyObject* history_append(PyObject*, PyObject* const* a, Py_ssize_t n_args) {
  if (n_args != 10) return answer(-1);
  return guarded([&]() -> long {
    Call c;
    int64_t B, n, ldt;
    const int32_t* tokens = c.mat<int32_t>(a[0], at::kInt, &B, &n, &ldt);
    const History h = history(c, a[1], a[2], a[3]);
    const int32_t* slots = c.vec<int32_t>(a[4], at::kInt, B);
    const int32_t* lens = c.vec<int32_t>(a[5], at::kInt, B);
    int32_t* status = c.vec<int32_t>(a[8], at::kInt, -1);
    const int32_t prompt = c.flag(a[6]), reset = c.flag(a[7]);
    void* stream = c.stream(a[9]);
    if (!c.ok || B > INT32_MAX || n > INT32_MAX || (!slots && B > h.n_slots)) return -1;
    sv_status st;
    Py_BEGIN_ALLOW_THREADS;
    st = g_history(tokens, ldt, lens, int32_t(n), slots, int32_t(B), prompt, reset, h.V,
                   int32_t(h.n_slots), h.counts, h.ldc, h.prompt, h.output, h.ldb, status, stream);
    Py_END_ALLOW_THREADS;
    return st;
  });
}

// logits, row0, draft_row0, draft_len, max_draft_len, draft_tokens, first_row, bonus_row, slots,
// counts, prompt_bits, output_bits, repetition, presence, frequency, bias_start, bias_tokens,
// bias_values, mask, mask_row, out, status, stream
PyObject* process_logits(PyObject*, PyObject* const* a, Py_ssize_t n_args) {
  if (n_args != 23) return answer(-1);
  return guarded([&]() -> long {
    Call c;
    if (!THPVariable_Check(a[0])) return -1;
    const at::ScalarType type = THPVariable_Unpack(a[0]).scalar_type();
    if (type != at::kBFloat16 && type != at::kFloat) return -1;
    int64_t rows, V, ld, r2, v2, ldo, B = 0, any;
    const void* logits = c.mat<void>(a[0], type, &rows, &V, &ld);
    void* out = c.mat<void>(a[20], type, &r2, &v2, &ldo);
    if (!c.ok || r2 != rows || v2 != V) return -1;
    if (a[3] == Py_None) return -1;
    const int32_t* draft_len = c.vec<int32_t>(a[3], at::kInt, -1, &B);
    const int64_t* row0 = c.vec<int64_t>(a[1], at::kLong, B);
    const int64_t* draft_row0 = c.vec<int64_t>(a[2], at::kLong, B);
    const int32_t* tokens = c.vec<int32_t>(a[5], at::kInt, -1, &any);
    const float* rep = c.vec<float>(a[12], at::kFloat, B);
    const float* pres = c.vec<float>(a[13], at::kFloat, B);
    const float* freq = c.vec<float>(a[14], at::kFloat, B);
    History h;
    const int32_t* slots = nullptr;
    if (rep || pres || freq) {
      h = history(c, a[9], a[10], a[11]);
      slots = c.vec<int32_t>(a[8], at::kInt, B);
      c.ok = c.ok && h.V == V && (slots || B <= h.n_slots);
    }
    const int32_t *bias_start = c.vec<int32_t>(a[15], at::kInt, B + 1), *bias_tokens = nullptr;
    const float* bias_values = nullptr;
    int64_t n_bias = 0;
    if (bias_start) {
      if (a[16] == Py_None || a[17] == Py_None) return -1;
      bias_tokens = c.vec<int32_t>(a[16], at::kInt, -1, &n_bias);
      bias_values = c.vec<float>(a[17], at::kFloat, n_bias);
    }
    const int32_t* mask_row = c.vec<int32_t>(a[19], at::kInt, rows);
    const uint32_t* mask = nullptr;
    int64_t n_mask = 0, words, ldm = 0;
    if (mask_row) {
      mask = c.mat<uint32_t>(a[18], at::kInt, &n_mask, &words, &ldm);
      c.ok = c.ok && words >= (V + 31) / 32 && n_mask <= INT32_MAX;
    }
    int32_t* status = c.vec<int32_t>(a[21], at::kInt, -1);
    const int32_t gmax = c.num32(a[4]), first = c.num32(a[6]), bonus = c.flag(a[7]);
    void* stream = c.stream(a[22]);
    if (!c.ok || B > INT32_MAX) return -1;
    sv_status st;
    Py_BEGIN_ALLOW_THREADS;
    st = g_process(logits, ld, out, ldo, type == at::kBFloat16 ? SV_BF16 : SV_F32, V, row0,
                   draft_row0, draft_len, gmax, first, bonus, tokens, int32_t(B), slots,
                   int32_t(h.n_slots), h.counts, h.ldc, h.prompt, h.output, h.ldb, rep, pres, freq,
                   bias_start, bias_tokens, bias_values, n_bias, mask, ldm, int32_t(n_mask),
                   mask_row, status, stream);
    Py_END_ALLOW_THREADS;
    return st;
  });
}

int64_t packed_row(int64_t H) { return (H + 31) / 32 * 16; }
int64_t scale_bytes(int64_t rows, int64_t H, int32_t format) {
  return (rows + 127) / 128 * ((H + 255) / 256) * (format == SV_FP4_E8M0_32 ? 1024 : 2048);
}

// An operand's packed rows and scales: contiguous bytes of the right number.
struct Operand {
  uint8_t *packed, *scales;
  float* row;
};

Operand operand(Call& c, PyObject* packed, PyObject* scales, PyObject* row, int64_t rows,
                int64_t H, int32_t format) {
  Operand o = {};
  int64_t n = 0;
  if (packed == Py_None || scales == Py_None || H < 1 ||
      (format != SV_FP4_E8M0_32 && format != SV_FP4_E4M3_16)) {
    c.ok = false;
    return o;
  }
  o.packed = c.vec<uint8_t>(packed, at::kByte, -1, &n);
  if (c.ok) {
    const at::Tensor& t = THPVariable_Unpack(packed);
    c.ok = t.dim() == 2 && t.size(0) == rows && t.size(1) == packed_row(H);
  }
  o.scales = c.vec<uint8_t>(scales, at::kByte, -1, &n);
  c.ok = c.ok && n == scale_bytes(rows, H, format);
  if (format == SV_FP4_E4M3_16) {
    o.row = c.vec<float>(row, at::kFloat, rows);
    c.ok = c.ok && (o.row || rows == 0);
  }
  return o;
}

// x, fmt, packed, scales, row_scales, values, status, stream
PyObject* quantize_fp4(PyObject*, PyObject* const* a, Py_ssize_t n_args) {
  if (n_args != 8) return answer(-1);
  return guarded([&]() -> long {
    Call c;
    if (!THPVariable_Check(a[0])) return -1;
    const at::ScalarType type = THPVariable_Unpack(a[0]).scalar_type();
    if (type != at::kBFloat16 && type != at::kFloat) return -1;
    int64_t rows, H, ldx, r2, h2, ldv = 0;
    const void* x = c.mat<void>(a[0], type, &rows, &H, &ldx);
    if (!c.ok) return -1;
    const int32_t format = c.num32(a[1]);
    const Operand o = operand(c, a[2], a[3], a[4], rows, H, format);
    void* values = nullptr;
    if (a[5] != Py_None) {
      values = c.mat<void>(a[5], at::kBFloat16, &r2, &h2, &ldv);
      c.ok = c.ok && r2 == rows && h2 == H;
    }
    int32_t* status = c.vec<int32_t>(a[6], at::kInt, -1);
    void* stream = c.stream(a[7]);
    if (!c.ok) return -1;
    sv_status st;
    Py_BEGIN_ALLOW_THREADS;
    st = g_quantize(x, type == at::kBFloat16 ? SV_BF16 : SV_F32, rows, H, ldx, format, o.packed,
                    o.scales, o.row, values, ldv, status, stream);
    Py_END_ALLOW_THREADS;
    return st;
  });
}

// x packed, scales, row_scales, M, w packed, scales, row_scales, V, H, fmt, out, status, stream
PyObject* project_fp4(PyObject*, PyObject* const* a, Py_ssize_t n_args) {
  if (n_args != 13) return answer(-1);
  return guarded([&]() -> long {
    Call c;
    const int64_t M = c.num(a[3]), V = c.num(a[7]), H = c.num(a[8]);
    const int32_t format = c.num32(a[9]);
    if (!c.ok || M < 0 || V < 1) return -1;
    const Operand x = operand(c, a[0], a[1], a[2], M, H, format);
    const Operand w = operand(c, a[4], a[5], a[6], V, H, format);
    if (!c.ok || !THPVariable_Check(a[10])) return -1;
    const at::ScalarType type = THPVariable_Unpack(a[10]).scalar_type();
    if (type != at::kBFloat16 && type != at::kFloat) return -1;
    int64_t rows, cols, ld;
    void* out = c.mat<void>(a[10], type, &rows, &cols, &ld);
    c.ok = c.ok && rows == M && cols == V;
    int32_t* status = c.vec<int32_t>(a[11], at::kInt, -1);
    void* stream = c.stream(a[12]);
    if (!c.ok) return -1;
    sv_status st;
    Py_BEGIN_ALLOW_THREADS;
    st = g_project(x.packed, x.scales, x.row, M, w.packed, w.scales, w.row, V, H, format, out,
                   type == at::kBFloat16 ? SV_BF16 : SV_F32, ld, status, stream);
    Py_END_ALLOW_THREADS;
    return st;
  });
}

// Addresses of spec_history_append, spec_process_logits, spec_quantize_fp4, spec_project_fp4.
PyObject* bind(PyObject*, PyObject* const* a, Py_ssize_t n_args) {
  void* at[4];
  if (n_args != 4) {
    PyErr_SetString(PyExc_TypeError, "bind takes four addresses");
    return nullptr;
  }
  for (int i = 0; i < 4; ++i) {
    at[i] = PyLong_AsVoidPtr(a[i]);
    if (!at[i]) {
      if (!PyErr_Occurred()) PyErr_SetString(PyExc_ValueError, "null address");
      return nullptr;
    }
  }
  g_history = reinterpret_cast<decltype(g_history)>(at[0]);
  g_process = reinterpret_cast<decltype(g_process)>(at[1]);
  g_quantize = reinterpret_cast<decltype(g_quantize)>(at[2]);
  g_project = reinterpret_cast<decltype(g_project)>(at[3]);
  Py_RETURN_NONE;
}

#define FAST(name) \
  {#name, reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(name)), METH_FASTCALL, nullptr}
PyMethodDef methods[] = {FAST(bind),         FAST(history_append), FAST(process_logits),
                         FAST(quantize_fp4), FAST(project_fp4),    {nullptr, nullptr, 0, nullptr}};

PyModuleDef module = {PyModuleDef_HEAD_INIT, "_fastcall", nullptr, -1, methods};

}  // namespace

PyMODINIT_FUNC PyInit__fastcall() { return PyModule_Create(&module); }
