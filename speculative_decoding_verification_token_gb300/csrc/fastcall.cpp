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
decltype(&spec_cache_append) g_cache_append;
decltype(&spec_tree_attention) g_attention;
decltype(&spec_tree_attention_workspace_bytes) g_attention_bytes;
decltype(&spec_tree_accept) g_accept;
decltype(&spec_cache_keep) g_keep;

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

// A tensor [rows, heads, D] with a dense last axis; the stride of an axis of one says nothing.
struct Heads {
  void* at = nullptr;
  int64_t rows = 0, heads = 0, D = 0, ld = 0, hs = 0;
};

Heads heads_of(Call& c, PyObject* o, at::ScalarType type) {
  Heads h;
  const at::Tensor* t = c.tensor(o, type);
  if (!t || t->dim() != 3 || (t->size(2) > 1 && t->stride(2) != 1)) {
    c.ok = false;
    return h;
  }
  h.rows = t->size(0), h.heads = t->size(1), h.D = t->size(2);
  h.ld = h.rows > 1 ? t->stride(0) : h.heads * h.D;
  h.hs = h.heads > 1 ? t->stride(1) : h.D;
  h.at = t->data_ptr();
  c.ok = c.ok && h.rows <= INT32_MAX && h.heads <= INT32_MAX && h.D <= INT32_MAX;
  return h;
}

// Two caches [pages, page size, heads, D] (or [layers, ...]) alike.
struct Caches {
  void *k = nullptr, *v = nullptr;
  int64_t layers = 1, pages = 0, page = 0, heads = 0, D = 0, ls = 0, ps = 0, ts = 0, hs = 0;
};

Caches caches_of(Call& c, PyObject* ko, PyObject* vo, bool layers) {
  Caches x;
  const at::Tensor *k = c.tensor(ko, at::kBFloat16), *v = c.tensor(vo, at::kBFloat16);
  if (!k || !v || (k->dim() != 4 && !(layers && k->dim() == 5)) || k->sizes() != v->sizes() ||
      k->strides() != v->strides() || (k->size(-1) > 1 && k->stride(-1) != 1)) {
    c.ok = false;
    return x;
  }
  auto stride = [&](int d) { return k->size(d) > 1 ? k->stride(d) : 0; };
  x.k = k->data_ptr(), x.v = v->data_ptr();
  x.pages = k->size(-4), x.page = k->size(-3), x.heads = k->size(-2), x.D = k->size(-1);
  x.ps = stride(-4), x.ts = stride(-3), x.hs = stride(-2);
  if (k->dim() == 5) x.layers = k->size(0), x.ls = stride(0);
  c.ok = c.ok && x.page <= INT32_MAX && x.heads <= INT32_MAX && x.D <= INT32_MAX &&
         x.layers <= INT32_MAX;
  return x;
}

// What the calls over the cache take alike: [B] lengths, a page table of B rows.
struct Table {
  int64_t B = 0, columns = 0, ld = 0;
  const int32_t *ctx_len = nullptr, *pages = nullptr;
};

Table table_of(Call& c, PyObject* lengths, PyObject* page_table, PyObject* ctx_len,
               const int32_t** length) {
  Table t;
  int64_t rows = 0;
  if (lengths == Py_None || page_table == Py_None || ctx_len == Py_None) c.ok = false;
  *length = c.vec<int32_t>(lengths, at::kInt, -1, &t.B);
  c.ok = c.ok && THPVariable_Unpack(lengths).dim() == 1;
  t.ctx_len = c.vec<int32_t>(ctx_len, at::kInt, t.B);
  if (c.ok) t.pages = c.mat<int32_t>(page_table, at::kInt, &rows, &t.columns, &t.ld);
  c.ok = c.ok && rows == t.B && t.B <= INT32_MAX && t.columns <= INT32_MAX;
  return t;
}

// q, k, v, k_cache, v_cache, page_table, ctx_len, row0, draft_len, max_draft_len, cos_sin, adjacent,
// parents, bonus_row, q_out, status, stream
PyObject* cache_append(PyObject*, PyObject* const* a, Py_ssize_t n_args) {
  if (n_args != 17) return answer(-1);
  return guarded([&]() -> long {
    Call c;
    if (!THPVariable_Check(a[1])) return -1;
    const at::ScalarType type = THPVariable_Unpack(a[1]).scalar_type();
    if (type != at::kBFloat16 && type != at::kFloat) return -1;
    const Heads k = heads_of(c, a[1], type), v = heads_of(c, a[2], type);
    Heads q, out;
    if (a[0] != Py_None) {
      q = heads_of(c, a[0], type);
      out = heads_of(c, a[14], at::kBFloat16);
      c.ok = c.ok && q.rows == k.rows && q.D == k.D && out.rows == k.rows &&
             out.heads == q.heads && out.D == k.D;
    }
    const Caches x = caches_of(c, a[3], a[4], false);
    const int32_t* length;
    const Table t = table_of(c, a[8], a[5], a[6], &length);
    if (!c.ok || v.rows != k.rows || v.heads != k.heads || v.D != k.D || x.heads != k.heads ||
        x.D != k.D || a[7] == Py_None)
      return -1;
    const int64_t* row0 = c.vec<int64_t>(a[7], at::kLong, t.B);
    const float* cos_sin = nullptr;
    int64_t positions = 0, rot = 0, ldc = 0;
    if (a[10] != Py_None) cos_sin = c.mat<float>(a[10], at::kFloat, &positions, &rot, &ldc);
    const int32_t* parents = c.vec<int32_t>(a[12], at::kInt, k.rows);
    int32_t* status = c.vec<int32_t>(a[15], at::kInt, -1);
    const int32_t gmax = c.num32(a[9]), adjacent = c.flag(a[11]), bonus = c.flag(a[13]);
    void* stream = c.stream(a[16]);
    if (!c.ok || rot > INT32_MAX) return -1;
    sv_status st;
    Py_BEGIN_ALLOW_THREADS;
    st = g_cache_append(q.at, q.ld, q.hs, k.at, k.ld, k.hs, v.at, v.ld, v.hs,
                        type == at::kBFloat16 ? SV_BF16 : SV_F32, k.rows, int32_t(q.heads),
                        int32_t(k.heads), int32_t(k.D), cos_sin, ldc, positions, int32_t(rot),
                        adjacent, row0, length, gmax, bonus, parents, int32_t(t.B), t.ctx_len,
                        t.pages, t.ld, int32_t(t.columns), out.at, out.ld, out.hs, x.k, x.v,
                        x.pages, int32_t(x.page), x.ps, x.ts, x.hs, status, stream);
    Py_END_ALLOW_THREADS;
    return st;
  });
}

// q, k_cache, v_cache, page_table, ctx_len, row0, draft_len, max_draft_len, parents, bonus_row,
// scale, out, lse, status, workspace, stream
PyObject* tree_attention(PyObject*, PyObject* const* a, Py_ssize_t n_args) {
  if (n_args != 16) return answer(-1);
  return guarded([&]() -> long {
    Call c;
    const Heads q = heads_of(c, a[0], at::kBFloat16), out = heads_of(c, a[11], at::kBFloat16);
    const Caches x = caches_of(c, a[1], a[2], false);
    const int32_t* length;
    const Table t = table_of(c, a[6], a[3], a[4], &length);
    if (!c.ok || out.rows != q.rows || out.heads != q.heads || out.D != q.D || x.D != q.D ||
        a[5] == Py_None || a[14] == Py_None)
      return -1;
    const int64_t* row0 = c.vec<int64_t>(a[5], at::kLong, t.B);
    const int32_t* parents = c.vec<int32_t>(a[8], at::kInt, q.rows);
    float* lse = nullptr;
    int64_t rows = q.rows, heads = q.heads, ldl = 0;
    if (a[12] != Py_None) lse = c.mat<float>(a[12], at::kFloat, &rows, &heads, &ldl);
    int32_t* status = c.vec<int32_t>(a[13], at::kInt, -1);
    int64_t ws_bytes = 0;
    uint8_t* ws = c.vec<uint8_t>(a[14], at::kByte, -1, &ws_bytes);
    const int32_t gmax = c.num32(a[7]), bonus = c.flag(a[9]);
    const double scale = PyFloat_AsDouble(a[10]);
    if (scale == -1.0 && PyErr_Occurred()) {
      PyErr_Clear();
      return -1;
    }
    void* stream = c.stream(a[15]);
    if (!c.ok || rows != q.rows || heads < q.heads) return -1;
    const size_t need = g_attention_bytes(int32_t(t.B), gmax, bonus, int32_t(q.heads),
                                          int32_t(x.heads), int32_t(q.D));
    if (size_t(ws_bytes) < need) return -1;
    sv_status st;
    Py_BEGIN_ALLOW_THREADS;
    st = g_attention(q.at, q.ld, q.hs, q.rows, int32_t(q.heads), int32_t(x.heads), int32_t(q.D),
                     float(scale), row0, length, gmax, bonus, parents, int32_t(t.B), t.ctx_len,
                     t.pages, t.ld, int32_t(t.columns), x.k, x.v, x.pages, int32_t(x.page), x.ps,
                     x.ts, x.hs, out.at, out.ld, out.hs, lse, ldl, status, ws, size_t(ws_bytes),
                     stream);
    Py_END_ALLOW_THREADS;
    return st;
  });
}

// sampled, draft_tokens, parents, row0, draft_row0, draft_len, max_draft_len, accepted_len,
// out_tokens, path, correction, status, stream
PyObject* tree_accept(PyObject*, PyObject* const* a, Py_ssize_t n_args) {
  if (n_args != 13) return answer(-1);
  return guarded([&]() -> long {
    Call c;
    for (int i : {0, 1, 3, 4, 5, 7, 8, 9, 10})
      if (a[i] == Py_None) return -1;
    int64_t rows = 0, drafts = 0, B = 0, r1 = 0, r2 = 0, w1 = 0, w2 = 0, ldo = 0, ldp = 0;
    const int32_t* sampled = c.vec<int32_t>(a[0], at::kInt, -1, &rows);
    const int32_t* tokens = c.vec<int32_t>(a[1], at::kInt, -1, &drafts);
    const int32_t* length = c.vec<int32_t>(a[5], at::kInt, -1, &B);
    const int32_t* parents = c.vec<int32_t>(a[2], at::kInt, rows);
    const int64_t* row0 = c.vec<int64_t>(a[3], at::kLong, B);
    const int64_t* draft_row0 = c.vec<int64_t>(a[4], at::kLong, B);
    int32_t* accepted = c.vec<int32_t>(a[7], at::kInt, B);
    int32_t* out = c.mat<int32_t>(a[8], at::kInt, &r1, &w1, &ldo);
    int32_t* path = c.mat<int32_t>(a[9], at::kInt, &r2, &w2, &ldp);
    int32_t* correction = c.vec<int32_t>(a[10], at::kInt, B);
    int32_t* status = c.vec<int32_t>(a[11], at::kInt, -1);
    const int32_t gmax = c.num32(a[6]);
    void* stream = c.stream(a[12]);
    if (!c.ok || THPVariable_Unpack(a[5]).dim() != 1 || r1 != B || r2 != B ||
        w1 < int64_t(gmax) + 1 || w2 < gmax || B > INT32_MAX)
      return -1;
    sv_status st;
    Py_BEGIN_ALLOW_THREADS;
    st = g_accept(sampled, tokens, parents, row0, draft_row0, length, gmax, int32_t(B), rows,
                  drafts, accepted, out, ldo, correction, path, ldp, status, stream);
    Py_END_ALLOW_THREADS;
    return st;
  });
}

// k_cache, v_cache, page_table, ctx_len, accepted_len, path, new_len, status, stream
PyObject* cache_keep(PyObject*, PyObject* const* a, Py_ssize_t n_args) {
  if (n_args != 9) return answer(-1);
  return guarded([&]() -> long {
    Call c;
    const Caches x = caches_of(c, a[0], a[1], true);
    const int32_t* accepted;
    const Table t = table_of(c, a[4], a[2], a[3], &accepted);
    if (!c.ok || a[6] == Py_None) return -1;
    const int32_t* path = nullptr;
    int64_t rows = t.B, n_path = INT32_MAX, ldp = 0;
    if (a[5] != Py_None) path = c.mat<int32_t>(a[5], at::kInt, &rows, &n_path, &ldp);
    int32_t* new_len = c.vec<int32_t>(a[6], at::kInt, t.B);
    int32_t* status = c.vec<int32_t>(a[7], at::kInt, -1);
    void* stream = c.stream(a[8]);
    if (!c.ok || rows != t.B || n_path > INT32_MAX) return -1;
    sv_status st;
    Py_BEGIN_ALLOW_THREADS;
    st = g_keep(accepted, path, ldp, int32_t(n_path), int32_t(t.B), t.ctx_len, t.pages, t.ld,
                int32_t(t.columns), x.k, x.v, int32_t(x.layers), x.ls, x.pages, int32_t(x.page),
                x.ps, x.ts, x.hs, int32_t(x.heads), int32_t(x.D), new_len, status, stream);
    Py_END_ALLOW_THREADS;
    return st;
  });
}

// Addresses of spec_history_append, spec_process_logits, spec_quantize_fp4, spec_project_fp4,
// spec_cache_append, spec_tree_attention and its workspace query, spec_tree_accept, spec_cache_keep.
PyObject* bind(PyObject*, PyObject* const* a, Py_ssize_t n_args) {
  void* at[9];
  if (n_args != 9) {
    PyErr_SetString(PyExc_TypeError, "bind takes nine addresses");
    return nullptr;
  }
  for (int i = 0; i < 9; ++i) {
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
  g_cache_append = reinterpret_cast<decltype(g_cache_append)>(at[4]);
  g_attention = reinterpret_cast<decltype(g_attention)>(at[5]);
  g_attention_bytes = reinterpret_cast<decltype(g_attention_bytes)>(at[6]);
  g_accept = reinterpret_cast<decltype(g_accept)>(at[7]);
  g_keep = reinterpret_cast<decltype(g_keep)>(at[8]);
  Py_RETURN_NONE;
}

#define FAST(name) \
  {#name, reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(name)), METH_FASTCALL, nullptr}
PyMethodDef methods[] = {FAST(bind),         FAST(history_append), FAST(process_logits),
                         FAST(quantize_fp4), FAST(project_fp4),    FAST(cache_append),
                         FAST(tree_attention), FAST(tree_accept),  FAST(cache_keep),
                         {nullptr, nullptr, 0, nullptr}};

PyModuleDef module = {PyModuleDef_HEAD_INIT, "_fastcall", nullptr, -1, methods};

}  // namespace

PyMODINIT_FUNC PyInit__fastcall() { return PyModule_Create(&module); }
