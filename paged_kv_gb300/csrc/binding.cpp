// The Python side of the serving operators' calls: checks of tensors and the
// unpacking of some two dozen arguments, which as Python code takes longer than
// the small calls' kernels.  Everything else is the C ABI's.  Each function
// takes its arguments by position, returns the C status, and raises TypeError or
// ValueError for a tensor the ABI cannot be given.

#include <Python.h>

#include <c10/cuda/CUDAStream.h>
#include <cuda_runtime_api.h>
#include <torch/csrc/autograd/python_variable.h>

#include <cmath>
#include <cstdint>

#include "../../include/pkv.h"

namespace {

// What a function unpacks; `bad` once an exception is set.  Every tensor has to be
// on GPU `device`, once that is known.
struct Args {
  PyObject* const* a;
  bool bad = false;
  int device = -1;

  template <typename... X>
  void fail(PyObject* type, const char* fmt, X... x) {
    if (!bad) PyErr_Format(type, fmt, x...);
    bad = true;
  }
  const at::Tensor* tensor(int i, const char* name) {
    if (bad) return nullptr;
    if (!THPVariable_Check(a[i])) {
      fail(PyExc_TypeError, "%s must be a CUDA tensor", name);
      return nullptr;
    }
    const at::Tensor& t = THPVariable_Unpack(a[i]);
    if (!t.is_cuda()) {
      fail(PyExc_TypeError, "%s must be a CUDA tensor", name);
      return nullptr;
    }
    if (device >= 0 && t.get_device() != device) {
      fail(PyExc_ValueError, "%s is on cuda:%d, not on cuda:%d", name,
           static_cast<int>(t.get_device()), device);
      return nullptr;
    }
    return &t;
  }
  bool none(int i) const { return a[i] == Py_None; }

  // Pointer of a contiguous tensor of at least n elements, or of None.
  template <typename P>
  P* flat(int i, at::ScalarType dtype, const char* name, int64_t n) {
    if (none(i)) return nullptr;
    const at::Tensor* t = tensor(i, name);
    if (t == nullptr) return nullptr;
    if (t->scalar_type() != dtype) {
      fail(PyExc_TypeError, "%s must be %s, got %s", name, c10::toString(dtype),
           c10::toString(t->scalar_type()));
    } else if (!t->is_contiguous()) {
      fail(PyExc_ValueError, "%s must be contiguous", name);
    } else if (t->numel() < n) {
      fail(PyExc_ValueError, "%s has %lld elements, needs %lld", name, (long long)t->numel(),
           (long long)n);
    }
    return bad ? nullptr : static_cast<P*>(t->data_ptr());
  }
  // The same of a matrix, and its shape (0, 0 for None).
  template <typename P>
  P* matrix(int i, at::ScalarType dtype, const char* name, int64_t* rows, int64_t* cols) {
    *rows = *cols = 0;
    P* p = flat<P>(i, dtype, name, 0);
    if (bad || none(i)) return p;
    const at::Tensor& t = THPVariable_Unpack(a[i]);
    if (t.dim() != 2) {
      fail(PyExc_ValueError, "%s must be 2-D", name);
      return nullptr;
    }
    *rows = t.size(0);
    *cols = t.size(1);
    return p;
  }
  // A [tokens, heads, head_dim] tensor of 16-bit elements.
  struct Rows {
    void* p = nullptr;
    int64_t token = 0, head = 0;
    int64_t n = 0, heads = 0;
    pkv_dtype dt = PKV_BF16;
  };
  Rows rows(int i, const char* name, int64_t n, int64_t heads, int64_t dim) {
    Rows r;
    const at::Tensor* t = tensor(i, name);
    if (t == nullptr) return r;
    if (t->scalar_type() == at::kBFloat16) {
      r.dt = PKV_BF16;
    } else if (t->scalar_type() == at::kHalf) {
      r.dt = PKV_FP16;
    } else {
      fail(PyExc_TypeError, "%s dtype %s is not bf16 or fp16", name,
           c10::toString(t->scalar_type()));
      return r;
    }
    if (t->dim() != 3 || (n >= 0 && t->size(0) != n) || (heads >= 0 && t->size(1) != heads) ||
        t->size(2) != dim || (t->stride(2) != 1 && t->size(2) > 1)) {
      fail(PyExc_ValueError, "%s must be [%s, %s, %lld] with unit last stride", name,
           n >= 0 ? "the tokens" : "tokens", heads >= 0 ? "the heads" : "heads", (long long)dim);
      return r;
    }
    r.p = t->data_ptr();
    r.n = t->size(0);
    r.heads = t->size(1);
    // The stride of a dimension of one is never used, and may hold any value.
    r.token = r.n > 1 ? t->stride(0) : 0;
    r.head = r.heads > 1 ? t->stride(1) : 0;
    return r;
  }
  int64_t integer(int i, const char* name) {
    if (bad) return 0;
    const long long x = PyLong_AsLongLong(a[i]);
    if (x == -1 && PyErr_Occurred()) bad = true;
    return x;
  }
  int int32(int i, const char* name) {
    const int64_t x = integer(i, name);
    if (!bad && (x < INT32_MIN || x > INT32_MAX)) fail(PyExc_ValueError, "%s is out of range", name);
    return static_cast<int>(x);
  }
  // A stream object, an integer handle, or None for the device's current one.
  pkv_stream_t stream(int i) {
    if (bad) return nullptr;
    if (none(i))
      return reinterpret_cast<pkv_stream_t>(c10::cuda::getCurrentCUDAStream(device).stream());
    PyObject* h = PyObject_GetAttrString(a[i], "cuda_stream");
    if (h == nullptr) {
      PyErr_Clear();
      h = a[i];
      Py_INCREF(h);
    }
    void* p = PyLong_AsVoidPtr(h);
    Py_DECREF(h);
    if (PyErr_Occurred()) bad = true;
    return static_cast<pkv_stream_t>(p);
  }
  const pkv_kv_cache* cache(int i) {
    return bad ? nullptr : static_cast<const pkv_kv_cache*>(PyLong_AsVoidPtr(a[i]));
  }
};

bool arity(Py_ssize_t n, Py_ssize_t want) {
  if (n == want) return true;
  PyErr_Format(PyExc_TypeError, "%zd arguments, expected %zd", n, want);
  return false;
}

// (cache, device, k, v, positions, out_loc, cos_sin, interleaved, q, q_out,
//  total_tokens, status, stream)
PyObject* append_kv(PyObject*, PyObject* const* a, Py_ssize_t n) {
  if (!arity(n, 13)) return nullptr;
  Args g{a};
  const pkv_kv_cache* c = g.cache(0);
  if (c == nullptr) return nullptr;
  g.device = g.int32(1, "device");
  const auto k = g.rows(2, "k", -1, c->kv_heads, c->head_dim);
  const auto v = g.rows(3, "v", k.n, c->kv_heads, c->head_dim);
  const auto* pos = g.flat<int32_t>(4, at::kInt, "positions", k.n);
  const auto* loc = g.flat<int32_t>(5, at::kInt, "out_loc", k.n);
  int64_t max_pos, rot;
  const auto* cs = g.matrix<float>(6, at::kFloat, "cos_sin", &max_pos, &rot);
  const int inter = g.int32(7, "interleaved");
  Args::Rows q, o;
  if (!g.none(8)) {
    q = g.rows(8, "q", k.n, -1, c->head_dim);
    o = g.rows(9, "q_out", k.n, q.heads, c->head_dim);
    if (!g.bad && (q.dt != k.dt || o.dt != k.dt))
      g.fail(PyExc_TypeError, "q and q_out must have k's dtype");
  } else if (!g.none(9)) {
    g.fail(PyExc_ValueError, "q_out given without q");
  }
  if (!g.bad && v.dt != k.dt) g.fail(PyExc_TypeError, "v must have k's dtype");
  const auto* total = g.flat<int64_t>(10, at::kLong, "total_tokens", 1);
  auto* status = g.flat<int32_t>(11, at::kInt, "status", 1);
  const pkv_stream_t s = g.stream(12);
  if (g.bad) return nullptr;
  return PyLong_FromLong(pkv_append_kv(
      c, k.p, k.token, k.head, v.p, v.token, v.head, k.dt, k.n, total, pos, loc, cs, max_pos,
      static_cast<int>(rot), inter, q.p, q.token, q.head, static_cast<int>(q.heads), o.p, o.token,
      o.head, status, s));
}

// (cache, device, q, out, lse, cached_len, device_len, table_idx, kv_begin,
//  max_q_len, page_table, sm_scale, window, status, workspace, stream, default)
// `default` is None, or the dict of the wrapper's own workspaces, with `workspace`
// None: by stream and device, each of them large enough for any call.  Where
// there is none, or the stream is being captured, (bytes needed, the stream's
// handle, the key, the capture's id or 0) comes back and nothing is launched.
PyObject* paged_attention(PyObject*, PyObject* const* a, Py_ssize_t n) {
  if (!arity(n, 17)) return nullptr;
  Args g{a};
  const pkv_kv_cache* c = g.cache(0);
  if (c == nullptr) return nullptr;
  g.device = g.int32(1, "device");
  const auto q = g.rows(2, "q", -1, -1, c->head_dim);
  const auto o = g.rows(3, "out", q.n, q.heads, c->head_dim);
  if (!g.bad && o.dt != q.dt) g.fail(PyExc_TypeError, "out must have q's dtype");
  auto* lse = g.flat<float>(4, at::kFloat, "lse", q.n * q.heads);
  const at::Tensor* lens = g.tensor(5, "cached_len");
  const int64_t b = lens != nullptr ? lens->numel() : 0;
  const auto* cached = g.flat<int32_t>(5, at::kInt, "cached_len", b);
  const auto* dev = g.flat<int32_t>(6, at::kInt, "device_len", b);
  const auto* table = g.flat<int32_t>(7, at::kInt, "table_idx", b);
  const auto* begin = g.flat<int32_t>(8, at::kInt, "kv_begin", b);
  const int max_q = g.int32(9, "max_q_len");
  int64_t rows, cols;
  const auto* pt = g.matrix<int32_t>(10, at::kInt, "page_table", &rows, &cols);
  double scale = 1.0 / std::sqrt(static_cast<double>(c->head_dim));
  if (!g.bad && !g.none(11)) {
    scale = PyFloat_AsDouble(a[11]);
    if (scale == -1.0 && PyErr_Occurred()) g.bad = true;
  }
  const int window = g.int32(12, "window");
  auto* status = g.flat<int32_t>(13, at::kInt, "status", 1);
  auto* ws = g.flat<uint8_t>(14, at::kByte, "workspace", 0);
  const pkv_stream_t s = g.stream(15);
  if (g.bad) return nullptr;
  if (b > INT32_MAX) {
    PyErr_SetString(PyExc_ValueError, "cached_len is too long");
    return nullptr;
  }
  size_t have = ws != nullptr ? THPVariable_Unpack(a[14]).numel() : 0;
  if (!g.none(16)) {
    // (User-space addresses have 48 bits at most.)
    const unsigned long long handle = reinterpret_cast<uintptr_t>(s);
    const unsigned long long key = handle << 8 | static_cast<unsigned>(g.device);
    cudaStreamCaptureStatus capture = cudaStreamCaptureStatusNone;
    unsigned long long id = 0;
    if (cudaStreamGetCaptureInfo(reinterpret_cast<cudaStream_t>(s), &capture, &id) != cudaSuccess ||
        capture == cudaStreamCaptureStatusNone)
      id = 0;
    PyObject* name = PyLong_FromUnsignedLongLong(key);
    if (name == nullptr) return nullptr;
    PyObject* own = id == 0 ? PyDict_GetItemWithError(a[16], name) : nullptr;  // borrowed
    Py_DECREF(name);
    if (own == nullptr) {
      if (PyErr_Occurred()) return nullptr;
      const size_t need = pkv_paged_attention_workspace_bytes(
          static_cast<int>(b), q.n, max_q, static_cast<int>(q.heads), c->kv_heads, c->head_dim);
      return Py_BuildValue("(KKKK)", static_cast<unsigned long long>(need), handle, key, id);
    }
    if (!THPVariable_Check(own)) {
      PyErr_SetString(PyExc_TypeError, "the default workspace is no tensor");
      return nullptr;
    }
    ws = static_cast<uint8_t*>(THPVariable_Unpack(own).data_ptr());
    have = THPVariable_Unpack(own).numel();
  }
  return PyLong_FromLong(pkv_paged_attention(
      c, q.p, q.token, q.head, static_cast<int>(q.heads), q.dt, q.n, o.p, o.token, o.head, lse,
      cached, dev, table, begin, static_cast<int>(b), max_q, pt, rows, cols,
      static_cast<float>(scale), window, status, ws, have, s));
}

// (logits, out, token_pool, table_idx, prompt_len, device_len, repetition,
//  presence, frequency, bias_ptr, bias_ids, bias_values, mask, status, stream)
PyObject* adjust_logits(PyObject*, PyObject* const* a, Py_ssize_t n) {
  if (!arity(n, 15)) return nullptr;
  Args g{a};
  const at::Tensor* x = THPVariable_Check(a[0]) ? &THPVariable_Unpack(a[0]) : nullptr;
  if (x == nullptr || !x->is_cuda() || x->dim() != 2 || (x->stride(1) != 1 && x->size(1) > 1)) {
    PyErr_SetString(PyExc_ValueError, "logits must be a 2-D CUDA tensor with unit column stride");
    return nullptr;
  }
  pkv_dtype dt = PKV_FP32;
  if (x->scalar_type() == at::kBFloat16) {
    dt = PKV_BF16;
  } else if (x->scalar_type() != at::kFloat) {
    PyErr_Format(PyExc_TypeError, "logits dtype %s is not fp32 or bf16",
                 c10::toString(x->scalar_type()));
    return nullptr;
  }
  g.device = static_cast<int>(x->get_device());
  const int64_t b = x->size(0), v = x->size(1);
  const at::Tensor* o = THPVariable_Check(a[1]) ? &THPVariable_Unpack(a[1]) : nullptr;
  if (o == nullptr || !o->is_cuda() || o->get_device() != g.device ||
      o->scalar_type() != x->scalar_type() || o->dim() != 2 || o->size(0) != b ||
      o->size(1) != v || (o->stride(1) != 1 && v > 1)) {
    PyErr_SetString(PyExc_ValueError,
                    "out must be a tensor of the logits' GPU, shape and dtype with unit column stride");
    return nullptr;
  }
  int64_t pr, pc;
  const auto* pool = g.matrix<int32_t>(2, at::kInt, "token_pool", &pr, &pc);
  const auto* table = g.flat<int32_t>(3, at::kInt, "table_idx", b);
  const auto* prompt = g.flat<int32_t>(4, at::kInt, "prompt_len", b);
  const auto* dev = g.flat<int32_t>(5, at::kInt, "device_len", b);
  const auto* rep = g.flat<float>(6, at::kFloat, "repetition", b);
  const auto* pres = g.flat<float>(7, at::kFloat, "presence", b);
  const auto* freq = g.flat<float>(8, at::kFloat, "frequency", b);
  const auto* ptr = g.flat<int32_t>(9, at::kInt, "bias_ptr", b + 1);
  const auto* ids = g.flat<int32_t>(10, at::kInt, "bias_ids", 0);
  const int64_t nb = !g.bad && !g.none(10) ? THPVariable_Unpack(a[10]).numel() : 0;
  const auto* vals = g.flat<float>(11, at::kFloat, "bias_values", nb);
  const int32_t* mask = nullptr;
  int64_t mask_stride = 0;
  if (!g.none(12)) {
    const at::Tensor* m = g.tensor(12, "mask");
    if (m != nullptr) {
      if (m->dim() != 2 || m->scalar_type() != at::kInt || (m->stride(1) != 1 && m->size(1) > 1) ||
          m->size(0) < b || m->size(1) < (v + 31) / 32)
        g.fail(PyExc_ValueError, "mask must be a CUDA int32 tensor [%lld, %lld] with unit column stride",
               (long long)b, (long long)((v + 31) / 32));
      mask = static_cast<const int32_t*>(m->data_ptr());
      mask_stride = m->size(0) > 1 ? m->stride(0) : m->size(1);
    }
  }
  auto* status = g.flat<int32_t>(13, at::kInt, "status", 1);
  const pkv_stream_t s = g.stream(14);
  if (g.bad) return nullptr;
  if (b > INT32_MAX || v > INT32_MAX) {
    PyErr_SetString(PyExc_ValueError, "logits are too large");
    return nullptr;
  }
  const int64_t xs = b > 1 ? x->stride(0) : v, os = b > 1 ? o->stride(0) : v;
  return PyLong_FromLong(pkv_adjust_logits(
      x->data_ptr(), xs, dt, static_cast<int>(b), static_cast<int>(v), o->data_ptr(), os, pool, pr,
      pc, table, prompt, dev, rep, pres, freq, ptr, ids, vals, nb, mask, mask_stride, status, s));
}

// C++ exceptions (a CUDA error in the lookup of a stream, say) end here.
template <PyObject* (*F)(PyObject*, PyObject* const*, Py_ssize_t)>
PyObject* guarded(PyObject* self, PyObject* const* a, Py_ssize_t n) {
  try {
    return F(self, a, n);
  } catch (const std::exception& e) {
    PyErr_SetString(PyExc_RuntimeError, e.what());
    return nullptr;
  }
}

template <PyObject* (*F)(PyObject*, PyObject* const*, Py_ssize_t)>
PyCFunction fast() {
  return reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(&guarded<F>));
}

PyMethodDef methods[] = {
    {"append_kv", fast<append_kv>(), METH_FASTCALL, nullptr},
    {"paged_attention", fast<paged_attention>(), METH_FASTCALL, nullptr},
    {"adjust_logits", fast<adjust_logits>(), METH_FASTCALL, nullptr},
    {nullptr, nullptr, 0, nullptr},
};

PyModuleDef module = {PyModuleDef_HEAD_INIT, "_binding", nullptr, -1, methods,
                      nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__binding() { return PyModule_Create(&module); }
