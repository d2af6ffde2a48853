// pa_torch.cpp -- the 8-bit cache calls on torch tensors without the
// interpreter between the tensors and the library: a small batch's kernels take
// 3 to 10 us, and reading eleven tensors' pointers, types and shapes from Python
// as much again (11 us of host time a call, 3 to 4 here, the launches included).
//
// Each function takes the tensors as the Python call of the same name does
// (positional, everything given), checks them and calls the library on the
// current stream.  It returns the library's code, or None where anything is
// not as the plain case has it (a type, a device, a shape, a stride): the
// caller then takes its own way, which names what is wrong.
#include <Python.h>

#include <c10/cuda/CUDAFunctions.h>
#include <c10/cuda/CUDAStream.h>
#include <torch/csrc/autograd/python_variable.h>

#include "../../include/pagedkv.h"

namespace {

constexpr int64_t kHq = PA_NUM_Q_HEADS, kHkv = PA_NUM_KV_HEADS, kD = PA_HEAD_DIM;

decltype(&pa_kv_append_rope_q8) g_append = nullptr;
decltype(&pa_prefill_append_rope_q8) g_prefill_append = nullptr;
decltype(&pa_decode_attention_q8) g_decode = nullptr;
decltype(&pa_prefill_attention_q8) g_prefill = nullptr;

// Reads a call's arguments; `ok` goes false at the first that is not plain.
struct Reader {
  PyObject *const *args;
  int dev;
  bool ok = true;

  const at::Tensor *tensor(int i) {
    if (!ok || !THPVariable_CheckExact(args[i])) {
      ok = false;
      return nullptr;
    }
    const at::Tensor &t = THPVariable_Unpack(args[i]);
    if (!t.is_cuda() || t.get_device() != dev || !t.is_contiguous()) ok = false;
    return &t;
  }
  template <class T>
  T *ptr(int i, at::ScalarType type, at::IntArrayRef shape) {
    const at::Tensor *t = tensor(i);
    if (!ok || t->scalar_type() != type || t->sizes() != shape) {
      ok = false;
      return nullptr;
    }
    return static_cast<T *>(t->data_ptr());
  }
  // at least n elements, whatever the shape
  template <class T>
  T *flat(int i, at::ScalarType type, int64_t n) {
    const at::Tensor *t = tensor(i);
    if (!ok || t->scalar_type() != type || t->numel() < n) {
      ok = false;
      return nullptr;
    }
    return static_cast<T *>(t->data_ptr());
  }
  uint16_t *bf16(int i, at::IntArrayRef shape) { return ptr<uint16_t>(i, at::kBFloat16, shape); }
  int layer(int i) {
    const long v = ok ? PyLong_AsLong(args[i]) : 0;
    if (ok && v == -1 && PyErr_Occurred()) {
      PyErr_Clear();
      ok = false;
    }
    if (v < -1 || v > INT_MAX) ok = false;
    return static_cast<int>(v);
  }
  float real(int i) {
    const double v = ok ? PyFloat_AsDouble(args[i]) : 0;
    if (ok && v == -1 && PyErr_Occurred()) {
      PyErr_Clear();
      ok = false;
    }
    return static_cast<float>(v);
  }
};

// kv_cache, kv_scales and block_table at i, i + 1 and j.
struct Cache {
  uint8_t *kv = nullptr;
  float *scales = nullptr;
  int32_t *table = nullptr;
  int64_t blocks = 0, page = 0, rows = 0, layers = 0, width = 0;
  Cache(Reader &r, int i, int j) {
    const at::Tensor *t = r.tensor(i);
    if (!r.ok) return;
    if ((t->scalar_type() != at::kFloat8_e4m3fn && t->scalar_type() != at::kByte) || t->dim() != 5 ||
        t->size(1) != 2 || t->size(3) != kHkv || t->size(4) != kD) {
      r.ok = false;
      return;
    }
    kv = static_cast<uint8_t *>(t->data_ptr());
    blocks = t->size(0);
    page = t->size(2);
    scales = r.ptr<float>(i + 1, at::kFloat, {blocks, 2, kHkv});
    const at::Tensor *b = r.tensor(j);
    if (!r.ok || b->scalar_type() != at::kInt || b->dim() != 3) {
      r.ok = false;
      return;
    }
    table = static_cast<int32_t *>(b->data_ptr());
    rows = b->size(0);
    layers = b->size(1);
    width = b->size(2);
    for (int64_t x : {blocks, page, rows, layers, width})
      if (x > INT_MAX) r.ok = false;
  }
};

PyObject *answer(bool ok, int rc) {
  if (!ok) Py_RETURN_NONE;
  return PyLong_FromLong(rc);
}

int64_t rows_of(PyObject *o) {
  if (!THPVariable_CheckExact(o)) return -1;
  const at::Tensor &t = THPVariable_Unpack(o);
  return t.dim() > 0 && t.size(0) <= INT_MAX ? t.size(0) : -1;
}

// k, v, q, q_out, [cu_tokens,] kv_cache, kv_scales, block_table, context_lens,
// layer, free_list, free_count, err (q and q_out: a tensor)
PyObject *append_call(PyObject *const *args, Py_ssize_t n_args, bool prompt) {
  const int o = prompt ? 5 : 4;   // kv_cache
  if (n_args != o + 8) Py_RETURN_NONE;
  try {
    Reader r{args, static_cast<int>(c10::cuda::current_device())};
    const Cache c(r, o, o + 2);
    const int64_t rows = prompt ? rows_of(args[0]) : c.rows;
    if (!r.ok || rows < 0) Py_RETURN_NONE;
    uint16_t *k = r.bf16(0, {rows, kHkv, kD}), *v = r.bf16(1, {rows, kHkv, kD});
    uint16_t *q = r.bf16(2, {rows, kHq, kD}), *q_out = r.bf16(3, {rows, kHq, kD});
    int32_t *cu = prompt ? r.ptr<int32_t>(4, at::kInt, {c.rows + 1}) : nullptr;
    int32_t *ctx = r.flat<int32_t>(o + 3, at::kInt, c.rows);
    const int layer = r.layer(o + 4);
    int32_t *list = r.flat<int32_t>(o + 5, at::kInt, c.blocks);
    int32_t *count = r.flat<int32_t>(o + 6, at::kInt, 1), *err = r.flat<int32_t>(o + 7, at::kInt, 1);
    if (!r.ok) Py_RETURN_NONE;
    void *st = c10::cuda::getCurrentCUDAStream(r.dev).stream();
    const int blocks = static_cast<int>(c.blocks), page = static_cast<int>(c.page),
              layers = static_cast<int>(c.layers), width = static_cast<int>(c.width),
              seqs = static_cast<int>(c.rows);
    const int rc =
        prompt ? g_prefill_append(k, v, q, q_out, static_cast<int>(rows), cu, c.kv, c.scales, blocks,
                                  page, c.table, layers, width, ctx, seqs, layer, list, count, err, st)
               : g_append(k, v, q, q_out, c.kv, c.scales, blocks, page, c.table, layers, width, ctx,
                          seqs, layer, list, count, err, st);
    return answer(true, rc);
  } catch (...) {
    Py_RETURN_NONE;   // (a torch error: the caller's way meets it too)
  }
}

PyObject *append(PyObject *, PyObject *const *args, Py_ssize_t n) { return append_call(args, n, false); }
PyObject *prefill_append(PyObject *, PyObject *const *args, Py_ssize_t n) {
  return append_call(args, n, true);
}

// out, q, kv_cache, kv_scales, block_table, context_lens, layer, scale, workspace, err
PyObject *decode(PyObject *, PyObject *const *args, Py_ssize_t n_args) {
  if (n_args != 10) Py_RETURN_NONE;
  try {
    Reader r{args, static_cast<int>(c10::cuda::current_device())};
    const Cache c(r, 2, 4);
    const at::Tensor *ts[2] = {r.tensor(0), r.tensor(1)};
    if (!r.ok) Py_RETURN_NONE;
    for (const at::Tensor *t : ts)
      if (t->scalar_type() != at::kBFloat16 || t->dim() != 3 || t->size(0) < c.rows ||
          t->size(1) != kHq || t->size(2) != kD)
        Py_RETURN_NONE;
    int32_t *ctx = r.flat<int32_t>(5, at::kInt, c.rows);
    const int layer = r.layer(6);
    const float scale = r.real(7);
    const at::Tensor *ws = r.tensor(8);
    int32_t *err = r.flat<int32_t>(9, at::kInt, 1);
    if (!r.ok) Py_RETURN_NONE;
    return answer(true, g_decode(static_cast<uint16_t *>(ts[0]->data_ptr()),
                                 static_cast<uint16_t *>(ts[1]->data_ptr()), c.kv, c.scales,
                                 static_cast<int>(c.blocks), static_cast<int>(c.page), c.table,
                                 static_cast<int>(c.layers), static_cast<int>(c.width), ctx,
                                 static_cast<int>(c.rows), layer, scale, ws->data_ptr(),
                                 static_cast<size_t>(ws->nbytes()), err,
                                 c10::cuda::getCurrentCUDAStream(r.dev).stream()));
  } catch (...) {
    Py_RETURN_NONE;
  }
}

// out, q, cu_tokens, kv_cache, kv_scales, block_table, context_lens, layer, scale, err
PyObject *prefill(PyObject *, PyObject *const *args, Py_ssize_t n_args) {
  if (n_args != 10) Py_RETURN_NONE;
  try {
    Reader r{args, static_cast<int>(c10::cuda::current_device())};
    const Cache c(r, 3, 5);
    const int64_t rows = rows_of(args[1]);
    if (!r.ok || rows < 0) Py_RETURN_NONE;
    uint16_t *out = r.bf16(0, {rows, kHq, kD}), *q = r.bf16(1, {rows, kHq, kD});
    int32_t *cu = r.ptr<int32_t>(2, at::kInt, {c.rows + 1});
    int32_t *ctx = r.flat<int32_t>(6, at::kInt, c.rows);
    const int layer = r.layer(7);
    const float scale = r.real(8);
    int32_t *err = r.flat<int32_t>(9, at::kInt, 1);
    if (!r.ok) Py_RETURN_NONE;
    return answer(true, g_prefill(out, q, static_cast<int>(rows), cu, c.kv, c.scales,
                                  static_cast<int>(c.blocks), static_cast<int>(c.page), c.table,
                                  static_cast<int>(c.layers), static_cast<int>(c.width), ctx,
                                  static_cast<int>(c.rows), layer, scale, err,
                                  c10::cuda::getCurrentCUDAStream(r.dev).stream()));
  } catch (...) {
    Py_RETURN_NONE;
  }
}

// The addresses of the library's four functions (the library is loaded once, by
// the caller).
PyObject *bind(PyObject *, PyObject *const *args, Py_ssize_t n_args) {
  void *f[4];
  if (n_args != 4) {
    PyErr_SetString(PyExc_TypeError, "bind takes four addresses");
    return nullptr;
  }
  for (int i = 0; i < 4; ++i)
    if (!(f[i] = PyLong_AsVoidPtr(args[i]))) {
      if (!PyErr_Occurred()) PyErr_SetString(PyExc_ValueError, "an address is 0");
      return nullptr;
    }
  g_append = reinterpret_cast<decltype(g_append)>(f[0]);
  g_prefill_append = reinterpret_cast<decltype(g_prefill_append)>(f[1]);
  g_decode = reinterpret_cast<decltype(g_decode)>(f[2]);
  g_prefill = reinterpret_cast<decltype(g_prefill)>(f[3]);
  Py_RETURN_NONE;
}

#define FAST(f) reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(f))
PyMethodDef kMethods[] = {{"bind", FAST(bind), METH_FASTCALL, nullptr},
                          {"append", FAST(append), METH_FASTCALL, nullptr},
                          {"prefill_append", FAST(prefill_append), METH_FASTCALL, nullptr},
                          {"decode", FAST(decode), METH_FASTCALL, nullptr},
                          {"prefill", FAST(prefill), METH_FASTCALL, nullptr},
                          {nullptr, nullptr, 0, nullptr}};
PyModuleDef kModule = {PyModuleDef_HEAD_INIT, "_pa_torch", nullptr, -1, kMethods,
                       nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__pa_torch() { return PyModule_Create(&kModule); }
