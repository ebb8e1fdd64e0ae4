// The quick way into the library for calls whose time on the GPU is a few microseconds: one C++ function per entry point
// that checks the tensors, takes the current stream and makes the call.  Where a check does not hold it returns None and
// has done nothing; the Python function then goes through its own checks, which name what is wrong.
#define PY_SSIZE_T_CLEAN
#include <Python.h>
#include <c10/cuda/CUDAFunctions.h>
#include <c10/cuda/CUDAStream.h>
#include <dlfcn.h>
#include <torch/csrc/autograd/python_variable.h>

#include "../../include/moe.h"

namespace {

using at::ScalarType;

decltype(&moe_quant_i8) p_quant = nullptr;
decltype(&moe_linear_i8) p_linear = nullptr;
decltype(&moe_layer_decode) p_layer = nullptr;

enum Kind { F32, I32, I8, BF16, BYTES };

bool is(ScalarType t, Kind k) {
  switch (k) {
    case F32: return t == ScalarType::Float;
    case I32: return t == ScalarType::Int;
    case I8: return t == ScalarType::Char;
    case BF16: return t == ScalarType::BFloat16 || t == ScalarType::Short || t == ScalarType::UInt16;
    case BYTES: return true;
  }
  return false;
}

// The tensor behind an argument if the library may be given its address: contiguous, on CUDA device dev, of this type and
// of at least n elements.
const at::Tensor* tensor(PyObject* o, Kind k, int64_t n, int dev) {
  if (!THPVariable_Check(o)) return nullptr;
  const at::Tensor& t = THPVariable_Unpack(o);
  if (!t.defined() || !t.is_cuda() || t.get_device() != dev || !is(t.scalar_type(), k) || t.numel() < n ||
      !t.is_contiguous())
    return nullptr;
  return &t;
}

bool address(PyObject* o, Kind k, int64_t n, int dev, void** p, bool optional = false) {
  if (o == Py_None) {
    *p = nullptr;
    return optional;
  }
  const at::Tensor* t = tensor(o, k, n, dev);
  if (!t) return false;
  *p = t->data_ptr();
  return true;
}

PyObject* none() { Py_RETURN_NONE; }

cudaStream_t stream(int dev) { return c10::cuda::getCurrentCUDAStream(static_cast<c10::DeviceIndex>(dev)).stream(); }

// The status of a call made without the interpreter's lock: a launch waits when the device's queue is full, and what it
// waits for may need another Python thread.  The arguments hold references to every tensor meanwhile.
template <class F>
PyObject* status(F call) {
  int32_t code;
  Py_BEGIN_ALLOW_THREADS
  code = call();
  Py_END_ALLOW_THREADS
  return PyLong_FromLong(code);
}

// load(path): take the entry points from the library.
PyObject* load(PyObject*, PyObject* path) {
  const char* s = PyUnicode_AsUTF8(path);
  if (!s) return nullptr;
  void* h = dlopen(s, RTLD_NOW | RTLD_LOCAL);
  if (h) {
    p_quant = reinterpret_cast<decltype(p_quant)>(dlsym(h, "moe_quant_i8"));
    p_linear = reinterpret_cast<decltype(p_linear)>(dlsym(h, "moe_linear_i8"));
    p_layer = reinterpret_cast<decltype(p_layer)>(dlsym(h, "moe_layer_decode"));
  }
  return PyBool_FromLong(p_quant && p_linear && p_layer);
}

// quant(x, q, scale, eps | None) -> status | None
PyObject* quant(PyObject*, PyObject* const* a, Py_ssize_t n) {
  if (n != 4 || !p_quant) return none();
  try {
    const int dev = c10::cuda::current_device();
    const double eps = a[3] == Py_None ? -1.0 : PyFloat_AsDouble(a[3]);
    if (PyErr_Occurred()) {
      PyErr_Clear();
      return none();
    }
    if (a[3] != Py_None && !(eps >= 0)) return none();
    const at::Tensor *x = tensor(a[0], BYTES, 0, dev), *q = tensor(a[1], I8, 0, dev);
    if (!x || !q || x->dim() != 2 || q->dim() != 2) return none();
    const bool bf = x->scalar_type() == ScalarType::BFloat16;
    if (!bf && x->scalar_type() != ScalarType::Float) return none();
    const int64_t T = x->size(0), H = x->size(1), ld = q->size(1);
    void* s;
    if (ld % 16 || ld < H || q->size(0) < T || T > MOE_MAX_TOKENS || H > MOE_I8_MAX_IN || !address(a[2], F32, T, dev, &s))
      return none();
    const cudaStream_t st = stream(dev);
    void *px = x->data_ptr(), *pq = q->data_ptr();
    return status([&] {
      return p_quant(px, bf, static_cast<int32_t>(T), static_cast<int32_t>(H), static_cast<float>(eps),
                     static_cast<int8_t*>(pq), ld, static_cast<float*>(s), st);
    });
  } catch (...) {
    return none();
  }
}

// linear(address of the moe_linear8, its device, q, qscale, out, out_mode, err_word | None) -> status | None
PyObject* linear(PyObject*, PyObject* const* a, Py_ssize_t n) {
  if (n != 7 || !p_linear) return none();
  try {
    const auto* W = static_cast<const moe_linear8*>(PyLong_AsVoidPtr(a[0]));
    const long dev = PyLong_AsLong(a[1]), mode = PyLong_AsLong(a[5]);
    if (PyErr_Occurred()) {
      PyErr_Clear();
      return none();
    }
    if (!W || dev != c10::cuda::current_device() || mode < 0 || mode > 2) return none();
    const at::Tensor* q = tensor(a[2], I8, 0, dev);
    if (!q || q->dim() != 2) return none();
    const int64_t T = q->size(0), ld = q->size(1);
    void *s, *out, *err;
    if (ld % 16 || ld < W->in_dim || T > MOE_MAX_TOKENS || !address(a[3], F32, T, dev, &s) ||
        !address(a[4], mode == 1 ? BF16 : F32, T * W->out_dim, dev, &out) || !address(a[6], I32, 1, dev, &err, true))
      return none();
    const cudaStream_t st = stream(static_cast<int>(dev));
    void* pq = q->data_ptr();
    return status([&] {
      return p_linear(W, static_cast<const int8_t*>(pq), ld, static_cast<const float*>(s), static_cast<int32_t>(T), out,
                      static_cast<int32_t>(mode), static_cast<int32_t*>(err), st);
    });
  } catch (...) {
    return none();
  }
}

// layer(address of the moe_layer, its device, u | None, x | None, eps, K, exec_idx | None, logits | None, idx, w, out, out_mode,
// workspace, err_word | None) -> status | None
PyObject* layer(PyObject*, PyObject* const* a, Py_ssize_t n) {
  if (n != 14 || !p_layer) return none();
  try {
    const auto* L = static_cast<const moe_layer*>(PyLong_AsVoidPtr(a[0]));
    const double eps = PyFloat_AsDouble(a[4]);
    const long layer_dev = PyLong_AsLong(a[1]), K = PyLong_AsLong(a[5]), mode = PyLong_AsLong(a[11]);
    if (PyErr_Occurred()) {
      PyErr_Clear();
      return none();
    }
    if (!L || K < 1 || K > 8 || mode < 0 || mode > 2) return none();
    const int dev = c10::cuda::current_device();
    if (layer_dev != dev) return none();
    const bool norm = a[3] != Py_None;
    const at::Tensor* rows = tensor(norm ? a[3] : a[2], norm ? F32 : BF16, 0, dev);
    if (!rows || rows->dim() != 2 || rows->size(1) != L->H || rows->size(0) > MOE_LAYER_DECODE_MAX_TOKENS) return none();
    const int64_t T = rows->size(0);
    void *u, *exec, *logits, *idx, *w, *out, *ws, *err;
    if (!address(a[2], BF16, T * L->H, dev, &u, norm) || !address(a[6], I32, T * K, dev, &exec, true) ||
        !address(a[7], F32, T * L->E, dev, &logits, true) || !address(a[8], I32, T * K, dev, &idx) ||
        !address(a[9], F32, T * K, dev, &w) || !address(a[10], mode == 1 ? BF16 : F32, T * L->H, dev, &out) ||
        !address(a[12], BYTES, 0, dev, &ws) || !address(a[13], I32, 1, dev, &err, true))
      return none();
    const at::Tensor& wt = THPVariable_Unpack(a[12]);
    const cudaStream_t st = stream(dev);
    const size_t ws_bytes = static_cast<size_t>(wt.numel()) * wt.element_size();
    const float* px = norm ? static_cast<const float*>(rows->data_ptr()) : nullptr;
    return status([&] {
      return p_layer(L, static_cast<uint16_t*>(u), px, static_cast<float>(eps), static_cast<int32_t>(T),
                     static_cast<int32_t>(K), static_cast<const int32_t*>(exec), static_cast<float*>(logits),
                     static_cast<int32_t*>(idx), static_cast<float*>(w), out, static_cast<int32_t>(mode), ws, ws_bytes,
                     static_cast<int32_t*>(err), st);
    });
  } catch (...) {
    return none();
  }
}

PyMethodDef methods[] = {
    {"load", load, METH_O, "take the entry points from the library at this path"},
    {"quant", reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(quant)), METH_FASTCALL, "moe_quant_i8"},
    {"linear", reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(linear)), METH_FASTCALL, "moe_linear_i8"},
    {"layer", reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(layer)), METH_FASTCALL, "moe_layer_decode"},
    {nullptr, nullptr, 0, nullptr}};

// The torch that this was built for: its classes are laid out as that one's.
constexpr char kTorch[] = "moe binding for torch " MOE_TORCH;

PyModuleDef module = {PyModuleDef_HEAD_INIT, "_binding", nullptr, -1, methods, nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__binding() {
  PyObject* m = PyModule_Create(&module);
  if (m && PyModule_AddStringConstant(m, "built_for", kTorch) < 0) {
    Py_DECREF(m);
    return nullptr;
  }
  return m;
}
