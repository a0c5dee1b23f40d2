// Argument marshalling of the Python binding's usual calls, as a CPython module.
//
// The calls around a decode step's GEMMs run for 3 to 12 us on the GPU, while
// checking arguments, allocating outputs and filling a foreign call from Python
// took 13 to 20 us on the host. These functions do the same in C++: they check
// what the binding checks, allocate through the same caching allocator on the
// same (current) stream, and call the library through the addresses the binding
// hands over (bind). A call they do not take -- an argument that the binding
// would refuse, a tensor that is not on the current device -- returns None, and
// the binding's own code goes through it and raises its errors. A status other
// than 0 comes back as a number.
#include <Python.h>

#include <ATen/cuda/EmptyTensor.h>
#include <c10/cuda/CUDAFunctions.h>
#include <c10/cuda/CUDAStream.h>
#include <torch/csrc/Exceptions.h>
#include <torch/csrc/autograd/python_variable.h>

#include "bsgemm.h"

namespace {

struct Entries {
  decltype(&bsgemm_fp8_gemm_fused) gemm_fused;
  decltype(&bsgemm_fp8_gemm_residual) gemm_residual;
  decltype(&bsgemm_rms_norm_quantize_fp8) norm;
  decltype(&bsgemm_rms_norm_backward) norm_backward;
  decltype(&bsgemm_rms_norm_backward_workspace) norm_backward_workspace;
  decltype(&bsgemm_activation_quantize_fp8) act;
  decltype(&bsgemm_activation_backward_quantize_fp8) act_backward;
  decltype(&bsgemm_activation_backward_workspace) act_backward_workspace;
};
Entries g_lib{};

using at::Tensor;

// The tensor of a Python object if it is dense and on the current CUDA device.
const Tensor* dense(PyObject* o, c10::DeviceIndex dev) {
  if (!THPVariable_Check(o)) return nullptr;
  const Tensor& t = THPVariable_Unpack(o);
  return t.layout() == at::kStrided && t.is_cuda() && t.device().index() == dev && t.is_contiguous() ? &t : nullptr;
}

// bsgemm_src_dtype of a matrix or vector, -1 for other types
int src_of(const Tensor& t) {
  return t.scalar_type() == at::kFloat ? BSGEMM_SRC_F32 : t.scalar_type() == at::kBFloat16 ? BSGEMM_SRC_BF16 : -1;
}

const Tensor* matrix(PyObject* o, c10::DeviceIndex dev) {
  const Tensor* t = dense(o, dev);
  return t && t->dim() == 2 && src_of(*t) >= 0 ? t : nullptr;
}

// a matrix of the same type and sizes as `like`
const Tensor* matrix_like(PyObject* o, const Tensor& like) {
  const Tensor* t = dense(o, like.device().index());
  return t && t->dim() == 2 && t->scalar_type() == like.scalar_type() && t->sizes() == like.sizes() ? t : nullptr;
}

const Tensor* floats(PyObject* o, c10::DeviceIndex dev, int64_t numel) {
  const Tensor* t = dense(o, dev);
  return t && t->scalar_type() == at::kFloat && t->numel() == numel ? t : nullptr;
}

// on the CPU-only machine there is no current device: tensors are then never CUDA ones
bool current_device(PyObject* first, c10::DeviceIndex& dev) {
  if (!THPVariable_Check(first) || !THPVariable_Unpack(first).is_cuda()) return false;
  dev = c10::cuda::current_device();
  return true;
}

Tensor empty(at::IntArrayRef sizes, at::ScalarType type, c10::DeviceIndex dev) {
  return at::detail::empty_cuda(sizes, type, c10::Device(c10::kCUDA, dev), std::nullopt);
}

bool known_gran(int64_t g) { return g == 64 || g == 128 || g == 256; }
int64_t blocks(int64_t n, int64_t g) { return (n + g - 1) / g; }

void* stream_of(c10::DeviceIndex dev) { return c10::cuda::getCurrentCUDAStream(dev).stream(); }

template <typename F>
int call(F&& f) {
  int st;
  Py_BEGIN_ALLOW_THREADS st = f();
  Py_END_ALLOW_THREADS return st;
}

PyObject* status(int st) { return PyLong_FromLong(st); }

PyObject* tuple_of(std::initializer_list<const Tensor*> ts) {
  PyObject* r = PyTuple_New(static_cast<Py_ssize_t>(ts.size()));
  if (!r) return nullptr;
  Py_ssize_t i = 0;
  for (const Tensor* t : ts) {
    PyObject* o = t ? THPVariable_Wrap(*t) : Py_NewRef(Py_None);
    if (!o) {
      Py_DECREF(r);
      return nullptr;
    }
    PyTuple_SET_ITEM(r, i++, o);
  }
  return r;
}

#define BSGT_ARGS(n) \
  if (nargs != (n) || !g_lib.norm) Py_RETURN_NONE
#define BSGT_INT(name, k)                   \
  const int64_t name = PyLong_AsLong(args[k]); \
  if (name == -1 && PyErr_Occurred()) {     \
    PyErr_Clear();                          \
    Py_RETURN_NONE;                         \
  }

// norm(x, weight, residual or None, eps, gran, fmt) -> (q, scales, h or None, rstd)
PyObject* norm(PyObject*, PyObject* const* args, Py_ssize_t nargs) {
  HANDLE_TH_ERRORS
  BSGT_ARGS(6);
  c10::DeviceIndex dev;
  if (!current_device(args[0], dev)) Py_RETURN_NONE;
  const Tensor* x = matrix(args[0], dev);
  const Tensor* w = dense(args[1], dev);
  if (!x || !w || src_of(*w) < 0 || w->numel() != x->size(1)) Py_RETURN_NONE;
  const Tensor* res = args[2] == Py_None ? nullptr : matrix_like(args[2], *x);
  if (!res && args[2] != Py_None) Py_RETURN_NONE;
  const double eps = PyFloat_AsDouble(args[3]);
  if (eps == -1.0 && PyErr_Occurred()) {
    PyErr_Clear();
    Py_RETURN_NONE;
  }
  BSGT_INT(gran, 4);
  BSGT_INT(fmt, 5);
  const int64_t rows = x->size(0), cols = x->size(1);
  if (!known_gran(gran) || rows == 0 || cols == 0) Py_RETURN_NONE;
  Tensor q = empty({rows, cols}, at::kByte, dev);
  Tensor scales = empty({blocks(rows, gran), blocks(cols, gran)}, at::kFloat, dev);
  Tensor rstd = empty({rows}, at::kFloat, dev);
  Tensor h;
  if (res) h = empty({rows, cols}, x->scalar_type(), dev);
  void* s = stream_of(dev);
  const int st = call([&] {
    return g_lib.norm(src_of(*x), src_of(*w), static_cast<int>(fmt), x->data_ptr(), res ? res->data_ptr() : nullptr,
                      w->data_ptr(), static_cast<float>(eps), rows, cols, static_cast<int>(gran),
                      res ? h.data_ptr() : nullptr, q.data_ptr(), static_cast<float*>(scales.data_ptr()),
                      static_cast<float*>(rstd.data_ptr()), s);
  });
  return st ? status(st) : tuple_of({&q, &scales, res ? &h : nullptr, &rstd});
  END_HANDLE_TH_ERRORS
}

// norm_backward(dy, h, weight, rstd, dresidual or None) -> (dx, dweight)
PyObject* norm_backward(PyObject*, PyObject* const* args, Py_ssize_t nargs) {
  HANDLE_TH_ERRORS
  BSGT_ARGS(5);
  c10::DeviceIndex dev;
  if (!current_device(args[0], dev)) Py_RETURN_NONE;
  const Tensor* dy = matrix(args[0], dev);
  if (!dy) Py_RETURN_NONE;
  const int64_t rows = dy->size(0), cols = dy->size(1);
  const Tensor* h = matrix_like(args[1], *dy);
  const Tensor* w = dense(args[2], dev);
  const Tensor* rstd = floats(args[3], dev, rows);
  const Tensor* skip = args[4] == Py_None ? nullptr : matrix_like(args[4], *dy);
  if (!h || !w || src_of(*w) < 0 || w->numel() != cols || !rstd || (!skip && args[4] != Py_None) || rows == 0 ||
      cols == 0)
    Py_RETURN_NONE;
  Tensor dx = empty({rows, cols}, dy->scalar_type(), dev);
  Tensor dw = empty({cols}, at::kFloat, dev);
  const size_t bytes = g_lib.norm_backward_workspace(rows, cols);
  Tensor ws = empty({static_cast<int64_t>(bytes)}, at::kByte, dev);
  void* s = stream_of(dev);
  const int st = call([&] {
    return g_lib.norm_backward(src_of(*dy), src_of(*w), dy->data_ptr(), h->data_ptr(), w->data_ptr(),
                               static_cast<const float*>(rstd->data_ptr()), skip ? skip->data_ptr() : nullptr, rows,
                               cols, dx.data_ptr(), static_cast<float*>(dw.data_ptr()), ws.data_ptr(), bytes, s);
  });
  return st ? status(st) : tuple_of({&dx, &dw});
  END_HANDLE_TH_ERRORS
}

// act(z, activation, gran, fmt) -> (q, scales)
PyObject* act(PyObject*, PyObject* const* args, Py_ssize_t nargs) {
  HANDLE_TH_ERRORS
  BSGT_ARGS(4);
  c10::DeviceIndex dev;
  if (!current_device(args[0], dev)) Py_RETURN_NONE;
  const Tensor* z = matrix(args[0], dev);
  if (!z) Py_RETURN_NONE;
  BSGT_INT(activation, 1);
  BSGT_INT(gran, 2);
  BSGT_INT(fmt, 3);
  const int64_t rows = z->size(0), cols = z->size(1);
  if (!known_gran(gran) || rows == 0 || cols == 0) Py_RETURN_NONE;
  Tensor q = empty({rows, cols}, at::kByte, dev);
  Tensor scales = empty({blocks(rows, gran), blocks(cols, gran)}, at::kFloat, dev);
  void* s = stream_of(dev);
  const int st = call([&] {
    return g_lib.act(src_of(*z), static_cast<int>(fmt), static_cast<int>(activation), z->data_ptr(), rows, cols,
                     static_cast<int>(gran), q.data_ptr(), static_cast<float*>(scales.data_ptr()), s);
  });
  return st ? status(st) : tuple_of({&q, &scales});
  END_HANDLE_TH_ERRORS
}

// act_backward(dout, z or None, activation, gran, fmt, whether dbias is wanted) -> (q, scales, dbias or None)
PyObject* act_backward(PyObject*, PyObject* const* args, Py_ssize_t nargs) {
  HANDLE_TH_ERRORS
  BSGT_ARGS(6);
  c10::DeviceIndex dev;
  if (!current_device(args[0], dev)) Py_RETURN_NONE;
  const Tensor* dout = matrix(args[0], dev);
  if (!dout) Py_RETURN_NONE;
  const Tensor* z = args[1] == Py_None ? nullptr : matrix_like(args[1], *dout);
  if (!z && args[1] != Py_None) Py_RETURN_NONE;
  BSGT_INT(activation, 2);
  BSGT_INT(gran, 3);
  BSGT_INT(fmt, 4);
  const int sums = PyObject_IsTrue(args[5]);
  const int64_t rows = dout->size(0), cols = dout->size(1);
  if (sums < 0 || !known_gran(gran) || rows == 0 || cols == 0 || (z != nullptr) != (activation != BSGEMM_ACT_NONE)) {
    PyErr_Clear();
    Py_RETURN_NONE;
  }
  Tensor q = empty({rows, cols}, at::kByte, dev);
  Tensor scales = empty({blocks(rows, gran), blocks(cols, gran)}, at::kFloat, dev);
  Tensor db, ws;
  size_t bytes = 0;
  if (sums) {
    db = empty({cols}, at::kFloat, dev);
    bytes = g_lib.act_backward_workspace(rows, cols, static_cast<int>(gran));
    if (bytes) ws = empty({static_cast<int64_t>(bytes)}, at::kByte, dev);
  }
  void* s = stream_of(dev);
  const int st = call([&] {
    return g_lib.act_backward(src_of(*dout), static_cast<int>(fmt), static_cast<int>(activation), dout->data_ptr(),
                              z ? z->data_ptr() : nullptr, rows, cols, static_cast<int>(gran), q.data_ptr(),
                              static_cast<float*>(scales.data_ptr()), sums ? static_cast<float*>(db.data_ptr()) : nullptr,
                              bytes ? ws.data_ptr() : nullptr, bytes, s);
  });
  return st ? status(st) : tuple_of({&q, &scales, sums ? &db : nullptr});
  END_HANDLE_TH_ERRORS
}

// FP8 format of an operand's codes, -1 if they are none (bytes are E4M3 here)
int format_of(const Tensor& t) {
  switch (t.scalar_type()) {
    case at::kByte:
    case at::kFloat8_e4m3fn: return BSGEMM_FP8_E4M3;
    case at::kFloat8_e5m2:   return BSGEMM_FP8_E5M2;
    default:                 return -1;
  }
}

// gemm(layout, gran, a, b, scale_a, scale_b, bias or None, activation, whether out is FP32, residual or None) -> out
PyObject* gemm(PyObject*, PyObject* const* args, Py_ssize_t nargs) {
  HANDLE_TH_ERRORS
  BSGT_ARGS(10);
  c10::DeviceIndex dev;
  if (!current_device(args[2], dev)) Py_RETURN_NONE;
  BSGT_INT(layout, 0);
  BSGT_INT(gran, 1);
  BSGT_INT(activation, 7);
  const int f32 = PyObject_IsTrue(args[8]);
  const Tensor* a = dense(args[2], dev);
  const Tensor* b = dense(args[3], dev);
  if (f32 < 0 || !known_gran(gran) || layout < 0 || layout > 3 || !a || !b || a->dim() != 2 || b->dim() != 2) {
    PyErr_Clear();
    Py_RETURN_NONE;
  }
  const int fa = format_of(*a), fb = format_of(*b);
  const bool a_t = layout == BSGEMM_LAYOUT_TN || layout == BSGEMM_LAYOUT_TT;   // A stored [K, M]
  const bool b_t = layout == BSGEMM_LAYOUT_NT || layout == BSGEMM_LAYOUT_TT;   // B stored [N, K]
  const int64_t M = a->size(a_t ? 1 : 0), K = a->size(a_t ? 0 : 1);
  const int64_t N = b->size(b_t ? 0 : 1);
  if (fa < 0 || fb < 0 || b->size(b_t ? 1 : 0) != K || M == 0 || N == 0 || K == 0) Py_RETURN_NONE;
  const Tensor* sa = floats(args[4], dev, blocks(M, gran) * blocks(K, gran));
  const Tensor* sb = floats(args[5], dev, blocks(N, gran) * blocks(K, gran));
  const Tensor* bias = args[6] == Py_None ? nullptr : floats(args[6], dev, N);
  if (!sa || !sb || (!bias && args[6] != Py_None)) Py_RETURN_NONE;
  const at::ScalarType type = f32 ? at::kFloat : at::kBFloat16;
  const Tensor* res = args[9] == Py_None ? nullptr : dense(args[9], dev);
  if (args[9] != Py_None &&
      (!res || res->scalar_type() != type || res->dim() != 2 || res->size(0) != M || res->size(1) != N))
    Py_RETURN_NONE;
  Tensor out = empty({M, N}, type, dev);
  bsgemm_epilogue epi{bias ? static_cast<const float*>(bias->data_ptr()) : nullptr, static_cast<int>(activation),
                      f32 ? BSGEMM_OUT_F32 : BSGEMM_OUT_BF16};
  void* s = stream_of(dev);
  const float* pa = static_cast<const float*>(sa->data_ptr());
  const float* pb = static_cast<const float*>(sb->data_ptr());
  const int lay = static_cast<int>(layout), g = static_cast<int>(gran);
  const int st = call([&] {
    return res ? g_lib.gemm_residual(lay, fa, fb, a->data_ptr(), b->data_ptr(), pa, pb, &epi, res->data_ptr(),
                                     out.data_ptr(), M, N, K, g, nullptr, s)
               : g_lib.gemm_fused(lay, fa, fb, a->data_ptr(), b->data_ptr(), pa, pb, &epi, out.data_ptr(), M, N, K, g,
                                  nullptr, s);
  });
  return st ? status(st) : THPVariable_Wrap(out);
  END_HANDLE_TH_ERRORS
}

// bind(addresses of the library's entry points, in the order of Entries)
PyObject* bind(PyObject*, PyObject* const* args, Py_ssize_t nargs) {
  constexpr Py_ssize_t n = sizeof(Entries) / sizeof(void*);
  void* p[n];
  if (nargs != n) {
    PyErr_Format(PyExc_TypeError, "bind takes %zd addresses", n);
    return nullptr;
  }
  for (Py_ssize_t i = 0; i < n; ++i) {
    p[i] = PyLong_AsVoidPtr(args[i]);
    if (!p[i]) {
      if (!PyErr_Occurred()) PyErr_SetString(PyExc_ValueError, "null entry point");
      return nullptr;
    }
  }
  g_lib.gemm_fused = reinterpret_cast<decltype(g_lib.gemm_fused)>(p[0]);
  g_lib.gemm_residual = reinterpret_cast<decltype(g_lib.gemm_residual)>(p[1]);
  g_lib.norm = reinterpret_cast<decltype(g_lib.norm)>(p[2]);
  g_lib.norm_backward = reinterpret_cast<decltype(g_lib.norm_backward)>(p[3]);
  g_lib.norm_backward_workspace = reinterpret_cast<decltype(g_lib.norm_backward_workspace)>(p[4]);
  g_lib.act = reinterpret_cast<decltype(g_lib.act)>(p[5]);
  g_lib.act_backward = reinterpret_cast<decltype(g_lib.act_backward)>(p[6]);
  g_lib.act_backward_workspace = reinterpret_cast<decltype(g_lib.act_backward_workspace)>(p[7]);
  Py_RETURN_NONE;
}

template <PyObject* (*F)(PyObject*, PyObject* const*, Py_ssize_t)>
PyMethodDef method(const char* name) {
  return {name, reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(F)), METH_FASTCALL, nullptr};
}

PyMethodDef g_methods[] = {method<bind>("bind"), method<norm>("norm"), method<norm_backward>("norm_backward"),
                           method<act>("act"), method<act_backward>("act_backward"), method<gemm>("gemm"),
                           {nullptr, nullptr, 0, nullptr}};
PyModuleDef g_module = {PyModuleDef_HEAD_INIT, "_bsgemm_torch", nullptr, -1, g_methods, nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__bsgemm_torch(void) { return PyModule_Create(&g_module); }
