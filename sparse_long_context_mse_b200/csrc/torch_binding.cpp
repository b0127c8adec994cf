// torch_binding.cpp -- the binding's argument checks in native code.
//
// A call of the library takes up to 17 tensors; checking each one's type,
// device, shape and layout from Python costs about a microsecond, several times
// what the launch itself costs.  `call` does all of it in one step:
//
//   call(entry, shape, kinds, tensors, stream) -> status of the entry point,
//       or -1 when a tensor is not what its kind says (the Python binding then
//       finds out which and raises)
//
// entry: the address of a C entry point (losa.h) that takes a losa_shape*, one
// pointer per tensor, for a workspace its size in bytes, and a stream; shape:
// the ctypes structure; kinds: one character per tensor (see `expect`); stream:
// a cudaStream_t as a number, or None for torch's current stream of the
// tensors' device.  The tensors' device is made current for the call.
#include <Python.h>

#include <ATen/core/Tensor.h>
#include <c10/cuda/CUDAFunctions.h>
#include <c10/cuda/CUDAGuard.h>
#include <c10/cuda/CUDAStream.h>
#include <torch/csrc/autograd/python_variable.h>

#include <algorithm>

#include "losa.h"

namespace {

constexpr int kMaxArgs = 18;
// losa_page_meta_size of the loaded library (set by `use`)
size_t (*g_page_meta_size)(const losa_shape*) = nullptr;

struct Want {
  at::ScalarType type;
  int nd;  // -1: any shape
  int64_t size[4];
};

// What a tensor of kind `c` has to be: Q queries, K prefix, 8 prefix codes, s page
// scales, b block, O and L rows of fp32 state, A active tokens, P page lists, U
// union counts, M page metadata, W workspace.  Lower-case o, l, a, p, u, m: the
// same, or None.
bool expect(char c, const losa_shape& sh, Want* w) {
  const int64_t S = sh.num_seqs, Hq = sh.n_q_heads, Hkv = sh.n_kv_heads, d = sh.head_dim,
                B = sh.block_size, ps = sh.page_size;
  if (ps < 1) return false;
  const int64_t Lc = sh.prefix_capacity > 0 ? sh.prefix_capacity : sh.prefix_len;
  const int64_t P = (sh.prefix_len + ps - 1) / ps, A = sh.n_active;
  const int64_t k = std::min<int64_t>(sh.token_budget / ps, P);
  const at::ScalarType dt = sh.dtype == LOSA_BF16 ? at::kBFloat16 : at::kFloat;
  switch (c) {
    case 'Q': *w = {dt, 4, {S, Hq, B, d}}; return true;
    case 'K': *w = {dt, 4, {S, Hkv, Lc, d}}; return true;
    case '8': *w = {at::kFloat8_e4m3fn, 4, {S, Hkv, Lc, d}}; return true;
    case 's': *w = {at::kFloat, 3, {S, Hkv, (Lc + ps - 1) / ps, 0}}; return true;
    case 'b': *w = {dt, 4, {S, Hkv, B, d}}; return true;
    case 'O': case 'o': *w = {at::kFloat, 4, {S, Hq, B, d}}; return true;
    case 'L': case 'l': *w = {at::kFloat, 3, {S, Hq, B, 0}}; return true;
    case 'A': case 'a': *w = {at::kInt, 3, {S, Hq, A, 0}}; return true;
    case 'P': case 'p': *w = {at::kInt, 4, {S, Hq, A, k}}; return true;
    case 'U': case 'u': *w = {at::kInt, 2, {S, Hkv, 0, 0}}; return true;
    case 'M': case 'm': *w = {at::kByte, 1, {static_cast<int64_t>(g_page_meta_size(&sh)), 0, 0, 0}}; return true;
    case 'W': *w = {at::kByte, -1, {0, 0, 0, 0}}; return true;
    default: return false;
  }
}

using Fn = int (*)(const void*, void*, void*, void*, void*, void*, void*, void*, void*, void*,
                   void*, void*, void*, void*, void*, void*, void*, void*, void*, void*, void*);

PyObject* call(PyObject*, PyObject* const* args, Py_ssize_t nargs) {
  if (nargs != 5 || !g_page_meta_size) {
    PyErr_SetString(PyExc_TypeError, "call(entry, shape, kinds, tensors, stream), after use()");
    return nullptr;
  }
  void* entry = PyLong_AsVoidPtr(args[0]);
  if (PyErr_Occurred()) return nullptr;
  Py_buffer buf;
  if (PyObject_GetBuffer(args[1], &buf, PyBUF_SIMPLE) != 0) return nullptr;
  losa_shape sh;
  const bool whole = buf.len == static_cast<Py_ssize_t>(sizeof(sh));
  if (whole) sh = *static_cast<const losa_shape*>(buf.buf);
  PyBuffer_Release(&buf);
  Py_ssize_t nk = 0;
  const char* kinds = PyUnicode_AsUTF8AndSize(args[2], &nk);
  if (!kinds) return nullptr;
  if (!whole || !PyTuple_Check(args[3]) || PyTuple_GET_SIZE(args[3]) != nk || nk > kMaxArgs) {
    PyErr_SetString(PyExc_TypeError, "call: a losa_shape, and one tensor per kind");
    return nullptr;
  }
  void* stream = nullptr;
  if (args[4] != Py_None) {
    stream = PyLong_AsVoidPtr(args[4]);
    if (PyErr_Occurred()) return nullptr;
  }
  void* a[kMaxArgs + 2] = {};
  int n = 0, dev = -1, rc = 0;
  try {  // (a tensor without strides or storage of its own throws when it is asked)
    for (Py_ssize_t i = 0; i < nk; ++i) {
      PyObject* o = PyTuple_GET_ITEM(args[3], i);
      Want w;
      if (!expect(kinds[i], sh, &w)) return PyLong_FromLong(-1);
      if (o == Py_None && kinds[i] >= 'a' && kinds[i] <= 'z' && kinds[i] != 's' && kinds[i] != 'b') {
        a[n++] = nullptr;
        continue;
      }
      if (!THPVariable_Check(o)) return PyLong_FromLong(-1);
      const at::Tensor& t = THPVariable_Unpack(o);
      if (t.layout() != c10::kStrided || !t.is_cuda() || t.scalar_type() != w.type ||
          !t.is_contiguous() || (dev >= 0 && t.get_device() != dev))
        return PyLong_FromLong(-1);
      dev = t.get_device();
      if (w.nd >= 0) {
        const auto sz = t.sizes();
        if (static_cast<int>(sz.size()) != w.nd) return PyLong_FromLong(-1);
        for (int j = 0; j < w.nd; ++j)
          if (sz[j] != w.size[j]) return PyLong_FromLong(-1);
      }
      a[n++] = t.data_ptr();
      if (kinds[i] == 'W') a[n++] = reinterpret_cast<void*>(t.numel());
    }
    if (dev < 0) return PyLong_FromLong(-1);
    c10::cuda::CUDAGuard guard(static_cast<c10::DeviceIndex>(dev));
    a[n] = args[4] == Py_None
               ? c10::cuda::getCurrentCUDAStream(static_cast<c10::DeviceIndex>(dev)).stream()
               : stream;
    // A launch waits while the device's queue is full, perhaps for work of another
    // Python thread: not under the interpreter's lock.  (Every parameter is a pointer
    // or of a pointer's size; the entry point reads those that it has.)
    PyThreadState* state = PyEval_SaveThread();
    rc = reinterpret_cast<Fn>(entry)(&sh, a[0], a[1], a[2], a[3], a[4], a[5], a[6], a[7], a[8], a[9],
                                     a[10], a[11], a[12], a[13], a[14], a[15], a[16], a[17], a[18],
                                     a[19]);
    PyEval_RestoreThread(state);
  } catch (const std::exception& e) {
    PyErr_SetString(PyExc_RuntimeError, e.what());
    return nullptr;
  }
  return PyLong_FromLong(rc);
}

PyObject* use(PyObject*, PyObject* arg) {
  void* f = PyLong_AsVoidPtr(arg);
  if (PyErr_Occurred()) return nullptr;
  g_page_meta_size = reinterpret_cast<size_t (*)(const losa_shape*)>(f);
  Py_RETURN_NONE;
}

PyMethodDef methods[] = {
    {"use", use, METH_O, "the address of the library's losa_page_meta_size"},
    {"call", reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(call)), METH_FASTCALL,
     "check a call's tensors and make it: see torch_binding.cpp"},
    {nullptr, nullptr, 0, nullptr}};
PyModuleDef module = {PyModuleDef_HEAD_INIT, "_binding", nullptr, -1, methods};

}  // namespace

PyMODINIT_FUNC PyInit__binding() { return PyModule_Create(&module); }
