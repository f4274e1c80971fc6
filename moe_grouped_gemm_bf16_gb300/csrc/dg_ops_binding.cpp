// CPython module `_binding`: calls of the operators around the GEMMs without
// ctypes, whose argument conversion took a third of a small call (a norm of 7
// rows: 3.7 us from Python through ctypes, 2.5 so, of which the launch is 1.7).
//
// open(path) takes the entry points out of the library at `path`; each function
// then has its entry point's positional arguments and returns its status.
// Pointers are None, an address, or an object with data_ptr() (a torch tensor).
#define PY_SSIZE_T_CLEAN
#include <Python.h>
#include <dlfcn.h>

#include <climits>
#include <cstddef>
#include <tuple>
#include <utility>

#include "dg.h"

namespace {

PyObject* g_data_ptr;   // "data_ptr"

bool convert(PyObject* o, long long* out) {
  *out = PyLong_AsLongLong(o);
  return *out != -1 || !PyErr_Occurred();
}

bool convert(PyObject* o, int* out) {
  long long v;
  if (!convert(o, &v)) return false;
  if (v < INT_MIN || v > INT_MAX) {
    PyErr_Format(PyExc_OverflowError, "%lld does not fit 32 bits", v);
    return false;
  }
  *out = static_cast<int>(v);
  return true;
}

bool convert(PyObject* o, float* out) {
  const double v = PyFloat_AsDouble(o);
  *out = static_cast<float>(v);
  return v != -1.0 || !PyErr_Occurred();
}

bool address(PyObject* o, void** out) {
  if (o == Py_None) {
    *out = nullptr;
  } else if (PyLong_Check(o)) {
    *out = PyLong_AsVoidPtr(o);
  } else {
    PyObject* v = PyObject_CallMethodNoArgs(o, g_data_ptr);
    if (!v) return false;
    *out = PyLong_AsVoidPtr(v);
    Py_DECREF(v);
  }
  return *out || !PyErr_Occurred();
}

template <class T>
bool convert(PyObject* o, T** out) {
  void* p;
  if (!address(o, &p)) return false;
  *out = static_cast<T*>(p);
  return true;
}

template <class... A>
using Entry = dg_status (*)(A...);

template <class... A, size_t... I>
PyObject* call(Entry<A...> f, PyObject* const* args, std::index_sequence<I...>) {
  std::tuple<A...> a;
  if (!(convert(args[I], &std::get<I>(a)) && ...)) return nullptr;
  dg_status s;
  Py_BEGIN_ALLOW_THREADS
  s = f(std::get<I>(a)...);
  Py_END_ALLOW_THREADS
  return PyLong_FromLong(s);
}

template <class... A>
PyObject* call(Entry<A...> f, const char* name, PyObject* const* args, Py_ssize_t n) {
  if (!f) {
    PyErr_SetString(PyExc_RuntimeError, "the library is not open");
    return nullptr;
  }
  if (n != static_cast<Py_ssize_t>(sizeof...(A))) {
    PyErr_Format(PyExc_TypeError, "%s takes %zd arguments (%zd given)", name,
                 static_cast<Py_ssize_t>(sizeof...(A)), n);
    return nullptr;
  }
  return call(f, args, std::index_sequence_for<A...>());
}

#define DG_ENTRIES(X)                       \
  X(rms_norm_quantize_fp8_1x128)            \
  X(rms_norm_quantize_fp8_1x128_ue8m0)      \
  X(rms_norm_backward)                      \
  X(swiglu_quantize_fp8_1x128)              \
  X(swiglu_quantize_fp8_1x128_ue8m0)        \
  X(swiglu_backward_fp8_1x128)              \
  X(m_grouped_gemm_bf16_nt_ragged)          \
  X(m_grouped_gemm_bf16_nn_ragged)          \
  X(k_grouped_gemm_bf16_tn_ragged)

#define DG_FUNCTION(name)                                                        \
  decltype(&dg_##name) p_##name;                                                 \
  PyObject* py_##name(PyObject*, PyObject* const* args, Py_ssize_t n) {          \
    return call(p_##name, #name, args, n);                                       \
  }
DG_ENTRIES(DG_FUNCTION)

PyObject* py_open(PyObject*, PyObject* path) {
  const char* file = PyUnicode_AsUTF8(path);
  if (!file) return nullptr;
  void* lib = dlopen(file, RTLD_NOW | RTLD_LOCAL);
  if (!lib) {
    PyErr_Format(PyExc_OSError, "%s", dlerror());
    return nullptr;
  }
#define DG_RESOLVE(name)                                                         \
  if (!(p_##name = reinterpret_cast<decltype(p_##name)>(dlsym(lib, "dg_" #name)))) { \
    PyErr_Format(PyExc_OSError, "%s has no dg_" #name, file);                    \
    return nullptr;                                                              \
  }
  DG_ENTRIES(DG_RESOLVE)
  Py_RETURN_NONE;
}

#define DG_METHOD(name) \
  {#name, reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(py_##name)), METH_FASTCALL, nullptr},
PyMethodDef g_methods[] = {DG_ENTRIES(DG_METHOD){"open", py_open, METH_O, nullptr},
                           {nullptr, nullptr, 0, nullptr}};

PyModuleDef g_module = {PyModuleDef_HEAD_INIT, "_binding", nullptr, -1, g_methods,
                        nullptr,               nullptr,    nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__binding() {
  g_data_ptr = PyUnicode_InternFromString("data_ptr");
  return g_data_ptr ? PyModule_Create(&g_module) : nullptr;
}
