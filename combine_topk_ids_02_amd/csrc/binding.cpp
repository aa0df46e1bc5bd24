// What costs most of a small call in the Python binding, in C++: looking at a
// tensor (type, shape, device, order) and passing the arguments on. A call of the
// norm with 8 tensors took 9 us on the host through ctypes alone; its kernel takes
// 3.4 us. Nothing is kept between calls, and nothing is decided here: a tensor that
// is not what a call needs gives None, and the Python code then says what is wrong
// with it. The package works without this module, only slower; it is used only
// where built_for() is what the library and torch are.

#include <Python.h>
#include <torch/csrc/Dtype.h>
#include <torch/csrc/autograd/python_variable.h>

#include <cstdint>
#include <utility>

#include "moe_dispatch.h"

#ifndef MOE_BUILT_FOR_TORCH
#error "the torch this is compiled against, as a string (torch.__version__)"
#endif

namespace {

// address(tensor, dtype, device index, shape): the tensor's address, if it is a
// contiguous tensor of this type and shape on this GPU; else None.
PyObject* address(PyObject*, PyObject* const* args, Py_ssize_t n) {
  if (n != 4 || !THPVariable_Check(args[0]) || !THPDtype_Check(args[1]) ||
      !PyLong_Check(args[2]) || !PyTuple_Check(args[3]))
    Py_RETURN_NONE;
  try {
    const at::Tensor& t = THPVariable_Unpack(args[0]);
    const long device = PyLong_AsLong(args[2]);
    if (t.scalar_type() != reinterpret_cast<THPDtype*>(args[1])->scalar_type ||
        !t.device().is_cuda() || t.device().index() != device || !t.is_contiguous())
      Py_RETURN_NONE;
    const auto sizes = t.sizes();
    if (Py_ssize_t(sizes.size()) != PyTuple_GET_SIZE(args[3])) Py_RETURN_NONE;
    for (size_t i = 0; i < sizes.size(); ++i) {
      const long long want = PyLong_AsLongLong(PyTuple_GET_ITEM(args[3], i));
      if (want != sizes[i] || (want == -1 && PyErr_Occurred())) {
        PyErr_Clear();
        Py_RETURN_NONE;
      }
    }
    return PyLong_FromVoidPtr(t.data_ptr());
  } catch (...) {
    Py_RETURN_NONE;
  }
}

// An argument of a library call from its Python object: an address (None: NULL) or
// a structure, or a number. `ok` turns false where it is neither. `kind` stands for
// the type in built_for().
template <typename T>
struct Arg;
template <typename T>
struct Arg<T*> {
  static constexpr char kind = 'p';
  static T* from(PyObject* o, bool& ok) {
    if (o == Py_None) return nullptr;
    if (PyLong_Check(o)) {
      void* p = PyLong_AsVoidPtr(o);
      if (!p && PyErr_Occurred()) ok = false;
      return static_cast<T*>(p);
    }
    Py_buffer b;  // a ctypes structure, which its caller keeps alive
    if (PyObject_GetBuffer(o, &b, PyBUF_SIMPLE) != 0) {
      ok = false;
      return nullptr;
    }
    T* p = static_cast<T*>(b.buf);
    PyBuffer_Release(&b);
    return p;
  }
};
template <typename T>
T whole(PyObject* o, bool& ok) {
  const long long v = PyLong_AsLongLong(o);
  if ((v == -1 && PyErr_Occurred()) || static_cast<long long>(static_cast<T>(v)) != v) ok = false;
  return static_cast<T>(v);
}
template <>
struct Arg<int> {
  static constexpr char kind = 'i';
  static int from(PyObject* o, bool& ok) { return whole<int>(o, ok); }
};
template <>
struct Arg<int64_t> {
  static constexpr char kind = 'q';
  static int64_t from(PyObject* o, bool& ok) { return whole<int64_t>(o, ok); }
};
template <>
struct Arg<size_t> {
  static constexpr char kind = 'n';
  static size_t from(PyObject* o, bool& ok) { return whole<size_t>(o, ok); }
};
template <>
struct Arg<float> {
  static constexpr char kind = 'f';
  static float from(PyObject* o, bool& ok) {
    const double v = PyFloat_AsDouble(o);
    if (v == -1.0 && PyErr_Occurred()) ok = false;
    return float(v);
  }
};

// One library function as a Python one that returns its status. `at` is its address
// in the loaded library (see bind).
template <auto Declared>
struct Entry;
template <typename... A, int (*Declared)(A...)>
struct Entry<Declared> {
  static inline int (*at)(A...) = nullptr;
  static constexpr char kinds[] = {Arg<A>::kind..., 0};

  template <size_t... I>
  static int run(PyObject* const* args, bool& ok, std::index_sequence<I...>) {
    std::tuple<A...> a{Arg<A>::from(args[I], ok)...};
    if (!ok) return 0;
    int status;
    Py_BEGIN_ALLOW_THREADS;
    status = at(std::get<I>(a)...);
    Py_END_ALLOW_THREADS;
    return status;
  }

  static PyObject* call(PyObject*, PyObject* const* args, Py_ssize_t n) {
    if (!at || n != Py_ssize_t(sizeof...(A))) {
      PyErr_SetString(PyExc_TypeError, "not bound, or another number of arguments");
      return nullptr;
    }
    bool ok = true;
    const int status = run(args, ok, std::index_sequence_for<A...>{});
    if (!ok) {
      if (!PyErr_Occurred()) PyErr_SetString(PyExc_OverflowError, "a number out of range");
      return nullptr;
    }
    return PyLong_FromLong(status);
  }

  static bool bind(PyObject* o) {
    at = reinterpret_cast<int (*)(A...)>(PyLong_AsVoidPtr(o));
    return at != nullptr;
  }
};

// built_for(): the library's version, torch's, and the kinds of the arguments of each
// function below that this module was compiled for. A file that an earlier build left
// would pass arguments on in an order or width that the library no longer takes.
PyObject* built_for(PyObject*, PyObject*) {
  return Py_BuildValue("(isssss)", MOE_DISPATCH_ABI_VERSION, MOE_BUILT_FOR_TORCH,
                       Entry<&moe_norm>::kinds, Entry<&moe_norm_backward>::kinds,
                       Entry<&moe_quantise_rows>::kinds, Entry<&moe_int8_product>::kinds);
}

// bind(address of each function below, in this order)
PyObject* bind(PyObject*, PyObject* const* args, Py_ssize_t n) {
  if (n != 4 || !Entry<&moe_norm>::bind(args[0]) || !Entry<&moe_norm_backward>::bind(args[1]) ||
      !Entry<&moe_quantise_rows>::bind(args[2]) || !Entry<&moe_int8_product>::bind(args[3])) {
    if (!PyErr_Occurred()) PyErr_SetString(PyExc_TypeError, "four addresses");
    return nullptr;
  }
  Py_RETURN_NONE;
}

#define FAST(name, f) {name, reinterpret_cast<PyCFunction>(f), METH_FASTCALL, nullptr}
PyMethodDef kMethods[] = {FAST("address", address),
                          {"built_for", built_for, METH_NOARGS, nullptr},
                          FAST("bind", bind),
                          FAST("moe_norm", Entry<&moe_norm>::call),
                          FAST("moe_norm_backward", Entry<&moe_norm_backward>::call),
                          FAST("moe_quantise_rows", Entry<&moe_quantise_rows>::call),
                          FAST("moe_int8_product", Entry<&moe_int8_product>::call),
                          {nullptr, nullptr, 0, nullptr}};
PyModuleDef kModule = {PyModuleDef_HEAD_INIT, "_binding", nullptr, -1, kMethods};

}  // namespace

PyMODINIT_FUNC PyInit__binding() { return PyModule_Create(&kModule); }
