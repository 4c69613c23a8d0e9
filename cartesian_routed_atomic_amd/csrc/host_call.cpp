// The host's part of the library's shortest calls, as a CPython module: the check of
// tensor arguments and the passing of arguments to the C entry points.  ctypes and
// Python take longer for it than the kernels of a single token run.
//   fits(dev, tensor, dtype, shape, tensor, dtype, shape, ...): whether every tensor
//     that is not None is contiguous, of its type and shape, and on device dev
//   entry(name, address): a callable of the C function at address, by the prototype
//     that omni.h gives it; tensors go as their data, None as NULL
#define PY_SSIZE_T_CLEAN
#include <torch/csrc/Dtype.h>
#include <torch/csrc/autograd/python_variable.h>

#include <climits>
#include <cstring>
#include <exception>
#include <tuple>
#include <utility>

#include "omni.h"

namespace {

bool argument_error(const char* what) {
  if (!PyErr_Occurred()) PyErr_SetString(PyExc_TypeError, what);
  return false;
}
template <typename T>
struct Argument {  // int and the header's enumerations
  static bool get(PyObject* o, T& v) {
    const long x = PyLong_AsLong(o);
    if (x == -1 && PyErr_Occurred()) return false;
    if (x < INT_MIN || x > INT_MAX) return argument_error("an int argument is out of range");
    v = static_cast<T>(x);
    return true;
  }
};
template <>
struct Argument<float> {
  static bool get(PyObject* o, float& v) {
    const double x = PyFloat_AsDouble(o);
    if (x == -1.0 && PyErr_Occurred()) return false;
    v = static_cast<float>(x);
    return true;
  }
};
template <>
struct Argument<size_t> {
  static bool get(PyObject* o, size_t& v) {
    v = PyLong_AsSize_t(o);
    return !(v == static_cast<size_t>(-1) && PyErr_Occurred());
  }
};
template <typename T>
struct Argument<T*> {
  static bool get(PyObject* o, T*& v) {
    if (o == Py_None) {
      v = nullptr;
    } else if (THPVariable_Check(o)) {
      try {  // a tensor may have no memory
        v = static_cast<T*>(const_cast<void*>(THPVariable_Unpack(o).const_data_ptr()));
      } catch (const std::exception& e) {
        return argument_error(e.what());
      }
    } else {
      v = static_cast<T*>(PyLong_AsVoidPtr(o));
      if (!v && PyErr_Occurred()) return argument_error("a pointer is a tensor, an int or None");
    }
    return true;
  }
};

template <typename... A, size_t... I>
PyObject* pass(omni_status (*f)(A...), PyObject* const* args, std::index_sequence<I...>) {
  std::tuple<A...> v{};
  if (!(Argument<A>::get(args[I], std::get<I>(v)) && ...)) return nullptr;
  omni_status st;
  Py_BEGIN_ALLOW_THREADS
  st = f(std::get<I>(v)...);
  Py_END_ALLOW_THREADS
  return PyLong_FromLong(st);
}
template <typename F>
struct Entry;
template <typename... A>
struct Entry<omni_status (*)(A...)> {
  static PyObject* call(PyObject* self, PyObject* const* args, Py_ssize_t n) {
    if (n != static_cast<Py_ssize_t>(sizeof...(A)))
      return PyErr_Format(PyExc_TypeError, "%d arguments, not %zd", static_cast<int>(sizeof...(A)), n);
    return pass(reinterpret_cast<omni_status (*)(A...)>(PyLong_AsVoidPtr(self)), args,
                std::index_sequence_for<A...>{});
  }
};

#define OMNI_ENTRY(name) \
  {#name, reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(Entry<decltype(&name)>::call)), \
   METH_FASTCALL, nullptr}
PyMethodDef entries[] = {
    OMNI_ENTRY(omni_microscale_rows),       OMNI_ENTRY(omni_microscaled_matmul),
    OMNI_ENTRY(omni_microscaled_expert_matmul), OMNI_ENTRY(omni_expert_route),
    OMNI_ENTRY(omni_expert_route_backward), OMNI_ENTRY(omni_residual_norm),
    OMNI_ENTRY(omni_residual_norm_backward),
};

PyObject* entry(PyObject*, PyObject* args) {
  const char* name;
  PyObject* address;
  if (!PyArg_ParseTuple(args, "sO!", &name, &PyLong_Type, &address)) return nullptr;
  for (PyMethodDef& m : entries)
    if (std::strcmp(m.ml_name, name) == 0) return PyCFunction_New(&m, address);
  return PyErr_Format(PyExc_KeyError, "%s", name);
}

// 1 or 0, or -1 with a Python error
int one_fits(const at::Tensor& t, PyObject* dtype, PyObject* shape, long dev) {
  try {  // tensors that are not strided have no sizes or memory to ask for
    if (t.layout() != at::kStrided || t.is_nested()) return 0;
    const auto sizes = t.sizes();
    if (t.scalar_type() != reinterpret_cast<THPDtype*>(dtype)->scalar_type || !t.is_cuda() ||
        t.get_device() != dev || static_cast<Py_ssize_t>(sizes.size()) != PyTuple_GET_SIZE(shape) ||
        !t.is_contiguous())
      return 0;
    for (size_t j = 0; j < sizes.size(); ++j) {
      const long long want = PyLong_AsLongLong(PyTuple_GET_ITEM(shape, j));
      if (want == -1 && PyErr_Occurred()) return -1;
      if (sizes[j] != want) return 0;
    }
    return 1;
  } catch (const std::exception&) {
    return 0;
  }
}
PyObject* fits(PyObject*, PyObject* const* args, Py_ssize_t n) {
  if (n % 3 != 1) return PyErr_Format(PyExc_TypeError, "a device, then tensor, dtype, shape each");
  const long dev = PyLong_AsLong(args[0]);
  if (dev == -1 && PyErr_Occurred()) return nullptr;
  for (Py_ssize_t i = 1; i < n; i += 3) {
    PyObject *o = args[i], *dtype = args[i + 1], *shape = args[i + 2];
    if (o == Py_None) continue;
    if (!THPVariable_Check(o) || !THPDtype_Check(dtype) || !PyTuple_Check(shape)) Py_RETURN_FALSE;
    const int fit = one_fits(THPVariable_Unpack(o), dtype, shape, dev);
    if (fit < 0) return nullptr;
    if (fit == 0) Py_RETURN_FALSE;
  }
  Py_RETURN_TRUE;
}

PyMethodDef methods[] = {
    {"entry", entry, METH_VARARGS, nullptr},
    {"fits", reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(fits)), METH_FASTCALL, nullptr},
    {nullptr, nullptr, 0, nullptr},
};
PyModuleDef module = {PyModuleDef_HEAD_INIT, "_host_call", nullptr, -1, methods,
                      nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__host_call() { return PyModule_Create(&module); }
