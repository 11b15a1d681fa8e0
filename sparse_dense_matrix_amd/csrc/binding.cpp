// binding.cpp -- the checks of the Python binding's attention tensors, as a
// Python module: type, shape and device against what the plan takes, then the
// pointer (and strides) that the C ABI takes.  From Python a tensor's attributes
// take 0.4 us, ten of them more than a launch; from here all of them 0.1 us.  It
// fits the torch that it was compiled with: torch_version is compared on import.
#include <Python.h>
#include <torch/csrc/Dtype.h>
#include <torch/csrc/autograd/python_variable.h>
#include <torch/version.h>

#include <cstdint>
#include <exception>

namespace {

// Whether t is a tensor of the shape and type that `want` = (shape, dtype) names
// on the device; the tensor itself, or null.
const at::Tensor *fits(PyObject *t, PyObject *want, PyObject *device) {
  if (!THPVariable_Check(t) || !PyTuple_Check(want) || PyTuple_GET_SIZE(want) != 2) return nullptr;
  PyObject *shape = PyTuple_GET_ITEM(want, 0), *dtype = PyTuple_GET_ITEM(want, 1);
  if (!PyTuple_Check(shape) || !THPDtype_Check(dtype) || !PyLong_Check(device)) return nullptr;
  const at::Tensor &x = THPVariable_Unpack(t);
  if (!x.defined() || x.layout() != at::kStrided || !x.is_cuda() || x.device().index() != PyLong_AsLong(device) ||
      x.scalar_type() != reinterpret_cast<THPDtype *>(dtype)->scalar_type || x.dim() != PyTuple_GET_SIZE(shape))
    return nullptr;
  for (int64_t i = 0; i < x.dim(); ++i) {
    PyObject *n = PyTuple_GET_ITEM(shape, i);
    if (!PyLong_Check(n) || PyLong_AsLongLong(n) != x.size(i)) return nullptr;
  }
  return &x;
}

// heads(t, want, device): the tensor of heads [batch][tokens][heads][dim] as the
// C ABI's struct, in bytes; None where it does not fit, False where the elements
// of a head are not consecutive.
PyObject *heads_of(PyObject *const *args) {
  const at::Tensor *x = fits(args[0], args[1], args[2]);
  if (!x || x->dim() != 4) {
    if (PyErr_Occurred()) return nullptr;
    Py_RETURN_NONE;
  }
  if (x->stride(3) != 1 && x->numel() > 0) Py_RETURN_FALSE;
  const int64_t out[4] = {static_cast<int64_t>(reinterpret_cast<intptr_t>(x->data_ptr())), x->stride(0), x->stride(1),
                          x->stride(2)};
  return PyBytes_FromStringAndSize(reinterpret_cast<const char *>(out), sizeof(out));
}

// flat(t, want, device): the pointer of a contiguous tensor; None and False as above.
PyObject *flat_of(PyObject *const *args) {
  const at::Tensor *x = fits(args[0], args[1], args[2]);
  if (!x) {
    if (PyErr_Occurred()) return nullptr;
    Py_RETURN_NONE;
  }
  if (!x->is_contiguous()) Py_RETURN_FALSE;
  return PyLong_FromVoidPtr(x->data_ptr());
}

// Tensors without memory of their own throw: no exception leaves the module.
template <PyObject *(*F)(PyObject *const *)>
PyObject *entry(PyObject *, PyObject *const *args, Py_ssize_t n) {
  if (n != 3) {
    PyErr_SetString(PyExc_TypeError, "three arguments: tensor, (shape, dtype), device");
    return nullptr;
  }
  try {
    return F(args);
  } catch (const std::exception &e) {
    PyErr_SetString(PyExc_RuntimeError, e.what());
  } catch (...) {
    PyErr_SetString(PyExc_RuntimeError, "unknown exception");
  }
  return nullptr;
}

PyMethodDef methods[] = {
    {"heads", reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(entry<heads_of>)), METH_FASTCALL, nullptr},
    {"flat", reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(entry<flat_of>)), METH_FASTCALL, nullptr},
    {nullptr, nullptr, 0, nullptr}};
PyModuleDef module = {PyModuleDef_HEAD_INIT, "_binding", nullptr, -1, methods, nullptr, nullptr, nullptr, nullptr};

}  // namespace

extern "C" __attribute__((visibility("default"))) PyObject *PyInit__binding() {
  PyObject *m = PyModule_Create(&module);
  if (m && PyModule_AddStringConstant(m, "torch_version", TORCH_VERSION) < 0) {
    Py_DECREF(m);
    return nullptr;
  }
  return m;
}
