// Python module _tensor_list: what the gradient calls need of a list of tensors, in one pass.
//
// The calls take hundreds of tensors, and addresses, sizes and types read through the tensors'
// Python attributes (five passes over a list, one call each) cost more than the kernels of short
// tensors: 70 tensors with outputs took 48 us a call, of which 11.6 in kernels, and 19 this way; on
// more than 100 short tensors the call was slower than elementary operations on one flat buffer.
#include <torch/csrc/Exceptions.h>
#include <torch/csrc/autograd/python_variable.h>

#include <cstdint>
#include <vector>

#include "../../include/intlora.h"

namespace {

struct List {
  std::vector<void*> pointers;
  std::vector<int64_t> numel;
  std::vector<int32_t> types;
};

// Fills `l` from the tensors of a list; false with a Python error set otherwise.
bool read(const char* name, PyObject* list, int device, List& l) {
  const Py_ssize_t n = PyList_GET_SIZE(list);
  l.pointers.resize(n);
  l.numel.resize(n);
  l.types.resize(n);
  Py_ssize_t other = -1;  // the first tensor of another type
  for (Py_ssize_t i = 0; i < n; ++i) {
    PyObject* o = PyList_GET_ITEM(list, i);
    if (!THPVariable_Check(o)) {
      PyErr_Format(PyExc_TypeError, "%s: expected tensors, got %s", name, Py_TYPE(o)->tp_name);
      return false;
    }
    const at::Tensor& t = THPVariable_Unpack(o);
    if (t.get_device() != device || !t.is_contiguous()) {
      PyErr_Format(PyExc_ValueError, "%s: expected contiguous tensors on the current device", name);
      return false;
    }
    l.pointers[i] = t.data_ptr();
    l.numel[i] = t.numel();
    switch (t.scalar_type()) {
      case at::kBFloat16: l.types[i] = INTLORA_BF16; break;
      case at::kHalf: l.types[i] = INTLORA_FP16; break;
      case at::kFloat: l.types[i] = INTLORA_FP32; break;
      default: other = other < 0 ? i : other;
    }
  }
  if (other < 0) return true;
  if (PyObject* dtype = PyObject_GetAttrString(PyList_GET_ITEM(list, other), "dtype")) {
    PyErr_Format(PyExc_ValueError, "%s: expected bf16, fp16 or fp32 tensors, got %S", name, dtype);
    Py_DECREF(dtype);
  }
  return false;
}

template <class T>
PyObject* bytes(const std::vector<T>& v) {
  return PyBytes_FromStringAndSize(reinterpret_cast<const char*>(v.data()), (Py_ssize_t)(v.size() * sizeof(T)));
}

// read(name, list, device) -> (addresses, element counts, INTLORA_* types), bytes of void*,
// int64 and int32 arrays.  `device` is the tensors' index (-1: host).
PyObject* py_read(PyObject*, PyObject* args) {
  HANDLE_TH_ERRORS
  const char* name;
  PyObject* list;
  int device;
  List l;
  if (!PyArg_ParseTuple(args, "sO!i", &name, &PyList_Type, &list, &device) || !read(name, list, device, l)) return nullptr;
  return Py_BuildValue("NNN", bytes(l.pointers), bytes(l.numel), bytes(l.types));
  END_HANDLE_TH_ERRORS
}

PyMethodDef methods[] = {
    {"read", py_read, METH_VARARGS, "read(name, list, device) -> addresses, element counts and types of the tensors"},
    {nullptr, nullptr, 0, nullptr}};
PyModuleDef module = {PyModuleDef_HEAD_INIT, "_tensor_list", nullptr, -1, methods, nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__tensor_list() { return PyModule_Create(&module); }
