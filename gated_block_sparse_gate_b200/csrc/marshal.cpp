// marshal.cpp — argument checks of the Python binding, on the tensors themselves.
//
// A call of a few microseconds on the GPU is otherwise outweighed by its argument checks:
// one to two microseconds a tensor in Python, some fifty nanoseconds here. Both functions only
// answer whether a tensor plainly has what is asked of it; anything else (another type, a
// view with a layout of its own, a mistake) is left to the binding's own checks, which
// accept or refuse it in words.
#include <torch/csrc/Dtype.h>
#include <torch/csrc/autograd/python_variable.h>

#include "gbs.h"

namespace {

// The tensor in t if it is plainly one on CUDA device `device` with one of the dtypes (a
// tuple) and that shape (None: any); else null.
const at::Tensor* plain(PyObject* t, PyObject* dtypes, PyObject* device, PyObject* shape) {
  if (!THPVariable_CheckExact(t) || !PyLong_Check(device)) return nullptr;
  const at::Tensor& x = THPVariable_Unpack(t);
  if (!x.defined() || x.layout() != at::kStrided || x.get_device() != PyLong_AsLong(device)) return nullptr;
  bool known = false;
  for (Py_ssize_t i = 0; i < PyTuple_GET_SIZE(dtypes) && !known; ++i) {
    PyObject* d = PyTuple_GET_ITEM(dtypes, i);
    known = THPDtype_Check(d) && reinterpret_cast<THPDtype*>(d)->scalar_type == x.scalar_type();
  }
  if (!known) return nullptr;
  if (shape == Py_None) return &x;
  const auto sizes = x.sizes();
  if (!PyTuple_Check(shape) || PyTuple_GET_SIZE(shape) != (Py_ssize_t)sizes.size()) return nullptr;
  for (size_t i = 0; i < sizes.size(); ++i)
    if (PyLong_AsLongLong(PyTuple_GET_ITEM(shape, i)) != sizes[i]) return nullptr;
  return &x;
}

// fits(t, dtypes, device_index, shape): plainly so and contiguous?
PyObject* fits(PyObject*, PyObject* const* a, Py_ssize_t n) {
  if (n != 4 || !PyTuple_Check(a[1])) {
    PyErr_SetString(PyExc_TypeError, "fits(t, dtypes, device_index, shape)");
    return nullptr;
  }
  try {
    const at::Tensor* x = plain(a[0], a[1], a[2], a[3]);
    if (PyErr_Occurred()) return nullptr;
    return PyBool_FromLong(x && x->is_contiguous());
  } catch (...) {  // a tensor without sizes or storage of its own: not plain
    Py_RETURN_FALSE;
  }
}

// heads(t, dtypes, device_index, shape, token_major, written): gbs_heads of a 4-D tensor
// as bytes; None if it is not plainly so, its channels are not contiguous or, where it is
// written, it is not contiguous.
PyObject* heads(PyObject*, PyObject* const* a, Py_ssize_t n) {
  if (n != 6 || !PyTuple_Check(a[1]) || !PyTuple_Check(a[3]) || PyTuple_GET_SIZE(a[3]) != 4) {
    PyErr_SetString(PyExc_TypeError, "heads(t, dtypes, device_index, shape, token_major, written)");
    return nullptr;
  }
  try {
    const at::Tensor* x = plain(a[0], a[1], a[2], a[3]);
    if (PyErr_Occurred()) return nullptr;
    if (!x || (a[5] == Py_True && !x->is_contiguous())) Py_RETURN_NONE;
    int64_t step[4];
    for (int i = 0; i < 4; ++i) step[i] = i < 3 && x->size(i) == 1 ? 0 : x->stride(i);  // (that of one is never followed)
    if (step[3] != 1) Py_RETURN_NONE;
    const int h_at = a[4] == Py_True ? 2 : 1;
    const gbs_heads h = {x->data_ptr(), step[0], step[h_at], step[3 - h_at]};
    return PyBytes_FromStringAndSize(reinterpret_cast<const char*>(&h), sizeof h);
  } catch (...) {
    Py_RETURN_NONE;
  }
}

PyMethodDef methods[] = {
    {"fits", reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(fits)), METH_FASTCALL,
     "whether a tensor plainly has a device, dtype and shape"},
    {"heads", reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(heads)), METH_FASTCALL,
     "gbs_heads of a tensor as bytes, or None"},
    {nullptr, nullptr, 0, nullptr}};
PyModuleDef module = {PyModuleDef_HEAD_INIT, "_marshal", nullptr, -1, methods, nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__marshal() { return PyModule_Create(&module); }
