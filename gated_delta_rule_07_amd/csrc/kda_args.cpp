// Python helper of the binding: one call that checks a tensor argument and gives its
// address.  A one-token call checks ten tensors, and five property reads of each from
// Python take as long as launching the kernel (0.40 us a tensor against 0.1 us here).
//
//   need(tensor, name, dtype, device_index, shape) -> address
// A tensor that is not a dense HIP tensor of this dtype, device and shape goes to the
// callable given to set_refuse with the same arguments, which says what is wrong.
//
//   rows(tensor, dtype, device_index) -> (address, tokens, heads, d, row stride) or None
// of a HIP tensor [n,H,d] or [B,T,H,d] of this dtype and device whose heads are dense and
// whose token rows are evenly spaced; None for any other.
//
//   torch_version: the PyTorch whose headers this was compiled against.  Its objects' layouts
// are read here, so the binding uses this module with that version only; a Python of
// another minor version is refused at import.
#define PY_SSIZE_T_CLEAN
#include <Python.h>
#include <stdio.h>

#include <torch/csrc/Dtype.h>
#include <torch/csrc/autograd/python_variable.h>

namespace {

PyObject* g_refuse = nullptr;

PyObject* set_refuse(PyObject*, PyObject* f) {
  Py_INCREF(f);
  Py_XSETREF(g_refuse, f);
  Py_RETURN_NONE;
}

bool fits(PyObject* const* args) {
  if (!THPVariable_Check(args[0]) || !THPDtype_Check(args[2]) || !PyLong_Check(args[3]) || !PyTuple_Check(args[4]))
    return false;
  const at::Tensor& t = THPVariable_Unpack(args[0]);
  const Py_ssize_t dim = PyTuple_GET_SIZE(args[4]);
  if (!t.defined() || t.layout() != at::kStrided || !t.is_cuda() || t.dim() != dim ||
      t.scalar_type() != reinterpret_cast<THPDtype*>(args[2])->scalar_type ||
      t.get_device() != PyLong_AsLongLong(args[3]) || !t.is_contiguous())
    return false;
  for (Py_ssize_t i = 0; i < dim; ++i)
    if (t.size(i) != PyLong_AsLongLong(PyTuple_GET_ITEM(args[4], i))) return false;
  return true;
}

PyObject* need(PyObject*, PyObject* const* args, Py_ssize_t n) {
  if (n != 5 || !g_refuse) {
    PyErr_SetString(PyExc_TypeError, "need(tensor, name, dtype, device_index, shape), after set_refuse");
    return nullptr;
  }
  try {
    if (fits(args) && !PyErr_Occurred()) return PyLong_FromVoidPtr(THPVariable_Unpack(args[0]).data_ptr());
  } catch (...) {  // (a tensor without storage, say: the callable below finds the words)
  }
  PyErr_Clear();
  return PyObject_Vectorcall(g_refuse, args, n, nullptr);
}

PyObject* rows(PyObject*, PyObject* const* args, Py_ssize_t n) {
  if (n != 3) {
    PyErr_SetString(PyExc_TypeError, "rows(tensor, dtype, device_index)");
    return nullptr;
  }
  if (!THPVariable_Check(args[0]) || !THPDtype_Check(args[1]) || !PyLong_Check(args[2])) Py_RETURN_NONE;
  try {
    const at::Tensor& t = THPVariable_Unpack(args[0]);
    const int64_t dim = t.defined() && t.layout() == at::kStrided ? t.dim() : 0;
    if (!t.is_cuda() || t.scalar_type() != reinterpret_cast<THPDtype*>(args[1])->scalar_type ||
        t.get_device() != PyLong_AsLongLong(args[2]) || (dim != 3 && dim != 4))
      Py_RETURN_NONE;
    const int64_t d = t.size(dim - 1), H = t.size(dim - 2), T = t.size(dim - 3), B = dim == 4 ? t.size(0) : 1;
    const int64_t row = dim == 4 && T <= 1 ? t.stride(0) : t.stride(dim - 3);
    if (B * T > 0 && ((d > 1 && t.stride(dim - 1) != 1) || (H > 1 && t.stride(dim - 2) != d))) Py_RETURN_NONE;
    if (B > 1 && T > 1 && t.stride(0) != T * row) Py_RETURN_NONE;
    return Py_BuildValue("(KLLLL)", (unsigned long long)(uintptr_t)t.data_ptr(), (long long)(B * T), (long long)H, (long long)d,
                         (long long)row);
  } catch (...) {
    PyErr_Clear();
    Py_RETURN_NONE;
  }
}

PyMethodDef methods[] = {
    {"rows", reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)(void)>(rows)), METH_FASTCALL, nullptr},
    {"need", reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)(void)>(need)), METH_FASTCALL, nullptr},
    {"set_refuse", set_refuse, METH_O, nullptr},
    {nullptr, nullptr, 0, nullptr}};
PyModuleDef module = {PyModuleDef_HEAD_INIT, "_kda_args", nullptr, -1, methods, nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__kda_args() {
  int major = 0, minor = 0;
  if (sscanf(Py_GetVersion(), "%d.%d", &major, &minor) != 2 || major != PY_MAJOR_VERSION || minor != PY_MINOR_VERSION) {
    PyErr_SetString(PyExc_ImportError, "_kda_args was built for another Python");
    return nullptr;
  }
  PyObject* m = PyModule_Create(&module);
  if (m && PyModule_AddStringConstant(m, "torch_version", KDA_TORCH_VERSION) != 0) Py_CLEAR(m);
  return m;
}
