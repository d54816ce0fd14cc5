// marshal.cpp -- the binding's check of one tensor argument, as a CPython extension.
//
// A call here takes three to five tensors, and asking one of them in Python for its device,
// layout, type, size and pointer costs 0.32 us of the 5.1 that a call with a launch takes on
// the host; from C it is 0.05 (four tensors: 4.0 us a call).
#include <torch/csrc/Dtype.h>
#include <torch/csrc/DynamicTypes.h>
#include <torch/csrc/autograd/python_variable.h>

namespace {

// the check in Python, which takes what is left to it here: objects that answer like a tensor but
// are none, or of a subclass whose answers may be its own, and sizes beyond 64 bits
PyObject* python_buf = nullptr;

// buf(t, name, n, kinds, device): _buf in __init__.py
PyObject* buf(PyObject*, PyObject* const* args, Py_ssize_t nargs) {
  if (nargs != 5 || !PyUnicode_Check(args[1]) || !(args[3] == Py_None || PyTuple_Check(args[3]))) {
    PyErr_SetString(PyExc_TypeError, "buf(t, name, n, kinds, device)");
    return nullptr;
  }
  PyObject *o = args[0], *name = args[1], *kinds = args[3];
  if (o == Py_None || PyLong_CheckExact(o)) {
    Py_INCREF(o);
    return o;
  }
  if (!THPVariable_CheckExact(o)) {  // a Parameter is taken as exact
    if (python_buf && PyObject_HasAttrString(o, "data_ptr")) return PyObject_Vectorcall(python_buf, args, nargs, nullptr);
    return PyErr_Format(PyExc_TypeError, "%U: %S is not a tensor, None or a pointer", name, Py_TYPE(o));
  }
  const long long n = PyLong_AsLongLong(args[2]);
  if (n == -1 && PyErr_Occurred()) {
    if (!python_buf || !PyErr_ExceptionMatches(PyExc_OverflowError)) return nullptr;
    PyErr_Clear();
    return PyObject_Vectorcall(python_buf, args, nargs, nullptr);
  }
  const long long device = PyLong_AsLongLong(args[4]);
  if (device == -1 && PyErr_Occurred()) return nullptr;
  try {
    const at::Tensor& t = THPVariable_Unpack(o);
    if (t.get_device() != device)
      return PyErr_Format(PyExc_ValueError, "%U: tensor is not on the current GPU device", name);
    if (!t.is_contiguous()) return PyErr_Format(PyExc_ValueError, "%U: tensor is not contiguous", name);
    if (kinds != Py_None) {
      PyObject* type = reinterpret_cast<PyObject*>(torch::getTHPDtype(t.scalar_type()));
      bool in = false;
      for (Py_ssize_t i = 0; i < PyTuple_GET_SIZE(kinds); ++i) in = in || PyTuple_GET_ITEM(kinds, i) == type;
      if (!in) return PyErr_Format(PyExc_ValueError, "%U: dtype %S, expected one of %S", name, type, kinds);
    }
    if (t.numel() < n)
      return PyErr_Format(PyExc_ValueError, "%U: %lld elements, %lld are needed", name,
                          static_cast<long long>(t.numel()), n);
    return PyLong_FromVoidPtr(t.data_ptr());
  } catch (const std::exception& e) {  // a tensor without storage, say
    return PyErr_Format(PyExc_RuntimeError, "%U: %s", name, e.what());
  }
}

PyObject* set_python(PyObject*, PyObject* f) {
  Py_INCREF(f);
  Py_XSETREF(python_buf, f);
  Py_RETURN_NONE;
}

PyMethodDef methods[] = {
    {"buf", reinterpret_cast<PyCFunction>(reinterpret_cast<void*>(buf)), METH_FASTCALL, nullptr},
    {"set_python", set_python, METH_O, nullptr},
    {nullptr}};
PyModuleDef module = {PyModuleDef_HEAD_INIT, "_marshal", nullptr, -1, methods};

}  // namespace

// torch_build: the torch whose layouts are compiled in; the binding asks before it uses buf
PyMODINIT_FUNC PyInit__marshal() {
  PyObject* m = PyModule_Create(&module);
  if (m && PyModule_AddStringConstant(m, "torch_build", MARSHAL_TORCH) < 0) Py_CLEAR(m);
  return m;
}
