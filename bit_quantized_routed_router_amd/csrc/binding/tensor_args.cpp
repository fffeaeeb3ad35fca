// Tensor arguments of the Python binding: checked against what a call reads
// and writes, and turned into the addresses that the C functions take.
//
//   addresses(name, device, args) -> list
//
// An argument that is a tuple (tensor, count, held) must be a contiguous
// tensor on GPU `device` that holds at least `count` values of the types
// `held` names, and becomes its address; None and an int in the tensor's
// place go through unchecked, as do arguments that are no tuples.  Host time of
// a combine call of 16 tokens, its launch included: 4.6 us; with the same
// checks in Python 6.4, with Python's loop without them 5.6.
#include <Python.h>
#include <torch/csrc/autograd/python_variable.h>

#include <exception>

namespace {

// what a tensor may hold: the library's type codes (bfloat16 also as its
// bits; a code that is none of them is the library's to refuse), int32, bytes
// of any type
enum Held { kF32 = 0, kBf16 = 1, kI32 = 100, kBytes = 101 };

bool holds(c10::ScalarType t, long held) {
  switch (held) {
    case kF32: return t == c10::ScalarType::Float;
    case kBf16: return t == c10::ScalarType::BFloat16 || t == c10::ScalarType::Short || t == c10::ScalarType::UInt16;
    case kI32: return t == c10::ScalarType::Int;
    default: return true;
  }
}
const char* held_name(long held) { return held == kF32 ? "float32" : held == kBf16 ? "bfloat16" : "int32"; }

// The address of item (tensor, count, held) as a new reference, or null with
// the error set.
PyObject* address(PyObject* name, long device, PyObject* item) {
  if (PyTuple_GET_SIZE(item) != 3) {
    PyErr_SetString(PyExc_TypeError, "expected (tensor, count, held)");
    return nullptr;
  }
  PyObject* obj = PyTuple_GET_ITEM(item, 0);
  if (!THPVariable_Check(obj)) {
    Py_INCREF(obj);
    return obj;
  }
  int past = 0;  // a count beyond 64 bits is more than any tensor holds
  const long long count = PyLong_AsLongLongAndOverflow(PyTuple_GET_ITEM(item, 1), &past);
  if (count == -1 && PyErr_Occurred()) return nullptr;
  const long held = PyLong_AsLong(PyTuple_GET_ITEM(item, 2));
  if (held == -1 && PyErr_Occurred()) return nullptr;
  const at::Tensor& t = THPVariable_Unpack(obj);
  if (!holds(t.scalar_type(), held))
    return PyErr_Format(PyExc_ValueError, "%U: a tensor of dtype %s where the call takes %s", name,
                        c10::toString(t.scalar_type()), held_name(held));
  const long long has = held == kBytes ? (long long)t.nbytes() : (long long)t.numel();
  if (past > 0 || has < count)
    return PyErr_Format(PyExc_ValueError, "%U: a tensor of %lld %s where the call takes %S", name, has,
                        held == kBytes ? "bytes" : "values", PyTuple_GET_ITEM(item, 1));
  if (!t.is_cuda() || t.get_device() != device || !t.is_contiguous())
    return PyErr_Format(PyExc_ValueError, "%U: tensors must be contiguous and on the current GPU", name);
  return PyLong_FromVoidPtr(t.data_ptr());
}

PyObject* addresses(PyObject*, PyObject* const* a, Py_ssize_t n) {
  if (n != 3 || !PyUnicode_Check(a[0]) || !PyTuple_Check(a[2])) {
    PyErr_SetString(PyExc_TypeError, "addresses(name, device, args)");
    return nullptr;
  }
  const long device = PyLong_AsLong(a[1]);
  if (device == -1 && PyErr_Occurred()) return nullptr;
  const Py_ssize_t m = PyTuple_GET_SIZE(a[2]);
  PyObject* out = PyList_New(m);
  if (!out) return nullptr;
  try {
    for (Py_ssize_t i = 0; i < m; ++i) {
      PyObject* v = PyTuple_GET_ITEM(a[2], i);
      if (PyTuple_CheckExact(v))
        v = address(a[0], device, v);
      else
        Py_INCREF(v);
      if (!v) {
        Py_DECREF(out);
        return nullptr;
      }
      PyList_SET_ITEM(out, i, v);
    }
  } catch (const std::exception& e) {  // a tensor without plain storage
    Py_DECREF(out);
    return PyErr_Format(PyExc_ValueError, "%U: %.300s", a[0], e.what());
  }
  return out;
}

PyMethodDef kMethods[] = {
    {"addresses", (PyCFunction)(void (*)(void))addresses, METH_FASTCALL,
     "addresses(name, device, args): the arguments with every (tensor, count, held) checked and as its address"},
    {nullptr, nullptr, 0, nullptr}};
PyModuleDef kModule = {PyModuleDef_HEAD_INIT, "_tensor_args", nullptr, -1, kMethods};

}  // namespace

PyMODINIT_FUNC PyInit__tensor_args() { return PyModule_Create(&kModule); }
