// marshal.cpp -- the binding's argument checks in C++: lists of rank tensors
// to arrays of their addresses.  A call of the attention operators names up to 40
// tensors; looked at from Python each costs about a microsecond, more than the
// kernels of a decode step.  Every function returns None where a check fails;
// the binding then repeats the checks in Python, which names what is wrong.
#define PY_SSIZE_T_CLEAN
#include <torch/csrc/Dtype.h>
#include <torch/csrc/autograd/python_variable.h>

#include <cstdint>

namespace {

constexpr Py_ssize_t MAX = 8;  // ranks

struct List {
  PyObject* items;
  Py_ssize_t n;
  at::ScalarType type;
  long device;
};

// (list, dtype, device, ...): the first three arguments of a call.
bool list_of(PyObject* const* args, List* l) {
  l->items = args[0];
  if (!PyList_CheckExact(l->items) && !PyTuple_CheckExact(l->items)) return false;
  l->n = PySequence_Fast_GET_SIZE(l->items);
  if (l->n < 1 || l->n > MAX || !THPDtype_Check(args[1])) return false;
  l->type = reinterpret_cast<THPDtype*>(args[1])->scalar_type;
  l->device = PyLong_AsLong(args[2]);
  return !PyErr_Occurred();
}

// The i-th tensor, if it has the call's type and device.
const at::Tensor* tensor_of(PyObject* o, at::ScalarType type, long device) {
  if (!THPVariable_Check(o)) return nullptr;
  const at::Tensor& t = THPVariable_Unpack(o);
  if (t.layout() != at::kStrided || t.scalar_type() != type || t.get_device() != device) return nullptr;
  return &t;
}

// contiguous(list, dtype, device, shape) -> the addresses, as bytes
PyObject* contiguous(PyObject*, PyObject* const* args, Py_ssize_t nargs) {
  List l;
  if (nargs != 4 || !list_of(args, &l) || !PyTuple_Check(args[3])) Py_RETURN_NONE;
  const Py_ssize_t dims = PyTuple_GET_SIZE(args[3]);
  int64_t shape[4];
  if (dims > 4) Py_RETURN_NONE;
  for (Py_ssize_t d = 0; d < dims; ++d) {
    shape[d] = PyLong_AsLongLong(PyTuple_GET_ITEM(args[3], d));
    if (PyErr_Occurred()) return nullptr;
  }
  uint64_t at[MAX];
  for (Py_ssize_t i = 0; i < l.n; ++i) {
    const at::Tensor* t = tensor_of(PySequence_Fast_GET_ITEM(l.items, i), l.type, l.device);
    if (!t || t->sizes() != at::IntArrayRef(shape, dims) || !t->is_contiguous()) Py_RETURN_NONE;
    at[i] = reinterpret_cast<uint64_t>(t->data_ptr());
  }
  return PyBytes_FromStringAndSize(reinterpret_cast<char*>(at), l.n * 8);
}

// rows(list, dtype, device, rows, heads, dim) -> (the addresses, elements from
// row to row): [rows, heads, dim] with each row's heads side by side
PyObject* rows(PyObject*, PyObject* const* args, Py_ssize_t nargs) {
  List l;
  if (nargs != 6 || !list_of(args, &l)) Py_RETURN_NONE;
  int64_t shape[3];
  for (int d = 0; d < 3; ++d) {
    shape[d] = PyLong_AsLongLong(args[3 + d]);
    if (PyErr_Occurred()) return nullptr;
  }
  uint64_t at[MAX];
  int64_t stride = shape[1] * shape[2];
  for (Py_ssize_t i = 0; i < l.n; ++i) {
    const at::Tensor* t = tensor_of(PySequence_Fast_GET_ITEM(l.items, i), l.type, l.device);
    if (!t || t->sizes() != at::IntArrayRef(shape, 3)) Py_RETURN_NONE;
    const at::IntArrayRef s = t->strides();
    if (shape[0] && shape[1] && (s[2] != 1 || (shape[1] > 1 && s[1] != shape[2]))) Py_RETURN_NONE;
    if (shape[0] > 1) {
      if (i && s[0] != stride) Py_RETURN_NONE;
      stride = s[0];
    }
    at[i] = reinterpret_cast<uint64_t>(t->data_ptr());
  }
  return Py_BuildValue("(y#L)", reinterpret_cast<char*>(at), l.n * 8, (long long)stride);
}

// vector(tensor, dtype, device, n) -> the address of a contiguous vector of n
PyObject* vector(PyObject*, PyObject* const* args, Py_ssize_t nargs) {
  if (nargs != 4 || !THPDtype_Check(args[1])) Py_RETURN_NONE;
  const long device = PyLong_AsLong(args[2]);
  const int64_t n = PyLong_AsLongLong(args[3]);
  if (PyErr_Occurred()) return nullptr;
  const at::Tensor* t = tensor_of(args[0], reinterpret_cast<THPDtype*>(args[1])->scalar_type, device);
  if (!t || t->dim() != 1 || t->size(0) != n || !t->is_contiguous()) Py_RETURN_NONE;
  return PyLong_FromUnsignedLongLong((unsigned long long)t->data_ptr());
}

// sequences(table, first, at, device) -> (addresses of the three, table stride,
// width, sequences)
PyObject* sequences(PyObject*, PyObject* const* args, Py_ssize_t nargs) {
  if (nargs != 4) Py_RETURN_NONE;
  const long device = PyLong_AsLong(args[3]);
  if (PyErr_Occurred()) return nullptr;
  const at::Tensor* t[3];
  for (int i = 0; i < 3; ++i) {
    t[i] = tensor_of(args[i], at::kInt, device);
    if (!t[i] || t[i]->dim() != (i ? 1 : 2)) Py_RETURN_NONE;
    const int64_t d = t[i]->dim() - 1;
    if (t[i]->size(d) > 1 && t[i]->stride(d) != 1) Py_RETURN_NONE;
  }
  const int64_t seqs = t[0]->size(0), width = t[0]->size(1), stride = seqs > 1 ? t[0]->stride(0) : width;
  if (t[1]->size(0) != seqs + 1 || t[2]->size(0) != seqs || stride < width) Py_RETURN_NONE;
  return Py_BuildValue("(KKKLLL)", (unsigned long long)t[0]->data_ptr(), (unsigned long long)t[1]->data_ptr(),
                       (unsigned long long)t[2]->data_ptr(), (long long)stride, (long long)width, (long long)seqs);
}

// A tensor without memory or with symbolic sizes throws when asked for them: a
// failed check as any other.
template <PyObject* (*F)(PyObject*, PyObject* const*, Py_ssize_t)>
PyObject* guarded(PyObject* self, PyObject* const* args, Py_ssize_t nargs) {
  try {
    return F(self, args, nargs);
  } catch (...) {
    PyErr_Clear();
    Py_RETURN_NONE;
  }
}

PyMethodDef METHODS[] = {
    {"contiguous", (PyCFunction)(void (*)(void))guarded<contiguous>, METH_FASTCALL, nullptr},
    {"rows", (PyCFunction)(void (*)(void))guarded<rows>, METH_FASTCALL, nullptr},
    {"vector", (PyCFunction)(void (*)(void))guarded<vector>, METH_FASTCALL, nullptr},
    {"sequences", (PyCFunction)(void (*)(void))guarded<sequences>, METH_FASTCALL, nullptr},
    {nullptr, nullptr, 0, nullptr},
};

PyModuleDef MODULE = {PyModuleDef_HEAD_INIT, "_marshal", nullptr, -1, METHODS, nullptr, nullptr, nullptr, nullptr};

}  // namespace

// BUILT_FOR: the torch and Python this was compiled against; the binding uses no other's.
PyMODINIT_FUNC PyInit__marshal() {
  PyObject* m = PyModule_Create(&MODULE);
  if (m && PyModule_AddStringConstant(m, "BUILT_FOR", BUILT_FOR) != 0) Py_CLEAR(m);
  return m;
}
