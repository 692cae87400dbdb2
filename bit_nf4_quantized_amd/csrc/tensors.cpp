// Checks and device addresses of torch tensors for the ctypes binding, as one
// call each: the binding of a call with a few tensors, or with hundreds, would
// otherwise spend longer on them in Python than the GPU on the call.
//
//   address(t, dtype, shape, device, name) -> int
//       the address of tensor t after the checks of api._need: a contiguous
//       device tensor of that dtype, shape (a tuple) and device index (-1: any)
//   stream() -> int
//       the current stream of the current device (torch's own accessor builds a
//       Python object for it: 2.9 us)
//   addresses(ts, dtype, device, name, numel=None) -> (bytes, bytes)
//       the addresses and element counts of a list of tensors, as arrays of
//       int64; with numel (such an array) the counts must equal it
//
//   empties(device, dtype, shape, dtype, shape, ...) -> tuple
//       new device tensors (1.3 us each from Python)
//
// dtype: 0 float32, 1 bfloat16, 2 int32, 3 int64, 4 float64, 5 uint8. Failed checks raise TypeError
// or ValueError; C++ exceptions end here as RuntimeError.
#define PY_SSIZE_T_CLEAN
#include <Python.h>

#include <string.h>

#include <exception>
#include <string>
#include <vector>

#include <ATen/ops/empty.h>
#include <c10/hip/HIPStream.h>
#include <torch/csrc/Exceptions.h>
#include <torch/csrc/autograd/python_variable.h>

namespace {

const c10::ScalarType kTypes[] = {c10::ScalarType::Float, c10::ScalarType::BFloat16, c10::ScalarType::Int,
                                  c10::ScalarType::Long, c10::ScalarType::Double,   c10::ScalarType::Byte};
constexpr int kTypeCount = 6;

// nullptr after setting a Python error
const at::Tensor* tensor_of(PyObject* o, int dtype, long device, const char* name) {
  if (!THPVariable_Check(o)) {
    PyErr_Format(PyExc_TypeError, "%s must be a torch tensor", name);
    return nullptr;
  }
  const at::Tensor& t = THPVariable_Unpack(o);
  if (!t.is_cuda()) {
    PyErr_Format(PyExc_ValueError, "%s must be a device tensor", name);
    return nullptr;
  }
  if (t.scalar_type() != kTypes[dtype]) {
    PyErr_Format(PyExc_TypeError, "%s must be %s, got %s", name, c10::toString(kTypes[dtype]),
                 c10::toString(t.scalar_type()));
    return nullptr;
  }
  if (device >= 0 && t.get_device() != device) {
    PyErr_Format(PyExc_ValueError, "%s must be on device %ld, got %ld", name, device, (long)t.get_device());
    return nullptr;
  }
  if (!t.is_contiguous()) {
    PyErr_Format(PyExc_ValueError, "%s must be contiguous", name);
    return nullptr;
  }
  return &t;
}

PyObject* address(PyObject*, PyObject* const* args, Py_ssize_t n) {
  if (n != 5 || !PyTuple_Check(args[2])) {
    PyErr_SetString(PyExc_TypeError, "address(tensor, dtype, shape, device, name)");
    return nullptr;
  }
  try {
    const long dtype = PyLong_AsLong(args[1]), device = PyLong_AsLong(args[3]);
    const char* name = PyUnicode_AsUTF8(args[4]);
    if (!name || PyErr_Occurred()) return nullptr;
    if (dtype < 0 || dtype >= kTypeCount) {
      PyErr_SetString(PyExc_ValueError, "unknown dtype number");
      return nullptr;
    }
    const at::Tensor* t = tensor_of(args[0], (int)dtype, device, name);
    if (!t) return nullptr;
    const auto sizes = t->sizes();
    bool same = (Py_ssize_t)sizes.size() == PyTuple_GET_SIZE(args[2]);
    for (size_t i = 0; same && i < sizes.size(); ++i) {
      const long long want = PyLong_AsLongLong(PyTuple_GET_ITEM(args[2], (Py_ssize_t)i));
      if (want == -1 && PyErr_Occurred()) return nullptr;
      same = want == (long long)sizes[i];
    }
    if (!same) {
      std::string got = "(";
      for (size_t i = 0; i < sizes.size(); ++i) got += (i ? ", " : "") + std::to_string(sizes[i]);
      PyErr_Format(PyExc_ValueError, "%s must have shape %R, got %s)", name, args[2], got.c_str());
      return nullptr;
    }
    return PyLong_FromVoidPtr(t->data_ptr());
  } catch (const std::exception& e) {
    PyErr_SetString(PyExc_RuntimeError, e.what());
    return nullptr;
  }
}

PyObject* addresses(PyObject*, PyObject* const* args, Py_ssize_t n) {
  if ((n != 4 && n != 5) || !PyList_Check(args[0])) {
    PyErr_SetString(PyExc_TypeError, "addresses(list, dtype, device, name, numel=None)");
    return nullptr;
  }
  try {
    const long dtype = PyLong_AsLong(args[1]), device = PyLong_AsLong(args[2]);
    const char* name = PyUnicode_AsUTF8(args[3]);
    if (!name || PyErr_Occurred()) return nullptr;
    if (dtype < 0 || dtype >= kTypeCount) {
      PyErr_SetString(PyExc_ValueError, "unknown dtype number");
      return nullptr;
    }
    const Py_ssize_t count = PyList_GET_SIZE(args[0]);
    const char* want = nullptr;
    if (n == 5 && args[4] != Py_None) {
      Py_ssize_t bytes = 0;
      if (PyBytes_AsStringAndSize(args[4], const_cast<char**>(&want), &bytes) < 0) return nullptr;
      if (bytes != count * 8) {
        PyErr_Format(PyExc_ValueError, "%s must be one tensor per parameter (%zd), got %zd", name, bytes / 8, count);
        return nullptr;
      }
    }
    std::vector<int64_t> ptrs((size_t)count), numel((size_t)count);
    for (Py_ssize_t i = 0; i < count; ++i) {
      const at::Tensor* t = tensor_of(PyList_GET_ITEM(args[0], i), (int)dtype, device, name);
      if (!t) return nullptr;
      ptrs[(size_t)i] = (int64_t)reinterpret_cast<uintptr_t>(t->data_ptr());
      numel[(size_t)i] = t->numel();
    }
    if (want && count && memcmp(want, numel.data(), (size_t)count * 8) != 0) {
      PyErr_Format(PyExc_ValueError, "%s must have the parameters' sizes", name);
      return nullptr;
    }
    PyObject* p = PyBytes_FromStringAndSize(reinterpret_cast<const char*>(ptrs.data()), count * 8);
    PyObject* q = PyBytes_FromStringAndSize(reinterpret_cast<const char*>(numel.data()), count * 8);
    PyObject* both = p && q ? PyTuple_Pack(2, p, q) : nullptr;
    Py_XDECREF(p);
    Py_XDECREF(q);
    return both;
  } catch (const std::exception& e) {
    PyErr_SetString(PyExc_RuntimeError, e.what());
    return nullptr;
  }
}

PyObject* stream(PyObject*, PyObject*) {
  try {
    return PyLong_FromVoidPtr(c10::hip::getCurrentHIPStream().stream());
  } catch (const std::exception& e) {
    PyErr_SetString(PyExc_RuntimeError, e.what());
    return nullptr;
  }
}

PyObject* empties(PyObject*, PyObject* const* args, Py_ssize_t n) {
  HANDLE_TH_ERRORS   // an allocator's error stays torch's own
  if (n % 2 == 0) throw torch::TypeError("empties(device, dtype, shape, ...)");
  const long device = PyLong_AsLong(args[0]);
  if (PyErr_Occurred()) throw python_error();
  const auto on = c10::TensorOptions().device(c10::Device(c10::DeviceType::CUDA, (c10::DeviceIndex)device));
  std::vector<at::Tensor> made;
  std::vector<int64_t> sizes;
  for (Py_ssize_t i = 1; i < n; i += 2) {
    const long dtype = PyLong_AsLong(args[i]);
    if (PyErr_Occurred()) throw python_error();
    if (dtype < 0 || dtype >= kTypeCount || !PyTuple_Check(args[i + 1]))
      throw torch::TypeError("empties(device, dtype, shape, ...)");
    sizes.clear();
    for (Py_ssize_t k = 0; k < PyTuple_GET_SIZE(args[i + 1]); ++k) {
      sizes.push_back(PyLong_AsLongLong(PyTuple_GET_ITEM(args[i + 1], k)));
      if (PyErr_Occurred()) throw python_error();
    }
    made.push_back(at::empty(sizes, on.dtype(kTypes[dtype])));
  }
  PyObject* out = PyTuple_New((Py_ssize_t)made.size());
  if (!out) throw python_error();
  for (size_t i = 0; i < made.size(); ++i) PyTuple_SET_ITEM(out, (Py_ssize_t)i, THPVariable_Wrap(made[i]));
  return out;
  END_HANDLE_TH_ERRORS
}

PyMethodDef kMethods[] = {
    {"address", reinterpret_cast<PyCFunction>(reinterpret_cast<void*>(address)), METH_FASTCALL,
     "address(tensor, dtype, shape, device, name): the checked device address"},
    {"addresses", reinterpret_cast<PyCFunction>(reinterpret_cast<void*>(addresses)), METH_FASTCALL,
     "addresses(list, dtype, device, name, numel=None): checked addresses and sizes"},
    {"empties", reinterpret_cast<PyCFunction>(reinterpret_cast<void*>(empties)), METH_FASTCALL,
     "empties(device, dtype, shape, ...): new device tensors"},
    {"stream", stream, METH_NOARGS, "stream(): the current stream of the current device"},
    {nullptr, nullptr, 0, nullptr}};

PyModuleDef kModule = {PyModuleDef_HEAD_INIT, "_tensors", "checked device addresses of torch tensors", -1, kMethods,
                       nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__tensors(void) { return PyModule_Create(&kModule); }
