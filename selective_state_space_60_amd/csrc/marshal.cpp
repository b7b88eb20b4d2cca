// The two per-call steps of the Python binding that touch every tensor, as a
// CPython module: reading what a descriptor depends on, and handing the data
// pointers to an entry point of libssm.  In Python they take 3 us of a decode
// step's call (ten tensors; a kernel launch is 2.5 us), here 0.4 us.
#include <Python.h>

#include <ATen/core/Tensor.h>
#include <torch/csrc/autograd/python_variable.h>

#include <cstdint>
#include <exception>
#include <string>

namespace {

constexpr Py_ssize_t kMaxTensors = 32;

// The tensor of an argument, null for None; a Python error and false otherwise.
bool tensor_of(PyObject* o, const at::Tensor** t) {
  *t = nullptr;
  if (o == Py_None) return true;
  if (!THPVariable_Check(o)) {
    PyErr_SetString(PyExc_TypeError, "expected a tensor or None");
    return false;
  }
  *t = &THPVariable_Unpack(o);
  return true;
}

template <class F>
PyObject* guarded(F f) {
  try {
    return f();
  } catch (const std::exception& e) {
    PyErr_SetString(PyExc_RuntimeError, e.what());
    return nullptr;
  }
}

// signature(tensors): type, device, sizes and strides of every tensor, as bytes.
PyObject* signature(PyObject*, PyObject* arg) {
  if (!PyTuple_Check(arg)) {
    PyErr_SetString(PyExc_TypeError, "signature takes a tuple");
    return nullptr;
  }
  return guarded([&]() -> PyObject* {
    std::string s;
    s.reserve(512);
    auto put = [&](int64_t v) { s.append((const char*)&v, sizeof(v)); };
    const Py_ssize_t n = PyTuple_GET_SIZE(arg);
    for (Py_ssize_t i = 0; i < n; ++i) {
      const at::Tensor* t;
      if (!tensor_of(PyTuple_GET_ITEM(arg, i), &t)) return nullptr;
      if (!t) {
        put(-1);
        continue;
      }
      const auto sizes = t->sizes(), strides = t->strides();
      const int64_t device = t->is_cuda() ? t->device().index() : -1;
      put((int64_t)sizes.size() << 32 | (int64_t)(uint8_t)t->scalar_type() << 16 | (device & 0xFFFF));
      for (const int64_t v : sizes) put(v);
      for (const int64_t v : strides) put(v);
    }
    return PyBytes_FromStringAndSize(s.data(), (Py_ssize_t)s.size());
  });
}

// launch(entry, descriptor, tensors, workspace, bytes, stream): the entry
// point's status.  All but the tensors are addresses or sizes; bytes < 0: an
// entry point without a workspace.
PyObject* launch(PyObject*, PyObject* const* args, Py_ssize_t nargs) {
  if (nargs != 6 || !PyTuple_Check(args[2])) {
    PyErr_SetString(PyExc_TypeError, "launch(entry, descriptor, tensors, workspace, bytes, stream)");
    return nullptr;
  }
  return guarded([&]() -> PyObject* {
    void* const entry = PyLong_AsVoidPtr(args[0]);
    void* const desc = PyLong_AsVoidPtr(args[1]);
    void* const ws = PyLong_AsVoidPtr(args[3]);
    const long long bytes = PyLong_AsLongLong(args[4]);
    void* const stream = PyLong_AsVoidPtr(args[5]);
    if (PyErr_Occurred()) return nullptr;
    const Py_ssize_t n = PyTuple_GET_SIZE(args[2]);
    if (!entry || n > kMaxTensors) {
      PyErr_SetString(PyExc_ValueError, "no entry point, or too many tensors");
      return nullptr;
    }
    void* ptrs[kMaxTensors];
    for (Py_ssize_t i = 0; i < n; ++i) {
      const at::Tensor* t;
      if (!tensor_of(PyTuple_GET_ITEM(args[2], i), &t)) return nullptr;
      ptrs[i] = t ? t->mutable_data_ptr() : nullptr;
    }
    int status;
    Py_BEGIN_ALLOW_THREADS
    if (bytes < 0)
      status = ((int (*)(const void*, const void*, void*))entry)(desc, ptrs, stream);
    else
      status = ((int (*)(const void*, const void*, void*, size_t, void*))entry)(desc, ptrs, ws, (size_t)bytes, stream);
    Py_END_ALLOW_THREADS
    return PyLong_FromLong(status);
  });
}

PyMethodDef methods[] = {
    {"signature", signature, METH_O, "Type, device, sizes and strides of a tuple of tensors, as bytes."},
    {"launch", (PyCFunction)(void (*)(void))launch, METH_FASTCALL, "Call an entry point on a tuple of tensors."},
    {nullptr, nullptr, 0, nullptr}};

PyModuleDef module = {PyModuleDef_HEAD_INIT, "_marshal", nullptr, -1, methods};

}  // namespace

PyMODINIT_FUNC PyInit__marshal(void) { return PyModule_Create(&module); }
