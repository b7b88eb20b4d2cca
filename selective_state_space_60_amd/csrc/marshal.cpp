// The per-call steps of the Python binding that touch every tensor, as a
// CPython module: reading what a descriptor depends on, allocating outputs and
// workspace, and handing the data pointers to an entry point of libssm.
// Reading and handing over take 3 us of a decode step's call in Python (ten
// tensors; a kernel launch is 2.5 us) and 0.4 us here.
#include <Python.h>

#include <ATen/ATen.h>
#include <torch/csrc/Dtype.h>
#include <torch/csrc/Exceptions.h>
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

// Exceptions become the Python errors that torch makes of its own (an
// allocation that fails is torch.OutOfMemoryError).
template <class F>
PyObject* guarded(F f) {
  try {
    return f();
  } catch (...) {
    torch::translate_exception_to_python(std::current_exception());
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

// The type of a dtype or, for None, of `t`; a Python error and false otherwise.
bool type_of(PyObject* o, const at::Tensor& t, at::ScalarType* type) {
  if (o == Py_None) {
    *type = t.scalar_type();
  } else if (THPDtype_Check(o)) {
    *type = reinterpret_cast<THPDtype*>(o)->scalar_type;
  } else {
    PyErr_SetString(PyExc_TypeError, "expected a dtype or None");
    return false;
  }
  return true;
}

// like(tensor, dtype): memory of the tensor's shape and, if it is dense, strides.
PyObject* like(PyObject*, PyObject* const* args, Py_ssize_t nargs) {
  const at::Tensor* t;
  if (nargs != 2) {
    PyErr_SetString(PyExc_TypeError, "like(tensor, dtype)");
    return nullptr;
  }
  if (!tensor_of(args[0], &t)) return nullptr;
  return guarded([&]() -> PyObject* {
    at::ScalarType type;
    if (!t) {
      PyErr_SetString(PyExc_TypeError, "expected a tensor");
      return nullptr;
    }
    if (!type_of(args[1], *t, &type)) return nullptr;
    at::AutoDispatchBelowADInplaceOrView plain;
    return THPVariable_Wrap(at::empty_like(*t, t->options().dtype(type)));
  });
}

// empty(tensor, shape, dtype): contiguous memory on the tensor's device.
PyObject* empty(PyObject*, PyObject* const* args, Py_ssize_t nargs) {
  const at::Tensor* t;
  if (nargs != 3 || !PyTuple_Check(args[1])) {
    PyErr_SetString(PyExc_TypeError, "empty(tensor, shape, dtype)");
    return nullptr;
  }
  if (!tensor_of(args[0], &t)) return nullptr;
  return guarded([&]() -> PyObject* {
    at::ScalarType type;
    if (!t) {
      PyErr_SetString(PyExc_TypeError, "expected a tensor");
      return nullptr;
    }
    if (!type_of(args[2], *t, &type)) return nullptr;
    at::DimVector shape;
    for (Py_ssize_t i = 0; i < PyTuple_GET_SIZE(args[1]); ++i) {
      shape.push_back(PyLong_AsLongLong(PyTuple_GET_ITEM(args[1], i)));
      if (PyErr_Occurred()) return nullptr;
    }
    at::AutoDispatchBelowADInplaceOrView plain;
    return THPVariable_Wrap(at::empty(shape, t->options().dtype(type)));
  });
}

// launch(entry, descriptor, tensors, written, bytes, stream): the entry point's
// status.  Entry, descriptor and stream are addresses.  written: bit i says that
// tensor i is written; the others are only read, so that a lazily copied one
// stays shared.  bytes: size of the workspace, which is allocated on the first
// tensor's device for the current stream; < 0: an entry point without one.
PyObject* launch(PyObject*, PyObject* const* args, Py_ssize_t nargs) {
  if (nargs != 6 || !PyTuple_Check(args[2])) {
    PyErr_SetString(PyExc_TypeError, "launch(entry, descriptor, tensors, written, bytes, stream)");
    return nullptr;
  }
  return guarded([&]() -> PyObject* {
    void* const entry = PyLong_AsVoidPtr(args[0]);
    void* const desc = PyLong_AsVoidPtr(args[1]);
    const unsigned long written = PyLong_AsUnsignedLong(args[3]);
    const long long bytes = PyLong_AsLongLong(args[4]);
    void* const stream = PyLong_AsVoidPtr(args[5]);
    if (PyErr_Occurred()) return nullptr;
    const Py_ssize_t n = PyTuple_GET_SIZE(args[2]);
    if (!entry || n > kMaxTensors) {
      PyErr_SetString(PyExc_ValueError, "no entry point, or too many tensors");
      return nullptr;
    }
    const void* ptrs[kMaxTensors];
    const at::Tensor* first = nullptr;
    // the written ones first: one that is read as well gets its own memory there
    for (const bool write : {true, false})
      for (Py_ssize_t i = 0; i < n; ++i) {
        const at::Tensor* t;
        if ((written >> i & 1) != write) continue;
        if (!tensor_of(PyTuple_GET_ITEM(args[2], i), &t)) return nullptr;
        ptrs[i] = !t ? nullptr : write ? t->mutable_data_ptr() : t->const_data_ptr();
        if (t && (!first || i == 0)) first = t;
      }
    at::Tensor ws;
    if (bytes > 0) {
      if (!first) {
        PyErr_SetString(PyExc_ValueError, "no tensor");
        return nullptr;
      }
      at::AutoDispatchBelowADInplaceOrView plain;
      ws = at::empty({(int64_t)bytes}, first->options().dtype(at::kByte));
    }
    int status;
    Py_BEGIN_ALLOW_THREADS
    if (bytes < 0)
      status = ((int (*)(const void*, const void*, void*))entry)(desc, ptrs, stream);
    else
      status = ((int (*)(const void*, const void*, void*, size_t, void*))entry)(
          desc, ptrs, bytes ? ws.mutable_data_ptr() : nullptr, (size_t)bytes, stream);
    Py_END_ALLOW_THREADS
    return PyLong_FromLong(status);
  });
}

PyMethodDef methods[] = {
    {"signature", signature, METH_O, "Type, device, sizes and strides of a tuple of tensors, as bytes."},
    {"like", (PyCFunction)(void (*)(void))like, METH_FASTCALL, "Memory like a tensor's, of a dtype or (None) its own."},
    {"empty", (PyCFunction)(void (*)(void))empty, METH_FASTCALL, "Contiguous memory on a tensor's device."},
    {"launch", (PyCFunction)(void (*)(void))launch, METH_FASTCALL, "Call an entry point on a tuple of tensors."},
    {nullptr, nullptr, 0, nullptr}};

PyModuleDef module = {PyModuleDef_HEAD_INIT, "_marshal", nullptr, -1, methods};

}  // namespace

PyMODINIT_FUNC PyInit__marshal(void) { return PyModule_Create(&module); }
