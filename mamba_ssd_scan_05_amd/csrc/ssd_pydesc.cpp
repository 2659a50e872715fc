// ssd_pydesc.cpp -- the CPython module _pydesc: ssd_tensor descriptors of torch
// tensors, read from the tensors in C++.  The Python binding builds the
// same descriptors from t.shape, t.stride() and t.data_ptr(), at 0.7 us a
// tensor: half the host time of a small call (10 tensors: 6.9 us there, here
// under 1 us).  Marshalling only; nothing is computed here.
#include <torch/csrc/autograd/python_variable.h>

#include <cstddef>
#include <exception>

#include "ssd.h"

namespace {

constexpr Py_ssize_t kMaxTensors = 32;

int dtype_code(at::ScalarType t) {
  switch (t) {
  case at::kFloat: return SSD_F32;
  case at::kBFloat16: return SSD_BF16;
  case at::kByte:
  case at::kBool: return SSD_U8;
  case at::kInt: return SSD_I32;
  case at::kLong: return SSD_I64;
  default: return 99; // rejected by the library as SSD_ERR_DTYPE
  }
}

// pack(tensor_or_None, ...) -> tuple of descriptors or None.  A descriptor is
// a bytes object, which ctypes passes as the address of its contents: the
// tuple owns them, so a call made in between (by a signal handler, a
// finalizer, another thread) leaves them alone.  The contents of a bytes object
// lie behind a header of whole words, aligned to 8 bytes as ssd_tensor needs.
static_assert(alignof(ssd_tensor) <= 8 && offsetof(PyBytesObject, ob_sval) % 8 == 0, "descriptors in bytes objects");
PyObject *pack(PyObject *, PyObject *const *args, Py_ssize_t n) {
  if (n > kMaxTensors) {
    PyErr_SetString(PyExc_ValueError, "too many tensors in one call");
    return nullptr;
  }
  PyObject *out = PyTuple_New(n);
  if (!out) return nullptr;
  for (Py_ssize_t i = 0; i < n; ++i) {
    PyObject *item = nullptr;
    if (args[i] == Py_None) {
      Py_INCREF(Py_None);
      item = Py_None;
    } else if (!THPVariable_Check(args[i])) {
      PyErr_Format(PyExc_TypeError, "argument %zd is a %s, not a tensor", i, Py_TYPE(args[i])->tp_name);
    } else {
      try {
        const at::Tensor &t = THPVariable_Unpack(args[i]);
        const int64_t nd = t.dim();
        if (nd > 4) {
          PyErr_SetString(PyExc_ValueError, "ssd tensors have at most 4 dimensions");
        } else {
          ssd_tensor d;
          d.data = t.numel() ? t.data_ptr() : nullptr;
          d.dtype = dtype_code(t.scalar_type());
          d.ndim = (int32_t)nd;
          for (int64_t k = 0; k < 4; ++k) {
            d.shape[k] = k < nd ? t.size(k) : 0;
            d.strides[k] = k < nd ? t.stride(k) : 0;
          }
          item = PyBytes_FromStringAndSize(reinterpret_cast<const char *>(&d), sizeof d);
        }
      } catch (const std::exception &e) {
        PyErr_SetString(PyExc_RuntimeError, e.what());
      }
    }
    if (!item) {
      Py_DECREF(out);
      return nullptr;
    }
    PyTuple_SET_ITEM(out, i, item);
  }
  return out;
}

PyMethodDef kMethods[] = {
    {"pack", (PyCFunction)(void (*)(void))pack, METH_FASTCALL, "descriptors of the given tensors"},
    {nullptr, nullptr, 0, nullptr}};
PyModuleDef kModule = {PyModuleDef_HEAD_INIT, "_pydesc", "ssd_tensor descriptors of torch tensors", -1, kMethods,
                       nullptr, nullptr, nullptr, nullptr};

} // namespace

extern "C" __attribute__((visibility("default"))) PyObject *PyInit__pydesc(void) { return PyModule_Create(&kModule); }
