// Python extension `_tensors`: what a list of torch tensors is made of, for the
// calls of libbfly that take many of them.  Reading address, size, type,
// device and contiguity of 96 gradients and their outputs through Python
// costs 50 us, four times what the GPU needs to clip them.
#include <torch/csrc/autograd/python_variable.h>

#include <cstdint>
#include <exception>

namespace {

// describe(tensors, device) -> (addresses, element counts, bfly_dtype values)
// as bytes of uint64, int64 and int32.  Every item has to be a contiguous
// float32 or bfloat16 tensor on GPU `device`.
PyObject* describe(PyObject*, PyObject* args) {
  PyObject* given = nullptr;
  int device = -1;
  if (!PyArg_ParseTuple(args, "Oi", &given, &device)) return nullptr;
  PyObject* items = PySequence_Fast(given, "a list or tuple of tensors is needed");
  if (!items) return nullptr;
  const Py_ssize_t n = PySequence_Fast_GET_SIZE(items);
  PyObject* at = PyBytes_FromStringAndSize(nullptr, n * 8);
  PyObject* numel = PyBytes_FromStringAndSize(nullptr, n * 8);
  PyObject* type = PyBytes_FromStringAndSize(nullptr, n * 4);
  PyObject* result = nullptr;
  if (at && numel && type) {
    auto* const a = reinterpret_cast<uint64_t*>(PyBytes_AS_STRING(at));
    auto* const c = reinterpret_cast<int64_t*>(PyBytes_AS_STRING(numel));
    auto* const t = reinterpret_cast<int32_t*>(PyBytes_AS_STRING(type));
    Py_ssize_t i = 0;
    try {
      for (; i < n; ++i) {
        PyObject* item = PySequence_Fast_GET_ITEM(items, i);
        if (!THPVariable_Check(item)) {
          PyErr_Format(PyExc_TypeError, "item %zd is not a tensor", i);
          break;
        }
        const at::Tensor& x = THPVariable_Unpack(item);
        const auto s = x.scalar_type();
        if (s != at::kFloat && s != at::kBFloat16) {
          PyErr_Format(PyExc_TypeError, "tensor %zd is neither float32 nor bfloat16", i);
          break;
        }
        if (!x.is_cuda() || x.get_device() != device) {
          PyErr_Format(PyExc_ValueError, "tensor %zd is not on GPU %d", i, device);
          break;
        }
        if (x.layout() != at::kStrided || !x.is_contiguous()) {
          PyErr_Format(PyExc_ValueError, "tensor %zd is not contiguous", i);
          break;
        }
        a[i] = reinterpret_cast<uint64_t>(x.data_ptr());
        c[i] = x.numel();
        t[i] = s == at::kBFloat16 ? 1 : 0;
      }
    } catch (const std::exception& e) {
      PyErr_Format(PyExc_RuntimeError, "tensor %zd: %s", i, e.what());
    }
    if (!PyErr_Occurred()) result = PyTuple_Pack(3, at, numel, type);
  }
  Py_XDECREF(at);
  Py_XDECREF(numel);
  Py_XDECREF(type);
  Py_DECREF(items);
  return result;
}

PyMethodDef methods[] = {
    {"describe", describe, METH_VARARGS, "addresses, element counts and types of tensors"},
    {nullptr, nullptr, 0, nullptr}};
PyModuleDef module = {PyModuleDef_HEAD_INIT, "_tensors", nullptr, -1, methods,
                      nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__tensors() { return PyModule_Create(&module); }
