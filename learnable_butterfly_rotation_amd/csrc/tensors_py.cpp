// Python extension `_tensors`: the checks of torch tensors before their
// addresses go into a call of libbfly.  Reading type, shape, device and
// contiguity of 96 gradients and their outputs through Python costs 50 us, four
// times what the GPU needs to clip them, and of the eight tensors of a norm 4 us,
// as long as its kernel takes for a token.
#define PY_SSIZE_T_CLEAN  // lengths of bytes as Py_ssize_t
#include <torch/csrc/autograd/python_variable.h>

#include <algorithm>
#include <cstdint>
#include <exception>
#include <utility>
#include <vector>

namespace {

// Whether two of n ranges of bytes share any (empty ranges share none).
bool overlap(const uint64_t* at, const int64_t* numel, const int32_t* type, Py_ssize_t n) {
  const auto bytes = [&](Py_ssize_t i) { return (uint64_t)numel[i] * (type[i] ? 2 : 4); };
  bool ordered = true;  // as views of one buffer mostly are
  uint64_t end = 0;
  for (Py_ssize_t i = 0; i < n && ordered; ++i) {
    if (!numel[i]) continue;
    ordered = at[i] >= end;
    end = at[i] + bytes(i);
  }
  if (ordered) return false;
  std::vector<std::pair<uint64_t, uint64_t>> r;
  for (Py_ssize_t i = 0; i < n; ++i)
    if (numel[i]) r.emplace_back(at[i], at[i] + bytes(i));
  std::sort(r.begin(), r.end());
  for (size_t i = 1; i < r.size(); ++i)
    if (r[i].first < r[i - 1].second) return true;
  return false;
}

// describe(tensors, device, distinct) -> (addresses, element counts, bfly_dtype
// values) as bytes of uint64, int64 and int32.  Every item has to be a
// contiguous float32 or bfloat16 tensor on GPU `device`; with `distinct`, no
// two of them may overlap.
PyObject* describe(PyObject*, PyObject* args) {
  PyObject* given = nullptr;
  int device = -1, distinct = 0;
  if (!PyArg_ParseTuple(args, "Oip", &given, &device, &distinct)) return nullptr;
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
      if (i == n && distinct && overlap(a, c, t, n))
        PyErr_SetString(PyExc_ValueError, "two of the tensors to write overlap");
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

// apart(inputs, outputs, element counts, types), as describe gives them for two
// lists of like tensors whose outputs do not overlap: whether an output shares
// bytes with an input other than, exactly, its own.
PyObject* apart(PyObject*, PyObject* args) {
  const char *in, *out, *count, *kind;
  Py_ssize_t in_len, out_len, count_len, kind_len;
  if (!PyArg_ParseTuple(args, "y#y#y#y#", &in, &in_len, &out, &out_len, &count, &count_len, &kind,
                        &kind_len))
    return nullptr;
  const Py_ssize_t n = kind_len / 4;
  if (kind_len % 4 || in_len != n * 8 || out_len != n * 8 || count_len != n * 8)
    return PyErr_Format(PyExc_ValueError, "apart() takes four lists of one length");
  const auto* const from = reinterpret_cast<const uint64_t*>(in);
  const auto* const to = reinterpret_cast<const uint64_t*>(out);
  const auto* const numel = reinterpret_cast<const int64_t*>(count);
  const auto* const type = reinterpret_cast<const int32_t*>(kind);
  const auto bytes = [&](Py_ssize_t i) { return (uint64_t)numel[i] * (type[i] ? 2 : 4); };
  try {
    std::vector<std::pair<uint64_t, Py_ssize_t>> outs;  // address, index
    outs.reserve(n);
    for (Py_ssize_t i = 0; i < n; ++i)
      if (numel[i]) outs.emplace_back(to[i], i);
    if (!std::is_sorted(outs.begin(), outs.end())) std::sort(outs.begin(), outs.end());
    for (Py_ssize_t i = 0; i < n; ++i) {
      if (!numel[i]) continue;
      // the first output that ends behind the input's start, and those after it
      auto o = std::upper_bound(outs.begin(), outs.end(), std::make_pair(from[i], n));
      if (o != outs.begin() && (o - 1)->first + bytes((o - 1)->second) > from[i]) --o;
      for (; o != outs.end() && o->first < from[i] + bytes(i); ++o)
        if (o->second != i || o->first != from[i]) Py_RETURN_FALSE;
    }
  } catch (const std::exception& e) {
    return PyErr_Format(PyExc_RuntimeError, "%s", e.what());
  }
  Py_RETURN_TRUE;
}

// The types that `at` is told to take, as bits.
int kind_of(at::ScalarType s) {
  switch (s) {
    case at::kFloat: return 1;
    case at::kBFloat16: return 2;
    case at::kHalf: return 4;
    case at::kChar: return 8;
    case at::kByte: return 16;
    case at::kFloat8_e4m3fn: return 32;
    case at::kInt: return 64;
    default: return 0;
  }
}

// at(name, tensor, shape, kinds, device) -> the address of a tensor that is
// contiguous, of this shape, of one of these types and on GPU `device`; None
// for None.
PyObject* address(PyObject*, PyObject* const* args, Py_ssize_t n) {
  if (n != 5) return PyErr_Format(PyExc_TypeError, "at() takes five arguments");
  PyObject *const name = args[0], *const item = args[1], *const shape = args[2];
  if (item == Py_None) Py_RETURN_NONE;
  if (!THPVariable_Check(item)) return PyErr_Format(PyExc_TypeError, "%S is not a tensor", name);
  if (!PyTuple_Check(shape))
    return PyErr_Format(PyExc_TypeError, "the shape of %S has to be a tuple", name);
  const long kinds = PyLong_AsLong(args[3]), device = PyLong_AsLong(args[4]);
  if (PyErr_Occurred()) return nullptr;
  try {
    const at::Tensor& x = THPVariable_Unpack(item);
    if (!(kind_of(x.scalar_type()) & kinds))
      return PyErr_Format(PyExc_TypeError, "%S has the wrong type", name);
    bool same = x.layout() == at::kStrided && x.dim() == PyTuple_GET_SIZE(shape);
    for (int64_t i = 0; same && i < x.dim(); ++i) {
      const long long v = PyLong_AsLongLong(PyTuple_GET_ITEM(shape, i));
      if (v == -1 && PyErr_Occurred()) return nullptr;
      same = x.size(i) == v;
    }
    if (!same || !x.is_contiguous())
      return PyErr_Format(PyExc_ValueError, "%S has to be contiguous of shape %R", name, shape);
    if (!x.is_cuda() || x.get_device() != device)
      return PyErr_Format(PyExc_ValueError, "%S has to be on GPU %ld", name, device);
    return PyLong_FromVoidPtr(x.data_ptr());
  } catch (const std::exception& e) {
    return PyErr_Format(PyExc_RuntimeError, "%S: %s", name, e.what());
  }
}

// scratch(workspace, device) -> its address and bytes; (None, 0) for None.
PyObject* scratch(PyObject*, PyObject* const* args, Py_ssize_t n) {
  if (n != 2) return PyErr_Format(PyExc_TypeError, "scratch() takes two arguments");
  const long device = PyLong_AsLong(args[1]);
  if (PyErr_Occurred()) return nullptr;
  if (args[0] == Py_None) return Py_BuildValue("Oi", Py_None, 0);
  if (!THPVariable_Check(args[0]))
    return PyErr_Format(PyExc_TypeError, "the workspace is not a tensor");
  try {
    const at::Tensor& x = THPVariable_Unpack(args[0]);
    if (!x.is_cuda() || x.get_device() != device || x.layout() != at::kStrided ||
        !x.is_contiguous())
      return PyErr_Format(PyExc_ValueError, "the workspace has to be contiguous and on GPU %ld",
                          device);
    return Py_BuildValue("KK", (unsigned long long)reinterpret_cast<uintptr_t>(x.data_ptr()),
                         (unsigned long long)x.nbytes());
  } catch (const std::exception& e) {
    return PyErr_Format(PyExc_RuntimeError, "the workspace: %s", e.what());
  }
}

PyMethodDef methods[] = {
    {"scratch", reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(scratch)),
     METH_FASTCALL, "a workspace's address and bytes"},
    {"at", reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(address)), METH_FASTCALL,
     "the address of a tensor that is as it has to be"},
    {"describe", describe, METH_VARARGS, "addresses, element counts and types of tensors"},
    {"apart", apart, METH_VARARGS, "whether outputs overlap no input but their own"},
    {nullptr, nullptr, 0, nullptr}};
PyModuleDef module = {PyModuleDef_HEAD_INIT, "_tensors", nullptr, -1, methods,
                      nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__tensors() { return PyModule_Create(&module); }
