// Python extension `_tensors`: the calls of libbfly that take many small
// tensors, from torch tensors to addresses and sizes.  Through Python and
// ctypes the checks of a norm's eight tensors and its seventeen arguments cost
// 2 us, beside 3 us for the launch and 3 us of the GPU for a token; reading 96
// gradients and their outputs alone 50 us.
#define PY_SSIZE_T_CLEAN  // lengths of bytes as Py_ssize_t
#include <torch/csrc/autograd/python_variable.h>

#include <algorithm>
#include <climits>
#include <cstdint>
#include <exception>
#include <initializer_list>
#include <utility>
#include <vector>

#include "bfly.h"

namespace {

// The library's functions, by the addresses that bind() was given.
struct Library {
  decltype(&bfly_rmsnorm) rmsnorm;
  decltype(&bfly_rmsnorm_backward) rmsnorm_backward;
  decltype(&bfly_lora_matmul) lora_matmul;
  decltype(&bfly_grad_clip) grad_clip;
} library;

// A Python error has been set.
struct Raised {};

template <typename... T>
[[noreturn]] void fail(PyObject* type, const char* format, T... v) {
  PyErr_Format(type, format, v...);
  throw Raised();
}

// The types that a tensor may have, as bits.
constexpr int kF32 = 1, kBF16 = 2, kF16 = 4, kBytes = 8, kI32 = 16, kI8 = 32, kE4M3 = 64,
              kRows = kF32 | kBF16;
int kind_of(at::ScalarType s) {
  switch (s) {
    case at::kFloat: return kF32;
    case at::kBFloat16: return kBF16;
    case at::kHalf: return kF16;
    case at::kByte: return kBytes;
    case at::kChar: return kI8;
    case at::kFloat8_e4m3fn: return kE4M3;
    case at::kInt: return kI32;
    default: return 0;
  }
}
bfly_dtype dtype_of(const at::Tensor* t) {
  return t && t->scalar_type() == at::kBFloat16 ? BFLY_BF16 : BFLY_F32;
}

// The arguments of a call in their order: the stream, the GPU, the call's own.
class Args {
 public:
  Args(PyObject* const* args, Py_ssize_t n, Py_ssize_t want) : next_(args) {
    if (n != want) fail(PyExc_TypeError, "%zd arguments are needed, not %zd", want, n);
    stream = PyLong_AsVoidPtr(*next_++);
    if (!stream && PyErr_Occurred()) throw Raised();
    device_ = (long)integer();
  }
  void* stream;

  long long integer() {
    const long long v = PyLong_AsLongLong(*next_++);
    if (v == -1 && PyErr_Occurred()) throw Raised();
    return v;
  }
  int32_t int32(const char* name) { return narrow(name, integer()); }
  bool none() const { return *next_ == Py_None; }
  void skip() { ++next_; }
  float real() {
    const double v = PyFloat_AsDouble(*next_++);
    if (v == -1.0 && PyErr_Occurred()) throw Raised();
    return (float)v;
  }
  static int32_t narrow(const char* name, int64_t v) {
    if (v > INT32_MAX || v < INT32_MIN) fail(PyExc_ValueError, "%s is too large", name);
    return (int32_t)v;
  }
  PyObject* object() { return *next_++; }

  // A tensor of `dims` axes whose sizes the call is made with.
  const at::Tensor& sized(const char* name, int64_t dims) const {
    if (!THPVariable_Check(*next_)) fail(PyExc_TypeError, "%s is not a tensor", name);
    const at::Tensor& x = THPVariable_Unpack(*next_);
    if (x.dim() != dims) fail(PyExc_ValueError, "%s has to have %d axes", name, (int)dims);
    return x;
  }
  // The next argument, contiguous, of one of these types and this shape (its
  // address with `at`); nullptr for None.
  const at::Tensor* tensor(const char* name, int kinds, std::initializer_list<int64_t> shape) {
    PyObject* const item = *next_++;
    if (item == Py_None) return nullptr;
    if (!THPVariable_Check(item)) fail(PyExc_TypeError, "%s is not a tensor", name);
    const at::Tensor& x = THPVariable_Unpack(item);
    if (!(kind_of(x.scalar_type()) & kinds)) fail(PyExc_TypeError, "%s has the wrong type", name);
    if (x.layout() != at::kStrided || x.sizes() != at::IntArrayRef(shape))
      fail(PyExc_ValueError, "%s has the wrong shape", name);
    contiguous(name, x);
    return &x;
  }
  void* at(const char* name, int kinds, std::initializer_list<int64_t> shape) {
    const at::Tensor* const x = tensor(name, kinds, shape);
    return x ? x->data_ptr() : nullptr;
  }
  // A workspace of any shape and type.
  void* scratch(size_t& bytes) {
    PyObject* const item = *next_++;
    bytes = 0;
    if (item == Py_None) return nullptr;
    if (!THPVariable_Check(item)) fail(PyExc_TypeError, "the workspace is not a tensor");
    const at::Tensor& x = THPVariable_Unpack(item);
    if (x.layout() != at::kStrided) fail(PyExc_ValueError, "the workspace has to be contiguous");
    contiguous("the workspace", x);
    bytes = x.nbytes();
    return x.data_ptr();
  }
  void contiguous(const char* name, const at::Tensor& x) {
    if (!x.is_contiguous()) fail(PyExc_ValueError, "%s has to be contiguous", name);
    if (!elsewhere_ && (!x.is_cuda() || x.get_device() != device_)) elsewhere_ = name;
  }
  // Last: whether all tensors are on the call's GPU.
  void on_the_gpu() const {
    if (elsewhere_) fail(PyExc_ValueError, "%s has to be on GPU %ld", elsewhere_, device_);
  }

 private:
  PyObject* const* next_;
  long device_;
  const char* elsewhere_ = nullptr;  // the first tensor that is not
};

void* address(const at::Tensor* t) { return t ? t->data_ptr() : nullptr; }

// What a call returns, or raises: f() gives the library's status.
template <typename F>
PyObject* guarded(F f) {
  try {
    return PyLong_FromLong((long)f());
  } catch (const Raised&) {
    return nullptr;
  } catch (const std::exception& e) {
    return PyErr_Format(PyExc_RuntimeError, "%s", e.what());
  }
}
// The library's own work, which may wait for a full queue, without the GIL.
template <typename F>
bfly_status released(F f) {
  PyThreadState* const state = PyEval_SaveThread();
  const bfly_status s = f();
  PyEval_RestoreThread(state);
  return s;
}

// rmsnorm(stream, device, eps, format, group, x, weight, y, codes, scales,
// residual, h, rstd); group None: one scale a row.
PyObject* rmsnorm(PyObject*, PyObject* const* args, Py_ssize_t count) {
  return guarded([&] {
    Args a(args, count, 13);
    const float eps = a.real();
    const int32_t format = a.int32("format");
    const bool by_row = a.none();
    int32_t group = 0;
    if (by_row) a.skip();
    else group = a.int32("group");
    const at::Tensor& like = a.sized("x", 2);
    const int64_t rows = like.size(0), n = like.size(1);
    const int32_t width = Args::narrow("a row", n);
    const at::Tensor* const x = a.tensor("x", kRows, {rows, n});
    const int same = kind_of(x->scalar_type());
    const at::Tensor* const weight = a.tensor("weight", kRows, {n});
    const at::Tensor* const y = a.tensor("y", kRows, {rows, n});
    // uint8 holds the bytes of either format, a type that names one only its own
    const int named = format == BFLY_Q8_E4M3 ? kE4M3 : kI8;
    void* const codes = a.at("codes", kBytes | named, {rows, n});
    if (by_row || !codes) group = width;
    void* const scales = a.at("scales", kF16, {rows, group > 0 ? n / group : 0});
    const void* const residual = a.at("residual", same, {rows, n});
    void* const h = a.at("h", same, {rows, n});
    void* const rstd = a.at("rstd", kF32, {rows});
    a.on_the_gpu();
    return released([&] {
      return library.rmsnorm(x->data_ptr(), dtype_of(x), residual, h, address(weight),
                             dtype_of(weight), address(y), dtype_of(y),
                             static_cast<uint8_t*>(codes), static_cast<uint16_t*>(scales),
                             static_cast<float*>(rstd), rows, width, eps, (bfly_q8)format, group,
                             a.stream);
    });
  });
}

// rmsnorm_backward(stream, device, h, weight, rstd, dy, dx, dweight, dh, workspace)
PyObject* rmsnorm_backward(PyObject*, PyObject* const* args, Py_ssize_t count) {
  return guarded([&] {
    Args a(args, count, 10);
    const at::Tensor& like = a.sized("h", 2);
    const int64_t rows = like.size(0), n = like.size(1);
    const int32_t width = Args::narrow("a row", n);
    const at::Tensor* const h = a.tensor("h", kRows, {rows, n});
    const at::Tensor* const weight = a.tensor("weight", kRows, {n});
    const void* const rstd = a.at("rstd", kF32, {rows});
    const at::Tensor* const dy = a.tensor("dy", kRows, {rows, n});
    const int same = dy ? kind_of(dy->scalar_type()) : kRows;
    void* const dx = a.at("dx", same, {rows, n});
    void* const dweight = a.at("dweight", kF32, {n});
    const void* const dh = a.at("dh", same, {rows, n});
    size_t bytes;
    void* const workspace = a.scratch(bytes);
    a.on_the_gpu();
    return released([&] {
      return library.rmsnorm_backward(h->data_ptr(), dtype_of(h), address(weight),
                                      dtype_of(weight), static_cast<const float*>(rstd),
                                      address(dy), dh, dx, dtype_of(dy),
                                      static_cast<float*>(dweight), rows, width, workspace, bytes,
                                      a.stream);
    });
  });
}

// lora_matmul(stream, device, x, lora_a, y, ids, lora_b, scaling, base, workspace)
PyObject* lora_matmul(PyObject*, PyObject* const* args, Py_ssize_t count) {
  return guarded([&] {
    Args a(args, count, 10);
    const at::Tensor& like = a.sized("x", 2);
    const int64_t rows = like.size(0), k = like.size(1);
    const void* const x = a.at("x", kBF16, {rows, k});
    const at::Tensor& as = a.sized("lora_a", 3);
    const int64_t num = as.size(0), rank = as.size(1);
    const void* const lora_a = a.at("lora_a", kBF16, {num, rank, k});
    const int64_t n_out = a.sized("y", 2).size(1);
    const at::Tensor* const y = a.tensor("y", kRows, {rows, n_out});
    const void* const ids = a.at("ids", kI32, {rows});
    const void* const lora_b = a.at("lora_b", kBF16, {num, n_out, rank});
    const void* const scaling = a.at("scaling", kF32, {num});
    const at::Tensor* const base = a.tensor("base", kRows, {rows, n_out});
    size_t bytes;
    void* const workspace = a.scratch(bytes);
    const int32_t n32 = Args::narrow("a row of y", n_out), k32 = Args::narrow("a row of x", k),
                  num32 = Args::narrow("the adapters' number", num),
                  rank32 = Args::narrow("the rank", rank);
    a.on_the_gpu();
    return released([&] {
      return library.lora_matmul(x, BFLY_BF16, static_cast<const int32_t*>(ids), lora_a, lora_b,
                                 static_cast<const float*>(scaling), address(base),
                                 dtype_of(base), address(y), dtype_of(y), rows, n32, k32, num32,
                                 rank32, workspace, bytes, a.stream);
    });
  });
}

// The addresses, element counts and types of a list of contiguous tensors.
struct List {
  std::vector<uint64_t> at;
  std::vector<int64_t> numel;
  std::vector<int32_t> type;

  size_t size() const { return at.size(); }
  uint64_t bytes(size_t i) const { return (uint64_t)numel[i] * (type[i] ? 2 : 4); }

  void read(PyObject* given, Args& a) {
    PyObject* const items = PySequence_Fast(given, "a list or tuple of tensors is needed");
    if (!items) throw Raised();
    struct Release {
      PyObject* o;
      ~Release() { Py_DECREF(o); }
    } release{items};
    const Py_ssize_t n = PySequence_Fast_GET_SIZE(items);
    at.reserve(n), numel.reserve(n), type.reserve(n);
    for (Py_ssize_t i = 0; i < n; ++i) {
      PyObject* const item = PySequence_Fast_GET_ITEM(items, i);
      if (!THPVariable_Check(item)) fail(PyExc_TypeError, "item %zd is not a tensor", i);
      const at::Tensor& x = THPVariable_Unpack(item);
      const int kind = kind_of(x.scalar_type());
      if (!(kind & kRows))
        fail(PyExc_TypeError, "tensor %zd is neither float32 nor bfloat16", i);
      if (x.layout() != at::kStrided) fail(PyExc_ValueError, "tensor %zd is not strided", i);
      a.contiguous("every tensor", x);
      at.push_back(reinterpret_cast<uint64_t>(x.data_ptr()));
      numel.push_back(x.numel());
      type.push_back(kind == kBF16);
    }
  }
  // The addresses and indexes of those with elements, by address.
  std::vector<std::pair<uint64_t, size_t>> by_address() const {
    std::vector<std::pair<uint64_t, size_t>> v;
    v.reserve(size());
    for (size_t i = 0; i < size(); ++i)
      if (numel[i]) v.emplace_back(at[i], i);
    if (!std::is_sorted(v.begin(), v.end())) std::sort(v.begin(), v.end());
    return v;
  }
};

// Whether no two of the tensors to write share bytes, nor one of them and a
// gradient that is not, exactly, its own.
const char* overlap(const List& in, const List& out) {
  const auto outs = out.by_address();
  for (size_t i = 1; i < outs.size(); ++i)
    if (outs[i].first < outs[i - 1].first + out.bytes(outs[i - 1].second))
      return "two of the tensors to write overlap";
  if (&in == &out) return nullptr;
  for (size_t i = 0; i < in.size(); ++i) {
    if (!in.numel[i]) continue;
    // the first output that ends behind the gradient's start, and those after it
    auto o = std::upper_bound(outs.begin(), outs.end(), std::make_pair(in.at[i], in.size()));
    if (o != outs.begin() && (o - 1)->first + out.bytes((o - 1)->second) > in.at[i]) --o;
    for (; o != outs.end() && o->first < in.at[i] + in.bytes(i); ++o)
      if (o->second != i || o->first != in.at[i])
        return "an output overlaps a gradient that is not its own";
  }
  return nullptr;
}

// grad_clip(stream, device, max_norm, norm, workspace, grads, outs)
PyObject* grad_clip(PyObject*, PyObject* const* args, Py_ssize_t count) {
  return guarded([&] {
    Args a(args, count, 7);
    const float max_norm = a.real();
    void* const norm = a.at("norm", kF32, {2});
    size_t bytes;
    void* const workspace = a.scratch(bytes);
    List grads, outs;
    grads.read(a.object(), a);
    const bool in_place = a.none();
    if (!in_place) {
      outs.read(a.object(), a);
      if (outs.numel != grads.numel || outs.type != grads.type)
        fail(PyExc_ValueError, "the outputs have to be like their gradients");
    }
    const List& to = in_place ? grads : outs;
    if (const char* const problem = overlap(grads, to)) fail(PyExc_ValueError, "%s", problem);
    if (grads.size() > INT32_MAX) fail(PyExc_ValueError, "too many tensors");
    a.on_the_gpu();
    return released([&] {
      return library.grad_clip((int32_t)grads.size(),
                               reinterpret_cast<const void* const*>(grads.at.data()),
                               reinterpret_cast<void* const*>(to.at.data()), grads.numel.data(),
                               grads.type.data(), max_norm, static_cast<float*>(norm), workspace,
                               bytes, a.stream);
    });
  });
}

// overlaps(addresses, output addresses or None, element counts, types), as
// tuples of numbers -> the problem that grad_clip would have with them, or None.
PyObject* overlaps(PyObject*, PyObject* args) {
  PyObject *in, *out, *numel, *type;
  if (!PyArg_ParseTuple(args, "O!OO!O!", &PyTuple_Type, &in, &out, &PyTuple_Type, &numel,
                        &PyTuple_Type, &type))
    return nullptr;
  const auto read = [&](PyObject* from, List& l) {
    const Py_ssize_t n = PyTuple_GET_SIZE(numel);
    if (!PyTuple_Check(from) || PyTuple_GET_SIZE(from) != n || PyTuple_GET_SIZE(type) != n)
      fail(PyExc_ValueError, "tuples of one length are needed");
    for (Py_ssize_t i = 0; i < n; ++i) {
      l.at.push_back(PyLong_AsUnsignedLongLong(PyTuple_GET_ITEM(from, i)));
      l.numel.push_back(PyLong_AsLongLong(PyTuple_GET_ITEM(numel, i)));
      l.type.push_back((int32_t)PyLong_AsLong(PyTuple_GET_ITEM(type, i)));
    }
    if (PyErr_Occurred()) throw Raised();
  };
  try {
    List grads, outs;
    read(in, grads);
    if (out != Py_None) read(out, outs);
    const char* const problem = overlap(grads, out == Py_None ? grads : outs);
    return problem ? PyUnicode_FromString(problem) : (Py_INCREF(Py_None), Py_None);
  } catch (const Raised&) {
    return nullptr;
  } catch (const std::exception& e) {
    return PyErr_Format(PyExc_RuntimeError, "%s", e.what());
  }
}

// bind(rmsnorm, rmsnorm_backward, lora_matmul, grad_clip): the addresses of
// the library's functions.
PyObject* bind(PyObject*, PyObject* const* args, Py_ssize_t count) {
  void* at[4];
  if (count != 4) return PyErr_Format(PyExc_TypeError, "bind() takes four addresses");
  for (int i = 0; i < 4; ++i)
    if (!(at[i] = PyLong_AsVoidPtr(args[i])))
      return PyErr_Occurred() ? nullptr : PyErr_Format(PyExc_ValueError, "a null address");
  library.rmsnorm = reinterpret_cast<decltype(library.rmsnorm)>(at[0]);
  library.rmsnorm_backward = reinterpret_cast<decltype(library.rmsnorm_backward)>(at[1]);
  library.lora_matmul = reinterpret_cast<decltype(library.lora_matmul)>(at[2]);
  library.grad_clip = reinterpret_cast<decltype(library.grad_clip)>(at[3]);
  Py_RETURN_NONE;
}

PyCFunction fast(PyObject* (*f)(PyObject*, PyObject* const*, Py_ssize_t)) {
  return reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(f));
}
PyMethodDef methods[] = {
    {"bind", fast(bind), METH_FASTCALL, "the library's functions"},
    {"rmsnorm", fast(rmsnorm), METH_FASTCALL, "bfly_rmsnorm's status"},
    {"rmsnorm_backward", fast(rmsnorm_backward), METH_FASTCALL, "bfly_rmsnorm_backward's status"},
    {"lora_matmul", fast(lora_matmul), METH_FASTCALL, "bfly_lora_matmul's status"},
    {"grad_clip", fast(grad_clip), METH_FASTCALL, "bfly_grad_clip's status"},
    {"overlaps", overlaps, METH_VARARGS, "what grad_clip would refuse in a list"},
    {nullptr, nullptr, 0, nullptr}};
PyModuleDef module = {PyModuleDef_HEAD_INIT, "_tensors", nullptr, -1, methods,
                      nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__tensors() { return PyModule_Create(&module); }
