// The operators' C entry points as Python calls: a torch tensor in the place of a forge_tensor or a pointer, None
// for NULL, whole numbers as they are. A small call is bound by the host's time; of about 8 us through ctypes, half
// went into the structures. Time of a call among others, through ctypes and here: a quantisation and an 8-bit product
// of one token 16.2 us and 11.5, the five calls of a small block of experts 37 and 25.5 (the launch itself is 3.2 to
// 3.9 of a call). What an entry point takes is read off its declaration. Checked here: types, dimensions, strides and devices
// of the tensors; all else in the entry points.
#define PY_SSIZE_T_CLEAN
#include <Python.h>
#include <ATen/ops/empty.h>
#include <dlfcn.h>
#include <torch/csrc/Dtype.h>
#include <torch/csrc/Exceptions.h>
#include <torch/csrc/autograd/python_variable.h>
#include <torch/version.h>

#include <stdexcept>
#include <string>
#include <tuple>
#include <type_traits>
#include <utility>

#include "forge.h"

namespace {

PyObject* g_error = nullptr;  // called with a status and the entry point's name: the exception to raise

struct PythonError {};  // already set

// The structures of a call's tensors, and the device of all of them.
struct Call {
  forge_tensor t[4 * FORGE_MAX_GROUP];
  int n = 0, device = -1;

  const at::Tensor& tensor(PyObject* o) {
    if (!THPVariable_Check(o)) throw std::invalid_argument("a tensor wanted");
    const at::Tensor& x = THPVariable_Unpack(o);
    const int d = x.is_cuda() ? x.get_device() : -2;
    if (device == -1) device = d;
    if (d != device || d < 0) throw std::invalid_argument("the tensors of a call live on one device");
    return x;
  }
};

int type_of(const at::Tensor& x) {
  switch (x.scalar_type()) {
    case at::kFloat: return FORGE_F32;
    case at::kBFloat16: return FORGE_BF16;
    case at::kChar: return FORGE_I8;
    default: throw std::invalid_argument(std::string("unsupported dtype ") + c10::toString(x.scalar_type()));
  }
}

// kind: 'm' rows of a matrix, 's' stacked matrices [experts, rows, cols], 'r' a vector as one row
forge_tensor* describe(Call& c, PyObject* o, char kind) {
  PyObject* factors = nullptr;
  if (PyTuple_Check(o) && PyTuple_GET_SIZE(o) == 2) {  // 8-bit rows and their factors
    factors = PyTuple_GET_ITEM(o, 1);
    o = PyTuple_GET_ITEM(o, 0);
  }
  const at::Tensor& x = c.tensor(o);
  if (c.n == static_cast<int>(sizeof(c.t) / sizeof(c.t[0]))) throw std::invalid_argument("too many tensors");
  forge_tensor& t = c.t[c.n++];
  const int64_t dim = x.dim();
  t = forge_tensor{nullptr, type_of(x), 0, 0, 0, 0, nullptr};
  if (kind == 'r') {
    if (dim != 1 || !x.is_contiguous()) throw std::invalid_argument("bias is a contiguous vector");
    t.rows = 1;
    t.cols = t.ld = x.size(0);
  } else if (kind == 's') {
    if (dim != 3) throw std::invalid_argument("stacked matrices [experts, out, in] wanted");
    const int64_t e = x.size(0), rows = x.size(1);
    t.rows = e * rows;
    t.cols = t.ld = x.size(2);
    if (x.numel() != 0) {
      if (x.stride(2) != 1 && t.cols > 1) throw std::invalid_argument("rows must be contiguous (stride(2) == 1)");
      if (rows > 1)
        t.ld = x.stride(1);
      else if (e > 1)
        t.ld = x.stride(0);
      if (e > 1 && x.stride(0) != rows * t.ld)
        throw std::invalid_argument("the rows of a stack follow one another in one pitch (stride(0) == out * stride(1))");
    }
  } else {
    if (dim != 2) throw std::invalid_argument("a matrix of two dimensions wanted");
    t.rows = x.size(0);
    t.cols = t.ld = x.size(1);
    if (x.numel() != 0) {
      if (x.stride(1) != 1 && t.cols > 1) throw std::invalid_argument("rows must be contiguous (stride(1) == 1)");
      if (t.rows > 1) t.ld = x.stride(0);
    }
  }
  if (x.numel() != 0) t.data = x.data_ptr();
  if (factors) {
    if (t.dtype != FORGE_I8) throw std::invalid_argument("int8 codes wanted beside factors");
    const at::Tensor& s = c.tensor(factors);
    if (s.scalar_type() != at::kFloat || s.numel() != t.rows || !s.is_contiguous())
      throw std::invalid_argument("factors of 8-bit rows: " + std::to_string(t.rows) + " contiguous float32 values wanted");
    if (t.rows) t.scale = static_cast<float*>(s.data_ptr());
  }
  return &t;
}

template <class T>
T take(Call& c, PyObject* o, char kind) {
  if constexpr (std::is_same_v<T, forge_tensor*> || std::is_same_v<T, const forge_tensor*>) {
    if (o == Py_None) return nullptr;
    if (!PyList_Check(o)) return describe(c, o, kind);
    forge_tensor* first = c.t + c.n;  // a group's, one after another
    for (Py_ssize_t i = 0; i < PyList_GET_SIZE(o); ++i) describe(c, PyList_GET_ITEM(o, i), kind);
    return first;
  } else if constexpr (std::is_pointer_v<T>) {
    if (o == Py_None) return nullptr;
    if (PyLong_Check(o)) {  // a stream
      void* p = PyLong_AsVoidPtr(o);
      if (!p && PyErr_Occurred()) throw PythonError{};
      return static_cast<T>(p);
    }
    const at::Tensor& x = c.tensor(o);
    return x.numel() == 0 ? nullptr : static_cast<T>(x.data_ptr());
  } else {
    static_assert(std::is_integral_v<T>, "an argument of another type");
    const long long v = PyLong_AsLongLong(o);
    if (v == -1 && PyErr_Occurred()) throw PythonError{};
    if (static_cast<long long>(static_cast<T>(v)) != v) throw std::invalid_argument("a whole number out of range");
    return static_cast<T>(v);
  }
}

template <class R, class... A, std::size_t... I>
PyObject* call(R (*fn)(A...), const char* name, const char* kinds, PyObject* const* args, Py_ssize_t n,
               std::index_sequence<I...>) {
  if (!fn) {
    PyErr_SetString(PyExc_RuntimeError, "the library is not loaded");
    return nullptr;
  }
  if (n != static_cast<Py_ssize_t>(sizeof...(A))) {
    PyErr_Format(PyExc_TypeError, "%s takes %zu arguments, not %zd", name, sizeof...(A), n);
    return nullptr;
  }
  try {
    Call c;
    const std::tuple<A...> a{take<A>(c, args[I], kinds[I])...};  // (in order)
    R r;
    Py_BEGIN_ALLOW_THREADS
    r = std::apply(fn, a);
    Py_END_ALLOW_THREADS
    if constexpr (sizeof(R) == 8) return PyLong_FromLongLong(r);
    if (r == FORGE_OK) Py_RETURN_NONE;
    PyObject* e = PyObject_CallFunction(g_error, "is", static_cast<int>(r), name);
    if (e) {
      PyErr_SetObject(reinterpret_cast<PyObject*>(Py_TYPE(e)), e);
      Py_DECREF(e);
    }
  } catch (const PythonError&) {
  } catch (const std::invalid_argument& e) {
    PyErr_Format(PyExc_ValueError, "%s: %s", name, e.what());
  } catch (const std::exception& e) {
    PyErr_Format(PyExc_RuntimeError, "%s: %s", name, e.what());
  }
  return nullptr;
}

// entry points, and what each of their arguments is (describe's kinds; . for all else)
#define FORGE_CALLS(X)                               \
  X(forge_expert_plan_workspace, "...")              \
  X(forge_expert_plan, ".........")                  \
  X(forge_expert_dispatch, "m..m.")                  \
  X(forge_expert_combine, "m...mm.")                 \
  X(forge_expert_combine_backward, "mm...m..")       \
  X(forge_expert_linear, "ms...mm.")                 \
  X(forge_expert_gated, "mss...mmm.")                \
  X(forge_expert_gated_dgrad, "msmm...mmm.")         \
  X(forge_expert_dgrad_group_workspace, ".....")     \
  X(forge_expert_dgrad_group_split, ".ms..m...")     \
  X(forge_expert_wgrad, "mm.....")                   \
  X(forge_quantize_rows, "mm.")                      \
  X(forge_linear_q8, "mmr.mm.")                      \
  X(forge_gated_q8, "mmm.m.")                        \
  X(forge_expert_linear_q8, "ms...m.")               \
  X(forge_expert_gated_q8, "mss...m.")

template <class R, class... A>
constexpr std::size_t arity(R (*)(A...)) {
  return sizeof...(A);
}

#define FORGE_DEFINE(NAME, KINDS)                                                                        \
  decltype(&NAME) p_##NAME = nullptr;                                                                    \
  PyObject* py_##NAME(PyObject*, PyObject* const* args, Py_ssize_t n) {                                  \
    constexpr std::size_t N = arity(static_cast<decltype(&NAME)>(nullptr));                              \
    static_assert(sizeof(KINDS) - 1 == N, "a kind for each argument");                                   \
    return call(p_##NAME, #NAME, KINDS, args, n, std::make_index_sequence<N>{});                         \
  }
FORGE_CALLS(FORGE_DEFINE)
#undef FORGE_DEFINE

// load(path, error): the library that the calls go to
PyObject* load(PyObject*, PyObject* args) {
  const char* path;
  PyObject* error;
  if (!PyArg_ParseTuple(args, "sO", &path, &error)) return nullptr;
  void* lib = dlopen(path, RTLD_NOW | RTLD_LOCAL);
  if (!lib) {
    PyErr_SetString(PyExc_ImportError, dlerror());
    return nullptr;
  }
#define FORGE_FIND(NAME, KINDS)                                                   \
  p_##NAME = reinterpret_cast<decltype(&NAME)>(dlsym(lib, #NAME));                \
  if (!p_##NAME) {                                                                \
    PyErr_SetString(PyExc_ImportError, "the library lacks " #NAME);               \
    return nullptr;                                                               \
  }
  FORGE_CALLS(FORGE_FIND)
#undef FORGE_FIND
  Py_XDECREF(g_error);
  Py_INCREF(error);
  g_error = error;
  Py_RETURN_NONE;
}

// empty(device index, dtype, *sizes): torch.empty on that device, without the time that parsing its arguments takes (of
// 1.25 us for a matrix); what torch.empty honours, deterministic fill and dispatch modes, at::empty does
PyObject* empty(PyObject*, PyObject* const* args, Py_ssize_t n) {
  HANDLE_TH_ERRORS
  if (n < 2 || !THPDtype_Check(args[1])) throw std::invalid_argument("empty(device index, dtype, *sizes) wanted");
  int64_t v[FORGE_MAX_GROUP + 1];
  const Py_ssize_t dims = n - 2;
  if (dims > FORGE_MAX_GROUP) throw std::invalid_argument("too many dimensions");
  for (Py_ssize_t i = 0; i <= dims; ++i) {  // (the device's index, then the sizes)
    v[i] = PyLong_AsLongLong(args[i ? i + 1 : 0]);
    if (v[i] == -1 && PyErr_Occurred()) return nullptr;
  }
  const auto options = at::TensorOptions()
                           .dtype(reinterpret_cast<THPDtype*>(args[1])->scalar_type)
                           .device(c10::Device(c10::kCUDA, static_cast<c10::DeviceIndex>(v[0])));
  struct Released {
    PyThreadState* state = PyEval_SaveThread();
    ~Released() { PyEval_RestoreThread(state); }
  };
  at::Tensor t;
  {
    Released gil;
    t = at::empty(at::IntArrayRef(v + 1, dims), options);
  }
  return THPVariable_Wrap(std::move(t));
  END_HANDLE_TH_ERRORS
}

PyMethodDef methods[] = {
    {"load", load, METH_VARARGS, nullptr},
    {"empty", reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(empty)), METH_FASTCALL, nullptr},
#define FORGE_METHOD(NAME, KINDS) \
  {#NAME, reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(py_##NAME)), METH_FASTCALL, nullptr},
    FORGE_CALLS(FORGE_METHOD)
#undef FORGE_METHOD
    {nullptr, nullptr, 0, nullptr}};

PyModuleDef module = {PyModuleDef_HEAD_INIT, "forge_calls", nullptr, -1, methods, nullptr, nullptr, nullptr, nullptr};

}  // namespace

// torch_version: the torch that this was compiled against, whose classes the code above has inlined
PyMODINIT_FUNC PyInit_forge_calls() {
  PyObject* m = PyModule_Create(&module);
  if (m && PyModule_AddStringConstant(m, "torch_version", TORCH_VERSION) < 0) Py_CLEAR(m);
  return m;
}
