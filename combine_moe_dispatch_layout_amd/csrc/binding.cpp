// binding.cpp -- the binding's hot path as a CPython extension: the facts about a
// tensor that a call checks, asked for at once, new outputs, and the library's
// entry points called without ctypes.  (A decode-sized call is bound by host
// time: a norm of one token took 8.1 us through Python and ctypes alone, 6.6 with
// the facts asked through the tensors' Python methods, 5.5 so.)
#define PY_SSIZE_T_CLEAN
#include <torch/csrc/Dtype.h>
#include <torch/csrc/Exceptions.h>
#include <torch/csrc/autograd/python_variable.h>

#include <ATen/ops/empty.h>

#include <climits>
#include <cstdint>
#include <cstring>
#include <tuple>
#include <type_traits>
#include <utility>

#include "moe_dispatch.h"

namespace {

// None, with no error left: the caller then says what is wrong.
PyObject* not_so() {
  PyErr_Clear();
  Py_RETURN_NONE;
}

// The tensor of `t` if it is a strided one of `dtype`, else null.
const at::Tensor* tensor_of(PyObject* t, PyObject* dtype) {
  if (!THPVariable_Check(t) || !THPDtype_Check(dtype)) return nullptr;
  const at::Tensor& v = THPVariable_Unpack(t);
  if (v.layout() != at::kStrided ||
      v.scalar_type() != reinterpret_cast<THPDtype*>(dtype)->scalar_type)
    return nullptr;
  return &v;
}

// A tuple of numbers.
template <typename... N>
PyObject* numbers(N... n) {
  PyObject* t = PyTuple_New(sizeof...(n));
  if (t == nullptr) return nullptr;
  Py_ssize_t at = 0;
  for (const long long v : {static_cast<long long>(n)...}) {
    PyObject* o = PyLong_FromLongLong(v);
    if (o == nullptr) {
      Py_DECREF(t);
      return nullptr;
    }
    PyTuple_SET_ITEM(t, at++, o);
  }
  return t;
}

long long address(const at::Tensor& t) { return (long long)(intptr_t)t.data_ptr(); }

// matrix(t, dtype) -> (device, rows, columns, row stride, address) of a 2-D
// tensor with unit column stride, or None.
PyObject* calls_matrix(PyObject*, PyObject* const* a, Py_ssize_t n) try {
  const at::Tensor* t = n == 2 ? tensor_of(a[0], a[1]) : nullptr;
  if (t == nullptr || t->dim() != 2 || t->stride(1) != 1) return not_so();
  return numbers(t->get_device(), t->size(0), t->size(1), t->stride(0), address(*t));
} catch (...) {
  return not_so();
}

// rows(t, dtype, rows, columns, device) -> (row stride, address), or None.
PyObject* calls_rows(PyObject*, PyObject* const* a, Py_ssize_t n) try {
  const at::Tensor* t = n == 5 ? tensor_of(a[0], a[1]) : nullptr;
  if (t == nullptr || t->dim() != 2 || t->stride(1) != 1 ||
      t->size(0) != PyLong_AsLongLong(a[2]) || t->size(1) != PyLong_AsLongLong(a[3]) ||
      t->get_device() != PyLong_AsLongLong(a[4]) || PyErr_Occurred())
    return not_so();
  return numbers(t->stride(0), address(*t));
} catch (...) {
  return not_so();
}

// flat(t, dtype, device, size0[, size1]) -> address of a contiguous tensor of
// that shape, or None.
PyObject* calls_flat(PyObject*, PyObject* const* a, Py_ssize_t n) try {
  const at::Tensor* t = n == 4 || n == 5 ? tensor_of(a[0], a[1]) : nullptr;
  if (t == nullptr || t->dim() != n - 3 || t->get_device() != PyLong_AsLongLong(a[2]) ||
      !t->is_contiguous())
    return not_so();
  for (Py_ssize_t i = 0; i < n - 3; ++i)
    if (t->size(i) != PyLong_AsLongLong(a[3 + i])) return not_so();
  if (PyErr_Occurred()) return not_so();
  return PyLong_FromLongLong(address(*t));
} catch (...) {
  return not_so();
}

// Other threads may run Python meanwhile.
struct Unlocked {
  PyThreadState* state = PyEval_SaveThread();
  ~Unlocked() { PyEval_RestoreThread(state); }
};

at::Tensor new_tensor(const at::Tensor& like, at::ScalarType type, at::IntArrayRef sizes) {
  const Unlocked unlocked;  // the allocator may wait for the GPU
  return at::empty(sizes, like.options().dtype(type));
}

// new(like, dtype, size0[, size1]) -> (a new contiguous tensor beside `like`, its
// address).
PyObject* calls_new(PyObject*, PyObject* const* a, Py_ssize_t n) {
  HANDLE_TH_ERRORS
  if (n < 3 || n > 4 || !THPVariable_Check(a[0]) || !THPDtype_Check(a[1]))
    return PyErr_Format(PyExc_TypeError, "new takes a tensor, a dtype and one or two sizes");
  int64_t sizes[2];
  for (Py_ssize_t i = 0; i < n - 2; ++i) sizes[i] = PyLong_AsLongLong(a[2 + i]);
  if (PyErr_Occurred()) return nullptr;
  at::Tensor t = new_tensor(THPVariable_Unpack(a[0]),
                            reinterpret_cast<THPDtype*>(a[1])->scalar_type,
                            at::IntArrayRef(sizes, n - 2));
  const long long at = address(t);
  PyObject* pair = PyTuple_New(2);
  if (pair == nullptr) return nullptr;
  PyTuple_SET_ITEM(pair, 0, THPVariable_Wrap(std::move(t)));
  PyTuple_SET_ITEM(pair, 1, PyLong_FromLongLong(at));
  if (PyTuple_GET_ITEM(pair, 0) == nullptr || PyTuple_GET_ITEM(pair, 1) == nullptr) {
    Py_DECREF(pair);
    return nullptr;
  }
  return pair;
  END_HANDLE_TH_ERRORS
}

// ---- the entry points ------------------------------------------------------------
// An argument as the library takes it; a wrong one leaves an error.
template <typename T>
T taken(PyObject* v) {
  if constexpr (std::is_pointer_v<T>) {
    return v == Py_None ? nullptr : static_cast<T>(PyLong_AsVoidPtr(v));
  } else if constexpr (std::is_same_v<T, float>) {
    return (float)PyFloat_AsDouble(v);
  } else if constexpr (std::is_same_v<T, size_t>) {
    return PyLong_AsSize_t(v);
  } else {
    static_assert(std::is_same_v<T, int32_t> || std::is_same_v<T, int64_t>);
    const long long n = PyLong_AsLongLong(v);
    if (sizeof(T) == 4 && (n > INT32_MAX || n < INT32_MIN))
      PyErr_SetString(PyExc_OverflowError, "a size that does not fit 32 bits");
    return (T)n;
  }
}

struct Entry {
  const char* name;
  void* at;
};
Entry entries[] = {{"moe_rms_norm", nullptr},      {"moe_rms_norm_backward", nullptr},
                   {"moe_router_logits", nullptr}, {"moe_router_logits_backward", nullptr},
                   {"moe_route", nullptr},         {"moe_route_backward", nullptr}};

// Calls entry WHICH, whose arguments the header declares as A.
template <int WHICH, typename... A, size_t... I>
PyObject* invoke(PyObject* const* a, Py_ssize_t n, std::index_sequence<I...>) {
  const Entry& e = entries[WHICH];
  if (n != (Py_ssize_t)sizeof...(A))
    return PyErr_Format(PyExc_TypeError, "%s takes %zd arguments, got %zd", e.name,
                        (Py_ssize_t)sizeof...(A), n);
  if (e.at == nullptr) return PyErr_Format(PyExc_RuntimeError, "%s is not bound", e.name);
  const std::tuple<A...> args{(PyErr_Occurred() ? A() : taken<A>(a[I]))...};
  if (PyErr_Occurred()) return nullptr;
  int rc;
  {
    const Unlocked unlocked;
    rc = std::apply(reinterpret_cast<int (*)(A...)>(e.at), args);
  }
  return PyLong_FromLong(rc);
}

// bind(name, address): where an entry point of the loaded library is.
PyObject* calls_bind(PyObject*, PyObject* args) {
  const char* name;
  PyObject* at;
  if (!PyArg_ParseTuple(args, "sO", &name, &at)) return nullptr;
  void* p = PyLong_AsVoidPtr(at);
  if (PyErr_Occurred()) return nullptr;
  for (Entry& e : entries)
    if (std::strcmp(e.name, name) == 0) {
      e.at = p;
      Py_RETURN_NONE;
    }
  return PyErr_Format(PyExc_ValueError, "no entry point %s", name);
}

using Call = PyObject* (*)(PyObject*, PyObject* const*, Py_ssize_t);
PyMethodDef method(const char* name, Call call) {
  return {name, reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(call)), METH_FASTCALL,
          nullptr};
}

// (The functions are named for their types alone: the library is found at run
// time, by load_library().)
template <int WHICH, typename F>
struct Of;
template <int WHICH, typename... A>
struct Of<WHICH, int (*)(A...)> {
  static PyObject* call(PyObject*, PyObject* const* a, Py_ssize_t n) {
    return invoke<WHICH, A...>(a, n, std::index_sequence_for<A...>{});
  }
};
#define MOE_ENTRY(which, name) method(#name, Of<which, decltype(&name)>::call)

PyMethodDef methods[] = {method("matrix", calls_matrix),
                         method("rows", calls_rows),
                         method("flat", calls_flat),
                         method("new", calls_new),
                         MOE_ENTRY(0, moe_rms_norm),
                         MOE_ENTRY(1, moe_rms_norm_backward),
                         MOE_ENTRY(2, moe_router_logits),
                         MOE_ENTRY(3, moe_router_logits_backward),
                         MOE_ENTRY(4, moe_route),
                         MOE_ENTRY(5, moe_route_backward),
                         {"bind", calls_bind, METH_VARARGS, nullptr},
                         {nullptr, nullptr, 0, nullptr}};

PyModuleDef module = {PyModuleDef_HEAD_INIT, "_binding", nullptr, -1, methods};

}  // namespace

PyMODINIT_FUNC PyInit__binding() { return PyModule_Create(&module); }
