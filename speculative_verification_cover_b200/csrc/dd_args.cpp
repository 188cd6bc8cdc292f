// Host side of the cached-decoding calls of the Python binding (dd.py): a tensor's type,
// shape, layout and device, and its address, in one call; and the library's entry points,
// with the signatures of dd.h. A decode step makes many small calls of eight tensors or so
// each: the same checks in Python take about 0.9 us a tensor, and ctypes 0.3 us an argument,
// together more than the kernels of the smallest steps.
#include <Python.h>

#include <torch/csrc/Dtype.h>
#include <torch/csrc/autograd/python_variable.h>

#include <climits>
#include <exception>
#include <tuple>
#include <type_traits>
#include <utility>
#include <vector>

#include "../../include/dd.h"

namespace {

// refuse(t, name, dtype, shape, gpu, rows) raises the error that says what is wrong.
PyObject* g_refuse = nullptr;

// Whether the tensor is as asked: shape and type on device `gpu`, contiguous or, with `rows`,
// contiguous in all dimensions but the first.
bool fits(const at::Tensor& t, at::ScalarType type, PyObject* shape, long gpu, bool rows) {
  const auto sizes = t.sizes();
  if (t.scalar_type() != type || (Py_ssize_t)sizes.size() != PyTuple_GET_SIZE(shape)) return false;
  if ((t.is_cpu() ? -1 : (long)t.get_device()) != gpu) return false;
  for (size_t i = 0; i < sizes.size(); ++i)
    if (PyLong_AsLongLong(PyTuple_GET_ITEM(shape, (Py_ssize_t)i)) != sizes[i]) return false;
  if (t.is_contiguous()) return true;
  if (!rows || sizes.empty() || sizes[0] < 2) return false;
  int64_t inner = 1;
  for (size_t i = sizes.size() - 1; i > 0; --i) {
    if (sizes[i] != 1 && t.stride((int64_t)i) != inner) return false;
    inner *= sizes[i];
  }
  return true;
}

// (t, name, dtype, shape, gpu): the address, or None to the caller's error.
PyObject* check(PyObject* const* args, Py_ssize_t n, bool rows) {
  if (n != 5 || !THPDtype_Check(args[2]) || !PyTuple_Check(args[3])) {
    PyErr_SetString(PyExc_TypeError, "expected (tensor, name, dtype, shape, gpu)");
    return nullptr;
  }
  const long gpu = PyLong_AsLong(args[4]);
  if (gpu == -1 && PyErr_Occurred()) return nullptr;
  try {
    if (THPVariable_Check(args[0])) {
      const at::Tensor& t = THPVariable_Unpack(args[0]);
      const bool ok = fits(t, reinterpret_cast<THPDtype*>(args[2])->scalar_type, args[3], gpu, rows);
      if (PyErr_Occurred()) return nullptr;  // a size that is no whole number
      if (ok) {
        const auto at = (unsigned long long)reinterpret_cast<uintptr_t>(t.data_ptr());
        return rows ? Py_BuildValue("KL", at, (long long)(t.dim() ? t.stride(0) : 0)) : PyLong_FromUnsignedLongLong(at);
      }
    }
  } catch (const std::exception& e) {
    PyErr_SetString(PyExc_RuntimeError, e.what());
    return nullptr;
  }
  if (!g_refuse) {
    PyErr_SetString(PyExc_RuntimeError, "no refusal is set");
    return nullptr;
  }
  return PyObject_CallFunctionObjArgs(g_refuse, args[0], args[1], args[2], args[3], args[4],
                                      rows ? Py_True : Py_False, nullptr);
}

PyObject* arg(PyObject*, PyObject* const* args, Py_ssize_t n) { return check(args, n, false); }
PyObject* rows(PyObject*, PyObject* const* args, Py_ssize_t n) { return check(args, n, true); }

PyObject* set_refuse(PyObject*, PyObject* f) {
  Py_INCREF(f);
  Py_XSETREF(g_refuse, f);
  Py_RETURN_NONE;
}

// (t, gpu): address and bytes of a caller's workspace, or None if it is no contiguous tensor there.
PyObject* workspace(PyObject*, PyObject* const* args, Py_ssize_t n) {
  if (n != 2) {
    PyErr_SetString(PyExc_TypeError, "expected (tensor, gpu)");
    return nullptr;
  }
  const long gpu = PyLong_AsLong(args[1]);
  if (gpu == -1 && PyErr_Occurred()) return nullptr;
  try {
    if (THPVariable_Check(args[0])) {
      const at::Tensor& t = THPVariable_Unpack(args[0]);
      if ((t.is_cpu() ? -1 : (long)t.get_device()) == gpu && t.is_contiguous())
        return Py_BuildValue("KK", (unsigned long long)reinterpret_cast<uintptr_t>(t.data_ptr()),
                             (unsigned long long)t.nbytes());
    }
  } catch (const std::exception& e) {
    PyErr_SetString(PyExc_RuntimeError, e.what());
    return nullptr;
  }
  Py_RETURN_NONE;
}

// ------------------------------------------------------------------ entry points
// A Python argument as the type of a parameter; false with a Python error.
template <typename T>
bool convert(PyObject* o, T& x) {
  if constexpr (std::is_pointer_v<T>) {
    x = o == Py_None ? nullptr : static_cast<T>(PyLong_AsVoidPtr(o));
  } else if constexpr (std::is_floating_point_v<T>) {
    x = (T)PyFloat_AsDouble(o);
  } else if constexpr (std::is_same_v<T, size_t>) {
    x = PyLong_AsSize_t(o);
  } else {  // int, int64_t or an enum
    const long long v = PyLong_AsLongLong(o);
    if (sizeof(T) == sizeof(int) && (v < INT_MIN || v > INT_MAX)) {
      PyErr_SetString(PyExc_OverflowError, "a size is beyond 32 bits");
      return false;
    }
    x = (T)v;
  }
  return !PyErr_Occurred();
}

template <typename... A, size_t... I>
PyObject* invoke(dd_status (*fn)(A...), PyObject* const* args, Py_ssize_t n, std::index_sequence<I...>) {
  if (!fn || n != (Py_ssize_t)sizeof...(A)) {
    PyErr_SetString(PyExc_TypeError, fn ? "wrong number of arguments" : "the library is not bound");
    return nullptr;
  }
  std::tuple<A...> v;
  if (!(convert(args[I], std::get<I>(v)) && ...)) return nullptr;
  dd_status st;
  Py_BEGIN_ALLOW_THREADS
  st = fn(std::get<I>(v)...);
  Py_END_ALLOW_THREADS
  return PyLong_FromLong(st);
}

// One entry point: its address in the library that dd.py loaded, and the call.
template <auto* kSignature>
struct Entry;
template <typename... A, dd_status (*kSignature)(A...)>
struct Entry<kSignature> {
  static inline dd_status (*fn)(A...) = nullptr;
  static PyObject* call(PyObject*, PyObject* const* args, Py_ssize_t n) {
    return invoke(fn, args, n, std::index_sequence_for<A...>{});
  }
  static PyObject* bind(PyObject*, PyObject* address) {
    fn = reinterpret_cast<dd_status (*)(A...)>(PyLong_AsVoidPtr(address));
    if (PyErr_Occurred()) return nullptr;
    Py_RETURN_NONE;
  }
};

// (parent, B, K, [src, dst, bytes a row, ...], stream): dd_beam_reorder of packed rows.
PyObject* reorder(PyObject*, PyObject* const* args, Py_ssize_t n) {
  const auto fn = Entry<&dd_beam_reorder>::fn;
  const int32_t* parent;
  int B, K;
  void* stream;
  if (!fn || n != 5 || !PyList_Check(args[3])) {
    PyErr_SetString(PyExc_TypeError, fn ? "expected (parent, B, K, list, stream)" : "the library is not bound");
    return nullptr;
  }
  if (!convert(args[0], parent) || !convert(args[1], B) || !convert(args[2], K) || !convert(args[4], stream))
    return nullptr;
  std::vector<dd_row_state> states((size_t)PyList_GET_SIZE(args[3]) / 3);
  for (size_t i = 0; i < states.size(); ++i) {
    dd_row_state& s = states[i];
    const auto item = [&](size_t e) { return PyList_GET_ITEM(args[3], (Py_ssize_t)(3 * i + e)); };
    if (!convert(item(0), s.src) || !convert(item(1), s.dst) || !convert(item(2), s.row_bytes)) return nullptr;
    s.src_stride = s.dst_stride = s.row_bytes;
  }
  dd_status st;
  Py_BEGIN_ALLOW_THREADS
  st = fn(parent, B, K, states.data(), (int)states.size(), stream);
  Py_END_ALLOW_THREADS
  return PyLong_FromLong(st);
}

PyCFunction fast(PyObject* (*f)(PyObject*, PyObject* const*, Py_ssize_t)) {
  return reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(f));
}

#define DD_ENTRY(name)                                      \
  {#name, fast(Entry<&name>::call), METH_FASTCALL, nullptr}, \
  {"bind_" #name, Entry<&name>::bind, METH_O, nullptr}

PyMethodDef g_methods[] = {
    {"arg", fast(arg), METH_FASTCALL, "Address of a contiguous tensor of the given type, shape and device."},
    {"rows", fast(rows), METH_FASTCALL, "Address and row stride of a tensor whose rows are contiguous."},
    {"workspace", fast(workspace), METH_FASTCALL, "Address and bytes of a workspace."},
    {"set_refuse", set_refuse, METH_O, "The function that raises what is wrong with a tensor."},
    DD_ENTRY(dd_paged_attention),
    DD_ENTRY(dd_cache_evict),
    DD_ENTRY(dd_beam_select),
    {"dd_beam_reorder", fast(reorder), METH_FASTCALL, nullptr},
    {"bind_dd_beam_reorder", Entry<&dd_beam_reorder>::bind, METH_O, nullptr},
    DD_ENTRY(dd_paged_fork),
    {nullptr, nullptr, 0, nullptr}};
PyModuleDef g_module = {PyModuleDef_HEAD_INIT, "_args", nullptr, -1, g_methods, nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__args() { return PyModule_Create(&g_module); }
