// Marshalling of the layer norm's and the linear layer's calls from Python:
// an entry takes the device's index, then the C entry's arguments in their
// order, tensors (or raw addresses, or None) in the place of pointers, and
// returns the status.  What an argument may be is read from the C entry's own
// parameter types.  A call of 24 arguments through ctypes, with the checks in
// Python, takes longer than the kernels of a single token.
#define PY_SSIZE_T_CLEAN
#include <Python.h>

#include <tuple>
#include <type_traits>
#include <utility>

#include "../../include/fp8q.h"

namespace {

// torch's dtypes (one object each for the process) that a pointer's type
// stands for, set by types().
PyObject *g_float = nullptr, *g_bfloat = nullptr, *g_codes = nullptr;
PyObject *s_dtype, *s_device, *s_pointer;

struct Call {
  long dev;               // of the operands; -1: none is a tensor yet
  long other = -2;        // a device that is not it
  bool host = false;      // an operand on no device
};

// The address an operand stands for.  `kind`: the dtypes it may have (null:
// any).  A wrong type raises at once, a wrong device once every type is right.
bool pointer(PyObject* o, PyObject* kind, const char* name, Call& c, void** out) {
  if (o == Py_None) {
    *out = nullptr;
    return true;
  }
  if (PyLong_Check(o)) {
    *out = PyLong_AsVoidPtr(o);
    return !PyErr_Occurred();
  }
  if (kind) {
    PyObject* t = PyObject_GetAttr(o, s_dtype);
    if (!t) return false;
    bool found = false;
    for (Py_ssize_t i = 0; i < PyTuple_GET_SIZE(kind); ++i) found = found || PyTuple_GET_ITEM(kind, i) == t;
    if (!found) PyErr_Format(PyExc_TypeError, "this operand is %s, got %S", name, t);
    Py_DECREF(t);
    if (!found) return false;
  }
  PyObject* d = PyObject_CallMethodNoArgs(o, s_device);
  if (!d) return false;
  const long dev = PyLong_AsLong(d);
  Py_DECREF(d);
  if (dev == -1 && PyErr_Occurred()) return false;
  if (dev < 0) c.host = true;
  else if (c.dev < 0) c.dev = dev;
  else if (dev != c.dev) c.other = dev;
  PyObject* p = PyObject_CallMethodNoArgs(o, s_pointer);
  if (!p) return false;
  *out = PyLong_AsVoidPtr(p);
  Py_DECREF(p);
  return !PyErr_Occurred();
}

template <typename T>
bool convert(PyObject* o, Call& c, T& v) {
  if constexpr (std::is_pointer_v<T>) {
    using E = std::remove_cv_t<std::remove_pointer_t<T>>;
    void* p;
    bool ok;
    if constexpr (std::is_same_v<E, float>) ok = pointer(o, g_float, "float32", c, &p);
    else if constexpr (std::is_same_v<E, uint16_t>) ok = pointer(o, g_bfloat, "bfloat16", c, &p);
    else if constexpr (std::is_same_v<E, uint8_t>) ok = pointer(o, g_codes, "FP8 codes", c, &p);
    else ok = pointer(o, nullptr, nullptr, c, &p);
    v = (T)p;
    return ok;
  } else if constexpr (std::is_floating_point_v<T>) {
    v = (T)PyFloat_AsDouble(o);
    return !PyErr_Occurred();
  } else {
    const long long x = PyLong_AsLongLong(o);
    v = (T)x;
    if (x == -1 && PyErr_Occurred()) return false;
    if (sizeof(T) == 4 && x != (long long)(int)x) {
      PyErr_SetString(PyExc_OverflowError, "this argument has 32 bits");
      return false;
    }
    return true;
  }
}

template <typename... P, size_t... I>
PyObject* invoke(int (*f)(P...), PyObject* const* a, Py_ssize_t n, std::index_sequence<I...>) {
  if (n != (Py_ssize_t)sizeof...(P) + 1)
    return PyErr_Format(PyExc_TypeError, "%zd arguments where there are %zd", n, (Py_ssize_t)sizeof...(P) + 1);
  Call c;
  c.dev = PyLong_AsLong(a[0]);
  if (c.dev == -1 && PyErr_Occurred()) return nullptr;
  std::tuple<P...> v;
  if (!(convert(a[I + 1], c, std::get<I>(v)) && ...)) return nullptr;
  if (c.host) return PyErr_Format(PyExc_ValueError, "this operand is not on a GPU");
  if (c.other >= 0)
    return PyErr_Format(PyExc_ValueError, "these operands share one device, got cuda:%ld and cuda:%ld", c.dev, c.other);
  int rc;
  // a full queue makes a launch wait
  Py_BEGIN_ALLOW_THREADS;
  rc = f(std::get<I>(v)...);
  Py_END_ALLOW_THREADS;
  return PyLong_FromLong(rc);
}

template <auto F>
struct Entry;
template <typename... P, int (*F)(P...)>
struct Entry<F> {
  static PyObject* call(PyObject*, PyObject* const* a, Py_ssize_t n) {
    return invoke(F, a, n, std::index_sequence_for<P...>{});
  }
};

PyObject* types(PyObject*, PyObject* args) {
  PyObject *f, *b, *c;
  if (!PyArg_ParseTuple(args, "O!O!O!", &PyTuple_Type, &f, &PyTuple_Type, &b, &PyTuple_Type, &c)) return nullptr;
  Py_XSETREF(g_float, Py_NewRef(f));
  Py_XSETREF(g_bfloat, Py_NewRef(b));
  Py_XSETREF(g_codes, Py_NewRef(c));
  Py_RETURN_NONE;
}

#define FP8Q_ENTRY(NAME_) {#NAME_, (PyCFunction)(void (*)(void))Entry<&NAME_>::call, METH_FASTCALL, nullptr}
PyMethodDef g_methods[] = {{"types", types, METH_VARARGS, nullptr},
                           FP8Q_ENTRY(fp8q_layernorm_1x128),
                           FP8Q_ENTRY(fp8q_layernorm_bwd),
                           FP8Q_ENTRY(fp8q_linear_blockscaled),
                           FP8Q_ENTRY(fp8q_linear_blockscaled_fast),
                           FP8Q_ENTRY(fp8q_linear_blockscaled_q),
                           FP8Q_ENTRY(fp8q_linear_blockscaled_q_fast),
                           FP8Q_ENTRY(fp8q_linear_bwd_q),
                           {nullptr, nullptr, 0, nullptr}};
PyModuleDef g_module = {PyModuleDef_HEAD_INIT, "_fp8q_call", nullptr, -1, g_methods, nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__fp8q_call(void) {
  s_dtype = PyUnicode_InternFromString("dtype");
  s_device = PyUnicode_InternFromString("get_device");
  s_pointer = PyUnicode_InternFromString("data_ptr");
  if (!s_dtype || !s_device || !s_pointer) return nullptr;
  return PyModule_Create(&g_module);
}
