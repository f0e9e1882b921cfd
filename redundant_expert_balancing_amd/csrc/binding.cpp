// Marshalling of the 8-bit integer experts' calls for Python: the checks of _lib.py's _q on every
// tensor, the current stream's handle, and the call. These calls serve single tokens, where
// the host's time counts: a call takes 3.1 us (3.7-3.9 on a slower host), nearly all of it the
// launch, against 5.2 (three tensors) to 6.2 us (six) with the checks in Python; one token through
// a dense product 12.2 -> 8.2 us with the rounding of its row.
//
// bind(addresses, current_device, current_stream) hands over the loaded library's functions and
// torch's two queries; each function below takes what the call of _lib.py of its name takes,
// raises ValueError for a tensor that must not reach a kernel, and returns the call's status.
#define PY_SSIZE_T_CLEAN
#include <Python.h>

#include <torch/csrc/autograd/python_variable.h>

#include "moonep.h"

namespace {

typedef __int128 wide;      // sizes formed from a shape's fields cannot overflow

struct Functions {
  decltype(&moonep_int_quantize) quantize;
  decltype(&moonep_int_quantize_weight) quantize_weight;
  decltype(&moonep_int_transpose_weight) transpose_weight;
  decltype(&moonep_int_prefetch_weight) prefetch_weight;
  decltype(&moonep_int_grouped_gemm) grouped_gemm;
  decltype(&moonep_int_grouped_gemm_swiglu) grouped_gemm_swiglu;
  decltype(&moonep_int_gemm) gemm;
  decltype(&moonep_int_gemm_swiglu) gemm_swiglu;
  decltype(&moonep_int_quantize_grad) quantize_grad;
} f;
PyObject *g_device = nullptr, *g_stream = nullptr;

// A call's arguments. The first one refused sets the Python error and ok to false; everything
// after that does nothing.
struct Call {
  PyObject* const* args;
  bool ok = true;
  int device = -1;          // of the tensors so far
  moonep_shape sh{};

  Call(PyObject* const* a, Py_ssize_t n, Py_ssize_t want) : args(a) {
    if (n != want) {
      PyErr_Format(PyExc_TypeError, "%zd arguments, expected %zd", n, want);
      ok = false;
      return;
    }
    Py_buffer view;
    if (PyObject_GetBuffer(a[0], &view, PyBUF_SIMPLE)) {
      ok = false;
      return;
    }
    if (view.len == Py_ssize_t(sizeof sh)) memcpy(&sh, view.buf, sizeof sh);
    else fail(PyExc_TypeError, "a moonep_shape is required");
    PyBuffer_Release(&view);
  }

  void fail(PyObject* type, const char* text) {
    PyErr_SetString(type, text);
    ok = false;
  }

  // A whole number: anything with __index__ (numpy's among them), no float and no text.
  int64_t integer(int i, const char* name) {
    if (!ok) return 0;
    if (PyUnicode_Check(args[i]) || PyBytes_Check(args[i])) {
      PyErr_Format(PyExc_ValueError, "%s: a whole number is required, got text", name);
      ok = false;
      return 0;
    }
    PyObject* v = PyNumber_Index(args[i]);
    const int64_t r = v ? PyLong_AsLongLong(v) : -1;
    Py_XDECREF(v);
    if (PyErr_Occurred()) ok = false;
    return r;
  }

  // Address of argument i: a contiguous GPU tensor of `type` with at least `need` bytes, on
  // the device of the others; None gives NULL where it may.
  void* tensor(int i, const char* name, wide need, at::ScalarType type, bool optional = false) {
    if (!ok) return nullptr;
    PyObject* o = args[i];
    if (o == Py_None && optional) return nullptr;
    if (!THPVariable_Check(o)) {
      PyErr_Format(PyExc_ValueError, "%s: a tensor is required", name);
      ok = false;
      return nullptr;
    }
    const at::Tensor& t = THPVariable_Unpack(o);
    if (!t.is_cuda()) {
      PyErr_Format(PyExc_ValueError, "%s: a GPU tensor is required, got one on %s", name,
                   t.device().str().c_str());
    } else if (!t.is_contiguous()) {
      PyErr_Format(PyExc_ValueError, "%s: the tensor must be contiguous", name);
    } else if (type != at::ScalarType::Undefined && t.scalar_type() != type) {
      PyErr_Format(PyExc_ValueError, "%s: dtype %s, expected %s", name, at::toString(t.scalar_type()),
                   at::toString(type));
    } else if (wide(t.nbytes()) < need) {
      PyErr_Format(PyExc_ValueError, "%s: %zu bytes, the call needs more", name, size_t(t.nbytes()));
    } else if (device >= 0 && t.get_device() != device) {
      PyErr_Format(PyExc_ValueError, "%s: on %s, the other tensors on cuda:%d", name,
                   t.device().str().c_str(), device);
    } else {
      device = int(t.get_device());
      return t.data_ptr();
    }
    ok = false;
    return nullptr;
  }

  // hipStream_t of argument i (None: torch's current one); the tensors have to be on the current
  // device, whose stream it is.
  void* stream(int i) {
    if (!ok) return nullptr;
    PyObject* d = PyObject_CallNoArgs(g_device);
    const long now = d ? PyLong_AsLong(d) : -1;
    Py_XDECREF(d);
    if (PyErr_Occurred()) {
      ok = false;
      return nullptr;
    }
    if (device >= 0 && now != device) {
      PyErr_Format(PyExc_ValueError, "tensors on cuda:%d, the current device is cuda:%ld", device, now);
      ok = false;
      return nullptr;
    }
    PyObject* o = args[i];
    PyObject* handle;
    if (o == Py_None) {
      PyObject* dev = PyLong_FromLong(now);
      handle = dev ? PyObject_CallOneArg(g_stream, dev) : nullptr;
      Py_XDECREF(dev);
    } else if (PyObject_HasAttrString(o, "cuda_stream")) {
      handle = PyObject_GetAttrString(o, "cuda_stream");
    } else {
      handle = Py_NewRef(o);
    }
    void* s = handle ? PyLong_AsVoidPtr(handle) : nullptr;
    Py_XDECREF(handle);
    if (PyErr_Occurred()) ok = false;
    return s;
  }

  at::ScalarType type() const { return sh.dtype == MOONEP_BF16 ? at::kBFloat16 : at::kFloat; }
  wide element() const { return sh.dtype == MOONEP_BF16 ? 2 : 4; }
  wide tokens() const { return wide(sh.R) * sh.S; }
  wide slots() const { return tokens() * sh.K; }
  wide weight_rows() const { return sh.E + wide(sh.R) * sh.B; }
  wide cu_bytes() const { return 4 * wide(sh.R) * (wide(sh.E) + sh.B + 1); }
};

wide row_bytes(wide width) { return 128 * ((width + 127) / 128); }
wide columns(wide Hp) { return 16 * ((Hp + 15) / 16); }
constexpr auto I8 = at::kChar;
constexpr auto I32 = at::kInt;
constexpr auto F32 = at::kFloat;

template <typename T>
T* as(void* p) { return static_cast<T*>(p); }

// The library's call, with Python's lock released: a launch waits where the GPU's queue is full,
// and other threads (or a host function of the queue that needs the lock) have to go on. Releasing
// and taking it again costs under 0.1 us a call. Taking it ends a daemon thread's stack where
// the interpreter is on its way out, so that must not happen in a destructor.
template <typename F, typename... A>
int unlocked(F call, A... a) {
  PyThreadState* const state = PyEval_SaveThread();
  int st;
  try {
    st = call(a...);
  } catch (...) {
    PyEval_RestoreThread(state);
    throw;
  }
  PyEval_RestoreThread(state);
  return st;
}

// Runs a call's body; C++ exceptions (a tensor without storage, for one) become Python's.
template <typename F>
PyObject* run(PyObject* const* args, Py_ssize_t n, Py_ssize_t want, F body) {
  try {
    Call c(args, n, want);
    const int st = c.ok ? body(c) : 0;
    return c.ok ? PyLong_FromLong(st) : nullptr;
  } catch (const std::exception& e) {
    PyErr_SetString(PyExc_RuntimeError, e.what());
    return nullptr;
  }
}

PyObject* quantize(PyObject*, PyObject* const* args, Py_ssize_t n) {
  return run(args, n, 7, [](Call& c) {      // shape, rows, width, src, q, scales, stream
    const int64_t rows = c.integer(1, "rows"), width = c.integer(2, "width");
    void* src = c.tensor(3, "src", wide(rows) * width * c.element(), c.type());
    void* q = c.tensor(4, "q", rows * row_bytes(width), I8);
    void* scales = c.tensor(5, "scales", 4 * wide(rows), F32);
    void* s = c.stream(6);
    if (width != int32_t(width)) return int(MOONEP_EINVAL);
    return c.ok ? unlocked(f.quantize, &c.sh, rows, int32_t(width), src, as<int8_t>(q), as<float>(scales), s)
                : 0;
  });
}

PyObject* quantize_weight(PyObject*, PyObject* const* args, Py_ssize_t n) {
  return run(args, n, 5, [](Call& c) {      // shape, w, wq, wscales, stream
    const wide cols = columns(c.sh.Hp);
    void* w = c.tensor(1, "w", wide(c.sh.E) * c.sh.H * c.sh.Hp * c.element(), c.type());
    void* wq = c.tensor(2, "wq", c.sh.E * cols * row_bytes(c.sh.H), I8);
    void* ws = c.tensor(3, "wscales", 4 * c.sh.E * cols, F32);
    void* s = c.stream(4);
    return c.ok ? unlocked(f.quantize_weight, &c.sh, w, as<int8_t>(wq), as<float>(ws), s) : 0;
  });
}

PyObject* transpose_weight(PyObject*, PyObject* const* args, Py_ssize_t n) {
  return run(args, n, 4, [](Call& c) {      // shape, wq, wqt, stream
    void* wq = c.tensor(1, "wq", c.sh.E * columns(c.sh.Hp) * row_bytes(c.sh.H), I8);
    void* wqt = c.tensor(2, "wqt", c.sh.E * columns(c.sh.H) * row_bytes(c.sh.Hp), I8);
    void* s = c.stream(3);
    return c.ok ? unlocked(f.transpose_weight, &c.sh, as<int8_t>(wq), as<int8_t>(wqt), s) : 0;
  });
}

PyObject* prefetch_weight(PyObject*, PyObject* const* args, Py_ssize_t n) {
  return run(args, n, 5, [](Call& c) {      // shape, replica_expert, wq, wscales, stream
    void* replica = c.tensor(1, "replica_expert", 4 * wide(c.sh.R) * c.sh.B, I32);
    const wide cols = c.weight_rows() * columns(c.sh.Hp);
    void* wq = c.tensor(2, "wq", cols * row_bytes(c.sh.H), I8);
    void* ws = c.tensor(3, "wscales", 4 * cols, F32, true);
    void* s = c.stream(4);
    return c.ok ? unlocked(f.prefetch_weight, &c.sh, as<int32_t>(replica), as<int8_t>(wq), as<float>(ws), s)
                : 0;
  });
}

// The operands of a product from argument i on (xq, xscales, [src_index,] wq, wscales)
struct Operands {
  void *xq, *xs, *index = nullptr, *wq, *ws;
  Operands(Call& c, int i, bool plan, wide rows, wide weights, wide W) {
    if (plan && c.args[i + 2] != Py_None) rows = c.tokens();
    xq = c.tensor(i, "xq", rows * row_bytes(c.sh.H), I8);
    xs = c.tensor(i + 1, "xscales", 4 * rows, F32);
    if (plan) index = c.tensor(i + 2, "src_index", 4 * c.slots(), I32, true);
    i += plan ? 3 : 2;
    const wide cols = weights * columns(W);
    wq = c.tensor(i, "wq", cols * row_bytes(c.sh.H), I8);
    ws = c.tensor(i + 1, "wscales", 4 * cols, F32, true);
  }
};

PyObject* grouped_gemm(PyObject*, PyObject* const* args, Py_ssize_t n) {
  // shape, xq, xscales, src_index, wq, wscales, cu_seqlens, c, ws, stream
  return run(args, n, 10, [](Call& c) {
    const Operands o(c, 1, true, c.slots(), c.weight_rows(), c.sh.Hp);
    void* cu = c.tensor(6, "cu_seqlens", c.cu_bytes(), I32);
    void* out = c.tensor(7, "c", 4 * c.slots() * c.sh.Hp, F32);
    void* ws = c.tensor(8, "ws", 0, at::ScalarType::Undefined);
    void* s = c.stream(9);
    return c.ok ? unlocked(f.grouped_gemm, &c.sh, as<int8_t>(o.xq), as<float>(o.xs), as<int32_t>(o.index),
                           as<int8_t>(o.wq), as<float>(o.ws), as<int32_t>(cu), as<float>(out), ws,
                           THPVariable_Unpack(c.args[8]).nbytes(), s)
                : 0;
  });
}

PyObject* grouped_gemm_swiglu(PyObject*, PyObject* const* args, Py_ssize_t n) {
  // shape, xq, xscales, src_index, wq, wscales, cu_seqlens, act, h_saved, ws, stream
  return run(args, n, 11, [](Call& c) {
    const wide act_bytes = c.slots() * c.sh.Hp * c.element();
    const Operands o(c, 1, true, c.slots(), c.weight_rows(), 2 * wide(c.sh.Hp));
    void* cu = c.tensor(6, "cu_seqlens", c.cu_bytes(), I32);
    void* act = c.tensor(7, "act", act_bytes, c.type());
    void* h = c.tensor(8, "h_saved", 2 * act_bytes, c.type(), true);
    void* ws = c.tensor(9, "ws", 0, at::ScalarType::Undefined);
    void* s = c.stream(10);
    return c.ok ? unlocked(f.grouped_gemm_swiglu, &c.sh, as<int8_t>(o.xq), as<float>(o.xs),
                           as<int32_t>(o.index), as<int8_t>(o.wq), as<float>(o.ws), as<int32_t>(cu), act, h,
                           ws, THPVariable_Unpack(c.args[9]).nbytes(), s)
                : 0;
  });
}

PyObject* gemm(PyObject*, PyObject* const* args, Py_ssize_t n) {
  return run(args, n, 9, [](Call& c) {      // shape, rows, xq, xscales, wq, wscales, add, c, stream
    const int64_t rows = c.integer(1, "rows");
    const wide bytes = 4 * wide(rows) * c.sh.Hp;
    const Operands o(c, 2, false, rows, 1, c.sh.Hp);
    void* add = c.tensor(6, "add", bytes, F32, true);
    void* out = c.tensor(7, "c", bytes, F32);
    void* s = c.stream(8);
    return c.ok ? unlocked(f.gemm, &c.sh, rows, as<int8_t>(o.xq), as<float>(o.xs), as<int8_t>(o.wq),
                           as<float>(o.ws), as<float>(add), as<float>(out), s)
                : 0;
  });
}

PyObject* gemm_swiglu(PyObject*, PyObject* const* args, Py_ssize_t n) {
  return run(args, n, 9, [](Call& c) {      // shape, rows, xq, xscales, wq, wscales, act, h_saved, stream
    const int64_t rows = c.integer(1, "rows");
    const wide bytes = wide(rows) * c.sh.Hp * c.element();
    const Operands o(c, 2, false, rows, 1, 2 * wide(c.sh.Hp));
    void* act = c.tensor(6, "act", bytes, c.type());
    void* h = c.tensor(7, "h_saved", 2 * bytes, c.type(), true);
    void* s = c.stream(8);
    return c.ok ? unlocked(f.gemm_swiglu, &c.sh, rows, as<int8_t>(o.xq), as<float>(o.xs), as<int8_t>(o.wq),
                           as<float>(o.ws), act, h, s)
                : 0;
  });
}

PyObject* quantize_grad(PyObject*, PyObject* const* args, Py_ssize_t n) {
  // shape, src, src_index, gates, wscales, cu_seqlens, q, scales, stream
  return run(args, n, 9, [](Call& c) {
    const wide slots = c.slots(), rows = c.args[2] == Py_None ? slots : c.tokens();
    void* src = c.tensor(1, "src", rows * c.sh.Hp * c.element(), c.type());
    void* index = c.tensor(2, "src_index", 4 * slots, I32, true);
    void* gates = c.tensor(3, "gates", 4 * slots, F32, true);
    const wide weights = c.args[5] == Py_None ? wide(1) : c.weight_rows();
    void* ws = c.tensor(4, "wscales", 4 * weights * columns(c.sh.Hp), F32);
    void* cu = c.tensor(5, "cu_seqlens", c.cu_bytes(), I32, true);
    void* q = c.tensor(6, "q", slots * row_bytes(c.sh.Hp), I8);
    void* scales = c.tensor(7, "scales", 4 * slots, F32);
    void* s = c.stream(8);
    return c.ok ? unlocked(f.quantize_grad, &c.sh, src, as<int32_t>(index), as<float>(gates), as<float>(ws),
                           as<int32_t>(cu), as<int8_t>(q), as<float>(scales), s)
                : 0;
  });
}

PyObject* bind(PyObject*, PyObject* args) {
  unsigned long long p[9];
  PyObject *device, *stream;
  if (!PyArg_ParseTuple(args, "(KKKKKKKKK)OO", &p[0], &p[1], &p[2], &p[3], &p[4], &p[5], &p[6], &p[7],
                        &p[8], &device, &stream))
    return nullptr;
  static_assert(sizeof f == sizeof p, "nine functions");
  memcpy(&f, p, sizeof f);
  Py_XSETREF(g_device, Py_NewRef(device));
  Py_XSETREF(g_stream, Py_NewRef(stream));
  Py_RETURN_NONE;
}

#define FAST(name) {#name, reinterpret_cast<PyCFunction>(reinterpret_cast<void*>(name)), METH_FASTCALL, nullptr}
PyMethodDef methods[] = {
    {"bind", bind, METH_VARARGS, nullptr},
    FAST(quantize), FAST(quantize_weight), FAST(transpose_weight), FAST(prefetch_weight),
    FAST(grouped_gemm), FAST(grouped_gemm_swiglu), FAST(gemm), FAST(gemm_swiglu), FAST(quantize_grad),
    {nullptr, nullptr, 0, nullptr}};
PyModuleDef module = {PyModuleDef_HEAD_INIT, "_binding", nullptr, -1, methods, nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__binding(void) { return PyModule_Create(&module); }
