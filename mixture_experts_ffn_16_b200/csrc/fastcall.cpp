// fastcall.cpp - the common case of the Python binding's token-dispatch and
// MXFP4 calls in native code: every argument a plain contiguous CUDA tensor of
// the right type and shape on the current device, work on its current stream.
// Then the checks and the call take 0.3 us around the launch's 2.1 us, where
// the same in Python and ctypes takes 3.6 us or more, longer than the smallest
// operators run.
//
// A function returns the library's status, or None for anything else: api.py
// then looks again and raises what is wrong, or makes the call itself (another
// stream, a tensor subclass).  Nothing is kept between calls but the library's
// function addresses (bind).
#include <Python.h>

#include <ATen/core/Tensor.h>
#include <c10/cuda/CUDAFunctions.h>
#include <c10/cuda/CUDAStream.h>
#include <torch/csrc/autograd/python_variable.h>

#include "moe.h"

namespace {

struct Library {
  decltype(&moe_sort_tokens) sort_tokens;
  decltype(&moe_dispatch) dispatch;
  decltype(&moe_dispatch_backward) dispatch_backward;
  decltype(&moe_undispatch) undispatch;
  decltype(&moe_undispatch_backward) undispatch_backward;
  decltype(&moe_quantize_fp4) quantize_fp4;
  decltype(&moe_dequantize_fp4) dequantize_fp4;
  decltype(&moe_dispatch_fp4) dispatch_fp4;
  decltype(&moe_matmul_fp4) matmul_fp4;
  decltype(&moe_swiglu_fp4) swiglu_fp4;
} lib;

constexpr auto kInt = at::kInt;
constexpr auto kFloat = at::kFloat;
constexpr auto kByte = at::kByte;

// The arguments of one call; `ok` turns false at the first that is not plain.
struct Call {
  PyObject* const* args;
  bool ok;
  int dev = -1;

  Call(PyObject* const* a, Py_ssize_t n, Py_ssize_t want) : args(a), ok(n == want) {}

  // Argument i as a contiguous CUDA tensor of n dimensions on the call's
  // device (the first tensor's, which must be the current one).
  const at::Tensor* tensor(int i, int n) { return ok ? check(args[i], n) : nullptr; }
  const at::Tensor* tensor(int i, int n, at::ScalarType type) {
    const at::Tensor* t = tensor(i, n);
    ok = ok && t->scalar_type() == type;
    return t;
  }
  // Argument i as the MXFP4 pair (codes, scales) of G x rows x K values; what
  // is negative is read from the codes.
  moe_fp4_tensor fp4(int i, int64_t& G, int64_t& rows, int64_t& K) {
    moe_fp4_tensor q = {nullptr, nullptr};
    ok = ok && PyTuple_CheckExact(args[i]) && PyTuple_GET_SIZE(args[i]) == 2;
    if (ok) pair(PyTuple_GET_ITEM(args[i], 0), PyTuple_GET_ITEM(args[i], 1), q, G, rows, K);
    return q;
  }
  moe_fp4_tensor fp4(int i, int j, int64_t& G, int64_t& rows, int64_t& K) {
    moe_fp4_tensor q = {nullptr, nullptr};
    if (ok) pair(args[i], args[j], q, G, rows, K);
    return q;
  }
  // The type code of a row tensor.
  int dtype(const at::Tensor* t) {
    if (!ok) return -1;
    switch (t->scalar_type()) {
      case at::kBFloat16: return MOE_BF16;
      case at::kHalf: return MOE_FP16;
      case at::kFloat: return MOE_FP32;
      default: ok = false; return -1;
    }
  }
  void is(bool condition) { ok = ok && condition; }
  moe_stream_t stream() const { return c10::cuda::getCurrentCUDAStream(static_cast<c10::DeviceIndex>(dev)).stream(); }

 private:
  const at::Tensor* check(PyObject* o, int n) {
    if (!THPVariable_CheckExact(o)) {
      ok = false;
      return nullptr;
    }
    const at::Tensor& t = THPVariable_Unpack(o);
    if (!t.is_cuda() || t.dim() != n || !t.is_contiguous() || t.is_neg() || t.is_conj()) {
      ok = false;
      return nullptr;
    }
    if (dev < 0) {
      dev = t.device().index();
      ok = dev == c10::cuda::current_device();
    } else {
      ok = dev == t.device().index();
    }
    return &t;
  }
  void pair(PyObject* c, PyObject* s, moe_fp4_tensor& q, int64_t& G, int64_t& rows, int64_t& K) {
    const at::Tensor* codes = check(c, 3);
    const at::Tensor* scales = ok ? check(s, 4) : nullptr;
    if (!ok) return;
    if (G < 0) G = codes->size(0);
    if (rows < 0) rows = codes->size(1);
    if (K < 0) K = 2 * codes->size(2);
    ok = codes->scalar_type() == kByte && scales->scalar_type() == kByte && codes->size(0) == G &&
         codes->size(1) == rows && 2 * codes->size(2) == K && scales->size(0) == G &&
         scales->size(1) == (K + 127) / 128 && scales->size(2) == rows && scales->size(3) == 4;
    q.codes = codes->data_ptr();
    q.scales = scales->data_ptr();
  }
};

int32_t i32(int64_t v) { return v > INT32_MAX ? INT32_MAX : static_cast<int32_t>(v); }   // INT32_MAX is refused
template <typename T>
T* ptr(const at::Tensor* t) { return static_cast<T*>(t->data_ptr()); }

// A library call without the interpreter's lock, as ctypes makes it: a launch
// may wait for room in a full queue whose next entry is a host function that
// wants the lock.
template <typename F, typename... A>
int call(F f, A... a) {
  PyThreadState* const state = PyEval_SaveThread();
  const int status = f(a...);
  PyEval_RestoreThread(state);
  return status;
}

// `body` returns the library's status; None where the call is not plain or an
// exception (of torch's) came up.
template <typename F>
PyObject* run(Call& c, F body) {
  try {
    const int status = body();
    if (c.ok) return PyLong_FromLong(status);
  } catch (...) {
  }
  Py_RETURN_NONE;
}

bool shaped(const at::Tensor* t, int64_t a, int64_t b) { return t->size(0) == a && t->size(1) == b; }

PyObject* sort_tokens(PyObject*, PyObject* const* a, Py_ssize_t n) {
  Call c(a, n, 4);
  return run(c, [&] {
    const at::Tensor *idx = c.tensor(0, 2, kInt), *off = c.tensor(1, 1, kInt), *row = c.tensor(2, 2, kInt),
                     *ws = c.tensor(3, 1, kByte);
    if (!c.ok) return 0;
    const int64_t T = idx->size(0), k = idx->size(1);
    c.is(shaped(row, T, k));
    return !c.ok ? 0
                 : call(lib.sort_tokens, i32(T), i32(k), i32(off->size(0) - 1), ptr<int32_t>(idx), ptr<int32_t>(off),
                        ptr<int32_t>(row), ws->data_ptr(), ws->numel(), c.stream());
  });
}

PyObject* dispatch(PyObject*, PyObject* const* a, Py_ssize_t n) {
  Call c(a, n, 3);
  return run(c, [&] {
    const at::Tensor *x = c.tensor(0, 2), *row = c.tensor(1, 2, kInt), *xs = c.tensor(2, 2);
    const int dt = c.dtype(x);
    if (!c.ok) return 0;
    const int64_t T = x->size(0), d = x->size(1), k = row->size(1);
    c.is(row->size(0) == T && shaped(xs, T * k, d) && xs->scalar_type() == x->scalar_type());
    return !c.ok ? 0
                 : call(lib.dispatch, i32(T), i32(k), i32(d), dt, x->data_ptr(), ptr<int32_t>(row), xs->data_ptr(),
                        c.stream());
  });
}

PyObject* dispatch_backward(PyObject*, PyObject* const* a, Py_ssize_t n) {
  Call c(a, n, 3);
  return run(c, [&] {
    const at::Tensor *dxs = c.tensor(0, 2), *row = c.tensor(1, 2, kInt), *dx = c.tensor(2, 2);
    const int dt = c.dtype(dx);
    if (!c.ok) return 0;
    const int64_t T = dx->size(0), d = dx->size(1), k = row->size(1);
    c.is(row->size(0) == T && shaped(dxs, T * k, d) && dxs->scalar_type() == dx->scalar_type());
    return !c.ok ? 0
                 : call(lib.dispatch_backward, i32(T), i32(k), i32(d), dt, dxs->data_ptr(), ptr<int32_t>(row),
                        dx->data_ptr(), c.stream());
  });
}

PyObject* undispatch(PyObject*, PyObject* const* a, Py_ssize_t n) {
  Call c(a, n, 4);
  return run(c, [&] {
    const at::Tensor *y = c.tensor(0, 2), *row = c.tensor(1, 2, kInt), *w = c.tensor(2, 2, kFloat),
                     *out = c.tensor(3, 2);
    const int dt = c.dtype(out);
    if (!c.ok) return 0;
    const int64_t T = out->size(0), d = out->size(1), k = row->size(1);
    c.is(row->size(0) == T && shaped(w, T, k) && shaped(y, T * k, d) && y->scalar_type() == out->scalar_type());
    return !c.ok ? 0
                 : call(lib.undispatch, i32(T), i32(k), i32(d), dt, y->data_ptr(), ptr<int32_t>(row), ptr<float>(w),
                        out->data_ptr(), c.stream());
  });
}

PyObject* undispatch_backward(PyObject*, PyObject* const* a, Py_ssize_t n) {
  Call c(a, n, 6);
  return run(c, [&] {
    const at::Tensor *dout = c.tensor(0, 2), *y = c.tensor(1, 2), *row = c.tensor(2, 2, kInt),
                     *w = c.tensor(3, 2, kFloat), *dy = c.tensor(4, 2), *dw = c.tensor(5, 2, kFloat);
    const int dt = c.dtype(dout);
    if (!c.ok) return 0;
    const int64_t T = dout->size(0), d = dout->size(1), k = row->size(1);
    c.is(row->size(0) == T && shaped(w, T, k) && shaped(dw, T, k) && shaped(y, T * k, d) && shaped(dy, T * k, d) &&
         y->scalar_type() == dout->scalar_type() && dy->scalar_type() == dout->scalar_type());
    return !c.ok ? 0
                 : call(lib.undispatch_backward, i32(T), i32(k), i32(d), dt, dout->data_ptr(), y->data_ptr(),
                        ptr<int32_t>(row), ptr<float>(w), dy->data_ptr(), ptr<float>(dw),
                        c.stream());
  });
}

PyObject* quantize_fp4(PyObject*, PyObject* const* a, Py_ssize_t n) {
  Call c(a, n, 3);
  return run(c, [&] {
    const at::Tensor* x = c.tensor(0, 3);
    const int dt = c.dtype(x);
    if (!c.ok) return 0;
    int64_t G = x->size(0), rows = x->size(1), K = x->size(2);
    const moe_fp4_tensor q = c.fp4(1, 2, G, rows, K);
    return !c.ok ? 0 : call(lib.quantize_fp4, i32(G), i32(rows), i32(K), dt, x->data_ptr(), &q, c.stream());
  });
}

PyObject* dequantize_fp4(PyObject*, PyObject* const* a, Py_ssize_t n) {
  Call c(a, n, 3);
  return run(c, [&] {
    const at::Tensor* x = c.tensor(2, 3);
    const int dt = c.dtype(x);
    if (!c.ok) return 0;
    int64_t G = x->size(0), rows = x->size(1), K = x->size(2);
    const moe_fp4_tensor q = c.fp4(0, 1, G, rows, K);
    return !c.ok ? 0 : call(lib.dequantize_fp4, i32(G), i32(rows), i32(K), dt, &q, x->data_ptr(), c.stream());
  });
}

PyObject* dispatch_fp4(PyObject*, PyObject* const* a, Py_ssize_t n) {
  Call c(a, n, 3);
  return run(c, [&] {
    const at::Tensor *x = c.tensor(0, 2), *row = c.tensor(1, 2, kInt);
    const int dt = c.dtype(x);
    if (!c.ok) return 0;
    const int64_t T = x->size(0), k = row->size(1);
    int64_t one = 1, rows = T * k, d = x->size(1);
    c.is(row->size(0) == T);
    const moe_fp4_tensor q = c.fp4(2, one, rows, d);
    return !c.ok ? 0
                 : call(lib.dispatch_fp4, i32(T), i32(k), i32(d), dt, x->data_ptr(), ptr<int32_t>(row), &q, c.stream());
  });
}

PyObject* matmul_fp4(PyObject*, PyObject* const* a, Py_ssize_t n) {
  Call c(a, n, 5);
  return run(c, [&] {
    int64_t one = 1, rows = -1, K = -1, E = -1, N = -1;
    const moe_fp4_tensor x = c.fp4(0, one, rows, K);
    const at::Tensor* off = c.tensor(1, 1, kInt);
    const moe_fp4_tensor W = c.fp4(2, E, N, K);
    const at::Tensor *out = c.tensor(3, 2), *ws = c.tensor(4, 1, kByte);
    const int dt = c.dtype(out);
    if (!c.ok) return 0;
    c.is(off->size(0) == E + 1 && shaped(out, rows, N));
    return !c.ok ? 0
                 : call(lib.matmul_fp4, i32(rows), i32(E), i32(N), i32(K),
                        &x, ptr<int32_t>(off), &W, dt, out->data_ptr(), ws->data_ptr(), ws->numel(), c.stream());
  });
}

PyObject* swiglu_fp4(PyObject*, PyObject* const* a, Py_ssize_t n) {
  Call c(a, n, 6);
  return run(c, [&] {
    int64_t one = 1, rows = -1, K = -1, E = -1, f = -1;
    const moe_fp4_tensor x = c.fp4(0, one, rows, K);
    const at::Tensor* off = c.tensor(1, 1, kInt);
    const moe_fp4_tensor Wg = c.fp4(2, E, f, K), Wu = c.fp4(3, E, f, K), h = c.fp4(4, one, rows, f);
    const at::Tensor* ws = c.tensor(5, 1, kByte);
    if (!c.ok) return 0;
    c.is(off->size(0) == E + 1);
    return !c.ok ? 0
                 : call(lib.swiglu_fp4, i32(rows), i32(E), i32(f), i32(K), &x, ptr<int32_t>(off), &Wg, &Wu, &h,
                        ws->data_ptr(), ws->numel(), c.stream());
  });
}

// bind(addresses): the library's functions in the order of Library.
PyObject* bind(PyObject*, PyObject* list) {
  constexpr Py_ssize_t count = sizeof(Library) / sizeof(void*);
  void* all[count];
  if (!PyTuple_Check(list) || PyTuple_GET_SIZE(list) != count) {
    PyErr_SetString(PyExc_TypeError, "bind: a tuple of the library's function addresses");
    return nullptr;
  }
  for (Py_ssize_t i = 0; i < count; ++i) {
    all[i] = PyLong_AsVoidPtr(PyTuple_GET_ITEM(list, i));
    if (PyErr_Occurred()) return nullptr;
  }
  static_assert(sizeof all == sizeof lib, "one address per function");
  memcpy(&lib, all, sizeof lib);
  Py_RETURN_NONE;
}

#define FAST(name) {#name, reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(name)), METH_FASTCALL, nullptr}
PyMethodDef methods[] = {{"bind", bind, METH_O, nullptr},
                         FAST(sort_tokens),
                         FAST(dispatch),
                         FAST(dispatch_backward),
                         FAST(undispatch),
                         FAST(undispatch_backward),
                         FAST(quantize_fp4),
                         FAST(dequantize_fp4),
                         FAST(dispatch_fp4),
                         FAST(matmul_fp4),
                         FAST(swiglu_fp4),
                         {nullptr, nullptr, 0, nullptr}};
PyModuleDef module = {PyModuleDef_HEAD_INIT, "_fastcall", nullptr, -1, methods};

}  // namespace

PyMODINIT_FUNC PyInit__fastcall() { return PyModule_Create(&module); }
