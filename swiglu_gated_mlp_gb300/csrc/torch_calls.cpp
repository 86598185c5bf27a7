// The 8-bit calls of _native.py for their common case: tensors as the kernels take
// them, on the current device and stream, outputs not given. Checks, allocation of the
// outputs and the C call are made here, as those kernels run for less time than the
// same steps take in Python (quantiser and projection of 1 token on a Grace host: 26 us
// of Python for 12 us on the GPU). Whatever else a call asks for, or has wrong, is
// answered with None, and the caller goes through its own checks, which name the fault.
#define PY_SSIZE_T_CLEAN
#include <Python.h>

#include <ATen/ops/empty.h>
#include <c10/cuda/CUDAFunctions.h>
#include <c10/cuda/CUDAStream.h>
#include <torch/csrc/Exceptions.h>
#include <torch/csrc/autograd/python_variable.h>

#include "swiglu.h"

namespace {

using at::Tensor;

bool has(const Tensor& t, at::ScalarType type, int device) {
  return t.is_cuda() && t.get_device() == device && t.scalar_type() == type && t.is_contiguous();
}

bool matrix(const Tensor& t, at::ScalarType type, int device) { return has(t, type, device) && t.dim() == 2; }

bool matrix(const Tensor& t, at::ScalarType type, int device, int64_t rows, int64_t cols) {
  return matrix(t, type, device) && t.size(0) == rows && t.size(1) == cols;
}

bool vector(const Tensor& t, int device, int64_t n) {
  return has(t, at::kFloat, device) && t.dim() == 1 && t.size(0) == n;
}

// A packed weight or a workspace of at least `bytes`.
bool buffer(const Tensor& t, int device, int64_t bytes) {
  return t.is_cuda() && t.get_device() == device && t.is_contiguous() && static_cast<int64_t>(t.nbytes()) >= bytes;
}

int64_t div_up(int64_t a, int64_t b) { return (a + b - 1) / b; }

// Scales of a checkpoint: [2, ceil(N / 128), M].
bool scales(const Tensor& t, int device, int64_t m, int64_t n) {
  return has(t, at::kFloat, device) && t.dim() == 3 && t.size(0) == 2 && t.size(1) == div_up(n, 128) && t.size(2) == m;
}

// The arguments of a call: tensors (of exactly torch's own classes), some of them None, and one size.
struct Args {
  PyObject* const* a;
  Py_ssize_t n;
  bool ok = true;
  const Tensor none;

  Args(PyObject* const* args, Py_ssize_t count, Py_ssize_t want) : a(args), n(count), ok(count == want) {}
  const Tensor& tensor(int i) {
    if (ok && THPVariable_CheckExact(a[i])) return THPVariable_Unpack(a[i]);
    ok = false;
    return none;
  }
  const Tensor& maybe(int i) {
    if (ok && a[i] == Py_None) return none;
    return tensor(i);
  }
  int64_t size(int i) {  // at most 31 bits, so that the sizes made from it do not overflow
    const int64_t v = ok && PyLong_CheckExact(a[i]) ? PyLong_AsLongLong(a[i]) : -1;
    if (v < 0 || v > 0x7fffffff) {
      PyErr_Clear();
      ok = false;
    }
    return v;
  }
};

// The current device, for a CUDA tensor; -1 for others.
int here(const Args& a, const Tensor& t) { return a.ok && t.is_cuda() ? c10::cuda::current_device() : -1; }

Tensor new_tensor(at::IntArrayRef shape, at::ScalarType type, const Tensor& beside) {
  return at::empty(shape, beside.options().dtype(type).requires_grad(false));
}

const float* floats(const Tensor& t) { return static_cast<const float*>(t.const_data_ptr()); }
const void* at_or_null(const Tensor& t) { return t.defined() ? t.const_data_ptr() : nullptr; }

// Runs the C call on the current stream of `device` without the interpreter's lock.
template <typename F>
bool run(int device, F call) {
  const swiglu_stream_t stream = c10::cuda::getCurrentCUDAStream(static_cast<c10::DeviceIndex>(device)).stream();
  swiglu_status_t st;
  Py_BEGIN_ALLOW_THREADS;
  st = call(stream);
  Py_END_ALLOW_THREADS;
  return st == SWIGLU_OK;
}

PyObject* wrapped(std::initializer_list<Tensor> ts) {
  PyObject* r = PyTuple_New(static_cast<Py_ssize_t>(ts.size()));
  if (!r) return nullptr;
  Py_ssize_t i = 0;
  for (const Tensor& t : ts) {
    PyObject* o = THPVariable_Wrap(t);
    if (!o) {
      Py_DECREF(r);
      return nullptr;
    }
    PyTuple_SET_ITEM(r, i++, o);
  }
  return r;
}

// (X) -> (Q, scale)
PyObject* quantize_int8(PyObject*, PyObject* const* args, Py_ssize_t n) {
  HANDLE_TH_ERRORS
  Args a(args, n, 1);
  const Tensor& x = a.tensor(0);
  const int device = here(a, x);
  if (device < 0 || !matrix(x, at::kBFloat16, device)) Py_RETURN_NONE;
  const int64_t m = x.size(0), k = x.size(1);
  const Tensor q = new_tensor({m, k}, at::kChar, x), s = new_tensor({m}, at::kFloat, x);
  if (!run(device, [&](swiglu_stream_t st) {
        return swiglu_quantize_int8(x.const_data_ptr(), q.data_ptr(), static_cast<float*>(s.data_ptr()), m, k, st);
      }))
    Py_RETURN_NONE;
  return wrapped({q, s});
  END_HANDLE_TH_ERRORS
}

// (A, scale_a, Wpacked, N, scale_w1, scale_w2, workspace or None) -> Y
PyObject* forward_int8(PyObject*, PyObject* const* args, Py_ssize_t n) {
  HANDLE_TH_ERRORS
  Args a(args, n, 7);
  const Tensor &x = a.tensor(0), &sa = a.tensor(1), &wp = a.tensor(2);
  const int64_t cols = a.size(3);
  const Tensor &s1 = a.tensor(4), &s2 = a.tensor(5);
  Tensor ws = a.maybe(6);
  const int device = here(a, x);
  if (device < 0 || !matrix(x, at::kChar, device)) Py_RETURN_NONE;
  const int64_t m = x.size(0), k = x.size(1);
  if (!vector(sa, device, m) || !vector(s1, device, cols) || !vector(s2, device, cols) ||
      !buffer(wp, device, div_up(cols, 128) * div_up(k, 128) * 32768) || (ws.defined() && !buffer(ws, device, 0)))
    Py_RETURN_NONE;
  const Tensor y = new_tensor({m, cols}, at::kBFloat16, x);
  if (!ws.defined()) ws = new_tensor({static_cast<int64_t>(swiglu_int8_workspace_bytes(m, k, cols))}, at::kByte, x);
  if (!run(device, [&](swiglu_stream_t st) {
        return swiglu_forward_int8(x.const_data_ptr(), floats(sa), wp.const_data_ptr(), floats(s1), floats(s2), y.data_ptr(),
                                   m, k, cols, ws.data_ptr(), ws.nbytes(), st);
      }))
    Py_RETURN_NONE;
  return THPVariable_Wrap(y);
  END_HANDLE_TH_ERRORS
}

// (Y, scale_y, W3packed, H, scale_w3, R or None, workspace or None) -> Out
PyObject* down_forward_int8(PyObject*, PyObject* const* args, Py_ssize_t n) {
  HANDLE_TH_ERRORS
  Args a(args, n, 7);
  const Tensor &x = a.tensor(0), &sy = a.tensor(1), &wp = a.tensor(2);
  const int64_t cols = a.size(3);
  const Tensor &s3 = a.tensor(4), &r = a.maybe(5);
  Tensor ws = a.maybe(6);
  const int device = here(a, x);
  if (device < 0 || !matrix(x, at::kChar, device)) Py_RETURN_NONE;
  const int64_t m = x.size(0), k = x.size(1);
  if (!vector(sy, device, m) || !vector(s3, device, cols) ||
      !buffer(wp, device, div_up(cols, 256) * div_up(k, 128) * 32768) ||
      (r.defined() && !matrix(r, at::kBFloat16, device, m, cols)) || (ws.defined() && !buffer(ws, device, 0)))
    Py_RETURN_NONE;
  const Tensor out = new_tensor({m, cols}, at::kBFloat16, x);
  if (!ws.defined()) ws = new_tensor({static_cast<int64_t>(swiglu_down_int8_workspace_bytes(m, k, cols))}, at::kByte, x);
  if (!run(device, [&](swiglu_stream_t st) {
        return swiglu_down_forward_int8(x.const_data_ptr(), floats(sy), wp.const_data_ptr(), floats(s3), at_or_null(r),
                                        out.data_ptr(), m, k, cols, ws.data_ptr(), ws.nbytes(), st);
      }))
    Py_RETURN_NONE;
  return THPVariable_Wrap(out);
  END_HANDLE_TH_ERRORS
}

// (A, Wpacked, N) -> (Y, gate, up, scale)
PyObject* forward_checkpoint(PyObject*, PyObject* const* args, Py_ssize_t n) {
  HANDLE_TH_ERRORS
  Args a(args, n, 3);
  const Tensor &x = a.tensor(0), &wp = a.tensor(1);
  const int64_t cols = a.size(2);
  const int device = here(a, x);
  if (device < 0 || !matrix(x, at::kBFloat16, device)) Py_RETURN_NONE;
  const int64_t m = x.size(0), k = x.size(1);
  if (!has(wp, at::kBFloat16, device) || wp.numel() < div_up(cols, 128) * div_up(k, 64) * 16384) Py_RETURN_NONE;
  const Tensor y = new_tensor({m, cols}, at::kBFloat16, x), gate = new_tensor({m, cols}, at::kChar, x),
               up = new_tensor({m, cols}, at::kChar, x), s = new_tensor({2, div_up(cols, 128), m}, at::kFloat, x);
  if (!run(device, [&](swiglu_stream_t st) {
        return swiglu_forward_checkpoint(x.const_data_ptr(), wp.const_data_ptr(), y.data_ptr(), gate.data_ptr(),
                                         up.data_ptr(), static_cast<float*>(s.data_ptr()), m, k, cols, st);
      }))
    Py_RETURN_NONE;
  return wrapped({y, gate, up, s});
  END_HANDLE_TH_ERRORS
}

// (gate, up, scale) -> Y
PyObject* checkpoint_output(PyObject*, PyObject* const* args, Py_ssize_t n) {
  HANDLE_TH_ERRORS
  Args a(args, n, 3);
  const Tensor &gate = a.tensor(0), &up = a.tensor(1), &s = a.tensor(2);
  const int device = here(a, gate);
  if (device < 0 || !matrix(gate, at::kChar, device)) Py_RETURN_NONE;
  const int64_t m = gate.size(0), cols = gate.size(1);
  if (!matrix(up, at::kChar, device, m, cols) || !scales(s, device, m, cols)) Py_RETURN_NONE;
  const Tensor y = new_tensor({m, cols}, at::kBFloat16, gate);
  if (!run(device, [&](swiglu_stream_t st) {
        return swiglu_checkpoint_output(gate.const_data_ptr(), up.const_data_ptr(), floats(s), y.data_ptr(), m, cols, st);
      }))
    Py_RETURN_NONE;
  return THPVariable_Wrap(y);
  END_HANDLE_TH_ERRORS
}

// (A, Wpacked, dY, gate, up, scale, scale_a or None, workspace or None) -> (dA, dW1, dW2)
PyObject* backward_checkpoint(PyObject*, PyObject* const* args, Py_ssize_t n) {
  HANDLE_TH_ERRORS
  Args a(args, n, 8);
  const Tensor &x = a.tensor(0), &wp = a.tensor(1), &dy = a.tensor(2), &gate = a.tensor(3), &up = a.tensor(4),
               &s = a.tensor(5), &sa = a.maybe(6);
  Tensor ws = a.maybe(7);
  const int device = here(a, gate);
  if (device < 0 || !matrix(gate, at::kChar, device)) Py_RETURN_NONE;
  const int64_t m = gate.size(0), cols = gate.size(1);
  if (!matrix(x, sa.defined() ? at::kChar : at::kBFloat16, device) || x.size(0) != m ||
      (sa.defined() && !vector(sa, device, m)) || !matrix(up, at::kChar, device, m, cols) ||
      !scales(s, device, m, cols) || !matrix(dy, at::kBFloat16, device, m, cols) || !has(wp, at::kBFloat16, device) ||
      wp.numel() < div_up(cols, 128) * div_up(x.size(1), 64) * 16384 || (ws.defined() && !buffer(ws, device, 0)))
    Py_RETURN_NONE;
  const int64_t k = x.size(1);
  const Tensor da = new_tensor({m, k}, at::kBFloat16, dy), dw1 = new_tensor({k, cols}, at::kBFloat16, dy),
               dw2 = new_tensor({k, cols}, at::kBFloat16, dy);
  if (!ws.defined())
    ws = new_tensor({static_cast<int64_t>(swiglu_backward_checkpoint_workspace_bytes(m, k, cols))}, at::kByte, dy);
  if (!run(device, [&](swiglu_stream_t st) {
        return swiglu_backward_checkpoint(x.const_data_ptr(), static_cast<const float*>(at_or_null(sa)), wp.const_data_ptr(),
                                          dy.const_data_ptr(), gate.const_data_ptr(), up.const_data_ptr(), floats(s),
                                          da.data_ptr(), dw1.data_ptr(), dw2.data_ptr(), m, k, cols, ws.data_ptr(),
                                          ws.nbytes(), st);
      }))
    Py_RETURN_NONE;
  return wrapped({da, dw1, dw2});
  END_HANDLE_TH_ERRORS
}

template <PyObject* (*F)(PyObject*, PyObject* const*, Py_ssize_t)>
PyCFunction fast() {
  return reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(F));
}

PyMethodDef methods[] = {{"quantize_int8", fast<quantize_int8>(), METH_FASTCALL, nullptr},
                         {"forward_int8", fast<forward_int8>(), METH_FASTCALL, nullptr},
                         {"down_forward_int8", fast<down_forward_int8>(), METH_FASTCALL, nullptr},
                         {"forward_checkpoint", fast<forward_checkpoint>(), METH_FASTCALL, nullptr},
                         {"checkpoint_output", fast<checkpoint_output>(), METH_FASTCALL, nullptr},
                         {"backward_checkpoint", fast<backward_checkpoint>(), METH_FASTCALL, nullptr},
                         {nullptr, nullptr, 0, nullptr}};
PyModuleDef module = {PyModuleDef_HEAD_INIT, "_torch_calls", nullptr, -1, methods, nullptr, nullptr, nullptr, nullptr};

}  // namespace

// built_for: the PyTorch and Python whose binary interfaces this file was compiled against.
PyMODINIT_FUNC PyInit__torch_calls() {
  PyObject* m = PyModule_Create(&module);
  if (m && PyModule_AddStringConstant(m, "built_for", SWIGLU_BUILT_FOR) != 0) {
    Py_DECREF(m);
    return nullptr;
  }
  return m;
}
