// Tensor arguments of the sequence operators: checks each torch tensor's type, device, shape and
// strides, allocates what the caller has not given, fills the C ABI's argument structure and calls it.
// Marshalling only, like the ctypes part of the package; it is native because the single-token calls
// take 4 us on the GPU, and the same checks in Python took 5 us of host time beside the launch's 3.7.
//
// Each function takes every argument by position (None where one is left out) and the stream's
// handle last, and returns the output tensor, or the sc_status of a refused call.
//
// No operator here has a gradient, so a tensor that asks for one is refused while gradients are recorded
// (its call would leave the graph without a word), and tensors written in place count their versions.
#include <Python.h>

#include <ATen/core/Tensor.h>
#include <ATen/ops/empty.h>
#include <c10/core/DeviceGuard.h>
#include <c10/core/GradMode.h>
#include <torch/csrc/autograd/python_variable.h>

#include <sstream>
#include <stdexcept>

#include "../../include/sparseconv.h"

namespace {

using at::Tensor;
using Shape = at::IntArrayRef;

[[noreturn]] void refuse(const std::string& what) { throw std::invalid_argument(what); }

const Tensor& tensor(PyObject* o, const char* name) {
  if (!THPVariable_Check(o)) refuse(std::string(name) + " must be a tensor");
  const Tensor& t = THPVariable_Unpack(o);
  if (t.requires_grad() && c10::GradMode::is_enabled())
    refuse(std::string(name) + " requires a gradient, and this operator has none: call it under torch.no_grad()");
  return t;
}

// The caller's tensor o (or None) has been written by a launch.
void written(PyObject* o) {
  if (o == Py_None) return;
  const Tensor& t = THPVariable_Unpack(o);
  if (!t.is_inference()) t.unsafeGetTensorImpl()->bump_version();
}

[[noreturn]] void refuse_tensor(const Tensor& t, const char* name, at::ScalarType type, Shape shape, const char* how) {
  std::ostringstream s;
  s << name << " must be a " << type << " tensor of shape " << shape << " on x's GPU, " << how << ": got " << t.sizes()
    << " " << t.scalar_type() << " on " << t.device() << ", strides " << t.strides();
  refuse(s.str());
}

// What every tensor of a call is held against.
struct Call {
  const Tensor& x;
  at::ScalarType type;
  at::Device device;

  explicit Call(const Tensor& x_) : x(x_), type(x_.scalar_type()), device(x_.device()) {
    if (!x.is_cuda() || (type != at::kFloat && type != at::kBFloat16 && type != at::kHalf))
      refuse("x must be a float32, bfloat16 or float16 tensor on the GPU");
  }
  int dtype() const { return type == at::kFloat ? SC_F32 : type == at::kBFloat16 ? SC_BF16 : SC_F16; }

  bool fits(const Tensor& t, at::ScalarType ty, Shape shape) const {
    return t.scalar_type() == ty && t.device() == device && t.sizes() == shape;
  }
  // an activation whose last axis (the positions) is contiguous where `positions` is set
  void activation(const Tensor& t, const char* name, Shape shape, bool positions) const {
    if (!fits(t, type, shape) || (positions && shape.back() > 1 && t.stride(-1) != 1))
      refuse_tensor(t, name, type, shape, positions ? "its last axis contiguous" : "strided");
  }
  template <class P>
  const P* dense(PyObject* o, const char* name, at::ScalarType ty, Shape shape) const {
    if (o == Py_None) return nullptr;
    const Tensor& t = tensor(o, name);
    if (!fits(t, ty, shape) || !t.is_contiguous()) refuse_tensor(t, name, ty, shape, "contiguous");
    return static_cast<const P*>(t.data_ptr());
  }
  // a pool of states; returns its slots
  int64_t states(PyObject* o, const char* name, at::ScalarType ty, int64_t D, int64_t per, void** p, int64_t* stride) const {
    const Tensor& t = tensor(o, name);
    const int64_t shape[3] = {t.dim() == 3 ? t.size(0) : 0, D, per};
    if (!fits(t, ty, shape) || (per > 0 && ((per > 1 && t.stride(2) != 1) || (D > 1 && t.stride(1) != per))))
      refuse_tensor(t, name, ty, shape, "each slot contiguous");
    *p = per ? t.data_ptr() : nullptr;
    *stride = shape[0] > 1 ? t.stride(0) : D * per;
    return shape[0];
  }
  // both pools; returns the number of slots (B where there is no pool).  A pool of none has no address, so
  // the library could not tell it from no pool at all.
  int32_t pools(PyObject* first, PyObject* last, PyObject* slots, at::ScalarType ty, int64_t B, int64_t D, int64_t per,
                const void** fp, void** lp, int64_t* fs, int64_t* ls) const {
    int64_t n = B;
    void* p = nullptr;
    *fp = *lp = nullptr;
    *fs = *ls = 0;
    if (first != Py_None) {
      n = states(first, "initial_state", ty, D, per, &p, fs);
      *fp = p;
    }
    if (last == first) {
      *lp = p;
      *ls = *fs;
    } else if (last != Py_None) {
      const int64_t m = states(last, "final_state", ty, D, per, lp, ls);
      if (first != Py_None && m != n) refuse("initial_state and final_state have different numbers of slots");
      n = m;
    }
    if (n == 0 && B > 0 && per > 0 && slots == Py_None) refuse("a pool of states without slots: fewer than sequences");
    return size(n);
  }
  static int32_t size(int64_t v) {
    if (v > INT32_MAX) refuse("a size is 2^31 or more");
    return (int32_t)v;
  }
  Tensor output(PyObject* o, Shape shape, bool positions) const {
    if (o == Py_None) return at::empty(shape, x.options());
    const Tensor& t = tensor(o, "out");
    activation(t, "out", shape, positions);
    return t;
  }
  Tensor workspace(PyObject* o, int64_t need) const {
    if (need == 0) return Tensor();
    if (o == Py_None) return at::empty({need}, x.options().dtype(at::kByte));
    const Tensor& t = tensor(o, "workspace");
    if (t.device() != device || !t.is_contiguous()) refuse("workspace must be a contiguous tensor on x's GPU");
    return t;
  }
};

void check(Py_ssize_t got, Py_ssize_t want) {
  if (got != want) refuse("wrong number of arguments");
}

PyObject* answer(sc_status s, const Tensor& out, PyObject* given_out, PyObject* final_state) {
  if (s != SC_OK) return PyLong_FromLong(s);
  written(given_out);
  written(final_state);
  return THPVariable_Wrap(out);
}

// x, weight, bias, silu, lengths, slots, initial_state, final_state, out, axes of x, stream
PyObject* causal_conv(PyObject* const* v, Py_ssize_t n) {
  check(n, 11);
  const Call c(tensor(v[0], "x"));
  const Tensor &x = c.x, &weight = tensor(v[1], "weight");
  const int64_t axes = PyLong_AsLong(v[9]);
  if (x.dim() != axes) refuse(axes == 2 ? "x must be (B, D)" : "x must be (B, D, L)");
  if (weight.dim() != 2) refuse("weight must be (D, K)");
  const c10::DeviceGuard guard(c.device);
  const int64_t B = x.size(0), D = x.size(1), L = axes == 3 ? x.size(2) : 1, K = weight.size(1);
  c.activation(x, "x", x.sizes(), axes == 3);
  sc_causal_conv a{};
  a.weight = c.dense<float>(v[1], "weight", at::kFloat, {D, K});
  a.bias = c.dense<float>(v[2], "bias", at::kFloat, {D});
  a.flags = PyObject_IsTrue(v[3]) ? SC_SEQ_SILU : 0;
  a.lengths = c.dense<int32_t>(v[4], "lengths", at::kInt, {B});
  a.slots = c.dense<int32_t>(v[5], "slots", at::kInt, {B});
  a.num_slots = c.pools(v[6], v[7], v[5], c.type, B, D, K - 1, &a.initial_state, &a.final_state, &a.initial_stride, &a.final_stride);
  const Tensor out = c.output(v[8], x.sizes(), axes == 3);
  a.x = x.data_ptr(), a.out = out.data_ptr();
  a.x_batch = x.stride(0), a.x_channel = x.stride(1), a.out_batch = out.stride(0), a.out_channel = out.stride(1);
  a.dtype = c.dtype(), a.B = c.size(B), a.D = c.size(D), a.L = c.size(L), a.K = c.size(K);
  return answer(sparseconv_causal_conv(&a, PyLong_AsVoidPtr(v[10])), out, v[8], v[7]);
}

// x, dt, A, B, C, D, z, dt_bias, softplus, lengths, slots, initial_state, final_state, out, workspace, axes of x, stream
PyObject* selective_scan(PyObject* const* v, Py_ssize_t n) {
  check(n, 17);
  const Call c(tensor(v[0], "x"));
  const Tensor &x = c.x, &dt = tensor(v[1], "dt"), &A = tensor(v[2], "A"), &Bm = tensor(v[3], "B"), &Cm = tensor(v[4], "C");
  const int64_t axes = PyLong_AsLong(v[15]);
  const bool prompt = axes == 3;
  if (x.dim() != axes) refuse(prompt ? "x must be (B, D, L)" : "x must be (B, D)");
  if (A.dim() != 2) refuse("A must be (D, N)");
  if (Bm.dim() != axes + 1) refuse(prompt ? "B must be (batch, groups, N, L)" : "B must be (batch, groups, N)");
  const c10::DeviceGuard guard(c.device);
  const int64_t B = x.size(0), D = x.size(1), L = prompt ? x.size(2) : 1, N = A.size(1), G = Bm.size(1);
  const int64_t bc[4] = {B, G, N, L};
  const Shape bshape(bc, prompt ? 4 : 3);
  c.activation(x, "x", x.sizes(), prompt);
  c.activation(dt, "dt", x.sizes(), prompt);
  c.activation(Bm, "B", bshape, prompt);
  c.activation(Cm, "C", bshape, prompt);
  sc_selective_scan a{};
  a.A = c.dense<float>(v[2], "A", at::kFloat, {D, N});
  a.skip = c.dense<float>(v[5], "D", at::kFloat, {D});
  if (v[6] != Py_None) {
    const Tensor& z = tensor(v[6], "z");
    c.activation(z, "z", x.sizes(), prompt);
    a.z = z.data_ptr(), a.z_batch = z.stride(0), a.z_channel = z.stride(1);
  }
  a.dt_bias = c.dense<float>(v[7], "dt_bias", at::kFloat, {D});
  a.flags = PyObject_IsTrue(v[8]) ? SC_SEQ_SOFTPLUS : 0;
  a.lengths = c.dense<int32_t>(v[9], "lengths", at::kInt, {B});
  a.slots = c.dense<int32_t>(v[10], "slots", at::kInt, {B});
  const void* first;
  void* last;
  a.num_slots = c.pools(v[11], v[12], v[10], at::kFloat, B, D, N, &first, &last, &a.initial_stride, &a.final_stride);
  a.initial_state = static_cast<const float*>(first), a.final_state = static_cast<float*>(last);
  const Tensor out = c.output(v[13], x.sizes(), prompt);
  a.x = x.data_ptr(), a.dt = dt.data_ptr(), a.b = Bm.data_ptr(), a.c = Cm.data_ptr(), a.out = out.data_ptr();
  a.x_batch = x.stride(0), a.x_channel = x.stride(1), a.dt_batch = dt.stride(0), a.dt_channel = dt.stride(1);
  a.out_batch = out.stride(0), a.out_channel = out.stride(1);
  a.b_batch = Bm.stride(0), a.b_group = Bm.stride(1), a.b_state = Bm.stride(2);
  a.c_batch = Cm.stride(0), a.c_group = Cm.stride(1), a.c_state = Cm.stride(2);
  a.dtype = c.dtype(), a.B = c.size(B), a.D = c.size(D), a.L = c.size(L), a.N = c.size(N), a.G = c.size(G);
  int64_t need = 0;
  if (const sc_status s = sparseconv_selective_scan_workspace(&a, &need)) return PyLong_FromLong(s);
  const Tensor ws = c.workspace(v[14], need);
  if (need) a.workspace = ws.data_ptr(), a.workspace_bytes = (int64_t)ws.nbytes();
  return answer(sparseconv_selective_scan(&a, PyLong_AsVoidPtr(v[16])), out, v[13], v[12]);
}

// x, down, up, index, scale, base, out, workspace, stream
PyObject* adapter_apply(PyObject* const* v, Py_ssize_t n) {
  check(n, 9);
  const Call c(tensor(v[0], "x"));
  const Tensor &x = c.x, &down = tensor(v[1], "down"), &up = tensor(v[2], "up");
  if (x.dim() != 3 || down.dim() != 3 || up.dim() != 3)
    refuse("x must be (B, C, L), down (adapters, R, C) and up (adapters, M, R)");
  const c10::DeviceGuard guard(c.device);
  const int64_t B = x.size(0), C = x.size(1), L = x.size(2), R = down.size(1), M = up.size(1), adapters = down.size(0);
  const int64_t shape[3] = {B, M, L};
  c.activation(x, "x", x.sizes(), true);
  sc_adapter a{};
  a.down = c.dense<void>(v[1], "down", c.type, {adapters, R, C});
  a.up = c.dense<void>(v[2], "up", c.type, {adapters, M, R});
  a.index = c.dense<int32_t>(v[3], "index", at::kInt, {B});
  a.scale = c.dense<float>(v[4], "scale", at::kFloat, {adapters});
  if (v[5] != Py_None) {
    const Tensor& base = tensor(v[5], "base");
    c.activation(base, "base", shape, true);
    a.base = base.data_ptr(), a.base_batch = base.stride(0), a.base_channel = base.stride(1);
  }
  const Tensor out = c.output(v[6], shape, true);
  a.x = x.data_ptr(), a.out = out.data_ptr();
  a.x_batch = x.stride(0), a.x_channel = x.stride(1), a.out_batch = out.stride(0), a.out_channel = out.stride(1);
  a.dtype = c.dtype(), a.B = c.size(B), a.C = c.size(C), a.M = c.size(M), a.L = c.size(L), a.R = c.size(R);
  a.adapters = c.size(adapters);
  int64_t need = 0;
  if (const sc_status s = sparseconv_adapter_workspace(&a, &need)) return PyLong_FromLong(s);
  const Tensor ws = c.workspace(v[7], need);
  if (need) a.workspace = ws.data_ptr(), a.workspace_bytes = (int64_t)ws.nbytes();
  return answer(sparseconv_adapter_apply(&a, PyLong_AsVoidPtr(v[8])), out, v[6], Py_None);
}

template <PyObject* (*F)(PyObject* const*, Py_ssize_t)>
PyObject* entry(PyObject*, PyObject* const* v, Py_ssize_t n) {
  try {
    PyObject* r = F(v, n);
    if (PyErr_Occurred()) {
      Py_XDECREF(r);
      return nullptr;
    }
    return r;
  } catch (const std::invalid_argument& e) {
    PyErr_SetString(PyExc_ValueError, e.what());
  } catch (const std::exception& e) {
    PyErr_SetString(PyExc_RuntimeError, e.what());
  }
  return nullptr;
}

template <PyObject* (*F)(PyObject* const*, Py_ssize_t)>
PyMethodDef method(const char* name) {
  return {name, reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(&entry<F>)), METH_FASTCALL, nullptr};
}

PyMethodDef methods[] = {method<causal_conv>("causal_conv"), method<selective_scan>("selective_scan"),
                         method<adapter_apply>("adapter_apply"), {nullptr, nullptr, 0, nullptr}};
PyModuleDef module = {PyModuleDef_HEAD_INIT, "_binding", nullptr, -1, methods, nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__binding() { return PyModule_Create(&module); }
