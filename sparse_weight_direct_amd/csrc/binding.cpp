// Tensor arguments of the sequence and attention operators: checks each torch tensor's type, device, shape and
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

#include <cmath>
#include <sstream>
#include <stdexcept>
#include <vector>

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

double number(PyObject* o) {
  const double v = PyFloat_AsDouble(o);
  if (v == -1.0 && PyErr_Occurred()) {
    PyErr_Clear();
    refuse("scale, cap and eps must be numbers");
  }
  return v;
}

// Both halves of a cache: k_pages (pages, G, P, D) and v_pages (pages, G, D, P), each page contiguous.
struct Pages {
  const Tensor &k, &v;
  int64_t pages, G, P, D;

  Pages(const Call& c, PyObject* ko, PyObject* vo, at::ScalarType type) : k(tensor(ko, "k_pages")), v(tensor(vo, "v_pages")) {
    if (k.dim() != 4 || v.dim() != 4) refuse("k_pages must be (pages, heads, positions, dims) and v_pages (pages, heads, dims, positions)");
    pages = k.size(0), G = k.size(1), P = k.size(2), D = k.size(3);
    check(c, k, "k_pages", type, {pages, G, P, D});
    check(c, v, "v_pages", type, {pages, G, D, P});
  }
  static void check(const Call& c, const Tensor& t, const char* name, at::ScalarType type, Shape shape) {
    int64_t per = 1;
    bool dense = true;
    for (int i = 3; i >= 1; i--) {
      if (shape[i] > 1 && t.stride(i) != per) dense = false;
      per *= shape[i];
    }
    if (!c.fits(t, type, shape) || !dense) refuse_tensor(t, name, type, shape, "each page contiguous");
  }
  int64_t stride(const Tensor& t) const { return pages > 1 ? t.stride(0) : G * P * D; }
};

// table (B, width): its rows may be part of a wider one.
const int32_t* table_of(const Call& c, PyObject* o, int64_t B, int64_t* width, int64_t* batch) {
  const Tensor& t = tensor(o, "table");
  *width = t.dim() == 2 ? t.size(1) : 0;
  const int64_t shape[2] = {B, *width};
  if (t.dim() != 2 || !c.fits(t, at::kInt, shape) || (*width > 1 && t.stride(1) != 1)) refuse_tensor(t, "table", at::kInt, shape, "its rows contiguous");
  *batch = B > 1 ? t.stride(0) : *width;
  return static_cast<const int32_t*>(t.data_ptr());
}

// q, k_pages, v_pages, table, past, lengths, prefix, slopes, scale, cap, window, out, workspace, axes of q, stream
PyObject* paged_attention(PyObject* const* v, Py_ssize_t n) {
  check(n, 15);
  const Call c(tensor(v[0], "q"));
  const Tensor& q = c.x;
  const int64_t axes = PyLong_AsLong(v[13]);
  const bool chunk = axes == 3;
  if (q.dim() != axes) refuse(chunk ? "q must be (B, H*D, L)" : "q must be (B, H*D)");
  const Pages pages(c, v[1], v[2], c.type);
  const c10::DeviceGuard guard(c.device);
  const int64_t B = q.size(0), D = pages.D, G = pages.G, L = chunk ? q.size(2) : 1;
  if (D == 0 || q.size(1) % D) refuse("q's channels are no multiple of the cache's dims");
  const int64_t H = q.size(1) / D;
  c.activation(q, "q", q.sizes(), chunk);
  sc_paged_attention a{};
  int64_t width;
  a.table = table_of(c, v[3], B, &width, &a.table_batch);
  a.past = c.dense<int32_t>(v[4], "past", at::kInt, {B});
  a.lengths = c.dense<int32_t>(v[5], "lengths", at::kInt, {B});
  a.prefix = c.dense<int32_t>(v[6], "prefix", at::kInt, {B});
  a.slopes = c.dense<float>(v[7], "slopes", at::kFloat, {H});
  a.scale = v[8] == Py_None ? (float)(1.0 / std::sqrt((double)D)) : (float)number(v[8]);
  a.cap = (float)number(v[9]);
  const long long window = PyLong_AsLongLong(v[10]);
  if (window == -1 && PyErr_Occurred()) return nullptr;
  if (window < 0) refuse("window must be 0 (none) or positive");
  Tensor out;
  if (v[11] == Py_None) {
    out = at::empty(q.sizes(), q.options());
  } else {
    out = tensor(v[11], "out");
    if (out.scalar_type() == at::kFloat && c.type != at::kFloat) {
      a.flags = SC_ATT_OUT_F32;
      if (!c.fits(out, at::kFloat, q.sizes()) || (chunk && L > 1 && out.stride(-1) != 1))
        refuse_tensor(out, "out", at::kFloat, q.sizes(), chunk ? "its last axis contiguous" : "strided");
    } else {
      c.activation(out, "out", q.sizes(), chunk);
    }
  }
  a.q = q.data_ptr(), a.out = out.data_ptr(), a.k_pages = pages.k.data_ptr(), a.v_pages = pages.v.data_ptr();
  a.q_batch = q.stride(0), a.q_channel = q.stride(1), a.out_batch = out.stride(0), a.out_channel = out.stride(1);
  a.k_page = pages.stride(pages.k), a.v_page = pages.stride(pages.v);
  a.dtype = c.dtype(), a.B = c.size(B), a.H = c.size(H), a.G = c.size(G), a.D = c.size(D), a.L = c.size(L), a.P = c.size(pages.P);
  a.width = c.size(width), a.pages = c.size(pages.pages);
  a.window = window > INT32_MAX ? 0 : (int32_t)window;  // positions end below 2^31
  int64_t need = 0;
  if (const sc_status s = sparseconv_paged_attention_workspace(&a, &need)) return PyLong_FromLong(s);
  const Tensor ws = c.workspace(v[12], need);
  if (need) a.workspace = ws.data_ptr(), a.workspace_bytes = (int64_t)ws.nbytes();
  return answer(sparseconv_paged_attention(&a, PyLong_AsVoidPtr(v[14])), out, v[11], Py_None);
}

// k, v, k_pages, v_pages, table, past, q, freqs, axes, positions, interleaved, lengths, out, axes of k, stream
PyObject* cache_append(PyObject* const* v, Py_ssize_t n) {
  check(n, 15);
  const Call c(tensor(v[0], "k"));
  const Tensor &k = c.x, &val = tensor(v[1], "v");
  const int64_t axes = PyLong_AsLong(v[13]);
  const bool chunk = axes == 3;
  if (k.dim() != axes) refuse(chunk ? "k must be (B, G*D, L)" : "k must be (B, G*D)");
  const at::ScalarType cache = tensor(v[2], "k_pages").scalar_type();
  if (cache != c.type && !(c.type == at::kFloat && (cache == at::kBFloat16 || cache == at::kHalf)))
    refuse("k_pages must be of k's type, or narrower than a float32 k");
  const Pages pages(c, v[2], v[3], cache);
  const c10::DeviceGuard guard(c.device);
  const int64_t B = k.size(0), G = pages.G, D = pages.D, L = chunk ? k.size(2) : 1;
  std::vector<int64_t> shape = {B, G * D};
  if (chunk) shape.push_back(L);
  c.activation(k, "k", shape, chunk);
  c.activation(val, "v", shape, chunk);
  sc_cache_append a{};
  int64_t width;
  a.table = table_of(c, v[4], B, &width, &a.table_batch);
  a.past = c.dense<int32_t>(v[5], "past", at::kInt, {B});
  a.lengths = c.dense<int32_t>(v[11], "lengths", at::kInt, {B});
  a.num_axes = 1;
  if (v[7] != Py_None) {
    const Tensor& freqs = tensor(v[7], "freqs");
    const int64_t pairs = freqs.dim() == 1 ? freqs.size(0) : 0;
    a.freqs = c.dense<double>(v[7], "freqs", at::kDouble, {pairs});
    a.axes = c.dense<int32_t>(v[8], "axes", at::kInt, {pairs});
    a.pairs = c.size(pairs);
    if (v[9] != Py_None) {
      const Tensor& p = tensor(v[9], "positions");
      const int64_t want[3] = {B, p.dim() == 3 ? p.size(1) : 0, L};
      if (p.dim() != 3 || want[1] < 1 || !c.fits(p, at::kInt, want) || (L > 1 && p.stride(2) != 1))
        refuse_tensor(p, "positions", at::kInt, want, "its last axis contiguous, (B, axes, L)");
      a.positions = static_cast<const int32_t*>(p.data_ptr());
      a.positions_batch = p.stride(0), a.positions_axis = p.stride(1), a.num_axes = c.size(want[1]);
    }
  } else if (v[8] != Py_None || v[9] != Py_None) {
    refuse("axes and positions need freqs");
  }
  a.flags = PyObject_IsTrue(v[10]) ? SC_ROT_INTERLEAVED : 0;
  Tensor out;
  if (v[6] != Py_None) {
    const Tensor& q = tensor(v[6], "q");
    if (q.dim() != axes || D == 0 || q.size(1) % D) refuse(chunk ? "q must be (B, H*D, L)" : "q must be (B, H*D)");
    std::vector<int64_t> qs = {B, q.size(1)};
    if (chunk) qs.push_back(L);
    c.activation(q, "q", qs, chunk);
    if (v[12] == Py_None) {
      out = at::empty(qs, k.options().dtype(cache));
    } else {
      out = tensor(v[12], "out");
      if (!c.fits(out, cache, qs) || (chunk && L > 1 && out.stride(-1) != 1))
        refuse_tensor(out, "out", cache, qs, chunk ? "its last axis contiguous" : "strided");
    }
    a.q = q.data_ptr(), a.q_out = out.data_ptr(), a.H = c.size(q.size(1) / D);
    a.q_batch = q.stride(0), a.q_channel = q.stride(1), a.q_out_batch = out.stride(0), a.q_out_channel = out.stride(1);
    if (q.size(1) == 0) refuse("q has no heads");
  } else if (v[12] != Py_None) {
    refuse("out without q");
  }
  a.k = k.data_ptr(), a.v = val.data_ptr(), a.k_pages = pages.k.data_ptr(), a.v_pages = pages.v.data_ptr();
  a.k_batch = k.stride(0), a.k_channel = k.stride(1), a.v_batch = val.stride(0), a.v_channel = val.stride(1);
  a.k_page = pages.stride(pages.k), a.v_page = pages.stride(pages.v);
  a.dtype = c.dtype(), a.cache_dtype = cache == at::kFloat ? SC_F32 : cache == at::kBFloat16 ? SC_BF16 : SC_F16;
  a.B = c.size(B), a.G = c.size(G), a.D = c.size(D), a.L = c.size(L), a.P = c.size(pages.P), a.width = c.size(width), a.pages = c.size(pages.pages);
  if (const sc_status s = sparseconv_cache_append(&a, PyLong_AsVoidPtr(v[14]))) return PyLong_FromLong(s);
  written(v[2]);
  written(v[3]);
  written(v[12]);
  if (v[6] == Py_None) Py_RETURN_NONE;
  return THPVariable_Wrap(out);
}

// pool, source, target, stream
PyObject* cache_copy(PyObject* const* v, Py_ssize_t n) {
  check(n, 4);
  const Tensor& pool = tensor(v[0], "pool");
  if (!pool.is_cuda() || pool.dim() < 3) refuse("pool must be a tensor (outer, pages, ...) on the GPU");
  int64_t per = 1;
  for (int64_t i = pool.dim() - 1; i >= 2; i--) {
    if (pool.size(i) > 1 && pool.stride(i) != per) refuse("each of pool's pages must be contiguous");
    per *= pool.size(i);
  }
  const c10::DeviceGuard guard(pool.device());
  sc_cache_copy a{};
  const Tensor* which[2] = {&tensor(v[1], "source"), &tensor(v[2], "target")};
  const int64_t count = which[0]->dim() == 1 ? which[0]->size(0) : 0, es = (int64_t)pool.element_size();
  for (int i = 0; i < 2; i++) {
    const Tensor& t = *which[i];
    if (t.scalar_type() != at::kInt || t.device() != pool.device() || t.dim() != 1 || t.size(0) != count || !t.is_contiguous())
      refuse_tensor(t, i ? "target" : "source", at::kInt, {count}, "contiguous");
  }
  a.pool = pool.data_ptr();
  a.source = static_cast<const int32_t*>(which[0]->data_ptr()), a.target = static_cast<const int32_t*>(which[1]->data_ptr());
  a.outer = Call::size(pool.size(0)), a.pages = Call::size(pool.size(1)), a.count = Call::size(count);
  a.page_bytes = per * es;
  a.page_stride = pool.size(1) > 1 ? pool.stride(1) * es : a.page_bytes;
  a.outer_stride = pool.size(0) > 1 ? pool.stride(0) * es : a.page_stride * pool.size(1);
  return answer(sparseconv_cache_copy(&a, PyLong_AsVoidPtr(v[3])), pool, v[0], Py_None);
}

// x, y, weight, bias, post_weight, post_bias, gate, scale, eps, center, sum, out, axes of x, stream
PyObject* residual_norm(PyObject* const* v, Py_ssize_t n) {
  check(n, 14);
  const Call c(tensor(v[0], "x"));
  const Tensor& x = c.x;
  const int64_t axes = PyLong_AsLong(v[12]);
  const bool chunk = axes == 3;
  if (x.dim() != axes) refuse(chunk ? "x must be (B, C, L)" : "x must be (B, C)");
  const c10::DeviceGuard guard(c.device);
  const int64_t B = x.size(0), C = x.size(1), L = chunk ? x.size(2) : 1;
  c.activation(x, "x", x.sizes(), chunk);
  sc_residual_norm a{};
  a.weight = c.dense<float>(v[2], "weight", at::kFloat, {C});
  a.bias = c.dense<float>(v[3], "bias", at::kFloat, {C});
  a.post_weight = c.dense<float>(v[4], "post_weight", at::kFloat, {C});
  a.post_bias = c.dense<float>(v[5], "post_bias", at::kFloat, {C});
  if (v[1] != Py_None) {
    const Tensor& y = tensor(v[1], "y");
    c.activation(y, "y", x.sizes(), chunk);
    a.y = y.data_ptr(), a.y_batch = y.stride(0), a.y_channel = y.stride(1);
  }
  if (v[6] != Py_None) {
    const Tensor& g = tensor(v[6], "gate");
    const int64_t two[2] = {B, C};
    if (g.dim() == 2) {
      c.activation(g, "gate", two, false);
    } else {
      c.activation(g, "gate", x.sizes(), chunk);
      a.gate_position = L > 1 ? 1 : 0;
    }
    a.gate = g.data_ptr(), a.gate_batch = g.stride(0), a.gate_channel = g.stride(1);
  }
  a.scale = (float)number(v[7]), a.eps = (float)number(v[8]);
  a.flags = PyObject_IsTrue(v[9]) ? SC_NORM_CENTER : 0;
  Tensor sum, out;
  if (v[1] != Py_None || v[10] != Py_None) {  // without y the sum is x
    sum = c.output(v[10], x.sizes(), chunk);
    a.sum = sum.data_ptr(), a.sum_batch = sum.stride(0), a.sum_channel = sum.stride(1);
  }
  if (a.weight || v[11] != Py_None) {
    if (v[11] == Py_None) {
      out = at::empty(x.sizes(), x.options());
    } else {
      out = tensor(v[11], "out");
      c.activation(out, "out", x.sizes(), chunk);
    }
    a.out = out.data_ptr(), a.out_batch = out.stride(0), a.out_channel = out.stride(1);
  }
  a.x = x.data_ptr(), a.x_batch = x.stride(0), a.x_channel = x.stride(1);
  a.dtype = c.dtype(), a.B = c.size(B), a.C = c.size(C), a.L = c.size(L);
  if (const sc_status s = sparseconv_residual_norm(&a, PyLong_AsVoidPtr(v[13]))) return PyLong_FromLong(s);
  written(v[10]);
  written(v[11]);
  PyObject* r = PyTuple_New(2);
  if (!r) return nullptr;
  auto item = [](const Tensor& t) {
    if (t.defined()) return THPVariable_Wrap(t);
    Py_INCREF(Py_None);
    return Py_None;
  };
  PyTuple_SET_ITEM(r, 0, sum.defined() ? item(sum) : item(x));
  PyTuple_SET_ITEM(r, 1, item(out));
  return r;
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
                         method<adapter_apply>("adapter_apply"), method<paged_attention>("paged_attention"),
                         method<cache_append>("cache_append"), method<cache_copy>("cache_copy"),
                         method<residual_norm>("residual_norm"), {nullptr, nullptr, 0, nullptr}};
PyModuleDef module = {PyModuleDef_HEAD_INIT, "_binding", nullptr, -1, methods, nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__binding() { return PyModule_Create(&module); }
