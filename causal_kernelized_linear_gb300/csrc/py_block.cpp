// CPython entry points of the block operators: argument checks,
// la_rows views of the tensors, output allocation, and the call into the C
// ABI (include/linattn.h).  No arithmetic.
//
// A decoding step's kernels take 3 to 10 µs, and marshalling the six to eight
// tensors of a call through ctypes took 13 µs; from here the whole call takes
// about 4 µs, 2.6 µs with a given output.  The functions are positional; _block.py names their arguments.
// The C ABI's functions are handed over by address (bind), so that the
// release and the LA_DEBUG library are used alike.
#include <Python.h>

#include <ATen/ATen.h>
#include <ATen/core/grad_mode.h>
#include <c10/cuda/CUDAGuard.h>
#include <c10/cuda/CUDAStream.h>
#include <torch/csrc/Exceptions.h>
#include <torch/csrc/autograd/function.h>
#include <torch/csrc/autograd/python_variable.h>

#include <array>
#include <cmath>
#include <optional>
#include <string>

#include "linattn.h"

namespace {

decltype(&la_linear) p_linear = nullptr;
decltype(&la_causal_conv) p_conv = nullptr;
decltype(&la_causal_conv_step) p_conv_step = nullptr;
decltype(&la_selective_scan) p_scan = nullptr;
decltype(&la_selective_step) p_step = nullptr;
decltype(&la_gated_delta) p_delta = nullptr;
decltype(&la_gated_delta_step) p_delta_step = nullptr;
decltype(&la_rms_norm) p_norm = nullptr;
decltype(&la_linear_e4m3) p_linear8 = nullptr;
PyObject* g_fail = nullptr;   // fail(function name, status): raises LinAttnError
PyObject* g_no_backward = nullptr;   // no_backward(function name, outputs, inputs): see _block.py

// Set when a check has raised a Python error; caught in every entry point.
struct Raised {};

template <typename... A>
[[noreturn]] void raise(PyObject* type, const char* format, A... args) {
  PyErr_Format(type, format, args...);
  throw Raised{};
}

const at::Tensor& tensor(PyObject* o, const char* name) {
  if (!THPVariable_Check(o)) raise(PyExc_TypeError, "%s must be a torch.Tensor", name);
  return THPVariable_Unpack(o);
}

const char* type_name(at::ScalarType t) {
  switch (t) {
    case at::kBFloat16: return "torch.bfloat16";
    case at::kFloat: return "torch.float32";
    case at::kFloat8_e4m3fn: return "torch.float8_e4m3fn";
    default: return "torch.int32";
  }
}

// The call's x: its type and device are what the other arguments must have.
struct Call {
  at::ScalarType type;
  la_dtype dtype;
  c10::Device device{c10::kCPU};
  std::optional<c10::cuda::CUDAGuard> on_device;
  std::optional<c10::cuda::CUDAStreamGuard> on_stream;
  la_stream stream = nullptr;

  explicit Call(const at::Tensor& x, const char* name = "x") : type(x.scalar_type()) {
    if (type != at::kBFloat16 && type != at::kFloat)
      raise(PyExc_ValueError, "%s: unsupported dtype (bf16 or fp32 wanted)", name);
    dtype = type == at::kBFloat16 ? LA_BF16 : LA_F32;
    device = x.device();
  }
  // bf16 results of 8-bit operands
  Call(const at::Tensor& x, at::ScalarType result) : type(result), dtype(LA_BF16), device(x.device()) {}

  void check(const at::Tensor& t, const char* name, at::ScalarType want) const {
    if (!t.is_cuda()) raise(PyExc_ValueError, "%s must be a CUDA tensor (no CPU path exists)", name);
    if (t.scalar_type() != want) raise(PyExc_ValueError, "%s must be %s", name, type_name(want));
    if (t.device() != device) raise(PyExc_ValueError, "%s must be on x's device", name);
    if (t.layout() != at::kStrided || t.is_conj() || t.is_neg())
      raise(PyExc_ValueError, "%s must be a plain strided tensor", name);
  }

  // The stream: None for the current one of x's device, a torch.cuda.Stream or
  // a handle.  With one given, allocations from here on belong to it, so that
  // they are not handed out again while work queued there still uses them.
  void use(PyObject* s) {
    on_device.emplace(device);
    if (s == Py_None) {
      stream = c10::cuda::getCurrentCUDAStream(device.index()).stream();
      return;
    }
    PyObject* h = PyObject_HasAttrString(s, "cuda_stream") ? PyObject_GetAttrString(s, "cuda_stream")
                                                           : PyNumber_Long(s);
    if (!h) throw Raised{};
    stream = static_cast<la_stream>(PyLong_AsVoidPtr(h));
    Py_DECREF(h);
    if (PyErr_Occurred()) throw Raised{};
    on_stream.emplace(c10::cuda::getStreamFromExternal(stream, device.index()));
  }

  at::Tensor empty(at::IntArrayRef shape, at::ScalarType t) const {
    return at::empty(shape, at::TensorOptions().dtype(t).device(device));
  }

  void last_axis(const at::Tensor& t, const char* name) const {
    if (t.stride(-1) != 1 && t.size(-1) != 1)
      raise(PyExc_ValueError, "%s's last axis must be contiguous", name);
  }

  // [B, n, d] (axes 3) or [B, d] (axes 2, n = 1).
  la_rows view(const at::Tensor& t, const char* name, int axes) const {
    if (t.dim() != axes)
      raise(PyExc_ValueError, "%s must have %d axes, not %d", name, axes, (int)t.dim());
    check(t, name, type);
    last_axis(t, name);
    if (axes == 3)
      return la_rows{t.data_ptr(), dtype, t.size(0), t.size(1), t.size(2), t.stride(0), t.stride(1)};
    return la_rows{t.data_ptr(), dtype, t.size(0), 1, t.size(1), t.stride(0), 0};
  }

  // [..., d] whose leading axes flatten to rows without a copy.
  la_rows matrix(const at::Tensor& t, const char* name) const { return matrix(t, name, type, dtype); }
  la_rows matrix(const at::Tensor& t, const char* name, at::ScalarType want, la_dtype as) const {
    const int64_t dim = t.dim();
    if (dim < 2) raise(PyExc_ValueError, "%s must have at least two axes", name);
    check(t, name, want);
    last_axis(t, name);
    int64_t rows = 1, stride = t.size(dim - 1);
    bool first = true;
    for (int64_t i = dim - 2; i >= 0; --i) {
      const int64_t size = t.size(i);
      if (size != 1 && t.numel() != 0) {
        if (first)
          stride = t.stride(i);
        else if (t.stride(i) != stride * rows)
          raise(PyExc_ValueError, "%s's leading axes must flatten without a copy", name);
        first = false;
      }
      rows *= size;
    }
    return la_rows{t.data_ptr(), as, 1, rows, t.size(dim - 1), 0, stride};
  }

  // [B, n, H, d] (axes 4) or [B, H, d] (axes 3, n = 1).
  la_heads heads(const at::Tensor& t, const char* name, int axes) const {
    if (t.dim() != axes)
      raise(PyExc_ValueError, "%s must have %d axes, not %d", name, axes, (int)t.dim());
    check(t, name, type);
    last_axis(t, name);
    if (axes == 4)
      return la_heads{t.data_ptr(), dtype, t.size(0), t.size(1), t.size(2), t.size(3),
                      t.stride(0), t.stride(1), t.stride(2)};
    return la_heads{t.data_ptr(), dtype, t.size(0), 1, t.size(1), t.size(2),
                    t.stride(0), 0, t.stride(1)};
  }

  // [B, n, H] (axes 3) or [B, H] of x's type or fp32.
  la_rows gate(const at::Tensor& t, const char* name, int axes) const {
    if (t.dim() != axes)
      raise(PyExc_ValueError, "%s must have %d axes, not %d", name, axes, (int)t.dim());
    const bool f32 = t.scalar_type() == at::kFloat;
    check(t, name, f32 ? at::kFloat : type);
    last_axis(t, name);
    const la_dtype as = f32 ? LA_F32 : dtype;
    if (axes == 3)
      return la_rows{t.data_ptr(), as, t.size(0), t.size(1), t.size(2), t.stride(0), t.stride(1)};
    return la_rows{t.data_ptr(), as, t.size(0), 1, t.size(1), t.stride(0), 0};
  }

  // A dense array of the given type and shape, or nullptr for None.
  void* dense(PyObject* o, const char* name, at::ScalarType want, at::IntArrayRef shape) const {
    if (o == Py_None) return nullptr;
    const at::Tensor& t = tensor(o, name);
    check(t, name, want);
    if (t.sizes() != shape) {
      std::string have = c10::str(t.sizes()), need = c10::str(shape);
      raise(PyExc_ValueError, "%s must have the shape %s, not %s", name, need.c_str(), have.c_str());
    }
    if (!t.is_contiguous()) raise(PyExc_ValueError, "%s must be contiguous", name);
    return t.data_ptr();
  }
};

la_activation activation(PyObject* o) {
  static const char* const names[] = {"none", "relu", "silu", "gelu", "softplus"};
  if (PyUnicode_Check(o))
    for (int i = 0; i < 5; ++i)
      if (PyUnicode_CompareWithASCIIString(o, names[i]) == 0) return (la_activation)i;
  raise(PyExc_ValueError, "activation must be one of none, relu, silu, gelu, softplus");
}

void done(const char* fn, la_status st) {
  if (st == LA_OK) return;
  PyObject* r = PyObject_CallFunction(g_fail, "si", fn, (int)st);
  Py_XDECREF(r);
  if (!PyErr_Occurred()) PyErr_Format(PyExc_RuntimeError, "%s failed (%d)", fn, (int)st);
  throw Raised{};
}

// Calls into the library without the interpreter's lock.
template <typename F>
la_status unlocked(F&& f) {
  la_status st;
  Py_BEGIN_ALLOW_THREADS
  st = f();
  Py_END_ALLOW_THREADS
  return st;
}

PyObject* wrap(PyObject* given, at::Tensor&& made) {
  if (given == Py_None) return THPVariable_Wrap(std::move(made));
  Py_INCREF(given);
  return given;
}

PyObject* pair(PyObject* first, at::Tensor&& second) {
  PyObject* s = THPVariable_Wrap(std::move(second));
  if (!s) {
    Py_DECREF(first);
    return nullptr;
  }
  PyObject* t = PyTuple_Pack(2, first, s);
  Py_DECREF(first);
  Py_DECREF(s);
  return t;
}

// Gradients: these functions have no backward.  Before the call, tensors that it
// would write in place (out, a step's state) may not be part of a graph that is
// being recorded; after it, what was written says so, and fresh outputs of inputs
// that require a gradient get a node that raises when it is asked for one.
struct Grads {
  PyObject* const* a;
  Py_ssize_t n;
  bool wanted = false;

  // the arguments of a call, the stream (the last of them) apart
  Grads(PyObject* const* args, Py_ssize_t count) : a(args), n(count - 1) {
    if (!at::GradMode::is_enabled()) return;
    for (Py_ssize_t i = 0; i < n && !wanted; ++i) wanted = requires_grad(a[i]);
  }
  static bool requires_grad(PyObject* o) {
    if (o == Py_None || PyBool_Check(o) || PyUnicode_Check(o)) return false;   // asking their class is slow
    return THPVariable_Check(o) && THPVariable_Unpack(o).requires_grad();
  }
  void out(PyObject* o) const {
    if (wanted && o != Py_None)
      raise(PyExc_ValueError, "no gradient passes through an out that is given, and an argument "
                              "requires one; call under torch.no_grad()");
  }
  // A state that one of these functions returned keeps its raising node.
  void in_place(PyObject* o, const char* name) const {
    if (!wanted || !requires_grad(o)) return;
    const auto& node = THPVariable_Unpack(o).grad_fn();
    if (!node || node->name() != "_NoBackwardBackward")
      raise(PyExc_ValueError, "%s requires a gradient and is updated in place; call under "
                              "torch.no_grad()", name);
  }
  static void written(PyObject* o) {
    if (o == Py_None) return;
    const at::Tensor& t = THPVariable_Unpack(o);
    if (!t.is_inference()) t.unsafeGetTensorImpl()->bump_version();
  }
  PyObject* result(const char* name, PyObject* r) const {
    if (!wanted || !r) return r;
    PyObject* inputs = PyList_New(0);
    for (Py_ssize_t i = 0; inputs && i < n; ++i)
      if (requires_grad(a[i]) && PyList_Append(inputs, a[i]) < 0) Py_CLEAR(inputs);
    PyObject* with = inputs ? PyObject_CallFunction(g_no_backward, "sOO", name, r, inputs) : nullptr;
    Py_XDECREF(inputs);
    Py_DECREF(r);
    return with;
  }
};

#define LA_PY_ENTRY(want)                                                        \
  HANDLE_TH_ERRORS                                                               \
  if (n != (want)) {                                                             \
    PyErr_Format(PyExc_TypeError, "%d arguments wanted, not %zd", (want), n);    \
    return nullptr;                                                              \
  }                                                                              \
  try {
#define LA_PY_END                                                                \
  }                                                                              \
  catch (const Raised&) {                                                        \
    return nullptr;                                                              \
  }                                                                              \
  END_HANDLE_TH_ERRORS

// x, weight, bias, activation, residual, out, stream
PyObject* linear(PyObject*, PyObject* const* a, Py_ssize_t n) {
  LA_PY_ENTRY(7)
  const at::Tensor& x = tensor(a[0], "x");
  Call call(x);
  const la_activation act = activation(a[3]);
  const la_rows xr = call.matrix(x, "x");
  const at::Tensor& w = tensor(a[1], "weight");
  if (w.dim() != 2) raise(PyExc_ValueError, "weight must be an [N, K] tensor");
  const la_rows wr = call.matrix(w, "weight");
  c10::SmallVector<int64_t, 5> shape(x.sizes().begin(), x.sizes().end());
  shape.back() = wr.n;
  const void* bias = call.dense(a[2], "bias", call.type, {wr.n});
  la_rows rr{};
  const bool has_res = a[4] != Py_None;
  if (has_res) {
    const at::Tensor& r = tensor(a[4], "residual");
    if (r.sizes() != at::IntArrayRef(shape))
      raise(PyExc_ValueError, "residual must have the shape %s", c10::str(at::IntArrayRef(shape)).c_str());
    rr = call.matrix(r, "residual");
  }
  const Grads grads(a, n);
  grads.out(a[5]);
  call.use(a[6]);
  at::Tensor made;
  if (a[5] == Py_None)
    made = call.empty(shape, call.type);
  else if (tensor(a[5], "out").sizes() != at::IntArrayRef(shape))
    raise(PyExc_ValueError, "out must have the shape %s", c10::str(at::IntArrayRef(shape)).c_str());
  la_rows out = call.matrix(a[5] == Py_None ? made : tensor(a[5], "out"), "out");
  done("la_linear", unlocked([&] {
         return p_linear(&xr, &wr, bias, act, has_res ? &rr : nullptr, &out, call.stream);
       }));
  grads.written(a[5]);
  return grads.result("linear", wrap(a[5], std::move(made)));
  LA_PY_END
}

// The [D, W] weight of a convolution.
const void* conv_weight(const Call& call, PyObject* o, int64_t D, int* width) {
  if (!THPVariable_Check(o) || THPVariable_Unpack(o).dim() != 2)
    raise(PyExc_ValueError, "weight must be a [D, W] tensor");
  const int64_t W = THPVariable_Unpack(o).size(1);
  *width = W > 1000 ? 1000 : (int)W;
  return call.dense(o, "weight", call.type, {D, W});
}

// x, weight, bias, activation, state, lengths, out, return_state, stream
PyObject* causal_conv(PyObject*, PyObject* const* a, Py_ssize_t n) {
  LA_PY_ENTRY(9)
  const at::Tensor& x = tensor(a[0], "x");
  Call call(x);
  const la_activation act = activation(a[3]);
  const la_rows xr = call.view(x, "x", 3);
  int W = 0;
  const void* w = conv_weight(call, a[1], xr.d, &W);
  const void* bias = call.dense(a[2], "bias", call.type, {xr.d});
  const std::array<int64_t, 3> state_shape{xr.B, W > 0 ? W - 1 : 0, xr.d};
  const void* state = call.dense(a[4], "state", call.type, state_shape);
  const auto* lens = static_cast<const int32_t*>(call.dense(a[5], "lengths", at::kInt, {xr.B}));
  const int want = PyObject_IsTrue(a[7]);
  if (want < 0) throw Raised{};
  const Grads grads(a, n);
  grads.out(a[6]);
  call.use(a[8]);
  at::Tensor made, after;
  if (a[6] == Py_None) made = call.empty(x.sizes(), call.type);
  la_rows out = call.view(a[6] == Py_None ? made : tensor(a[6], "out"), "out", 3);
  if (want) after = call.empty(state_shape, call.type);
  done("la_causal_conv", unlocked([&] {
         return p_conv(&xr, w, W, bias, act, state, lens, &out, want ? after.data_ptr() : nullptr,
                       call.stream);
       }));
  grads.written(a[6]);
  PyObject* r = wrap(a[6], std::move(made));
  return grads.result("causal_conv", want && r ? pair(r, std::move(after)) : r);
  LA_PY_END
}

// state, x, weight, bias, activation, out, stream
PyObject* causal_conv_step(PyObject*, PyObject* const* a, Py_ssize_t n) {
  LA_PY_ENTRY(7)
  const at::Tensor& x = tensor(a[1], "x");
  Call call(x);
  const la_activation act = activation(a[4]);
  const la_rows xr = call.view(x, "x", 2);
  int W = 0;
  const void* w = conv_weight(call, a[2], xr.d, &W);
  const void* bias = call.dense(a[3], "bias", call.type, {xr.d});
  tensor(a[0], "state");
  void* state = call.dense(a[0], "state", call.type, {xr.B, W > 0 ? W - 1 : 0, xr.d});
  const Grads grads(a, n);
  grads.out(a[5]);
  grads.in_place(a[0], "state");
  call.use(a[6]);
  at::Tensor made;
  if (a[5] == Py_None) made = call.empty(x.sizes(), call.type);
  la_rows out = call.view(a[5] == Py_None ? made : tensor(a[5], "out"), "out", 2);
  done("la_causal_conv_step",
       unlocked([&] { return p_conv_step(state, &xr, w, W, bias, act, &out, call.stream); }));
  grads.written(a[0]);
  grads.written(a[5]);
  return grads.result("causal_conv_step", wrap(a[5], std::move(made)));
  LA_PY_END
}

// What the scan and its step share: x, dt, a, b, c, skip, gate, dt_bias, softplus.
struct ScanCall {
  la_rows x, dt, b, c, gate;
  const float *a, *skip, *bias;
  int64_t S;
  bool gated;
  int softplus;

  ScanCall(const Call& call, PyObject* const* p, int axes) {
    x = call.view(tensor(p[0], "x"), "x", axes);
    dt = call.view(tensor(p[1], "dt"), "dt", axes);
    if (!THPVariable_Check(p[2]) || THPVariable_Unpack(p[2]).dim() != 2)
      raise(PyExc_ValueError, "a must be a [D, S] tensor");
    S = THPVariable_Unpack(p[2]).size(1);
    if (S > (1 << 20)) raise(PyExc_ValueError, "a has too many states");
    a = static_cast<const float*>(call.dense(p[2], "a", at::kFloat, {x.d, S}));
    b = call.view(tensor(p[3], "b"), "b", axes);
    c = call.view(tensor(p[4], "c"), "c", axes);
    skip = static_cast<const float*>(call.dense(p[5], "skip", at::kFloat, {x.d}));
    gated = p[6] != Py_None;
    if (gated) gate = call.view(tensor(p[6], "gate"), "gate", axes);
    bias = static_cast<const float*>(call.dense(p[7], "dt_bias", at::kFloat, {x.d}));
    softplus = PyObject_IsTrue(p[8]);
    if (softplus < 0) throw Raised{};
  }
};

// x, dt, a, b, c, skip, gate, dt_bias, softplus, state, lengths, out, return_state, stream
PyObject* selective_scan(PyObject*, PyObject* const* a, Py_ssize_t n) {
  LA_PY_ENTRY(14)
  const at::Tensor& x = tensor(a[0], "x");
  Call call(x);
  const ScanCall s(call, a, 3);
  const std::array<int64_t, 3> state_shape{s.x.B, s.x.d, s.S};
  const auto* state = static_cast<const float*>(call.dense(a[9], "state", at::kFloat, state_shape));
  const auto* lens = static_cast<const int32_t*>(call.dense(a[10], "lengths", at::kInt, {s.x.B}));
  const int want = PyObject_IsTrue(a[12]);
  if (want < 0) throw Raised{};
  const Grads grads(a, n);
  grads.out(a[11]);
  call.use(a[13]);
  at::Tensor made, after;
  if (a[11] == Py_None) made = call.empty(x.sizes(), call.type);
  la_rows out = call.view(a[11] == Py_None ? made : tensor(a[11], "out"), "out", 3);
  if (want) after = call.empty(state_shape, at::kFloat);
  done("la_selective_scan", unlocked([&] {
         return p_scan(&s.x, &s.dt, s.a, (int)s.S, &s.b, &s.c, s.skip, s.gated ? &s.gate : nullptr,
                       s.bias, s.softplus, state, lens, &out,
                       want ? static_cast<float*>(after.data_ptr()) : nullptr, call.stream);
       }));
  grads.written(a[11]);
  PyObject* r = wrap(a[11], std::move(made));
  return grads.result("selective_scan", want && r ? pair(r, std::move(after)) : r);
  LA_PY_END
}

// state, x, dt, a, b, c, skip, gate, dt_bias, softplus, out, stream
PyObject* selective_step(PyObject*, PyObject* const* a, Py_ssize_t n) {
  LA_PY_ENTRY(12)
  const at::Tensor& x = tensor(a[1], "x");
  Call call(x);
  const ScanCall s(call, a + 1, 2);
  tensor(a[0], "state");
  auto* state = static_cast<float*>(call.dense(a[0], "state", at::kFloat, {s.x.B, s.x.d, s.S}));
  const Grads grads(a, n);
  grads.out(a[10]);
  grads.in_place(a[0], "state");
  call.use(a[11]);
  at::Tensor made;
  if (a[10] == Py_None) made = call.empty(x.sizes(), call.type);
  la_rows out = call.view(a[10] == Py_None ? made : tensor(a[10], "out"), "out", 2);
  done("la_selective_step", unlocked([&] {
         return p_step(state, &s.x, &s.dt, s.a, (int)s.S, &s.b, &s.c, s.skip,
                       s.gated ? &s.gate : nullptr, s.bias, s.softplus, &out, call.stream);
       }));
  grads.written(a[0]);
  grads.written(a[10]);
  return grads.result("selective_step", wrap(a[10], std::move(made)));
  LA_PY_END
}

float number(PyObject* o, const char* name) {
  const double v = PyFloat_AsDouble(o);
  if (v == -1.0 && PyErr_Occurred()) {
    PyErr_Clear();
    raise(PyExc_TypeError, "%s must be a number", name);
  }
  return (float)v;
}

int truth(PyObject* o) {
  const int v = PyObject_IsTrue(o);
  if (v < 0) throw Raised{};
  return v;
}

// What the rule and its step share: q, k, v, dt, a, beta, dt_bias, softplus, sigmoid,
// normalize, scale.
struct DeltaCall {
  la_heads q, k, v;
  la_rows dt, beta;
  const float *a, *bias;
  int softplus, sigmoid, normalize;
  float scale;

  DeltaCall(const Call& call, PyObject* const* p, int axes) {
    q = call.heads(tensor(p[0], "q"), "q", axes);
    k = call.heads(tensor(p[1], "k"), "k", axes);
    v = call.heads(tensor(p[2], "v"), "v", axes);
    dt = call.gate(tensor(p[3], "dt"), "dt", axes - 1);
    tensor(p[4], "a");
    a = static_cast<const float*>(call.dense(p[4], "a", at::kFloat, {v.H}));
    beta = call.gate(tensor(p[5], "beta"), "beta", axes - 1);
    bias = static_cast<const float*>(call.dense(p[6], "dt_bias", at::kFloat, {v.H}));
    softplus = truth(p[7]);
    sigmoid = truth(p[8]);
    normalize = truth(p[9]);
    scale = p[10] == Py_None ? 1.f / sqrtf((float)q.d) : number(p[10], "scale");
  }
  std::array<int64_t, 4> state_shape() const { return {v.B, v.H, q.d, v.d}; }
};

// q, k, v, dt, a, beta, dt_bias, softplus, sigmoid, normalize, scale, state, lengths, out,
// return_state, stream
PyObject* gated_delta(PyObject*, PyObject* const* a, Py_ssize_t n) {
  LA_PY_ENTRY(16)
  Call call(tensor(a[0], "q"), "q");
  const DeltaCall s(call, a, 4);
  const auto state_shape = s.state_shape();
  const auto* state = static_cast<const float*>(call.dense(a[11], "state", at::kFloat, state_shape));
  const auto* lens = static_cast<const int32_t*>(call.dense(a[12], "lengths", at::kInt, {s.v.B}));
  const int want = truth(a[14]);
  const Grads grads(a, n);
  grads.out(a[13]);
  call.use(a[15]);
  at::Tensor made, after;
  if (a[13] == Py_None) made = call.empty({s.v.B, s.v.n, s.v.H, s.v.d}, call.type);
  la_heads out = call.heads(a[13] == Py_None ? made : tensor(a[13], "out"), "out", 4);
  if (want) after = call.empty(state_shape, at::kFloat);
  done("la_gated_delta", unlocked([&] {
         return p_delta(&s.q, &s.k, &s.v, &s.dt, s.a, &s.beta, s.bias, s.softplus, s.sigmoid,
                        s.normalize, s.scale, state, lens, &out,
                        want ? static_cast<float*>(after.data_ptr()) : nullptr, call.stream);
       }));
  grads.written(a[13]);
  PyObject* r = wrap(a[13], std::move(made));
  return grads.result("gated_delta", want && r ? pair(r, std::move(after)) : r);
  LA_PY_END
}

// state, q, k, v, dt, a, beta, dt_bias, softplus, sigmoid, normalize, scale, out, stream
PyObject* gated_delta_step(PyObject*, PyObject* const* a, Py_ssize_t n) {
  LA_PY_ENTRY(14)
  Call call(tensor(a[1], "q"), "q");
  const DeltaCall s(call, a + 1, 3);
  tensor(a[0], "state");
  auto* state = static_cast<float*>(call.dense(a[0], "state", at::kFloat, s.state_shape()));
  const Grads grads(a, n);
  grads.out(a[12]);
  grads.in_place(a[0], "state");
  call.use(a[13]);
  at::Tensor made;
  if (a[12] == Py_None) made = call.empty({s.v.B, s.v.H, s.v.d}, call.type);
  la_heads out = call.heads(a[12] == Py_None ? made : tensor(a[12], "out"), "out", 3);
  done("la_gated_delta_step", unlocked([&] {
         return p_delta_step(state, &s.q, &s.k, &s.v, &s.dt, s.a, &s.beta, s.bias, s.softplus,
                             s.sigmoid, s.normalize, s.scale, &out, call.stream);
       }));
  grads.written(a[0]);
  grads.written(a[12]);
  return grads.result("gated_delta_step", wrap(a[12], std::move(made)));
  LA_PY_END
}

// x, weight, group, eps, gate, residual, quantize, out, sum_out, stream
PyObject* rms_norm(PyObject*, PyObject* const* a, Py_ssize_t n) {
  LA_PY_ENTRY(10)
  const at::Tensor& x = tensor(a[0], "x");
  Call call(x);
  const la_rows xr = call.matrix(x, "x");
  int64_t group = xr.d;
  const void* weight = nullptr;
  if (a[2] != Py_None) {
    group = PyLong_AsLongLong(a[2]);
    if (PyErr_Occurred()) throw Raised{};
  }
  if (a[1] != Py_None) {
    const at::Tensor& w = tensor(a[1], "weight");
    if (w.dim() != 1) raise(PyExc_ValueError, "weight must have one axis");
    if (a[2] == Py_None) group = w.size(0);
    weight = call.dense(a[1], "weight", call.type, {group});
  }
  if (group < 1 || xr.d % group)
    raise(PyExc_ValueError, "x's last axis must be a multiple of the norm's group (%lld)", (long long)group);
  const float eps = number(a[3], "eps");
  la_rows rows[4];   // gate, residual, sum, out
  auto like_x = [&](PyObject* o, const char* name, la_rows* to) {
    if (o == Py_None) return false;
    const at::Tensor& t = tensor(o, name);
    if (t.sizes() != x.sizes())
      raise(PyExc_ValueError, "%s must have the shape %s", name, c10::str(x.sizes()).c_str());
    *to = call.matrix(t, name);
    return true;
  };
  const bool gated = like_x(a[4], "gate", rows), added = like_x(a[5], "residual", rows + 1);
  const bool quantize = truth(a[6]);
  const Grads grads(a, n);
  grads.out(a[7]);
  grads.out(a[8]);
  if (a[8] != Py_None && !added) raise(PyExc_ValueError, "sum_out needs a residual");
  call.use(a[9]);
  at::Tensor made, scale, sum;
  if (a[7] == Py_None) made = call.empty(x.sizes(), quantize ? at::kFloat8_e4m3fn : call.type);
  const at::Tensor& out = a[7] == Py_None ? made : tensor(a[7], "out");
  if (out.sizes() != x.sizes())
    raise(PyExc_ValueError, "out must have the shape %s", c10::str(x.sizes()).c_str());
  rows[3] = quantize ? call.matrix(out, "out", at::kFloat8_e4m3fn, LA_E4M3) : call.matrix(out, "out");
  if (quantize) scale = call.empty(x.sizes().slice(0, x.dim() - 1), at::kFloat);
  if (added && !like_x(a[8], "sum_out", rows + 2)) {
    sum = call.empty(x.sizes(), call.type);
    rows[2] = call.matrix(sum, "sum_out");
  }
  done("la_rms_norm", unlocked([&] {
         return p_norm(&xr, weight, group, eps, added ? rows + 1 : nullptr, gated ? rows : nullptr,
                       rows + 3, quantize ? static_cast<float*>(scale.data_ptr()) : nullptr,
                       added ? rows + 2 : nullptr, call.stream);
       }));
  grads.written(a[7]);
  grads.written(a[8]);
  PyObject* r[3] = {wrap(a[7], std::move(made)), nullptr, nullptr};
  int count = 1;
  if (quantize) r[count++] = THPVariable_Wrap(std::move(scale));
  if (added) r[count++] = wrap(a[8], std::move(sum));
  bool ok = true;
  for (int i = 0; i < count; ++i) ok = ok && r[i];
  PyObject* all = !ok ? nullptr : count == 1 ? Py_NewRef(r[0]) : PyTuple_New(count);
  for (int i = 0; i < count; ++i) {
    if (all && count > 1)
      PyTuple_SET_ITEM(all, i, r[i]);
    else
      Py_XDECREF(r[i]);
  }
  return grads.result("rms_norm", all);
  LA_PY_END
}

// x, x_scale, weight, weight_scale, bias, activation, residual, out, stream
PyObject* linear_e4m3(PyObject*, PyObject* const* a, Py_ssize_t n) {
  LA_PY_ENTRY(9)
  const at::Tensor& x = tensor(a[0], "x");
  Call call(x, at::kBFloat16);
  const la_activation act = activation(a[5]);
  const la_rows xr = call.matrix(x, "x", at::kFloat8_e4m3fn, LA_E4M3);
  tensor(a[1], "x_scale");
  const auto* xs = static_cast<const float*>(
      call.dense(a[1], "x_scale", at::kFloat, x.sizes().slice(0, x.dim() - 1)));
  const at::Tensor& w = tensor(a[2], "weight");
  if (w.dim() != 2) raise(PyExc_ValueError, "weight must be an [N, K] tensor");
  const la_rows wr = call.matrix(w, "weight", at::kFloat8_e4m3fn, LA_E4M3);
  tensor(a[3], "weight_scale");
  const auto* ws = static_cast<const float*>(call.dense(a[3], "weight_scale", at::kFloat, {wr.n}));
  c10::SmallVector<int64_t, 5> shape(x.sizes().begin(), x.sizes().end());
  shape.back() = wr.n;
  const void* bias = call.dense(a[4], "bias", call.type, {wr.n});
  la_rows rr{};
  const bool has_res = a[6] != Py_None;
  if (has_res) {
    const at::Tensor& r = tensor(a[6], "residual");
    if (r.sizes() != at::IntArrayRef(shape))
      raise(PyExc_ValueError, "residual must have the shape %s", c10::str(at::IntArrayRef(shape)).c_str());
    rr = call.matrix(r, "residual");
  }
  const Grads grads(a, n);
  grads.out(a[7]);
  call.use(a[8]);
  at::Tensor made;
  if (a[7] == Py_None)
    made = call.empty(shape, call.type);
  else if (tensor(a[7], "out").sizes() != at::IntArrayRef(shape))
    raise(PyExc_ValueError, "out must have the shape %s", c10::str(at::IntArrayRef(shape)).c_str());
  la_rows out = call.matrix(a[7] == Py_None ? made : tensor(a[7], "out"), "out");
  done("la_linear_e4m3", unlocked([&] {
         return p_linear8(&xr, xs, &wr, ws, bias, act, has_res ? &rr : nullptr, &out, call.stream);
       }));
  grads.written(a[7]);
  return grads.result("linear_e4m3", wrap(a[7], std::move(made)));
  LA_PY_END
}

// bind(fail, no_backward, addresses of the nine C functions in the order above)
PyObject* bind(PyObject*, PyObject* const* a, Py_ssize_t n) {
  if (n != 11) {
    PyErr_SetString(PyExc_TypeError, "bind(fail, no_backward, nine addresses)");
    return nullptr;
  }
  void* p[9];
  for (int i = 0; i < 9; ++i) {
    p[i] = PyLong_AsVoidPtr(a[i + 2]);
    if (PyErr_Occurred()) return nullptr;
  }
  p_linear = reinterpret_cast<decltype(p_linear)>(p[0]);
  p_conv = reinterpret_cast<decltype(p_conv)>(p[1]);
  p_conv_step = reinterpret_cast<decltype(p_conv_step)>(p[2]);
  p_scan = reinterpret_cast<decltype(p_scan)>(p[3]);
  p_step = reinterpret_cast<decltype(p_step)>(p[4]);
  p_delta = reinterpret_cast<decltype(p_delta)>(p[5]);
  p_delta_step = reinterpret_cast<decltype(p_delta_step)>(p[6]);
  p_norm = reinterpret_cast<decltype(p_norm)>(p[7]);
  p_linear8 = reinterpret_cast<decltype(p_linear8)>(p[8]);
  Py_INCREF(a[0]);
  Py_XSETREF(g_fail, a[0]);
  Py_INCREF(a[1]);
  Py_XSETREF(g_no_backward, a[1]);
  Py_RETURN_NONE;
}

#define LA_PY_METHOD(f) {#f, reinterpret_cast<PyCFunction>(reinterpret_cast<void*>(f)), METH_FASTCALL, nullptr}
PyMethodDef g_methods[] = {LA_PY_METHOD(bind),           LA_PY_METHOD(linear),
                           LA_PY_METHOD(causal_conv),    LA_PY_METHOD(causal_conv_step),
                           LA_PY_METHOD(selective_scan), LA_PY_METHOD(selective_step),
                           LA_PY_METHOD(gated_delta),    LA_PY_METHOD(gated_delta_step),
                           LA_PY_METHOD(rms_norm),       LA_PY_METHOD(linear_e4m3),
                           {nullptr, nullptr, 0, nullptr}};
PyModuleDef g_module = {PyModuleDef_HEAD_INIT, "la_block", nullptr, -1, g_methods,
                        nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit_la_block() { return PyModule_Create(&g_module); }
