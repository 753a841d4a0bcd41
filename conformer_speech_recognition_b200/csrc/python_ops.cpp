// Python marshalling of the streaming-block operators (module _ops, used by gam.py).
//
// A call of one of these operators can take a few microseconds on the GPU, and a
// frame's step makes many of them; checking a dozen tensors attribute by attribute
// in Python took 10 to 15 microseconds a call, most of a step.  These functions do
// the same checks on the tensors themselves, allocate missing outputs and call the
// C entry point.  They compute nothing.  The entry points' addresses and the
// exception class come from gam.py, which owns the library.
#include <c10/cuda/CUDAGuard.h>
#include <c10/cuda/CUDAStream.h>
#include <torch/csrc/autograd/python_variable.h>

#include <ATen/core/grad_mode.h>
#include <c10/core/AutogradState.h>
#include <ATen/ops/empty.h>

#include <initializer_list>
#include <optional>
#include <string>

#include "../../include/gam.h"

namespace {

struct Entry {
  decltype(&gam_last_error) last_error;
  decltype(&gam_quant_linear) quant_linear;
  decltype(&gam_short_conv) short_conv;
  decltype(&gam_selective_scan) selective_scan;
  decltype(&gam_residual_norm) residual_norm;
} g_entry;
PyObject* g_error = nullptr;  // gam.GamError(status, message)

struct Refused {
  int status;
  std::string message;
};

[[noreturn]] void refuse(int status, const std::string& message) { throw Refused{status, message}; }

const at::Tensor& tensor(PyObject* o, const char* name) {
  if (!THPVariable_Check(o) || !THPVariable_Unpack(o).is_cuda())
    refuse(GAM_ERR_INVALID_ARG, std::string(name) + " must be a CUDA tensor");
  return THPVariable_Unpack(o);
}

int dtype_code(const at::Tensor& t, const char* name) {
  switch (t.scalar_type()) {
    case at::kFloat: return GAM_DTYPE_F32;
    case at::kHalf: return GAM_DTYPE_F16;
    case at::kBFloat16: return GAM_DTYPE_BF16;
    default: refuse(GAM_ERR_INVALID_ARG, std::string(name) + " must be float32, float16 or bfloat16");
  }
}

// The device and stream of a call, taken from its first tensor.  With a stream given,
// outputs allocated here belong to it.
struct Call {
  c10::DeviceIndex dev;
  c10::cuda::OptionalCUDAGuard device;
  std::optional<c10::cuda::CUDAStreamGuard> own;
  void* raw;

  Call(const at::Tensor& t, PyObject* stream) : dev(t.get_device()) {
    device.set_index(dev);
    if (stream != Py_None) {
      raw = PyLong_AsVoidPtr(stream);
      if (PyErr_Occurred()) throw PyErr_Occurred();
      own.emplace(c10::cuda::getStreamFromExternal(static_cast<cudaStream_t>(raw), dev));
    } else {
      raw = c10::cuda::getCurrentCUDAStream(dev).stream();
    }
  }

  // A tensor's gradient, which these operators do not give, is not dropped in silence.
  static void no_gradient(const at::Tensor& t, const char* name) {
    // a forward-mode tangent does not make a tensor require a gradient, and no_grad does not switch it off
    if (c10::AutogradState::get_tls_state().get_fw_grad_mode() && t._fw_grad(0).defined())
      refuse(GAM_ERR_INVALID_ARG, std::string(name) + " carries a forward-mode gradient, which this operator does not "
                                                      "pass on: call it with detached tensors");
    if (t.requires_grad() && at::GradMode::is_enabled())
      refuse(GAM_ERR_INVALID_ARG, std::string(name) + " requires a gradient, which this operator does not give: call it "
                                                      "under torch.no_grad() or with detached tensors");
  }

  // A number, or a tensor that holds one.
  static float number(PyObject* o, const char* name) {
    if (THPVariable_Check(o)) no_gradient(THPVariable_Unpack(o), name);
    const double v = PyFloat_AsDouble(o);
    if (PyErr_Occurred()) throw PyErr_Occurred();
    return (float)v;
  }

  // Address of a tensor of this shape and type on the call's device; its last dimension
  // is contiguous (`packed`: all of it).  None is 0 where `optional`.
  void* arg(PyObject* o, const char* name, at::IntArrayRef shape, at::ScalarType type, bool packed,
            bool optional = false) const {
    if (optional && o == Py_None) return nullptr;
    const at::Tensor& t = tensor(o, name);
    if (t.scalar_type() != type)
      refuse(GAM_ERR_INVALID_ARG, std::string(name) + " must be " + c10::toString(type) + ", got " +
                                      c10::toString(t.scalar_type()));
    if (t.get_device() != dev)
      refuse(GAM_ERR_INVALID_ARG, std::string(name) + " is on cuda:" + std::to_string(t.get_device()) +
                                      ", expected cuda:" + std::to_string(dev));
    if (t.sizes() != shape) {
      std::string want;
      for (int64_t v : shape) want += (want.empty() ? "" : ", ") + std::to_string(v);
      refuse(GAM_ERR_INVALID_ARG, std::string(name) + " must have shape [" + want + "]");
    }
    no_gradient(t, name);
    if (packed ? !t.is_contiguous() : shape.back() > 1 && t.stride(-1) != 1)
      refuse(GAM_ERR_INVALID_ARG, packed ? std::string(name) + " must be contiguous"
                                         : std::string("the last dimension of ") + name + " must be contiguous");
    if (t.is_neg())  // its memory holds the negated values
      refuse(GAM_ERR_INVALID_ARG, std::string(name) + " is a lazily negated view: call it with resolve_neg()");
    return t.data_ptr();
  }

  // An output: the one given, or a new one.
  PyObject* out(PyObject* o, at::IntArrayRef shape, at::ScalarType type) const {
    if (o != Py_None) return Py_NewRef(o);
    return THPVariable_Wrap(at::empty(shape, at::TensorOptions().dtype(type).device(c10::kCUDA, dev)));
  }

  // The status of a call that writes these tensors: what was given counts as changed in place (autograd then notices
  // if a backward pass has saved it).
  void check(gam_status s, std::initializer_list<PyObject*> written) const {
    if (s != GAM_OK) refuse(s, g_entry.last_error(nullptr));
    for (PyObject* o : written) {
      const at::Tensor& t = THPVariable_Unpack(o);
      if (!t.is_inference()) t.unsafeGetTensorImpl()->bump_version();
    }
  }
};

struct Owned {  // a new reference that a refusal drops
  PyObject* p;
  explicit Owned(PyObject* o) : p(o) {
    if (!p) throw PyErr_Occurred();
  }
  ~Owned() { Py_XDECREF(p); }
  Owned(const Owned&) = delete;
  PyObject* release() {
    PyObject* r = p;
    p = nullptr;
    return r;
  }
};

int code(PyObject* o) { return (int)PyLong_AsLong(o); }

template <typename F>
PyObject* guarded(Py_ssize_t given, Py_ssize_t want, F&& body) {
  if (given != want) {
    PyErr_SetString(PyExc_TypeError, "wrong number of arguments");
    return nullptr;
  }
  try {
    return body();
  } catch (const Refused& r) {
    PyObject* e = PyObject_CallFunction(g_error, "is", r.status, r.message.c_str());
    if (e) {
      PyErr_SetObject(g_error, e);
      Py_DECREF(e);
    }
  } catch (const std::exception& e) {
    if (!PyErr_Occurred()) PyErr_SetString(PyExc_RuntimeError, e.what());
  } catch (PyObject*) {  // already set
  }
  return nullptr;
}

PyObject* pair_of(Owned& a, Owned& b) {
  PyObject* r = PyTuple_New(2);
  if (r) {
    PyTuple_SET_ITEM(r, 0, a.release());
    PyTuple_SET_ITEM(r, 1, b.release());
  }
  return r;
}

// x, packed, scale, bias, act, out, stream
PyObject* quant_linear(PyObject*, PyObject* const* a, Py_ssize_t n_args) {
  return guarded(n_args, 7, [&] {
    const at::Tensor &x = tensor(a[0], "x"), &w = tensor(a[1], "packed");
    const int dt = dtype_code(x, "x");
    if (x.dim() != 2 || w.dim() != 2) refuse(GAM_ERR_INVALID_ARG, "x must be [rows, k] and packed [n, k / 2]");
    const int64_t rows = x.size(0), k = x.size(1), n = w.size(0);
    if (k % 64) refuse(GAM_ERR_SHAPE, "k must be a multiple of 64");
    if (rows > INT32_MAX || n > INT32_MAX || k > INT32_MAX) refuse(GAM_ERR_CAPACITY, "a dimension passes 2^31");
    const Call call(x, a[6]);
    const auto type = x.scalar_type();
    Owned out(call.out(a[5], {rows, n}, type));
    void* y = call.arg(out.p, "out", {rows, n}, type, false);
    call.check(g_entry.quant_linear(
        call.arg(a[0], "x", {rows, k}, type, false), dt, x.stride(0),
        (const uint8_t*)call.arg(a[1], "packed", {n, k / 2}, at::kByte, true),
        call.arg(a[2], "scale", {n, k / 64}, at::kHalf, true),
        (const float*)call.arg(a[3], "bias", {n}, at::kFloat, true, true), code(a[4]), (int)rows, (int)n, (int)k, y,
        THPVariable_Unpack(out.p).stride(0), call.raw), {out.p});
    return out.release();
  });
}

// x, weight, bias, act, lengths, state, out, state_out, stream
PyObject* short_conv(PyObject*, PyObject* const* a, Py_ssize_t n_args) {
  return guarded(n_args, 9, [&] {
    const at::Tensor &x = tensor(a[0], "x"), &w = tensor(a[1], "weight");
    const int dt = dtype_code(x, "x");
    if (x.dim() != 3 || w.dim() != 2) refuse(GAM_ERR_INVALID_ARG, "x must be [batch, t, d] and weight [d, taps]");
    const int64_t B = x.size(0), t = x.size(1), d = x.size(2), taps = w.size(1);
    if (B > INT32_MAX || t > INT32_MAX || d > INT32_MAX) refuse(GAM_ERR_CAPACITY, "a dimension passes 2^31");
    if (taps < 2 || taps > 8) refuse(GAM_ERR_SHAPE, "taps must be 2 .. 8");
    const Call call(x, a[8]);
    const auto type = x.scalar_type();
    Owned out(call.out(a[6], {B, t, d}, type)), state(call.out(a[7], {B, taps - 1, d}, type));
    void* y = call.arg(out.p, "out", {B, t, d}, type, false);
    void* so = call.arg(state.p, "state_out", {B, taps - 1, d}, type, true);
    const at::Tensor& ot = THPVariable_Unpack(out.p);
    call.check(g_entry.short_conv(
        call.arg(a[0], "x", {B, t, d}, type, false), dt, x.stride(0), x.stride(1),
        (const float*)call.arg(a[1], "weight", {d, taps}, at::kFloat, true),
        (const float*)call.arg(a[2], "bias", {d}, at::kFloat, true, true), (int)taps, code(a[3]), (int)B, (int)t, (int)d,
        (const int32_t*)call.arg(a[4], "lengths", {B}, at::kInt, true, true),
        call.arg(a[5], "state", {B, taps - 1, d}, type, true, true), so, y, ot.stride(0), ot.stride(1), call.raw), {out.p, state.p});
    return pair_of(out, state);
  });
}

// x, dt, a, b, c, d_skip, z, dt_bias, dt_softplus, lengths, state, out, state_out, stream
PyObject* selective_scan(PyObject*, PyObject* const* a, Py_ssize_t n_args) {
  return guarded(n_args, 14, [&] {
    const at::Tensor &x = tensor(a[0], "x"), &rates = tensor(a[2], "a");
    gam_scan_args p = {};
    p.dtype = dtype_code(x, "x");
    if (x.dim() != 3 || rates.dim() != 2) refuse(GAM_ERR_INVALID_ARG, "x must be [batch, t, d] and a [d, n]");
    const int64_t B = x.size(0), t = x.size(1), d = x.size(2), n = rates.size(1);
    if (B > INT32_MAX || t > INT32_MAX || d > INT32_MAX) refuse(GAM_ERR_CAPACITY, "a dimension passes 2^31");
    if (n < 1 || n > 64) refuse(GAM_ERR_SHAPE, "n must be 1 .. 64");
    const Call call(x, a[13]);
    const auto type = x.scalar_type();
    Owned out(call.out(a[11], {B, t, d}, type)), state(call.out(a[12], {B, d, n}, at::kFloat));
    auto strided = [&](PyObject* o, const char* name, int64_t last, int64_t& bs, int64_t& rs, bool optional = false) {
      void* q = call.arg(o, name, {B, t, last}, type, false, optional);
      if (o != Py_None) bs = THPVariable_Unpack(o).stride(0), rs = THPVariable_Unpack(o).stride(1);
      return q;
    };
    p.y = strided(out.p, "out", d, p.y_batch_stride, p.y_row_stride);
    p.state_out = (float*)call.arg(state.p, "state_out", {B, d, n}, at::kFloat, true);
    p.x = strided(a[0], "x", d, p.x_batch_stride, p.x_row_stride);
    p.dt = strided(a[1], "dt", d, p.dt_batch_stride, p.dt_row_stride);
    p.a = (const float*)call.arg(a[2], "a", {d, n}, at::kFloat, true);
    p.b = strided(a[3], "b", n, p.b_batch_stride, p.b_row_stride);
    p.c = strided(a[4], "c", n, p.c_batch_stride, p.c_row_stride);
    p.d_skip = (const float*)call.arg(a[5], "d_skip", {d}, at::kFloat, true, true);
    p.z = strided(a[6], "z", d, p.z_batch_stride, p.z_row_stride, true);
    p.dt_bias = (const float*)call.arg(a[7], "dt_bias", {d}, at::kFloat, true, true);
    p.dt_softplus = PyObject_IsTrue(a[8]);
    if (p.dt_softplus < 0) throw PyErr_Occurred();
    p.lengths = (const int32_t*)call.arg(a[9], "lengths", {B}, at::kInt, true, true);
    p.state_in = (const float*)call.arg(a[10], "state", {B, d, n}, at::kFloat, true, true);
    p.batch = (int)B, p.t_max = (int)t, p.d = (int)d, p.n = (int)n;
    call.check(g_entry.selective_scan(&p, call.raw), {out.p, state.p});
    return pair_of(out, state);
  });
}

// x, y, alpha, layer_scale, gate, gate_act, post, post_weight, post_bias, pre, pre_weight, pre_bias, eps, x_out, out, stream
PyObject* residual_norm(PyObject*, PyObject* const* a, Py_ssize_t n_args) {
  return guarded(n_args, 16, [&] {
    const at::Tensor &x = tensor(a[0], "x"), &y = tensor(a[1], "y");
    gam_residual_norm_args p = {};
    p.x_dtype = dtype_code(x, "x");
    p.dtype = dtype_code(y, "y");
    if (x.dim() != 2) refuse(GAM_ERR_INVALID_ARG, "x must be [rows, d]");
    const int64_t rows = x.size(0), d = x.size(1);
    if (d > INT32_MAX) refuse(GAM_ERR_CAPACITY, "d above 16384");
    const Call call(x, a[15]);
    const auto xt = x.scalar_type(), yt = y.scalar_type();
    Owned x_out(call.out(a[13], {rows, d}, xt)), out(call.out(a[14], {rows, d}, yt));
    auto row = [&](PyObject* o, const char* name, at::ScalarType type, int64_t& stride) {
      void* q = call.arg(o, name, {rows, d}, type, false);
      stride = THPVariable_Unpack(o).stride(0);
      return q;
    };
    auto vec = [&](PyObject* o, const char* name) {
      return (const float*)call.arg(o, name, {d}, at::kFloat, true, true);
    };
    p.x = row(a[0], "x", xt, p.x_stride);
    p.y = row(a[1], "y", yt, p.y_stride);
    p.x_out = row(x_out.p, "x_out", xt, p.x_out_stride);
    p.u = row(out.p, "out", yt, p.u_stride);
    p.alpha = call.number(a[2], "alpha");
    p.layer_scale = vec(a[3], "layer_scale");
    p.gate_rows = 1;
    if (a[4] != Py_None) {
      const at::Tensor& g = tensor(a[4], "gate");
      if (g.dim() != 2) refuse(GAM_ERR_INVALID_ARG, "gate must be [gate_rows, d]");
      p.gate_rows = g.size(0);
      p.gate = call.arg(a[4], "gate", {p.gate_rows, d}, yt, false);
      p.gate_stride = g.stride(0);
    }
    p.gate_act = code(a[5]);
    p.post_norm = code(a[6]);
    p.post_weight = vec(a[7], "post_weight");
    p.post_bias = vec(a[8], "post_bias");
    p.pre_norm = code(a[9]);
    p.pre_weight = vec(a[10], "pre_weight");
    p.pre_bias = vec(a[11], "pre_bias");
    p.eps = call.number(a[12], "eps");
    p.rows = rows, p.d = (int)d;
    call.check(g_entry.residual_norm(&p, call.raw), {x_out.p, out.p});
    return pair_of(x_out, out);
  });
}

// The entry points' addresses in the order of Entry, then the exception class.
PyObject* bind(PyObject*, PyObject* args) {
  unsigned long long f[5];
  PyObject* error;
  if (!PyArg_ParseTuple(args, "KKKKKO", &f[0], &f[1], &f[2], &f[3], &f[4], &error)) return nullptr;
  g_entry.last_error = reinterpret_cast<decltype(g_entry.last_error)>(f[0]);
  g_entry.quant_linear = reinterpret_cast<decltype(g_entry.quant_linear)>(f[1]);
  g_entry.short_conv = reinterpret_cast<decltype(g_entry.short_conv)>(f[2]);
  g_entry.selective_scan = reinterpret_cast<decltype(g_entry.selective_scan)>(f[3]);
  g_entry.residual_norm = reinterpret_cast<decltype(g_entry.residual_norm)>(f[4]);
  Py_XSETREF(g_error, Py_NewRef(error));
  Py_RETURN_NONE;
}

PyMethodDef methods[] = {
    {"bind", bind, METH_VARARGS, nullptr},
    {"quant_linear", reinterpret_cast<PyCFunction>(quant_linear), METH_FASTCALL, nullptr},
    {"short_conv", reinterpret_cast<PyCFunction>(short_conv), METH_FASTCALL, nullptr},
    {"selective_scan", reinterpret_cast<PyCFunction>(selective_scan), METH_FASTCALL, nullptr},
    {"residual_norm", reinterpret_cast<PyCFunction>(residual_norm), METH_FASTCALL, nullptr},
    {nullptr, nullptr, 0, nullptr}};

PyModuleDef module = {PyModuleDef_HEAD_INIT, "_ops", "Marshalling of the streaming-block operators.", -1, methods};

}  // namespace

// The attribute built_for also leaves its text in the file, where the build looks for it.
PyMODINIT_FUNC PyInit__ops() {
  PyObject* m = PyModule_Create(&module);
  if (m && PyModule_AddStringConstant(m, "built_for", GAM_BUILT_FOR) < 0) Py_CLEAR(m);
  return m;
}
