// The sequence operators on torch tensors: argument checks, allocation of the
// outputs and the workspace, the current stream, and the call of the C ABI
// (cnhwc_seq.h).  A single token's kernel takes a few microseconds; done in
// Python the same steps took 9 to 12, here 2 to 3.
//
// Every function is documented in sequence.py, which passes its arguments on.
// Wrong tensors raise TypeError or ValueError, a status of the library the
// error class that set_error() was given.
#include <ATen/ATen.h>
#include <c10/core/DeviceGuard.h>
#include <c10/hip/HIPFunctions.h>
#include <c10/hip/HIPStream.h>
#include <torch/csrc/Exceptions.h>
#include <torch/csrc/utils/pybind.h>

#include <optional>
#include <string>
#include <tuple>

#include "cnhwc_seq.h"

namespace {

namespace py = pybind11;
using at::Tensor;
using Opt = std::optional<Tensor>;

PyObject* g_error = nullptr;  // the class of library errors

int32_t dtype_code(const Tensor& t, const char* name) {
  if (!t.is_cuda()) throw py::type_error(std::string(name) + " must be a GPU torch tensor");
  switch (t.scalar_type()) {
    case at::kFloat: return CNHWC_F32;
    case at::kHalf: return CNHWC_F16;
    case at::kBFloat16: return CNHWC_BF16;
    default: throw py::type_error("unsupported dtype " + std::string(at::toString(t.scalar_type())));
  }
}

std::string shape_of(at::IntArrayRef s) {
  std::string r = "(";
  for (size_t i = 0; i < s.size(); ++i) r += (i ? ", " : "") + std::to_string(s[i]);
  return r + ")";
}

// t on x's device, of this dtype and shape; dense, or with a channel stride of 1.
const Tensor& like(const Tensor& t, const char* name, const Tensor& x, at::ScalarType dtype, at::IntArrayRef shape,
                   bool dense = true) {
  if (!t.is_cuda() || t.get_device() != x.get_device())
    throw py::type_error(std::string(name) + " must be a torch tensor on cuda:" + std::to_string(x.get_device()));
  if (t.scalar_type() != dtype)
    throw py::type_error(std::string(name) + " must be " + at::toString(dtype) + ", got " +
                         at::toString(t.scalar_type()));
  if (t.sizes() != shape)
    throw py::value_error(std::string(name) + " must have shape " + shape_of(shape) + ", got " + shape_of(t.sizes()));
  if (dense) {
    if (!t.is_contiguous()) throw py::value_error(std::string(name) + " must be contiguous");
  } else if (t.stride(-1) != 1 && t.size(-1) != 1) {
    throw py::value_error(std::string(name) + " must have a channel stride of 1");
  }
  return t;
}

void like(const Opt& t, const char* name, const Tensor& x, at::ScalarType dtype, at::IntArrayRef shape,
          bool dense = true) {
  if (t) like(*t, name, x, dtype, shape, dense);
}

Tensor dense_like(const Tensor& t) { return at::empty(t.sizes(), t.options()); }
Opt dense_like(const Opt& t) { return t ? Opt(dense_like(*t)) : Opt(); }

Tensor output(const Opt& out, const Tensor& x) {
  if (!out) return dense_like(x);
  return like(*out, "out", x, x.scalar_type(), x.sizes());
}

template <typename T = void>
T* ptr(const Tensor& t) { return static_cast<T*>(t.data_ptr()); }
template <typename T = void>
T* ptr(const Opt& t) { return t ? static_cast<T*>(t->data_ptr()) : nullptr; }

Tensor workspace(const Opt& given, uint64_t need, const Tensor& x) {
  if (!given) return at::empty({int64_t(need)}, x.options().dtype(at::kByte));
  if (!given->is_cuda() || given->get_device() != x.get_device())
    throw py::type_error("workspace must be a torch tensor on cuda:" + std::to_string(x.get_device()));
  if (!given->is_contiguous()) throw py::value_error("workspace must be contiguous");
  return *given;
}
uint64_t bytes_of(const Tensor& t) { return uint64_t(t.numel()) * t.element_size(); }

void raise_status(int st, const char* name) {
  if (st == CNHWC_OK) return;
  py::object e = py::reinterpret_borrow<py::object>(g_error)(st, name);
  PyErr_SetObject(g_error, e.ptr());
  throw py::error_already_set();
}

// f(stream) on x's device and its current stream.
template <typename F>
void launch(const Tensor& x, const char* name, F&& f) {
  const auto dev = static_cast<c10::DeviceIndex>(x.get_device());
  void* stream = c10::hip::getCurrentHIPStream(dev).stream();
  if (dev == c10::hip::current_device()) {
    raise_status(f(stream), name);
  } else {
    const c10::DeviceGuard guard(x.device());
    raise_status(f(stream), name);
  }
}

// x [..., C] as n, l, c and the strides of n and l, without a copy.
struct Rows {
  int64_t n, l, c, stride[2];
};
Rows rows_of(const Tensor& t, const char* name) {
  if (t.dim() < 1) throw py::value_error(std::string(name) + " must be [..., C]");
  if (t.stride(-1) != 1 && t.size(-1) != 1)
    throw py::value_error(std::string(name) + " must have a channel stride of 1");
  const int64_t c = t.size(-1);
  if (t.dim() == 1) return {1, 1, c, {0, 0}};
  if (t.dim() == 2) return {1, t.size(0), c, {0, t.stride(0)}};
  // the dimensions before the last two collapse to one stride
  const int64_t lead = t.dim() - 2;
  int64_t n = 1, step = 0;
  for (int64_t i = lead - 1; i >= 0; --i) {
    if (t.size(i) == 1) continue;
    if (n == 1) step = t.stride(i);
    else if (t.numel() > 0 && t.stride(i) != step * n)
      throw py::value_error(std::string(name) + ": the leading dimensions must collapse to one stride");
    n *= t.size(i);
  }
  return {n, t.size(-2), c, {step, t.stride(-2)}};
}

// ---------------------------------------------------------------- layer norm

at::ScalarType norm_params(const Opt& weight, const Opt& bias, const Tensor& x) {
  if (!weight) {
    if (bias) throw py::value_error("bias needs weight");
    return x.scalar_type();
  }
  const at::ScalarType wd = weight->scalar_type();
  if (wd != x.scalar_type() && wd != at::kFloat)
    throw py::type_error("weight must be a " + std::string(at::toString(x.scalar_type())) + " or Float tensor");
  like(*weight, "weight", x, wd, {x.size(-1)});
  like(bias, "bias", x, wd, {x.size(-1)});
  return wd;
}

cnhwc_layer_norm_desc_t norm_desc(const Tensor& x, const Rows& r, const Rows& g, at::ScalarType wd, double eps) {
  const int32_t code = dtype_code(x, "x");
  return {code, wd == at::kFloat ? int32_t(CNHWC_F32) : code, r.n, r.l, r.c, {r.stride[0], r.stride[1]},
          {g.stride[0], g.stride[1]}, float(eps), 0};
}

py::object layer_norm(const Tensor& x, const Opt& weight, const Opt& bias, double eps, bool stats, const Opt& out) {
  dtype_code(x, "x");
  const Rows r = rows_of(x, "x");
  const at::ScalarType wd = norm_params(weight, bias, x);
  const Tensor y = output(out, x);
  Opt mean, rstd;
  if (stats) {
    mean = at::empty(x.sizes().slice(0, x.dim() - 1), x.options().dtype(at::kFloat));
    rstd = dense_like(mean);
  }
  if (r.n * r.l > 0) {
    const cnhwc_layer_norm_desc_t d = norm_desc(x, r, r, wd, eps);
    launch(x, "cnhwc_layer_norm_fwd", [&](void* s) {
      return cnhwc_layer_norm_fwd(&d, ptr(x), ptr(weight), ptr(bias), ptr(y), ptr<float>(mean), ptr<float>(rstd), s);
    });
  }
  return stats ? py::cast(std::make_tuple(y, *mean, *rstd)) : py::cast(y);
}

std::tuple<Tensor, Opt, Opt> layer_norm_backward(const Tensor& dy, const Tensor& x, const Tensor& mean,
                                                 const Tensor& rstd, const Opt& weight, const Opt& given) {
  dtype_code(x, "x");
  const Rows r = rows_of(x, "x");
  const Rows g = rows_of(like(dy, "dy", x, x.scalar_type(), x.sizes(), false), "dy");
  const at::IntArrayRef lead = x.sizes().slice(0, x.dim() - 1);
  like(mean, "mean", x, at::kFloat, lead);
  like(rstd, "rstd", x, at::kFloat, lead);
  const at::ScalarType wd = norm_params(weight, Opt(), x);
  const Tensor dx = dense_like(x);
  const Opt dw = dense_like(weight), db = dense_like(weight);
  if (r.n * r.l == 0) {
    if (dw) dw->zero_(), db->zero_();
    return {dx, dw, db};
  }
  const cnhwc_layer_norm_desc_t d = norm_desc(x, r, g, wd, 0.0);
  uint64_t need = 0;
  raise_status(cnhwc_layer_norm_bwd_workspace(&d, dw.has_value(), &need), "cnhwc_layer_norm_bwd_workspace");
  const Tensor ws = workspace(given, need, x);
  launch(x, "cnhwc_layer_norm_bwd", [&](void* s) {
    return cnhwc_layer_norm_bwd(&d, ptr(dy), ptr(x), ptr<float>(mean), ptr<float>(rstd), ptr(weight), ptr(dx),
                                ptr(dw), ptr(db), ptr(ws), bytes_of(ws), s);
  });
  return {dx, dw, db};
}

// ---------------------------------------------------------------- causal convolution

cnhwc_causal_conv_desc_t conv_check(const Tensor& x, const Tensor& w, const Opt& bias, int32_t act, const Opt& state,
                                    const Opt& lengths, int64_t dims) {
  cnhwc_causal_conv_desc_t d{};
  d.dtype = dtype_code(x, "x");
  if (x.dim() != dims) throw py::value_error(dims == 3 ? "x must be [N,L,C]" : "x must be [N,C]");
  const int64_t n = x.size(0), c = x.size(-1);
  if (x.stride(-1) != 1 && c != 1) throw py::value_error("x must have a channel stride of 1");
  if (w.dim() != 2 || w.size(0) != c || w.size(1) < 1)
    throw py::value_error("w must be [C,K] with x's channels and K >= 1");
  const int64_t k = w.size(1);
  like(w, "w", x, x.scalar_type(), w.sizes());
  like(bias, "bias", x, x.scalar_type(), {c});
  like(state, "state", x, x.scalar_type(), {n, k - 1, c});
  like(lengths, "lengths", x, at::kInt, {n});
  d.activation = act;
  d.n = n;
  d.l = dims == 3 ? x.size(1) : 1;
  d.c = c;
  d.k = int32_t(k < INT32_MAX ? k : INT32_MAX);
  d.x_stride[0] = x.stride(0);
  d.x_stride[1] = dims == 3 ? x.stride(1) : 0;
  return d;
}

// With one tap the state has no elements, and so no address.
py::object causal_conv1d(const Tensor& x, const Tensor& w, const Opt& bias, int32_t act, const Opt& state,
                         const Opt& lengths, bool return_state, const Opt& out) {
  const cnhwc_causal_conv_desc_t d = conv_check(x, w, bias, act, state, lengths, 3);
  const Tensor y = output(out, x);
  Opt last;
  if (return_state) last = at::empty({d.n, d.k - 1, d.c}, x.options());
  if (x.numel() > 0) {
    launch(x, "cnhwc_causal_conv_fwd", [&](void* s) {
      return cnhwc_causal_conv_fwd(&d, ptr(x), ptr(w), ptr(bias), ptr(state), ptr<int32_t>(lengths), ptr(y),
                                   ptr(last), s);
    });
  } else if (last) {
    if (state) last->copy_(*state);
    else last->zero_();
  }
  return last ? py::cast(std::make_tuple(y, *last)) : py::cast(y);
}

std::tuple<Tensor, Tensor, Opt, Opt> causal_conv1d_backward(const Tensor& dy, const Tensor& x, const Tensor& w,
                                                            const Opt& bias, int32_t act, const Opt& state,
                                                            const Opt& lengths, const Opt& dlast, const Opt& given) {
  cnhwc_causal_conv_desc_t d = conv_check(x, w, bias, act, state, lengths, 3);
  like(dy, "dy", x, x.scalar_type(), x.sizes(), false);
  like(dlast, "dstate", x, x.scalar_type(), {d.n, d.k - 1, d.c});
  d.dy_stride[0] = dy.stride(0);
  d.dy_stride[1] = dy.stride(1);
  const Tensor dx = dense_like(x), dw = dense_like(w);
  const Opt db = dense_like(bias), ds = dense_like(state);
  if (x.numel() == 0) {
    dw.zero_();
    if (db) db->zero_();
    if (ds) dlast ? ds->copy_(*dlast) : ds->zero_();
    return {dx, dw, db, ds};
  }
  uint64_t need = 0;
  raise_status(cnhwc_causal_conv_bwd_workspace(&d, &need), "cnhwc_causal_conv_bwd_workspace");
  const Tensor ws = workspace(given, need, x);
  launch(x, "cnhwc_causal_conv_bwd", [&](void* s) {
    return cnhwc_causal_conv_bwd(&d, ptr(dy), ptr(dlast), ptr(x), ptr(w), ptr(bias), ptr(state),
                                 ptr<int32_t>(lengths), ptr(dx), ptr(dw), ptr(db), ptr(ds), ptr(ws), bytes_of(ws), s);
  });
  return {dx, dw, db, ds};
}

Tensor causal_conv1d_step(const Tensor& x, const Opt& state, const Tensor& w, const Opt& bias, int32_t act,
                          const Opt& state_out, const Opt& out) {
  const cnhwc_causal_conv_desc_t d = conv_check(x, w, bias, act, state, Opt(), 2);
  if (!state) throw py::value_error("state is required");
  like(state_out, "state_out", x, x.scalar_type(), state->sizes());
  const Tensor y = output(out, x);
  if (x.numel() > 0)
    launch(x, "cnhwc_causal_conv_step", [&](void* s) {
      return cnhwc_causal_conv_step(&d, ptr(x), ptr(state), ptr(w), ptr(bias), ptr(y),
                                    state_out ? ptr(state_out) : ptr(state), s);
    });
  return y;
}

// ---------------------------------------------------------------- selective scan

struct Scan {
  cnhwc_scan_desc_t d{};
  cnhwc_scan_inputs_t in{};
};

Scan scan_check(const Tensor& u, const Tensor& delta, const Tensor& a, const Tensor& b, const Tensor& c,
                const Opt& skip, const Opt& gate, const Opt& bias, bool softplus, const Opt& state,
                const Opt& lengths, int64_t dims) {
  Scan r;
  cnhwc_scan_desc_t& d = r.d;
  d.dtype = dtype_code(u, "u");
  if (u.dim() != dims) throw py::value_error(dims == 3 ? "u must be [N,L,D]" : "u must be [N,D]");
  const int64_t n = u.size(0), l = dims == 3 ? u.size(1) : 1, wide = u.size(-1);
  if (a.dim() != 2 || a.size(0) != wide || a.size(1) < 1)
    throw py::value_error("a must be [D,S] with u's channels and S >= 1");
  const int64_t s = a.size(1);
  const at::ScalarType dt = u.scalar_type();
  const int64_t bc3[3] = {n, l, s}, bc2[2] = {n, s};
  const at::IntArrayRef bc = dims == 3 ? at::IntArrayRef(bc3, 3) : at::IntArrayRef(bc2, 2);
  like(u, "u", u, dt, u.sizes(), false);
  like(delta, "delta", u, dt, u.sizes(), false);
  like(a, "a", u, at::kFloat, a.sizes());
  like(b, "b", u, dt, bc, false);
  like(c, "c", u, dt, bc, false);
  like(skip, "skip", u, at::kFloat, {wide});
  like(gate, "gate", u, dt, u.sizes(), false);
  like(bias, "delta_bias", u, at::kFloat, {wide});
  like(state, "state", u, at::kFloat, {n, wide, s});
  like(lengths, "lengths", u, at::kInt, {n});
  d.softplus = softplus;
  d.n = n;
  d.l = l;
  d.d = wide;
  d.s = int32_t(s < INT32_MAX ? s : INT32_MAX);
  auto strides = [&](const Tensor& t, int64_t (&to)[2]) {
    to[0] = t.stride(0);
    to[1] = dims == 3 ? t.stride(1) : 0;
  };
  strides(u, d.u_stride);
  strides(delta, d.delta_stride);
  strides(b, d.b_stride);
  strides(c, d.c_stride);
  if (gate) strides(*gate, d.gate_stride);
  r.in = {ptr(u), ptr(delta), ptr<float>(a), ptr(b), ptr(c), ptr<float>(skip), ptr(gate), ptr<float>(bias),
          ptr<float>(state), ptr<int32_t>(lengths)};
  return r;
}

py::object selective_scan(const Tensor& u, const Tensor& delta, const Tensor& a, const Tensor& b, const Tensor& c,
                          const Opt& skip, const Opt& gate, const Opt& bias, bool softplus, const Opt& state,
                          const Opt& lengths, bool return_state, const Opt& out, const Opt& given) {
  const Scan r = scan_check(u, delta, a, b, c, skip, gate, bias, softplus, state, lengths, 3);
  const Tensor y = output(out, u);
  Opt last;
  if (return_state) last = at::empty({r.d.n, r.d.d, int64_t(r.d.s)}, a.options());
  if (u.numel() > 0) {
    uint64_t need = 0;
    raise_status(cnhwc_scan_fwd_workspace(&r.d, &need), "cnhwc_scan_fwd_workspace");
    const Tensor ws = workspace(given, need, u);
    launch(u, "cnhwc_scan_fwd", [&](void* s) {
      return cnhwc_scan_fwd(&r.d, &r.in, ptr(y), ptr<float>(last), ptr(ws), bytes_of(ws), s);
    });
  } else if (last) {
    if (state) last->copy_(*state);
    else last->zero_();
  }
  return last ? py::cast(std::make_tuple(y, *last)) : py::cast(y);
}

using Grads = std::tuple<Tensor, Tensor, Tensor, Tensor, Tensor, Opt, Opt, Opt, Opt>;
Grads selective_scan_backward(const Tensor& dy, const Tensor& u, const Tensor& delta, const Tensor& a, const Tensor& b,
                              const Tensor& c, const Opt& skip, const Opt& gate, const Opt& bias, bool softplus,
                              const Opt& state, const Opt& lengths, const Opt& dlast, const Opt& given) {
  Scan r = scan_check(u, delta, a, b, c, skip, gate, bias, softplus, state, lengths, 3);
  like(dy, "dy", u, u.scalar_type(), u.sizes(), false);
  like(dlast, "dstate", u, at::kFloat, {r.d.n, r.d.d, int64_t(r.d.s)});
  r.d.dy_stride[0] = dy.stride(0);
  r.d.dy_stride[1] = dy.stride(1);
  const Grads g{dense_like(u), dense_like(delta), dense_like(a), dense_like(b), dense_like(c),
                dense_like(skip), dense_like(gate), dense_like(bias), dense_like(state)};
  const auto& [du, dd, da, db, dc, dskip, dgate, dbias, dstate] = g;
  if (u.numel() == 0) {
    for (const Tensor* t : {&du, &dd, &da, &db, &dc}) t->zero_();
    for (const Opt* t : {&dskip, &dgate, &dbias})
      if (*t) (*t)->zero_();
    if (dstate) dlast ? dstate->copy_(*dlast) : dstate->zero_();
    return g;
  }
  uint64_t need = 0;
  raise_status(cnhwc_scan_bwd_workspace(&r.d, &need), "cnhwc_scan_bwd_workspace");
  const Tensor ws = workspace(given, need, u);
  const cnhwc_scan_grads_t out{ptr(du), ptr(dd), ptr<float>(da), ptr(db), ptr(dc), ptr<float>(dskip), ptr(dgate),
                               ptr<float>(dbias), ptr<float>(dstate)};
  launch(u, "cnhwc_scan_bwd", [&](void* s) {
    return cnhwc_scan_bwd(&r.d, &r.in, ptr(dy), ptr<float>(dlast), &out, ptr(ws), bytes_of(ws), s);
  });
  return g;
}

Tensor selective_scan_step(const Tensor& u, const Tensor& delta, const Tensor& a, const Tensor& b, const Tensor& c,
                           const Opt& state, const Opt& skip, const Opt& gate, const Opt& bias, bool softplus,
                           const Opt& state_out, const Opt& out) {
  const Scan r = scan_check(u, delta, a, b, c, skip, gate, bias, softplus, state, Opt(), 2);
  if (!state) throw py::value_error("state is required");
  like(state_out, "state_out", u, at::kFloat, state->sizes());
  const Tensor y = output(out, u);
  if (u.numel() > 0)
    launch(u, "cnhwc_scan_step", [&](void* s) {
      return cnhwc_scan_step(&r.d, &r.in, ptr(y), state_out ? ptr<float>(state_out) : ptr<float>(state), s);
    });
  return y;
}

}  // namespace

PYBIND11_MODULE(_seq, m) {
  m.def("set_error", [](py::object cls) { g_error = cls.release().ptr(); });
  // torch's own errors (an allocation that fails) keep their Python types
  m.def("layer_norm", torch::wrap_pybind_function(layer_norm));
  m.def("layer_norm_backward", torch::wrap_pybind_function(layer_norm_backward));
  m.def("causal_conv1d", torch::wrap_pybind_function(causal_conv1d));
  m.def("causal_conv1d_backward", torch::wrap_pybind_function(causal_conv1d_backward));
  m.def("causal_conv1d_step", torch::wrap_pybind_function(causal_conv1d_step));
  m.def("selective_scan", torch::wrap_pybind_function(selective_scan));
  m.def("selective_scan_backward", torch::wrap_pybind_function(selective_scan_backward));
  m.def("selective_scan_step", torch::wrap_pybind_function(selective_scan_step));
}
