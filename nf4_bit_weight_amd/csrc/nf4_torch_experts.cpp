// Argument marshalling of the expert calls (nf4_experts.h) and of the products
// in 8-bit integers (nf4_int8.h) for Python, and the autograd nodes of the former.  As in
// nf4_torch.cpp, every function takes its arguments by position (experts.py and
// int8.py name them) and returns the results, or the status of a C call that
// failed.  Nothing here computes.
#include "nf4_torch.hpp"

#include <torch/csrc/Dtype.h>

#include "../../include/nf4_experts.h"
#include "../../include/nf4_int8.h"

namespace {

using torch::autograd::AutogradContext;
using torch::autograd::variable_list;

int32_t small(int64_t v, const char* name) {
  if (v < INT32_MIN || v > INT32_MAX) refuse(name, " is out of range: ", v);
  return static_cast<int32_t>(v);
}
int32_t small(PyObject* o, const char* name) { return small(integer(o, name), name); }
double number(PyObject* o, const char* name) {
  const double v = PyFloat_AsDouble(o);
  if (PyErr_Occurred()) {
    PyErr_Clear();
    refuse(name, " must be a number");
  }
  return v;
}

int dtype_of(const Tensor& t, const char* name) {
  if (t.scalar_type() == at::kFloat) return NF4_DTYPE_F32;
  if (t.scalar_type() == at::kBFloat16) return NF4_DTYPE_BF16;
  refuse(name, " must be float32 or bfloat16, got ", t.scalar_type());
}
void on_device(const Tensor& t, const char* name) {
  if (!t.is_cuda()) refuse(name, " must be a device tensor");
}

// A [rows, n] tensor of the calls' types whose rows may be strided.
struct Matrix {
  c10::Device dev{c10::kCPU};
  at::ScalarType type = at::kFloat;
  void* p = nullptr;
  int dtype = 0;
  int64_t rows = 0, n = 0, stride = 0;
};
Matrix matrix(const Tensor& t, const char* name, const c10::Device* dev = nullptr) {
  if (t.dim() != 2) refuse(name, " must have two dimensions, got ", t.sizes());
  on_device(t, name);
  if (dev && t.device() != *dev) refuse(name, " is on ", t.device(), ", expected ", *dev);
  Matrix m{t.device(), t.scalar_type(), t.data_ptr(), dtype_of(t, name), t.size(0), t.size(1), t.size(1)};
  if (t.numel() == 0) return m;
  if (m.n > 1 && t.stride(1) != 1) refuse(name, ": the elements of a row must be contiguous");
  if (m.rows > 1) m.stride = t.stride(0);
  return m;
}

// What the differentiable calls make of their input: float32 or bfloat16 (other types as
// float32), the elements of a row contiguous.
Tensor native(const Tensor& t, const char* name) {
  on_device(t, name);
  if (!t.is_floating_point()) refuse(name, " must be a floating point tensor, got ", t.scalar_type());
  const bool fits = t.scalar_type() == at::kFloat || t.scalar_type() == at::kBFloat16;
  const Tensor x = fits ? t : t.to(at::kFloat);
  return x.dim() != 2 || x.numel() == 0 || x.size(1) == 1 || x.stride(1) == 1 ? x : x.contiguous();
}
Tensor native_dense(const Tensor& t, const char* name) { return native(t, name).contiguous(); }

bool records(std::initializer_list<const Tensor*> inputs) {
  if (!at::GradMode::is_enabled()) return false;
  for (const Tensor* t : inputs)
    if (t->defined() && t->requires_grad()) return true;
  return false;
}
void once_only(const char* name, const Tensor& grad) {
  if (at::GradMode::is_enabled()) throw std::runtime_error(std::string(name) + ": its backward pass is not differentiable (create_graph)");
  if (grad.defined() && grad._fw_grad(0).defined())
    throw std::runtime_error(std::string(name) + ": the gradient carries a forward-mode tangent, and the backward pass has no forward derivative");
}

// ---- routing -------------------------------------------------------------------

struct Route {
  int32_t k = 0, groups = 1, top_groups = 1;
  bool sigmoid = false, top2 = false, renorm = false;
  float scale = 1.0f;
};
float positive(double s) {
  const float f = static_cast<float>(s);
  if (!(f > 0.0f) || !std::isfinite(f)) refuse("scale must be positive and finite, got ", s);
  return f;
}
struct Routed {
  Tensor weights, experts, offsets, tokens, slots;
  int status = 0;
};
// Numbers `at` .. of `all` as a tensor of their own.  (The four results of integers share one
// allocation: at a batch of new tokens allocating takes as long as the kernel.)
Tensor part_of(const Tensor& all, int64_t at, at::IntArrayRef shape) {
  auto impl = c10::make_intrusive<at::TensorImpl>(c10::Storage(all.storage()), all.key_set(), all.dtype());
  impl->set_storage_offset(at);
  impl->set_sizes_contiguous(shape);
  return Tensor(std::move(impl));
}
Routed run_route(const Tensor& logits, const Tensor& bias, const Route& r) {
  const Matrix l = matrix(logits, "logits");
  const int32_t E = small(l.n, "the number of experts");
  if (r.k < 1 || r.k > E) refuse("top_k must be 1 to the ", E, " experts, got ", r.k);
  if (r.groups < 1 || E % r.groups) refuse(E, " experts do not divide into ", r.groups, " groups");
  if (r.top_groups < 1 || r.top_groups > r.groups) refuse("top_groups must be 1 to ", r.groups, ", got ", r.top_groups);
  if (bias.defined()) need(bias, "bias", at::kFloat, E, &l.dev);
  const size_t bytes = nf4_expert_plan_workspace(l.rows, r.k, E);
  if (bytes == SIZE_MAX) return {{}, {}, {}, {}, {}, NF4_ERR_UNSUPPORTED};
  const int64_t n = l.rows * r.k;
  const Tensor all = fresh({3 * n + E + 1}, at::kInt, l.dev);
  Routed o{fresh({l.rows, r.k}, at::kFloat, l.dev), part_of(all, 0, {l.rows, r.k}), part_of(all, 3 * n, {E + 1}), part_of(all, n, {n}),
           part_of(all, 2 * n, {l.rows, r.k})};
  const On on(l.dev);
  const Tensor ws = new_workspace(bytes, l.dev);
  o.status = nf4_route_fwd(l.p, l.dtype, l.stride, l.rows, E, r.k, bias.defined() ? bias.data_ptr<float>() : nullptr, r.sigmoid,
                           r.groups, r.top_groups, r.top2, r.renorm, r.scale, o.weights.data_ptr<float>(),
                           o.experts.data_ptr<int32_t>(), o.offsets.data_ptr<int32_t>(), o.tokens.data_ptr<int32_t>(),
                           o.slots.data_ptr<int32_t>(), ptr(ws), ws.defined() ? ws.nbytes() : 0, on.stream);
  return o;
}
int run_route_bwd(const Tensor& grad, const Tensor& logits, const Tensor& weights, const Tensor& experts, const Route& r, Tensor& out) {
  const Matrix l = matrix(logits, "logits");
  if (experts.dim() != 2 || experts.size(0) != l.rows) refuse("experts must be [", l.rows, ", top_k], got ", experts.sizes());
  const int32_t k = small(experts.size(1), "top_k"), E = small(l.n, "the number of experts");
  need(experts, "experts", at::kInt, -1, &l.dev);
  need(weights, "weights", at::kFloat, l.rows * k, &l.dev);
  need(grad, "grad_weights", at::kFloat, l.rows * k, &l.dev);
  out = fresh({l.rows, l.n}, l.type, l.dev);
  const On on(l.dev);
  return nf4_route_bwd(grad.data_ptr<float>(), l.p, l.dtype, l.stride, l.rows, E, k, weights.data_ptr<float>(),
                       experts.data_ptr<int32_t>(), r.sigmoid, r.renorm, r.scale, out.data_ptr(), on.stream);
}

// Differentiable in the logits.  (Nodes in C++, as in nf4_torch.cpp: tensors are saved
// through save_for_backward only, and the backward runs without the interpreter.)
struct RouteNode : torch::autograd::Function<RouteNode> {
  static variable_list forward(AutogradContext* ctx, const Tensor& logits, const std::optional<Tensor>& bias, const Route& r) {
    const Tensor l = native(logits, "logits");
    const Routed o = run_route(l, bias ? *bias : Tensor(), r);
    ok(o.status, "nf4_route_fwd");
    ctx->mark_non_differentiable({o.experts, o.offsets, o.tokens, o.slots});
    ctx->set_materialize_grads(false);                         // no zeros for the integers
    ctx->save_for_backward({l, o.weights, o.experts});
    ctx->saved_data["sigmoid"] = r.sigmoid;
    ctx->saved_data["renorm"] = r.renorm;
    ctx->saved_data["scale"] = static_cast<double>(r.scale);
    ctx->saved_data["type"] = logits.scalar_type();
    return {o.weights, o.experts, o.offsets, o.tokens, o.slots};
  }
  static variable_list backward(AutogradContext* ctx, variable_list grad) {
    once_only("nf4_route", grad[0]);
    if (!grad[0].defined()) return {Tensor(), Tensor(), Tensor()};
    const auto s = ctx->get_saved_variables();
    Route r;
    r.sigmoid = ctx->saved_data["sigmoid"].toBool();
    r.renorm = ctx->saved_data["renorm"].toBool();
    r.scale = static_cast<float>(ctx->saved_data["scale"].toDouble());
    Tensor out;
    ok(run_route_bwd(native_dense(grad[0], "grad_weights").to(at::kFloat), s[0], s[1], s[2], r, out), "nf4_route_bwd");
    return {out.to(ctx->saved_data["type"].toScalarType()), Tensor(), Tensor()};
  }
};

// (logits, top_k, sigmoid, bias, groups, top_groups, top2, renormalize, scale)
PyObject* route(PyObject* const* a) {
  no_tangents({{"logits", a[0]}, {"bias", a[3]}});
  const Tensor& logits = tensor(a[0], "logits");
  Route r;
  r.k = small(a[1], "top_k");
  r.sigmoid = truth(a[2], "score");
  r.groups = small(a[4], "groups");
  r.top_groups = small(a[5], "top_groups");
  r.top2 = truth(a[6], "group_score");
  r.renorm = truth(a[7], "renormalize");
  r.scale = positive(number(a[8], "scale"));
  const Tensor bias = given(a[3]) ? tensor(a[3], "bias") : Tensor();
  on_device(logits, "logits");
  if (records({&bias})) refuse("bias requires a gradient, which this call does not carry: it only moves the choice");
  if (records({&logits})) {
    check_capture({{"logits", &logits}}, logits.device());
    const variable_list o = RouteNode::apply(logits, bias.defined() ? std::optional<Tensor>(bias) : std::nullopt, r);
    return several(o[0], o[1], o[2], o[3], o[4]);
  }
  const Routed o = run_route(native(logits, "logits"), bias, r);
  return o.status ? PyLong_FromLong(o.status) : several(o.weights, o.experts, o.offsets, o.tokens, o.slots);
}

// (grad_weights, logits, weights, experts, sigmoid, renormalize, scale)
PyObject* route_bwd(PyObject* const* a) {
  no_tangents({{"grad_weights", a[0]}, {"logits", a[1]}, {"weights", a[2]}});
  Route r;
  r.sigmoid = truth(a[4], "score");
  r.renorm = truth(a[5], "renormalize");
  r.scale = positive(number(a[6], "scale"));
  Tensor out;
  const int st = run_route_bwd(tensor(a[0], "grad_weights"), tensor(a[1], "logits"), tensor(a[2], "weights"), tensor(a[3], "experts"), r, out);
  return st ? PyLong_FromLong(st) : wrap(out);
}

// (experts, E)
PyObject* expert_plan(PyObject* const* a) {
  const Tensor& experts = tensor(a[0], "experts");
  const int32_t E = small(a[1], "E");
  if (experts.dim() != 2) refuse("experts must be [T, top_k], got ", experts.sizes());
  need(experts, "experts", at::kInt, -1, nullptr);
  const c10::Device dev = experts.device();
  const int64_t T = experts.size(0);
  const int32_t k = small(experts.size(1), "top_k");
  const size_t bytes = nf4_expert_plan_workspace(T, k, E);
  if (bytes == SIZE_MAX) return PyLong_FromLong(E < 1 || k < 1 ? NF4_ERR_SHAPE : NF4_ERR_UNSUPPORTED);
  const Tensor offsets = fresh({E + 1}, at::kInt, dev), tokens = fresh({T * k}, at::kInt, dev), slots = fresh({T, k}, at::kInt, dev);
  const On on(dev);
  const Tensor ws = new_workspace(bytes, dev);
  const int st = nf4_expert_plan(experts.data_ptr<int32_t>(), T, k, E, offsets.data_ptr<int32_t>(), tokens.data_ptr<int32_t>(),
                                 slots.data_ptr<int32_t>(), ptr(ws), ws.defined() ? ws.nbytes() : 0, on.stream);
  return st ? PyLong_FromLong(st) : several(offsets, tokens, slots);
}

// ---- rows to and from the experts --------------------------------------------------

struct Slots {
  int64_t T = 0;
  int32_t k = 0;
  const int32_t *slots = nullptr, *end = nullptr;
};
Slots slots_of(const Tensor& slots, const Tensor& offsets, const c10::Device& dev) {
  if (slots.dim() != 2) refuse("slots must be [T, top_k], got ", slots.sizes());
  need(slots, "slots", at::kInt, -1, &dev);
  Slots s{slots.size(0), small(slots.size(1), "top_k"), slots.data_ptr<int32_t>(), nullptr};
  if (!offsets.defined()) return s;
  need(offsets, "offsets", at::kInt, -1, &dev);
  if (offsets.dim() != 1 || offsets.numel() < 2) refuse("offsets must be [E + 1]");
  s.end = offsets.data_ptr<int32_t>() + offsets.numel() - 1;
  return s;
}
void dense(const Tensor& t, const char* name, int64_t rows, int64_t n, at::ScalarType type, const c10::Device& dev) {
  if (t.dim() != 2 || t.size(0) != rows || (n >= 0 && t.size(1) != n))
    refuse(name, " must be [", rows, ", ", n >= 0 ? std::to_string(n) : "H", "], got ", t.sizes());
  need(t, name, type, -1, &dev);
}

int run_gather(const Tensor& x, const Tensor& slots, const Tensor& offsets, Tensor& out) {
  const Matrix m = matrix(x, "x");
  const Slots s = slots_of(slots, offsets, m.dev);
  if (m.rows != s.T) refuse("x has ", m.rows, " rows, the routing ", s.T, " tokens");
  const bool fill = !out.defined();
  if (fill) out = fresh({s.T * s.k, m.n}, m.type, m.dev);
  else dense(out, "out", s.T * s.k, m.n, m.type, m.dev);
  const On on(m.dev);
  return nf4_expert_gather(m.p, m.dtype, m.stride, s.T, m.n, s.k, s.slots, s.end, out.data_ptr(), fill, on.stream);
}
int run_gather_bwd(const Tensor& grad, const Tensor& slots, Tensor& out) {
  const Matrix m = matrix(grad, "grad_rows");
  const Slots s = slots_of(slots, Tensor(), m.dev);
  dense(grad, "grad_rows", s.T * s.k, -1, m.type, m.dev);
  out = fresh({s.T, m.n}, m.type, m.dev);
  const On on(m.dev);
  return nf4_expert_gather_bwd(m.p, m.dtype, s.T, m.n, s.k, s.slots, out.data_ptr(), on.stream);
}
int run_combine(const Tensor& rows, const Tensor& weights, const Tensor& slots, Tensor& out) {
  const Matrix m = matrix(rows, "rows");
  const Slots s = slots_of(slots, Tensor(), m.dev);
  dense(rows, "rows", s.T * s.k, -1, m.type, m.dev);
  dense(weights, "weights", s.T, s.k, at::kFloat, m.dev);
  if (!out.defined()) out = fresh({s.T, m.n}, m.type, m.dev);
  else dense(out, "out", s.T, m.n, m.type, m.dev);
  const On on(m.dev);
  return nf4_expert_combine_fwd(m.p, m.dtype, s.T, m.n, s.k, weights.data_ptr<float>(), s.slots, out.data_ptr(), on.stream);
}
int run_combine_bwd(const Tensor& grad, const Tensor& rows, const Tensor& weights, const Tensor& slots, const Tensor& offsets,
                    bool want_rows, bool want_weights, Tensor& grad_rows, Tensor& grad_weights) {
  const Matrix g = matrix(grad, "grad_out");
  const Slots s = slots_of(slots, offsets, g.dev);
  if (g.rows != s.T) refuse("grad_out has ", g.rows, " rows, the routing ", s.T, " tokens");
  dense(rows, "rows", s.T * s.k, g.n, g.type, g.dev);
  dense(weights, "weights", s.T, s.k, at::kFloat, g.dev);
  if (want_rows) grad_rows = fresh({s.T * s.k, g.n}, g.type, g.dev);
  if (want_weights) grad_weights = fresh({s.T, s.k}, at::kFloat, g.dev);
  const On on(g.dev);
  return nf4_expert_combine_bwd(g.p, g.stride, rows.data_ptr(), g.dtype, s.T, g.n, s.k, weights.data_ptr<float>(), s.slots, s.end,
                                ptr(grad_rows), static_cast<float*>(ptr(grad_weights)), want_rows, on.stream);
}

struct GatherNode : torch::autograd::Function<GatherNode> {
  static Tensor forward(AutogradContext* ctx, const Tensor& x, const Tensor& slots, const Tensor& offsets) {
    Tensor out;
    ok(run_gather(native(x, "x"), slots, offsets, out), "nf4_expert_gather");
    ctx->save_for_backward({slots});
    ctx->saved_data["type"] = x.scalar_type();
    return out.to(x.scalar_type());
  }
  static variable_list backward(AutogradContext* ctx, variable_list grad) {
    once_only("nf4_expert_gather", grad[0]);
    const auto s = ctx->get_saved_variables();
    Tensor out;
    ok(run_gather_bwd(native_dense(grad[0], "grad_rows"), s[0], out), "nf4_expert_gather_bwd");
    return {out.to(ctx->saved_data["type"].toScalarType()), Tensor(), Tensor()};
  }
};
struct CombineNode : torch::autograd::Function<CombineNode> {
  static Tensor forward(AutogradContext* ctx, const Tensor& rows, const Tensor& weights, const Tensor& slots, const Tensor& offsets) {
    const Tensor r = native_dense(rows, "rows"), w = native_dense(weights, "weights").to(at::kFloat);
    slots_of(slots, offsets, r.device());                      // refused here, not in the backward pass
    Tensor out;
    ok(run_combine(r, w, slots, out), "nf4_expert_combine_fwd");
    ctx->save_for_backward({r, w, slots, offsets});
    ctx->saved_data["rows"] = rows.scalar_type();
    ctx->saved_data["weights"] = weights.scalar_type();
    return out.to(rows.scalar_type());
  }
  static variable_list backward(AutogradContext* ctx, variable_list grad) {
    once_only("nf4_expert_combine", grad[0]);
    const auto s = ctx->get_saved_variables();
    const Tensor g = native(grad[0], "grad_out").to(s[0].scalar_type());
    Tensor gr, gw;
    ok(run_combine_bwd(g, s[0], s[1], s[2], s[3], ctx->needs_input_grad(0), ctx->needs_input_grad(1), gr, gw), "nf4_expert_combine_bwd");
    return {gr.defined() ? gr.to(ctx->saved_data["rows"].toScalarType()) : gr,
            gw.defined() ? gw.to(ctx->saved_data["weights"].toScalarType()) : gw, Tensor(), Tensor()};
  }
};

// (x, slots, offsets, out)
PyObject* expert_gather(PyObject* const* a) {
  no_tangents({{"x", a[0]}, {"out", a[3]}});
  const Tensor &x = tensor(a[0], "x"), &slots = tensor(a[1], "slots"), &offsets = tensor(a[2], "offsets");
  Tensor out = given(a[3]) ? tensor(a[3], "out") : Tensor();
  on_device(x, "x");
  if (records({&x, &out})) {
    if (out.defined()) refuse("out carries no gradient: leave it out, or call under torch.no_grad()");
    check_capture({{"x", &x}}, x.device());
    return wrap(GatherNode::apply(x, slots, offsets));
  }
  if (out.defined()) {
    const int st = run_gather(x, slots, offsets, out);
    return st ? PyLong_FromLong(st) : wrap(out);
  }
  const int st = run_gather(native(x, "x"), slots, offsets, out);
  return st ? PyLong_FromLong(st) : wrap(out.to(x.scalar_type()));
}

// (grad_rows, slots)
PyObject* expert_gather_bwd(PyObject* const* a) {
  no_tangents({{"grad_rows", a[0]}});
  Tensor out;
  const int st = run_gather_bwd(tensor(a[0], "grad_rows"), tensor(a[1], "slots"), out);
  return st ? PyLong_FromLong(st) : wrap(out);
}

// (rows, weights, slots, offsets, out)
PyObject* expert_combine(PyObject* const* a) {
  no_tangents({{"rows", a[0]}, {"weights", a[1]}, {"out", a[4]}});
  const Tensor &rows = tensor(a[0], "rows"), &weights = tensor(a[1], "weights"), &slots = tensor(a[2], "slots"),
               &offsets = tensor(a[3], "offsets");
  Tensor out = given(a[4]) ? tensor(a[4], "out") : Tensor();
  on_device(rows, "rows");
  on_device(weights, "weights");
  if (records({&rows, &weights, &out})) {
    if (out.defined()) refuse("out carries no gradient: leave it out, or call under torch.no_grad()");
    check_capture({{"rows", &rows}, {"weights", &weights}}, rows.device());
    return wrap(CombineNode::apply(rows, weights, slots, offsets));
  }
  if (out.defined()) {
    const int st = run_combine(rows, weights, slots, out);
    return st ? PyLong_FromLong(st) : wrap(out);
  }
  const int st = run_combine(native_dense(rows, "rows"), native_dense(weights, "weights").to(at::kFloat), slots, out);
  return st ? PyLong_FromLong(st) : wrap(out.to(rows.scalar_type()));
}

// (grad_out, rows, weights, slots, offsets)
PyObject* expert_combine_bwd(PyObject* const* a) {
  no_tangents({{"grad_out", a[0]}, {"rows", a[1]}, {"weights", a[2]}});
  Tensor gr, gw;
  const int st = run_combine_bwd(tensor(a[0], "grad_out"), tensor(a[1], "rows"), tensor(a[2], "weights"), tensor(a[3], "slots"),
                                 tensor(a[4], "offsets"), true, true, gr, gw);
  return st ? PyLong_FromLong(st) : several(gr, gw);
}

// ---- 8-bit integers ------------------------------------------------------------------

// (x)
PyObject* int8_quantize(PyObject* const* a) {
  no_derivatives({{"x", a[0]}});
  const Matrix m = matrix(tensor(a[0], "x"), "x");
  const Tensor q = fresh({m.rows, nf4_int8_row_bytes(m.n)}, at::kChar, m.dev), scale = fresh({m.rows}, at::kFloat, m.dev);
  const On on(m.dev);
  const int st = nf4_int8_quantize(m.p, m.dtype, m.stride, m.rows, m.n, q.data_ptr<int8_t>(), scale.data_ptr<float>(), on.stream);
  return st ? PyLong_FromLong(st) : several(q, scale);
}

struct Product {
  c10::Device dev{c10::kCPU};
  const void* x = nullptr;
  int x_dtype = 0, y_dtype = 0;
  int64_t stride = 0, rows = 0, N = 0, K = 0;
  const float *x_scale = nullptr, *scale = nullptr, *bias = nullptr;
  const int8_t* q = nullptr;
  at::ScalarType y_type = at::kBFloat16;
};
// a: x, x_scale, q, scale, N, K, bias, out_dtype; experts: rows of the weight are experts * N
Product product_of(PyObject* const* a, int64_t experts) {
  Product p;
  const Tensor &x = tensor(a[0], "x"), &q = tensor(a[2], "q"), &scale = tensor(a[3], "scale");
  p.N = integer(a[4], "N");
  p.K = integer(a[5], "K");
  if (p.N < 0 || p.K < 0) refuse("N and K must not be negative");
  const int64_t pitch = nf4_int8_row_bytes(p.K);
  if (given(a[1])) {
    if (x.dim() != 2 || x.size(1) != pitch) refuse("x's integers must be [M, ", pitch, "], got ", x.sizes());
    need(x, "x", at::kChar, -1, nullptr);
    p.dev = x.device();
    p.x = x.data_ptr();
    p.x_dtype = NF4_DTYPE_I8;
    p.rows = x.size(0);
    const Tensor& xs = tensor(a[1], "x_scale");
    need(xs, "x_scale", at::kFloat, p.rows, &p.dev);
    p.x_scale = xs.data_ptr<float>();
  } else {
    const Matrix m = matrix(x, "x");
    if (m.n != p.K) refuse("x must be [M, ", p.K, "], got ", x.sizes());
    p.dev = m.dev;
    p.x = m.p;
    p.x_dtype = m.dtype;
    p.rows = m.rows;
    p.stride = m.stride;
    p.y_type = m.type;
  }
  if (q.dim() != 2 || q.size(1) != pitch || q.size(0) / experts != p.N || q.size(0) % experts)
    refuse("the weight's integers must be [", experts > 1 ? std::to_string(experts) + " * " : "", p.N, ", ", pitch, "], got ", q.sizes());
  need(q, "q", at::kChar, -1, &p.dev);
  need(scale, "scale", at::kFloat, q.size(0), &p.dev);
  p.q = q.data_ptr<int8_t>();
  p.scale = scale.data_ptr<float>();
  if (given(a[6])) {
    const Tensor& b = tensor(a[6], "bias");
    need(b, "bias", at::kFloat, p.N, &p.dev);
    p.bias = b.data_ptr<float>();
  }
  if (given(a[7])) {
    if (!THPDtype_Check(a[7])) refuse("out_dtype must be a torch.dtype");
    p.y_type = reinterpret_cast<THPDtype*>(a[7])->scalar_type;
  }
  if (p.y_type != at::kFloat && p.y_type != at::kBFloat16) refuse("out_dtype must be float32 or bfloat16, got ", p.y_type);
  p.y_dtype = p.y_type == at::kFloat ? NF4_DTYPE_F32 : NF4_DTYPE_BF16;
  return p;
}
Tensor product_out(PyObject* o, const Product& p, int64_t M, bool& fill) {
  fill = !given(o);
  if (fill) return fresh({M, p.N}, p.y_type, p.dev);
  const Tensor& t = tensor(o, "out");
  dense(t, "out", M, p.N, p.y_type, p.dev);
  return t;
}

// (x, x_scale, q, scale, N, K, bias, out_dtype, out, ws)
PyObject* int8_matmul(PyObject* const* a) {
  no_derivatives({{"x", a[0]}, {"x_scale", a[1]}, {"scale", a[3]}, {"bias", a[6]}, {"out", a[8]}});
  const Product p = product_of(a, 1);
  bool fill;
  const Tensor out = product_out(a[8], p, p.rows, fill);
  const On on(p.dev);
  const Tensor ws = given(a[9]) ? given_workspace(a[9], p.dev)
                                : new_workspace(nf4_int8_workspace(p.x_dtype, p.rows, p.rows, p.N, p.K, 0), p.dev);
  const int st = nf4_int8_matmul(p.x, p.x_dtype, p.stride, p.x_scale, p.rows, p.q, p.scale, p.N, p.K, p.bias, out.data_ptr(), p.y_dtype,
                                 ptr(ws), ws.defined() ? ws.nbytes() : 0, on.stream);
  return st ? PyLong_FromLong(st) : wrap(out);
}

// (x, x_scale, q, scale, N, K, None, out_dtype, out, ws, offsets, E, tokens)
PyObject* int8_grouped(PyObject* const* a) {
  no_derivatives({{"x", a[0]}, {"x_scale", a[1]}, {"scale", a[3]}, {"out", a[8]}});
  const int32_t E = small(a[11], "E");
  if (E < 1) refuse("E must be at least 1, got ", E);
  const Product p = product_of(a, E);
  const Tensor& offsets = tensor(a[10], "offsets");
  need(offsets, "offsets", at::kInt, static_cast<int64_t>(E) + 1, &p.dev);
  const int32_t* tokens = nullptr;
  int64_t M = p.rows;
  if (given(a[12])) {
    const Tensor& t = tensor(a[12], "tokens");
    need(t, "tokens", at::kInt, -1, &p.dev);
    M = t.numel();
    tokens = t.data_ptr<int32_t>();
    if (M == 0) tokens = nullptr;
    else if (p.rows == 0) refuse("tokens name rows of an empty x");
  }
  bool fill;
  const Tensor out = product_out(a[8], p, M, fill);
  if (M == 0) return wrap(out);
  const On on(p.dev);
  const Tensor ws = given(a[9]) ? given_workspace(a[9], p.dev)
                                : new_workspace(nf4_int8_workspace(p.x_dtype, p.rows, M, p.N, p.K, E), p.dev);
  const int st = nf4_int8_grouped_matmul(p.x, p.x_dtype, p.stride, p.x_scale, p.rows, tokens, offsets.data_ptr<int32_t>(), E, M, p.q,
                                         p.scale, p.N, p.K, out.data_ptr(), p.y_dtype, fill, ptr(ws), ws.defined() ? ws.nbytes() : 0,
                                         on.stream);
  return st ? PyLong_FromLong(st) : wrap(out);
}

PyMethodDef methods[] = {
    method<route, 9>("route"),
    method<route_bwd, 7>("route_bwd"),
    method<expert_plan, 2>("expert_plan"),
    method<expert_gather, 4>("expert_gather"),
    method<expert_gather_bwd, 2>("expert_gather_bwd"),
    method<expert_combine, 5>("expert_combine"),
    method<expert_combine_bwd, 5>("expert_combine_bwd"),
    method<int8_quantize, 1>("int8_quantize"),
    method<int8_matmul, 10>("int8_matmul"),
    method<int8_grouped, 13>("int8_grouped"),
    {nullptr, nullptr, 0, nullptr},
};

}  // namespace

PyMethodDef* nf4_expert_methods() { return methods; }
