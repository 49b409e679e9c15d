// Argument marshalling of the attention calls (nf4_attn.h) for Python: checks of
// tensors, allocation of results and workspaces, the current stream of the
// tensors' device, the C call, and the autograd node of the prompt's attention.  The kernels of a decode step take a few
// microseconds, less than the same checks take in the interpreter.  Nothing
// here computes.
//
// Every function takes its arguments by position (attention.py names them) and
// returns the results, or the status of a C call that failed.
#include <Python.h>

#include <ATen/core/Tensor.h>
#include <ATen/ops/empty.h>
#include <c10/core/DeviceGuard.h>
#include <c10/hip/HIPStream.h>
#include <torch/csrc/Exceptions.h>
#include <torch/csrc/autograd/custom_function.h>
#include <torch/csrc/autograd/function.h>
#include <torch/csrc/autograd/python_variable.h>
#include <torch/csrc/autograd/variable.h>

#include <cmath>
#include <initializer_list>
#include <optional>
#include <sstream>
#include <stdexcept>
#include <string>
#include <utility>

#include "../../include/nf4_attn.h"

namespace {

using at::Tensor;

struct Refused : std::runtime_error {
  using std::runtime_error::runtime_error;
};
template <typename... A>
[[noreturn]] void refuse(const A&... a) {
  std::ostringstream s;
  (s << ... << a);
  throw Refused(s.str());
}

const Tensor& tensor(PyObject* o, const char* name) {
  if (!THPVariable_Check(o)) refuse(name, " must be a tensor");
  return THPVariable_Unpack(o);
}
bool given(PyObject* o) { return o != Py_None; }

long long integer(PyObject* o, const char* name) {
  const long long v = PyLong_AsLongLong(o);
  if (v == -1 && PyErr_Occurred()) {
    PyErr_Clear();
    refuse(name, " must be an integer");
  }
  return v;
}
bool truth(PyObject* o, const char* name) {
  const int t = PyObject_IsTrue(o);
  if (t < 0) {
    PyErr_Clear();
    refuse(name, " must be true or false");
  }
  return t == 1;
}

// No call has a forward derivative: a tangent would be lost without a word.
using Named = std::initializer_list<std::pair<const char*, PyObject*>>;
void no_tangents(const Named& inputs) {
  for (const auto& [name, o] : inputs)
    if (given(o) && tensor(o, name)._fw_grad(0).defined())
      refuse(name, " carries a forward-mode tangent, and this call has no forward derivative");
}

// Rotation and cache have no gradient either: an input that wants one is refused
// while gradients are recorded, not returned without its history.
void no_derivatives(const Named& inputs) {
  no_tangents(inputs);
  if (!at::GradMode::is_enabled()) return;
  for (const auto& [name, o] : inputs)
    if (given(o) && tensor(o, name).requires_grad())
      refuse(name, " requires a gradient, which this call does not carry: detach it, or call under torch.no_grad()");
}

void need(const Tensor& t, const char* name, at::ScalarType dtype, int64_t numel, const c10::Device* device) {
  if (!t.is_cuda()) refuse(name, " must be a device tensor");
  if (!t.is_contiguous()) refuse(name, " must be contiguous");
  if (t.scalar_type() != dtype) refuse(name, " must be ", dtype, ", got ", t.scalar_type());
  if (numel >= 0 && t.numel() != numel) refuse(name, " must have ", numel, " elements, got ", t.numel());
  if (device && t.device() != *device) refuse(name, " is on ", t.device(), ", expected ", *device);
}

struct Cache {
  c10::Device dev{c10::kCPU};
  int64_t P = 0;
  int32_t page = 0, H = 0, D = 0;
  uint8_t *kc = nullptr, *vc = nullptr;
  float *ks = nullptr, *vs = nullptr;
};
Cache cache_of(PyObject* const* a) {
  const Tensor &kc = tensor(a[0], "k_codes"), &ks = tensor(a[1], "k_scale"), &vc = tensor(a[2], "v_codes"),
               &vs = tensor(a[3], "v_scale");
  if (kc.dim() != 4) refuse("k_codes must be [pages, kv_heads, page, head_dim / 2]");
  const auto s = kc.sizes();
  if (s[3] != 32 && s[3] != 64) refuse("the cache's head_dim must be 64 or 128, got ", 2 * s[3]);
  if (s[2] < 16 || s[2] % 16 || s[2] > INT32_MAX) refuse("the cache's page must be a multiple of 16 tokens, got ", s[2]);
  if (s[1] < 1 || s[1] > 1024) refuse("the cache must have 1 to 1024 key heads, got ", s[1]);
  const c10::Device dev = kc.device();
  const int64_t n = kc.numel();
  need(kc, "k_codes", at::kByte, -1, nullptr);
  need(vc, "v_codes", at::kByte, n, &dev);
  need(ks, "k_scale", at::kFloat, n / 32, &dev);
  need(vs, "v_scale", at::kFloat, n / 32, &dev);
  return Cache{dev, s[0], static_cast<int32_t>(s[2]), static_cast<int32_t>(s[1]), static_cast<int32_t>(2 * s[3]),
               kc.data_ptr<uint8_t>(), vc.data_ptr<uint8_t>(), ks.data_ptr<float>(), vs.data_ptr<float>()};
}
#define CACHE_ARGS(c) c.kc, c.ks, c.vc, c.vs, c.P, c.page, c.H, c.D

struct Seqs {
  const int32_t *offsets = nullptr, *lengths = nullptr, *table = nullptr;
  int32_t B = 0, width = 0;
};
Seqs seqs_of(PyObject* lengths, PyObject* table, PyObject* offsets, int64_t rows, const c10::Device& dev) {
  const Tensor &ln = tensor(lengths, "lengths"), &pt = tensor(table, "page_table");
  need(ln, "lengths", at::kInt, -1, &dev);
  need(pt, "page_table", at::kInt, -1, &dev);
  if (ln.dim() != 1 || pt.dim() != 2 || pt.size(0) != ln.size(0)) refuse("lengths must be [B] and page_table [B, width]");
  if (ln.size(0) > INT32_MAX || pt.size(1) > INT32_MAX) refuse("lengths or page_table are too large");
  Seqs s{nullptr, ln.data_ptr<int32_t>(), pt.data_ptr<int32_t>(), static_cast<int32_t>(ln.size(0)),
         static_cast<int32_t>(pt.size(1))};
  if (given(offsets)) {
    const Tensor& off = tensor(offsets, "offsets");
    need(off, "offsets", at::kInt, s.B + 1, &dev);
    s.offsets = off.data_ptr<int32_t>();
  } else if (rows != s.B) {
    refuse("without offsets there is one row per sequence: ", rows, " rows, ", s.B, " sequences");
  }
  return s;
}
#define SEQ_ARGS(s) s.offsets, s.lengths, s.B, s.table, s.width

struct Rows {
  void* p = nullptr;
  int64_t stride = 0, T = 0;
  int32_t H = 0;
};
// A [T, heads, D] bf16 tensor whose rows may be strided.
Rows rows_of(const Tensor& t, const char* name, int64_t heads, int64_t D, int64_t T, const c10::Device& dev) {
  if (t.dim() != 3 || t.size(2) != D || (heads >= 0 && t.size(1) != heads))
    refuse(name, " must be [T, ", heads >= 0 ? std::to_string(heads) : "heads", ", ", D, "], got ", t.sizes());
  if (T >= 0 && t.size(0) != T) refuse(name, " has ", t.size(0), " rows, expected ", T);
  if (!t.is_cuda()) refuse(name, " must be a device tensor");
  if (t.scalar_type() != at::kBFloat16) refuse(name, " must be ", at::kBFloat16, ", got ", t.scalar_type());
  if (t.device() != dev) refuse(name, " is on ", t.device(), ", expected ", dev);
  if (t.size(1) > 1024) refuse(name, " has more than 1024 heads");
  Rows r{t.data_ptr(), 0, t.size(0), static_cast<int32_t>(t.size(1))};
  if (t.numel() == 0) return r;
  if (t.stride(2) != 1 || (r.H > 1 && t.stride(1) != D) || (r.T > 1 && t.stride(0) % 8))
    refuse(name, ": the heads of a row must be contiguous and rows a multiple of 8 elements apart");
  if (r.T > 1) r.stride = t.stride(0);
  return r;
}

Rows rows_of(PyObject* o, const char* name, int64_t heads, int64_t D, int64_t T, const c10::Device& dev) {
  return rows_of(tensor(o, name), name, heads, D, T, dev);
}

int32_t groups(int64_t Hq, int64_t H) {
  if (Hq < 1 || H < 1 || Hq % H) refuse(Hq, " query heads do not divide over ", H, " key heads");
  return static_cast<int32_t>(Hq);
}

Tensor fresh(at::IntArrayRef shape, at::ScalarType dtype, const c10::Device& dev) {
  return at::empty(shape, at::TensorOptions().dtype(dtype).device(dev));
}
// The caller's result tensor (rows outside every sequence are then left
// alone), or a new one (they are filled).
Tensor result(PyObject* o, const char* name, int64_t T, int64_t H, int64_t D, const c10::Device& dev, bool& fill) {
  fill = !given(o);
  if (fill) return fresh({T, H, D}, at::kBFloat16, dev);
  const Tensor& t = tensor(o, name);
  need(t, name, at::kBFloat16, T * H * D, &dev);
  return t;
}
Tensor new_workspace(size_t bytes, const c10::Device& dev) {
  if (bytes == SIZE_MAX) bytes = 0;                            // the call itself says why
  return bytes ? fresh({static_cast<int64_t>(bytes)}, at::kByte, dev) : Tensor();
}
Tensor given_workspace(PyObject* o, const c10::Device& dev) {
  const Tensor& t = tensor(o, "ws");
  if (!t.is_cuda()) refuse("ws must be a device tensor");
  if (!t.is_contiguous()) refuse("ws must be contiguous");
  if (t.device() != dev) refuse("ws is on ", t.device(), ", expected ", dev);
  return t;
}
void* ptr(const Tensor& t) { return t.defined() ? t.data_ptr() : nullptr; }

using Scale = std::optional<double>;
Scale scale_arg(PyObject* o) {
  if (!given(o)) return {};
  const double s = PyFloat_AsDouble(o);
  if (PyErr_Occurred()) {
    PyErr_Clear();
    refuse("scale must be a number");
  }
  return s;
}
float scale_of(const Scale& given_scale, int32_t D) {
  const double s = given_scale ? *given_scale : 1.0 / std::sqrt(static_cast<double>(D));
  const float f = static_cast<float>(s);
  if (!(f > 0.0f) || !std::isfinite(f)) refuse("scale must be positive and finite, got ", s);
  return f;
}

// The tensors' device is made current, its current stream takes the work.
struct On {
  c10::DeviceGuard guard;
  void* stream;
  explicit On(const c10::Device& dev) : guard(dev), stream(c10::hip::getCurrentHIPStream(dev.index()).stream()) {}
};

PyObject* wrap(const Tensor& t) {
  if (!t.defined()) Py_RETURN_NONE;
  return THPVariable_Wrap(t);
}
template <typename... T>
PyObject* several(const T&... t) {
  PyObject* out = PyTuple_New(sizeof...(t));
  if (!out) return nullptr;
  Py_ssize_t i = 0;
  for (const Tensor* x : {&t...}) {
    PyObject* w = wrap(*x);
    if (!w) {
      Py_DECREF(out);
      return nullptr;
    }
    PyTuple_SET_ITEM(out, i++, w);
  }
  return out;
}

// (k_codes, k_scale, v_codes, v_scale, k, v, lengths, page_table, offsets, inv_freq, interleaved, q, return_k, q_out, k_out)
PyObject* kv_append(PyObject* const* a) {
  no_derivatives({{"k_scale", a[1]}, {"v_scale", a[3]}, {"k", a[4]}, {"v", a[5]}, {"inv_freq", a[9]}, {"q", a[11]}});
  const Cache c = cache_of(a);
  const Rows k = rows_of(a[4], "k", c.H, c.D, -1, c.dev), v = rows_of(a[5], "v", c.H, c.D, k.T, c.dev);
  const Seqs s = seqs_of(a[6], a[7], a[8], k.T, c.dev);
  const float* inv = nullptr;
  const bool interleaved = truth(a[10], "interleaved");
  int64_t rotary = 0;
  if (given(a[9])) {
    const Tensor& f = tensor(a[9], "inv_freq");
    need(f, "inv_freq", at::kFloat, -1, &c.dev);
    rotary = 2 * f.numel();
    if (rotary > c.D || rotary % 16)
      refuse("inv_freq must have a multiple of 8 elements, at most ", c.D / 2, ", got ", f.numel());
    inv = f.data_ptr<float>();
  }
  Rows q;
  Tensor q_out, k_out;
  bool fill = true;
  int32_t Hq = c.H;
  if (given(a[11])) {
    q = rows_of(a[11], "q", -1, c.D, k.T, c.dev);
    Hq = groups(q.H, c.H);
    q_out = result(a[13], "q_out", k.T, Hq, c.D, c.dev, fill);
  } else if (given(a[13])) {
    refuse("q_out without q");
  }
  if (truth(a[12], "return_k") || given(a[14])) {
    bool kfill;
    k_out = result(a[14], "k_out", k.T, c.H, c.D, c.dev, kfill);
    if (given(a[11]) && kfill != fill) refuse("pass both of q_out and k_out, or neither");
    fill = kfill;
  }
  const On on(c.dev);
  const int st = nf4_kv_append(q.p, q.stride, k.p, k.stride, v.p, v.stride, k.T, Hq, SEQ_ARGS(s), inv,
                               static_cast<int32_t>(rotary), interleaved, CACHE_ARGS(c), ptr(q_out), ptr(k_out), fill,
                               on.stream);
  return st ? PyLong_FromLong(st) : several(q_out, k_out);
}

// (k_codes, k_scale, v_codes, v_scale, lengths, page_table, offsets, rows, k_out, v_out)
PyObject* kv_dequantize(PyObject* const* a) {
  no_derivatives({{"k_scale", a[1]}, {"v_scale", a[3]}});
  const Cache c = cache_of(a);
  int64_t T;
  if (given(a[7])) {
    T = integer(a[7], "rows");
    if (T < 0) refuse("rows must not be negative, got ", T);
  } else {
    if (given(a[6])) refuse("with offsets, pass the number of rows");
    T = tensor(a[4], "lengths").numel();
  }
  const Seqs s = seqs_of(a[4], a[5], a[6], T, c.dev);
  if (given(a[8]) != given(a[9])) refuse("pass both of k_out and v_out, or neither");
  bool fill;
  const Tensor k_out = result(a[8], "k_out", T, c.H, c.D, c.dev, fill), v_out = result(a[9], "v_out", T, c.H, c.D, c.dev, fill);
  const On on(c.dev);
  const int st = nf4_kv_dequantize(T, SEQ_ARGS(s), CACHE_ARGS(c), ptr(k_out), ptr(v_out), fill, on.stream);
  return st ? PyLong_FromLong(st) : several(k_out, v_out);
}

// (k_codes, k_scale, v_codes, v_scale, q, lengths, page_table, offsets, scale, out, ws)
PyObject* kv_attention(PyObject* const* a) {
  no_derivatives({{"k_scale", a[1]}, {"v_scale", a[3]}, {"q", a[4]}});
  const Cache c = cache_of(a);
  const Rows q = rows_of(a[4], "q", -1, c.D, -1, c.dev);
  const int32_t Hq = groups(q.H, c.H);
  const Seqs s = seqs_of(a[5], a[6], a[7], q.T, c.dev);
  const float scale = scale_of(scale_arg(a[8]), c.D);
  bool fill;
  const Tensor out = result(a[9], "out", q.T, Hq, c.D, c.dev, fill);
  const On on(c.dev);
  const Tensor ws = given(a[10]) ? given_workspace(a[10], c.dev)
                                 : new_workspace(nf4_kv_attention_workspace(q.T, s.B, Hq, c.H, c.D, s.width, c.page), c.dev);
  const int st = nf4_kv_attention(q.p, q.stride, q.T, Hq, SEQ_ARGS(s), CACHE_ARGS(c), scale, ptr(out), fill, ptr(ws),
                                  ws.defined() ? ws.nbytes() : 0, on.stream);
  return st ? PyLong_FromLong(st) : wrap(out);
}

struct Prompt {
  c10::Device dev{c10::kCPU};
  Rows q, k, v;
  int32_t B = 0, D = 0;
  const int32_t* offsets = nullptr;
  float scale = 0.0f;
};
Prompt prompt_of(const Tensor& q, const Tensor& k, const Tensor& v, const Tensor& offsets, const Scale& scale) {
  Prompt p;
  if (q.dim() != 3 || (q.size(2) != 64 && q.size(2) != 128)) refuse("q must be [T, Hq, D] with D 64 or 128, got ", q.sizes());
  p.dev = q.device();
  p.D = static_cast<int32_t>(q.size(2));
  p.q = rows_of(q, "q", -1, p.D, -1, p.dev);
  p.k = rows_of(k, "k", -1, p.D, p.q.T, p.dev);
  p.v = rows_of(v, "v", p.k.H, p.D, p.q.T, p.dev);
  groups(p.q.H, p.k.H);
  need(offsets, "offsets", at::kInt, -1, &p.dev);
  if (offsets.dim() != 1 || offsets.numel() < 1 || offsets.numel() > INT32_MAX) refuse("offsets must be [B + 1]");
  p.B = static_cast<int32_t>(offsets.numel() - 1);
  p.offsets = offsets.data_ptr<int32_t>();
  p.scale = scale_of(scale, p.D);
  return p;
}
#define PROMPT_ARGS(p) p.q.p, p.q.stride, p.k.p, p.k.stride, p.v.p, p.v.stride

int run_forward(const Prompt& p, const Tensor& out, const Tensor& rest, const Tensor& lse, bool fill) {
  const On on(p.dev);
  return nf4_prompt_attention_fwd(PROMPT_ARGS(p), p.q.T, p.offsets, p.B, p.q.H, p.k.H, p.D, p.scale, ptr(out), ptr(rest),
                                  static_cast<float*>(ptr(lse)), fill, on.stream);
}
struct Grads {
  Tensor q, k, v;
};
int run_backward(const Prompt& p, const Tensor& grad_out, const Tensor& out, const Tensor& rest, const Tensor& lse, PyObject* ws_arg,
             Grads& grads) {
  const int64_t T = p.q.T, n = T * p.q.H * p.D;
  const Rows g = rows_of(grad_out, "grad_out", p.q.H, p.D, T, p.dev);
  need(out, "out", at::kBFloat16, n, &p.dev);
  if (rest.defined()) need(rest, "out_rest", at::kBFloat16, n, &p.dev);
  need(lse, "lse", at::kFloat, T * p.q.H, &p.dev);
  grads = Grads{fresh({T, p.q.H, p.D}, at::kBFloat16, p.dev), fresh({T, p.k.H, p.D}, at::kBFloat16, p.dev),
                fresh({T, p.k.H, p.D}, at::kBFloat16, p.dev)};
  const On on(p.dev);
  const bool own = !ws_arg || !given(ws_arg);
  const size_t bytes = nf4_prompt_attention_bwd_workspace(T, p.B, p.q.H, p.k.H, p.D);
  const Tensor ws = own ? new_workspace(bytes, p.dev) : given_workspace(ws_arg, p.dev);
  return nf4_prompt_attention_bwd(g.p, g.stride, PROMPT_ARGS(p), out.data_ptr(), ptr(rest), lse.data_ptr<float>(), T,
                                  p.offsets, p.B, p.q.H, p.k.H, p.D, p.scale, ptr(grads.q), ptr(grads.k), ptr(grads.v), 1,
                                  ptr(ws), ws.defined() ? ws.nbytes() : 0, on.stream);
}

// (q, k, v, offsets, scale, out, for_backward)
PyObject* prompt_fwd(PyObject* const* a) {
  no_tangents({{"q", a[0]}, {"k", a[1]}, {"v", a[2]}});
  const Prompt p = prompt_of(tensor(a[0], "q"), tensor(a[1], "k"), tensor(a[2], "v"), tensor(a[3], "offsets"), scale_arg(a[4]));
  bool fill;
  const Tensor out = result(a[5], "out", p.q.T, p.q.H, p.D, p.dev, fill);
  Tensor rest, lse;
  const bool keep = truth(a[6], "for_backward");
  if (keep) {
    rest = fresh({p.q.T, p.q.H, p.D}, at::kBFloat16, p.dev);
    lse = fresh({p.q.H, p.q.T}, at::kFloat, p.dev);
  }
  const int st = run_forward(p, out, rest, lse, fill);
  if (st) return PyLong_FromLong(st);
  return keep ? several(out, rest, lse) : wrap(out);
}

// (grad_out, q, k, v, out, out_rest, lse, offsets, scale, ws)
PyObject* prompt_bwd(PyObject* const* a) {
  no_tangents({{"grad_out", a[0]}, {"q", a[1]}, {"k", a[2]}, {"v", a[3]}, {"out", a[4]}, {"out_rest", a[5]}, {"lse", a[6]}});
  const Prompt p = prompt_of(tensor(a[1], "q"), tensor(a[2], "k"), tensor(a[3], "v"), tensor(a[7], "offsets"), scale_arg(a[8]));
  Grads g;
  const int st = run_backward(p, tensor(a[0], "grad_out"), tensor(a[4], "out"), given(a[5]) ? tensor(a[5], "out_rest") : Tensor(),
                          tensor(a[6], "lse"), a[9], g);
  return st ? PyLong_FromLong(st) : several(g.q, g.k, g.v);
}

// t [T, heads, D] as the kernels take it: bf16, the heads of a row contiguous,
// rows 16-byte aligned and at most 2^24 elements apart.
Tensor head_rows(const Tensor& t) {
  const Tensor x = t.scalar_type() == at::kBFloat16 ? t : t.to(at::kBFloat16);
  if (x.dim() != 3 || x.numel() == 0) return x;
  const bool fits = x.stride(2) == 1 && (x.size(1) == 1 || x.stride(1) == x.size(2)) &&
                    (x.size(0) == 1 || (x.stride(0) % 8 == 0 && x.stride(0) <= 1 << 24)) && reinterpret_cast<uintptr_t>(x.data_ptr()) % 16 == 0;
  return fits ? x : x.clone(at::MemoryFormat::Contiguous);
}
// Raises a failed C call as the package does (NF4Error with its status), from
// autograd's thread too.
void ok(int status, const char* name) {
  if (!status) return;
  const PyGILState_STATE gil = PyGILState_Ensure();
  PyObject* lib = PyImport_ImportModule("nf4_bit_weight_amd._lib");
  PyObject* none = lib ? PyObject_CallMethod(lib, "check", "si", name, status) : nullptr;
  Py_XDECREF(none);
  Py_XDECREF(lib);
  python_error e;
  e.persist();
  PyGILState_Release(gil);
  throw e;
}

// Causal attention over packed sequences, differentiable in q, k and v.  Saved
// are the bf16 operands, the output with what its rounding took, and each
// row's log-sum-exp: tensors only, through save_for_backward, so that saved-tensor
// hooks and activation checkpointing see them.  (A node in C++: its backward
// runs on autograd's thread without the interpreter.)
struct PromptAttention : torch::autograd::Function<PromptAttention> {
  static Tensor forward(torch::autograd::AutogradContext* ctx, const Tensor& q, const Tensor& k, const Tensor& v,
                        const Tensor& offsets, double scale) {
    const Tensor q2 = head_rows(q), k2 = head_rows(k), v2 = head_rows(v);
    const Prompt p = prompt_of(q2, k2, v2, offsets, scale);
    // refused here, not in a backward pass that cannot start
    if (nf4_prompt_attention_bwd_workspace(p.q.T, p.B, p.q.H, p.k.H, p.D) == SIZE_MAX)
      ok(NF4_ERR_UNSUPPORTED, "nf4_prompt_attention_bwd");
    const Tensor out = fresh({p.q.T, p.q.H, p.D}, at::kBFloat16, p.dev), rest = fresh({p.q.T, p.q.H, p.D}, at::kBFloat16, p.dev),
                 lse = fresh({p.q.H, p.q.T}, at::kFloat, p.dev);
    ok(run_forward(p, out, rest, lse, true), "nf4_prompt_attention_fwd");
    ctx->save_for_backward({q2, k2, v2, out, rest, lse, offsets});
    ctx->saved_data["scale"] = scale;
    ctx->saved_data["q"] = q.scalar_type();
    ctx->saved_data["k"] = k.scalar_type();
    ctx->saved_data["v"] = v.scalar_type();
    return out.to(q.scalar_type());
  }
  static torch::autograd::variable_list backward(torch::autograd::AutogradContext* ctx, torch::autograd::variable_list grad) {
    if (at::GradMode::is_enabled())
      throw std::runtime_error("nf4_prompt_attention: its backward pass is not differentiable (create_graph)");
    if (grad[0].defined() && grad[0]._fw_grad(0).defined())
      throw std::runtime_error("nf4_prompt_attention: grad_out carries a forward-mode tangent, and the backward pass has no forward derivative");
    const auto s = ctx->get_saved_variables();
    const Prompt p = prompt_of(s[0], s[1], s[2], s[6], ctx->saved_data["scale"].toDouble());
    Grads g;
    ok(run_backward(p, head_rows(grad[0]), s[3], s[4], s[5], nullptr, g), "nf4_prompt_attention_bwd");
    auto as = [&](const char* name, const Tensor& x, int i) {
      return ctx->needs_input_grad(i) ? x.to(ctx->saved_data[name].toScalarType()) : Tensor();
    };
    return {as("q", g.q, 0), as("k", g.k, 1), as("v", g.v, 2), Tensor(), Tensor()};
  }
};

// While a graph is being captured, the gradients of leaves go through their
// accumulators.  One that a living eager graph made belongs to the eager stream,
// and autograd would make that stream wait inside the capture, which ends it,
// and the process with it.  So such a leaf is refused here, in the forward call.
void check_capture(std::initializer_list<std::pair<const char*, const Tensor*>> inputs, const c10::Device& dev) {
  const auto now = c10::hip::getCurrentHIPStream(dev.index());
  hipStreamCaptureStatus status = hipStreamCaptureStatusNone;
  if (hipStreamIsCapturing(now.stream(), &status) != hipSuccess || status != hipStreamCaptureStatusActive) return;
  for (const auto& [name, t] : inputs) {
    if (!t->requires_grad() || !t->is_leaf()) continue;
    const auto acc = torch::autograd::impl::try_get_grad_accumulator(*t);
    const auto stream = acc ? acc->stream() : std::nullopt;
    if (stream && stream->id() != now.id())
      refuse(name, " is captured while an eager graph of the same leaf lives: drop that graph first, or pass a detached leaf");
  }
}

// (q, k, v, offsets, scale): any floating dtype and layout, differentiable
PyObject* prompt_attention(PyObject* const* a) {
  no_tangents({{"q", a[0]}, {"k", a[1]}, {"v", a[2]}});
  const Tensor &q = tensor(a[0], "q"), &k = tensor(a[1], "k"), &v = tensor(a[2], "v"), &offsets = tensor(a[3], "offsets");
  for (const Tensor* t : {&q, &k, &v})
    if (!t->is_cuda()) refuse("q, k and v must be device tensors");
  if (q.dim() != 3) refuse("q must be [T, Hq, D] with D 64 or 128, got ", q.sizes());
  const Scale given_scale = scale_arg(a[4]);
  if (at::GradMode::is_enabled() && (q.requires_grad() || k.requires_grad() || v.requires_grad())) {
    check_capture({{"q", &q}, {"k", &k}, {"v", &v}}, q.device());
    const double scale = given_scale ? *given_scale : 1.0 / std::sqrt(static_cast<double>(q.size(2)));
    return wrap(PromptAttention::apply(q, k, v, offsets, scale));
  }
  const Tensor q2 = head_rows(q), k2 = head_rows(k), v2 = head_rows(v);
  const Prompt p = prompt_of(q2, k2, v2, offsets, given_scale);
  const Tensor out = fresh({p.q.T, p.q.H, p.D}, at::kBFloat16, p.dev);
  const int st = run_forward(p, out, Tensor(), Tensor(), true);
  return st ? PyLong_FromLong(st) : wrap(out.to(q.scalar_type()));
}

template <PyObject* (*F)(PyObject* const*), int N>
PyObject* call(PyObject*, PyObject* const* args, Py_ssize_t n) {
  if (n != N) {
    PyErr_Format(PyExc_TypeError, "%d arguments expected, got %zd", N, n);
    return nullptr;
  }
  HANDLE_TH_ERRORS                                             // torch's own: out of memory, no device
  try {
    return F(args);
  } catch (const Refused& e) {
    PyErr_SetString(PyExc_ValueError, e.what());
    return nullptr;
  }
  END_HANDLE_TH_ERRORS
}
template <PyObject* (*F)(PyObject* const*), int N>
PyMethodDef method(const char* name) {
  return {name, reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(&call<F, N>)), METH_FASTCALL, nullptr};
}

PyMethodDef methods[] = {
    method<kv_append, 15>("kv_append"),   method<kv_dequantize, 10>("kv_dequantize"),
    method<kv_attention, 11>("kv_attention"), method<prompt_fwd, 7>("prompt_fwd"),
    method<prompt_bwd, 10>("prompt_bwd"), method<prompt_attention, 5>("prompt_attention"), {nullptr, nullptr, 0, nullptr},
};
PyModuleDef module = {PyModuleDef_HEAD_INIT, "_nf4_torch", nullptr, -1, methods, nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__nf4_torch() { return PyModule_Create(&module); }
