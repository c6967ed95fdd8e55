// The layers as torch operations: checks of tensors, allocation, the autograd
// nodes and the calls of the C ABI (include/shampoo.h).  In C++ because a small
// layer's time is the host's: autograd runs a backward pass on a thread of its
// own, where Python costs twice what it does on the caller's.  Forward and
// backward of small fp32 matrices, bound by the host, with nodes in Python -> here:
// 1001 x 1537 activation 87 -> 43 us (torch's own silu takes 41), 333 x 1001 LayerNorm
// 137 -> 51 to 78, 1001 x 1537 join 200 -> 99 to 120, of which its kernels take 37; the
// host's part varies from box to box.
#include <ATen/ATen.h>
#include <ATen/hip/impl/HIPStreamMasqueradingAsCUDA.h>
#include <c10/core/DeviceGuard.h>
#include <c10/core/impl/TorchDispatchModeTLS.h>
#include <c10/hip/HIPStream.h>
#include <torch/csrc/autograd/custom_function.h>
#include <torch/csrc/jit/frontend/tracer.h>
#include <torch/csrc/utils/pybind.h>

#include <cmath>
#include <optional>
#include <sstream>

#include "../../include/shampoo.h"

namespace py = pybind11;
using at::Tensor;
using torch::autograd::AutogradContext;
using torch::autograd::variable_list;
using OptTensor = std::optional<Tensor>;

namespace {

template <class... T>
[[noreturn]] void refuse(const T&... parts) {
  std::ostringstream s;
  (s << ... << parts);
  throw py::value_error(s.str());
}

// Raises capi.ShampooError (callers' threads; the backward pass's raise RuntimeError).
void check(int rc, const char* where) {
  if (rc == SHAMPOO_OK) return;
  py::gil_scoped_acquire gil;
  py::module_::import("inverse_root_preconditioning_amd.capi").attr("check")(rc, where);
}
void check_backward(int rc, const char* where) {
  TORCH_CHECK(rc == SHAMPOO_OK, where, ": ", shampoo_strerror(rc), " (code ", rc, ")");
}

// A trace would hold the allocation of the outputs and not the call that fills them.
void refuse_trace() {
  using c10::impl::TorchDispatchModeKey;
  if (!torch::jit::tracer::isTracing() &&
      !c10::impl::TorchDispatchModeTLS::get_mode(TorchDispatchModeKey::PROXY).has_value())
    return;
  py::gil_scoped_acquire gil;
  PyErr_SetString(PyExc_NotImplementedError, "the layers cannot be recorded in a trace");
  throw py::error_already_set();
}

int type_of(const Tensor& t) {
  if (t.scalar_type() == at::kFloat) return SHAMPOO_T_F32;
  return t.scalar_type() == at::kBFloat16 ? SHAMPOO_T_BF16 : -1;
}

int checked_type(const Tensor& t, const char* name) {
  const int type = type_of(t);
  if (type < 0 || !t.is_cuda()) refuse(name, " must be a float32 or bfloat16 CUDA tensor");
  if (t.dim() == 0) refuse(name, " must have a dimension");
  return type;
}

hipStream_t stream_of(const Tensor& t) { return c10::hip::getCurrentHIPStream(t.get_device()).stream(); }

int64_t padded(int64_t cols) { return (cols + 31) / 32 * 32; }
// Codes and scales of an MX8 matrix, rounded up so that another may follow.
int64_t mx8_bytes(int64_t rows, int64_t cols) {
  const int64_t n = rows * padded(cols);
  return (n + n / 32 + 15) / 16 * 16;
}
struct Copy {
  uint8_t *codes = nullptr, *scales = nullptr;
};
Copy copy_at(const Tensor& buf, int64_t index, int64_t rows, int64_t cols) {
  Copy c;
  c.codes = static_cast<uint8_t*>(buf.data_ptr()) + index * mx8_bytes(rows, cols);
  c.scales = c.codes + rows * padded(cols);
  return c;
}

// A tensor's memory.  One that only stands for others (a wrapper subclass) has none, and an address of 0 would
// say that the argument is not there.
void* memory_of(const Tensor& t) {
  void* const p = t.data_ptr();
  if (p == nullptr && t.numel() > 0) refuse("a tensor without memory of its own (a wrapper of others)");
  return p;
}

// A tensor as a matrix of evenly spaced rows of its last dimension: itself or a copy.
struct Rows {
  Tensor t;
  int64_t ld = 0;
  void* ptr() const { return memory_of(t); }
};
Rows rows_of(const Tensor& t) {
  if (t.is_neg()) return rows_of(t.resolve_neg());  // a view that negates what is in memory
  const int64_t n = t.dim();
  if (t.is_contiguous()) return {t, t.size(-1)};
  if (n > 1 && t.numel() > 0 && t.stride(-1) == 1 && t.stride(-2) >= t.size(-1)) {
    bool even = true;
    for (int64_t i = n - 2; i > 0 && even; --i) even = t.stride(i - 1) == t.stride(i) * t.size(i);
    if (even) return {t, t.stride(-2)};
  }
  return {t.contiguous(), t.size(-1)};
}

int64_t lead(at::IntArrayRef sizes) {
  int64_t n = 1;
  for (size_t i = 0; i + 1 < sizes.size(); ++i) n *= sizes[i];
  return n;
}

bool wants_gradient(std::initializer_list<const OptTensor*> tensors) {
  if (!at::GradMode::is_enabled()) return false;
  for (const OptTensor* t : tensors)
    if (t->has_value() && (*t)->requires_grad()) return true;
  return false;
}

Tensor or_undefined(const OptTensor& t) { return t ? *t : Tensor(); }

// In a backward pass that is captured into a graph: a gradient that goes on to a node of another stream
// (the accumulator of a leaf of which a graph from before the capture still lives) would
// make that stream wait for the captured one, in autograd's own thread, which ends the process.
void check_captured(const Tensor& given) {
  const hipStream_t now = stream_of(given);
  hipStreamCaptureStatus status;
  auto captured = [&](hipStream_t s) {  // the default stream cannot be, nor be asked during another's capture
    return s != nullptr && hipStreamIsCapturing(s, &status) == hipSuccess && status != hipStreamCaptureStatusNone;
  };
  if (!captured(now)) return;
  const auto node = torch::autograd::get_current_node();
  if (node == nullptr) return;
  for (const auto& edge : node->next_edges()) {
    const auto to = edge.function ? edge.function->stream() : std::nullopt;
    TORCH_CHECK(!to || to->device_index() != given.get_device() ||
                    captured(c10::hip::HIPStreamMasqueradingAsCUDA(*to).stream()),
                "a graph of these tensors from before the capture still lives: free it (its outputs), or capture "
                "the backward pass on its stream");
  }
}

// A gradient that is asked for with create_graph: differentiating it again is an
// error instead of a graph that lacks this layer.
struct Once : torch::autograd::Function<Once> {
  static Tensor forward(AutogradContext*, const Tensor&, const Tensor& gradient) { return gradient.view_as(gradient); }
  static variable_list backward(AutogradContext*, variable_list) {
    TORCH_CHECK(false, "the layers form no gradients of gradients");
  }
};
variable_list finish(variable_list out) {
  if (at::GradMode::is_enabled()) {
    for (Tensor& t : out)
      if (t.defined()) t = Once::apply(at::zeros({1}, t.options()).requires_grad_(), t);
  }
  return out;
}

// ---------------------------------------------------------------------------
// Activations
// ---------------------------------------------------------------------------

struct ActState : torch::CustomClassHolder {
  int act = 0, type = 0;
  bool packed = false, gated = false, low = false;
  std::vector<int64_t> shape;
  int64_t rows = 0, cols = 0;
};

std::pair<Tensor, Tensor> act_forward(const ActState& s, const Tensor& a, const OptTensor& b, bool low) {
  const c10::DeviceGuard guard(a.device());
  std::vector<int64_t> sizes = s.shape;
  sizes.back() = s.cols;
  Tensor y = at::empty(sizes, a.options()), buf;
  const bool any = s.rows > 0 && s.cols > 0;
  if (low) buf = at::empty({(s.gated ? 2 : 1) * mx8_bytes(s.rows, s.cols)}, a.options().dtype(at::kByte));
  if (!any) return {y, buf};
  const Rows ra = rows_of(a);
  Rows rb;
  const void* pb = nullptr;
  if (s.packed) {
    pb = static_cast<const uint8_t*>(ra.ptr()) + s.cols * a.element_size();
    rb.ld = ra.ld;
  } else if (b) {
    rb = rows_of(*b);
    pb = rb.ptr();
  }
  Copy ca, cb;
  if (low) {
    ca = copy_at(buf, 0, s.rows, s.cols);
    if (s.gated) cb = copy_at(buf, 1, s.rows, s.cols);
  }
  check(shampoo_activation(s.act, ra.ptr(), ra.ld, pb, rb.ld, s.rows, s.cols, s.type, y.data_ptr(), s.cols, ca.codes,
                           ca.scales, cb.codes, cb.scales, stream_of(a)),
        "shampoo_activation");
  return {y, buf};
}

struct Activation : torch::autograd::Function<Activation> {
  static Tensor forward(AutogradContext* ctx, const Tensor& a, const OptTensor& b, c10::intrusive_ptr<ActState> s) {
    auto [y, buf] = act_forward(*s, a, b, s->low);
    if (s->low) {
      ctx->save_for_backward({buf});
    } else {
      ctx->save_for_backward({a, or_undefined(b)});
    }
    ctx->saved_data["state"] = c10::IValue::make_capsule(s);
    return y;
  }

  static variable_list backward(AutogradContext* ctx, variable_list grads) {
    const auto held = ctx->saved_data["state"].toCapsule();
    const ActState& s = static_cast<const ActState&>(*held);
    const variable_list saved = ctx->get_saved_variables();
    const Tensor& given = grads[0];
    const c10::DeviceGuard guard(given.device());
    check_captured(given);
    const bool need_a = ctx->needs_input_grad(0), need_b = s.gated && !s.packed && ctx->needs_input_grad(1);
    variable_list out(3);
    if (need_a) out[0] = at::empty(s.shape, given.options());
    if (need_b) out[1] = at::empty(s.shape, given.options());
    if (s.rows > 0 && s.cols > 0) {
      const Rows dy = rows_of(given);
      Rows a, b;
      const void *pa = nullptr, *pb = nullptr;
      Copy ca, cb;
      if (s.low) {
        ca = copy_at(saved[0], 0, s.rows, s.cols);
        if (s.gated) cb = copy_at(saved[0], 1, s.rows, s.cols);
      } else {
        a = rows_of(saved[0]);
        pa = a.ptr();
        if (s.packed) {
          pb = static_cast<const uint8_t*>(pa) + s.cols * given.element_size();
          b.ld = a.ld;
        } else if (s.gated) {
          b = rows_of(saved[1]);
          pb = b.ptr();
        }
      }
      const int64_t ld = s.shape.back();
      void* const da = need_a ? out[0].data_ptr() : nullptr;
      void* const db = s.packed ? static_cast<uint8_t*>(da) + s.cols * given.element_size()
                       : need_b ? out[1].data_ptr()
                                : nullptr;
      check_backward(shampoo_activation_backward(s.act, dy.ptr(), dy.ld, pa, a.ld, pb, b.ld, ca.codes, ca.scales,
                                                 cb.codes, cb.scales, s.gated, s.rows, s.cols, s.type, da, ld, db, ld,
                                                 stream_of(given)),
                     "shampoo_activation_backward");
    }
    return finish(std::move(out));
  }
};

Tensor activate(const Tensor& a, const OptTensor& b, bool packed, int64_t act, bool low) {
  refuse_trace();
  auto s = c10::make_intrusive<ActState>();
  s->type = checked_type(a, "x");
  s->act = (int)act;
  s->packed = packed;
  s->gated = packed || b.has_value();
  s->low = low;
  s->shape = a.sizes().vec();
  const int64_t width = a.size(-1);
  if (packed && width % 2 != 0) refuse("x has ", width, " columns: two halves are needed");
  if (b && (b->sizes() != a.sizes() || b->scalar_type() != a.scalar_type() || b->device() != a.device()))
    refuse("x and b differ in shape, type or device");
  s->cols = packed ? width / 2 : width;
  s->rows = lead(a.sizes());
  const OptTensor x = a;
  if (wants_gradient({&x, &b})) return Activation::apply(a, b, s);
  return act_forward(*s, a, b, false).first;
}

// ---------------------------------------------------------------------------
// Norms and joins
// ---------------------------------------------------------------------------

enum { kR, kY, kW1, kB1, kGate, kW2, kB2, kInputs };

struct JoinState : torch::CustomClassHolder {
  std::vector<int64_t> shape;
  shampoo_join j = {};  // without addresses
  bool join = false, low = false, keep_r = false, keep_y = false;
  at::ScalarType stream_type, branch_type;
  int edge[kInputs];  // which of autograd's inputs each is (-1: not given)
};

struct Inputs {
  Tensor t[kInputs];
};

// Parameters, dense, with their addresses in the description.
void place_parameters(shampoo_join& j, Inputs& in) {
  auto place = [&](int i, const void*& ptr, int64_t& type) {
    if (!in.t[i].defined()) return;
    if (!in.t[i].is_contiguous() || in.t[i].is_neg()) in.t[i] = in.t[i].resolve_neg().contiguous();
    ptr = memory_of(in.t[i]);
    type = type_of(in.t[i]);
  };
  place(kW1, j.after.weight, j.after.weight_dtype);
  place(kB1, j.after.bias, j.after.bias_dtype);
  place(kGate, j.gate, j.gate_dtype);
  place(kW2, j.before.weight, j.before.weight_dtype);
  place(kB2, j.before.bias, j.before.bias_dtype);
}

void place_kept(shampoo_join& j, const JoinState& s, const Tensor& buf, const Tensor& stats) {
  if (buf.defined()) {
    int64_t i = 0;
    if (s.keep_r) {
      const Copy c = copy_at(buf, i++, j.rows, j.cols);
      j.residual_codes = c.codes;
      j.residual_scales = c.scales;
    }
    if (s.keep_y) {
      const Copy c = copy_at(buf, i, j.rows, j.cols);
      j.branch_codes = c.codes;
      j.branch_scales = c.scales;
    }
  }
  if (stats.defined()) {
    float* p = static_cast<float*>(stats.data_ptr());
    if (j.after.kind != SHAMPOO_NORM_NONE) {
      j.after_stats = p;
      p += 2 * j.rows;
    }
    if (j.before.kind != SHAMPOO_NORM_NONE) j.before_stats = p;
  }
}

struct Kept {
  Tensor h, u, buf, stats;
};

Kept join_forward(const JoinState& s, Inputs in, bool keep) {
  const Tensor& residual = in.t[kR];
  const c10::DeviceGuard guard(residual.device());
  Kept k;
  shampoo_join j = s.j;
  const bool n1 = j.after.kind != SHAMPOO_NORM_NONE, n2 = j.before.kind != SHAMPOO_NORM_NONE;
  if (s.join) k.h = at::empty(s.shape, residual.options());
  if (n2) k.u = at::empty(s.shape, residual.options().dtype(s.branch_type));
  if (keep) {
    // as bytes: what rounds saved tensors of floating point leaves them alone
    if (n1 || n2) k.stats = at::empty({((int)n1 + (int)n2) * j.rows * 8}, residual.options().dtype(at::kByte));
    if (s.low && (s.keep_r || s.keep_y))
      k.buf = at::empty({((int)s.keep_r + (int)s.keep_y) * mx8_bytes(j.rows, j.cols)}, residual.options().dtype(at::kByte));
  }
  if (j.rows == 0 || j.cols == 0) return k;
  place_parameters(j, in);
  const Rows r = rows_of(residual);
  j.residual = r.ptr();
  j.ld_residual = r.ld;
  Rows y;
  if (s.join) {
    y = rows_of(in.t[kY]);
    j.branch = y.ptr();
    j.ld_branch = y.ld;
  }
  place_kept(j, s, k.buf, k.stats);
  check(shampoo_join_forward(&j, s.join ? k.h.data_ptr() : nullptr, j.cols, n2 ? k.u.data_ptr() : nullptr, j.cols,
                             stream_of(residual)),
        "shampoo_join_forward");
  return k;
}

struct Join : torch::autograd::Function<Join> {
  static variable_list forward(AutogradContext* ctx, const Tensor& r, const OptTensor& y, const OptTensor& w1,
                               const OptTensor& b1, const OptTensor& gate, const OptTensor& w2, const OptTensor& b2,
                               c10::intrusive_ptr<JoinState> s) {
    const Inputs in = {{r, or_undefined(y), or_undefined(w1), or_undefined(b1), or_undefined(gate), or_undefined(w2),
                        or_undefined(b2)}};
    const Kept k = join_forward(*s, in, true);
    variable_list saved(in.t, in.t + kInputs);
    if (s->low || !s->keep_r) saved[kR] = Tensor();
    if (s->low || !s->keep_y) saved[kY] = Tensor();
    saved.push_back(k.buf);
    saved.push_back(k.stats);
    ctx->save_for_backward(std::move(saved));
    ctx->set_materialize_grads(false);
    int n = 0;
    for (int i = 0; i < kInputs; ++i) s->edge[i] = in.t[i].defined() ? n++ : -1;
    ctx->saved_data["state"] = c10::IValue::make_capsule(s);
    variable_list out;
    if (k.h.defined()) out.push_back(k.h);
    if (k.u.defined()) out.push_back(k.u);
    return out;
  }

  static variable_list backward(AutogradContext* ctx, variable_list grads) {
    const auto held = ctx->saved_data["state"].toCapsule();
    const JoinState& s = static_cast<const JoinState&>(*held);
    variable_list out(kInputs + 1);
    shampoo_join j = s.j;
    const bool n2 = j.before.kind != SHAMPOO_NORM_NONE;
    const Tensor dh = s.join ? grads.front() : Tensor(), du = n2 ? grads.back() : Tensor();
    if (!dh.defined() && !du.defined()) return out;
    const Tensor& given = dh.defined() ? dh : du;
    const c10::DeviceGuard guard(given.device());
    check_captured(given);
    variable_list saved = ctx->get_saved_variables();
    const bool any = j.rows > 0 && j.cols > 0;
    for (int i = 0; i < kInputs; ++i) {
      if (s.edge[i] < 0 || !ctx->needs_input_grad(s.edge[i]) || (i >= kW2 && !du.defined())) continue;
      const at::TensorOptions options =
          given.options().dtype(i == kR ? s.stream_type : i == kY ? s.branch_type : saved[i].scalar_type());
      const at::IntArrayRef sizes = i <= kY ? at::IntArrayRef(s.shape) : saved[i].sizes();
      out[i] = any ? at::empty(sizes, options) : at::zeros(sizes, options);
    }
    if (any) {
      Inputs in;
      for (int i = kW1; i < kInputs; ++i) in.t[i] = saved[i];
      place_parameters(j, in);
      // where only the copies are read, an address that says there is such an input
      Rows r{given, j.cols}, y{given, j.cols};
      if (saved[kR].defined()) r = rows_of(saved[kR]);
      if (saved[kY].defined()) y = rows_of(saved[kY]);
      j.residual = r.ptr();
      j.ld_residual = r.ld;
      j.branch = s.join ? y.ptr() : nullptr;
      j.ld_branch = y.ld;
      place_kept(j, s, saved[kInputs], saved[kInputs + 1]);
      shampoo_join_grads g = {};
      Rows rh, ru;
      if (dh.defined()) {
        rh = rows_of(dh);
        g.d_h = rh.ptr();
        g.ld_d_h = rh.ld;
      }
      if (du.defined()) {
        ru = rows_of(du);
        g.d_u = ru.ptr();
        g.ld_d_u = ru.ld;
      }
      auto at = [&](int i) { return out[i].defined() ? out[i].data_ptr() : nullptr; };
      g.d_residual = at(kR);
      g.d_branch = at(kY);
      g.ld_d_residual = g.ld_d_branch = j.cols;
      g.d_after_weight = at(kW1);
      g.d_after_bias = at(kB1);
      g.d_gate = at(kGate);
      g.d_before_weight = at(kW2);
      g.d_before_bias = at(kB2);
      const int64_t size = (int64_t)shampoo_join_backward_workspace_bytes(&j, &g);
      const Tensor ws = at::empty({size}, given.options().dtype(at::kByte));
      check_backward(shampoo_join_backward(&j, &g, ws.data_ptr(), (size_t)size, stream_of(given)),
                     "shampoo_join_backward");
    }
    return finish(std::move(out));
  }
};

void check_vector(const OptTensor& v, const char* name, const Tensor& like) {
  if (!v) return;
  if (type_of(*v) < 0 || v->device() != like.device())
    refuse(name, " must be a float32 or bfloat16 tensor on ", like.device().str());
  if (v->dim() != 1 || v->size(0) != like.size(-1)) refuse(name, " has shape ", v->sizes(), ", expected [", like.size(-1), "]");
}

// Kind of a gate for rows of `shape`, and how many rows share a row of it.
int64_t gate_kind(const Tensor& gate, at::IntArrayRef shape, int64_t* run) {
  const at::IntArrayRef size = gate.sizes();
  const size_t n = shape.size() - 1;
  *run = std::max<int64_t>(lead(shape), 1);
  if (size.size() == 1 && size[0] == shape[n]) return SHAMPOO_GATE_ROWS;
  if (size.size() == n + 1) {
    if (size[n] == 1 && size.slice(0, n) == shape.slice(0, n)) {
      *run = 0;
      return SHAMPOO_GATE_TOKEN;
    }
    // leading dimensions as they are, then ones, then the columns
    size_t k = 0;
    while (k < n && size[k] == shape[k]) ++k;
    bool good = size[n] == shape[n];
    for (size_t i = k; i < n; ++i) good = good && size[i] == 1;
    if (good) {
      int64_t rows = 1;
      for (size_t i = k; i < n; ++i) rows *= shape[i];
      *run = std::max<int64_t>(rows, 1);
      return SHAMPOO_GATE_ROWS;
    }
  }
  refuse("gate has shape ", size, "; expected [", shape[n], "], a number or a row of ", shape[n],
         " for each row or run of the rows of ", shape);
}

std::pair<Tensor, Tensor> join(const Tensor& residual, const OptTensor& branch, int64_t kind1, double eps1,
                               const OptTensor& w1, const OptTensor& b1, const OptTensor& gate, double scale,
                               int64_t kind2, double eps2, const OptTensor& w2, const OptTensor& b2, bool to_bf16,
                               bool low) {
  refuse_trace();
  auto s = c10::make_intrusive<JoinState>();
  shampoo_join& j = s->j;
  j.stream_dtype = checked_type(residual, branch ? "residual" : "x");
  s->join = branch.has_value();
  s->stream_type = s->branch_type = residual.scalar_type();
  if (branch) {
    checked_type(*branch, "branch");
    if (branch->sizes() != residual.sizes() || branch->device() != residual.device())
      refuse("residual and branch differ in shape or device");
    s->branch_type = branch->scalar_type();
    if (s->branch_type != s->stream_type && s->stream_type != at::kFloat)
      refuse("a ", s->branch_type, " branch of a ", s->stream_type, " residual");
  } else if (to_bf16) {
    s->branch_type = at::kBFloat16;
  }
  j.branch_dtype = s->branch_type == at::kFloat ? SHAMPOO_T_F32 : SHAMPOO_T_BF16;
  check_vector(w1, "after.weight", residual);
  check_vector(b1, "after.bias", residual);
  check_vector(w2, branch ? "before.weight" : "the norm's weight", residual);
  check_vector(b2, branch ? "before.bias" : "the norm's bias", residual);
  if (!std::isfinite(scale)) refuse("scale must be finite");
  s->shape = residual.sizes().vec();
  j.rows = lead(s->shape);
  j.cols = s->shape.back();
  j.scale = scale;
  j.after.kind = kind1;
  j.after.eps = eps1;
  j.before.kind = kind2;
  j.before.eps = eps2;
  if (gate) {
    if (type_of(*gate) < 0 || gate->device() != residual.device())
      refuse("gate must be a float32 or bfloat16 tensor on ", residual.device().str());
    j.gate_kind = gate_kind(*gate, s->shape, &j.gate_rows);
  }
  s->low = low;
  s->keep_r = kind2 != SHAMPOO_NORM_NONE;
  s->keep_y = s->join && (kind1 != SHAMPOO_NORM_NONE || gate || kind2 != SHAMPOO_NORM_NONE);
  const OptTensor r = residual;
  if (wants_gradient({&r, &branch, &w1, &b1, &gate, &w2, &b2})) {
    const variable_list out = Join::apply(residual, branch, w1, b1, gate, w2, b2, s);
    return {s->join ? out.front() : Tensor(), s->keep_r ? out.back() : Tensor()};
  }
  const Kept k = join_forward(*s, Inputs{{residual, or_undefined(branch), or_undefined(w1), or_undefined(b1),
                                          or_undefined(gate), or_undefined(w2), or_undefined(b2)}}, false);
  return {k.h, k.u};
}

}  // namespace

PYBIND11_MODULE(_layers, m) {
  if (shampoo_abi_version() != SHAMPOO_ABI_VERSION) throw py::import_error("libshampoo_mi355x.so ABI version mismatch");
  m.def("activate", &activate, py::call_guard<py::gil_scoped_release>());
  m.def("join", &join, py::call_guard<py::gil_scoped_release>());
}
