// The operators' calls for torch tensors: checks,
// outputs, workspaces and the automatic differentiation behind
// learned_optimizer_step_amd/layers.py, built into _layers.so.  It calls the C
// ABI of the liblopt.so that lopt.load_library() loaded; no kernel is here.
//
// It is compiled, unlike the optimizer's ctypes binding, because these calls
// are many and short and half of them run on autograd's own thread: the same
// in Python took 14 us for a norm's forward call and 124 us for the forward and
// backward of 8 rows through autograd; compiled they take 7 and 43 (x * 2 and
// its backward, in torch alone: 27).
#include <c10/core/DeviceGuard.h>
#include <c10/hip/HIPStream.h>
#include <torch/csrc/autograd/custom_function.h>
#include <torch/csrc/autograd/functions/basic_ops.h>
#include <torch/csrc/utils/pybind.h>

#include <dlfcn.h>

#include <algorithm>
#include <optional>
#include <stdexcept>
#include <string>
#include <tuple>
#include <type_traits>
#include <vector>

#include "../../include/lopt.h"

namespace {

using at::Tensor;
using torch::autograd::AutogradContext;
using torch::autograd::Function;
using torch::autograd::variable_list;
using Maybe = std::optional<Tensor>;

// The library's calls, looked up in the one that the optimizer's steps run from (LOPT_LIBRARY can name another than the
// one beside this file).
struct Library {
  decltype(&lopt_norm_forward) norm_forward;
  decltype(&lopt_norm_backward_workspace) norm_backward_workspace;
  decltype(&lopt_norm_backward) norm_backward;
  decltype(&lopt_residual_norm_forward) residual_norm_forward;
  decltype(&lopt_residual_norm_backward_workspace) residual_norm_backward_workspace;
  decltype(&lopt_residual_norm_backward) residual_norm_backward;
  decltype(&lopt_embedding_forward) embedding_forward;
  decltype(&lopt_embedding_backward_workspace) embedding_backward_workspace;
  decltype(&lopt_embedding_backward) embedding_backward;
  decltype(&lopt_distill_forward) distill_forward;
  decltype(&lopt_distill_backward) distill_backward;
  decltype(&lopt_linear_ce_forward_workspace) linear_ce_forward_workspace;
  decltype(&lopt_linear_ce_forward) linear_ce_forward;
  decltype(&lopt_linear_ce_backward_workspace) linear_ce_backward_workspace;
  decltype(&lopt_linear_ce_backward) linear_ce_backward;
  decltype(&lopt_adamw_state_bytes) adamw_state_bytes;
  decltype(&lopt_adamw_step) adamw_step;
  decltype(&lopt_adamw_moments) adamw_moments;
  decltype(&lopt_last_error) last_error;
};
Library lib;

void bind(uintptr_t handle) {
  Library l;
  const auto find = [&](auto& call, const char* name) {
    call = reinterpret_cast<std::decay_t<decltype(call)>>(dlsym(reinterpret_cast<void*>(handle), name));
    if (!call) throw pybind11::import_error(std::string(name) + " is missing in the liblopt.so that is loaded");
  };
  find(l.norm_forward, "lopt_norm_forward");
  find(l.norm_backward_workspace, "lopt_norm_backward_workspace");
  find(l.norm_backward, "lopt_norm_backward");
  find(l.residual_norm_forward, "lopt_residual_norm_forward");
  find(l.residual_norm_backward_workspace, "lopt_residual_norm_backward_workspace");
  find(l.residual_norm_backward, "lopt_residual_norm_backward");
  find(l.embedding_forward, "lopt_embedding_forward");
  find(l.embedding_backward_workspace, "lopt_embedding_backward_workspace");
  find(l.embedding_backward, "lopt_embedding_backward");
  find(l.distill_forward, "lopt_distill_forward");
  find(l.distill_backward, "lopt_distill_backward");
  find(l.linear_ce_forward_workspace, "lopt_linear_ce_forward_workspace");
  find(l.linear_ce_forward, "lopt_linear_ce_forward");
  find(l.linear_ce_backward_workspace, "lopt_linear_ce_backward_workspace");
  find(l.linear_ce_backward, "lopt_linear_ce_backward");
  find(l.adamw_state_bytes, "lopt_adamw_state_bytes");
  find(l.adamw_step, "lopt_adamw_step");
  find(l.adamw_moments, "lopt_adamw_moments");
  find(l.last_error, "lopt_last_error");
  lib = l;
}

// A call that liblopt refused: lopt.LoptError in Python.
struct Refused : std::runtime_error {
  int status;
  Refused(int s, const char* message) : std::runtime_error(message), status(s) {}
};

void check(lopt_status s) {
  if (s != LOPT_OK) throw Refused(int(s), lib.last_error());
}

[[noreturn]] void bad(const std::string& message) { throw pybind11::value_error(message); }

std::string show(at::IntArrayRef shape) {
  std::string s = "(";
  for (size_t i = 0; i < shape.size(); ++i) s += (i ? ", " : "") + std::to_string(shape[i]);
  return s + ")";
}

int32_t dtype_code(at::ScalarType t, const char* name) {
  if (t == at::kFloat) return LOPT_F32;
  if (t == at::kBFloat16) return LOPT_BF16;
  if (t == at::kHalf) return LOPT_F16;
  bad(std::string(name) + " must be float32, bfloat16 or float16, not " + c10::toString(t));
}

int32_t id_bytes(const Tensor& t, const char* name) {
  if (t.scalar_type() == at::kInt) return 4;
  if (t.scalar_type() == at::kLong) return 8;
  bad(std::string(name) + " must be int32 or int64, not " + c10::toString(t.scalar_type()));
}

void on(c10::Device device, const Tensor& t, const char* name) {
  if (t.device() != device) bad(std::string(name) + " is on " + t.device().str() + ", not on " + device.str());
}

c10::Device gpu(const Tensor& t, const char* name) {
  if (!t.is_cuda()) bad(std::string(name) + " must be on the GPU: there is no CPU path");
  return t.device();
}

// t as rows of its last dimension, with unit stride in a row and rows that do
// not overlap; a copy where t is not laid out so.
struct Matrix {
  Tensor t;
  int64_t rows, cols, ld;
  void* data() const { return t.data_ptr(); }
};

Matrix matrix(const Tensor& x, const char* name) {
  if (x.dim() == 0) bad(std::string(name) + " needs at least one dimension");
  const int64_t cols = x.size(-1);
  if (cols < 1) bad(std::string(name) + ": the last dimension is empty");
  if (x.is_contiguous()) return {x, x.numel() / cols, cols, cols};
  Tensor t = x.dim() == 2 ? x : x.reshape({-1, cols});
  if ((t.stride(1) != 1 && cols > 1) || (t.size(0) > 1 && t.stride(0) < cols)) t = t.contiguous();
  return {t, t.size(0), cols, t.stride(0)};
}

// A vector of n elements of the device, contiguous; undefined for none.
Tensor vector(const Maybe& t, int64_t n, c10::Device device, const char* name) {
  if (!t || !t->defined()) return Tensor();
  if (t->dim() != 1 || t->size(0) != n) bad(std::string(name) + " must have shape (" + std::to_string(n) + ",), not " + show(t->sizes()));
  on(device, *t, name);
  return t->contiguous();
}

void* ptr(const Tensor& t) { return t.defined() ? t.data_ptr() : nullptr; }

Tensor empty(at::IntArrayRef shape, at::ScalarType t, c10::Device device) {
  return at::empty(shape, at::TensorOptions().dtype(t).device(device));
}

// A change in place, which autograd looks for in what it has saved.
void changed(const Tensor& t) {
  if (!t.is_inference()) t.unsafeGetTensorImpl()->bump_version();
}

// A caller's contiguous output, which the call will write, or a new one.
Tensor output(const Maybe& t, at::IntArrayRef shape, c10::Device device, at::ScalarType type, const char* name) {
  if (!t) return empty(shape, type, device);
  if (t->sizes() != shape || !t->is_contiguous() || t->device() != device)
    bad(std::string(name) + " must be a contiguous tensor of shape " + show(shape) + " on " + device.str());
  dtype_code(t->scalar_type(), name);
  changed(*t);
  return *t;
}

void* stream(c10::Device device) { return c10::hip::getCurrentHIPStream(device.index()).stream(); }

// Gradients of a backward pass that is itself differentiated: an error when
// something is differentiated through them, as for once_differentiable.
variable_list differentiable_once(variable_list grads) {
  if (!at::GradMode::is_enabled()) return grads;
  for (Tensor& g : grads)
    if (g.defined())
      g = (*std::make_shared<torch::autograd::DelayedError>("the gradients of this operator cannot be differentiated", 1))(
          {g.requires_grad() ? g : g.detach().requires_grad_(true)})[0];
  return grads;
}

// ---------------------------------------------------------------------------
// norms

// (y, statistics): the mean and rstd of the rows (RMS: rstd alone) as the rows of one matrix
std::tuple<Tensor, Tensor> norm_forward(const Tensor& x, const Maybe& weight, const Maybe& bias, double eps, bool rms) {
  const c10::Device device = gpu(x, "x");
  const int32_t code = dtype_code(x.scalar_type(), "x");
  const Matrix m = matrix(x, "x");
  const Tensor w = vector(weight, m.cols, device, "weight"), b = vector(bias, m.cols, device, "bias");
  if (rms && b.defined()) bad("an RMS norm has no bias");
  if (w.defined() && b.defined() && w.scalar_type() != b.scalar_type()) bad("weight and bias must have the same type");
  const int32_t wcode = w.defined() ? dtype_code(w.scalar_type(), "weight") : b.defined() ? dtype_code(b.scalar_type(), "bias") : LOPT_F32;
  const c10::DeviceGuard guard(device);
  Tensor y = empty(x.sizes(), x.scalar_type(), device);
  Tensor stats = empty({rms ? 1 : 2, m.rows}, at::kFloat, device);
  float* at = static_cast<float*>(stats.data_ptr());
  check(lib.norm_forward(rms ? LOPT_NORM_RMS : LOPT_NORM_LAYER, m.rows, m.cols, code, m.data(), m.ld, ptr(w), ptr(b), wcode,
                          float(eps), y.data_ptr(), m.cols, rms ? nullptr : at, rms ? at : at + m.rows, stream(device)));
  return {y, stats};
}

struct NormGrads {
  Tensor dx, dw, db;
};

NormGrads norm_backward(const Tensor& dy, const Tensor& x, const Maybe& weight, const float* mean, const float* rstd, bool rms,
                        const Maybe& grad_weight, const Maybe& grad_bias, bool accumulate, bool need_x, bool need_weight,
                        bool need_bias, std::optional<at::ScalarType> grad_dtype) {
  const c10::Device device = gpu(x, "x");
  on(device, dy, "grad_y");
  const int32_t code = dtype_code(x.scalar_type(), "x");
  if (dy.sizes() != x.sizes() || dy.scalar_type() != x.scalar_type()) bad("grad_y must have the shape and type of x");
  const Matrix m = matrix(x, "x"), g = matrix(dy, "grad_y");
  const Tensor w = vector(weight, m.cols, device, "weight");
  if (rms && (need_bias || grad_bias)) bad("an RMS norm has no bias");
  if (accumulate && ((need_weight && !grad_weight) || (need_bias && !grad_bias))) bad("accumulate needs the buffers to add to");
  const at::ScalarType make = grad_dtype ? *grad_dtype : w.defined() ? w.scalar_type() : at::kFloat;
  const c10::DeviceGuard guard(device);
  NormGrads out;
  if (need_x) out.dx = empty(x.sizes(), x.scalar_type(), device);
  if (need_weight) out.dw = output(grad_weight, {m.cols}, device, make, "grad_weight");
  if (need_bias) out.db = output(grad_bias, {m.cols}, device, need_weight ? out.dw.scalar_type() : make, "grad_bias");
  if (need_weight && need_bias && out.dw.scalar_type() != out.db.scalar_type())
    bad("grad_weight and grad_bias must have the same type");
  const Tensor& gw = need_weight ? out.dw : out.db;
  Tensor ws;
  size_t bytes = 0;
  if (gw.defined()) {
    check(lib.norm_backward_workspace(m.rows, m.cols, &bytes));
    ws = empty({int64_t(bytes)}, at::kByte, device);
  }
  check(lib.norm_backward(rms ? LOPT_NORM_RMS : LOPT_NORM_LAYER, m.rows, m.cols, code, g.data(), g.ld, m.data(), m.ld, ptr(w),
                           w.defined() ? dtype_code(w.scalar_type(), "weight") : LOPT_F32, mean, rstd, ptr(out.dx), m.cols,
                           ptr(out.dw), ptr(out.db), gw.defined() ? dtype_code(gw.scalar_type(), "grad_weight") : LOPT_F32,
                           accumulate, ptr(ws), bytes, stream(device)));
  return out;
}

class Norm : public Function<Norm> {
 public:
  static Tensor forward(AutogradContext* ctx, const Tensor& x, const Maybe& weight, const Maybe& bias, double eps, bool rms) {
    auto [y, stats] = norm_forward(x, weight, bias, eps, rms);
    ctx->save_for_backward({x, weight ? *weight : Tensor(), stats});
    ctx->saved_data["rms"] = rms;
    if (bias) ctx->saved_data["bias"] = bias->scalar_type();
    return y;
  }
  static variable_list backward(AutogradContext* ctx, variable_list grads) {
    const variable_list saved = ctx->get_saved_variables();
    const Tensor &x = saved[0], &w = saved[1], &stats = saved[2];
    const bool rms = ctx->saved_data["rms"].toBool(), biased = ctx->saved_data.count("bias") != 0;
    // edges are those of the tensors that there are
    const bool nw = w.defined() && ctx->needs_input_grad(1), nb = biased && ctx->needs_input_grad(w.defined() ? 2 : 1);
    std::optional<at::ScalarType> type;
    if (biased && !w.defined()) type = ctx->saved_data["bias"].toScalarType();
    const float* at = static_cast<const float*>(stats.data_ptr());
    const bool some = stats.size(1) != 0;
    NormGrads g = norm_backward(grads[0], x, w.defined() ? Maybe(w) : std::nullopt, rms || !some ? nullptr : at,
                                !some ? nullptr : rms ? at : at + stats.size(1), rms, std::nullopt, std::nullopt, false,
                                ctx->needs_input_grad(0), nw, nb, type);
    return differentiable_once({g.dx, g.dw, g.db, Tensor(), Tensor()});
  }
};

// ---------------------------------------------------------------------------
// the residual update with its norms

struct Residual {
  float alpha, beta;
  bool rms, post, pre;
};

// The vectors and the gate of a call, checked against rows of x's kind.
struct ResidualParams {
  Tensor w1, b1, w2, b2, row_gate;   // row_gate: a vector, the same for every row
  std::optional<Matrix> own_gate;    // a gate like y
  at::ScalarType type = at::kFloat;
  int32_t gate_kind() const { return own_gate ? LOPT_GATE_MATRIX : row_gate.defined() ? LOPT_GATE_VECTOR : LOPT_GATE_NONE; }
  const void* gate() const { return own_gate ? own_gate->data() : ptr(row_gate); }
  int64_t ldg() const { return own_gate ? own_gate->ld : 0; }

  ResidualParams(const Tensor& y, int64_t cols, const Residual& o, const Maybe& gate, const Maybe& post_weight, const Maybe& post_bias,
                 const Maybe& weight, const Maybe& bias) {
    const c10::Device device = y.device();
    w1 = vector(post_weight, cols, device, "post_weight");
    b1 = vector(post_bias, cols, device, "post_bias");
    w2 = vector(weight, cols, device, "weight");
    b2 = vector(bias, cols, device, "bias");
    if (!o.post && (w1.defined() || b1.defined())) bad("post_weight and post_bias are of the norm of y, which post=False leaves out");
    if (!o.pre && (w2.defined() || b2.defined())) bad("weight and bias are of the norm of h, which pre=False leaves out");
    if (!o.post && !o.pre) bad("neither norm: post and pre are False");
    if (o.rms && (b1.defined() || b2.defined())) bad("an RMS norm has no bias");
    if (gate && gate->defined()) {
      // of one row alone, a gate of y's own type is like y, one of another type a vector
      if (gate->dim() == 1 && (y.dim() != 1 || gate->scalar_type() != y.scalar_type())) {
        row_gate = vector(gate, cols, device, "gate");
      } else {
        on(device, *gate, "gate");
        if (gate->sizes() != y.sizes() || gate->scalar_type() != y.scalar_type()) bad("gate must be a vector of the last dimension, or have y's shape and type");
        own_gate = matrix(*gate, "gate");
      }
    }
    bool first = true;
    for (const Tensor* t : {&w1, &b1, &w2, &b2, &row_gate}) {
      if (!t->defined()) continue;
      if (!first && t->scalar_type() != type) bad("the weights, the biases and a gate vector must have the same type");
      type = t->scalar_type();
      first = false;
    }
    dtype_code(type, "weight");
  }
};

struct ResidualOut {
  Tensor h, z, stats;
};

ResidualOut residual_forward(const Tensor& x, const Tensor& y, const Maybe& gate, const Maybe& post_weight, const Maybe& post_bias,
                             const Maybe& weight, const Maybe& bias, double eps, const Residual& o) {
  const c10::Device device = gpu(x, "x");
  on(device, y, "y");
  const int32_t code = dtype_code(x.scalar_type(), "x");
  if (y.sizes() != x.sizes() || y.scalar_type() != x.scalar_type()) bad("y must have the shape and type of x");
  const Matrix mx = matrix(x, "x"), my = matrix(y, "y");
  const ResidualParams p(y, my.cols, o, gate, post_weight, post_bias, weight, bias);
  const c10::DeviceGuard guard(device);
  ResidualOut out;
  out.h = empty(x.sizes(), x.scalar_type(), device);
  if (o.pre) out.z = empty(x.sizes(), x.scalar_type(), device);
  out.stats = empty({4, mx.rows}, at::kFloat, device);
  check(lib.residual_norm_forward(o.rms ? LOPT_NORM_RMS : LOPT_NORM_LAYER, o.post, o.pre, mx.rows, mx.cols, code, mx.data(), mx.ld,
                                  my.data(), my.ld, p.gate_kind(), p.gate(), p.ldg(), ptr(p.w1), ptr(p.b1), ptr(p.w2), ptr(p.b2),
                                  dtype_code(p.type, "weight"), o.alpha, o.beta, float(eps), out.h.data_ptr(), mx.cols, ptr(out.z),
                                  mx.cols, static_cast<float*>(out.stats.data_ptr()), stream(device)));
  return out;
}

struct ResidualNeeds {
  bool x, y, gate, w1, b1, w2, b2;
};
struct ResidualBuffers {
  Maybe gate, w1, b1, w2, b2;
};
struct ResidualGrads {
  Tensor dx, dy, dgate, w1, b1, w2, b2;
};

ResidualGrads residual_backward(const Tensor& dh, const Tensor& dz, const Tensor& y, const Tensor& h, const Tensor& stats, const Maybe& gate,
                                const Maybe& post_weight, const Maybe& post_bias, const Maybe& weight, const Residual& o,
                                const ResidualNeeds& need, const ResidualBuffers& to, bool accumulate, std::optional<at::ScalarType> grad_dtype) {
  const c10::Device device = gpu(y, "y");
  const int32_t code = dtype_code(y.scalar_type(), "y");
  const auto like = [&](const Tensor& t, const char* name) -> std::optional<Matrix> {
    if (!t.defined()) return std::nullopt;
    on(device, t, name);
    if (t.sizes() != y.sizes() || t.scalar_type() != y.scalar_type()) bad(std::string(name) + " must have the shape and type of y");
    return matrix(t, name);
  };
  const Matrix my = matrix(y, "y");
  const auto mdh = like(dh, "grad_h"), mdz = like(dz, "grad_z"), mh = like(h, "h");
  if (o.pre && !mh) bad("h is missing");
  if (!o.pre && mdz) bad("grad_z is of the norm of h, which pre=False leaves out");
  on(device, stats, "stats");
  if (stats.scalar_type() != at::kFloat || !stats.is_contiguous() || stats.sizes() != at::IntArrayRef({4, my.rows}))
    bad("stats must be the forward call's");
  const ResidualParams p(y, my.cols, o, gate, post_weight, post_bias, weight, std::nullopt);
  const c10::DeviceGuard guard(device);
  ResidualGrads g;
  at::ScalarType make = grad_dtype.value_or(p.type), made = at::kFloat;
  bool first = true;
  const auto sum = [&](bool wanted, const Maybe& buffer, const char* name) {
    if (!wanted) return Tensor();
    if (accumulate && !buffer) bad("accumulate needs the buffers to add to");
    Tensor t = output(buffer, {my.cols}, device, first ? make : made, name);
    if (!first && t.scalar_type() != made) bad("the vectors' gradients must have the same type");
    made = t.scalar_type();
    first = false;
    return t;
  };
  // a given buffer's type is that of the others
  for (const Maybe* b : {&to.gate, &to.w1, &to.b1, &to.w2, &to.b2})
    if (*b && !grad_dtype) make = (*b)->scalar_type();
  g.w1 = sum(o.post && need.w1, to.w1, "grad_post_weight");
  g.b1 = sum(o.post && !o.rms && need.b1, to.b1, "grad_post_bias");
  g.w2 = sum(o.pre && need.w2, to.w2, "grad_weight");
  g.b2 = sum(o.pre && !o.rms && need.b2, to.b2, "grad_bias");
  if (p.own_gate) {
    if (to.gate) bad("grad_gate is for a gate vector");
    if (need.gate) g.dgate = empty(y.sizes(), y.scalar_type(), device);
  } else {
    g.dgate = sum(p.row_gate.defined() && need.gate, to.gate, "grad_gate");
  }
  if (need.x) g.dx = empty(y.sizes(), y.scalar_type(), device);
  if (need.y) g.dy = empty(y.sizes(), y.scalar_type(), device);
  Tensor ws;
  size_t bytes = 0;
  if (!first) {
    check(lib.residual_norm_backward_workspace(my.rows, my.cols, &bytes));
    ws = empty({int64_t(bytes)}, at::kByte, device);
  }
  const auto data = [](const std::optional<Matrix>& m) { return m ? m->data() : nullptr; };
  const auto ld = [](const std::optional<Matrix>& m) { return m ? m->ld : 0; };
  check(lib.residual_norm_backward(o.rms ? LOPT_NORM_RMS : LOPT_NORM_LAYER, o.post, o.pre, my.rows, my.cols, code, data(mdh), ld(mdh),
                                   data(mdz), ld(mdz), my.data(), my.ld, o.pre ? data(mh) : nullptr, ld(mh),
                                   static_cast<const float*>(stats.data_ptr()), p.gate_kind(), p.gate(), p.ldg(), ptr(p.w1), ptr(p.b1),
                                   ptr(p.w2), dtype_code(p.type, "weight"), o.alpha, o.beta, ptr(g.dx), my.cols, ptr(g.dy), my.cols,
                                   ptr(g.dgate), my.cols, ptr(g.w1), ptr(g.b1), ptr(g.w2), ptr(g.b2),
                                   first ? LOPT_F32 : dtype_code(made, "a gradient"), accumulate, ptr(ws), bytes, stream(device)));
  return g;
}

class ResidualNorm : public Function<ResidualNorm> {
 public:
  static variable_list forward(AutogradContext* ctx, const Tensor& x, const Tensor& y, const Maybe& gate, const Maybe& post_weight,
                               const Maybe& post_bias, const Maybe& weight, const Maybe& bias, double eps, double alpha, double beta,
                               bool rms, bool post, bool pre) {
    const Residual o{float(alpha), float(beta), rms, post, pre};
    ResidualOut out = residual_forward(x, y, gate, post_weight, post_bias, weight, bias, eps, o);
    const auto some = [](const Maybe& t) { return t ? *t : Tensor(); };
    ctx->set_materialize_grads(false);
    // h is read by its norm's gradient alone: without that norm a caller may change it in place
    ctx->save_for_backward({y, some(gate), some(post_weight), some(post_bias), some(weight), pre ? out.h : Tensor(), out.stats});
    ctx->saved_data["flags"] = int64_t(rms) | int64_t(post) << 1 | int64_t(pre) << 2 | int64_t(bool(gate)) << 3 | int64_t(bool(post_weight)) << 4 |
                               int64_t(bool(post_bias)) << 5 | int64_t(bool(weight)) << 6 | int64_t(bool(bias)) << 7;
    ctx->saved_data["alpha"] = alpha;
    ctx->saved_data["beta"] = beta;
    for (const Maybe* v : {&post_weight, &post_bias, &weight, &bias})   // the gradients' type: that of the vectors
      if (*v) ctx->saved_data["type"] = (*v)->scalar_type();
    if (!pre) return {out.h};
    return {out.h, out.z};
  }
  static variable_list backward(AutogradContext* ctx, variable_list grads) {
    const variable_list s = ctx->get_saved_variables();
    const int64_t flags = ctx->saved_data["flags"].toInt();
    const auto flag = [&](int k) { return (flags >> k & 1) != 0; };
    const Residual o{float(ctx->saved_data["alpha"].toDouble()), float(ctx->saved_data["beta"].toDouble()), flag(0), flag(1), flag(2)};
    // edges are those of the tensors that there are
    size_t edge = 2;
    const auto needs = [&](int k) { return flag(k) && ctx->needs_input_grad(edge++); };
    ResidualNeeds need{ctx->needs_input_grad(0), ctx->needs_input_grad(1), needs(3), needs(4), needs(5), needs(6), needs(7)};
    const Tensor dh = grads[0], dz = o.pre ? grads[1] : Tensor();
    ResidualGrads g;
    if (dh.defined() || dz.defined()) {
      const auto maybe = [](const Tensor& t) { return t.defined() ? Maybe(t) : Maybe(); };
      std::optional<at::ScalarType> type;
      if (ctx->saved_data.count("type")) type = ctx->saved_data["type"].toScalarType();
      g = residual_backward(dh, dz, s[0], s[5], s[6], maybe(s[1]), maybe(s[2]), maybe(s[3]), maybe(s[4]), o, need, {}, false, type);
    }
    return differentiable_once({g.dx, g.dy, g.dgate, g.w1, g.b1, g.w2, g.b2, Tensor(), Tensor(), Tensor(), Tensor(), Tensor(), Tensor()});
  }
};

// ---------------------------------------------------------------------------
// embedding

Tensor embedding_forward(const Tensor& ids, const Tensor& weight, double scale, int64_t row0, std::optional<at::ScalarType> dtype) {
  const c10::Device device = gpu(weight, "weight");
  on(device, ids, "ids");
  const int32_t code = dtype_code(weight.scalar_type(), "weight"), nb = id_bytes(ids, "ids");
  if (weight.dim() != 2) bad("weight must have two dimensions");
  const Matrix w = matrix(weight, "weight");
  const Tensor i = ids.contiguous();
  const at::ScalarType type = dtype.value_or(weight.scalar_type());
  const int32_t ocode = dtype_code(type, "dtype");
  const c10::DeviceGuard guard(device);
  c10::SmallVector<int64_t, 5> shape(ids.sizes().begin(), ids.sizes().end());
  shape.push_back(w.cols);
  Tensor out = empty(shape, type, device);
  check(lib.embedding_forward(i.numel(), i.data_ptr(), nb, w.rows, w.cols, row0, w.data(), w.ld, code, float(scale),
                               out.data_ptr(), w.cols, ocode, stream(device)));
  return out;
}

Tensor embedding_backward(const Tensor& dout, const Tensor& ids, int64_t rows, double scale, int64_t row0, const Maybe& to,
                          bool accumulate, at::ScalarType dtype) {
  const c10::Device device = gpu(dout, "grad_out");
  on(device, ids, "ids");
  const int32_t code = dtype_code(dout.scalar_type(), "grad_out"), nb = id_bytes(ids, "ids");
  if (dout.dim() == 0 || dout.sizes().slice(0, dout.dim() - 1) != ids.sizes())
    bad("grad_out must have the shape of ids and one dimension more");
  const Matrix g = matrix(dout, "grad_out");
  if (accumulate && !to) bad("accumulate needs a buffer to add to");
  if (rows < 0) bad("rows must not be negative");
  const Tensor i = ids.contiguous();
  const c10::DeviceGuard guard(device);
  Tensor dw = output(to, {rows, g.cols}, device, dtype, "out");
  size_t bytes = 0;
  check(lib.embedding_backward_workspace(g.rows, rows, g.cols, &bytes));
  const Tensor ws = empty({int64_t(bytes)}, at::kByte, device);
  check(lib.embedding_backward(g.rows, i.data_ptr(), nb, g.data(), g.ld, code, rows, g.cols, row0, float(scale), dw.data_ptr(),
                                g.cols, dtype_code(dw.scalar_type(), "dtype"), accumulate, ws.data_ptr(), bytes, stream(device)));
  return dw;
}

class Embedding : public Function<Embedding> {
 public:
  static Tensor forward(AutogradContext* ctx, const Tensor& ids, const Tensor& weight, double scale, int64_t row0,
                        std::optional<at::ScalarType> dtype) {
    ctx->save_for_backward({ids});
    ctx->saved_data["rows"] = weight.dim() == 2 ? weight.size(0) : 0;
    ctx->saved_data["scale"] = scale;
    ctx->saved_data["row0"] = row0;
    ctx->saved_data["dtype"] = weight.scalar_type();
    return embedding_forward(ids, weight, scale, row0, dtype);
  }
  static variable_list backward(AutogradContext* ctx, variable_list grads) {
    Tensor dw;
    if (ctx->needs_input_grad(1))
      dw = embedding_backward(grads[0], ctx->get_saved_variables()[0], ctx->saved_data["rows"].toInt(),
                              ctx->saved_data["scale"].toDouble(), ctx->saved_data["row0"].toInt(), std::nullopt, false,
                              ctx->saved_data["dtype"].toScalarType());
    return differentiable_once({Tensor(), dw, Tensor(), Tensor(), Tensor()});
  }
};

// ---------------------------------------------------------------------------
// distillation from a teacher's top logits

struct Lists {
  c10::Device device;
  int32_t code, nb, ucode;
  Matrix z, i, u;
};

Lists lists(const Tensor& logits, const Tensor& ids, const Tensor& teacher) {
  const c10::Device device = gpu(logits, "logits");
  on(device, ids, "teacher_ids");
  on(device, teacher, "teacher_logits");
  if (logits.dim() == 0 || ids.sizes() != teacher.sizes() || ids.dim() != logits.dim() ||
      ids.sizes().slice(0, ids.dim() - 1) != logits.sizes().slice(0, ids.dim() - 1))
    bad("teacher_ids and teacher_logits must have one shape, the logits' but for the last dimension");
  return {device, dtype_code(logits.scalar_type(), "logits"), id_bytes(ids, "teacher_ids"),
          dtype_code(teacher.scalar_type(), "teacher_logits"), matrix(logits, "logits"), matrix(ids, "teacher_ids"),
          matrix(teacher, "teacher_logits")};
}

std::tuple<Tensor, Tensor> distill_forward(const Tensor& logits, const Tensor& ids, const Tensor& teacher, double temperature) {
  const Lists l = lists(logits, ids, teacher);
  const at::IntArrayRef shape = logits.sizes().slice(0, logits.dim() - 1);
  const c10::DeviceGuard guard(l.device);
  Tensor loss = empty(shape, at::kFloat, l.device), lse = empty(shape, at::kFloat, l.device);
  check(lib.distill_forward(l.z.rows, l.z.cols, l.code, l.z.data(), l.z.ld, int32_t(std::min<int64_t>(l.i.cols, INT32_MAX)),
                             l.i.data(), l.i.ld, l.nb, l.u.data(), l.u.ld, l.ucode, float(temperature),
                             static_cast<float*>(loss.data_ptr()), static_cast<float*>(lse.data_ptr()), stream(l.device)));
  return {loss, lse};
}

Tensor distill_backward(const Tensor& grad_loss, const Tensor& logits, const Tensor& ids, const Tensor& teacher, const Tensor& lse,
                        double temperature, const Maybe& to) {
  const Lists l = lists(logits, ids, teacher);
  const at::IntArrayRef shape = logits.sizes().slice(0, logits.dim() - 1);
  const auto a_row = [&](const Tensor& t, const char* name) {
    on(l.device, t, name);
    if (t.scalar_type() != at::kFloat || t.sizes() != shape) bad(std::string(name) + " must be float32, one value a row of logits");
  };
  a_row(grad_loss, "grad_loss");
  a_row(lse, "lse");
  const c10::DeviceGuard guard(l.device);
  Tensor dz = output(to, logits.sizes(), l.device, logits.scalar_type(), "out");
  if (dz.scalar_type() != logits.scalar_type()) bad("out must have the type of logits");
  Tensor g = grad_loss.dim() == 1 ? grad_loss : grad_loss.reshape({-1});
  if (g.numel() > 1 && g.stride(0) >= (int64_t(1) << 28)) g = g.contiguous();
  const int64_t step = g.numel() > 1 ? g.stride(0) : 0;   // a single element's stride can be anything
  const Tensor s = lse.contiguous();
  check(lib.distill_backward(l.z.rows, l.z.cols, l.code, static_cast<const float*>(g.data_ptr()), step, l.z.data(), l.z.ld,
                              int32_t(std::min<int64_t>(l.i.cols, INT32_MAX)), l.i.data(), l.i.ld, l.nb, l.u.data(), l.u.ld,
                              l.ucode, float(temperature), static_cast<const float*>(s.data_ptr()), dz.data_ptr(), l.z.cols,
                              stream(l.device)));
  return dz;
}

class Distill : public Function<Distill> {
 public:
  static Tensor forward(AutogradContext* ctx, const Tensor& logits, const Tensor& ids, const Tensor& teacher, double temperature) {
    auto [loss, lse] = distill_forward(logits, ids, teacher, temperature);
    ctx->save_for_backward({logits, ids, teacher, lse});
    ctx->saved_data["temperature"] = temperature;
    return loss;
  }
  static variable_list backward(AutogradContext* ctx, variable_list grads) {
    const variable_list s = ctx->get_saved_variables();
    Tensor dz;
    if (ctx->needs_input_grad(0))
      dz = distill_backward(grads[0], s[0], s[1], s[2], s[3], ctx->saved_data["temperature"].toDouble(), std::nullopt);
    return differentiable_once({dz, Tensor(), Tensor(), Tensor()});
  }
};

// ---------------------------------------------------------------------------
// cross entropy of a linear layer's logits

struct Linear {
  c10::Device device;
  int32_t code, nb;
  Matrix x, w;
  Tensor targets;
};

Linear linear(const Tensor& x, const Tensor& weight, const Tensor& targets) {
  const c10::Device device = gpu(x, "x");
  on(device, weight, "weight");
  on(device, targets, "targets");
  const int32_t code = dtype_code(x.scalar_type(), "x"), nb = id_bytes(targets, "targets");
  if (x.dim() == 0 || targets.sizes() != x.sizes().slice(0, x.dim() - 1)) bad("targets must have the shape of x but for the last dimension");
  if (weight.dim() != 2 || weight.size(1) != x.size(-1)) bad("weight must have two dimensions, the second of x's last size");
  if (weight.scalar_type() != x.scalar_type()) bad("weight must have the type of x");
  if (weight.size(0) == 0) bad("weight: no entries");
  return {device, code, nb, matrix(x, "x"), matrix(weight, "weight"), targets.contiguous()};
}

std::tuple<Tensor, Tensor> linear_ce_forward(const Tensor& x, const Tensor& weight, const Tensor& targets) {
  const Linear l = linear(x, weight, targets);
  const c10::DeviceGuard guard(l.device);
  Tensor loss = empty(targets.sizes(), at::kFloat, l.device), lse = empty(targets.sizes(), at::kFloat, l.device);
  size_t bytes = 0;
  check(lib.linear_ce_forward_workspace(l.x.rows, l.x.cols, l.w.rows, l.code, &bytes));
  const Tensor ws = empty({int64_t(bytes)}, at::kByte, l.device);
  check(lib.linear_ce_forward(l.x.rows, l.x.cols, l.w.rows, l.code, l.x.data(), l.x.ld, l.w.data(), l.w.ld, l.targets.data_ptr(), l.nb,
                              static_cast<float*>(loss.data_ptr()), static_cast<float*>(lse.data_ptr()), ws.data_ptr(), bytes,
                              stream(l.device)));
  return {loss, lse};
}

std::tuple<Tensor, Tensor> linear_ce_backward(const Tensor& grad_loss, const Tensor& x, const Tensor& weight, const Tensor& targets,
                                              const Tensor& lse, const Maybe& to, bool accumulate, bool need_x, bool need_weight,
                                              std::optional<at::ScalarType> grad_dtype) {
  const Linear l = linear(x, weight, targets);
  for (const auto& [t, name] : {std::pair<const Tensor*, const char*>{&grad_loss, "grad_loss"}, {&lse, "lse"}}) {
    on(l.device, *t, name);
    if (t->scalar_type() != at::kFloat || t->sizes() != targets.sizes()) bad(std::string(name) + " must be float32, one value a token");
  }
  if (accumulate && need_weight && !to) bad("accumulate needs a buffer to add to");
  const c10::DeviceGuard guard(l.device);
  Tensor dx, dw;
  if (need_x) dx = empty(x.sizes(), x.scalar_type(), l.device);
  if (need_weight) dw = output(to, {l.w.rows, l.w.cols}, l.device, grad_dtype.value_or(weight.scalar_type()), "grad_weight");
  Tensor g = grad_loss.dim() == 1 ? grad_loss : grad_loss.reshape({-1});
  if (g.numel() > 1 && g.stride(0) >= (int64_t(1) << 28)) g = g.contiguous();
  const int64_t step = g.numel() > 1 ? g.stride(0) : 0;   // a single element's stride can be anything
  const Tensor s = lse.contiguous();
  size_t bytes = 0;
  check(lib.linear_ce_backward_workspace(l.x.rows, l.x.cols, l.w.rows, l.code, &bytes));
  const Tensor ws = empty({int64_t(bytes)}, at::kByte, l.device);
  check(lib.linear_ce_backward(l.x.rows, l.x.cols, l.w.rows, l.code, static_cast<const float*>(g.data_ptr()), step, l.x.data(), l.x.ld,
                               l.w.data(), l.w.ld, l.targets.data_ptr(), l.nb, static_cast<const float*>(s.data_ptr()), ptr(dx), l.x.cols,
                               ptr(dw), l.w.cols, dw.defined() ? dtype_code(dw.scalar_type(), "grad_weight") : LOPT_F32, accumulate,
                               ws.data_ptr(), bytes, stream(l.device)));
  return {dx, dw};
}

class LinearCe : public Function<LinearCe> {
 public:
  static Tensor forward(AutogradContext* ctx, const Tensor& x, const Tensor& weight, const Tensor& targets) {
    auto [loss, lse] = linear_ce_forward(x, weight, targets);
    ctx->save_for_backward({x, weight, targets, lse});
    return loss;
  }
  static variable_list backward(AutogradContext* ctx, variable_list grads) {
    const variable_list s = ctx->get_saved_variables();
    auto [dx, dw] = linear_ce_backward(grads[0], s[0], s[1], s[2], s[3], std::nullopt, false, ctx->needs_input_grad(0), ctx->needs_input_grad(1),
                                       std::nullopt);
    return differentiable_once({dx, dw, Tensor()});
  }
};

// ---------------------------------------------------------------------------
// AdamW

at::ScalarType moment_type(int64_t bits) { return bits == 8 ? at::kByte : at::kFloat; }

size_t moment_bytes(int64_t n, int64_t bits) {
  size_t bytes = 0;
  check(lib.adamw_state_bytes(n, int32_t(bits), &bytes));
  return bytes;
}

Tensor adamw_state(const Tensor& param, int64_t bits) {
  const c10::Device device = gpu(param, "param");
  const size_t bytes = moment_bytes(param.numel(), bits);
  return at::zeros({int64_t(bytes / c10::elementSize(moment_type(bits)))}, at::TensorOptions().dtype(moment_type(bits)).device(device));
}

void check_state(const Tensor& s, int64_t n, int64_t bits, c10::Device device, const std::string& name) {
  on(device, s, name.c_str());
  const size_t need = moment_bytes(n, bits);
  if (s.scalar_type() != moment_type(bits) || !s.is_contiguous() || s.nbytes() < need)
    bad(name + " must be contiguous, " + c10::toString(moment_type(bits)) + " and of " + std::to_string(need) + " bytes");
}

void adamw_step(const std::vector<Tensor>& params, const std::vector<Maybe>& grads, const std::vector<Tensor>& states,
                const Tensor& step, const std::vector<double>& lr, double beta1, double beta2, double eps,
                const std::vector<double>& weight_decay, int64_t bits, int64_t seed) {
  const size_t n = params.size();
  if (grads.size() != n || states.size() != n) bad("params, grads and states must be lists of one length");
  for (const auto* v : {&lr, &weight_decay})
    if (v->size() != 1 && v->size() != n) bad("lr and weight_decay must be numbers, or one a parameter");
  const c10::Device device = gpu(step, "step");
  if (step.scalar_type() != at::kLong || step.numel() != 2 || !step.is_contiguous()) bad("step must be a contiguous int64 tensor of two elements");
  std::vector<lopt_adamw_tensor> ts(n);
  std::vector<Tensor> keep;
  for (size_t i = 0; i < n; ++i) {
    const Tensor& p = params[i];
    const auto name = [&](const char* what) { return std::string(what) + " " + std::to_string(i); };
    on(device, p, name("parameter").c_str());
    if (!p.is_contiguous()) bad(name("parameter") + " must be contiguous");
    check_state(states[i], p.numel(), bits, device, name("state"));
    ts[i] = {p.data_ptr(), nullptr, states[i].data_ptr(), p.numel(), lr[lr.size() == 1 ? 0 : i],
             weight_decay[weight_decay.size() == 1 ? 0 : i], dtype_code(p.scalar_type(), "a parameter"), 0};
    if (!grads[i]) continue;
    Tensor g = *grads[i];
    if (g.layout() != at::kStrided) bad(name("gradient") + " must be dense");
    on(device, g, name("gradient").c_str());
    if (g.sizes() != p.sizes()) bad(name("gradient") + " must have the shape of its parameter");
    if (!g.is_contiguous()) keep.push_back(g = g.contiguous());
    ts[i].grad = g.data_ptr();
    ts[i].g_dtype = dtype_code(g.scalar_type(), "a gradient");
  }
  const c10::DeviceGuard guard(device);
  check(lib.adamw_step(ts.data(), int32_t(n), int32_t(bits), beta1, beta2, eps, uint32_t(seed),
                       static_cast<int64_t*>(step.data_ptr()), stream(device)));
  changed(step);
  for (size_t i = 0; i < n; ++i)
    if (grads[i]) {
      changed(params[i]);
      changed(states[i]);
    }
}

std::tuple<Tensor, Tensor> adamw_moments(const Tensor& state, int64_t n, int64_t bits, at::ScalarType dtype) {
  const c10::Device device = gpu(state, "state");
  check_state(state, n, bits, device, "state");
  const int32_t code = dtype_code(dtype, "dtype");
  const c10::DeviceGuard guard(device);
  Tensor m = empty({n}, dtype, device), v = empty({n}, dtype, device);
  check(lib.adamw_moments(state.data_ptr(), n, int32_t(bits), code, m.data_ptr(), v.data_ptr(), stream(device)));
  return {m, v};
}

std::optional<at::ScalarType> scalar_type(const pybind11::object& dtype) {
  if (dtype.is_none()) return std::nullopt;
  if (!THPDtype_Check(dtype.ptr())) throw pybind11::type_error("dtype must be a torch.dtype");
  return reinterpret_cast<THPDtype*>(dtype.ptr())->scalar_type;
}

}  // namespace

PYBIND11_MODULE(_layers, m) {
  namespace py = pybind11;
  bind(py::module_::import("learned_optimizer_step_amd.lopt").attr("load_library")().attr("_handle").cast<uintptr_t>());
  py::register_local_exception_translator([](std::exception_ptr p) {
    try {
      if (p) std::rethrow_exception(p);
    } catch (const Refused& e) {
      const py::object type = py::module_::import("learned_optimizer_step_amd.lopt").attr("LoptError");
      PyErr_SetObject(type.ptr(), type(e.status, e.what()).ptr());
    }
  });
  m.def("norm_forward", [](const Tensor& x, const Maybe& w, const Maybe& b, double eps, bool rms) {
    auto [y, stats] = norm_forward(x, w, b, eps, rms);
    return std::make_tuple(y, rms ? Maybe() : Maybe(stats.select(0, 0)), stats.select(0, rms ? 0 : 1));
  });
  m.def("norm_backward", [](const Tensor& dy, const Tensor& x, const Maybe& weight, const Maybe& mean, const Maybe& rstd, bool rms,
                            const Maybe& gw, const Maybe& gb, bool accumulate, bool need_x, bool need_weight, bool need_bias,
                            const py::object& dtype) {
    const c10::Device device = gpu(x, "x");
    const int64_t rows = x.dim() && x.size(-1) ? x.numel() / x.size(-1) : 0;
    const auto stat = [&](const Maybe& t, const char* name) -> const float* {
      if (!t) bad(std::string(name) + " is missing");
      if (t->scalar_type() != at::kFloat || t->dim() != 1 || t->size(0) != rows || !t->is_contiguous() || t->device() != device)
        bad(std::string(name) + " must be a contiguous float32 vector of " + std::to_string(rows) + " values on x's device");
      return static_cast<const float*>(t->data_ptr());
    };
    const NormGrads g = norm_backward(dy, x, weight, rms ? nullptr : stat(mean, "mean"), stat(rstd, "rstd"), rms, gw, gb, accumulate,
                                      need_x, need_weight, need_bias, scalar_type(dtype));
    const auto maybe = [](const Tensor& t) { return t.defined() ? Maybe(t) : Maybe(); };
    return std::make_tuple(maybe(g.dx), maybe(g.dw), maybe(g.db));
  });
  m.def("norm", [](const Tensor& x, const Maybe& w, const Maybe& b, double eps, bool rms) { return Norm::apply(x, w, b, eps, rms); });
  m.def("residual_norm_forward", [](const Tensor& x, const Tensor& y, const Maybe& gate, const Maybe& w1, const Maybe& b1, const Maybe& w2,
                                    const Maybe& b2, double eps, double alpha, double beta, bool rms, bool post, bool pre) {
    const ResidualOut out = residual_forward(x, y, gate, w1, b1, w2, b2, eps, {float(alpha), float(beta), rms, post, pre});
    return std::make_tuple(out.h, pre ? Maybe(out.z) : Maybe(), out.stats);
  });
  m.def("residual_norm_backward", [](const Maybe& dh, const Maybe& dz, const Tensor& y, const Maybe& h, const Tensor& stats, const Maybe& gate,
                                     const Maybe& w1, const Maybe& b1, const Maybe& w2, double alpha, double beta, bool rms, bool post,
                                     bool pre, bool need_x, bool need_y, bool need_params, const Maybe& ggate, const Maybe& gw1,
                                     const Maybe& gb1, const Maybe& gw2, const Maybe& gb2, bool accumulate, const py::object& dtype) {
    const auto some = [](const Maybe& t) { return t ? *t : Tensor(); };
    const bool n = need_params;
    const ResidualGrads g = residual_backward(some(dh), some(dz), y, some(h), stats, gate, w1, b1, w2, {float(alpha), float(beta), rms, post, pre},
                                              {need_x, need_y, n, n, n, n, n}, {ggate, gw1, gb1, gw2, gb2}, accumulate, scalar_type(dtype));
    const auto maybe = [](const Tensor& t) { return t.defined() ? Maybe(t) : Maybe(); };
    return std::make_tuple(maybe(g.dx), maybe(g.dy), maybe(g.dgate), maybe(g.w1), maybe(g.b1), maybe(g.w2), maybe(g.b2));
  });
  m.def("residual_norm", [](const Tensor& x, const Tensor& y, const Maybe& gate, const Maybe& w1, const Maybe& b1, const Maybe& w2, const Maybe& b2,
                            double eps, double alpha, double beta, bool rms, bool post, bool pre) {
    const variable_list out = ResidualNorm::apply(x, y, gate, w1, b1, w2, b2, eps, alpha, beta, rms, post, pre);
    return std::make_tuple(out[0], pre ? Maybe(out[1]) : Maybe());
  });
  m.def("embedding_forward", [](const Tensor& ids, const Tensor& w, double scale, int64_t row0, const py::object& dtype) {
    return embedding_forward(ids, w, scale, row0, scalar_type(dtype));
  });
  m.def("embedding_backward", [](const Tensor& d, const Tensor& ids, int64_t rows, double scale, int64_t row0, const Maybe& out,
                                 bool accumulate, const py::object& dtype) {
    return embedding_backward(d, ids, rows, scale, row0, out, accumulate, scalar_type(dtype).value_or(at::kFloat));
  });
  m.def("embedding", [](const Tensor& ids, const Tensor& w, double scale, int64_t row0, const py::object& dtype) {
    return Embedding::apply(ids, w, scale, row0, scalar_type(dtype));
  });
  m.def("linear_ce_forward", &linear_ce_forward);
  m.def("linear_ce_backward", [](const Tensor& g, const Tensor& x, const Tensor& w, const Tensor& targets, const Tensor& lse, const Maybe& to,
                                 bool accumulate, bool need_x, bool need_weight, const py::object& dtype) {
    auto [dx, dw] = linear_ce_backward(g, x, w, targets, lse, to, accumulate, need_x, need_weight, scalar_type(dtype));
    return std::make_tuple(need_x ? Maybe(dx) : Maybe(), need_weight ? Maybe(dw) : Maybe());
  });
  m.def("linear_ce", [](const Tensor& x, const Tensor& w, const Tensor& targets) { return LinearCe::apply(x, w, targets); });
  m.def("adamw_state", &adamw_state);
  m.def("adamw_step", &adamw_step);
  m.def("adamw_moments", [](const Tensor& state, int64_t n, int64_t bits, const py::object& dtype) {
    return adamw_moments(state, n, bits, scalar_type(dtype).value_or(at::kFloat));
  });
  m.def("distill_forward", &distill_forward);
  m.def("distill_backward", &distill_backward);
  m.def("distill", [](const Tensor& z, const Tensor& ids, const Tensor& u, double temperature) {
    if (u.requires_grad()) bad("the loss has no gradient for teacher_logits: detach them");
    return Distill::apply(z, ids, u, temperature);
  });
}
