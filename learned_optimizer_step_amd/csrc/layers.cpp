// The norm, embedding and distillation calls for torch tensors: checks,
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
  decltype(&lopt_embedding_forward) embedding_forward;
  decltype(&lopt_embedding_backward_workspace) embedding_backward_workspace;
  decltype(&lopt_embedding_backward) embedding_backward;
  decltype(&lopt_distill_forward) distill_forward;
  decltype(&lopt_distill_backward) distill_backward;
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
  find(l.embedding_forward, "lopt_embedding_forward");
  find(l.embedding_backward_workspace, "lopt_embedding_backward_workspace");
  find(l.embedding_backward, "lopt_embedding_backward");
  find(l.distill_forward, "lopt_distill_forward");
  find(l.distill_backward, "lopt_distill_backward");
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

// A caller's contiguous output, which the call will write, or a new one.
Tensor output(const Maybe& t, at::IntArrayRef shape, c10::Device device, at::ScalarType type, const char* name) {
  if (!t) return empty(shape, type, device);
  if (t->sizes() != shape || !t->is_contiguous() || t->device() != device)
    bad(std::string(name) + " must be a contiguous tensor of shape " + show(shape) + " on " + device.str());
  dtype_code(t->scalar_type(), name);
  // a change in place, which autograd looks for in what it has saved
  if (!t->is_inference()) t->unsafeGetTensorImpl()->bump_version();
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
  m.def("distill_forward", &distill_forward);
  m.def("distill_backward", &distill_backward);
  m.def("distill", [](const Tensor& z, const Tensor& ids, const Tensor& u, double temperature) {
    if (u.requires_grad()) bad("the loss has no gradient for teacher_logits: detach them");
    return Distill::apply(z, ids, u, temperature);
  });
}
