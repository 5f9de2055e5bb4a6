// C ABI of the operators around the learned optimizer's step (norms, embedding,
// distillation loss, linear cross entropy, AdamW): validation, then the launches of lopt_ops.h.  Nothing is
// allocated and nothing waits; the calls may be captured into a graph.
#include <hip/hip_runtime.h>

#include <algorithm>
#include <cmath>
#include <string>
#include <tuple>
#include <vector>

#include "../../include/lopt.h"
#include "lopt_error.h"
#include "lopt_ops.h"

using namespace lopt;

namespace {

constexpr int64_t kMaxDim = int64_t(1) << 31;     // rows and columns stay below
constexpr int64_t kMaxIds = int64_t(1) << 27;     // tokens of one embedding gradient
constexpr int64_t kMaxSpan = int64_t(1) << 60;    // bytes of one matrix stay below

int64_t elem_bytes(int32_t dtype) { return dtype == LOPT_F32 ? 4 : 2; }

void check_dtype(int32_t dtype, const char* name) {
  if (dtype != LOPT_F32 && dtype != LOPT_BF16 && dtype != LOPT_F16)
    fail(LOPT_ERR_INVALID_ARGUMENT, std::string(name) + ": unknown element type");
}

void check_dims(int64_t rows, int64_t cols) {
  if (rows < 0 || cols < 1) fail(LOPT_ERR_INVALID_ARGUMENT, "rows must be >= 0 and cols >= 1");
  if (rows >= kMaxDim || cols >= kMaxDim) fail(LOPT_ERR_UNSUPPORTED, "rows and cols must be below 2^31");
}

// A device buffer of a call: what the call reads or writes there.
struct Buffer {
  const char* name;
  uintptr_t a, b;   // [a, b)
  bool written;
};

struct Buffers {
  static constexpr size_t kMost = 20;   // no call has more
  Buffer list[kMost];
  size_t count = 0;

  void add(const char* name, const void* p, int64_t bytes, int64_t align, bool written) {
    const uintptr_t a = reinterpret_cast<uintptr_t>(p);
    if (!p) fail(LOPT_ERR_INVALID_ARGUMENT, std::string(name) + " is NULL");
    if (a % uintptr_t(align)) fail(LOPT_ERR_UNSUPPORTED, std::string(name) + " is not aligned to its elements");
    list[count++] = {name, a, a + uintptr_t(bytes), written};
  }
  // rows x cols elements of size `size`, rows `ld` elements apart
  void matrix(const char* name, const void* p, int64_t rows, int64_t cols, int64_t ld, int64_t size, bool written) {
    if (rows > 1) {
      if (ld < cols) fail(LOPT_ERR_INVALID_ARGUMENT, std::string(name) + ": rows overlap (row stride below the row's length)");
      if (ld >= kMaxSpan / size / rows) fail(LOPT_ERR_UNSUPPORTED, std::string(name) + " is too large");
    }
    if (rows == 0) return;   // nothing is read or written
    add(name, p, ((rows - 1) * (rows > 1 ? ld : 0) + cols) * size, size, written);
  }
  void no_overlap() const {
    for (size_t i = 0; i < count; ++i)
      for (size_t j = i + 1; j < count; ++j) {
        const Buffer &x = list[i], &y = list[j];
        if ((x.written || y.written) && x.a < y.b && y.a < x.b)
          fail(LOPT_ERR_INVALID_ARGUMENT, std::string(x.name) + " and " + y.name + " overlap");
      }
  }
};

void check_workspace(const void* ws, size_t have, size_t need) {
  if (need == 0) return;
  if (!ws || have < need)
    fail(LOPT_ERR_WORKSPACE, "workspace of " + std::to_string(have) + " bytes, " + std::to_string(need) + " needed");
  if (reinterpret_cast<uintptr_t>(ws) & 255u) fail(LOPT_ERR_WORKSPACE, "workspace is not 256-byte aligned");
}

void check_kind(int32_t kind) {
  if (kind != LOPT_NORM_LAYER && kind != LOPT_NORM_RMS) fail(LOPT_ERR_INVALID_ARGUMENT, "unknown kind of norm");
}

void check_ids(int32_t id_bytes) {
  if (id_bytes != 4 && id_bytes != 8) fail(LOPT_ERR_INVALID_ARGUMENT, "ids must be 4- or 8-byte integers");
}

void check_temperature(float tau) {
  // the loss has the factor tau^2, exponents the factor log2(e) / tau
  if (!std::isfinite(tau) || !(tau > 0.f) || !std::isfinite(1.5f / tau) || !std::isfinite(tau * tau))
    fail(LOPT_ERR_INVALID_ARGUMENT, "temperature must be finite and > 0, and so must its square and 1.5 / temperature");
}

size_t norm_bytes(int64_t rows, int64_t cols) {
  return size_t(norm_backward_blocks(rows, cols)) * 2 * size_t(cols) * sizeof(float);
}

void check_embedding(int64_t n_ids, int64_t rows, int64_t cols, int64_t row0) {
  check_dims(rows, cols);
  if (cols > (int64_t(1) << 30)) fail(LOPT_ERR_UNSUPPORTED, "embedding rows of more than 2^30 columns");
  if (n_ids < 0) fail(LOPT_ERR_INVALID_ARGUMENT, "negative number of ids");
  if (n_ids > kMaxIds) fail(LOPT_ERR_UNSUPPORTED, "more than 2^27 ids in one call");
  if (row0 < 0 || row0 > (int64_t(1) << 40)) fail(LOPT_ERR_INVALID_ARGUMENT, "row0 must lie in [0, 2^40]");
}

void check_residual(int32_t kind, int32_t post, int32_t pre, int32_t gate_kind, float alpha, float beta) {
  check_kind(kind);
  if (!post && !pre) fail(LOPT_ERR_INVALID_ARGUMENT, "neither norm: post and pre are 0");
  if (gate_kind < LOPT_GATE_NONE || gate_kind > LOPT_GATE_MATRIX) fail(LOPT_ERR_INVALID_ARGUMENT, "unknown kind of gate");
  if (!std::isfinite(alpha) || !std::isfinite(beta)) fail(LOPT_ERR_INVALID_ARGUMENT, "alpha and beta must be finite");
}

void check_linear_ce(int64_t rows, int64_t cols, int64_t vocab, int32_t dtype) {
  if (rows < 0 || cols < 1 || vocab < 1) fail(LOPT_ERR_INVALID_ARGUMENT, "rows must be >= 0, cols and vocab >= 1");
  if (rows > (int64_t(1) << 24) || cols > (int64_t(1) << 20)) fail(LOPT_ERR_UNSUPPORTED, "more than 2^24 rows or 2^20 columns");
  const int64_t tiles = (vocab + 255) / 256;
  // a grid has room for fewer than 2^32 threads: 512 a tile of 256 x 256, and with few rows 256 a tile of 64
  if (vocab > (int64_t(1) << 30) - 64) fail(LOPT_ERR_UNSUPPORTED, "vocab must be at most 2^30 - 64");
  if (tiles * ((rows + 255) / 256) >= (int64_t(1) << 23)) fail(LOPT_ERR_UNSUPPORTED, "vocab / 256 * rows / 256 must be below 2^23");
  check_dtype(dtype, "x");
}

void check_state_bits(int32_t bits) {
  if (bits != 8 && bits != 32) fail(LOPT_ERR_INVALID_ARGUMENT, "state_bits must be 8 or 32");
}

void check_moments(int64_t n, int32_t bits) {
  check_state_bits(bits);
  if (n < 1) fail(LOPT_ERR_INVALID_ARGUMENT, "a tensor needs at least one element");
  if (n > (int64_t(1) << 38)) fail(LOPT_ERR_UNSUPPORTED, "a tensor of more than 2^38 elements");
}

size_t moment_bytes(int64_t n, int32_t bits) {
  return size_t((n + kMomentBlock - 1) / kMomentBlock) * size_t(bits == 32 ? 8 * kMomentBlock : 2 * kMomentBlock + 16);
}

}  // namespace

extern "C" {

lopt_status lopt_norm_forward(int32_t kind, int64_t rows, int64_t cols, int32_t dtype, const void* x, int64_t ldx,
                              const void* weight, const void* bias, int32_t w_dtype, float eps, void* y, int64_t ldy,
                              float* mean, float* rstd, void* stream) {
  return guarded([&] {
    check_kind(kind);
    check_dims(rows, cols);
    check_dtype(dtype, "x");
    if (weight || bias) check_dtype(w_dtype, "weight");
    if (!(eps >= 0.f) || !std::isfinite(eps)) fail(LOPT_ERR_INVALID_ARGUMENT, "eps must be finite and >= 0");
    const bool rms = kind == LOPT_NORM_RMS;
    if (rms && (bias || mean)) fail(LOPT_ERR_INVALID_ARGUMENT, "an RMS norm has no bias and no mean");
    Buffers bufs;
    bufs.matrix("x", x, rows, cols, ldx, elem_bytes(dtype), false);
    bufs.matrix("y", y, rows, cols, ldy, elem_bytes(dtype), true);
    if (rows && weight) bufs.add("weight", weight, cols * elem_bytes(w_dtype), elem_bytes(w_dtype), false);
    if (rows && bias) bufs.add("bias", bias, cols * elem_bytes(w_dtype), elem_bytes(w_dtype), false);
    if (rows && mean) bufs.add("mean", mean, rows * 4, 4, true);
    if (rows && rstd) bufs.add("rstd", rstd, rows * 4, 4, true);
    bufs.no_overlap();
    NormForward a{};
    a.x = x; a.w = weight; a.b = bias; a.y = y; a.mean = mean; a.rstd = rstd;
    a.rows = rows; a.cols = cols; a.ldx = ldx; a.ldy = ldy;
    a.dtype = dtype; a.wdtype = w_dtype; a.rms = rms; a.eps = eps;
    hip_check(launch_norm_forward(a, static_cast<hipStream_t>(stream)), "norm forward");
  });
}

lopt_status lopt_norm_backward_workspace(int64_t rows, int64_t cols, size_t* bytes) {
  return guarded([&] {
    if (!bytes) fail(LOPT_ERR_INVALID_ARGUMENT, "bytes is NULL");
    check_dims(rows, cols);
    *bytes = norm_bytes(rows, cols);
  });
}

lopt_status lopt_norm_backward(int32_t kind, int64_t rows, int64_t cols, int32_t dtype, const void* dy, int64_t lddy,
                               const void* x, int64_t ldx, const void* weight, int32_t w_dtype, const float* mean,
                               const float* rstd, void* dx, int64_t lddx, void* dweight, void* dbias, int32_t g_dtype,
                               int32_t accumulate, void* workspace, size_t ws_bytes, void* stream) {
  return guarded([&] {
    check_kind(kind);
    check_dims(rows, cols);
    check_dtype(dtype, "x");
    if (weight) check_dtype(w_dtype, "weight");
    if (dweight || dbias) check_dtype(g_dtype, "dweight");
    const bool rms = kind == LOPT_NORM_RMS;
    if (rms && (dbias || mean)) fail(LOPT_ERR_INVALID_ARGUMENT, "an RMS norm has no bias and no mean");
    if (rows && (!rstd || (!rms && !mean))) fail(LOPT_ERR_INVALID_ARGUMENT, "mean or rstd is NULL");
    Buffers bufs;
    const int64_t size = elem_bytes(dtype);
    bufs.matrix("dy", dy, rows, cols, lddy, size, false);
    bufs.matrix("x", x, rows, cols, ldx, size, false);
    if (dx) bufs.matrix("dx", dx, rows, cols, lddx, size, true);
    if (weight) bufs.add("weight", weight, cols * elem_bytes(w_dtype), elem_bytes(w_dtype), false);
    if (rows && mean) bufs.add("mean", mean, rows * 4, 4, false);
    if (rows && rstd) bufs.add("rstd", rstd, rows * 4, 4, false);
    if (dweight) bufs.add("dweight", dweight, cols * elem_bytes(g_dtype), elem_bytes(g_dtype), true);
    if (dbias) bufs.add("dbias", dbias, cols * elem_bytes(g_dtype), elem_bytes(g_dtype), true);
    if (dweight || dbias) {
      const size_t need = norm_bytes(rows, cols);
      check_workspace(workspace, ws_bytes, need);
      if (need) bufs.add("workspace", workspace, int64_t(need), 256, true);
    }
    bufs.no_overlap();
    NormBackward a{};
    a.dy = dy; a.x = x; a.w = weight; a.mean = mean; a.rstd = rstd; a.dx = dx; a.dw = dweight; a.db = dbias;
    a.part = static_cast<float*>(workspace);
    a.rows = rows; a.cols = cols; a.lddy = lddy; a.ldx = ldx; a.lddx = lddx;
    a.dtype = dtype; a.wdtype = w_dtype; a.gdtype = g_dtype; a.rms = rms; a.accumulate = accumulate != 0;
    hip_check(launch_norm_backward(a, static_cast<hipStream_t>(stream)), "norm backward");
  });
}

lopt_status lopt_residual_norm_forward(int32_t kind, int32_t post, int32_t pre, int64_t rows, int64_t cols, int32_t dtype,
                                       const void* x, int64_t ldx, const void* y, int64_t ldy, int32_t gate_kind,
                                       const void* gate, int64_t ldg, const void* post_weight, const void* post_bias,
                                       const void* weight, const void* bias, int32_t w_dtype, float alpha, float beta,
                                       float eps, void* h, int64_t ldh, void* z, int64_t ldz, float* stats, void* stream) {
  return guarded([&] {
    check_residual(kind, post, pre, gate_kind, alpha, beta);
    check_dims(rows, cols);
    check_dtype(dtype, "x");
    if (post_weight || post_bias || weight || bias || gate_kind == LOPT_GATE_VECTOR) check_dtype(w_dtype, "weight");
    if (!(eps >= 0.f) || !std::isfinite(eps)) fail(LOPT_ERR_INVALID_ARGUMENT, "eps must be finite and >= 0");
    const bool rms = kind == LOPT_NORM_RMS;
    if (rms && (post_bias || bias)) fail(LOPT_ERR_INVALID_ARGUMENT, "an RMS norm has no bias");
    if (!post && (post_weight || post_bias)) fail(LOPT_ERR_INVALID_ARGUMENT, "post_weight or post_bias without the norm of y");
    if (!pre && (weight || bias || z)) fail(LOPT_ERR_INVALID_ARGUMENT, "weight, bias or z without the norm of h");
    Buffers bufs;
    const int64_t size = elem_bytes(dtype), wsize = elem_bytes(w_dtype);
    const auto vec = [&](const char* name, const void* p) {
      if (rows && p) bufs.add(name, p, cols * wsize, wsize, false);
    };
    bufs.matrix("x", x, rows, cols, ldx, size, false);
    bufs.matrix("y", y, rows, cols, ldy, size, false);
    if (gate_kind == LOPT_GATE_MATRIX) bufs.matrix("gate", gate, rows, cols, ldg, size, false);
    else if (gate_kind == LOPT_GATE_VECTOR && rows) bufs.add("gate", gate, cols * wsize, wsize, false);
    vec("post_weight", post_weight);
    vec("post_bias", post_bias);
    vec("weight", weight);
    vec("bias", bias);
    bufs.matrix("h", h, rows, cols, ldh, size, true);
    if (pre) bufs.matrix("z", z, rows, cols, ldz, size, true);
    if (rows && stats) bufs.add("stats", stats, 16 * rows, 4, true);
    bufs.no_overlap();
    ResidualForward a{};
    a.x = x; a.y = y; a.gate = gate; a.w1 = post_weight; a.b1 = post_bias; a.w2 = weight; a.b2 = bias;
    a.h = h; a.z = z; a.stats = stats;
    a.rows = rows; a.cols = cols; a.ldx = ldx; a.ldy = ldy; a.ldg = ldg; a.ldh = ldh; a.ldz = ldz;
    a.dtype = dtype; a.wdtype = w_dtype; a.gate_kind = gate_kind; a.rms = rms; a.post = post != 0; a.pre = pre != 0;
    a.alpha = alpha; a.beta = beta; a.eps = eps;
    hip_check(launch_residual_forward(a, static_cast<hipStream_t>(stream)), "residual norm forward");
  });
}

lopt_status lopt_residual_norm_backward_workspace(int64_t rows, int64_t cols, size_t* bytes) {
  return guarded([&] {
    if (!bytes) fail(LOPT_ERR_INVALID_ARGUMENT, "bytes is NULL");
    check_dims(rows, cols);
    *bytes = residual_backward_bytes(rows, cols);
  });
}

lopt_status lopt_residual_norm_backward(int32_t kind, int32_t post, int32_t pre, int64_t rows, int64_t cols, int32_t dtype,
                                        const void* dh, int64_t lddh, const void* dz, int64_t lddz, const void* y, int64_t ldy,
                                        const void* h, int64_t ldh, const float* stats, int32_t gate_kind, const void* gate,
                                        int64_t ldg, const void* post_weight, const void* post_bias, const void* weight,
                                        int32_t w_dtype, float alpha, float beta, void* dx, int64_t lddx, void* dy,
                                        int64_t lddy, void* dgate, int64_t lddg, void* dpost_weight, void* dpost_bias,
                                        void* dweight, void* dbias, int32_t g_dtype, int32_t accumulate, void* workspace,
                                        size_t ws_bytes, void* stream) {
  return guarded([&] {
    check_residual(kind, post, pre, gate_kind, alpha, beta);
    check_dims(rows, cols);
    check_dtype(dtype, "y");
    const bool rms = kind == LOPT_NORM_RMS, vector_gate = gate_kind == LOPT_GATE_VECTOR;
    if (post_weight || post_bias || weight || vector_gate) check_dtype(w_dtype, "weight");
    void* const sums[5] = {dpost_weight, dpost_bias, dweight, dbias, vector_gate ? dgate : nullptr};
    const bool any = std::any_of(sums, sums + 5, [](const void* p) { return p != nullptr; });
    if (any) check_dtype(g_dtype, "dweight");
    if (rms && (post_bias || dpost_bias || dbias)) fail(LOPT_ERR_INVALID_ARGUMENT, "an RMS norm has no bias");
    if (!post && (post_weight || post_bias || dpost_weight || dpost_bias))
      fail(LOPT_ERR_INVALID_ARGUMENT, "post_weight, post_bias or a gradient of theirs without the norm of y");
    if (!pre && (weight || dweight || dbias || dz)) fail(LOPT_ERR_INVALID_ARGUMENT, "weight, dz or a gradient of the weight or bias without the norm of h");
    if (gate_kind == LOPT_GATE_NONE && dgate) fail(LOPT_ERR_INVALID_ARGUMENT, "dgate without a gate");
    Buffers bufs;
    const int64_t size = elem_bytes(dtype), wsize = elem_bytes(w_dtype), gsize = elem_bytes(g_dtype);
    const auto vec = [&](const char* name, const void* p, int64_t s, bool written) {
      if (p && (rows || written)) bufs.add(name, p, cols * s, s, written);
    };
    if (dh) bufs.matrix("dh", dh, rows, cols, lddh, size, false);
    if (dz) bufs.matrix("dz", dz, rows, cols, lddz, size, false);
    bufs.matrix("y", y, rows, cols, ldy, size, false);
    if (pre) bufs.matrix("h", h, rows, cols, ldh, size, false);
    if (rows) bufs.add("stats", stats, 16 * rows, 4, false);
    if (gate_kind == LOPT_GATE_MATRIX) bufs.matrix("gate", gate, rows, cols, ldg, size, false);
    else if (vector_gate && rows) bufs.add("gate", gate, cols * wsize, wsize, false);
    vec("post_weight", post_weight, wsize, false);
    vec("post_bias", post_bias, wsize, false);
    vec("weight", weight, wsize, false);
    if (dx) bufs.matrix("dx", dx, rows, cols, lddx, size, true);
    if (dy) bufs.matrix("dy", dy, rows, cols, lddy, size, true);
    if (dgate && !vector_gate) bufs.matrix("dgate", dgate, rows, cols, lddg, size, true);
    const char* const names[5] = {"dpost_weight", "dpost_bias", "dweight", "dbias", "dgate"};
    for (int k = 0; k < 5; ++k) vec(names[k], sums[k], gsize, true);
    if (any) {
      const size_t need = residual_backward_bytes(rows, cols);
      check_workspace(workspace, ws_bytes, need);
      if (need) bufs.add("workspace", workspace, int64_t(need), 256, true);
    }
    bufs.no_overlap();
    ResidualBackward a{};
    a.dh = dh; a.dz = dz; a.y = y; a.h = h; a.stats = stats; a.gate = gate;
    a.w1 = post_weight; a.b1 = post_bias; a.w2 = weight; a.dx = dx; a.dy = dy; a.dgate = vector_gate ? nullptr : dgate;
    std::copy(sums, sums + 5, a.sums);
    a.part = any ? static_cast<float*>(workspace) : nullptr;
    a.rows = rows; a.cols = cols; a.lddh = lddh; a.lddz = lddz; a.ldy = ldy; a.ldh = ldh; a.ldg = ldg;
    a.lddx = lddx; a.lddy = lddy; a.lddg = lddg;
    a.dtype = dtype; a.wdtype = w_dtype; a.gdtype = g_dtype; a.gate_kind = gate_kind; a.rms = rms; a.post = post != 0;
    a.pre = pre != 0; a.accumulate = accumulate != 0; a.alpha = alpha; a.beta = beta;
    hip_check(launch_residual_backward(a, static_cast<hipStream_t>(stream)), "residual norm backward");
  });
}

lopt_status lopt_embedding_forward(int64_t n_ids, const void* ids, int32_t id_bytes, int64_t rows, int64_t cols, int64_t row0,
                                   const void* table, int64_t ldt, int32_t t_dtype, float scale, void* out, int64_t ldo,
                                   int32_t o_dtype, void* stream) {
  return guarded([&] {
    check_embedding(n_ids, rows, cols, row0);
    check_ids(id_bytes);
    check_dtype(t_dtype, "table");
    check_dtype(o_dtype, "out");
    if (!std::isfinite(scale)) fail(LOPT_ERR_INVALID_ARGUMENT, "scale must be finite");
    Buffers bufs;
    if (n_ids) bufs.add("ids", ids, n_ids * id_bytes, id_bytes, false);
    bufs.matrix("table", table, rows, cols, ldt, elem_bytes(t_dtype), false);
    bufs.matrix("out", out, n_ids, cols, ldo, elem_bytes(o_dtype), true);
    bufs.no_overlap();
    EmbeddingForward a{};
    a.ids = ids; a.table = table; a.out = out;
    a.n_ids = n_ids; a.rows = rows; a.cols = cols; a.row0 = row0; a.ldt = ldt; a.ldo = ldo;
    a.id_bytes = id_bytes; a.tdtype = t_dtype; a.odtype = o_dtype; a.scale = scale;
    hip_check(launch_embedding_forward(a, static_cast<hipStream_t>(stream)), "embedding forward");
  });
}

lopt_status lopt_embedding_backward_workspace(int64_t n_ids, int64_t rows, int64_t cols, size_t* bytes) {
  return guarded([&] {
    if (!bytes) fail(LOPT_ERR_INVALID_ARGUMENT, "bytes is NULL");
    check_embedding(n_ids, rows, cols, 0);
    *bytes = embedding_backward_bytes(n_ids, rows, cols);
  });
}

lopt_status lopt_embedding_backward(int64_t n_ids, const void* ids, int32_t id_bytes, const void* dout, int64_t ldd,
                                    int32_t d_dtype, int64_t rows, int64_t cols, int64_t row0, float scale, void* dtable,
                                    int64_t ldt, int32_t g_dtype, int32_t accumulate, void* workspace, size_t ws_bytes,
                                    void* stream) {
  return guarded([&] {
    check_embedding(n_ids, rows, cols, row0);
    check_ids(id_bytes);
    check_dtype(d_dtype, "dout");
    check_dtype(g_dtype, "dtable");
    if (!std::isfinite(scale)) fail(LOPT_ERR_INVALID_ARGUMENT, "scale must be finite");
    Buffers bufs;
    if (n_ids) bufs.add("ids", ids, n_ids * id_bytes, id_bytes, false);
    bufs.matrix("dout", dout, n_ids, cols, ldd, elem_bytes(d_dtype), false);
    bufs.matrix("dtable", dtable, rows, cols, ldt, elem_bytes(g_dtype), true);
    const size_t need = embedding_backward_bytes(n_ids, rows, cols);
    check_workspace(workspace, ws_bytes, need);
    if (need) bufs.add("workspace", workspace, int64_t(need), 256, true);
    bufs.no_overlap();
    if (rows == 0) return;
    EmbeddingBackward a{};
    a.ids = ids; a.dout = dout; a.dtable = dtable; a.ws = static_cast<unsigned char*>(workspace);
    a.n_ids = n_ids; a.rows = rows; a.cols = cols; a.row0 = row0; a.ldd = ldd; a.ldt = ldt;
    a.id_bytes = id_bytes; a.dtype = d_dtype; a.gdtype = g_dtype; a.accumulate = accumulate != 0; a.scale = scale;
    hip_check(launch_embedding_backward(a, static_cast<hipStream_t>(stream)), "embedding backward");
  });
}

lopt_status lopt_distill_forward(int64_t rows, int64_t cols, int32_t dtype, const void* logits, int64_t ldz, int32_t top,
                                 const void* ids, int64_t ldi, int32_t id_bytes, const void* teacher, int64_t ldu,
                                 int32_t u_dtype, float temperature, float* loss, float* lse, void* stream) {
  return guarded([&] {
    check_dims(rows, cols);
    check_dtype(dtype, "logits");
    check_dtype(u_dtype, "teacher");
    check_ids(id_bytes);
    check_temperature(temperature);
    if (top < 1) fail(LOPT_ERR_INVALID_ARGUMENT, "top must be >= 1");
    if (top > LOPT_MAX_TOP) fail(LOPT_ERR_UNSUPPORTED, "lists of more than LOPT_MAX_TOP entries");
    Buffers bufs;
    bufs.matrix("logits", logits, rows, cols, ldz, elem_bytes(dtype), false);
    bufs.matrix("ids", ids, rows, top, ldi, id_bytes, false);
    bufs.matrix("teacher", teacher, rows, top, ldu, elem_bytes(u_dtype), false);
    if (rows && loss) bufs.add("loss", loss, rows * 4, 4, true);
    if (rows && lse) bufs.add("lse", lse, rows * 4, 4, true);
    bufs.no_overlap();
    DistillForward a{};
    a.z = logits; a.ids = ids; a.u = teacher; a.loss = loss; a.lse = lse;
    a.rows = rows; a.cols = cols; a.ldz = ldz; a.ldi = ldi; a.ldu = ldu;
    a.top = top; a.dtype = dtype; a.udtype = u_dtype; a.id_bytes = id_bytes;
    a.tau = temperature; a.inv_tau = 1.f / temperature;
    hip_check(launch_distill_forward(a, static_cast<hipStream_t>(stream)), "distill forward");
  });
}

lopt_status lopt_distill_backward(int64_t rows, int64_t cols, int32_t dtype, const float* dloss, int64_t dloss_stride,
                                  const void* logits, int64_t ldz, int32_t top, const void* ids, int64_t ldi,
                                  int32_t id_bytes, const void* teacher, int64_t ldu, int32_t u_dtype, float temperature,
                                  const float* lse, void* dlogits, int64_t lddz, void* stream) {
  return guarded([&] {
    check_dims(rows, cols);
    check_dtype(dtype, "logits");
    check_dtype(u_dtype, "teacher");
    check_ids(id_bytes);
    check_temperature(temperature);
    if (top < 1) fail(LOPT_ERR_INVALID_ARGUMENT, "top must be >= 1");
    if (top > LOPT_MAX_TOP) fail(LOPT_ERR_UNSUPPORTED, "lists of more than LOPT_MAX_TOP entries");
    if (dloss_stride < 0 || dloss_stride >= (int64_t(1) << 28)) fail(LOPT_ERR_INVALID_ARGUMENT, "dloss_stride must lie in [0, 2^28)");
    Buffers bufs;
    const bool in_place = dlogits == logits && (lddz == ldz || rows <= 1);
    if (!in_place) bufs.matrix("logits", logits, rows, cols, ldz, elem_bytes(dtype), false);
    bufs.matrix("dlogits", dlogits, rows, cols, lddz, elem_bytes(dtype), true);
    bufs.matrix("ids", ids, rows, top, ldi, id_bytes, false);
    bufs.matrix("teacher", teacher, rows, top, ldu, elem_bytes(u_dtype), false);
    if (rows) bufs.add("dloss", dloss, ((rows - 1) * dloss_stride + 1) * 4, 4, false);
    if (rows) bufs.add("lse", lse, rows * 4, 4, false);
    bufs.no_overlap();
    DistillBackward a{};
    a.dloss = dloss; a.z = logits; a.ids = ids; a.u = teacher; a.lse = lse; a.dz = dlogits;
    a.rows = rows; a.cols = cols; a.lddl = dloss_stride; a.ldz = ldz; a.ldi = ldi; a.ldu = ldu; a.lddz = lddz;
    a.top = top; a.dtype = dtype; a.udtype = u_dtype; a.id_bytes = id_bytes;
    a.tau = temperature; a.inv_tau = 1.f / temperature;
    hip_check(launch_distill_backward(a, static_cast<hipStream_t>(stream)), "distill backward");
  });
}

lopt_status lopt_linear_ce_forward_workspace(int64_t rows, int64_t cols, int64_t vocab, int32_t dtype, size_t* bytes) {
  return guarded([&] {
    if (!bytes) fail(LOPT_ERR_INVALID_ARGUMENT, "bytes is NULL");
    check_linear_ce(rows, cols, vocab, dtype);
    *bytes = linear_ce_bytes(rows, vocab, cols, dtype, false);
  });
}

lopt_status lopt_linear_ce_backward_workspace(int64_t rows, int64_t cols, int64_t vocab, int32_t dtype, size_t* bytes) {
  return guarded([&] {
    if (!bytes) fail(LOPT_ERR_INVALID_ARGUMENT, "bytes is NULL");
    check_linear_ce(rows, cols, vocab, dtype);
    *bytes = linear_ce_bytes(rows, vocab, cols, dtype, true);
  });
}

lopt_status lopt_linear_ce_forward(int64_t rows, int64_t cols, int64_t vocab, int32_t dtype, const void* x, int64_t ldx,
                                   const void* w, int64_t ldw, const void* targets, int32_t id_bytes, float* loss, float* lse,
                                   void* workspace, size_t ws_bytes, void* stream) {
  return guarded([&] {
    check_linear_ce(rows, cols, vocab, dtype);
    check_ids(id_bytes);
    Buffers bufs;
    bufs.matrix("x", x, rows, cols, ldx, elem_bytes(dtype), false);
    if (rows) {
      bufs.matrix("w", w, vocab, cols, ldw, elem_bytes(dtype), false);
      bufs.add("targets", targets, rows * id_bytes, id_bytes, false);
      if (loss) bufs.add("loss", loss, rows * 4, 4, true);
      if (lse) bufs.add("lse", lse, rows * 4, 4, true);
      const size_t need = linear_ce_bytes(rows, vocab, cols, dtype, false);
      check_workspace(workspace, ws_bytes, need);
      bufs.add("workspace", workspace, int64_t(need), 256, true);
    }
    bufs.no_overlap();
    LinearCeForward a{};
    a.x = x; a.w = w; a.targets = targets; a.loss = loss; a.lse = lse; a.ws = static_cast<unsigned char*>(workspace);
    a.rows = rows; a.cols = cols; a.vocab = vocab; a.ldx = ldx; a.ldw = ldw; a.dtype = dtype; a.id_bytes = id_bytes;
    hip_check(launch_linear_ce_forward(a, static_cast<hipStream_t>(stream)), "linear cross entropy forward");
  });
}

lopt_status lopt_linear_ce_backward(int64_t rows, int64_t cols, int64_t vocab, int32_t dtype, const float* dloss,
                                    int64_t dloss_stride, const void* x, int64_t ldx, const void* w, int64_t ldw,
                                    const void* targets, int32_t id_bytes, const float* lse, void* dx, int64_t lddx, void* dw,
                                    int64_t lddw, int32_t g_dtype, int32_t accumulate, void* workspace, size_t ws_bytes,
                                    void* stream) {
  return guarded([&] {
    check_linear_ce(rows, cols, vocab, dtype);
    check_ids(id_bytes);
    if (dw) check_dtype(g_dtype, "dw");
    if (dloss_stride < 0 || dloss_stride >= (int64_t(1) << 28)) fail(LOPT_ERR_INVALID_ARGUMENT, "dloss_stride must lie in [0, 2^28)");
    Buffers bufs;
    bufs.matrix("x", x, rows, cols, ldx, elem_bytes(dtype), false);
    if (rows) {
      bufs.matrix("w", w, vocab, cols, ldw, elem_bytes(dtype), false);
      bufs.add("targets", targets, rows * id_bytes, id_bytes, false);
      bufs.add("dloss", dloss, ((rows - 1) * dloss_stride + 1) * 4, 4, false);
      bufs.add("lse", lse, rows * 4, 4, false);
      const size_t need = linear_ce_bytes(rows, vocab, cols, dtype, true);
      check_workspace(workspace, ws_bytes, need);
      bufs.add("workspace", workspace, int64_t(need), 256, true);
    }
    if (dx) bufs.matrix("dx", dx, rows, cols, lddx, elem_bytes(dtype), true);
    if (dw) bufs.matrix("dw", dw, vocab, cols, lddw, elem_bytes(g_dtype), true);
    bufs.no_overlap();
    if (!dx && !dw) return;
    LinearCeBackward a{};
    a.dloss = dloss; a.x = x; a.w = w; a.targets = targets; a.lse = lse; a.dx = dx; a.dw = dw;
    a.ws = static_cast<unsigned char*>(workspace);
    a.rows = rows; a.cols = cols; a.vocab = vocab; a.lddl = dloss_stride; a.ldx = ldx; a.ldw = ldw; a.lddx = lddx; a.lddw = lddw;
    a.dtype = dtype; a.id_bytes = id_bytes; a.gdtype = g_dtype; a.accumulate = accumulate != 0;
    hip_check(launch_linear_ce_backward(a, static_cast<hipStream_t>(stream)), "linear cross entropy backward");
  });
}

lopt_status lopt_adamw_state_bytes(int64_t n, int32_t state_bits, size_t* bytes) {
  return guarded([&] {
    if (!bytes) fail(LOPT_ERR_INVALID_ARGUMENT, "bytes is NULL");
    check_moments(n, state_bits);
    *bytes = moment_bytes(n, state_bits);
  });
}

lopt_status lopt_adamw_step(const lopt_adamw_tensor* ts, int32_t n, int32_t state_bits, double beta1, double beta2,
                            double eps, uint32_t seed, int64_t* step, void* stream) {
  return guarded([&] {
    if (n < 0) fail(LOPT_ERR_INVALID_ARGUMENT, "negative number of tensors");
    if (n && !ts) fail(LOPT_ERR_INVALID_ARGUMENT, "ts is NULL");
    check_state_bits(state_bits);
    for (const double b : {beta1, beta2})
      if (!(b >= 0.0 && b < 1.0)) fail(LOPT_ERR_INVALID_ARGUMENT, "beta1 and beta2 must lie in [0, 1)");
    if (!(eps >= 0.0) || !std::isfinite(float(eps))) fail(LOPT_ERR_INVALID_ARGUMENT, "eps must be finite and >= 0");
    if (n == 0) return;
    std::vector<Buffer> bufs;
    bufs.reserve(3 * size_t(n) + 1);
    const auto add = [&](const std::string& name, const void* p, int64_t bytes, uintptr_t align, bool written) {
      const uintptr_t at = reinterpret_cast<uintptr_t>(p);
      if (!p) fail(LOPT_ERR_INVALID_ARGUMENT, name + " is NULL");
      if (at % align) fail(LOPT_ERR_UNSUPPORTED, name + " is not aligned to " + std::to_string(align) + " bytes");
      bufs.push_back({nullptr, at, at + uintptr_t(bytes), written});
    };
    add("step", step, 16, 8, true);
    // launches of one pair of types, in the order of the list
    std::vector<std::pair<std::pair<int32_t, int32_t>, std::vector<int32_t>>> groups;
    int64_t bytes = 0;
    for (int32_t i = 0; i < n; ++i) {
      const lopt_adamw_tensor& t = ts[i];
      const auto name = [&](const char* what) { return std::string(what) + " of tensor " + std::to_string(i); };
      check_moments(t.n, state_bits);
      check_dtype(t.p_dtype, "param");
      if (t.grad) check_dtype(t.g_dtype, "grad");
      if (!std::isfinite(float(t.lr)) || !std::isfinite(float(t.lr * t.weight_decay)))
        fail(LOPT_ERR_INVALID_ARGUMENT, name("lr or weight_decay") + " is not finite");
      const int64_t p = elem_bytes(t.p_dtype), s = int64_t(moment_bytes(t.n, state_bits));
      add(name("param"), t.param, t.n * p, uintptr_t(p), true);
      add(name("state"), t.state, s, 16, true);
      if (!t.grad) continue;
      const int64_t g = elem_bytes(t.g_dtype);
      add(name("grad"), t.grad, t.n * g, uintptr_t(g), false);
      bytes += t.n * (p + g) + s;
      const std::pair<int32_t, int32_t> types(t.p_dtype, t.g_dtype);
      auto at = std::find_if(groups.begin(), groups.end(), [&](const auto& x) { return x.first == types; });
      if (at == groups.end()) at = groups.insert(at, {types, {}});
      at->second.push_back(i);
    }
    // by address: a buffer may begin before the last written one ends, or, if written, before any does
    std::sort(bufs.begin(), bufs.end(), [](const Buffer& x, const Buffer& y) { return std::tie(x.a, x.b) < std::tie(y.a, y.b); });
    uintptr_t any = 0, written = 0;
    for (const Buffer& b : bufs) {
      if (b.a < (b.written ? any : written)) fail(LOPT_ERR_INVALID_ARGUMENT, "params, states, gradients or step overlap");
      any = std::max(any, b.b);
      if (b.written) written = std::max(written, b.b);
    }
    AdamwLaunch a{};
    a.b1 = float(beta1); a.c1 = float(1.0 - beta1); a.b2 = float(beta2); a.c2 = float(1.0 - beta2);
    a.log_b1 = std::log(beta1); a.log_b2 = std::log(beta2);   // -inf of 0: no correction
    a.eps = float(eps); a.seed = seed; a.step = reinterpret_cast<unsigned long long*>(step);
    const bool once = bytes > 200'000'000;   // what the memory-side cache does not hold until the next step
    if (groups.empty()) groups.push_back({{LOPT_F32, LOPT_F32}, {}});   // only the count
    for (size_t k = 0; k < groups.size(); ++k) {
      const auto& [types, list] = groups[k];
      size_t next = 0;
      do {
        a.count = 0;
        a.first[0] = 0;
        while (next < list.size() && a.count < kMaxAdamw) {
          const lopt_adamw_tensor& t = ts[list[next]];
          const int64_t chunks = adamw_chunks(t.n);
          if (a.count && a.first[a.count] + chunks > (int64_t(1) << 31)) break;
          a.e[a.count] = {t.param, t.grad, t.state, t.n, float(t.lr), float(1.0 - t.lr * t.weight_decay)};
          a.place[a.count] = uint32_t(list[next]);
          a.first[a.count + 1] = a.first[a.count] + uint32_t(chunks);
          ++a.count;
          ++next;
        }
        a.advance = next == list.size() && k + 1 == groups.size();
        hip_check(launch_adamw(a, types.first, types.second, state_bits, once, static_cast<hipStream_t>(stream)), "adamw");
      } while (next < list.size());
    }
  });
}

lopt_status lopt_adamw_moments(const void* state, int64_t n, int32_t state_bits, int32_t dtype, void* m, void* v,
                               void* stream) {
  return guarded([&] {
    check_moments(n, state_bits);
    check_dtype(dtype, "m");
    Buffers bufs;
    bufs.add("state", state, int64_t(moment_bytes(n, state_bits)), 16, false);
    if (m) bufs.add("m", m, n * elem_bytes(dtype), elem_bytes(dtype), true);
    if (v) bufs.add("v", v, n * elem_bytes(dtype), elem_bytes(dtype), true);
    bufs.no_overlap();
    if (!m && !v) return;
    hip_check(launch_adamw_moments(state, n, state_bits, dtype, m, v, static_cast<hipStream_t>(stream)), "adamw moments");
  });
}

}  // extern "C"
