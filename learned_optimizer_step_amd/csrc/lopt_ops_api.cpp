// C ABI of the operators that produce a step's gradients (norms, embedding,
// distillation loss): validation, then the launches of lopt_ops.h.  Nothing is
// allocated and nothing waits; the calls may be captured into a graph.
#include <hip/hip_runtime.h>

#include <cmath>
#include <string>

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
  static constexpr size_t kMost = 12;   // no call has more
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

}  // extern "C"
