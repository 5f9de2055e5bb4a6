// Launches of the gradient-producing operators, called by lopt_ops_api.cpp
// with validated arguments.  Not part of the public ABI.
#pragma once

#include <stddef.h>
#include <stdint.h>

#include <hip/hip_runtime.h>

namespace lopt {

// Element types as the ABI numbers them (lopt_dtype).
enum : int32_t { kF32 = 0, kBF16 = 1, kF16 = 2 };

// ---- layer norm and RMS norm (lopt_norm_forward.hip, lopt_norm_backward.hip) ----
struct NormForward {
  const void* x;
  const void* w;   // NULL: 1
  const void* b;   // NULL: 0
  void* y;
  float* mean;     // NULL: not written (always for RMS)
  float* rstd;     // NULL: not written
  int64_t rows, cols, ldx, ldy;
  int32_t dtype, wdtype, rms;
  float eps;
};

struct NormBackward {
  const void* dy;
  const void* x;
  const void* w;      // NULL: 1
  const float* mean;  // NULL for RMS
  const float* rstd;
  void* dx;           // NULL: not computed
  void* dw;           // NULL: not computed
  void* db;           // NULL: not computed (always for RMS)
  float* part;        // workspace: [blocks][2 cols] partial sums (RMS: [blocks][cols])
  int64_t rows, cols, lddy, ldx, lddx;
  int32_t dtype, wdtype, gdtype, rms, accumulate;
};

// Blocks of the backward pass, each with one partial sum per column and gradient.
int64_t norm_backward_blocks(int64_t rows, int64_t cols);
hipError_t launch_norm_forward(const NormForward& a, hipStream_t s);
hipError_t launch_norm_backward(const NormBackward& a, hipStream_t s);

// ---- embedding (lopt_embedding.hip) ----
struct EmbeddingForward {
  const void* ids;
  const void* table;
  void* out;
  int64_t n_ids, rows, cols, row0, ldt, ldo;
  int32_t id_bytes, tdtype, odtype;
  float scale;
};

struct EmbeddingBackward {
  const void* ids;
  const void* dout;
  void* dtable;
  unsigned char* ws;
  int64_t n_ids, rows, cols, row0, ldd, ldt;
  int32_t id_bytes, dtype, gdtype, accumulate;
  float scale;
};

size_t embedding_backward_bytes(int64_t n_ids, int64_t rows, int64_t cols);
hipError_t launch_embedding_forward(const EmbeddingForward& a, hipStream_t s);
hipError_t launch_embedding_backward(const EmbeddingBackward& a, hipStream_t s);

// ---- distillation from a teacher's top logits (lopt_distill.hip) ----
constexpr int kMaxTop = 1024;   // entries of a teacher's list

struct DistillForward {
  const void* z;       // student logits
  const void* ids;     // [rows][top], row stride ldi
  const void* u;       // teacher logits [rows][top], row stride ldu
  float* loss;
  float* lse;
  int64_t rows, cols, ldz, ldi, ldu;
  int32_t top, dtype, udtype, id_bytes;
  float inv_tau, tau;
};

struct DistillBackward {
  const float* dloss;  // row stride lddl (0: one value for all rows)
  const void* z;
  const void* ids;
  const void* u;
  const float* lse;
  void* dz;
  int64_t rows, cols, lddl, ldz, ldi, ldu, lddz;
  int32_t top, dtype, udtype, id_bytes;
  float inv_tau, tau;
};

hipError_t launch_distill_forward(const DistillForward& a, hipStream_t s);
hipError_t launch_distill_backward(const DistillBackward& a, hipStream_t s);

}  // namespace lopt
