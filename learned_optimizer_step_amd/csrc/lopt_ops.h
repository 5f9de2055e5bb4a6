// Launches of the operators around the learned optimizer's step, called by lopt_ops_api.cpp
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

// ---- residual update with its norms (lopt_residual_norm_forward.hip, lopt_residual_norm_backward.hip) ----
enum : int32_t { kNoGate = 0, kGateVector = 1, kGateMatrix = 2 };

struct ResidualForward {
  const void* x;
  const void* y;
  const void* gate;   // vector: type wdtype; matrix: type dtype
  const void* w1;     // of the norm of y; NULL: 1
  const void* b1;     // NULL: 0
  const void* w2;     // of the norm of h
  const void* b2;
  void* h;
  void* z;            // NULL without the second norm
  float* stats;       // [4][rows]: mean and rstd of y, mean and rstd of h; NULL: not written
  int64_t rows, cols, ldx, ldy, ldg, ldh, ldz;
  int32_t dtype, wdtype, gate_kind, rms, post, pre;
  float alpha, beta, eps;
};

struct ResidualBackward {
  const void* dh;     // NULL: 0
  const void* dz;     // NULL: 0
  const void* y;
  const void* h;
  const float* stats;
  const void* gate;
  const void* w1;
  const void* b1;
  const void* w2;
  void* dx;           // NULL: not computed, as those below
  void* dy;
  void* dgate;
  void* sums[5];      // gradients of w1, b1, w2, b2 and of a gate vector
  float* part;        // workspace
  int64_t rows, cols, lddh, lddz, ldy, ldh, ldg, lddx, lddy, lddg;
  int32_t dtype, wdtype, gdtype, gate_kind, rms, post, pre, accumulate;
  float alpha, beta;
};

size_t residual_backward_bytes(int64_t rows, int64_t cols);
hipError_t launch_residual_forward(const ResidualForward& a, hipStream_t s);
hipError_t launch_residual_backward(const ResidualBackward& a, hipStream_t s);

// ---- cross entropy of a linear layer's logits (lopt_linear_ce.hip) ----
struct LinearCeForward {
  const void* x;        // [rows][cols]
  const void* w;        // [vocab][cols]
  const void* targets;
  float* loss;          // NULL: not written, as lse
  float* lse;
  unsigned char* ws;
  int64_t rows, cols, vocab, ldx, ldw;
  int32_t dtype, id_bytes;
};

struct LinearCeBackward {
  const float* dloss;   // lddl apart
  const void* x;
  const void* w;
  const void* targets;
  const float* lse;
  void* dx;             // NULL: not computed, as dw
  void* dw;
  unsigned char* ws;
  int64_t rows, cols, vocab, lddl, ldx, ldw, lddx, lddw;
  int32_t dtype, id_bytes, gdtype, accumulate;
};

size_t linear_ce_bytes(int64_t rows, int64_t vocab, int64_t cols, int32_t dtype, bool backward_pass);
hipError_t launch_linear_ce_forward(const LinearCeForward& a, hipStream_t s);
hipError_t launch_linear_ce_backward(const LinearCeBackward& a, hipStream_t s);

// ---- AdamW over a list of tensors (lopt_adamw.hip) ----
constexpr int64_t kMomentBlock = 256;   // elements of a block of moments
constexpr int kMaxAdamw = 80;           // tensors of one launch

struct AdamwEntry {
  void* p;
  const void* g;
  void* s;       // moments
  int64_t n;
  float lr;
  float decay;   // 1 - lr wd
};

struct AdamwLaunch {
  AdamwEntry e[kMaxAdamw];
  uint32_t first[kMaxAdamw + 1];   // chunks of the tensors before each one, and of all
  uint32_t place[kMaxAdamw];       // in the caller's list
  int32_t count, advance;          // advance: the step counter goes on when this launch ends
  float b1, c1, b2, c2, eps;       // c = 1 - b
  uint32_t seed;
  double log_b1, log_b2;
  unsigned long long* step;        // t, and a ticket that is 0 between launches
};

int64_t adamw_chunks(int64_t n);
hipError_t launch_adamw(const AdamwLaunch& a, int32_t pdtype, int32_t gdtype, int32_t bits, bool once, hipStream_t s);
hipError_t launch_adamw_moments(const void* state, int64_t n, int32_t bits, int32_t dtype, void* m, void* v, hipStream_t s);

}  // namespace lopt
