// Row layouts of the residual update's kernels, shared by the forward and backward pass.
#pragma once

#include "lopt_norm.h"

namespace lopt {

// Longer rows are read again for each of their sums (the *_long kernels).
constexpr int64_t kLongestResidualRow = 8192;

// Calls f(RowLayout) for the layout that holds rows of n columns: 8 elements a
// thread, as up to eight vectors of parameters and sums stay in registers beside
// a row's four and the next one's.  The widest rows take 16, as 1024 threads
// would leave 128 registers each.  Neither has room for all of it: with 16 the backward kernels of two norms keep up to 436
// bytes of a thread in scratch memory (4096 x 8192 bf16, layer norms, backward: 203 us, 343 with 1024 threads; its bytes take 63).
template <class F>
auto with_residual_layout(int64_t n, F&& f) {
  if (n <= 64) return f(RowLayout<8, 8, 256>());     // eight rows in a wave
  if (n <= 512) return f(RowLayout<8, 64, 256>());
  if (n <= 1024) return f(RowLayout<8, 128, 128>());
  if (n <= 2048) return f(RowLayout<8, 256, 256>());
  if (n <= 4096) return f(RowLayout<8, 512, 512>());
  return f(RowLayout<16, 512, 512>());
}

// Calls f(mode) for rows of n columns: the vectors of rows that are whole
// numbers of them are those of kTail too.
template <class T, class L, class F>
void with_residual_mode(int64_t n, F&& f) {
  if constexpr (L::TPR == 8) {
    if (n < kVec<T>) return f(std::integral_constant<int, kTiny>());
  }
  f(std::integral_constant<int, kTail>());
}

// Moments of a row of which z, the norm of a rounded number, is the reader: a
// last bit of it decides where a rounding falls, so the row's sums are added up
// in 64 bits (up to 16 numbers of a thread in fp32), and its reciprocal root is the nearest float.
__device__ __forceinline__ void residual_mean(Moments& m, double sum, double inv_n) {
  const double mu = sum * inv_n;
  m.mean = float(mu);
  m.rest = float(mu - double(m.mean));
}
// s2: the sum of (x - mean)^2
__device__ __forceinline__ void residual_spread(Moments& m, double s2, double inv_n, float eps) {
  const double v = fmax(fma(-double(m.rest), double(m.rest), s2 * inv_n), 0.0) + double(eps);
  const double r = __builtin_amdgcn_rsq(v);
  m.rstd = float(fma(0.5 * r, fma(-v * r, r, 1.0), r));
  if (!(s2 <= double(FLT_MAX))) m.rstd = s2 > 0.0 ? 0.f : NAN;   // more than a float holds, or a NaN
}

// The thread's vectors of a row as they are loaded, and their elements, 0 where they are not its own.
template <class T, class At>
struct RowPacks {
  Pack<T, At::V> p[At::NV];
  __device__ __forceinline__ void load(const At& at, const T* row) {
#pragma unroll
    for (int k = 0; k < At::NV; ++k) p[k] = at[k].load(row);
  }
  __device__ __forceinline__ void open(const At& at, float (&x)[At::NV * At::V]) const {
#pragma unroll
    for (int k = 0; k < At::NV; ++k)
#pragma unroll
      for (int i = 0; i < At::V; ++i) x[k * At::V + i] = at[k].own(i) ? to_f32(p[k].v[i]) : 0.f;
  }
};
template <class T, class At>
__device__ __forceinline__ void store_row(const At& at, T* row, const float (&x)[At::NV * At::V]) {
#pragma unroll
  for (int k = 0; k < At::NV; ++k) {
    Pack<T, At::V> p;
#pragma unroll
    for (int i = 0; i < At::V; ++i) p.v[i] = from_f32<T>(x[k * At::V + i]);
    at[k].store(row, p);
  }
}

}  // namespace lopt
