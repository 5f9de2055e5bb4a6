// Row layouts of the norm kernels, shared by the forward and backward pass.
#pragma once

#include <cfloat>
#include <type_traits>
#include <utility>

#include "lopt_ops.h"
#include "lopt_ops_device.h"

namespace lopt {

// A row is held in registers by TPR threads, E elements each, as E / kVec
// 16-byte vectors TPR vectors apart; a block of BLOCK threads holds
// BLOCK / TPR rows at a time.  Rows longer than kLongestRow are read again for
// each of the sums (the *_long kernels).
constexpr int64_t kLongestRow = 16384;

template <int E_, int TPR_, int BLOCK_>
struct RowLayout {
  static constexpr int E = E_, TPR = TPR_, BLOCK = BLOCK_, ROWS = BLOCK_ / TPR_;
};

// Calls f(RowLayout) for the layout that holds rows of n columns (n <=
// kLongestRow).  Above 2048 columns the passes differ: the forward pass has
// registers to spare, so 16 elements a thread and more rows in flight (3000 x
// 6000 bf16: a fifth less time with 512 threads a row than with 1024; 20000 x
// 3001: 15 % less with 256 than with 512); the backward pass, with its sums,
// has not (a fifth less with 1024 than with 512; 8 % less with 512 than 256).
template <class F>
auto with_short_layout(int64_t n, F&& f) {
  if (n <= 64) return f(RowLayout<8, 8, 256>());     // eight rows in a wave
  if (n <= 512) return f(RowLayout<8, 64, 256>());
  if (n <= 1024) return f(RowLayout<16, 64, 256>());
  return f(RowLayout<8, 256, 256>());
}
template <class F>
auto with_forward_layout(int64_t n, F&& f) {
  if (n <= 2048) return with_short_layout(n, f);
  if (n <= 4096) return f(RowLayout<16, 256, 256>());
  if (n <= 8192) return f(RowLayout<16, 512, 512>());
  return f(RowLayout<16, 1024, 1024>());
}
template <class F>
auto with_backward_layout(int64_t n, F&& f) {
  if (n <= 2048) return with_short_layout(n, f);
  if (n <= 4096) return f(RowLayout<8, 512, 512>());
  if (n <= 8192) return f(RowLayout<8, 1024, 1024>());
  return f(RowLayout<16, 1024, 1024>());
}

// The thread's vectors of a row of n columns.
template <class T, class L, int MODE_>
struct RowAt {
  static constexpr int V = kVec<T>, NV = L::E / V, MODE = MODE_;
  RowVec<T, V, MODE> vec[NV];

  template <size_t... K>
  __device__ __forceinline__ RowAt(int lane, int n, std::index_sequence<K...>)
      : vec{RowVec<T, V, MODE>((int(K) * L::TPR + lane) * V, n)...} {}
  __device__ __forceinline__ RowAt(int lane, int n) : RowAt(lane, n, std::make_index_sequence<NV>()) {}
  __device__ __forceinline__ const RowVec<T, V, MODE>& operator[](int k) const { return vec[k]; }
};

// Calls f(mode) for rows of n columns; only the smallest layout sees rows shorter than a vector.
template <class T, class L, class F>
void with_mode(int64_t n, F&& f) {
  const int mode = row_mode(n, kVec<T>);
  if (mode == kWhole) f(std::integral_constant<int, kWhole>());
  else if constexpr (L::TPR == 8) {
    if (mode == kTail) f(std::integral_constant<int, kTail>());
    else f(std::integral_constant<int, kTiny>());
  } else f(std::integral_constant<int, kTail>());
}

// The thread's elements of a vector of weights; `fill` for all if there is
// none.  The type is branched on once, around loads that do not wait for each
// other (with a branch for each of them, 768 weights took 16 us to load).
template <class W, class At, int E>
__device__ __forceinline__ void load_weights_as(const At& at, const void* p, float (&w)[E]) {
  Pack<W, At::V> v[At::NV];
#pragma unroll
  for (int k = 0; k < At::NV; ++k) v[k] = at[k].load(static_cast<const W*>(p));
#pragma unroll
  for (int k = 0; k < At::NV; ++k)
#pragma unroll
    for (int i = 0; i < At::V; ++i) w[k * At::V + i] = to_f32(v[k].v[i]);
}
template <class At, int E>
__device__ __forceinline__ void load_weights(const At& at, const void* p, int dtype, float fill, float (&w)[E]) {
  if (!p) {
#pragma unroll
    for (int e = 0; e < E; ++e) w[e] = fill;
  } else if (dtype == kF32) {
    load_weights_as<float>(at, p, w);
  } else if (dtype == kBF16) {
    load_weights_as<bf16>(at, p, w);
  } else {
    load_weights_as<f16>(at, p, w);
  }
}

// Sums over the TPR threads of a row.  Across waves the sums go through LDS;
// `turn` alternates two buffers, so one barrier a call is enough (a wave that
// writes a buffer again has passed the barrier of the call between).
template <int TPR, int N, class S = float>
struct RowSum {
  static constexpr int W = TPR > 64 ? TPR / 64 : 1;
  S (*red)[W][N];
  int turn = 0;

  __device__ __forceinline__ void operator()(S (&v)[N]) {
#pragma unroll
    for (int i = 0; i < N; ++i) v[i] = lanes_sum<(TPR < 64 ? TPR : 64)>(v[i]);
    if constexpr (W > 1) {
      const int w = threadIdx.x >> 6;
      if ((threadIdx.x & 63) == 0)
#pragma unroll
        for (int i = 0; i < N; ++i) red[turn][w][i] = v[i];
      __syncthreads();
#pragma unroll
      for (int i = 0; i < N; ++i) {
        S t[W];
#pragma unroll
        for (int k = 0; k < W; ++k) t[k] = red[turn][k][i];
#pragma unroll
        for (int o = 1; o < W; o *= 2)
#pragma unroll
          for (int k = 0; k < W; k += 2 * o) t[k] += t[k + o];
        v[i] = t[0];
      }
      turn ^= 1;
    }
  }
};

// The mean comes from a sum in 64 bits: fp32's would be off by 2^-24 of the
// values' size, which is much of the spread of a row far from zero, and much of
// a mean that cancels (65536 x 200 fp32: 28 us, 25 with fp32 sums; bf16, whose
// threads add in fp32 without roundings, within 2 %).  What fp32 cannot hold of it goes into the spread and
// the output.
struct Moments {
  float mean, rest, rstd;   // mu = mean + rest
};

__device__ __forceinline__ Moments mean_of(double sum, int64_t n) {
  Moments m;
  const double mu = sum / double(n);
  m.mean = float(mu);
  m.rest = float(mu - double(m.mean));
  m.rstd = 0.f;
  return m;
}

// s2: the sum of (x - mean)^2; inv_n: the rounded 1 / n.  The product of the two is off by its rounding in every element
// of every row (the mean square of 41 ones is not 1): what it leaves of s2 gives the quotient's last bit (131072 x 128
// bf16 RMS: 27.1 us, 26.6 without it and 28.6 with a division).
__device__ __forceinline__ void spread(Moments& m, float s2, float n, float inv_n, float eps) {
  const float q = s2 * inv_n, mean2 = fmaf(fmaf(-q, n, s2), inv_n, q);
  const float var = fmaxf(mean2 - m.rest * m.rest, 0.f);
  m.rstd = 1.f / sqrtf(var + eps);
  // fmaxf drops a NaN: a row that holds one has no norm; one whose squares add up to more than fp32 holds has rstd 0
  if (!(s2 <= FLT_MAX)) m.rstd = s2 == INFINITY ? 0.f : s2;
}

template <class F>
hipError_t with_type(int32_t dtype, F&& f) {
  if (dtype == kF32) return f(float());
  if (dtype == kBF16) return f(bf16());
  return f(f16());
}

}  // namespace lopt
