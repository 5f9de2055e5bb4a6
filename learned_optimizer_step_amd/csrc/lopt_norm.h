// Row layouts of the norm kernels, shared by the forward and backward pass.
#pragma once

#include <utility>

#include "lopt_ops.h"
#include "lopt_ops_device.h"

namespace lopt {

// A row is held in registers by TPR threads, E elements each, as E / kVec
// 16-byte vectors TPR vectors apart; a block of BLOCK threads holds
// BLOCK / TPR rows at a time.  The layouts, by the longest row each takes:
//   TPR 8,    E 8   up to    64 columns (eight rows in a wave)
//   TPR 64,   E 8   up to   512
//   TPR 64,   E 16  up to  1024
//   TPR 256,  E 8   up to  2048
//   TPR 256,  E 16  up to  4096
//   TPR 1024, E 8   up to  8192
//   TPR 1024, E 16  up to 16384
// Longer rows are read again for each of the sums (the *_long kernels).
constexpr int64_t kLongestRow = 16384;

template <int E_, int TPR_, int BLOCK_>
struct RowLayout {
  static constexpr int E = E_, TPR = TPR_, BLOCK = BLOCK_, ROWS = BLOCK_ / TPR_;
};

// Calls f(RowLayout) for the layout that holds rows of n columns (n <= kLongestRow).
template <class F>
auto with_layout(int64_t n, F&& f) {
  if (n <= 64) return f(RowLayout<8, 8, 256>());
  if (n <= 512) return f(RowLayout<8, 64, 256>());
  if (n <= 1024) return f(RowLayout<16, 64, 256>());
  if (n <= 2048) return f(RowLayout<8, 256, 256>());
  if (n <= 4096) return f(RowLayout<16, 256, 256>());
  if (n <= 8192) return f(RowLayout<8, 1024, 1024>());
  return f(RowLayout<16, 1024, 1024>());
}

// The thread's elements of a vector of n weights; `fill` where there is none.
// The type is branched on once, around loads that do not wait for each other.
template <class L, int V, class W>
__device__ __forceinline__ void load_weights_as(const void* p, int lane, int n, float fill, float (&w)[L::E]) {
#pragma unroll
  for (int k = 0; k < L::E / V; ++k) {
    const int c = (k * L::TPR + lane) * V;
    if (c + V <= n) {
      const Pack<W, V> v = *reinterpret_cast<const Pack<W, V>*>(static_cast<const W*>(p) + c);
#pragma unroll
      for (int i = 0; i < V; ++i) w[k * V + i] = to_f32(v.v[i]);
    } else {
#pragma unroll
      for (int i = 0; i < V; ++i) w[k * V + i] = c + i < n ? to_f32(static_cast<const W*>(p)[c + i]) : fill;
    }
  }
}
template <class L, int V>
__device__ __forceinline__ void load_weights(const void* p, int dtype, int lane, int n, float fill, float (&w)[L::E]) {
  if (!p) {
#pragma unroll
    for (int e = 0; e < L::E; ++e) w[e] = fill;
  } else if (dtype == kF32) {
    load_weights_as<L, V, float>(p, lane, n, fill, w);
  } else if (dtype == kBF16) {
    load_weights_as<L, V, bf16>(p, lane, n, fill, w);
  } else {
    load_weights_as<L, V, f16>(p, lane, n, fill, w);
  }
}

// Sums over the TPR threads of a row.  Across waves the sums go through LDS;
// `turn` alternates two buffers, so one barrier a call is enough (a wave that
// writes a buffer again has passed the barrier of the call between).
template <int TPR, int N>
struct RowSum {
  static constexpr int W = TPR > 64 ? TPR / 64 : 1;
  float (*red)[W][N];
  int turn = 0;

  __device__ __forceinline__ void operator()(float (&v)[N]) {
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
        float s = red[turn][0][i];
#pragma unroll
        for (int k = 1; k < W; ++k) s += red[turn][k][i];
        v[i] = s;
      }
      turn ^= 1;
    }
  }
};

template <class F>
hipError_t with_type(int32_t dtype, F&& f) {
  if (dtype == kF32) return f(float());
  if (dtype == kBF16) return f(bf16());
  return f(f16());
}

}  // namespace lopt
