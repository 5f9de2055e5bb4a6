// Forward pass of layer norm and RMS norm:
//   mu = mean x (RMS: 0), rstd = (mean (x - mu)^2 + eps)^(-1/2), y = (x - mu) rstd w + b
// per row.  Bound by HBM: x is read and y written once; the row stays in
// registers between the two sums and the output.
#include <hip/hip_runtime.h>

#include "lopt_norm.h"

namespace lopt {
namespace {

// One rounding of x's mean costs |mu| 2^-24, which is much of the spread of a
// row far from zero: the second sum also adds up x - mu, and its mean goes
// into mu, the spread and the output.
struct Moments {
  float mean, rest, rstd;   // mu = mean + rest
};

__device__ __forceinline__ Moments finish(float mean, float s1, float s2, float inv_n, float eps) {
  Moments m;
  m.mean = mean;
  m.rest = s1 * inv_n;
  const float var = fmaxf(s2 * inv_n - m.rest * m.rest, 0.f);
  m.rstd = 1.f / sqrtf(var + eps);
  // fmaxf drops a NaN: a row that holds one has no norm
  if (s2 != s2) m.rstd = s2;
  return m;
}

template <class T, class L, int MODE>
__global__ __launch_bounds__(L::BLOCK) void k_norm_forward(NormForward a) {
  constexpr int V = kVec<T>, NV = L::E / V;
  __shared__ float red[2][L::TPR > 64 ? L::TPR / 64 : 1][2];
  RowSum<L::TPR, 2> row_sum{red};
  const int lane = threadIdx.x % L::TPR;
  const int n = int(a.cols);
  const float inv_n = 1.f / float(n);

  RowAt<T, L, MODE> at(lane, n);
  // the weights stay in registers for all rows of the thread
  float w[L::E], b[L::E];
  load_weights(at, a.w, a.wdtype, 1.f, w);
  load_weights(at, a.b, a.wdtype, 0.f, b);

  const int64_t stride = int64_t(gridDim.x) * L::ROWS;
  // every thread of a block makes the same number of rounds (barriers inside)
  for (int64_t r0 = int64_t(blockIdx.x) * L::ROWS; r0 < a.rows; r0 += stride) {
    const int64_t r = r0 + threadIdx.x / L::TPR;
    const bool row = L::ROWS == 1 || r < a.rows;
    const T* xr = static_cast<const T*>(a.x) + (row ? r : 0) * a.ldx;
    float x[L::E];
    float v[2] = {0.f, 0.f};
    Pack<T, V> p[NV];
#pragma unroll
    for (int k = 0; k < NV; ++k) p[k] = at[k].load(xr);
#pragma unroll
    for (int k = 0; k < NV; ++k)
#pragma unroll
      for (int i = 0; i < V; ++i) {
        x[k * V + i] = to_f32(p[k].v[i]);
        v[0] += at[k].own(i) ? x[k * V + i] : 0.f;
      }
    float mean = 0.f;
    if (!a.rms) {
      row_sum(v);
      mean = v[0] * inv_n;
    }
    v[0] = v[1] = 0.f;
#pragma unroll
    for (int k = 0; k < NV; ++k)
#pragma unroll
      for (int i = 0; i < V; ++i) {
        float& d = x[k * V + i];
        d -= mean;
        const float o = at[k].own(i) ? d : 0.f;
        v[0] += o;
        v[1] = fmaf(o, o, v[1]);
      }
    row_sum(v);
    const Moments m = finish(mean, a.rms ? 0.f : v[0], v[1], inv_n, a.eps);
    if (!row) continue;
    T* yr = static_cast<T*>(a.y) + r * a.ldy;
#pragma unroll
    for (int k = 0; k < NV; ++k) {
#pragma unroll
      for (int i = 0; i < V; ++i)
        p[k].v[i] = from_f32<T>(fmaf((x[k * V + i] - m.rest) * m.rstd, w[k * V + i], b[k * V + i]));
      at[k].store(yr, p[k]);
    }
    if (lane == 0) {
      if (a.mean) a.mean[r] = m.mean + m.rest;
      if (a.rstd) a.rstd[r] = m.rstd;
    }
  }
}

// Rows longer than kLongestRow: one block a row, read once per sum and once
// for the output.
template <class T>
__global__ __launch_bounds__(1024) void k_norm_forward_long(NormForward a) {
  constexpr int V = kVec<T>;
  __shared__ float red[2][16][2];
  RowSum<1024, 2> row_sum{red};
  const int64_t n = a.cols;
  const float inv_n = 1.f / float(n);
  for (int64_t r = blockIdx.x; r < a.rows; r += gridDim.x) {
    const T* xr = static_cast<const T*>(a.x) + r * a.ldx;
    float mean = 0.f, v[2] = {0.f, 0.f};
    if (!a.rms) {
      for (int64_t c = threadIdx.x * V; c < n; c += 1024 * V) {
        const Pack<T, V> p = load_pack<T, V>(xr, c, n);
#pragma unroll
        for (int i = 0; i < V; ++i) v[i & 1] += to_f32(p.v[i]);
      }
      row_sum(v);
      mean = (v[0] + v[1]) * inv_n;
    }
    v[0] = v[1] = 0.f;
    for (int64_t c = threadIdx.x * V; c < n; c += 1024 * V) {
      const Pack<T, V> p = load_pack<T, V>(xr, c, n);
#pragma unroll
      for (int i = 0; i < V; ++i)
        if (c + i < n) {
          const float d = to_f32(p.v[i]) - mean;
          v[0] += d;
          v[1] = fmaf(d, d, v[1]);
        }
    }
    row_sum(v);
    const Moments m = finish(mean, a.rms ? 0.f : v[0], v[1], inv_n, a.eps);
    T* yr = static_cast<T*>(a.y) + r * a.ldy;
    for (int64_t c = threadIdx.x * V; c < n; c += 1024 * V) {
      Pack<T, V> p = load_pack<T, V>(xr, c, n);
#pragma unroll
      for (int i = 0; i < V; ++i)
        if (c + i < n) {
          const float w = a.w ? load_any(a.w, a.wdtype, c + i) : 1.f;
          const float b = a.b ? load_any(a.b, a.wdtype, c + i) : 0.f;
          p.v[i] = from_f32<T>(fmaf((to_f32(p.v[i]) - mean - m.rest) * m.rstd, w, b));
        }
      store_pack<T, V>(yr, c, n, p);
    }
    if (threadIdx.x == 0) {
      if (a.mean) a.mean[r] = m.mean + m.rest;
      if (a.rstd) a.rstd[r] = m.rstd;
    }
  }
}

}  // namespace

hipError_t launch_norm_forward(const NormForward& a, hipStream_t s) {
  if (a.rows == 0) return hipSuccess;
  return with_type(a.dtype, [&](auto t) {
    using T = decltype(t);
    if (a.cols > kLongestRow) {
      k_norm_forward_long<T><<<dim3(unsigned(a.rows < 4096 ? a.rows : 4096)), dim3(1024), 0, s>>>(a);
      return hipGetLastError();
    }
    return with_forward_layout(a.cols, [&](auto l) {
      using L = decltype(l);
      const int64_t need = (a.rows + L::ROWS - 1) / L::ROWS, most = int64_t(2048) * 256 / L::BLOCK;
      const dim3 grid(unsigned(need < most ? need : most)), block(L::BLOCK);
      with_mode<T, L>(a.cols, [&](auto mode) { k_norm_forward<T, L, mode()><<<grid, block, 0, s>>>(a); });
      return hipGetLastError();
    });
  });
}

}  // namespace lopt
