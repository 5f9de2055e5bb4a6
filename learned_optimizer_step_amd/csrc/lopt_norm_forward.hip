// Forward pass of layer norm and RMS norm:
//   mu = mean x (RMS: 0), rstd = (mean (x - mu)^2 + eps)^(-1/2), y = (x - mu) rstd w + b
// per row.  Bound by HBM: x is read and y written once; the row stays in
// registers between the two sums and the output.
#include <hip/hip_runtime.h>

#include "lopt_norm.h"

namespace lopt {
namespace {

template <class T, class L, int MODE>
__global__ __launch_bounds__(L::BLOCK) void k_norm_forward(NormForward a) {
  constexpr int V = kVec<T>, NV = L::E / V;
  constexpr int W = L::TPR > 64 ? L::TPR / 64 : 1;
  __shared__ double red1[2][W][1];
  __shared__ float red2[2][W][1];
  RowSum<L::TPR, 1, double> row_sum1{red1};
  RowSum<L::TPR, 1> row_sum2{red2};
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
    Pack<T, V> p[NV];
#pragma unroll
    for (int k = 0; k < NV; ++k) p[k] = at[k].load(xr);
#pragma unroll
    for (int k = 0; k < NV; ++k)
#pragma unroll
      for (int i = 0; i < V; ++i) x[k * V + i] = to_f32(p[k].v[i]);
    Moments m{};
    if (!a.rms) {
      // 16-bit values: a thread's few add up in fp32 without a rounding, unless their sizes differ by more than 2^8
      using Sum = std::conditional_t<sizeof(T) == 4, double, float>;
      Sum part[2] = {0, 0};
#pragma unroll
      for (int k = 0; k < NV; ++k)
#pragma unroll
        for (int i = 0; i < V; ++i) part[i & 1] += Sum(at[k].own(i) ? x[k * V + i] : 0.f);
      double sum[1] = {double(part[0]) + double(part[1])};
      row_sum1(sum);
      m = mean_of(sum[0], n);
    }
    float s2[1] = {0.f};
#pragma unroll
    for (int k = 0; k < NV; ++k)
#pragma unroll
      for (int i = 0; i < V; ++i) {
        float& d = x[k * V + i];
        d -= m.mean;
        const float o = at[k].own(i) ? d : 0.f;
        s2[0] = fmaf(o, o, s2[0]);
      }
    row_sum2(s2);
    spread(m, s2[0], float(n), inv_n, a.eps);
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
      if (a.mean) a.mean[r] = m.mean;
      if (a.rstd) a.rstd[r] = m.rstd;
    }
  }
}

// Rows longer than kLongestRow: one block a row, read once per sum and once
// for the output.
template <class T>
__global__ __launch_bounds__(1024) void k_norm_forward_long(NormForward a) {
  constexpr int V = kVec<T>;
  __shared__ double red1[2][16][1];
  __shared__ float red2[2][16][1];
  RowSum<1024, 1, double> row_sum1{red1};
  RowSum<1024, 1> row_sum2{red2};
  const int64_t n = a.cols;
  const float inv_n = 1.f / float(n);
  for (int64_t r = blockIdx.x; r < a.rows; r += gridDim.x) {
    const T* xr = static_cast<const T*>(a.x) + r * a.ldx;
    Moments m{};
    if (!a.rms) {
      double sum[1] = {0.0};
      for (int64_t c = threadIdx.x * V; c < n; c += 1024 * V) {
        const Pack<T, V> p = load_pack<T, V>(xr, c, n);
#pragma unroll
        for (int i = 0; i < V; ++i) sum[0] += double(to_f32(p.v[i]));
      }
      row_sum1(sum);
      m = mean_of(sum[0], n);
    }
    float s2[1] = {0.f};
    for (int64_t c = threadIdx.x * V; c < n; c += 1024 * V) {
      const Pack<T, V> p = load_pack<T, V>(xr, c, n);
#pragma unroll
      for (int i = 0; i < V; ++i)
        if (c + i < n) {
          const float d = to_f32(p.v[i]) - m.mean;
          s2[0] = fmaf(d, d, s2[0]);
        }
    }
    row_sum2(s2);
    spread(m, s2[0], float(n), inv_n, a.eps);
    T* yr = static_cast<T*>(a.y) + r * a.ldy;
    for (int64_t c = threadIdx.x * V; c < n; c += 1024 * V) {
      Pack<T, V> p = load_pack<T, V>(xr, c, n);
#pragma unroll
      for (int i = 0; i < V; ++i)
        if (c + i < n) {
          const float w = a.w ? load_any(a.w, a.wdtype, c + i) : 1.f;
          const float b = a.b ? load_any(a.b, a.wdtype, c + i) : 0.f;
          p.v[i] = from_f32<T>(fmaf((to_f32(p.v[i]) - m.mean - m.rest) * m.rstd, w, b));
        }
      store_pack<T, V>(yr, c, n, p);
    }
    if (threadIdx.x == 0) {
      if (a.mean) a.mean[r] = m.mean;
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
