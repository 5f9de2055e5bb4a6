// The residual update between two blocks with the norms on both sides of it, per row:
//   u = norm1(y) (or y),  h = alpha x + beta gate u,  z = norm2(h)
// where h is rounded to its type first: z is the norm of what is kept.
// Bound by HBM: x and y (and a gate matrix) are read once, h and z written
// once; the row stays in registers through both norms, and so do the vectors of
// parameters for all rows of a block.  A block's next row is loaded before the sums of this one
// (65536 x 2048 bf16, RMS: 205 to 230 us, 4.7 to 5.2 TB/s; a copy reaches 5.1).
#include <hip/hip_runtime.h>

#include "lopt_residual_norm.h"

namespace lopt {
namespace {

// h as it is kept: an fp32 number first, also where one instruction could round the sum to fp16 at once.
template <class T>
__device__ __forceinline__ T kept(float h) {
  if constexpr (std::is_same_v<T, f16>) asm("" : "+v"(h));
  return from_f32<T>(h);
}

template <class T, class L, int MODE>
__global__ __launch_bounds__(L::BLOCK) void k_residual_forward(ResidualForward a) {
  constexpr int V = kVec<T>, NV = L::E / V, E = L::E;
  constexpr int W = L::TPR > 64 ? L::TPR / 64 : 1;
  __shared__ double red[2][W][1];
  RowSum<L::TPR, 1, double> row_sum{red};
  const int lane = threadIdx.x % L::TPR;
  const int n = int(a.cols);
  const double inv_n = 1.0 / double(n);

  RowAt<T, L, MODE> at(lane, n);
  float w1[E], b1[E], gate[E], w2[E], b2[E];
  load_weights(at, a.post ? a.w1 : nullptr, a.wdtype, 1.f, w1);
  load_weights(at, a.post ? a.b1 : nullptr, a.wdtype, 0.f, b1);
  load_weights(at, a.gate_kind == kGateVector ? a.gate : nullptr, a.wdtype, 1.f, gate);
  load_weights(at, a.pre ? a.w2 : nullptr, a.wdtype, 1.f, w2);
  load_weights(at, a.pre ? a.b2 : nullptr, a.wdtype, 0.f, b2);

  // mean and deviation of a row; v: the row less its mean, 0 where it is not the thread's
  const auto moments = [&](float (&v)[E]) {
    Moments m{};
    if (!a.rms) {
      using Sum = std::conditional_t<sizeof(T) == 4, double, float>;   // as the norm's: 16-bit values add up without a rounding
      Sum part[2] = {0, 0};
#pragma unroll
      for (int e = 0; e < E; ++e) part[e & 1] += Sum(v[e]);
      double sum[1] = {double(part[0]) + double(part[1])};
      row_sum(sum);
      residual_mean(m, sum[0], inv_n);
    }
    float part[2] = {0.f, 0.f};
#pragma unroll
    for (int k = 0; k < NV; ++k)
#pragma unroll
      for (int i = 0; i < V; ++i) {
        float& d = v[k * V + i];
        d = at[k].own(i) ? d - m.mean : 0.f;
        part[i & 1] = fmaf(d, d, part[i & 1]);
      }
    double s2[1] = {double(part[0]) + double(part[1])};
    row_sum(s2);
    residual_spread(m, s2[0], inv_n, a.eps);
    return m;
  };

  struct Row {
    RowPacks<T, RowAt<T, L, MODE>> x, y, gate;
  };
  const auto load = [&](int64_t r0) {
    const int64_t r = r0 + threadIdx.x / L::TPR, rr = r < a.rows ? r : 0;
    Row p;
    p.y.load(at, static_cast<const T*>(a.y) + rr * a.ldy);
    p.x.load(at, static_cast<const T*>(a.x) + rr * a.ldx);
    if (a.gate_kind == kGateMatrix) p.gate.load(at, static_cast<const T*>(a.gate) + rr * a.ldg);
    return p;
  };
  const int64_t stride = int64_t(gridDim.x) * L::ROWS, first = int64_t(blockIdx.x) * L::ROWS;
  Row next = load(first);
  // every thread of a block makes the same number of rounds (barriers inside)
  for (int64_t r0 = first; r0 < a.rows; r0 += stride) {
    const int64_t r = r0 + threadIdx.x / L::TPR;
    const bool row = L::ROWS == 1 || r < a.rows;
    const Row now = next;
    if (r0 + stride < a.rows) next = load(r0 + stride);
    float x[E], u[E];
    now.y.open(at, u);
    now.x.open(at, x);
    if (a.gate_kind == kGateMatrix) now.gate.open(at, gate);
    if (a.post) {
      const Moments m = moments(u);
#pragma unroll
      for (int e = 0; e < E; ++e) u[e] = fmaf((u[e] - m.rest) * m.rstd, w1[e], b1[e]);
      if (a.stats && row && lane == 0) {
        a.stats[r] = m.mean;
        a.stats[a.rows + r] = m.rstd;
      }
    }
#pragma unroll
    for (int k = 0; k < NV; ++k)
#pragma unroll
      for (int i = 0; i < V; ++i) {
        const int e = k * V + i;
        const float h = to_f32(kept<T>(fmaf(a.alpha, x[e], a.beta * (gate[e] * u[e]))));
        x[e] = at[k].own(i) ? h : 0.f;
      }
    if (row) store_row(at, static_cast<T*>(a.h) + r * a.ldh, x);
    if (!a.pre) continue;
    const Moments m = moments(x);
    if (!row) continue;
#pragma unroll
    for (int e = 0; e < E; ++e) x[e] = fmaf((x[e] - m.rest) * m.rstd, w2[e], b2[e]);
    store_row(at, static_cast<T*>(a.z) + r * a.ldz, x);
    if (a.stats && lane == 0) {
      a.stats[2 * a.rows + r] = m.mean;
      a.stats[3 * a.rows + r] = m.rstd;
    }
  }
}

// Rows longer than kLongestResidualRow: one block a row, read again for every
// sum.  A thread reads only what it wrote itself of h.
template <class T>
__global__ __launch_bounds__(1024) void k_residual_forward_long(ResidualForward a) {
  constexpr int V = kVec<T>;
  __shared__ double red[2][16][1];
  RowSum<1024, 1, double> row_sum{red};
  const int64_t n = a.cols;
  const double inv_n = 1.0 / double(n);
  const auto moments = [&](const T* row) {
    Moments m{};
    if (!a.rms) {
      double sum[1] = {0.0};
      for (int64_t c = threadIdx.x * V; c < n; c += 1024 * V) {
        const Pack<T, V> p = load_pack<T, V>(row, c, n);
#pragma unroll
        for (int i = 0; i < V; ++i) sum[0] += double(to_f32(p.v[i]));
      }
      row_sum(sum);
      residual_mean(m, sum[0], inv_n);
    }
    double s2[1] = {0.0};   // a vector's squares in fp32, the vectors' in 64 bits
    for (int64_t c = threadIdx.x * V; c < n; c += 1024 * V) {
      const Pack<T, V> p = load_pack<T, V>(row, c, n);
      float part = 0.f;
#pragma unroll
      for (int i = 0; i < V; ++i)
        if (c + i < n) {
          const float d = to_f32(p.v[i]) - m.mean;
          part = fmaf(d, d, part);
        }
      s2[0] += double(part);
    }
    row_sum(s2);
    residual_spread(m, s2[0], inv_n, a.eps);
    return m;
  };
  const auto param = [&](const void* p, int64_t c, float fill) { return p ? load_any(p, a.wdtype, c) : fill; };
  for (int64_t r = blockIdx.x; r < a.rows; r += gridDim.x) {
    const T* yr = static_cast<const T*>(a.y) + r * a.ldy;
    const T* xr = static_cast<const T*>(a.x) + r * a.ldx;
    const T* gr = a.gate_kind == kGateMatrix ? static_cast<const T*>(a.gate) + r * a.ldg : nullptr;
    T* hr = static_cast<T*>(a.h) + r * a.ldh;
    Moments m1{};
    if (a.post) m1 = moments(yr);
    for (int64_t c = threadIdx.x * V; c < n; c += 1024 * V) {
      const Pack<T, V> py = load_pack<T, V>(yr, c, n), px = load_pack<T, V>(xr, c, n);
      Pack<T, V> p;
#pragma unroll
      for (int i = 0; i < V; ++i) {
        if (c + i >= n) continue;
        float u = to_f32(py.v[i]);
        if (a.post) u = fmaf((u - m1.mean - m1.rest) * m1.rstd, param(a.w1, c + i, 1.f), param(a.b1, c + i, 0.f));
        const float g = gr ? to_f32(gr[c + i]) : a.gate_kind == kGateVector ? load_any(a.gate, a.wdtype, c + i) : 1.f;
        p.v[i] = kept<T>(fmaf(a.alpha, to_f32(px.v[i]), a.beta * (g * u)));
      }
      store_pack<T, V>(hr, c, n, p);
    }
    if (a.stats && a.post && threadIdx.x == 0) {
      a.stats[r] = m1.mean;
      a.stats[a.rows + r] = m1.rstd;
    }
    if (!a.pre) continue;
    const Moments m2 = moments(hr);
    T* zr = static_cast<T*>(a.z) + r * a.ldz;
    for (int64_t c = threadIdx.x * V; c < n; c += 1024 * V) {
      Pack<T, V> p = load_pack<T, V>(static_cast<const T*>(hr), c, n);
#pragma unroll
      for (int i = 0; i < V; ++i)
        if (c + i < n)
          p.v[i] = from_f32<T>(fmaf((to_f32(p.v[i]) - m2.mean - m2.rest) * m2.rstd, param(a.w2, c + i, 1.f), param(a.b2, c + i, 0.f)));
      store_pack<T, V>(zr, c, n, p);
    }
    if (a.stats && threadIdx.x == 0) {
      a.stats[2 * a.rows + r] = m2.mean;
      a.stats[3 * a.rows + r] = m2.rstd;
    }
  }
}

}  // namespace

hipError_t launch_residual_forward(const ResidualForward& a, hipStream_t s) {
  if (a.rows == 0) return hipSuccess;
  return with_type(a.dtype, [&](auto t) {
    using T = decltype(t);
    if (a.cols > kLongestResidualRow) {
      k_residual_forward_long<T><<<dim3(unsigned(a.rows < 4096 ? a.rows : 4096)), dim3(1024), 0, s>>>(a);
      return hipGetLastError();
    }
    return with_residual_layout(a.cols, [&](auto l) {
      using L = decltype(l);
      const int64_t need = (a.rows + L::ROWS - 1) / L::ROWS, most = int64_t(2048) * 256 / L::BLOCK;
      const dim3 grid(unsigned(need < most ? need : most)), block(L::BLOCK);
      with_residual_mode<T, L>(a.cols, [&](auto mode) { k_residual_forward<T, L, mode()><<<grid, block, 0, s>>>(a); });
      return hipGetLastError();
    });
  });
}

}  // namespace lopt
