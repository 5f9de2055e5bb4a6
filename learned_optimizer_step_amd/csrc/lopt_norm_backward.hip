// Backward pass of layer norm and RMS norm.  With xh = (x - mu) rstd and
// a = dy w, per row of n columns:
//   dx = rstd (a - xh mean(a xh) - mean(a))      (RMS: without mean(a))
//   dw = sum over rows of dy xh,  db = sum over rows of dy
// Bound by HBM: x and dy are read once, dx is written once.  x and dy have no
// further reader, and are read past the caches (65536 x 768 bf16: 64 to 56 us);
// so is dx written if the memory-side cache could not hold it for its reader
// (65536 x 2048 bf16 RMS, 268 MB: 147 to 140 us; 16384 x 2048: 46 to 51, not so).  Each thread adds
// up dw and db of its columns over the rows of its block in registers; the
// blocks' sums go to the workspace and a second kernel adds them in the order
// of the blocks, so the result has the same bits every time.
#include <hip/hip_runtime.h>

#include <algorithm>

#include "lopt_norm.h"

namespace lopt {
namespace {

template <class T, class L, bool RMS, int MODE, bool PASS_BY = false>
__global__ __launch_bounds__(L::BLOCK) void k_norm_backward(NormBackward a) {
  constexpr int V = kVec<T>, NV = L::E / V, E = L::E;
  __shared__ float red[2][L::TPR > 64 ? L::TPR / 64 : 1][2];
  RowSum<L::TPR, 2> row_sum{red};
  const int lane = threadIdx.x % L::TPR;
  const int n = int(a.cols);
  const float inv_n = 1.f / float(n);

  float w[E], dw[E], db[RMS ? 1 : E];
  RowAt<T, L, MODE> at(lane, n);
  load_weights(at, a.w, a.wdtype, 1.f, w);
#pragma unroll
  for (int e = 0; e < E; ++e) {
    dw[e] = 0.f;
    if (!RMS) db[e] = 0.f;
  }

  const int64_t stride = int64_t(gridDim.x) * L::ROWS;
  for (int64_t r0 = int64_t(blockIdx.x) * L::ROWS; r0 < a.rows; r0 += stride) {
    const int64_t r = r0 + threadIdx.x / L::TPR;
    const bool row = L::ROWS == 1 || r < a.rows;
    const int64_t rr = row ? r : 0;
    const T* xr = static_cast<const T*>(a.x) + rr * a.ldx;
    const T* gr = static_cast<const T*>(a.dy) + rr * a.lddy;
    const float mean = RMS ? 0.f : a.mean[rr], rstd = a.rstd[rr];
    float xh[E], g[E];
    float v[2] = {0.f, 0.f};
    Pack<T, V> px[NV], pg[NV];
#pragma unroll
    for (int k = 0; k < NV; ++k) {
      if constexpr (MODE == kWhole || PASS_BY) {
        px[k] = at[k].load_once(xr);
        pg[k] = at[k].load_once(gr);
      } else {   // unaligned vectors share cache lines with their neighbours: 5003 x 1025 fp32 20 us, 23 past the caches
        px[k] = at[k].load(xr);
        pg[k] = at[k].load(gr);
      }
    }
#pragma unroll
    for (int k = 0; k < NV; ++k)
#pragma unroll
      for (int i = 0; i < V; ++i) {
        const bool own = row && at[k].own(i);
        xh[k * V + i] = own ? (to_f32(px[k].v[i]) - mean) * rstd : 0.f;
        g[k * V + i] = own ? to_f32(pg[k].v[i]) : 0.f;
      }
#pragma unroll
    for (int e = 0; e < E; ++e) {
      dw[e] = fmaf(g[e], xh[e], dw[e]);
      if (!RMS) db[e] += g[e];
      g[e] *= w[e];
      v[0] = fmaf(g[e], xh[e], v[0]);
      v[1] += g[e];
    }
    if (!a.dx) continue;   // the same for every thread
    row_sum(v);
    if (!row) continue;
    const float c1 = v[0] * inv_n, c2 = RMS ? 0.f : v[1] * inv_n;
    T* dr = static_cast<T*>(a.dx) + r * a.lddx;
#pragma unroll
    for (int k = 0; k < NV; ++k) {
#pragma unroll
      for (int i = 0; i < V; ++i) px[k].v[i] = from_f32<T>(rstd * (g[k * V + i] - fmaf(xh[k * V + i], c1, c2)));
      at[k].template store<PASS_BY>(dr, px[k]);
    }
  }
  if (!a.dw && !a.db) return;

  // the block's sums: the row groups of a wave, then the waves in order
  constexpr int GROUPS = L::ROWS > 1 ? L::BLOCK / 64 : 1;   // waves that hold the same columns
  float* out = a.part + size_t(blockIdx.x) * size_t(RMS ? n : 2 * n);
  if constexpr (GROUPS == 1) {
#pragma unroll
    for (int k = 0; k < NV; ++k)
#pragma unroll
      for (int i = 0; i < V; ++i) {
        const int c = at[k].at + i;
        if (at[k].own(i)) {
          out[c] = dw[k * V + i];
          if (!RMS) out[n + c] = db[k * V + i];
        }
      }
  } else {
    constexpr int LPW = L::TPR < 64 ? L::TPR : 64;   // lanes of a wave with columns of their own
    __shared__ float sums[RMS ? 1 : 2][GROUPS][E * LPW];
    if constexpr (LPW == 8)
#pragma unroll
      for (int e = 0; e < E; ++e) {
        dw[e] = groups_sum(dw[e]);
        if (!RMS) db[e] = groups_sum(db[e]);
      }
    const int wave = threadIdx.x >> 6;
    if ((threadIdx.x & 63) < LPW)
#pragma unroll
      for (int e = 0; e < E; ++e) {
        sums[0][wave][e * LPW + lane] = dw[e];
        if (!RMS) sums[RMS ? 0 : 1][wave][e * LPW + lane] = db[e];
      }
    __syncthreads();
    // a column is the own element of the thread and vector that it falls to; the last vector of kTail has moved back
    const int moved = MODE == kTail ? (n + V - 1) / V * V - n : 0;
    for (int c = threadIdx.x; c < n; c += L::BLOCK) {
      const int vec = c / V, i = c % V + (vec == n / V ? moved : 0), at = ((vec / LPW) * V + i) * LPW + vec % LPW;
#pragma unroll
      for (int k = 0; k < (RMS ? 1 : 2); ++k) {
        float t = sums[k][0][at];
#pragma unroll
        for (int g = 1; g < GROUPS; ++g) t += sums[k][g][at];
        out[k * n + c] = t;
      }
    }
  }
}

// Rows longer than kLongestRow: dx with one block a row, dw and db by column
// strips over the rows.
template <class T>
__global__ __launch_bounds__(1024) void k_norm_backward_long(NormBackward a) {
  constexpr int V = kVec<T>;
  __shared__ float red[2][16][2];
  RowSum<1024, 2> row_sum{red};
  const int64_t n = a.cols;
  const float inv_n = 1.f / float(n);
  for (int64_t r = blockIdx.x; r < a.rows; r += gridDim.x) {
    const T* xr = static_cast<const T*>(a.x) + r * a.ldx;
    const T* gr = static_cast<const T*>(a.dy) + r * a.lddy;
    T* dr = static_cast<T*>(a.dx) + r * a.lddx;
    const float mean = a.rms ? 0.f : a.mean[r], rstd = a.rstd[r];
    float v[2] = {0.f, 0.f};
    for (int64_t c = threadIdx.x * V; c < n; c += 1024 * V) {
      const Pack<T, V> px = load_pack<T, V>(xr, c, n), pg = load_pack<T, V>(gr, c, n);
#pragma unroll
      for (int i = 0; i < V; ++i)
        if (c + i < n) {
          const float g = to_f32(pg.v[i]) * (a.w ? load_any(a.w, a.wdtype, c + i) : 1.f);
          v[0] = fmaf(g, (to_f32(px.v[i]) - mean) * rstd, v[0]);
          v[1] += g;
        }
    }
    row_sum(v);
    const float c1 = v[0] * inv_n, c2 = a.rms ? 0.f : v[1] * inv_n;
    for (int64_t c = threadIdx.x * V; c < n; c += 1024 * V) {
      const Pack<T, V> px = load_pack<T, V>(xr, c, n), pg = load_pack<T, V>(gr, c, n);
      Pack<T, V> p;
#pragma unroll
      for (int i = 0; i < V; ++i) {
        const float g = to_f32(pg.v[i]) * (a.w && c + i < n ? load_any(a.w, a.wdtype, c + i) : 1.f);
        p.v[i] = from_f32<T>(rstd * (g - fmaf((to_f32(px.v[i]) - mean) * rstd, c1, c2)));
      }
      store_pack<T, V>(dr, c, n, p);
    }
  }
}

// Column sums of a strip of 1024 elements over every gridDim.y-th row.
template <class T>
__global__ __launch_bounds__(256) void k_norm_columns_long(NormBackward a) {
  constexpr int V = 4;
  const int64_t n = a.cols, c = (int64_t(blockIdx.x) * 256 + threadIdx.x) * V;
  if (c >= n) return;
  float dw[V] = {}, db[V] = {};
  for (int64_t r = blockIdx.y; r < a.rows; r += gridDim.y) {
    const float mean = a.rms ? 0.f : a.mean[r], rstd = a.rstd[r];
    const Pack<T, V> px = load_pack<T, V>(static_cast<const T*>(a.x) + r * a.ldx, c, n);
    const Pack<T, V> pg = load_pack<T, V>(static_cast<const T*>(a.dy) + r * a.lddy, c, n);
#pragma unroll
    for (int i = 0; i < V; ++i) {
      const float g = to_f32(pg.v[i]);
      dw[i] = fmaf(g, (to_f32(px.v[i]) - mean) * rstd, dw[i]);
      db[i] += g;
    }
  }
  float* out = a.part + size_t(blockIdx.y) * size_t(a.rms ? n : 2 * n);
#pragma unroll
  for (int i = 0; i < V; ++i)
    if (c + i < n) {
      out[c + i] = dw[i];
      if (!a.rms) out[n + c + i] = db[i];
    }
}

// dw and db from the blocks' sums: 32 columns a block at a time, 32 threads a
// column, each adding up every 32nd block's sum; the 32 results are added in
// order.
constexpr int64_t kJoinBlocks = 1 << 20;   // a grid has room for 2^32 - 1 threads a dimension
__global__ __launch_bounds__(1024) void k_norm_weight_grad(NormBackward a, int64_t blocks) {
  __shared__ float s[32][33];
  const int64_t n = a.cols, width = a.rms ? n : 2 * n;
  const int g = threadIdx.x / 32;
  for (int64_t c0 = int64_t(blockIdx.x) * 32; c0 < width; c0 += int64_t(gridDim.x) * 32) {
    const int64_t c = c0 + threadIdx.x % 32;
    float sum = 0.f;
    if (c < width) {
#pragma unroll 8
      for (int64_t b = g; b < blocks; b += 32) sum += a.part[b * width + c];
    }
    s[g][threadIdx.x % 32] = sum;
    __syncthreads();
    if (g == 0 && c < width) {
      sum = 0.f;
#pragma unroll
      for (int k = 0; k < 32; ++k) sum += s[k][threadIdx.x];
      void* out = c < n ? a.dw : a.db;
      const int64_t i = c < n ? c : c - n;
      if (out) store_any(out, a.gdtype, i, a.accumulate ? load_any(out, a.gdtype, i) + sum : sum);
    }
    __syncthreads();   // s is written again
  }
}

}  // namespace

int64_t norm_backward_blocks(int64_t rows, int64_t cols) {
  if (rows <= 0) return 0;
  if (cols > kLongestRow) return std::min<int64_t>(rows, 64);
  return with_backward_layout(cols, [&](auto l) {
    using L = decltype(l);
    // two rounds of rows a block (fewer sums to join) once every compute unit has a block
    const int64_t need = (rows + L::ROWS - 1) / L::ROWS, cap = int64_t(1024) * 256 / L::BLOCK;
    return std::min<int64_t>(std::max<int64_t>(std::min<int64_t>(need, 256), (need + 1) / 2), cap);
  });
}

hipError_t launch_norm_backward(const NormBackward& a, hipStream_t s) {
  const int64_t blocks = norm_backward_blocks(a.rows, a.cols);
  const bool sums = a.dw || a.db;
  if (a.rows > 0 && (sums || a.dx)) {
    const hipError_t e = with_type(a.dtype, [&](auto t) {
      using T = decltype(t);
      if (a.cols > kLongestRow) {
        if (a.dx) k_norm_backward_long<T><<<dim3(unsigned(std::min<int64_t>(a.rows, 4096))), dim3(1024), 0, s>>>(a);
        if (sums) {
          const dim3 grid(unsigned((a.cols + 1023) / 1024), unsigned(blocks));
          k_norm_columns_long<T><<<grid, dim3(256), 0, s>>>(a);
        }
        return hipGetLastError();
      }
      return with_backward_layout(a.cols, [&](auto l) {
        using L = decltype(l);
        const dim3 grid{unsigned(blocks)}, block{L::BLOCK};
        if constexpr (L::TPR > 8)
          if (a.rows * a.cols * int64_t(sizeof(T)) > 200'000'000) {
            with_mode<T, L>(a.cols, [&](auto mode) {
              if (a.rms) k_norm_backward<T, L, true, mode(), true><<<grid, block, 0, s>>>(a);
              else k_norm_backward<T, L, false, mode(), true><<<grid, block, 0, s>>>(a);
            });
            return hipGetLastError();
          }
        with_mode<T, L>(a.cols, [&](auto mode) {
          if (a.rms) k_norm_backward<T, L, true, mode()><<<grid, block, 0, s>>>(a);
          else k_norm_backward<T, L, false, mode()><<<grid, block, 0, s>>>(a);
        });
        return hipGetLastError();
      });
    });
    if (e != hipSuccess) return e;
  }
  if (!sums) return hipSuccess;
  const int64_t width = a.rms ? a.cols : 2 * a.cols;
  k_norm_weight_grad<<<dim3(unsigned(std::min<int64_t>((width + 31) / 32, kJoinBlocks))), dim3(1024), 0, s>>>(a, blocks);
  return hipGetLastError();
}

}  // namespace lopt
