// Backward pass of the residual update with its norms.  Per row of n columns, with
// hh = (h - mean2) rstd2, yh = (y - mean1) rstd1 and u = yh w1 + b1 (or y):
//   D  = dh + rstd2 (a - hh mean(a hh) - mean(a)),  a = dz w2     (RMS: without mean(a))
//   dx = alpha D,  E = beta D,  dgate = E u,  du = E gate
//   dy = rstd1 (b - yh mean(b yh) - mean(b)),  b = du w1         (or du)
// The means that the forward pass kept are floats; what they leave of a row far
// from zero, in units of its spread, is the mean that (h - mean2) rstd2 still
// has, and is taken off hh and yh.
// And over the rows dw2 = sum dz hh, db2 = sum dz, dw1 = sum du yh, db1 = sum du
// and a gate vector's sum of dgate.
// Bound by HBM: dh, dz, y, h (and a gate matrix) are read once, dx and dy (and
// the matrix's gradient) written once; a block's next row is loaded before the sums of this one.  Each thread adds up its columns'
// sums over the rows of its block in registers; the blocks' sums go to the workspace and a
// second kernel adds them in the order of the blocks: the same bits every time (65536 x 2048
// bf16, RMS: 305 to 335 us, 4.8 to 5.3 TB/s, and 5 for the second kernel).
#include <hip/hip_runtime.h>

#include <algorithm>

#include "lopt_residual_norm.h"

namespace lopt {
namespace {

// Whether a row lies farther from zero than it is wide.  In others half a step of the mean is below the roundings of
// (x - mean) rstd themselves, and nothing is taken off (65536 x 2048 bf16, layer norm of y alone: 194 us, 202 with the sums taken
// of every row, 191 without any; norms on both sides 346, 336 without).
__device__ __forceinline__ bool is_far(float mean, float rstd) { return fabsf(mean) * rstd > 1.f; }

enum : int { kW1 = 0, kB1 = 1, kW2 = 2, kB2 = 3, kGate = 4, kSums = 5 };   // of ResidualBackward::sums

template <class T, class L, int MODE, bool RMS, bool POST, bool PRE>
__global__ __launch_bounds__(L::BLOCK) void k_residual_backward(ResidualBackward a) {
  constexpr int V = kVec<T>, NV = L::E / V, E = L::E;
  __shared__ float red[2][L::TPR > 64 ? L::TPR / 64 : 1][2], red_left[2][L::TPR > 64 ? L::TPR / 64 : 1][2];
  RowSum<L::TPR, 2> row_sum{red}, left_sum{red_left};
  const int lane = threadIdx.x % L::TPR;
  const int n = int(a.cols);
  const float inv_n = 1.f / float(n);

  RowAt<T, L, MODE> at(lane, n);
  float w1[E], b1[E], gate[E], w2[E], sum[kSums][E];
  if (POST) load_weights(at, a.w1, a.wdtype, 1.f, w1);
  if (POST) load_weights(at, a.gate_kind != kNoGate ? a.b1 : nullptr, a.wdtype, 0.f, b1);
  load_weights(at, a.gate_kind == kGateVector ? a.gate : nullptr, a.wdtype, 1.f, gate);
  if (PRE) load_weights(at, a.w2, a.wdtype, 1.f, w2);
#pragma unroll
  for (int k = 0; k < kSums; ++k)
#pragma unroll
    for (int e = 0; e < E; ++e) sum[k][e] = 0.f;

  struct Row {
    RowPacks<T, RowAt<T, L, MODE>> y, h, dh, dz, gate;
    float mean1, rstd1, mean2, rstd2;
  };
  const auto load = [&](int64_t r0) {
    const int64_t r = r0 + threadIdx.x / L::TPR, rr = r < a.rows ? r : 0;
    Row p;
    p.y.load(at, static_cast<const T*>(a.y) + rr * a.ldy);
    if (PRE) p.h.load(at, static_cast<const T*>(a.h) + rr * a.ldh);
    if (a.dh) p.dh.load(at, static_cast<const T*>(a.dh) + rr * a.lddh);
    if (PRE && a.dz) p.dz.load(at, static_cast<const T*>(a.dz) + rr * a.lddz);
    if (a.gate_kind == kGateMatrix) p.gate.load(at, static_cast<const T*>(a.gate) + rr * a.ldg);
    p.mean1 = POST && !RMS ? a.stats[rr] : 0.f;
    p.rstd1 = POST ? a.stats[a.rows + rr] : 0.f;
    p.mean2 = PRE && !RMS ? a.stats[2 * a.rows + rr] : 0.f;
    p.rstd2 = PRE ? a.stats[3 * a.rows + rr] : 0.f;
    return p;
  };
  const int64_t stride = int64_t(gridDim.x) * L::ROWS, first = int64_t(blockIdx.x) * L::ROWS;
  Row next = load(first);
  for (int64_t r0 = first; r0 < a.rows; r0 += stride) {
    const int64_t r = r0 + threadIdx.x / L::TPR;
    const bool row = L::ROWS == 1 || r < a.rows;
    const Row now = next;
    if (r0 + stride < a.rows) next = load(r0 + stride);
    float d[E], y[E], h[E], dz[E];
    now.y.open(at, y);
    if (PRE) now.h.open(at, h);
    if (a.dh) now.dh.open(at, d);
    if (PRE && a.dz) now.dz.open(at, dz);
    if (a.gate_kind == kGateMatrix) now.gate.open(at, gate);
    const float mean1 = now.mean1, rstd1 = now.rstd1, mean2 = now.mean2, rstd2 = now.rstd2;
#pragma unroll
    for (int e = 0; e < E; ++e)
      if (!a.dh || !row) d[e] = 0.f;
    if (PRE)
#pragma unroll
      for (int k = 0; k < NV; ++k)
#pragma unroll
        for (int i = 0; i < V; ++i) h[k * V + i] = row && at[k].own(i) ? (h[k * V + i] - mean2) * rstd2 : 0.f;
    if (POST)
#pragma unroll
      for (int k = 0; k < NV; ++k)
#pragma unroll
        for (int i = 0; i < V; ++i) y[k * V + i] = row && at[k].own(i) ? (y[k * V + i] - mean1) * rstd1 : 0.f;
    if constexpr (!RMS) {
      const bool far1 = POST && is_far(mean1, rstd1), far2 = PRE && is_far(mean2, rstd2);
      if (far1 || far2) {   // the same for all threads of a row, and where a row's sum has a barrier a block has one row
        float v[2] = {0.f, 0.f};
#pragma unroll
        for (int e = 0; e < E; ++e) {
          if (PRE) v[0] += h[e];
          if (POST) v[1] += y[e];
        }
        left_sum(v);
        const float left2 = far2 ? v[0] * inv_n : 0.f, left1 = far1 ? v[1] * inv_n : 0.f;
#pragma unroll
        for (int k = 0; k < NV; ++k)
#pragma unroll
          for (int i = 0; i < V; ++i)
            if (row && at[k].own(i)) {
              if (PRE) h[k * V + i] -= left2;
              if (POST) y[k * V + i] -= left1;
            }
      }
    }
    if (PRE) {
      float v[2] = {0.f, 0.f};
#pragma unroll
      for (int e = 0; e < E; ++e) {
        if (!a.dz || !row) dz[e] = 0.f;
        sum[kW2][e] = fmaf(dz[e], h[e], sum[kW2][e]);
        if (!RMS) sum[kB2][e] += dz[e];
        dz[e] *= w2[e];
        v[0] = fmaf(dz[e], h[e], v[0]);
        v[1] += dz[e];
      }
      row_sum(v);
      const float c1 = v[0] * inv_n, c2 = RMS ? 0.f : v[1] * inv_n;
#pragma unroll
      for (int k = 0; k < NV; ++k)
#pragma unroll
        for (int i = 0; i < V; ++i) {
          const int e = k * V + i;
          const float x = fmaf(rstd2, dz[e] - fmaf(h[e], c1, c2), d[e]);
          d[e] = row && at[k].own(i) ? x : 0.f;
        }
    }
    if (a.dx && row) {
      float x[E];
#pragma unroll
      for (int e = 0; e < E; ++e) x[e] = a.alpha * d[e];
      store_row(at, static_cast<T*>(a.dx) + r * a.lddx, x);
    }
#pragma unroll
    for (int e = 0; e < E; ++e) d[e] *= a.beta;
    if (a.gate_kind != kNoGate) {
      float x[E];
#pragma unroll
      for (int e = 0; e < E; ++e) x[e] = d[e] * (POST ? fmaf(y[e], w1[e], b1[e]) : y[e]);
      if (a.gate_kind == kGateVector) {
#pragma unroll
        for (int e = 0; e < E; ++e)
          if (row) sum[kGate][e] += x[e];
      } else if (a.dgate && row) {
        store_row(at, static_cast<T*>(a.dgate) + r * a.lddg, x);
      }
#pragma unroll
      for (int e = 0; e < E; ++e) d[e] *= gate[e];
    }
    if (POST) {
      float v[2] = {0.f, 0.f};
#pragma unroll
      for (int k = 0; k < NV; ++k)
#pragma unroll
        for (int i = 0; i < V; ++i) {
          const int e = k * V + i;
          if (!row || !at[k].own(i)) d[e] = 0.f;   // a gate may be no number where nothing is the thread's
          sum[kW1][e] = fmaf(d[e], y[e], sum[kW1][e]);
          if (!RMS) sum[kB1][e] += d[e];
          d[e] *= w1[e];
          v[0] = fmaf(d[e], y[e], v[0]);
          v[1] += d[e];
        }
      if (a.dy) {
        row_sum(v);
        const float c1 = v[0] * inv_n, c2 = RMS ? 0.f : v[1] * inv_n;
#pragma unroll
        for (int e = 0; e < E; ++e) d[e] = rstd1 * (d[e] - fmaf(y[e], c1, c2));
      }
    }
    if (a.dy && row) store_row(at, static_cast<T*>(a.dy) + r * a.lddy, d);
  }
  if (!a.part) return;

  // the block's sums, those that there are one behind the other: the row groups of a wave, then the waves in order
  constexpr int GROUPS = L::ROWS > 1 ? L::BLOCK / 64 : 1;   // waves that hold the same columns
  constexpr int LPW = L::TPR < 64 ? L::TPR : 64;            // lanes of a wave with columns of their own
  __shared__ float joined[GROUPS > 1 ? GROUPS : 1][GROUPS > 1 ? E * LPW : 1];
  float* out = a.part + size_t(blockIdx.x) * size_t(kSums) * size_t(n);
#pragma unroll
  for (int k = 0; k < kSums; ++k) {
    if (!a.sums[k]) continue;
    if constexpr (GROUPS == 1) {
#pragma unroll
      for (int q = 0; q < NV; ++q)
#pragma unroll
        for (int i = 0; i < V; ++i)
          if (at[q].own(i)) out[at[q].at + i] = sum[k][q * V + i];
    } else {
      if constexpr (LPW == 8)
#pragma unroll
        for (int e = 0; e < E; ++e) sum[k][e] = groups_sum(sum[k][e]);
      __syncthreads();   // of the sum before, everything is read
      if ((threadIdx.x & 63) < LPW)
#pragma unroll
        for (int e = 0; e < E; ++e) joined[threadIdx.x >> 6][e * LPW + lane] = sum[k][e];
      __syncthreads();
      // a column is the own element of the thread and vector that it falls to; the last vector of kTail has moved back
      const int moved = MODE == kTail ? (n + V - 1) / V * V - n : 0;
      for (int c = threadIdx.x; c < n; c += L::BLOCK) {
        const int vec = c / V, i = c % V + (vec == n / V ? moved : 0), from = ((vec / LPW) * V + i) * LPW + vec % LPW;
        float t = joined[0][from];
#pragma unroll
        for (int g = 1; g < GROUPS; ++g) t += joined[g][from];
        out[c] = t;
      }
    }
    out += n;
  }
}

// Rows longer than kLongestResidualRow: one block a row.  Up to kLongBlocks rows, each leaves its columns' sums itself; of more,
// the two means of the second norm's gradient and what the kept means leave stay in the workspace for the column sums.
constexpr int64_t kLongBlocks = 64;
struct LongRow {
  float mean1, rstd1, mean2, rstd2, c1, c2, left1, left2;
};
template <class T>
struct LongElement {   // column c of a row
  float hh, dz, d, u, yh, e, du;
  __device__ __forceinline__ LongElement(const ResidualBackward& a, const LongRow& m, int64_t r, int64_t c) {
    const auto param = [&](const void* p, float fill) { return p ? load_any(p, a.wdtype, c) : fill; };
    hh = a.pre ? (to_f32(static_cast<const T*>(a.h)[r * a.ldh + c]) - m.mean2) * m.rstd2 - m.left2 : 0.f;
    dz = a.pre && a.dz ? to_f32(static_cast<const T*>(a.dz)[r * a.lddz + c]) : 0.f;
    d = a.dh ? to_f32(static_cast<const T*>(a.dh)[r * a.lddh + c]) : 0.f;
    if (a.pre) d = fmaf(m.rstd2, dz * param(a.w2, 1.f) - fmaf(hh, m.c1, m.c2), d);
    const float y = to_f32(static_cast<const T*>(a.y)[r * a.ldy + c]);
    yh = a.post ? (y - m.mean1) * m.rstd1 - m.left1 : 0.f;
    u = a.post ? fmaf(yh, param(a.w1, 1.f), param(a.b1, 0.f)) : y;
    e = a.beta * d;
    du = e * (a.gate_kind == kGateVector ? load_any(a.gate, a.wdtype, c)
              : a.gate_kind == kGateMatrix ? to_f32(static_cast<const T*>(a.gate)[r * a.ldg + c]) : 1.f);
  }
};
__device__ __forceinline__ LongRow long_row(const ResidualBackward& a, int64_t r) {
  LongRow m{};
  if (a.post && !a.rms) m.mean1 = a.stats[r];
  if (a.post) m.rstd1 = a.stats[a.rows + r];
  if (a.pre && !a.rms) m.mean2 = a.stats[2 * a.rows + r];
  if (a.pre) m.rstd2 = a.stats[3 * a.rows + r];
  return m;
}

struct ColumnSums {   // of one column, over some rows
  float sum[kSums] = {};
  template <class T>
  __device__ __forceinline__ void add(const LongElement<T>& x) {
    sum[kW1] = fmaf(x.du, x.yh, sum[kW1]);
    sum[kB1] += x.du;
    sum[kW2] = fmaf(x.dz, x.hh, sum[kW2]);
    sum[kB2] += x.dz;
    sum[kGate] = fmaf(x.e, x.u, sum[kGate]);
  }
  // those that are wanted, one behind the other
  __device__ __forceinline__ void store(const ResidualBackward& a, int64_t block, int64_t c) const {
    float* out = a.part + size_t(block) * size_t(kSums) * size_t(a.cols) + c;
#pragma unroll
    for (int k = 0; k < kSums; ++k)
      if (a.sums[k]) {
        *out = sum[k];
        out += a.cols;
      }
  }
};

template <class T>
__global__ __launch_bounds__(1024) void k_residual_backward_long(ResidualBackward a, float* means) {
  __shared__ float red[2][16][2];
  RowSum<1024, 2> row_sum{red};
  const int64_t n = a.cols;
  const float inv_n = 1.f / float(n);
  for (int64_t r = blockIdx.x; r < a.rows; r += gridDim.x) {
    LongRow m = long_row(a, r);
    const bool far1 = !a.rms && a.post && is_far(m.mean1, m.rstd1), far2 = !a.rms && a.pre && is_far(m.mean2, m.rstd2);
    if (far1 || far2) {
      float v[2] = {0.f, 0.f};
      for (int64_t c = threadIdx.x; c < n; c += 1024) {
        if (far2) v[0] += to_f32(static_cast<const T*>(a.h)[r * a.ldh + c]) - m.mean2;
        if (far1) v[1] += to_f32(static_cast<const T*>(a.y)[r * a.ldy + c]) - m.mean1;
      }
      row_sum(v);
      if (far2) m.left2 = v[0] * inv_n * m.rstd2;
      if (far1) m.left1 = v[1] * inv_n * m.rstd1;
    }
    if (a.pre) {
      float v[2] = {0.f, 0.f};
      for (int64_t c = threadIdx.x; c < n; c += 1024) {
        const LongElement<T> x(a, m, r, c);
        const float b = x.dz * (a.w2 ? load_any(a.w2, a.wdtype, c) : 1.f);
        v[0] = fmaf(b, x.hh, v[0]);
        v[1] += b;
      }
      row_sum(v);
      m.c1 = v[0] * inv_n;
      m.c2 = a.rms ? 0.f : v[1] * inv_n;
    }
    if (means && threadIdx.x == 0) {
      means[4 * r] = m.c1;
      means[4 * r + 1] = m.c2;
      means[4 * r + 2] = m.left1;
      means[4 * r + 3] = m.left2;
    }
    float v[2] = {0.f, 0.f};
    for (int64_t c = threadIdx.x; c < n; c += 1024) {
      const LongElement<T> x(a, m, r, c);
      if (a.part && !means) {
        ColumnSums s;
        s.add(x);
        s.store(a, r, c);
      }
      if (a.dx) static_cast<T*>(a.dx)[r * a.lddx + c] = from_f32<T>(a.alpha * x.d);
      if (a.gate_kind == kGateMatrix && a.dgate) static_cast<T*>(a.dgate)[r * a.lddg + c] = from_f32<T>(x.e * x.u);
      if (a.post) {
        const float b = x.du * (a.w1 ? load_any(a.w1, a.wdtype, c) : 1.f);
        v[0] = fmaf(b, x.yh, v[0]);
        v[1] += b;
      } else if (a.dy) {
        static_cast<T*>(a.dy)[r * a.lddy + c] = from_f32<T>(x.du);
      }
    }
    if (!a.post || !a.dy) continue;
    row_sum(v);
    const float c1 = v[0] * inv_n, c2 = a.rms ? 0.f : v[1] * inv_n;
    for (int64_t c = threadIdx.x; c < n; c += 1024) {
      const LongElement<T> x(a, m, r, c);
      const float b = x.du * (a.w1 ? load_any(a.w1, a.wdtype, c) : 1.f);
      static_cast<T*>(a.dy)[r * a.lddy + c] = from_f32<T>(m.rstd1 * (b - fmaf(x.yh, c1, c2)));
    }
  }
}

// Column sums over every gridDim.y-th row; means: four floats a row.
template <class T>
__global__ __launch_bounds__(256) void k_residual_columns_long(ResidualBackward a, const float* means) {
  const int64_t n = a.cols, c = int64_t(blockIdx.x) * 256 + threadIdx.x;
  if (c >= n) return;
  ColumnSums s;
  for (int64_t r = blockIdx.y; r < a.rows; r += gridDim.y) {
    LongRow m = long_row(a, r);
    m.c1 = means[4 * r];
    m.c2 = means[4 * r + 1];
    m.left1 = means[4 * r + 2];
    m.left2 = means[4 * r + 3];
    s.add(LongElement<T>(a, m, r, c));
  }
  s.store(a, blockIdx.y, c);
}

// The parameters' gradients from the blocks' sums: 32 columns a block at a time, 32
// threads a column, each adding up every 32nd block's sum; the 32 results are added in order.
__global__ __launch_bounds__(1024) void k_residual_join(ResidualBackward a, int64_t blocks) {
  __shared__ float s[32][33];
  const int64_t n = a.cols, pitch = int64_t(kSums) * n;
  const int g = threadIdx.x / 32;
  int64_t width = 0;
#pragma unroll
  for (int k = 0; k < kSums; ++k) width += a.sums[k] ? n : 0;
  for (int64_t c0 = int64_t(blockIdx.x) * 32; c0 < width; c0 += int64_t(gridDim.x) * 32) {
    const int64_t c = c0 + threadIdx.x % 32;
    float t = 0.f;
    if (c < width) {
#pragma unroll 8
      for (int64_t b = g; b < blocks; b += 32) t += a.part[b * pitch + c];
    }
    s[g][threadIdx.x % 32] = t;
    __syncthreads();
    if (g == 0 && c < width) {
      t = 0.f;
#pragma unroll
      for (int k = 0; k < 32; ++k) t += s[k][threadIdx.x];
      int64_t i = c;
      bool done = false;
#pragma unroll
      for (int k = 0; k < kSums; ++k)
        if (a.sums[k] && !done) {
          if (i < n) {
            store_any(a.sums[k], a.gdtype, i, a.accumulate ? load_any(a.sums[k], a.gdtype, i) + t : t);
            done = true;
          }
          i -= n;
        }
    }
    __syncthreads();   // s is written again
  }
}

int64_t backward_blocks(int64_t rows, int64_t cols) {
  if (rows <= 0) return 0;
  if (cols > kLongestResidualRow) return std::min<int64_t>(rows, kLongBlocks);
  return with_residual_layout(cols, [&](auto l) {
    using L = decltype(l);
    // two rounds of rows a block (fewer sums to join) once every compute unit has a block, and no more blocks than are resident
    // together (65536 x 2048 bf16, RMS: 358 us with 1024 blocks of 256 threads, 321 with 512)
    const int64_t need = (rows + L::ROWS - 1) / L::ROWS, cap = int64_t(512) * 256 / L::BLOCK;
    return std::min<int64_t>(std::max<int64_t>(std::min<int64_t>(need, 256), (need + 1) / 2), cap);
  });
}

}  // namespace

size_t residual_backward_bytes(int64_t rows, int64_t cols) {
  const size_t sums = size_t(kSums) * size_t(cols) * sizeof(float);   // of a block
  size_t bytes = size_t(backward_blocks(rows, cols)) * sums;
  if (cols > kLongestResidualRow) {   // four floats a row, two of them in the room of whole blocks' sums
    const size_t half = size_t(rows) * 2 * sizeof(float);
    bytes += half + (rows > kLongBlocks ? (half + sums - 1) / sums * sums : 0);
  }
  return bytes;
}

hipError_t launch_residual_backward(const ResidualBackward& args, hipStream_t s) {
  ResidualBackward a = args;
  const int64_t blocks = backward_blocks(a.rows, a.cols);
  int64_t width = 0;
  for (void* p : a.sums) width += p ? a.cols : 0;
  if (!width) a.part = nullptr;
  if (a.rows > 0) {
    const hipError_t e = with_type(a.dtype, [&](auto t) {
      using T = decltype(t);
      if (a.cols > kLongestResidualRow) {
        float* means = a.part && a.rows > kLongBlocks ? a.part + size_t(blocks) * size_t(kSums) * size_t(a.cols) : nullptr;
        k_residual_backward_long<T><<<dim3(unsigned(std::min<int64_t>(a.rows, 4096))), dim3(1024), 0, s>>>(a, means);
        if (means) k_residual_columns_long<T><<<dim3(unsigned((a.cols + 255) / 256), unsigned(blocks)), dim3(256), 0, s>>>(a, means);
        return hipGetLastError();
      }
      return with_residual_layout(a.cols, [&](auto l) {
        using L = decltype(l);
        const dim3 grid{unsigned(blocks)}, block{L::BLOCK};
        with_residual_mode<T, L>(a.cols, [&](auto mode) {
          const auto norms = [&](auto rms) {
            if (a.post && a.pre) k_residual_backward<T, L, mode(), rms(), true, true><<<grid, block, 0, s>>>(a);
            else if (a.post) k_residual_backward<T, L, mode(), rms(), true, false><<<grid, block, 0, s>>>(a);
            else k_residual_backward<T, L, mode(), rms(), false, true><<<grid, block, 0, s>>>(a);
          };
          if (a.rms) norms(std::true_type());
          else norms(std::false_type());
        });
        return hipGetLastError();
      });
    });
    if (e != hipSuccess) return e;
  }
  if (!width) return hipSuccess;
  k_residual_join<<<dim3(unsigned(std::min<int64_t>((width + 31) / 32, 1 << 20))), dim3(1024), 0, s>>>(a, blocks);
  return hipGetLastError();
}

}  // namespace lopt
