// Distillation from a teacher's top logits.  Per row, with the student's
// logits z (V of them), the teacher's list of ids i_k and logits u_k and a
// temperature tau:
//   p_k  = exp(u_k / tau) / sum_j exp(u_j / tau)
//   L    = log sum_v exp(z_v / tau)
//   loss = tau^2 sum_k p_k (log p_k - z_{i_k} / tau + L)
//   dz_v = g tau (exp(z_v / tau - L) - sum over k with i_k = v of p_k)
// An entry whose id lies outside [0, V) or whose logit is -inf is absent; a
// row without entries has loss 0 and gradient 0 whatever its logits are.
// Bound by HBM: the forward pass reads z once (the running maximum and sum of
// the softmax in one pass), the backward pass reads z and writes dz.
#include <hip/hip_runtime.h>

#include <algorithm>

#include "lopt_ops.h"
#include "lopt_ops_device.h"

namespace lopt {
namespace {

constexpr float kLog2e = 1.44269504088896340736f;
constexpr float kLn2 = 0.693147180559945309417f;

__device__ __forceinline__ float exp2_hw(float x) { return __builtin_amdgcn_exp2f(x); }

// Sum and maximum over a block of W waves, the same bits on every thread.
template <int W, class Op>
__device__ __forceinline__ float block_reduce(float x, float* red, Op op) {
  x = lanes_reduce<64>(x, op);
  __syncthreads();
  if ((threadIdx.x & 63) == 0) red[threadIdx.x >> 6] = x;
  __syncthreads();
  float s = red[0];
#pragma unroll
  for (int k = 1; k < W; ++k) s = op(s, red[k]);
  return s;
}

// The teacher's list of one row in LDS: id (-1: absent), probability, and for
// the loss log p.  Returns whether the row has an entry.
struct Teacher {
  int id[kMaxTop];
  float p[kMaxTop];
};

template <int B>
__device__ __forceinline__ bool load_teacher(Teacher& t, float* red, const void* ids, const void* u, int64_t row, int64_t ldi,
                                             int64_t ldu, int top, int64_t cols, int id_bytes, int udtype, float inv_tau,
                                             float& top_u, float& log_sum) {
  float most = -INFINITY;
  bool nan = false;
  for (int k = threadIdx.x; k < top; k += B) {
    const int64_t id = id_bytes == 8 ? static_cast<const int64_t*>(ids)[row * ldi + k]
                                     : int64_t(static_cast<const int32_t*>(ids)[row * ldi + k]);
    const float x = load_any(u, udtype, row * ldu + k) * inv_tau;
    const bool there = id >= 0 && id < cols && x != -INFINITY;
    t.id[k] = there ? int(id) : -1;
    t.p[k] = x;
    if (there) {
      most = fmaxf(most, x);
      nan |= x != x;
    }
  }
  const bool any = __syncthreads_or(most != -INFINITY || nan);
  if (!any) return false;
  most = block_reduce<B / 64>(most, red, Max());
  float sum = 0.f;
  for (int k = threadIdx.x; k < top; k += B) {
    const float e = t.id[k] >= 0 ? exp2_hw((t.p[k] - most) * kLog2e) : 0.f;
    sum += e;
  }
  sum = block_reduce<B / 64>(sum, red, Add());
  top_u = most;
  log_sum = logf(sum);
  return true;
}

// ---------------------------------------------------------------------------
// Forward: one block a row.
template <class T, int B>
__global__ __launch_bounds__(B) void k_distill_forward(DistillForward a) {
  constexpr int V = kVec<T>, W = B / 64, U = 4;
  __shared__ Teacher t;
  __shared__ float red[W];
  const int64_t n = a.cols;
  const float c = a.inv_tau * kLog2e;
  for (int64_t r = blockIdx.x; r < a.rows; r += gridDim.x) {
    const T* z = static_cast<const T*>(a.z) + r * a.ldz;
    // running maximum m of z and sum s of exp((z - m) / tau), per thread
    float m = -INFINITY, s = 0.f;
    auto take = [&](const Pack<T, V>* p, int count) {
      float top = m;
#pragma unroll
      for (int k = 0; k < U; ++k)
        if (k < count)
#pragma unroll
          for (int i = 0; i < V; ++i) top = fmaxf(top, to_f32(p[k].v[i]));
      const float mc = top == -INFINITY ? 0.f : top * c;   // all -inf so far: every term is exp(-inf) = 0
      s *= exp2_hw((m == -INFINITY ? -INFINITY : m * c - mc));
#pragma unroll
      for (int k = 0; k < U; ++k)
        if (k < count)
#pragma unroll
          for (int i = 0; i < V; ++i) s += exp2_hw(fmaf(to_f32(p[k].v[i]), c, -mc));
      m = top;
    };
    int64_t j = threadIdx.x * V;
    for (; j + int64_t(U - 1) * B * V + V <= n; j += int64_t(U) * B * V) {
      Pack<T, V> p[U];
#pragma unroll
      for (int k = 0; k < U; ++k) p[k] = *reinterpret_cast<const Pack<T, V>*>(z + j + int64_t(k) * B * V);
      take(p, U);
    }
    for (; j < n; j += int64_t(B) * V) {
      Pack<T, V> p[U];
      if (j + V <= n) {
        p[0] = *reinterpret_cast<const Pack<T, V>*>(z + j);
      } else {
#pragma unroll
        for (int i = 0; i < V; ++i) p[0].v[i] = j + i < n ? z[j + i] : from_f32<T>(-INFINITY);
      }
      take(p, 1);
    }
    const float top = block_reduce<W>(m, red, Max());
    const float mc = top == -INFINITY ? 0.f : top * c;
    s *= exp2_hw(m == -INFINITY ? -INFINITY : m * c - mc);
    s = block_reduce<W>(s, red, Add());
    const float lse = kLn2 * (mc + log2f(s));

    float top_u, log_sum, loss = 0.f;
    if (load_teacher<B>(t, red, a.ids, a.u, r, a.ldi, a.ldu, a.top, n, a.id_bytes, a.udtype, a.inv_tau, top_u, log_sum)) {
      for (int k = threadIdx.x; k < a.top; k += B)
        if (t.id[k] >= 0) {
          const float logp = t.p[k] - top_u - log_sum, p = exp2_hw(logp * kLog2e);
          // p that rounds to 0 has no term, whatever the student's logit
          if (p != 0.f) loss = fmaf(p, logp - fmaf(to_f32(z[t.id[k]]), a.inv_tau, -lse), loss);
        }
      loss = block_reduce<W>(loss, red, Add()) * a.tau * a.tau;
    }
    if (threadIdx.x == 0) {
      if (a.loss) a.loss[r] = loss;
      if (a.lse) a.lse[r] = lse;
    }
    __syncthreads();   // the list is written again
  }
}

// ---------------------------------------------------------------------------
// Backward: a block writes a part of a row, the softmax first and then, over
// it, the elements that the teacher lists.  dz may be z: a block reads what it
// needs of its part before it writes there, and no other block reads it.
template <class T, int B>
__global__ __launch_bounds__(B) void k_distill_backward(DistillBackward a, int parts) {
  constexpr int V = kVec<T>, W = B / 64, U = 4;
  __shared__ Teacher t;
  __shared__ float listed[kMaxTop];
  __shared__ float red[W];
  const int64_t n = a.cols;
  const int64_t width = ((n + parts - 1) / parts + V - 1) / V * V;
  const int64_t units = a.rows * parts;
  for (int64_t unit = blockIdx.x; unit < units; unit += gridDim.x) {
    const int64_t r = unit / parts, first = (unit - r * parts) * width, last = std::min<int64_t>(n, first + width);
    const T* z = static_cast<const T*>(a.z) + r * a.ldz;
    T* dz = static_cast<T*>(a.dz) + r * a.lddz;
    float top_u, log_sum;
    const bool some = load_teacher<B>(t, red, a.ids, a.u, r, a.ldi, a.ldu, a.top, n, a.id_bytes, a.udtype, a.inv_tau, top_u, log_sum);
    if (!some) {
      for (int64_t j = first + threadIdx.x * V; j < last; j += int64_t(B) * V) store_pack<T, V>(dz, j, last, Pack<T, V>{});
      __syncthreads();
      continue;
    }
    const float lse = a.lse[r], scale = a.dloss[r * a.lddl] * a.tau;
    auto grad = [&](float x) { return exp2_hw(fmaf(x, a.inv_tau, -lse) * kLog2e); };
    // the entries in this part: the first of those with one id takes them all
    unsigned mine = 0;   // this thread's such entries
    for (int k = threadIdx.x; k < a.top; k += B) {
      const int id = t.id[k];
      if (id < first || id >= last) continue;
      float p = 0.f;
      int lead = k;
      for (int j = 0; j < a.top; ++j)
        if (t.id[j] == id) {
          if (j < lead) lead = j;
          p += exp2_hw((t.p[j] - top_u - log_sum) * kLog2e);
        }
      if (lead != k) continue;
      listed[k] = scale * (grad(to_f32(z[id])) - p);
      mine |= 1u << (k / B);
    }
    __syncthreads();
    int64_t j = first + threadIdx.x * V;
    for (; j + int64_t(U - 1) * B * V + V <= last; j += int64_t(U) * B * V) {
      Pack<T, V> p[U];
#pragma unroll
      for (int k = 0; k < U; ++k) p[k] = *reinterpret_cast<const Pack<T, V>*>(z + j + int64_t(k) * B * V);
#pragma unroll
      for (int k = 0; k < U; ++k) {
#pragma unroll
        for (int i = 0; i < V; ++i) p[k].v[i] = from_f32<T>(scale * grad(to_f32(p[k].v[i])));
        *reinterpret_cast<Pack<T, V>*>(dz + j + int64_t(k) * B * V) = p[k];
      }
    }
    for (; j < last; j += int64_t(B) * V) {
      Pack<T, V> p = load_pack<T, V>(z, j, last);
#pragma unroll
      for (int i = 0; i < V; ++i) p.v[i] = from_f32<T>(scale * grad(to_f32(p.v[i])));
      store_pack<T, V>(dz, j, last, p);
    }
    __syncthreads();
    for (int k = threadIdx.x; k < a.top; k += B)
      if (mine >> (k / B) & 1) dz[t.id[k]] = from_f32<T>(listed[k]);
    __syncthreads();   // the list is written again
  }
}

template <class F>
hipError_t with_type(int32_t dtype, F&& f) {
  if (dtype == kF32) return f(float());
  if (dtype == kBF16) return f(bf16());
  return f(f16());
}

}  // namespace

hipError_t launch_distill_forward(const DistillForward& a, hipStream_t s) {
  if (a.rows == 0) return hipSuccess;
  return with_type(a.dtype, [&](auto t) {
    using T = decltype(t);
    const dim3 grid(unsigned(std::min<int64_t>(a.rows, 1 << 20)));
    if (a.cols >= 8192) k_distill_forward<T, 512><<<grid, dim3(512), 0, s>>>(a);
    else k_distill_forward<T, 128><<<grid, dim3(128), 0, s>>>(a);
    return hipGetLastError();
  });
}

hipError_t launch_distill_backward(const DistillBackward& a, hipStream_t s) {
  if (a.rows == 0) return hipSuccess;
  return with_type(a.dtype, [&](auto t) {
    using T = decltype(t);
    // few rows: several blocks a row
    const int64_t parts = std::max<int64_t>(1, std::min<int64_t>(512 / a.rows, (a.cols + 8191) / 8192));
    const dim3 grid(unsigned(std::min<int64_t>(a.rows * parts, 1 << 20)));
    k_distill_backward<T, 256><<<grid, dim3(256), 0, s>>>(a, int(parts));
    return hipGetLastError();
  });
}

}  // namespace lopt
