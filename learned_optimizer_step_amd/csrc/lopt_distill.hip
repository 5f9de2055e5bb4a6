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

#include <cfloat>

#include <algorithm>
#include <type_traits>

#include "lopt_ops.h"
#include "lopt_ops_device.h"

namespace lopt {
namespace {

// The memory-side cache holds 256 MB.  The forward pass reads what does not fit
// it with the non-temporal hint and leaves the last rows' logits there; the
// backward pass begins with those, and its writes pass the cache by (4096 x
// 50257 bf16, 412 MB: 68 + 146 us; no hints and the same order in both 117 +
// 153; hints on all reads 67 + 163; kept bytes of 100 to 250 MB within 2 %).
constexpr int64_t kKeptBytes = 200'000'000;
constexpr float kLog2e = 1.44269504088896340736f;
constexpr float kLn2 = 0.693147180559945309417f;
constexpr float kFar = 1 << 20;   // scaled logits beyond this are taken for differences: see k_distill_forward

__device__ __forceinline__ float exp2_hw(float x) { return __builtin_amdgcn_exp2f(x); }

// Entry k of a row's list: its logit, -inf if it is absent, and its id.  The logit is scaled after the list's largest is
// taken off: a product with 1 / tau first can overflow, and costs half a step of the logits' common offset.
struct Entry {
  float u;
  int64_t id;
};
template <class Args>
__device__ __forceinline__ Entry load_entry(const Args& a, int64_t r, int k) {
  Entry e;
  e.id = a.id_bytes == 8 ? static_cast<const int64_t*>(a.ids)[r * a.ldi + k]
                         : int64_t(static_cast<const int32_t*>(a.ids)[r * a.ldi + k]);
  e.u = load_any(a.u, a.udtype, r * a.ldu + k);
  if (e.id < 0 || e.id >= a.cols) e.u = -INFINITY;
  return e;
}

// Elements of a row's part [first, last) before its first 16-byte border, and
// the number of whole vectors behind it.
struct Cut {
  int64_t lead, vecs;
};
template <class T>
__device__ __forceinline__ Cut cut_at_16(const T* z, int64_t n) {
  constexpr int V = kVec<T>;
  const int64_t to_border = int64_t((16 - (reinterpret_cast<uintptr_t>(z) & 15)) & 15) / int64_t(sizeof(T));
  const int64_t lead = to_border < n ? to_border : n;
  return {lead, (n - lead) / V};
}

// ---------------------------------------------------------------------------
// Forward: one block a row.  The list's entries and the logits they name are
// loaded first and stay in registers; the row is read once with a running
// maximum and sum per thread; two exchanges over the block end it (the maxima
// of both sides, then three sums).  With m the row's largest logit, u' the
// list's, e_k = exp((u_k - u') / tau), E their sum and s = sum exp((z - m) / tau):
//   loss / tau^2 = sum_k e_k ((u_k - u') - (z_(i_k) - m)) / tau / E - log E + log s,
// small terms all of them, whatever the logits' common offset is.
template <class T, int B, int NE>
__global__ __launch_bounds__(B) void k_distill_forward(DistillForward a) {
  constexpr int V = kVec<T>, W = B / 64, U = 4;
  __shared__ float maxima[2][W], sums[3][W];
  const int64_t n = a.cols;
  const float c = a.inv_tau * kLog2e;
  const int wave = threadIdx.x >> 6, lane = threadIdx.x & 63;
  for (int64_t r = blockIdx.x; r < a.rows; r += gridDim.x) {
    const T* z = static_cast<const T*>(a.z) + r * a.ldz;
    float u[NE], zk[NE];
    float top_u = -INFINITY;
    bool nan = false;
#pragma unroll
    for (int e = 0; e < NE; ++e) {
      u[e] = -INFINITY;
      zk[e] = 0.f;
      const int k = e * B + int(threadIdx.x);
      if (k < a.top) {
        const Entry t = load_entry(a, r, k);
        u[e] = t.u;
        if (t.u != -INFINITY) zk[e] = to_f32(z[t.id]);
        top_u = fmaxf(top_u, t.u);
        nan |= t.u != t.u;
      }
    }
    if (nan) top_u = NAN;

    // running maximum m of z and sum s of 2^(z c - mc), per thread, with mc the rounded m c: the sum is rescaled by that
    // same number, as half a step of m c (2^-19 at 60) is more than the sum's own roundings.  A thread may see nothing but
    // masks of -1e9 or the type's lowest value, whose m c overflows or has half steps that are exponents of their own: mc
    // is held within kFar, where half a step is 2^-5 or less (any mc is right for the sum, and such terms vanish)
    float m = -INFINITY, s = 0.f, mc = 0.f;
    const auto rise = [&](float top) {
      const float old = mc;
      mc = top == -INFINITY ? 0.f : fminf(fmaxf(top * c, -kFar), kFar);   // all -inf so far: terms are 2^-inf = 0
      asm("" : "+v"(mc));                      // one number for all its uses: no fma takes the product's place
      s = m == -INFINITY ? 0.f * s : s * exp2_hw(old - mc);
      m = top;
    };
    const auto take = [&](auto const&... packs) {
      float top = m;
      ([&] {
#pragma unroll
        for (int i = 0; i < V; ++i) top = fmaxf(top, to_f32(packs.v[i]));
      }(), ...);
      rise(top);
      ([&] {
        float t = 0.f;
#pragma unroll
        for (int i = 0; i < V; ++i) t += exp2_hw(fmaf(to_f32(packs.v[i]), c, -mc));
        s += t;
      }(), ...);
    };
    // single elements up to the first 16-byte border and behind the last one: rows of an odd length begin anywhere, and
    // unaligned vectors take a fifth more time (4096 x 50257 bf16: 112 us for 96)
    const auto [lead, vecs] = cut_at_16(z, n);
    const int64_t tail = lead + vecs * V;
    const Pack<T, V>* zv = reinterpret_cast<const Pack<T, V>*>(z + lead);
    int64_t j = threadIdx.x;
    const auto read = [&](auto const& ld) {
      for (; j + (U - 1) * B < vecs; j += U * B) take(ld(j), ld(j + B), ld(j + 2 * B), ld(j + 3 * B));
      for (; j < vecs; j += B) take(ld(j));
    };
    if ((a.rows - r) * n * int64_t(sizeof(T)) > kKeptBytes) read([&](int64_t i) { return load_stream(zv + i); });
    else read([&](int64_t i) { return zv[i]; });
    if (int64_t(threadIdx.x) < lead + n - tail) {
      const int64_t i = int64_t(threadIdx.x) < lead ? int64_t(threadIdx.x) : tail + threadIdx.x - lead;
      Pack<T, 1> p;
      p.v[0] = z[i];
      const float x = to_f32(p.v[0]);
      rise(fmaxf(m, x));
      s += exp2_hw(fmaf(x, c, -mc));
    }

    const float wave_m = lanes_reduce<64>(m, Max());
    const float wave_u = lanes_reduce<64>(top_u == top_u ? top_u : INFINITY, Max());   // NaN as +inf: gives NaN below
    if (lane == 0) {
      maxima[0][wave] = wave_m;
      maxima[1][wave] = wave_u;
    }
    __syncthreads();
    float mz = maxima[0][0], mu = maxima[1][0];
#pragma unroll
    for (int k = 1; k < W; ++k) {
      mz = fmaxf(mz, maxima[0][k]);
      mu = fmaxf(mu, maxima[1][k]);
    }
    rise(mz);
    const bool far = mz != -INFINITY && !(fabsf(mz * c) <= kFar);
    if (far) {   // the row's largest logit is out there itself: its sum again, of differences
      s = 0.f;
      for (int64_t i = threadIdx.x; i < n; i += B) s += exp2_hw((to_f32(z[i]) - mz) * c);
    }
    float es = 0.f, eu = 0.f;
#pragma unroll
    for (int e = 0; e < NE; ++e)
      if (u[e] != -INFINITY) {
        const float d = u[e] - mu, p = exp2_hw(d * c);
        es += p;
        // p that rounds to 0 has no term, whatever the student's logit
        if (p != 0.f) eu = fmaf(p, (d - (zk[e] - mz)) * a.inv_tau, eu);
      }
    s = lanes_sum<64>(s);
    es = lanes_sum<64>(es);
    eu = lanes_sum<64>(eu);
    if (lane == 0) {
      sums[0][wave] = s;
      sums[1][wave] = es;
      sums[2][wave] = eu;
    }
    __syncthreads();
    if (threadIdx.x == 0) {
      s = sums[0][0], es = sums[1][0], eu = sums[2][0];
#pragma unroll
      for (int k = 1; k < W; ++k) {
        s += sums[0][k];
        es += sums[1][k];
        eu += sums[2][k];
      }
      // from the rounded m c to m c itself; one logarithm of s / es, as that of two is lost in their difference
      const float rest = mz == -INFINITY || far ? 0.f : fmaf(mz, c, -mc);
      if (a.lse) {
        // below the least number that one, as the gradient of -inf would be no number
        const float lse = fmaf(mz, a.inv_tau, kLn2 * (log2f(s) - rest));
        a.lse[r] = far && lse == -INFINITY ? -FLT_MAX : lse;
      }
      if (a.loss) a.loss[r] = mu == -INFINITY ? 0.f : a.tau * (a.tau * fmaf(kLn2, log2f(s / es) - rest, eu / es));   // tau^2 alone can vanish
    }
    // the next row's exchanges write `maxima` after this barrier's reads of it, and `sums` after its own first barrier
  }
}

// ---------------------------------------------------------------------------
// Backward: a block writes a part of a row, the softmax first and then, over
// it, the elements that the teacher lists.  dz may be z: a block reads what it
// needs of its part before it writes there, and no other block reads it.
// An id that is listed more than once is written by its first entry, which
// adds up the p of all in their order.
template <class T, int B, int NE>
__global__ __launch_bounds__(B) void k_distill_backward(DistillBackward a, int parts) {
  constexpr int V = kVec<T>, W = B / 64, U = 4;
  __shared__ int4 ids4[NE * B / 4];   // -1: absent
  __shared__ float prob[NE * B];
  __shared__ float maxima[W], sums[W];
  int* ids = reinterpret_cast<int*>(ids4);
  const int64_t n = a.cols;
  const int64_t width = ((n + parts - 1) / parts + V - 1) / V * V;
  const int64_t units = a.rows * parts;
  const int wave = threadIdx.x >> 6, lane = threadIdx.x & 63;
  for (int64_t turn = blockIdx.x; turn < units; turn += gridDim.x) {
    const int64_t unit = units - 1 - turn;
    const int64_t r = unit / parts, first = std::min<int64_t>(n, (unit - r * parts) * width), last = std::min<int64_t>(n, first + width);
    const T* z = static_cast<const T*>(a.z) + r * a.ldz;
    T* dz = static_cast<T*>(a.dz) + r * a.lddz;
    const float lse = a.lse[r], scale = a.dloss[r * a.lddl] * a.tau;

    float u[NE], mine[NE];   // mine: the element that the entry writes
    float top_u = -INFINITY;
    bool nan = false;
    unsigned writes = 0;     // this thread's entries that write
#pragma unroll
    for (int e = 0; e < NE; ++e) {
      u[e] = -INFINITY;
      mine[e] = 0.f;
      const int k = e * B + int(threadIdx.x);
      if (k < a.top) {
        const Entry t = load_entry(a, r, k);
        u[e] = t.u;
        ids[k] = t.u != -INFINITY ? int(t.id) : -1;
        if (t.u != -INFINITY && t.id >= first && t.id < last) {
          mine[e] = to_f32(z[t.id]);
          writes |= 1u << e;
        }
        top_u = fmaxf(top_u, t.u);
        nan |= t.u != t.u;
      } else if (k < (a.top + 3) / 4 * 4) {
        ids[k] = -1;
      }
    }
    if (nan) top_u = INFINITY;   // gives NaN below
    top_u = lanes_reduce<64>(top_u, Max());
    if (lane == 0) maxima[wave] = top_u;
    __syncthreads();
    top_u = maxima[0];
#pragma unroll
    for (int k = 1; k < W; ++k) top_u = fmaxf(top_u, maxima[k]);
    float sum = 0.f;
#pragma unroll
    for (int e = 0; e < NE; ++e) {
      const int k = e * B + int(threadIdx.x);
      if (k < a.top) {
        const float p = u[e] == -INFINITY ? 0.f : exp2_hw((u[e] - top_u) * (a.inv_tau * kLog2e));
        prob[k] = p;
        sum += p;
      }
    }
    sum = lanes_sum<64>(sum);
    if (lane == 0) sums[wave] = sum;
    __syncthreads();
    sum = sums[0];
#pragma unroll
    for (int k = 1; k < W; ++k) sum += sums[k];

    const bool some = top_u != -INFINITY;
    // a probability is at most 1: half a step of a large lse is an exponent of its own (NaN stays NaN)
    const auto softmax = [&](float x) { return exp2_hw(__builtin_elementwise_minimum(fmaf(x, a.inv_tau, -lse) * kLog2e, 0.f)); };
    const auto grad = [&](float x) { return from_f32<T>(some ? scale * softmax(x) : 0.f); };
#pragma unroll
    for (int e = 0; e < NE; ++e)
      if (writes >> e & 1) {
        const int k = e * B + int(threadIdx.x), id = ids[k];
        int equal = 0;
        for (int q = 0; q < (a.top + 3) / 4; ++q) {
          const int4 o = ids4[q];
          equal += (o.x == id) + (o.y == id) + (o.z == id) + (o.w == id);
        }
        float p = prob[k];
        if (equal > 1) {   // listed more than once
          p = 0.f;
          for (int q = 0; q < a.top; ++q)
            if (ids[q] == id) {
              if (q < k) writes &= ~(1u << e);
              p += prob[q];
            }
        }
        mine[e] = scale * (softmax(mine[e]) - p / sum);
      }
    __syncthreads();   // the listed logits of this part are read: dz may be z

    const auto [lead, vecs] = cut_at_16(z + first, last - first);
    const Pack<T, V>* zv = reinterpret_cast<const Pack<T, V>*>(z + first + lead);
    Pack<T, V>* dv = reinterpret_cast<Pack<T, V>*>(dz + first + lead);
    int64_t j = threadIdx.x;
    for (; j + (U - 1) * B < vecs; j += U * B) {
      Pack<T, V> p[U];
#pragma unroll
      for (int k = 0; k < U; ++k) p[k] = load_stream(zv + j + k * B);
#pragma unroll
      for (int k = 0; k < U; ++k) settle(p[k]);
#pragma unroll
      for (int k = 0; k < U; ++k) {
#pragma unroll
        for (int i = 0; i < V; ++i) p[k].v[i] = grad(to_f32(p[k].v[i]));
        store_stream(dv + j + k * B, p[k]);
      }
    }
    for (; j < vecs; j += B) {
      Pack<T, V> p = zv[j];
#pragma unroll
      for (int i = 0; i < V; ++i) p.v[i] = grad(to_f32(p.v[i]));
      dv[j] = p;
    }
    const int64_t tail = lead + vecs * V;
    if (int64_t(threadIdx.x) < lead + (last - first) - tail) {
      const int64_t i = first + (int64_t(threadIdx.x) < lead ? int64_t(threadIdx.x) : tail + threadIdx.x - lead);
      dz[i] = grad(to_f32(z[i]));
    }
    __syncthreads();   // the softmax is written; the list is written again after this
#pragma unroll
    for (int e = 0; e < NE; ++e)
      if (writes >> e & 1) dz[ids[e * B + int(threadIdx.x)]] = from_f32<T>(mine[e]);
    __syncthreads();
  }
}

template <class F>
hipError_t with_type(int32_t dtype, F&& f) {
  if (dtype == kF32) return f(float());
  if (dtype == kBF16) return f(bf16());
  return f(f16());
}

}  // namespace

// Calls f(threads, entries a thread) for `units` rows or parts of `cols`
// logits and lists of `top`.  Small blocks keep more rows in flight where a
// row is short next to its exchanges (9000 x 3000 bf16, forward + backward:
// 16 + 30 us with 64 or 128 threads, 18 + 46 with 256, 32 + 76 with 512; 6000 x
// 12000: 32 + 63, 29 + 61, 26 + 51, 33 + 60); with too few rows for the chip
// large ones (1 x 50257: 8 us with 128, 4 with 512).
template <class F>
void with_block(int64_t units, int64_t cols, int top, F&& f) {
  const auto entries = [&](auto b) {
    if (top <= b()) f(b, std::integral_constant<int, 1>());
    else f(b, std::integral_constant<int, kMaxTop / b()>());
  };
  int threads = cols < 2048 ? 64 : cols < 8192 ? 128 : cols < 32768 ? 256 : 512;
  while (threads < 512 && units * threads < 256 * 512 && cols > threads * 16) threads *= 2;
  if (threads == 64) entries(std::integral_constant<int, 64>());
  else if (threads == 128) entries(std::integral_constant<int, 128>());
  else if (threads == 256) entries(std::integral_constant<int, 256>());
  else entries(std::integral_constant<int, 512>());
}

hipError_t launch_distill_forward(const DistillForward& a, hipStream_t s) {
  if (a.rows == 0) return hipSuccess;
  return with_type(a.dtype, [&](auto t) {
    using T = decltype(t);
    const dim3 grid(unsigned(std::min<int64_t>(a.rows, 1 << 20)));
    with_block(a.rows, a.cols, a.top, [&](auto b, auto ne) { k_distill_forward<T, b(), ne()><<<grid, dim3(b()), 0, s>>>(a); });
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
    with_block(a.rows * parts, a.cols, a.top, [&](auto b, auto ne) { k_distill_backward<T, b(), ne()><<<grid, dim3(b()), 0, s>>>(a, int(parts)); });
    return hipGetLastError();
  });
}

}  // namespace lopt
