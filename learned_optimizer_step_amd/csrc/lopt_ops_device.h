// Device helpers shared by the gradient-producing operators (norms, embedding,
// distillation loss): element types, rows read in 16-byte vectors from any
// element-aligned address, reductions over a wave and over a block.
#pragma once

#include <hip/hip_runtime.h>

#include <stdint.h>

namespace lopt {

typedef __bf16 bf16;
typedef _Float16 f16;

template <class T>
__device__ __forceinline__ float to_f32(T x) { return float(x); }
// One rounding, to nearest even (v_cvt_pk_bf16_f32 / v_cvt_f16_f32).
template <class T>
__device__ __forceinline__ T from_f32(float x) { return T(x); }

// N elements at an address aligned to one element only: gfx950 reads and
// writes global memory at any alignment, so these are single 16-byte (or
// shorter) accesses.
template <class T, int N>
struct __attribute__((packed, aligned(sizeof(T)))) Pack {
  T v[N];
};

// Elements of a 16-byte access.
template <class T>
constexpr int kVec = 16 / int(sizeof(T));

// Elements [c, c + N) of a row of n elements; 0 behind its end.
template <class T, int N>
__device__ __forceinline__ Pack<T, N> load_pack(const T* row, int64_t c, int64_t n) {
  Pack<T, N> p;
  if (c + N <= n) {
    p = *reinterpret_cast<const Pack<T, N>*>(row + c);
  } else {
#pragma unroll
    for (int i = 0; i < N; ++i) p.v[i] = c + i < n ? row[c + i] : T(0.f);
  }
  return p;
}

template <class T, int N>
__device__ __forceinline__ void store_pack(T* row, int64_t c, int64_t n, const Pack<T, N>& p) {
  if (c + N <= n) {
    *reinterpret_cast<Pack<T, N>*>(row + c) = p;
  } else {
#pragma unroll
    for (int i = 0; i < N; ++i)
      if (c + i < n) row[c + i] = p.v[i];
  }
}

// An element of a vector whose type is known at run time (0 fp32, 1 bf16, 2 fp16).
__device__ __forceinline__ float load_any(const void* p, int dtype, int64_t i) {
  if (dtype == 0) return static_cast<const float*>(p)[i];
  if (dtype == 1) return float(static_cast<const bf16*>(p)[i]);
  return float(static_cast<const f16*>(p)[i]);
}
__device__ __forceinline__ void store_any(void* p, int dtype, int64_t i, float x) {
  if (dtype == 0) static_cast<float*>(p)[i] = x;
  else if (dtype == 1) static_cast<bf16*>(p)[i] = bf16(x);
  else static_cast<f16*>(p)[i] = f16(x);
}

template <int CTRL>
__device__ __forceinline__ float dpp(float x) {
  return __builtin_bit_cast(float, __builtin_amdgcn_update_dpp(0, __builtin_bit_cast(int, x), CTRL, 0xf, 0xf, true));
}

// x of the wave's lanes with bit 4 (16) or bit 5 (32) of the lane number
// cleared, and with it set, in every lane: the row swaps of gfx950.
struct Two {
  float a, b;
};
__device__ __forceinline__ Two swap16(float x) {
  const auto r = __builtin_amdgcn_permlane16_swap(__float_as_uint(x), __float_as_uint(x), false, false);
  return {__uint_as_float(r[0]), __uint_as_float(r[1])};
}
__device__ __forceinline__ Two swap32(float x) {
  const auto r = __builtin_amdgcn_permlane32_swap(__float_as_uint(x), __float_as_uint(x), false, false);
  return {__uint_as_float(r[0]), __uint_as_float(r[1])};
}

// Butterflies over aligned groups of W lanes (W = 8 or 64); every lane gets
// the result, the same bits on all of them.  Lane exchanges are DPP moves
// within 16 lanes and the row swaps of gfx950 beyond, no LDS traffic.
struct Add {
  __device__ __forceinline__ float operator()(float a, float b) const { return a + b; }
};
struct Max {
  __device__ __forceinline__ float operator()(float a, float b) const { return fmaxf(a, b); }
};
template <int W, class Op>
__device__ __forceinline__ float lanes_reduce(float x, Op op) {
  x = op(x, dpp<0xB1>(x));    // quad_perm 1,0,3,2
  x = op(x, dpp<0x4E>(x));    // quad_perm 2,3,0,1
  x = op(x, dpp<0x141>(x));   // mirror within 8 lanes
  if constexpr (W > 8) {
    x = op(x, dpp<0x140>(x));   // mirror within 16 lanes
    const Two a = swap16(x);
    x = op(a.a, a.b);
    const Two b = swap32(x);
    x = op(b.a, b.b);
  }
  return x;
}
template <int W>
__device__ __forceinline__ float lanes_sum(float x) { return lanes_reduce<W>(x, Add()); }

// Sum over the lanes of the same place in their group of 8 (the groups of a wave added up).
__device__ __forceinline__ float groups_sum(float x) {
  x += dpp<0x128>(x);   // row_ror 8: the other group of the 16 lanes
  const Two a = swap16(x);
  x = a.a + a.b;
  const Two b = swap32(x);
  return b.a + b.b;
}

}  // namespace lopt
