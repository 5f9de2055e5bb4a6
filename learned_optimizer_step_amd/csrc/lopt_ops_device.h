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

// Waits here for a load into p.  One counter covers a wave's loads and stores,
// so a wait behind branches with stores in them waits for all of those too;
// a batch of loads settled together is waited for once.
template <class T, int N>
__device__ __forceinline__ void settle(Pack<T, N>& p) {
  struct Words {
    uint32_t w[sizeof(T) * N / 4];
  };
  Words u = __builtin_bit_cast(Words, p);
#pragma unroll
  for (int i = 0; i < int(sizeof(T) * N / 4); ++i) asm volatile("" : "+v"(u.w[i]));
  p = __builtin_bit_cast(Pack<T, N>, u);
}

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

// An 8- or 16-byte vector that is read or written once: with the non-temporal hint it
// takes no room in the caches from what is read again.
template <int BYTES>
struct StreamWords {
  typedef uint32_t type __attribute__((ext_vector_type(BYTES / 4), aligned(2)));
};
template <class T, int N>
__device__ __forceinline__ Pack<T, N> load_stream(const Pack<T, N>* p) {
  typedef typename StreamWords<sizeof(T) * N>::type Words;
  return __builtin_bit_cast(Pack<T, N>, __builtin_nontemporal_load(reinterpret_cast<const Words*>(p)));
}
template <class T, int N>
__device__ __forceinline__ void store_stream(Pack<T, N>* p, const Pack<T, N>& x) {
  typedef typename StreamWords<sizeof(T) * N>::type Words;
  __builtin_nontemporal_store(__builtin_bit_cast(Words, x), reinterpret_cast<Words*>(p));
}

// A row of n elements cut into vectors of V, one at column c = V, 2 V, ... for
// each thread, so that loads need no branch (branches around loads make the
// compiler wait for each one):
//   MODE kWhole  n is a multiple of V
//   MODE kTail   the last vector moves back to end with the row; elements that
//                it shares with the one before it are not its own
//   MODE kTiny   n < V: element by element
// Threads behind the row's end load its last vector and own nothing.
enum : int { kWhole = 0, kTail = 1, kTiny = 2 };
inline int row_mode(int64_t n, int v) { return n < v ? kTiny : n % v ? kTail : kWhole; }

template <class T, int V, int MODE>
struct RowVec {
  int c, at, n;   // the thread's columns begin at c; its vector is read at `at`

  __device__ __forceinline__ RowVec(int c_, int n_) : c(c_), at(MODE == kTiny ? c_ : c_ < n_ - V ? c_ : n_ - V), n(n_) {}
  // element i of the vector is the thread's own (column at + i)
  __device__ __forceinline__ bool own(int i) const {
    if (MODE == kWhole) return c < n;
    if (MODE == kTail) return c < n && at + i >= c;
    return c + i < n;
  }
  template <class U = T>
  __device__ __forceinline__ Pack<U, V> load(const U* row) const {
    Pack<U, V> p;
    if constexpr (MODE == kTiny) {
#pragma unroll
      for (int i = 0; i < V; ++i) p.v[i] = c + i < n ? row[c + i] : U(0.f);
    } else {
      p = *reinterpret_cast<const Pack<U, V>*>(row + at);
    }
    return p;
  }
  template <class U = T>
  __device__ __forceinline__ Pack<U, V> load_once(const U* row) const {
    if constexpr (MODE == kTiny) return load(row);
    else return load_stream(reinterpret_cast<const Pack<U, V>*>(row + at));
  }
  // ONCE: it is not read again soon (known at compile time: of two stores that
  // differ by the hint alone the compiler makes one without it)
  template <bool ONCE = false, class U = T>
  __device__ __forceinline__ void store(U* row, const Pack<U, V>& p) const {
    if (MODE != kTiny && c + V <= n) {
      if constexpr (ONCE) store_stream(reinterpret_cast<Pack<U, V>*>(row + at), p);
      else *reinterpret_cast<Pack<U, V>*>(row + at) = p;
    } else if (MODE != kWhole) {
#pragma unroll
      for (int i = 0; i < V; ++i)
        if (own(i)) row[at + i] = p.v[i];
    }
  }
};

// The same for a slab of columns of a long row, [slab0, slab0 + 64 V): the
// row's address and slab0 are wave-uniform, so an access is a scalar base and
// a 32-bit offset.
template <int V, int MODE>
struct SlabVec {
  int64_t base;   // elements from the row's first to where offsets count from
  int c, at, n;   // as RowVec, from the slab's first column
  uint32_t off;

  __device__ __forceinline__ SlabVec(int64_t slab0, int c_, int64_t cols) : c(c_), n(cols - slab0 < 65536 ? int(cols - slab0) : 65536) {
    at = MODE == kTail && c > n - V ? n - V : c;   // n < V in a row's last slab: into the slab before
    const int back = MODE == kTail && slab0 > 0 ? V : 0;
    base = slab0 - back;
    off = MODE == kTiny || c < n || MODE == kTail ? uint32_t(at + back) : 0;
  }
  __device__ __forceinline__ bool own(int i) const {
    if (MODE == kWhole) return c < n;
    return c + i < n + (c - at) && at + i >= c && c < n;
  }
  template <class U>
  __device__ __forceinline__ Pack<U, V> load(const U* row) const {
    Pack<U, V> p;
    if constexpr (MODE == kTiny) {
#pragma unroll
      for (int i = 0; i < V; ++i) p.v[i] = c + i < n ? row[c + i] : U(0.f);
    } else {
      p = *reinterpret_cast<const Pack<U, V>*>(row + base + off);
    }
    return p;
  }
  template <class U>
  __device__ __forceinline__ Pack<U, V> load_once(const U* row) const {
    if constexpr (MODE == kTiny) return load(row);
    else return load_stream(reinterpret_cast<const Pack<U, V>*>(row + base + off));
  }
  template <class U>
  __device__ __forceinline__ void store(U* row, const Pack<U, V>& p) const {
    if (MODE != kTiny && c + V <= n) {
      *reinterpret_cast<Pack<U, V>*>(row + base + off) = p;
    } else if (MODE != kWhole) {
#pragma unroll
      for (int i = 0; i < V; ++i)
        if (own(i)) row[base + off + i] = p.v[i];
    }
  }
};

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

// The same sum in 64 bits; the exchanges move the two halves of a value.
struct Halves {
  float lo, hi;
};
template <int W>
__device__ __forceinline__ double lanes_sum(double x) {
  const auto join = [](float lo, float hi) { return __builtin_bit_cast(double, Halves{lo, hi}); };
  Halves h = __builtin_bit_cast(Halves, x);
  x += join(dpp<0xB1>(h.lo), dpp<0xB1>(h.hi));
  h = __builtin_bit_cast(Halves, x);
  x += join(dpp<0x4E>(h.lo), dpp<0x4E>(h.hi));
  h = __builtin_bit_cast(Halves, x);
  x += join(dpp<0x141>(h.lo), dpp<0x141>(h.hi));
  if constexpr (W > 8) {
    h = __builtin_bit_cast(Halves, x);
    x += join(dpp<0x140>(h.lo), dpp<0x140>(h.hi));
    h = __builtin_bit_cast(Halves, x);
    Two lo = swap16(h.lo), hi = swap16(h.hi);
    x = join(lo.a, hi.a) + join(lo.b, hi.b);
    h = __builtin_bit_cast(Halves, x);
    lo = swap32(h.lo), hi = swap32(h.hi);
    x = join(lo.a, hi.a) + join(lo.b, hi.b);
  }
  return x;
}

// Sum over the lanes of the same place in their group of 8 (the groups of a wave added up).
__device__ __forceinline__ float groups_sum(float x) {
  x += dpp<0x128>(x);   // row_ror 8: the other group of the 16 lanes
  const Two a = swap16(x);
  x = a.a + a.b;
  const Two b = swap32(x);
  return b.a + b.b;
}

}  // namespace lopt
