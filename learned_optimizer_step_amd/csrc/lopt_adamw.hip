// AdamW over a list of tensors, moments in 32 bits or in 8.  With t = 1, 2, ...
//   m <- b1 m + (1 - b1) g,  v <- b2 v + (1 - b2) g^2
//   p <- p (1 - lr wd) - lr / (1 - b1^t) m / (sqrt(v / (1 - b2^t)) + eps)
// Bound by HBM: p, m and v are read and written once, g is read once (fp32: 28
// bytes an element with 32-bit moments, 16.1 with 8-bit ones).  ViT-B/16 with 32-bit moments:
// 408 us, 5.9 TB/s; GPT-2 355M with 8-bit ones 1028 (median of its kernels' trace; at best 958), 5.6; 92.6M bf16 elements
// with 8-bit ones 294 (283), 3.2: the codes' arithmetic and the ends of 13 launches.
//
// The list travels as a kernel argument, kMaxAdamw tensors a launch: nothing is
// uploaded, so gradients may lie elsewhere at every step, and a captured launch
// holds its own list.  A wave takes chunks of kChunk elements of one tensor and
// finds the tensor in the launch's running sum of chunks; tensors of any sizes
// fill the same grid.
//
// The step counter is on the device, so that a captured step counts as it is
// replayed: every wave reads it first.  A short last launch advances it itself, by
// its last block to finish (a ticket: some 40 ns a block, one after the other;
// 2048 of them took 60 us of 547); behind a longer one a launch of one thread does.
//
// 8-bit moments: a block of 256 numbers shares an exponent e, which puts its
// largest in the highest binade of the codes.  m has a sign, 4 bits of exponent
// and 3 of mantissa (2^14 from the largest normal code to the least, and 3 bits
// below), v no sign and 5 bits of exponent (2^30).  Codes are rounded up or down
// at random, in proportion to what is left: v changes by a thousandth a step
// with b2 = 0.999, which rounding to the nearest of 3 bits would lose every
// time, and the codes could neither rise nor decay.  A number is rounded by
// adding 16 random bits below the code's last bit: codes follow from the fp32
// moment and these bits alone.  The 32 random bits of an element are a hash of
// the seed, t, the tensor's place in the list and the element's number.  A v
// that is not 0 does not round to 0, as its root divides.
#include <hip/hip_runtime.h>

#include <cfloat>

#include <algorithm>
#include <cmath>
#include <type_traits>

#include "lopt_ops.h"
#include "lopt_ops_device.h"

namespace lopt {
namespace {

// A wave's chunk is two of the moments' blocks, and a list gets a wave for every
// chunk (ViT-B/16 fp32: 408 us, 439 with 2048 blocks of four-block chunks in a
// loop; GPT-2 355M with 8-bit moments and their decoding 1447, 1540).
constexpr int kPerLane = 4, kBlocks = 2;
constexpr unsigned kMostTickets = 64;   // blocks
constexpr unsigned kMostBlocks = 1u << 24;   // of 256 threads: a grid has room for 2^32 threads
constexpr int kChunk = 64 * kPerLane * kBlocks;
static_assert(kMomentBlock == 64 * kPerLane, "a wave holds a block of moments");
static_assert(sizeof(AdamwLaunch) <= 4096, "kernel arguments");

// a b + c d as two products and a sum, each rounded: what the moments' codes
// are rounded from can be computed elsewhere to the last bit.
__device__ __forceinline__ float weighted(float a, float b, float c, float d) {
#pragma clang fp contract(off)
  return a * b + c * d;
}
__device__ __forceinline__ float square(float x) {
#pragma clang fp contract(off)
  return x * x;
}

// A bijection of 32-bit numbers that scatters neighbours (the finalizer of MurmurHash3).
__device__ __forceinline__ uint32_t mix(uint32_t x) {
  x = (x ^ (x >> 16)) * 0x85EBCA6Bu;
  x = (x ^ (x >> 13)) * 0xC2B2AE35u;
  return x ^ (x >> 16);
}

struct Highest {   // of non-negative floats by their bits, a NaN above all
  __device__ __forceinline__ float operator()(float a, float b) const { return __uint_as_float(max(__float_as_uint(a), __float_as_uint(b))); }
};

// Codes of FIELDS exponents over 3 bits of mantissa, as the highest bits of a
// float: scaled by 2^kScale and the block's exponent, a code's exponent is the
// float's own field, and numbers below the least exponent are denormal floats
// as they are among the codes.
template <int FIELDS>
struct Codes {
  static constexpr int kScale = 128 - FIELDS;
  // Exponent of a block whose largest number is `top`: the next one where top could round up out of the codes.
  static __device__ __forceinline__ int exponent(float top) {
    const int e = int((__float_as_uint(top) + 0x100000u) >> 23) - 127;
    return min(max(e, -100), 127);
  }
  // x >= 0 scaled: its code from bit 20 on, and what is left of it below.  Numbers below the least exponent come rounded to
  // 2^-20 of a code's step; `down` makes that the one below, so that a sum with random bits goes as high as x's own does.
  static __device__ __forceinline__ uint32_t scaled(float x, int e) { return __float_as_uint(__builtin_ldexpf(x, -e - kScale)); }
  static __device__ __forceinline__ uint32_t down(uint32_t bits, float x, int e) { return bits - (__builtin_ldexpf(__uint_as_float(bits), e + kScale) > x); }
  // bits: the code in its place, from bit 20 on
  static __device__ __forceinline__ float decode(uint32_t bits, int e) { return __builtin_ldexpf(__uint_as_float(bits), e + kScale); }
};
typedef Codes<16> CodesM;
typedef Codes<32> CodesV;
constexpr uint32_t kLeastNormal = 0x800000;   // float's bits
constexpr uint32_t kNotANumber = 255;   // of a block's exponent: a NaN or an infinity is in it

// Byte k of x, its low 7 or 8 bits, from bit 20 on.
template <int K, uint32_t MASK>
__device__ __forceinline__ uint32_t from_byte(uint32_t x) {
  return (K < 2 ? x << (20 - 8 * K) : K == 2 ? x << 4 : x >> 4) & MASK << 20;
}

struct Factors {
  float size;   // 1 / (1 - b1^t)
  float root;   // (1 - b2^t)^(-1/2)
  uint32_t key;
};

// 4 elements of a lane from its place in a tensor of n elements; 0 behind the end.
template <class T, bool FULL, bool ONCE>
__device__ __forceinline__ void load4(const T* base, int64_t i, int64_t n, float (&x)[4]) {
  Pack<T, 4> p;
  if constexpr (FULL && ONCE) p = load_stream(reinterpret_cast<const Pack<T, 4>*>(base + i));
  else if constexpr (FULL) p = *reinterpret_cast<const Pack<T, 4>*>(base + i);
  else p = load_pack<T, 4>(base, i, n);
#pragma unroll
  for (int k = 0; k < 4; ++k) x[k] = to_f32(p.v[k]);
}
template <class T, bool FULL, bool ONCE>
__device__ __forceinline__ void store4(T* base, int64_t i, int64_t n, const float (&x)[4]) {
  Pack<T, 4> p;
#pragma unroll
  for (int k = 0; k < 4; ++k) p.v[k] = from_f32<T>(x[k]);
  if constexpr (FULL && ONCE) store_stream(reinterpret_cast<Pack<T, 4>*>(base + i), p);
  else if constexpr (FULL) *reinterpret_cast<Pack<T, 4>*>(base + i) = p;
  else store_pack<T, 4>(base, i, n, p);
}

// Block `at` (of 256 elements) of a tensor's moments.
template <int BITS>
struct Moments;

template <>
struct Moments<32> {
  static constexpr int64_t kBytes = 2 * kMomentBlock * 4;
  float m[4], v[4];
  template <bool ONCE>
  __device__ __forceinline__ void load(const unsigned char* s, int lane) {
    const float* f = reinterpret_cast<const float*>(s);
    load4<float, true, ONCE>(f, lane * 4, 0, m);
    load4<float, true, ONCE>(f + kMomentBlock, lane * 4, 0, v);
  }
  __device__ __forceinline__ void open() {}
  template <bool ONCE>
  __device__ __forceinline__ void store(unsigned char* s, int lane, uint32_t, int64_t) const {
    float* f = reinterpret_cast<float*>(s);
    store4<float, true, ONCE>(f, lane * 4, 0, m);
    store4<float, true, ONCE>(f + kMomentBlock, lane * 4, 0, v);
  }
};

template <>
struct Moments<8> {
  static constexpr int64_t kBytes = 2 * kMomentBlock + 16;
  uint32_t cm, cv, e;
  float m[4], v[4];
  template <bool ONCE>
  __device__ __forceinline__ void load(const unsigned char* s, int lane) {
    cm = reinterpret_cast<const uint32_t*>(s)[lane];
    cv = reinterpret_cast<const uint32_t*>(s + kMomentBlock)[lane];
    e = *reinterpret_cast<const uint32_t*>(s + 2 * kMomentBlock);
  }
  __device__ __forceinline__ void open() {
    const uint32_t both = __builtin_amdgcn_readfirstlane(e), bm = both & 255, bv = both >> 8 & 255;
    open_one<0>(int(bm) - 100, int(bv) - 100);
    open_one<1>(int(bm) - 100, int(bv) - 100);
    open_one<2>(int(bm) - 100, int(bv) - 100);
    open_one<3>(int(bm) - 100, int(bv) - 100);
    if (bm == kNotANumber || bv == kNotANumber) {
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        if (bm == kNotANumber) m[k] = NAN;
        if (bv == kNotANumber) v[k] = NAN;
      }
    }
  }
  template <int K>
  __device__ __forceinline__ void open_one(int em, int ev) {
    const float x = CodesM::decode(from_byte<K, 127>(cm), em);
    m[K] = __uint_as_float(__float_as_uint(x) | (cm << (24 - 8 * K) & 0x80000000u));
    v[K] = CodesV::decode(from_byte<K, 255>(cv), ev);
  }
  template <bool ONCE>
  __device__ __forceinline__ void store(unsigned char* s, int lane, uint32_t key, int64_t i) const {
    float tm = 0.f, tv = 0.f;
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      tm = Highest()(tm, fabsf(m[k]));
      tv = Highest()(tv, fabsf(v[k]));
    }
    tm = lanes_reduce<64>(tm, Highest());
    tv = lanes_reduce<64>(tv, Highest());
    const bool bm = !(tm < INFINITY), bv = !(tv < INFINITY);
    const int em = bm ? 0 : CodesM::exponent(tm), ev = bv ? 0 : CodesV::exponent(tv);
    // 0x9E3779B9 times the upper half: the same for the block
    const uint32_t base = key + uint32_t(i) + 0x9E3779B9u * uint32_t(uint64_t(i) >> 32);
    uint32_t bits_m[4], bits_v[4], least = ~0u;
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      bits_m[k] = CodesM::scaled(fabsf(m[k]), em);
      bits_v[k] = CodesV::scaled(v[k], ev);
      least = min(least, min(bits_m[k], bits_v[k]));
    }
    if (least < kLeastNormal) {
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        bits_m[k] = CodesM::down(bits_m[k], fabsf(m[k]), em);
        bits_v[k] = CodesV::down(bits_v[k], v[k], ev);
      }
    }
    uint32_t pm = 0, pv = 0, signs = 0;
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      const uint32_t r = mix(base + k);   // 16 bits under a code's last one for each moment
      pm |= min((bits_m[k] + ((r & 0xFFFF) << 4)) >> 20, 127u) << 8 * k;
      signs |= (__float_as_uint(m[k]) >> 24 & 128) << 8 * k;
      // a v that is not 0 has a code that is not
      pv |= min(max((bits_v[k] + (r >> 16 << 4)) >> 20, min(__float_as_uint(v[k]), 1u)), 255u) << 8 * k;
    }
    pm |= signs & (pm + 0x7F7F7F7Fu);   // no sign without a code
    reinterpret_cast<uint32_t*>(s)[lane] = bm ? 0u : pm;
    reinterpret_cast<uint32_t*>(s + kMomentBlock)[lane] = bv ? 0u : pv;
    if (lane == 0)
      *reinterpret_cast<uint32_t*>(s + 2 * kMomentBlock) = (bm ? kNotANumber : uint32_t(em + 100)) | (bv ? kNotANumber : uint32_t(ev + 100)) << 8;
  }
};

template <class P, class G, int BITS, bool FULL, bool ONCE>
__device__ __forceinline__ void chunk_step(const AdamwLaunch& a, const AdamwEntry& t, int64_t start, const Factors& f, uint32_t key, int lane) {
  P* p = static_cast<P*>(t.p);
  const G* g = static_cast<const G*>(t.g);
  unsigned char* s = static_cast<unsigned char*>(t.s) + start / kMomentBlock * Moments<BITS>::kBytes;
  const float size = t.lr * f.size;
  float xp[kBlocks][4], xg[kBlocks][4];
  Moments<BITS> mo[kBlocks];
  const int64_t i0 = start + lane * 4;
#pragma unroll
  for (int b = 0; b < kBlocks; ++b)
    if (FULL || start + b * kMomentBlock < t.n) {
      load4<P, FULL, ONCE>(p, i0 + b * kMomentBlock, t.n, xp[b]);
      load4<G, FULL, ONCE>(g, i0 + b * kMomentBlock, t.n, xg[b]);
      mo[b].template load<ONCE>(s + b * Moments<BITS>::kBytes, lane);
    }
#pragma unroll
  for (int b = 0; b < kBlocks; ++b)
    if (FULL || start + b * kMomentBlock < t.n) {
      mo[b].open();
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        float &m = mo[b].m[k], &v = mo[b].v[k];
        m = weighted(m, a.b1, xg[b][k], a.c1);
        v = weighted(v, a.b2, square(xg[b][k]), a.c2);
        // root and quotient of the hardware, one step off each; a v below the least normal float counts as that
        const float d = __builtin_amdgcn_sqrtf(__builtin_elementwise_maximum(v, FLT_MIN)) * f.root + a.eps;
        xp[b][k] = xp[b][k] * t.decay - size * m * __builtin_amdgcn_rcpf(d);
      }
      store4<P, FULL, ONCE>(p, i0 + b * kMomentBlock, t.n, xp[b]);
      mo[b].template store<ONCE>(s + b * Moments<BITS>::kBytes, lane, key, i0 + b * kMomentBlock);
    }
}

template <class P, class G, int BITS, bool ONCE>
__global__ __launch_bounds__(256) void k_adamw(AdamwLaunch a) {
  const int lane = threadIdx.x & 63;
  const int64_t t = int64_t(__hip_atomic_load(a.step, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT)) + 1;
  Factors f;
  // 1 - b^t = -expm1(t log b), in 64 bits: b near 1 leaves little of it
  f.size = float(1.0 / -expm1(double(t) * a.log_b1));
  f.root = float(1.0 / sqrt(-expm1(double(t) * a.log_b2)));
  f.key = mix(mix(uint32_t(t)) ^ a.seed);
  const uint32_t wave = blockIdx.x * 4 + (threadIdx.x >> 6), waves = gridDim.x * 4;
  for (uint32_t c = __builtin_amdgcn_readfirstlane(wave); c < a.first[a.count]; c += waves) {
    int lo = 0, hi = a.count;   // the tensor with first[lo] <= c < first[lo + 1]
    while (hi - lo > 1) {
      const int mid = (lo + hi) >> 1;
      if (a.first[mid] <= c) lo = mid;
      else hi = mid;
    }
    const AdamwEntry& e = a.e[lo];
    const int64_t start = int64_t(c - a.first[lo]) * kChunk;
    const uint32_t key = mix(f.key + a.place[lo]);
    if (start + kChunk <= e.n) chunk_step<P, G, BITS, true, ONCE>(a, e, start, f, key, lane);
    else chunk_step<P, G, BITS, false, ONCE>(a, e, start, f, key, lane);
  }
  if (a.advance) {
    __syncthreads();   // the block's waves have read the counter
    if (threadIdx.x == 0) {
      unsigned long long* step = a.step;
      const unsigned long long ticket = __hip_atomic_fetch_add(step + 1, 1ull, __ATOMIC_ACQ_REL, __HIP_MEMORY_SCOPE_AGENT);
      if (ticket == gridDim.x - 1) {
        __hip_atomic_store(step + 1, 0ull, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
        __hip_atomic_store(step, (unsigned long long)t, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
      }
    }
  }
}

__global__ void k_adamw_advance(unsigned long long* step) { *step += 1; }

template <class T, int BITS, bool ONCE>
__global__ __launch_bounds__(256) void k_adamw_moments(const unsigned char* s, int64_t n, T* m, T* v) {
  const int lane = threadIdx.x & 63;
  const int64_t blocks = (n + kMomentBlock - 1) / kMomentBlock;
  for (int64_t b = int64_t(blockIdx.x) * 4 + (threadIdx.x >> 6); b < blocks; b += int64_t(gridDim.x) * 4) {
    Moments<BITS> mo;
    mo.template load<ONCE>(s + b * Moments<BITS>::kBytes, lane);
    mo.open();
    const int64_t at = b * kMomentBlock + lane * 4;
    if ((b + 1) * kMomentBlock <= n) {
      if (m) store4<T, true, ONCE>(m, at, n, mo.m);
      if (v) store4<T, true, ONCE>(v, at, n, mo.v);
    } else {
      if (m) store4<T, false, false>(m, at, n, mo.m);
      if (v) store4<T, false, false>(v, at, n, mo.v);
    }
  }
}

template <class F>
hipError_t with_type(int32_t dtype, F&& f) {
  if (dtype == kF32) return f(float());
  if (dtype == kBF16) return f(bf16());
  return f(f16());
}

}  // namespace

int64_t adamw_chunks(int64_t n) { return (n + kChunk - 1) / kChunk; }

hipError_t launch_adamw(const AdamwLaunch& args, int32_t pdtype, int32_t gdtype, int32_t bits, bool once, hipStream_t s) {
  AdamwLaunch a = args;
  const int64_t need = (int64_t(a.first[a.count]) + 3) / 4;
  const dim3 grid(unsigned(std::max<int64_t>(1, std::min<int64_t>(need, kMostBlocks - 1))));
  const bool behind = a.advance && grid.x > kMostTickets;
  if (behind) a.advance = 0;
  const hipError_t e = with_type(pdtype, [&](auto p) {
    return with_type(gdtype, [&](auto g) {
      using P = decltype(p);
      using G = decltype(g);
      if (bits == 32) {
        if (once) k_adamw<P, G, 32, true><<<grid, dim3(256), 0, s>>>(a);
        else k_adamw<P, G, 32, false><<<grid, dim3(256), 0, s>>>(a);
      } else {
        if (once) k_adamw<P, G, 8, true><<<grid, dim3(256), 0, s>>>(a);
        else k_adamw<P, G, 8, false><<<grid, dim3(256), 0, s>>>(a);
      }
      return hipGetLastError();
    });
  });
  if (e != hipSuccess || !behind) return e;
  k_adamw_advance<<<dim3(1), dim3(1), 0, s>>>(a.step);
  return hipGetLastError();
}

hipError_t launch_adamw_moments(const void* state, int64_t n, int32_t bits, int32_t dtype, void* m, void* v, hipStream_t s) {
  const int64_t blocks = (n + kMomentBlock - 1) / kMomentBlock;
  const dim3 grid(unsigned(std::min<int64_t>((blocks + 3) / 4, kMostBlocks - 1)));
  const bool once = n > 50'000'000;
  return with_type(dtype, [&](auto t) {
    using T = decltype(t);
    const unsigned char* p = static_cast<const unsigned char*>(state);
    const auto run = [&](auto bits) {
      if (once) k_adamw_moments<T, bits(), true><<<grid, dim3(256), 0, s>>>(p, n, static_cast<T*>(m), static_cast<T*>(v));
      else k_adamw_moments<T, bits(), false><<<grid, dim3(256), 0, s>>>(p, n, static_cast<T*>(m), static_cast<T*>(v));
    };
    if (bits == 32) run(std::integral_constant<int, 32>());
    else run(std::integral_constant<int, 8>());
    return hipGetLastError();
  });
}

}  // namespace lopt
