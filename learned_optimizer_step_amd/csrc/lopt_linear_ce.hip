// Cross entropy of a linear layer's logits, which are never kept.  With x (N
// tokens of D), the weight w (V x D), z = x w^T and a target t per token:
//   lse = log sum_v exp(z_v),  loss = lse - z_t
//   G = g (exp(z - lse) - onehot(t)),  dx = G w,  dw = G^T x
// Forward: one product whose tiles end in the running maximum and sum of their
// part of the vocabulary.  Backward: the vocabulary in pieces; of each, the
// product again, its tiles ending in G, which is kept for the piece alone, and
// from it the piece's share of dx and its rows of dw.  Bound by the matrix
// units: 2 N V D operations forward, 6 N V D backward.  bf16: forward 8192 tokens of
// 32000 x 2048 814 to 930 us (1320 to 1155 TFLOP/s, on several cards and in a trace; the library's plain product of that size takes 901),
// both passes 4096 of 50257 x 1024 1680 to 1755 us (1004 to 961 TFLOP/s; the library's
// plain product of that size reaches 866).
#include <hip/hip_runtime.h>

#include <algorithm>
#include <type_traits>

#include "lopt_ops.h"
#include "lopt_ops_device.h"

namespace lopt {
namespace {

constexpr float kLog2e = 1.44269504088896340736f;
constexpr float kLn2 = 0.693147180559945309417f;
__device__ __forceinline__ float exp2_hw(float x) { return __builtin_amdgcn_exp2f(x); }

// ---------------------------------------------------------------------------
// The product C[m][n] = sum_k A[m][k] B[n][k] of a block: WM x WN waves of FM x
// FN matrix instructions of 16 x 16 each.  Under load the card's power sets the
// clock, and these do more for it than those of 32 x 32 (registers of random
// bf16 numbers alone: 2066 TFLOP/s, 1848).  Operands go to LDS in stages of 128
// bytes of k, straight from memory.  An operand may lie with k contiguous
// ("rows") or with m or n contiguous ("columns", a transposed read from LDS):
// no operand is ever transposed in memory.
template <int FM_, int FN_, int WM_, int WN_>
struct Tile {
  static constexpr int FM = FM_, FN = FN_, WM = WM_, WN = WN_;
  static constexpr int M = 16 * FM * WM, N = 16 * FN * WN, WAVES = WM * WN, THREADS = 64 * WAVES;
  static constexpr int STAGE = (M + N) * 128;   // bytes
};
// The large tile reads least from the caches for its operations; where its tiles
// are fewer than the compute units, smaller ones.
typedef Tile<8, 4, 2, 4> Large;    // 256 x 256, one block a compute unit
typedef Tile<4, 4, 2, 2> Middle;   // 128 x 128, two
typedef Tile<2, 2, 2, 2> Small;    // 64 x 64
constexpr int kTile = 256;         // tokens and pieces are filled up to whole tiles of any size

typedef uint32_t u32x4 __attribute__((ext_vector_type(4)));
typedef short s16x4 __attribute__((ext_vector_type(4)));
typedef bf16 bf16x8 __attribute__((ext_vector_type(8)));
typedef f16 f16x8 __attribute__((ext_vector_type(8)));
typedef float f32x4 __attribute__((ext_vector_type(4)));
#define LDS_PTR(T, p) ((__attribute__((address_space(3))) T*)(p))
#define GLOBAL_PTR(p) ((const __attribute__((address_space(1))) void*)(p))

template <class T>
__device__ __forceinline__ void multiply(f32x4& c, u32x4 a, u32x4 b) {
  if constexpr (std::is_same_v<T, bf16>) {
    c = __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(bf16x8, a), __builtin_bit_cast(bf16x8, b), c, 0, 0, 0);
  } else if constexpr (std::is_same_v<T, f16>) {
    c = __builtin_amdgcn_mfma_f32_16x16x32_f16(__builtin_bit_cast(f16x8, a), __builtin_bit_cast(f16x8, b), c, 0, 0, 0);
  } else {
    const f32x4 x = __builtin_bit_cast(f32x4, a), y = __builtin_bit_cast(f32x4, b);
#pragma unroll
    for (int e = 0; e < 4; ++e) c = __builtin_amdgcn_mfma_f32_16x16x4f32(x[e], y[e], c, 0, 0, 0);
  }
}

struct Operand {
  const char* p;
  int64_t ld;     // bytes from a row to the next (rows), from one k to the next (columns)
  int64_t last;   // the last row, or the last k, that there is: those behind it read it again
  int64_t edge;   // columns: the byte in a k where the last 16 begin
};

// Columns: what one read takes at several k lies in different banks.  The place of a 16-byte piece of k's row is its own
// number with these bits turned: 16-bit elements, 32 bytes at each of the k 0-3 and 8-11 of 32; fp32, 64 bytes at every 4th k of 16.
template <int S, int R>
__device__ __forceinline__ int turned(int k) {
  if (S == 4) return (k >> 2 & 3) << 2;
  return R == 64 ? ((k >> 1 & 1) | (k >> 3 & 1) << 1) << 1 : ((k & 3) | (k >> 3 & 1) << 2) << 1;
}

// R rows (or columns) of one operand of a stage: R / 8 loads of a wave, shared by the block's waves.
template <class T, bool COLUMNS, int R, int WAVES>
struct Loader {
  static constexpr int S = sizeof(T), kStep = 128 / S, COUNT = R / 8 / WAVES, PER = R * S / 16;   // PER: 16-byte pieces of a k (columns)
  const char* p[COUNT];
  int64_t ld, left;   // left: k from the next stage's first to the last one

  // k of load i's piece in a stage
  __device__ __forceinline__ static int k_of(int i, int wave, int lane) { return (wave * COUNT + i) * (64 / PER) + lane / PER; }

  __device__ __forceinline__ void begin(const Operand& o, int64_t tile0, int64_t k0, int wave, int lane) {
    ld = o.ld;
    left = o.last - k0;
#pragma unroll
    for (int i = 0; i < COUNT; ++i) {
      if constexpr (!COLUMNS) {
        // 8 rows of 128 bytes; 16-byte piece c of row r lies in place c ^ (r / 2 % 8), so that a read of 16 rows at one k meets every bank once
        const int r = (wave * COUNT + i) * 8 + lane / 8, c = (lane % 8) ^ (r / 2 % 8);
        p[i] = o.p + min(tile0 + r, o.last) * ld + k0 * S + c * 16;
      } else {
        const int k = k_of(i, wave, lane), c = (lane % PER) ^ turned<S, R>(k);
        p[i] = o.p + (k0 + k) * ld + min(tile0 * S + c * 16, o.edge);
      }
    }
  }
  // The next stage into `to`.
  __device__ __forceinline__ void load(char* to, int wave, int lane) {
#pragma unroll
    for (int i = 0; i < COUNT; ++i) {
      const char* from = p[i];
      if (COLUMNS && left < kStep - 1) {
        const int64_t behind = k_of(i, wave, lane) - left;
        if (behind > 0) from -= behind * ld;   // the last k
      }
      __builtin_amdgcn_global_load_lds(GLOBAL_PTR(from), LDS_PTR(void, to + (wave * COUNT + i) * 1024), 16, 0, 0);
      p[i] += COLUMNS ? kStep * ld : 128;
    }
    left -= kStep;
  }
};

// 16 rows (m or n, from row0) at half j of a stage, as the matrix instructions
// take them: lane l has row l % 16 and quarter l / 16 of the half's 64 bytes of k.
template <class T, bool COLUMNS, int R>
__device__ __forceinline__ u32x4 fragment(const char* s, int row0, int j, int lane) {
  const int i = lane % 16, g = lane / 16;
  if constexpr (!COLUMNS) {
    return *reinterpret_cast<const u32x4*>(s + (row0 + i) * 128 + (((4 * j + g) ^ (i / 2 % 8)) * 16));
  } else if constexpr (sizeof(T) == 2) {
    // 4 k of 16 columns a read: this lane's address is that of k i / 4 and columns i % 4 * 4, what it gets is column i
    const int k = 32 * j + 8 * g + i / 4;
    const char* at = s + k * (2 * R) + ((((row0 / 8) ^ turned<2, R>(k)) + (i & 3) / 2) * 16 + (i & 1) * 8);
    const s16x4 x = __builtin_amdgcn_ds_read_tr16_b64_v4i16(LDS_PTR(s16x4, at));
    const s16x4 y = __builtin_amdgcn_ds_read_tr16_b64_v4i16(LDS_PTR(s16x4, s + (k + 4) * (2 * R) + ((((row0 / 8) ^ turned<2, R>(k + 4)) + (i & 3) / 2) * 16 + (i & 1) * 8)));
    return __builtin_bit_cast(u32x4, __builtin_shufflevector(x, y, 0, 1, 2, 3, 4, 5, 6, 7));
  } else {
    const int k = 16 * j + 4 * g;
    const uint32_t* at = reinterpret_cast<const uint32_t*>(s + k * (4 * R) + (((row0 / 4) ^ turned<4, R>(k)) * 16 + i * 4));
    u32x4 v;
#pragma unroll
    for (int e = 0; e < 4; ++e) v[e] = at[e * R];
    return v;
  }
}

template <class C>
using Acc = f32x4[C::FM][C::FN];

// acc = the block's product over `steps` stages from k0.  A stage is four steps:
// both halves of k times both halves of a wave's rows of m, whose fragments are
// read a step ahead, between the matrix instructions; the next stage's first
// ones during this one's last step, so the barrier between stages stands before
// that.  The loads of a stage go out in two parts, B's a step and a half after
// A's.  (8192 x 32000 x 2048 bf16 on one unit: 914 us with reads and loads each
// at once, 864 with the reads between, 852 with the loads after the step, 800 with
// them in two parts.  A fragment more in registers and a longer way for the loads: no less.)
// All of LDS is read when it returns.
template <class T, bool AC, bool BC, class C>
__device__ __forceinline__ void product(Acc<C>& acc, const Operand& a, const Operand& b, int64_t m0, int64_t n0, int64_t k0, int64_t steps, char* lds) {
  constexpr int HM = C::FM / 2;
  const int wave = threadIdx.x >> 6, lane = threadIdx.x & 63, wm = wave % C::WM, wn = wave / C::WM;
#pragma unroll
  for (int i = 0; i < C::FM; ++i)
#pragma unroll
    for (int k = 0; k < C::FN; ++k) acc[i][k] = f32x4{0.f, 0.f, 0.f, 0.f};
  if (steps <= 0) return;
  Loader<T, AC, C::M, C::WAVES> la;
  Loader<T, BC, C::N, C::WAVES> lb;
  la.begin(a, m0, k0, wave, lane);
  lb.begin(b, n0, k0, wave, lane);
  const auto load_a = [&](int64_t s) { la.load(lds + (s & 1) * C::STAGE, wave, lane); };
  const auto load_b = [&](int64_t s) { lb.load(lds + (s & 1) * C::STAGE + C::M * 128, wave, lane); };
  u32x4 fa[2][HM], fb[2][C::FN];
  const auto read_a = [&](u32x4 (&f)[HM], const char* stage, int j, int half) {
#pragma unroll
    for (int i = 0; i < HM; ++i) f[i] = fragment<T, AC, C::M>(stage, (wm * C::FM + half * HM + i) * 16, j, lane);
  };
  const auto read_b = [&](u32x4 (&f)[C::FN], const char* stage, int j) {
#pragma unroll
    for (int i = 0; i < C::FN; ++i) f[i] = fragment<T, BC, C::N>(stage + C::M * 128, (wn * C::FN + i) * 16, j, lane);
  };
  const auto step = [&](int j, int half) {
#pragma unroll
    for (int i = 0; i < HM; ++i)
#pragma unroll
      for (int k = 0; k < C::FN; ++k) multiply<T>(acc[half * HM + i][k], fa[half][i], fb[j][k]);
#pragma unroll
    for (int q = 0; q < HM * C::FN / 4; ++q) {   // four matrix instructions, two fragments
      __builtin_amdgcn_sched_group_barrier(0x008, 4, 0);
      __builtin_amdgcn_sched_group_barrier(0x100, (AC || BC) && sizeof(T) == 2 ? 4 : 2, 0);
    }
    __builtin_amdgcn_sched_barrier(0);
  };
  load_a(0);
  load_b(0);
  __builtin_amdgcn_s_waitcnt(0x0f70);   // vmcnt(0): this wave's part of the stage is there
  __syncthreads();
  if (steps > 1) {
    load_a(1);
    load_b(1);
  }
  read_b(fb[0], lds, 0);
  read_a(fa[0], lds, 0, 0);
  for (int64_t s = 0; s < steps; ++s) {
    const char *now = lds + (s & 1) * C::STAGE, *next = lds + (~s & 1) * C::STAGE;
    read_a(fa[1], now, 0, 1);
    step(0, 0);
    if (s > 0 && s + 1 < steps) load_b(s + 1);
    read_b(fb[1], now, 1);
    read_a(fa[0], now, 1, 0);
    step(0, 1);
    read_a(fa[1], now, 1, 1);
    step(1, 0);
    __builtin_amdgcn_s_waitcnt(0x0070);   // vmcnt(0) lgkmcnt(0): the next stage is there, this one is read
    __syncthreads();
    if (s + 1 < steps) {
      read_b(fb[0], next, 0);
      read_a(fa[0], next, 0, 0);
    }
    step(1, 1);
    if (s + 2 < steps) load_a(s + 2);
  }
}

// Element e of acc[i][k] is C[m][n] with these, from the block's first.
template <class C>
__device__ __forceinline__ int tile_m(int i, int e) {
  const int wave = threadIdx.x >> 6;
  return ((wave % C::WM) * C::FM + i) * 16 + (threadIdx.x & 63) / 16 * 4 + e;
}
template <class C>
__device__ __forceinline__ int tile_n(int k) {
  const int wave = threadIdx.x >> 6;
  return ((wave / C::WM) * C::FN + k) * 16 + threadIdx.x % 16;
}

// Calls store(n, m, numbers) for 16 bytes of type S at a time of the block's tile, C[m..][n] = value(i, k): each wave turns
// its part of the tile in its own part of LDS, so that what it stores lies in rows of 256 bytes and more.  (Stored from the
// registers, in pieces of 32 bytes, 16384 x 1024 bf16 took 30 us more.)
template <class S, class C, class Value, class Store>
__device__ __forceinline__ void store_tile(char* lds, Value value, Store store) {
  constexpr int SZ = sizeof(S), V = 16 / SZ, ROW = C::FM * 16 * SZ, CHUNKS = ROW / 16, MASK = CHUNKS < 16 ? CHUNKS - 1 : 15;
  constexpr int OWN = 2 * C::STAGE / C::WAVES, PASSES = C::FN * 16 * ROW > OWN ? C::FN * 16 * ROW / OWN : 1, K = C::FN / PASSES;
  const int wave = threadIdx.x >> 6, lane = threadIdx.x & 63, i16 = lane % 16, g = lane / 16;
  const int m0 = (wave % C::WM) * C::FM * 16, n0 = (wave / C::WM) * C::FN * 16;
  char* own = lds + wave * OWN;
#pragma unroll
  for (int pass = 0; pass < PASSES; ++pass) {
#pragma unroll
    for (int k = 0; k < K; ++k)
#pragma unroll
      for (int i = 0; i < C::FM; ++i) {
        const f32x4 x = value(i, pass * K + k);
        Pack<S, 4> p;
#pragma unroll
        for (int e = 0; e < 4; ++e) p.v[e] = from_f32<S>(x[e]);
        const int at = (i * 16 + g * 4) * SZ;   // byte in the row; the 16-byte pieces of row n are turned by n
        *reinterpret_cast<Pack<S, 4>*>(own + (k * 16 + i16) * ROW + ((at / 16) ^ (i16 & MASK)) * 16 + at % 16) = p;
      }
    // the wave's own reads come after its own writes
#pragma unroll
    for (int t = 0; t < K * 16 * CHUNKS / 64; ++t) {
      const int piece = t * 64 + lane, r = piece / CHUNKS, c = piece % CHUNKS;
      const Pack<S, V> p = *reinterpret_cast<const Pack<S, V>*>(own + r * ROW + ((c ^ (r & MASK)) * 16));
      store(n0 + pass * K * 16 + r, m0 + c * V, p);
    }
  }
}

// Over the four lanes with one n.
template <class Op>
__device__ __forceinline__ float rows_reduce(float x, Op op) {
  const Two a = swap16(x);
  x = op(a.a, a.b);
  const Two b = swap32(x);
  return op(b.a, b.b);
}

// A block's tile, and its part of a split sum.  Blocks go to the eight dies in turn, each with a cache
// of its own: a die gets neighbours, 8 tiles of m by a run of n at a time, and few of the parts (4096 of
// 50257 x 1024 bf16, backward 16 us less than with every part on every die).
struct Place {
  int64_t m, n;
  uint32_t split;
};
__device__ __forceinline__ Place place(uint32_t mt, uint32_t nt) {
  const uint32_t per = gridDim.x / 8, rest = gridDim.x % 8, die = blockIdx.x % 8;
  uint32_t id = die * per + min(die, rest) + blockIdx.x / 8;
  const uint32_t split = id / (mt * nt);
  id -= split * mt * nt;
  const uint32_t group = id / (8 * nt), first = group * 8, rows = min(8u, mt - first), in = id - group * 8 * nt;
  return {first + in % rows, in / rows, split};
}

// What the backward pass keeps on the device: tokens with a target (the others
// have no gradient), and the power of two that G is scaled by.
struct Header {
  int32_t n;
  float scale, inv_scale;
};

// A token of those with a target.
struct Row {
  float lse;      // of its logits
  float g;        // its gradient, scaled
  int32_t target;
  int32_t from;   // its row of x
};

__device__ __forceinline__ int64_t load_id(const void* ids, int32_t bytes, int64_t i) {
  return bytes == 8 ? static_cast<const int64_t*>(ids)[i] : int64_t(static_cast<const int32_t*>(ids)[i]);
}

// ---------------------------------------------------------------------------
// Forward

struct Stats {
  Operand w, x;
  const void* targets;
  float2* part;    // [vocabulary tile][n]: largest logit, and the sum of exp of the rest
  float* hit;      // the target's logit
  int64_t v0, vend, n, steps;
  uint32_t mt, nt;
  int32_t id_bytes;
};

template <class T, class C>
__global__ __launch_bounds__(C::THREADS, 2) void k_ce_stats(Stats a) {
  __shared__ __attribute__((aligned(1024))) char lds[2 * C::STAGE];
  const Place t = place(a.mt, a.nt);
  const int64_t m0 = t.m * C::M, n0 = t.n * C::N;
  Acc<C> acc;
  product<T, false, false, C>(acc, a.w, a.x, m0, n0, 0, a.steps, lds);
  const int64_t v0 = a.v0 + m0;
  if (v0 + C::M > a.vend) {
#pragma unroll
    for (int i = 0; i < C::FM; ++i)
#pragma unroll
      for (int e = 0; e < 4; ++e)
        if (v0 + tile_m<C>(i, e) >= a.vend)
#pragma unroll
          for (int k = 0; k < C::FN; ++k) acc[i][k][e] = -INFINITY;
  }
  float2(*red)[C::N] = reinterpret_cast<float2(*)[C::N]>(lds);
  const int wave = threadIdx.x >> 6;
#pragma unroll
  for (int k = 0; k < C::FN; ++k) {
    const int64_t tok = n0 + tile_n<C>(k);
    const int64_t at = tok < a.n ? load_id(a.targets, a.id_bytes, tok) - v0 : -1;
    const bool here = at >= 0 && at < C::M && v0 + at < a.vend;
    if (__ballot(here)) {
#pragma unroll
      for (int i = 0; i < C::FM; ++i)
#pragma unroll
        for (int e = 0; e < 4; ++e)
          if (here && at == tile_m<C>(i, e)) a.hit[tok] = acc[i][k][e];
    }
    float m = -INFINITY;
#pragma unroll
    for (int i = 0; i < C::FM; ++i)
#pragma unroll
      for (int e = 0; e < 4; ++e) m = fmaxf(m, acc[i][k][e]);
    m = rows_reduce(m, Max());
    const float mc = m == -INFINITY ? 0.f : m;
    float s = 0.f;
#pragma unroll
    for (int i = 0; i < C::FM; ++i)
#pragma unroll
      for (int e = 0; e < 4; ++e) s += exp2_hw((acc[i][k][e] - mc) * kLog2e);
    s = rows_reduce(s, Add());
    if ((threadIdx.x & 63) < 16) red[wave % C::WM][tile_n<C>(k)] = make_float2(m, s);
  }
  __syncthreads();
  if (threadIdx.x < C::N && n0 + threadIdx.x < a.n) {
    float m = -INFINITY, s = 0.f;
#pragma unroll
    for (int q = 0; q < C::WM; ++q) m = fmaxf(m, red[q][threadIdx.x].x);
    const float mc = m == -INFINITY ? 0.f : m;
#pragma unroll
    for (int q = 0; q < C::WM; ++q) s = fmaf(red[q][threadIdx.x].y, exp2_hw((red[q][threadIdx.x].x - mc) * kLog2e), s);
    a.part[v0 / C::M * a.n + n0 + threadIdx.x] = make_float2(m, s);
  }
}

// Per token, the tiles' maxima and sums in their order: 32 tokens a block, 32 threads a token with every 32nd tile each.
__global__ __launch_bounds__(1024) void k_ce_loss(const float2* part, int64_t tiles, int64_t n, int64_t vocab, const void* targets, int32_t id_bytes,
                                                  const float* hit, float* loss, float* lse) {
  __shared__ float2 red[32][33];
  const int i = threadIdx.x % 32, q = threadIdx.x / 32;
  const int64_t tok = int64_t(blockIdx.x) * 32 + i;
  float m = -INFINITY, s = 0.f;
  if (tok < n) {
    for (int64_t t = q; t < tiles; t += 32 * 8) {
      float2 x[8];
#pragma unroll
      for (int k = 0; k < 8; ++k) x[k] = t + 32 * k < tiles ? part[(t + 32 * k) * n + tok] : make_float2(-INFINITY, 0.f);
      const float old = m;
#pragma unroll
      for (int k = 0; k < 8; ++k) m = fmaxf(m, x[k].x);
      const float mc = m == -INFINITY ? 0.f : m;
      s = old == -INFINITY ? s : s * exp2_hw((old - mc) * kLog2e);   // 0 or NaN so far: whatever the tiles hold, m may be far below 0
#pragma unroll
      for (int k = 0; k < 8; ++k) s = fmaf(x[k].y, exp2_hw((x[k].x - mc) * kLog2e), s);
    }
  }
  red[q][i] = make_float2(m, s);
  __syncthreads();
  if (q || tok >= n) return;
  m = -INFINITY;
#pragma unroll
  for (int k = 0; k < 32; ++k) m = fmaxf(m, red[k][i].x);
  const float mc = m == -INFINITY ? 0.f : m;
  s = 0.f;
#pragma unroll
  for (int k = 0; k < 32; ++k) s = fmaf(red[k][i].y, exp2_hw((red[k][i].x - mc) * kLog2e), s);
  const float log_s = kLn2 * log2f(s);
  if (lse) lse[tok] = m + log_s;
  if (loss) {
    const int64_t t = load_id(targets, id_bytes, tok);
    loss[tok] = t >= 0 && t < vocab ? (m - hit[tok]) + log_s : 0.f;   // small terms, whatever the logits' common offset is
  }
}

// ---------------------------------------------------------------------------
// Rows laid out for the product: 16-byte aligned, filled up with zeros to whole stages of k.

template <class T>
__global__ __launch_bounds__(256) void k_ce_pack(const T* from, int64_t ld, int64_t rows, int64_t cols, T* to, int64_t dp) {
  constexpr int V = kVec<T>;
  const int64_t per = dp / V, all = rows * per;
  for (int64_t i = int64_t(blockIdx.x) * 256 + threadIdx.x; i < all; i += int64_t(gridDim.x) * 256) {
    const int64_t r = i / per, c = (i - r * per) * V;
    reinterpret_cast<Pack<T, V>*>(to + r * dp + c)[0] = load_pack<T, V>(from + r * ld, c, cols);
  }
}

// The tokens with a target, in their order: rows[k] of the k-th, pos[r] its k (-1: none); the scale of G.  At most 64 blocks
// with a run of tokens each, 1024 at a time; a block counts the targets before its run itself (65536 tokens bf16: 12 us, one block 48).
__global__ __launch_bounds__(1024) void k_ce_rows(int64_t n, int64_t vocab, const void* targets, int32_t id_bytes, const float* g, int64_t g_stride,
                                                  const float* lse, int32_t scaled, Header* head, Row* rows, int32_t* pos) {
  __shared__ int32_t count[16];
  __shared__ float most[16];
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  const int64_t run = ((n + 1023) / 1024 + gridDim.x - 1) / gridDim.x * 1024, begin = blockIdx.x * run, end = min(begin + run, n);
  if (begin >= n) return;
  float scale = 1.f;
  if (scaled) {   // |G| up to 2^11: fp16's smallest steps are then 2^-35 to 2^-34 of the largest gradient
    float top = 0.f;
    for (int64_t r0 = threadIdx.x; r0 < n; r0 += 1024 * 8) {
#pragma unroll
      for (int k = 0; k < 8; ++k) {
        const int64_t r = min(r0 + 1024 * k, n - 1), t = load_id(targets, id_bytes, r);
        const float x = fabsf(g[r * g_stride]);
        top = t >= 0 && t < vocab && x < INFINITY ? fmaxf(top, x) : top;
      }
    }
    top = lanes_reduce<64>(top, Max());
    if (lane == 0) most[wave] = top;
    __syncthreads();
    for (int k = 0; k < 16; ++k) top = fmaxf(top, most[k]);
    const int e = int(__float_as_uint(top) >> 23) - 127;   // floor of the logarithm, of normal numbers
    const int k = 10 - e;
    if (top > 0.f) scale = __builtin_ldexpf(1.f, k < -126 ? -126 : k > 126 ? 126 : k);
  }
  struct Token {
    int64_t target;
    float lse, g;
  };
  const auto load = [&](int64_t r) {
    r = min(r, n - 1);
    return Token{load_id(targets, id_bytes, r), lse[r], g[r * g_stride]};
  };
  Token next = load(begin + threadIdx.x);
  int32_t before = 0;
  for (int64_t r0 = threadIdx.x; r0 < begin; r0 += 1024 * 8) {
#pragma unroll
    for (int k = 0; k < 8; ++k) {
      const int64_t r = min(r0 + 1024 * k, begin - 1), t = load_id(targets, id_bytes, r);
      before += r0 + 1024 * k < begin && t >= 0 && t < vocab ? 1 : 0;
    }
  }
#pragma unroll
  for (int d = 1; d < 64; d *= 2) before += __shfl_xor(before, d);
  if (lane == 0) count[wave] = before;
  __syncthreads();
  before = 0;
#pragma unroll
  for (int k = 0; k < 16; ++k) before += count[k];
  __syncthreads();   // count is written again
  for (int64_t r0 = begin; r0 < end; r0 += 1024) {
    const int64_t r = r0 + threadIdx.x;
    const Token now = next;
    next = load(r + 1024);
    const bool there = r < n && now.target >= 0 && now.target < vocab;
    const uint64_t mask = __ballot(there);
    const int32_t mine = __popcll(mask & ((1ull << lane) - 1));
    if (lane == 0) count[wave] = __popcll(mask);
    __syncthreads();
    int32_t at = before, all = 0;
#pragma unroll
    for (int k = 0; k < 16; ++k) {
      if (k < wave) at += count[k];
      all += count[k];
    }
    if (there) rows[at + mine] = {now.lse, now.g * scale, int32_t(now.target), int32_t(r)};
    if (r < n) pos[r] = there ? at + mine : -1;
    before += all;
    __syncthreads();   // count is written again
  }
  if (end == n && threadIdx.x == 0) *head = {before, scale, 1.f / scale};
}

// The rows of x of those tokens, and zeros up to a whole tile.
template <class T>
__global__ __launch_bounds__(256) void k_ce_gather(const T* x, int64_t ldx, int64_t cols, const Header* head, Row* rows, T* to, int64_t dp) {
  constexpr int V = kVec<T>;
  const int64_t n = head->n, all_rows = (n + kTile - 1) / kTile * kTile, per = dp / V, all = all_rows * per;
  for (int64_t i = int64_t(blockIdx.x) * 256 + threadIdx.x; i < all; i += int64_t(gridDim.x) * 256) {
    const int64_t r = i / per, c = (i - r * per) * V;
    Pack<T, V> p;
    if (r < n) {
      p = load_pack<T, V>(x + rows[r].from * ldx, c, cols);
    } else {
#pragma unroll
      for (int k = 0; k < V; ++k) p.v[k] = T(0.f);
      if (c == 0) rows[r] = {0.f, 0.f, -1, -1};
    }
    reinterpret_cast<Pack<T, V>*>(to + r * dp + c)[0] = p;
  }
}

// ---------------------------------------------------------------------------
// Backward

struct Grad {
  Operand w, x;
  const Header* head;
  const Row* rows;
  void* out;       // G of the piece: [tokens][width]
  int64_t v0, vend, width, steps;
  uint32_t mt, nt;
};

template <class T, class C>
__global__ __launch_bounds__(C::THREADS, 2) void k_ce_grad(Grad a) {
  __shared__ __attribute__((aligned(1024))) char lds[2 * C::STAGE];
  const Place t = place(a.mt, a.nt);
  const int64_t m0 = t.m * C::M, n0 = t.n * C::N;
  if (n0 >= a.head->n) return;
  Acc<C> acc;
  product<T, false, false, C>(acc, a.w, a.x, m0, n0, 0, a.steps, lds);
  const int64_t v0 = a.v0 + m0;
  Row rows[C::FN];
#pragma unroll
  for (int k = 0; k < C::FN; ++k) rows[k] = a.rows[n0 + tile_n<C>(k)];
  const bool edge = v0 + C::M > a.vend || n0 + C::N > a.head->n;   // 0 behind the vocabulary and the tokens, whatever the logits are there
  T* out = static_cast<T*>(a.out) + n0 * a.width + m0;
  store_tile<T, C>(
      lds,
      [&](int i, int k) {
        const int m = tile_m<C>(i, 0);
        const int64_t target = rows[k].target - v0;
        f32x4 v;
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          // the difference first: lse, which may be large, is not rounded again.  A probability is at most 1, whatever half a
          // step of lse is (NaN stays NaN)
          const float x = exp2_hw(__builtin_elementwise_minimum((acc[i][k][e] - rows[k].lse) * kLog2e, 0.f));
          v[e] = edge && (v0 + m + e >= a.vend || rows[k].target < 0) ? 0.f : rows[k].g * (x - (target == m + e ? 1.f : 0.f));
        }
        return v;
      },
      [&](int n, int m, const Pack<T, kVec<T>>& p) { *reinterpret_cast<Pack<T, kVec<T>>*>(out + n * a.width + m) = p; });
}

// A product's tiles as fp32 sums: C[m][n] at out[split][n][m].
struct Sums {
  Operand a, b;
  const Header* head;
  float* out;
  int64_t ldo, pitch;        // of a row n, of a split
  int64_t k;                 // the whole sum's length; unused where it goes over the tokens
  uint32_t mt, nt;
  int32_t splits, add;       // add: to what the piece before left
};

// Splits share the stages of k; the first ones take one more where they do not divide.
__device__ __forceinline__ void share(int64_t steps, int32_t splits, int64_t z, int64_t& first, int64_t& count) {
  const int64_t per = steps / splits, rest = steps % splits;
  first = z * per + min(z, rest);
  count = per + (z < rest ? 1 : 0);
}

template <class T, bool BC, class C>
__global__ __launch_bounds__(C::THREADS, 2) void k_ce_sums(Sums a) {
  __shared__ __attribute__((aligned(1024))) char lds[2 * C::STAGE];
  constexpr int kStep = 128 / int(sizeof(T));
  const int64_t n = a.head->n;
  const Place t = place(a.mt, a.nt);
  const int64_t z = t.split;
  const int64_t m0 = t.m * C::M, n0 = t.n * C::N;
  if (!BC && n0 >= n) return;   // n: tokens
  int64_t first, count;
  share(((BC ? n : a.k) + kStep - 1) / kStep, a.splits, z, first, count);
  Acc<C> acc;
  product<T, true, BC, C>(acc, a.a, a.b, m0, n0, first * kStep, count, lds);
  float* out = a.out + z * a.pitch + n0 * a.ldo + m0;
  const int cols = int(min(int64_t(C::M), a.ldo - m0));
  store_tile<float, C>(
      lds, [&](int i, int k) { return acc[i][k]; },
      [&](int n, int m, const Pack<float, 4>& p) {
        if (m >= cols) return;
        Pack<float, 4>* to = reinterpret_cast<Pack<float, 4>*>(out + n * a.ldo + m);
        Pack<float, 4> x = p;
        if (a.add) {
          const Pack<float, 4> old = *to;
#pragma unroll
          for (int e = 0; e < 4; ++e) x.v[e] += old.v[e];
        }
        *to = x;
      });
}

// dw of the piece's rows, from the whole sum over the tokens.
struct WeightGrad {
  Operand a, b;
  const Header* head;
  void* out;        // row 0 of the piece
  int64_t ldo, rows, cols;
  uint32_t mt, nt;
  int32_t dtype, accumulate;
};

template <class T, class C>
__global__ __launch_bounds__(C::THREADS, 2) void k_ce_weight(WeightGrad a) {
  __shared__ __attribute__((aligned(1024))) char lds[2 * C::STAGE];
  constexpr int kStep = 128 / int(sizeof(T));
  const Place t = place(a.mt, a.nt);
  const int64_t m0 = t.m * C::M, n0 = t.n * C::N;
  Acc<C> acc;
  product<T, true, true, C>(acc, a.a, a.b, m0, n0, 0, (int64_t(a.head->n) + kStep - 1) / kStep, lds);
  const float inv = a.head->inv_scale;
  const int rows = int(min(int64_t(C::N), a.rows - n0)), cols = int(min(int64_t(C::M), a.cols - m0));
  const auto value = [&](int i, int k) { return acc[i][k] * inv; };
  const auto write = [&](auto type) {
    using W = decltype(type);
    W* out = static_cast<W*>(a.out) + n0 * a.ldo + m0;
    if (a.accumulate) {   // added before the rounding
      store_tile<float, C>(lds, value, [&](int n, int m, const Pack<float, 4>& p) {
        if (n >= rows || m >= cols) return;
        Pack<W, 4> x = load_pack<W, 4>(out + n * a.ldo, m, cols);
#pragma unroll
        for (int e = 0; e < 4; ++e) x.v[e] = from_f32<W>(to_f32(x.v[e]) + p.v[e]);
        store_pack<W, 4>(out + n * a.ldo, m, cols, x);
      });
    } else {
      store_tile<W, C>(lds, value, [&](int n, int m, const Pack<W, kVec<W>>& p) {
        if (n >= rows || m >= cols) return;
        // the gradient's reader comes later, G's next piece now: past the caches (34 of 1795 us)
        if (m + kVec<W> <= cols) store_stream(reinterpret_cast<Pack<W, kVec<W>>*>(out + n * a.ldo + m), p);
        else store_pack<W, kVec<W>>(out + n * a.ldo, m, cols, p);
      });
    }
  };
  if (a.dtype == kF32) write(float());
  else if (a.dtype == kBF16) write(bf16());
  else write(f16());
}

// Rows of fp32 sums, their splits added in order: dx (pos: the token's row of the sums, -1: zeros) or, without pos, dw.
__global__ __launch_bounds__(256) void k_ce_join(const float* sums, int64_t ld, int64_t pitch, int32_t splits, const Header* head, const int32_t* pos,
                                                 int64_t rows, int64_t cols, void* out, int64_t ldo, int32_t dtype, int32_t accumulate) {
  const float inv = head->inv_scale;
  const int64_t per = (cols + 3) / 4, all = rows * per;
  for (int64_t i = int64_t(blockIdx.x) * 256 + threadIdx.x; i < all; i += int64_t(gridDim.x) * 256) {
    const int64_t r = i / per, c = (i - r * per) * 4, from = pos ? pos[r] : r;
    f32x4 v = {0.f, 0.f, 0.f, 0.f};
    if (from >= 0) {
      const float* at = sums + from * ld + c;
      int32_t z = 0;
      for (; z + 4 <= splits; z += 4) {
        f32x4 x[4];
#pragma unroll
        for (int k = 0; k < 4; ++k) x[k] = *reinterpret_cast<const f32x4*>(at + (z + k) * pitch);
#pragma unroll
        for (int k = 0; k < 4; ++k) v += x[k];
      }
      for (; z < splits; ++z) v += *reinterpret_cast<const f32x4*>(at + z * pitch);
    }
#pragma unroll
    for (int k = 0; k < 4; ++k)
      if (c + k < cols) store_any(out, dtype, r * ldo + c + k, (accumulate ? load_any(out, dtype, r * ldo + c + k) : 0.f) + inv * v[k]);
  }
}

// A matrix of zeros: the gradient of a weight without tokens.
__global__ __launch_bounds__(256) void k_ce_zero(void* out, int64_t ldo, int64_t rows, int64_t cols, int32_t dtype) {
  for (int64_t i = int64_t(blockIdx.x) * 256 + threadIdx.x; i < rows * cols; i += int64_t(gridDim.x) * 256) store_any(out, dtype, i / cols * ldo + i % cols, 0.f);
}

template <class F>
hipError_t with_type(int32_t dtype, F&& f) {
  if (dtype == kF32) return f(float());
  if (dtype == kBF16) return f(bf16());
  return f(f16());
}

int64_t up(int64_t x, int64_t to) { return (x + to - 1) / to * to; }
int64_t size_of(int32_t dtype) { return dtype == kF32 ? 4 : 2; }

// A tile of a product of m x n, and in how many parts the sum over k goes.
enum : int { kLarge = 0, kMiddle = 1, kSmall = 2 };
struct Shape {
  int tile;
  int32_t splits;
};
constexpr int64_t kUnits = 256;   // compute units
int64_t tiles_of(int64_t m, int64_t n, int tile) {
  const int64_t t = 256 >> tile;
  return ((m + t - 1) / t) * ((n + t - 1) / t);
}
// Whole sums: the largest tile that n fills by more than half and that gives most compute units one (bf16, forward: 2048 tokens
// of 32000 x 1024 122 us with the large, 154 and 212 with the smaller ones; 100 of 50257 x 1024 40, 32 and 39; 4096 of 1000 x
// 512 26, 19 and 18).
int whole_tile(int64_t m, int64_t n) {
  for (int tile = kLarge; tile < kSmall; ++tile)
    if (n > 128 >> tile && tiles_of(m, n, tile) >= kUnits * 3 / 4) return tile;
  return kSmall;
}
// Sums that may be split: the largest tile that does with parts of at least 16, 8 and 4 stages (backward, with each for both
// sums: 2048 tokens of 32000 x 1024 430, 633 and 892 us; 512 of 10000 x 512 82, 62 and 83; 3 of 1000 x 65 56, 37 and 28).
Shape split_tile(int64_t m, int64_t n, int64_t steps) {
  for (int tile = kLarge; tile < kSmall; ++tile) {
    if (n <= 128 >> tile) continue;
    const int64_t tiles = tiles_of(m, n, tile), most = std::max<int64_t>(1, steps / (16 >> tile));
    if (tiles * most >= kUnits * 3 / 4) return {tile, int32_t(std::max<int64_t>(1, std::min(most, kUnits / tiles)))};
  }
  const int64_t tiles = tiles_of(m, n, kSmall), most = std::max<int64_t>(1, steps / 4);
  return {kSmall, int32_t(std::max<int64_t>(1, std::min(most, kUnits / tiles)))};
}
template <class F>
void with_tile(int tile, F&& f) {
  if (tile == kLarge) f(Large());
  else if (tile == kMiddle) f(Middle());
  else f(Small());
}
template <class C>
uint32_t count(int64_t x, bool m) { return uint32_t((x + (m ? C::M : C::N) - 1) / (m ? C::M : C::N)); }

// Where things lie in the workspace.
struct Plan {
  int64_t s, np, dp;             // element bytes; tokens and columns filled up
  int64_t width;                 // of a piece of the vocabulary
  Shape sx;                      // of dx: its splits are kept from piece to piece
  int64_t bytes = 0;
  int64_t take(int64_t n) {
    const int64_t at = bytes;
    bytes += up(n, 1024);
    return at;
  }
  int64_t part, hit, x, w, head, rows, pos, g, sum_x, sum_w;
};

Shape x_shape(const Plan& p, int64_t n, int64_t width) { return split_tile(p.dp, n, width * p.s / 128); }
Shape w_shape(const Plan& p, int64_t rows) { return split_tile(p.dp, rows, p.np * p.s / 128); }

constexpr int64_t kPieceBytes = int64_t(128) << 20;   // of G, or of a piece of the weight that is laid out anew

Plan plan(int64_t n, int64_t vocab, int64_t cols, int32_t dtype, bool backward) {
  Plan p{};
  p.s = size_of(dtype);
  p.np = up(n, kTile);
  p.dp = up(cols, 128 / p.s);
  const int64_t all = up(vocab, kTile);
  const int64_t most = std::max(backward ? p.np : 0, p.dp) * p.s;
  p.width = std::min(all, std::max<int64_t>(kPieceBytes / most / kTile, 4) * kTile);
  if (p.width < all && backward) {
    // whole rounds of tiles: their number, times the tokens' tiles, a multiple of the compute units
    int64_t tiles = p.width / kTile, whole = kUnits;
    for (int64_t nt = p.np / kTile; nt % 2 == 0 && whole > 1; nt /= 2) whole /= 2;
    if (tiles > whole) p.width = tiles / whole * whole * kTile;
  }
  p.x = p.take((backward ? p.np : n) * p.dp * p.s);
  p.w = p.take(p.width * p.dp * p.s);
  if (!backward) {
    p.part = p.take(all / (256 >> whole_tile(std::min(vocab, p.width), n)) * n * 8);   // a weight that is not in pieces has no smaller tiles
    p.hit = p.take(n * 4);
    return p;
  }
  p.head = p.take(sizeof(Header));
  p.rows = p.take(p.np * int64_t(sizeof(Row)));
  p.pos = p.take(n * 4);
  p.g = p.take(p.np * p.width * p.s);
  p.sx = x_shape(p, n, p.width);
  p.sum_x = p.take(p.sx.splits * p.np * p.dp * 4);
  // the pieces and the last one
  int64_t most_w = 0;
  for (const int64_t rows : {std::min(vocab, p.width), (vocab - 1) % p.width + 1}) {
    const Shape w = w_shape(p, rows);
    if (w.splits > 1) most_w = std::max(most_w, w.splits * up(rows, kTile) * p.dp * 4);
  }
  p.sum_w = p.take(most_w);
  return p;
}

bool direct(const void* p, int64_t ld, int64_t cols, int64_t s) {
  return reinterpret_cast<uintptr_t>(p) % 16 == 0 && ld * s % 16 == 0 && cols * s % 128 == 0;
}

template <class T>
void pack(const void* from, int64_t ld, int64_t rows, int64_t cols, void* to, int64_t dp, hipStream_t s) {
  const int64_t blocks = (rows * (dp / kVec<T>) + 255) / 256;
  k_ce_pack<T><<<dim3(unsigned(std::min<int64_t>(blocks, 8192))), dim3(256), 0, s>>>(static_cast<const T*>(from), ld, rows, cols, static_cast<T*>(to), dp);
}

template <class T>
hipError_t forward(const LinearCeForward& a, hipStream_t s) {
  const Plan p = plan(a.rows, a.vocab, a.cols, a.dtype, false);
  unsigned char* ws = a.ws;
  Stats g{};
  g.steps = p.dp * p.s / 128;
  g.n = a.rows;
  g.targets = a.targets;
  g.id_bytes = a.id_bytes;
  g.part = reinterpret_cast<float2*>(ws + p.part);
  g.hit = reinterpret_cast<float*>(ws + p.hit);
  if (direct(a.x, a.ldx, a.cols, p.s)) {
    g.x = {static_cast<const char*>(a.x), a.ldx * p.s, a.rows - 1, 0};
  } else {
    pack<T>(a.x, a.ldx, a.rows, a.cols, ws + p.x, p.dp, s);
    g.x = {reinterpret_cast<const char*>(ws + p.x), p.dp * p.s, a.rows - 1, 0};
  }
  const bool whole = direct(a.w, a.ldw, a.cols, p.s);
  const int64_t width = whole ? a.vocab : p.width;
  const int tile = whole_tile(std::min(a.vocab, width), a.rows);
  for (int64_t v0 = 0; v0 < a.vocab; v0 += width) {
    const int64_t rows = std::min(width, a.vocab - v0);
    const char* w = static_cast<const char*>(a.w) + v0 * a.ldw * p.s;
    if (whole) {
      g.w = {w, a.ldw * p.s, rows - 1, 0};
    } else {
      pack<T>(w, a.ldw, rows, a.cols, ws + p.w, p.dp, s);
      g.w = {reinterpret_cast<const char*>(ws + p.w), p.dp * p.s, rows - 1, 0};
    }
    g.v0 = v0;
    g.vend = v0 + rows;
    with_tile(tile, [&](auto c) {
      using C = decltype(c);
      g.mt = count<C>(rows, true);
      g.nt = count<C>(a.rows, false);
      k_ce_stats<T, C><<<dim3(g.mt * g.nt), dim3(C::THREADS), 0, s>>>(g);
    });
  }
  const int64_t parts = (a.vocab + (256 >> tile) - 1) / (256 >> tile);
  k_ce_loss<<<dim3(unsigned((a.rows + 31) / 32)), dim3(1024), 0, s>>>(g.part, parts, a.rows, a.vocab, a.targets, a.id_bytes, g.hit, a.loss, a.lse);
  return hipGetLastError();
}

template <class T>
hipError_t backward(const LinearCeBackward& a, hipStream_t s) {
  const Plan p = plan(a.rows, a.vocab, a.cols, a.dtype, true);
  unsigned char* ws = a.ws;
  Header* head = reinterpret_cast<Header*>(ws + p.head);
  Row* rows = reinterpret_cast<Row*>(ws + p.rows);
  int32_t* pos = reinterpret_cast<int32_t*>(ws + p.pos);
  T* x = reinterpret_cast<T*>(ws + p.x);
  k_ce_rows<<<dim3(unsigned(std::min<int64_t>((a.rows + 1023) / 1024, 64))), dim3(1024), 0, s>>>(a.rows, a.vocab, a.targets, a.id_bytes, a.dloss, a.lddl, a.lse, a.dtype == kF16, head, rows, pos);
  const int64_t blocks = (p.np * (p.dp / kVec<T>) + 255) / 256;
  k_ce_gather<T><<<dim3(unsigned(std::min<int64_t>(blocks, 8192))), dim3(256), 0, s>>>(static_cast<const T*>(a.x), a.ldx, a.cols, head, rows, x, p.dp);
  const Operand xr{reinterpret_cast<const char*>(x), p.dp * p.s, p.np - 1, 0}, xc{xr.p, xr.ld, p.np - 1, p.dp * p.s - 16};
  const bool whole = direct(a.w, a.ldw, a.cols, p.s);
  float* sum_x = reinterpret_cast<float*>(ws + p.sum_x);
  float* sum_w = reinterpret_cast<float*>(ws + p.sum_w);
  char* G = reinterpret_cast<char*>(ws + p.g);
  for (int64_t v0 = 0; v0 < a.vocab; v0 += p.width) {
    const int64_t n = std::min(p.width, a.vocab - v0);
    const char* w = static_cast<const char*>(a.w) + v0 * a.ldw * p.s;
    int64_t ldw = a.ldw * p.s;
    if (!whole) {
      pack<T>(w, a.ldw, n, a.cols, ws + p.w, p.dp, s);
      w = reinterpret_cast<const char*>(ws + p.w);
      ldw = p.dp * p.s;
    }
    Grad g{};
    g.w = {w, ldw, n - 1, 0};
    g.x = xr;
    g.head = head;
    g.rows = rows;
    g.out = G;
    g.v0 = v0;
    g.vend = v0 + n;
    g.width = p.width;
    g.steps = p.dp * p.s / 128;
    // whole tiles of any size: what the sums below read of G is written
    with_tile(whole_tile(n, a.rows), [&](auto c) {
      using C = decltype(c);
      g.mt = count<C>(up(n, kTile), true);
      g.nt = count<C>(p.np, false);
      k_ce_grad<T, C><<<dim3(g.mt * g.nt), dim3(C::THREADS), 0, s>>>(g);
    });
    if (a.dx) {
      Sums q{};
      q.a = {w, ldw, n - 1, p.dp * p.s - 16};
      q.b = {G, p.width * p.s, p.np - 1, 0};
      q.head = head;
      q.out = sum_x;
      q.ldo = p.dp;
      q.pitch = p.np * p.dp;
      q.k = up(n, kTile);
      q.splits = p.sx.splits;
      q.add = v0 > 0;
      with_tile(p.sx.tile, [&](auto c) {
        using C = decltype(c);
        q.mt = count<C>(p.dp, true);
        q.nt = count<C>(a.rows, false);
        k_ce_sums<T, false, C><<<dim3(q.mt * q.nt * unsigned(q.splits)), dim3(C::THREADS), 0, s>>>(q);
      });
    }
    if (a.dw) {
      const Operand gc{G, p.width * p.s, p.np - 1, p.width * p.s - 16};
      char* out = static_cast<char*>(a.dw) + v0 * a.lddw * size_of(a.gdtype);
      const Shape shape = w_shape(p, n);
      if (shape.splits > 1) {
        Sums q{};
        q.a = xc;
        q.b = gc;
        q.head = head;
        q.out = sum_w;
        q.ldo = p.dp;
        q.pitch = up(n, kTile) * p.dp;
        q.splits = shape.splits;
        with_tile(shape.tile, [&](auto c) {
          using C = decltype(c);
          q.mt = count<C>(p.dp, true);
          q.nt = count<C>(n, false);
          k_ce_sums<T, true, C><<<dim3(q.mt * q.nt * unsigned(q.splits)), dim3(C::THREADS), 0, s>>>(q);
        });
        const int64_t work = (n * ((a.cols + 3) / 4) + 255) / 256;
        k_ce_join<<<dim3(unsigned(std::min<int64_t>(work, 8192))), dim3(256), 0, s>>>(sum_w, p.dp, q.pitch, q.splits, head, nullptr, n, a.cols, out, a.lddw,
                                                                                    a.gdtype, a.accumulate);
      } else {
        WeightGrad q{};
        q.a = xc;
        q.b = gc;
        q.head = head;
        q.out = out;
        q.ldo = a.lddw;
        q.rows = n;
        q.cols = a.cols;
        q.dtype = a.gdtype;
        q.accumulate = a.accumulate;
        with_tile(shape.tile, [&](auto c) {
          using C = decltype(c);
          q.mt = count<C>(p.dp, true);
          q.nt = count<C>(n, false);
          k_ce_weight<T, C><<<dim3(q.mt * q.nt), dim3(C::THREADS), 0, s>>>(q);
        });
      }
    }
  }
  if (a.dx) {
    const int64_t work = (a.rows * ((a.cols + 3) / 4) + 255) / 256;
    k_ce_join<<<dim3(unsigned(std::min<int64_t>(work, 8192))), dim3(256), 0, s>>>(sum_x, p.dp, p.np * p.dp, p.sx.splits, head, pos, a.rows, a.cols, a.dx, a.lddx,
                                                                                a.dtype, 0);
  }
  return hipGetLastError();
}

}  // namespace

size_t linear_ce_bytes(int64_t rows, int64_t vocab, int64_t cols, int32_t dtype, bool backward_pass) {
  return rows ? size_t(plan(rows, vocab, cols, dtype, backward_pass).bytes) : 0;
}

hipError_t launch_linear_ce_forward(const LinearCeForward& a, hipStream_t s) {
  if (a.rows == 0) return hipSuccess;
  return with_type(a.dtype, [&](auto t) { return forward<decltype(t)>(a, s); });
}

hipError_t launch_linear_ce_backward(const LinearCeBackward& a, hipStream_t s) {
  if (a.rows == 0) {
    if (a.dw && !a.accumulate) k_ce_zero<<<dim3(4096), dim3(256), 0, s>>>(a.dw, a.lddw, a.vocab, a.cols, a.gdtype);
    return hipGetLastError();
  }
  return with_type(a.dtype, [&](auto t) { return backward<decltype(t)>(a, s); });
}

}  // namespace lopt
