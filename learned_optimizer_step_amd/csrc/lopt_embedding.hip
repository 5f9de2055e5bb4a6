// Token embedding and its gradient.
//   out[t] = scale W[ids[t] - row0]      (0 where the id is no row of W)
//   dW[v]  = scale sum over t with ids[t] - row0 = v of dout[t]
// Both are bound by HBM.  The gradient sorts the token positions by id with a
// stable radix sort, so a row's tokens are summed in the order of their
// positions and the result has the same bits every time: no float atomics.
#include <hip/hip_runtime.h>

#include <algorithm>

#include "lopt_ops.h"
#include "lopt_ops_device.h"

namespace lopt {
namespace {

// The sort.  A list of up to kOneBlock tokens is sorted by one block in LDS in
// one launch (4096 tokens: 9.5 us; as two launches a pass 15 and their gaps;
// 16384: 31 against 19).
constexpr int kSortBlock = 1024;
constexpr int64_t kOneBlock = 8192;
constexpr int64_t kMarkedRows = 262144;   // rows that one block marks
constexpr int kTile = 1024;       // tokens a block of a longer sort takes at a time (4096: twice the time a pass)
constexpr int kMaxTiles = 256;    // blocks of the sort
constexpr int kDigits = 256;      // 8 bits a pass

constexpr int64_t kFew = 128;     // tokens that k_embedding_few takes (77 of 1000 x 65: 5 us, 13 with a sort)
constexpr int64_t kFewWaves = 1 << 24;   // its waves, each in a grid of at most 2^32 - 1 threads; more take the sort's path

// The sums: see k_embedding_sum.
constexpr int kSumVec = 4;        // columns of a lane
constexpr int kSumAhead = 8;      // tokens loaded at a time, while those before them are added up
constexpr int kReach = 8;         // tokens that a chunk takes from the next one to end a run

// Row of the table that an id names, `rows` if none.
__device__ __forceinline__ uint32_t row_of(const void* ids, int id_bytes, int64_t t, int64_t row0, int64_t rows) {
  const int64_t id = id_bytes == 8 ? static_cast<const int64_t*>(ids)[t] : int64_t(static_cast<const int32_t*>(ids)[t]);
  // row0 is within [0, 2^40], so an id at or above it gives a difference that is an int64_t
  if (id < row0) return uint32_t(rows);
  const int64_t v = id - row0;
  return uint32_t(v < rows ? v : rows);
}

// ---------------------------------------------------------------------------
// Forward: TPR threads write 8 TPR columns of one token.
template <class TT, class TO, int TPR, int MODE>
__global__ __launch_bounds__(256) void k_embedding_forward(EmbeddingForward a) {
  constexpr int V = 8;
  const int64_t slabs = (a.cols + V * TPR - 1) / (V * TPR), units = a.n_ids * slabs;
  for (int64_t u = int64_t(blockIdx.x) * (256 / TPR) + threadIdx.x / TPR; u < units; u += int64_t(gridDim.x) * (256 / TPR)) {
    const int64_t t = slabs == 1 ? u : u / slabs;
    const uint32_t v = row_of(a.ids, a.id_bytes, t, a.row0, a.rows);
    const bool there = int64_t(v) < a.rows;
    const RowVec<TT, V, MODE> at(int((u - t * slabs) * (V * TPR)) + int(threadIdx.x % TPR) * V, int(a.cols));
    Pack<TT, V> p{};
    if (there) p = at.load(static_cast<const TT*>(a.table) + int64_t(v) * a.ldt);
    Pack<TO, V> o;
#pragma unroll
    for (int i = 0; i < V; ++i) o.v[i] = from_f32<TO>(there ? to_f32(p.v[i]) * a.scale : 0.f);
    at.store(static_cast<TO*>(a.out) + t * a.ldo, o);
  }
}

// ---------------------------------------------------------------------------
// Workspace of the gradient.
struct Work {
  uint32_t *key[2], *val[2];   // tokens' rows and positions, by turns
  uint32_t* hist;              // [tiles][256] digits of a pass
  unsigned char* touched;      // rows that some token names, if `marks`
  uint32_t* crossing;          // number of runs that cross a chunk's border, then the chunks they begin in
  float* part;                 // [chunks][2][cols]: sums of runs that cross a chunk's first / last token
  int64_t tiles, rounds, chunks;
  int32_t chunk;               // tokens of a chunk
  int32_t passes;
  int32_t marks;
  int32_t sorted;              // which key and val hold the sorted tokens
  size_t bytes;
};

size_t up(size_t x) { return (x + 255) / 256 * 256; }

Work layout(unsigned char* ws, int64_t n, int64_t rows, int64_t cols) {
  Work w{};
  const int64_t tiles = (n + kTile - 1) / kTile;
  w.rounds = std::max<int64_t>(1, (tiles + kMaxTiles - 1) / kMaxTiles);
  w.tiles = std::max<int64_t>(1, (tiles + w.rounds - 1) / w.rounds);
  // long chunks leave fewer sums of crossing runs, as long as the chip has waves (four to eight per SIMD)
  const int64_t slabs = (cols + 64 * kSumVec - 1) / (64 * kSumVec);
  w.chunk = 8;
  for (const int c : {16, 32, 48})
    if (n / c * slabs >= 4096) w.chunk = c;
  w.chunks = (n + w.chunk - 1) / w.chunk;
  w.passes = 1;
  while (w.passes < 4 && (uint64_t(rows) >> (8 * w.passes)) != 0) ++w.passes;
  w.sorted = n <= kOneBlock ? 0 : w.passes & 1;
  size_t at = 0;
  auto take = [&](size_t bytes) {
    unsigned char* p = ws ? ws + at : nullptr;
    at += up(bytes);
    return p;
  };
  for (int k = 0; k < 2; ++k) {
    w.key[k] = reinterpret_cast<uint32_t*>(take(size_t(n) * 4));
    w.val[k] = reinterpret_cast<uint32_t*>(take(size_t(n) * 4));
  }
  w.hist = reinterpret_cast<uint32_t*>(take(size_t(w.tiles) * kDigits * 4));
  w.marks = n > kOneBlock || rows <= kMarkedRows;   // one block takes long to clear the marks of more
  w.touched = take(w.marks ? size_t(rows) : 0);
  w.crossing = reinterpret_cast<uint32_t*>(take(size_t(w.chunks + 1) * 4));
  w.part = reinterpret_cast<float*>(take(size_t(w.chunks) * 2 * size_t(cols) * 4));
  w.bytes = at;
  return w;
}

// The sort's launches keep few compute units busy, so blocks behind the sort's
// clear the gradient meanwhile: see launch_embedding_backward.  What is written
// here is not read again soon, and passes the caches by (65,536 tokens of
// 32,000 x 2048: 150 us for everything with ordinary accesses, 135 so, 122 with
// dout read that way too).
struct Clear {
  uint16_t* to;             // 2-byte units
  int64_t row, ld;          // units of a row
  int64_t first, last;      // this launch's rows
  const unsigned char* touched;   // rows that some token names, which are left; NULL: clear every row
};

__device__ __forceinline__ void clear_vector(const Clear& c, int64_t r, int64_t i) {
  const Pack<uint16_t, 8> zero{};
  uint16_t* row = c.to + r * c.ld;
  if (i + 8 <= c.row) store_stream(reinterpret_cast<Pack<uint16_t, 8>*>(row + i), zero);
  else store_pack<uint16_t, 8>(row, i, c.row, zero);
}

// The rows' 16-byte vectors in one sequence.  Every row: a vector a thread in
// many short blocks, as a grid that stays and strides writes slower (206 MB:
// 34 us, 41 with 1024 blocks).  Unmarked rows: a grid that strides and looks
// up four marks at a time (65,536 tokens of 32,000 x 2048: 120 us for
// everything, 130 with short blocks); row and place in it are carried along.
template <int THREADS>
__device__ __forceinline__ void clear_block(const Clear& c, int64_t block, int64_t blocks) {
  const uint32_t per = uint32_t((c.row + 7) / 8), last = uint32_t(c.last);
  if (!c.touched) {
    const int64_t end = (c.last - c.first) * per;
    for (int64_t at = block * THREADS + threadIdx.x; at < end; at += blocks * THREADS) {
      const int64_t turn = at / per;
      clear_vector(c, c.first + turn, (at - turn * per) * 8);
    }
    return;
  }
  constexpr int U = 4;
  // within a turn, and from a turn's last to the next one's first
  const uint32_t step_r = THREADS / per, step_i = THREADS - step_r * per;
  const int64_t jump = (blocks * U - U + 1) * THREADS;
  const uint32_t jump_r = uint32_t(jump / per), jump_i = uint32_t(jump - int64_t(jump_r) * per);
  const int64_t at = block * (THREADS * U) + threadIdx.x;
  uint32_t r = uint32_t(c.first + at / per), i = uint32_t(at % per);
  const auto go = [&](uint32_t dr, uint32_t di) {
    r += dr;
    i += di;
    if (i >= per) {
      i -= per;
      ++r;
    }
  };
  while (r < last) {
    uint32_t rs[U], is[U];
    bool skip[U];
#pragma unroll
    for (int k = 0; k < U; ++k) {
      rs[k] = r;
      is[k] = i;
      skip[k] = r >= last || c.touched[r];
      if (k + 1 < U) go(step_r, step_i);
    }
    go(jump_r, jump_i);
#pragma unroll
    for (int k = 0; k < U; ++k)
      if (!skip[k]) clear_vector(c, rs[k], int64_t(is[k]) * 8);
  }
}

// Digits of every tile; the first pass reads the ids.
__global__ __launch_bounds__(kSortBlock) void k_embedding_digits(EmbeddingBackward a, Work w, int pass, Clear clear) {
  if (int64_t(blockIdx.x) >= w.tiles) {
    clear_block<kSortBlock>(clear, blockIdx.x - w.tiles, gridDim.x - w.tiles);
    return;
  }
  __shared__ uint32_t hist[kDigits];
  for (int d = threadIdx.x; d < kDigits; d += kSortBlock) hist[d] = 0;
  if (pass == 0) {
    if (blockIdx.x == 0 && threadIdx.x == 0) w.crossing[0] = 0;
    if (!a.accumulate)
      for (int64_t v = (int64_t(blockIdx.x) * kSortBlock + threadIdx.x) * 16; v < a.rows; v += w.tiles * kSortBlock * 16)
        store_pack<unsigned char, 16>(w.touched, v, a.rows, Pack<unsigned char, 16>{});
  }
  __syncthreads();
  const int64_t first = int64_t(blockIdx.x) * w.rounds * kTile, last = std::min<int64_t>(a.n_ids, first + w.rounds * kTile);
#pragma unroll 4
  for (int64_t t = first + threadIdx.x; t < last; t += kSortBlock) {
    const uint32_t key = pass == 0 ? row_of(a.ids, a.id_bytes, t, a.row0, a.rows) : w.key[pass & 1][t];
    atomicAdd(&hist[(key >> (8 * pass)) & 255], 1u);
  }
  __syncthreads();
  for (int d = threadIdx.x; d < kDigits; d += kSortBlock) w.hist[int64_t(blockIdx.x) * kDigits + d] = hist[d];
}

// Exclusive scan of one value per digit over the first 256 threads of a block.
__device__ __forceinline__ uint32_t scan_digits(uint32_t x, uint32_t* wave_total) {
  const int lane = threadIdx.x & 63;
  uint32_t inc = x;
#pragma unroll
  for (int o = 1; o < 64; o <<= 1) {
    const uint32_t y = __shfl_up(inc, o);
    if (lane >= o) inc += y;
  }
  if (threadIdx.x < kDigits && lane == 63) wave_total[threadIdx.x >> 6] = inc;
  __syncthreads();
  uint32_t before = 0;
  if (threadIdx.x < kDigits)
    for (int k = 0; k < int(threadIdx.x >> 6); ++k) before += wave_total[k];
  __syncthreads();
  return before + inc - x;
}

// The lanes of the wave with this lane's digit.
__device__ __forceinline__ uint64_t same_digit(uint32_t digit) {
  uint64_t m = ~uint64_t(0);
#pragma unroll
  for (int b = 0; b < 8; ++b) {
    const bool bit = (digit >> b) & 1;
    const uint64_t set = __ballot(bit);
    m &= bit ? set : ~set;
  }
  return m;
}

constexpr int kSortWaves = kSortBlock / 64;

// rank[j]: the wave's tokens before token j of this lane with its digit, by
// the order of the tokens (64 consecutive ones for each j); count: the wave's
// tokens of every digit.
template <int N>
__device__ __forceinline__ void rank_wave(const uint32_t (&key)[N], int shift, uint32_t* count, uint32_t (&rank)[N]) {
  const int lane = threadIdx.x & 63;
#pragma unroll
  for (int j = 0; j < N; ++j) {
    const uint32_t digit = (key[j] >> shift) & 255;
    const uint64_t same = same_digit(digit), lower = same & ((uint64_t(1) << lane) - 1);
    rank[j] = count[digit] + __popcll(lower);
    // the wave's reads of its counts come before its writes, and those before the next reads
    __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
    __builtin_amdgcn_wave_barrier();
    if (lower == 0) count[digit] += __popcll(same);
    __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
    __builtin_amdgcn_wave_barrier();
  }
}

__device__ __forceinline__ void clear_counts(uint32_t (&count)[kSortWaves][kDigits]) {
  uint4* c = reinterpret_cast<uint4*>(&count[0][0]);
  for (int i = threadIdx.x; i < kSortWaves * kDigits / 4; i += kSortBlock) c[i] = uint4{0, 0, 0, 0};
}

// All of a short list in one block: every pass in LDS.  Behind the list's end
// the keys are all ones and stay last (the sort is stable).
template <int N>
__global__ __launch_bounds__(kSortBlock) void k_embedding_sort(EmbeddingBackward a, Work w, Clear clear) {
  if (blockIdx.x > 0) {
    clear_block<kSortBlock>(clear, blockIdx.x - 1, gridDim.x - 1);
    return;
  }
  __shared__ uint32_t count[kSortWaves][kDigits];
  __shared__ uint32_t skey[kSortBlock * N], sval[kSortBlock * N];
  __shared__ uint32_t wave_total[4];
  const int wave = threadIdx.x >> 6, first = wave * 64 * N + (threadIdx.x & 63);
  const int n = int(a.n_ids);
  uint32_t key[N], val[N], rank[N];
#pragma unroll
  for (int j = 0; j < N; ++j) {
    const int t = first + j * 64;
    key[j] = t < n ? row_of(a.ids, a.id_bytes, t, a.row0, a.rows) : ~uint32_t(0);
    val[j] = uint32_t(t);
  }
  if (threadIdx.x == 0) w.crossing[0] = 0;
  if (w.marks && !a.accumulate) {
    for (int64_t v = int64_t(threadIdx.x) * 16; v < a.rows; v += kSortBlock * 16)
      store_pack<unsigned char, 16>(w.touched, v, a.rows, Pack<unsigned char, 16>{});
    __syncthreads();
#pragma unroll
    for (int j = 0; j < N; ++j)
      if (int64_t(key[j]) < a.rows) w.touched[key[j]] = 1;
  }
  for (int pass = 0; pass < w.passes; ++pass) {
    clear_counts(count);
    __syncthreads();
    rank_wave<N>(key, 8 * pass, count[wave], rank);
    __syncthreads();
    uint32_t total = 0;
    if (threadIdx.x < kDigits)
#pragma unroll
      for (int k = 0; k < kSortWaves; ++k) total += count[k][threadIdx.x];
    uint32_t at = scan_digits(total, wave_total);
    if (threadIdx.x < kDigits)
#pragma unroll
      for (int k = 0; k < kSortWaves; ++k) {
        const uint32_t c = count[k][threadIdx.x];
        count[k][threadIdx.x] = at;
        at += c;
      }
    __syncthreads();
#pragma unroll
    for (int j = 0; j < N; ++j) {
      const uint32_t to = count[wave][(key[j] >> (8 * pass)) & 255] + rank[j];
      skey[to] = key[j];
      sval[to] = val[j];
    }
    __syncthreads();
    if (pass + 1 < w.passes)
#pragma unroll
      for (int j = 0; j < N; ++j) {
        key[j] = skey[first + j * 64];
        val[j] = sval[first + j * 64];
      }
  }
  for (int t = threadIdx.x; t < n; t += kSortBlock) {
    w.key[0][t] = skey[t];
    w.val[0][t] = sval[t];
  }
}

// One stable pass over a long list: every token goes behind the tokens of
// lower digits and the earlier ones of its own.
__global__ __launch_bounds__(kSortBlock) void k_embedding_place(EmbeddingBackward a, Work w, int pass, Clear clear) {
  if (int64_t(blockIdx.x) >= w.tiles) {
    clear_block<kSortBlock>(clear, blockIdx.x - w.tiles, gridDim.x - w.tiles);
    return;
  }
  constexpr int N = kTile / kSortBlock;
  __shared__ uint32_t count[kSortWaves][kDigits];
  __shared__ uint32_t base[kDigits];
  __shared__ uint32_t wave_total[4];
  const int wave = threadIdx.x >> 6;

  // tokens of each digit, and those of the tiles before this block's: four threads a digit
  uint32_t total = 0, before = 0;
  {
    const int d = threadIdx.x & 255, q = threadIdx.x >> 8;
#pragma unroll 8
    for (int64_t b = q; b < w.tiles; b += 4) {
      const uint32_t h = w.hist[b * kDigits + d];
      before += b < int64_t(blockIdx.x) ? h : 0;
      total += h;
    }
    count[q][d] = total;
    count[q + 4][d] = before;
    __syncthreads();
    if (threadIdx.x < kDigits) {
      total = count[0][d] + count[1][d] + count[2][d] + count[3][d];
      before = count[4][d] + count[5][d] + count[6][d] + count[7][d];
    } else {
      total = 0;
    }
  }
  const uint32_t start = scan_digits(total, wave_total);
  if (threadIdx.x < kDigits) base[threadIdx.x] = start + before;

  for (int64_t round = 0; round < w.rounds; ++round) {
    const int64_t first = (int64_t(blockIdx.x) * w.rounds + round) * kTile + wave * 64 * N + (threadIdx.x & 63);
    uint32_t key[N], val[N], rank[N];
#pragma unroll
    for (int j = 0; j < N; ++j) {
      const int64_t t = first + j * 64;
      key[j] = ~uint32_t(0);   // behind the list's end: last in its tile
      val[j] = uint32_t(t);
      if (t < a.n_ids) {
        if (pass == 0) {
          key[j] = row_of(a.ids, a.id_bytes, t, a.row0, a.rows);
          if (!a.accumulate && int64_t(key[j]) < a.rows) w.touched[key[j]] = 1;
        } else {
          key[j] = w.key[pass & 1][t];
          val[j] = w.val[pass & 1][t];
        }
      }
    }
    __syncthreads();
    clear_counts(count);
    __syncthreads();
    rank_wave<N>(key, 8 * pass, count[wave], rank);
    __syncthreads();
    if (threadIdx.x < kDigits) {
      uint32_t at = base[threadIdx.x];
#pragma unroll
      for (int k = 0; k < kSortWaves; ++k) {
        const uint32_t c = count[k][threadIdx.x];
        count[k][threadIdx.x] = at;
        at += c;
      }
      base[threadIdx.x] = at;
    }
    __syncthreads();
#pragma unroll
    for (int j = 0; j < N; ++j)
      if (first + j * 64 < a.n_ids) {
        const uint32_t to = count[wave][(key[j] >> (8 * pass)) & 255] + rank[j];
        w.key[(pass + 1) & 1][to] = key[j];
        w.val[(pass + 1) & 1][to] = val[j];
      }
  }
}

// x, a vector of sums of a row's columns, into the gradient's row.
template <class TG, int V, int MODE>
__device__ __forceinline__ void store_row(const EmbeddingBackward& a, TG* to, const SlabVec<V, MODE>& at, const float (&x)[V]) {
  Pack<TG, V> p{};
  if (a.accumulate) p = at.load(static_cast<const TG*>(to));
#pragma unroll
  for (int i = 0; i < V; ++i) p.v[i] = from_f32<TG>(to_f32(p.v[i]) + x[i] * a.scale);
  at.store(to, p);
}

// Lanes from the first on that hold `key`.
__device__ __forceinline__ int leading(uint32_t lane_key, uint32_t key) {
  const uint64_t other = __ballot(lane_key != key);
  return other ? __builtin_ctzll(other) : 64;
}

// A lane's 64-bit value, uniform.
__device__ __forceinline__ uint64_t of_lane(uint64_t x, int lane) {
  return uint64_t(uint32_t(__builtin_amdgcn_readlane(uint32_t(x >> 32), lane))) << 32 |
         uint32_t(__builtin_amdgcn_readlane(uint32_t(x), lane));
}

// One chunk of sorted tokens over the slab of columns from slab0.
template <class TD, class TG, int MODE>
__device__ __forceinline__ void sum_chunk(const EmbeddingBackward& a, const Work& w, int64_t chunk, int64_t slab0) {
  constexpr int V = kSumVec, U = kSumAhead;
  const int lane = threadIdx.x & 63;
  const uint32_t* skey = w.key[w.sorted];
  const uint32_t* sval = w.val[w.sorted];
  const uint32_t none = uint32_t(a.rows);
  // the chunk's tokens and kReach + 1 behind it, one a lane
  const int64_t p0 = chunk * w.chunk, left = a.n_ids - p0;
  const int own = int(std::min<int64_t>(left, w.chunk));
  const int64_t mine = p0 + (lane < left ? lane : left - 1);
  uint32_t lane_key = skey[mine], lane_val = sval[mine];
  uint32_t prev = skey[p0 > 0 ? p0 - 1 : 0];
  if (p0 == 0) prev = none;
  if (lane >= left || lane >= w.chunk + kReach + 1) lane_key = none;
  if (lane_key == none) lane_val = 0;   // tokens of no row are read as token 0 and left out
  // tokens that the chunk before takes, and tokens taken from the chunk behind
  const int head = leading(lane_key, prev);
  const int first = prev != none && head <= kReach ? head : 0;
  const uint32_t last = __builtin_amdgcn_readlane(lane_key, own - 1);
  const int more = own < w.chunk ? 0 : leading(__shfl_down(lane_key, own), last);
  const int n = more <= kReach ? own + more : own;
  const bool ends = more <= kReach;   // the last run ends here
  const uint32_t begin = __builtin_amdgcn_readlane(lane_key, first < own ? first : 0);
  if (first >= own || begin == none) return;   // all of it belongs to the chunk before, or to no row
  bool inside = begin != prev;                 // the run began in this chunk
  // bit i: token i + 1 is of another row than token i
  const uint64_t change = __ballot(lane_key != uint32_t(__shfl_down(lane_key, 1)));
  const uint64_t from = uint64_t(lane_val) * uint64_t(a.ldd) * sizeof(TD), to = uint64_t(lane_key) * uint64_t(a.ldt) * sizeof(TG);
  const SlabVec<V, MODE> at(slab0, lane * V, a.cols);
  const char* dout = static_cast<const char*>(a.dout);
  char* dtable = static_cast<char*>(a.dtable);
  float acc[V] = {};
  float* part = w.part + size_t(chunk) * 2 * size_t(a.cols);
  const auto leave = [&](float* to) {
    Pack<float, V> p;
#pragma unroll
    for (int i = 0; i < V; ++i) p.v[i] = acc[i];
    at.store(to, p);
  };
  Pack<TD, V> p[U], q[U];
  const auto load = [&](Pack<TD, V>(&x)[U], int i0) {
#pragma unroll
    for (int j = 0; j < U; ++j) x[j] = at.load_once(reinterpret_cast<const TD*>(dout + of_lane(from, i0 + j < n ? i0 + j : n - 1)));
  };
  load(q, first);
  for (int i0 = first; i0 < n; i0 += U) {
#pragma unroll
    for (int j = 0; j < U; ++j) {
      settle(q[j]);
      p[j] = q[j];
    }
    if (i0 + U < n) load(q, i0 + U);
#pragma unroll
    for (int j = 0; j < U; ++j) {
      const int i = i0 + j;
      if (i >= n) break;
#pragma unroll
      for (int k = 0; k < V; ++k) acc[k] += to_f32(p[j].v[k]);
      if (i + 1 < n && (change >> i & 1)) {   // the run ends here
        if (inside) store_row<TG>(a, reinterpret_cast<TG*>(dtable + of_lane(to, i)), at, acc);
        else leave(part);
        inside = true;
#pragma unroll
        for (int k = 0; k < V; ++k) acc[k] = 0.f;
        if (uint32_t(__builtin_amdgcn_readlane(lane_key, i + 1)) == none) return;
      }
    }
  }
  if (inside && ends) {
    store_row<TG>(a, reinterpret_cast<TG*>(dtable + of_lane(to, n - 1)), at, acc);
  } else if (inside) {
    leave(part + a.cols);
    if (slab0 == 0 && lane == 0) w.crossing[1 + atomicAdd(w.crossing, 1u)] = uint32_t(chunk);
  } else {
    leave(part);
  }
}

// Sums of the sorted tokens: a wave takes `chunk` of them in order over 64
// 16-byte vectors of columns, and writes a row where its run of equal keys
// ends.  A run that has at most kReach tokens behind the chunk's border is taken
// to its end, and the next chunk leaves them out; one that goes on further
// leaves its sum in the workspace: slot 0 if it began before the chunk, slot 1
// if it began in it.
// 65,536 tokens of 32,000 x 2048, bf16 to fp32: 68 us for 241 MB of dout and
// 102 MB of rows, 5.0 TB/s (95 through the caches, whose lines were written
// back meanwhile).
template <class TD, class TG, int MODE>
__global__ __launch_bounds__(256) void k_embedding_sum(EmbeddingBackward a, Work w, int64_t sum_blocks, Clear clear) {
  if (int64_t(blockIdx.x) >= sum_blocks) {
    clear_block<256>(clear, blockIdx.x - sum_blocks, gridDim.x - sum_blocks);
    return;
  }
  constexpr int S = 64 * kSumVec;
  const int64_t slabs = (a.cols + S - 1) / S, units = w.chunks * slabs;
  const int64_t step = sum_blocks * 4;
  for (int64_t unit = int64_t(blockIdx.x) * 4 + __builtin_amdgcn_readfirstlane(threadIdx.x >> 6); unit < units; unit += step)
    sum_chunk<TD, TG, MODE>(a, w, unit / slabs, unit % slabs * S);
}

// A handful of tokens (at most 128) of a small table, in one launch without a
// sort: each wave holds all ids, two a lane.  The wave of the first token of a
// row (and a slab of columns) adds up the row's tokens; waves behind those
// clear the rows that no token names.
template <class TD, class TG, int MODE>
__global__ __launch_bounds__(256) void k_embedding_few(EmbeddingBackward a, int64_t sum_waves) {
  constexpr int V = kSumVec, U = 4, VG = kVec<TG>;
  const int lane = threadIdx.x & 63, n = int(a.n_ids);
  const uint32_t none = uint32_t(a.rows);
  const uint32_t lo = lane < n ? row_of(a.ids, a.id_bytes, lane, a.row0, a.rows) : none;
  const uint32_t hi = 64 + lane < n ? row_of(a.ids, a.id_bytes, 64 + lane, a.row0, a.rows) : none;
  const int64_t wave = int64_t(blockIdx.x) * 4 + __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  if (wave >= sum_waves) {
    if (a.accumulate) return;   // the last block's waves without work
    const Pack<TG, VG> zero{};
    for (int64_t r = wave - sum_waves; r < a.rows; r += int64_t(gridDim.x) * 4 - sum_waves) {
      if (__ballot(lo == uint32_t(r) || hi == uint32_t(r))) continue;
      TG* row = static_cast<TG*>(a.dtable) + r * a.ldt;
      for (int64_t c = lane * VG; c < a.cols; c += 64 * VG) store_pack<TG, VG>(row, c, a.cols, zero);
    }
    return;
  }
  const int64_t slabs = (a.cols + 64 * V - 1) / (64 * V);
  const int t = int(wave / slabs);
  if (t >= n) return;
  const uint32_t key = t < 64 ? __builtin_amdgcn_readlane(lo, t) : __builtin_amdgcn_readlane(hi, t - 64);
  uint64_t same_lo = __ballot(lo == key), same_hi = __ballot(hi == key);
  const int first = same_lo ? __builtin_ctzll(same_lo) : 64 + __builtin_ctzll(same_hi);
  if (key == none || first != t) return;
  const SlabVec<V, MODE> at(wave % slabs * (64 * V), lane * V, a.cols);
  float acc[V] = {};
  int left = __popcll(same_lo) + __popcll(same_hi);
  while (left > 0) {
    Pack<TD, V> p[U];
    int i = 0;
#pragma unroll
    for (int j = 0; j < U; ++j) {
      if (j < left) {   // the next token; behind the last one that one again
        i = same_lo ? __builtin_ctzll(same_lo) : 64 + __builtin_ctzll(same_hi);
        if (same_lo) same_lo &= same_lo - 1;
        else same_hi &= same_hi - 1;
      }
      p[j] = at.load(static_cast<const TD*>(a.dout) + int64_t(i) * a.ldd);
    }
#pragma unroll
    for (int j = 0; j < U; ++j)
      if (j < left)
#pragma unroll
        for (int k = 0; k < V; ++k) acc[k] += to_f32(p[j].v[k]);
    left -= U;
  }
  store_row<TG>(a, static_cast<TG*>(a.dtable) + int64_t(key) * a.ldt, at, acc);
}

// Runs that cross chunks: one block a run and 256 columns adds up the chunks'
// sums, four waves a quarter each, the quarters in order.  The list of runs
// comes in any order, each run's sum does not.
constexpr int kJoinWaves = 4;
template <class TG, int MODE>
__global__ __launch_bounds__(64 * kJoinWaves) void k_embedding_join(EmbeddingBackward a, Work w, unsigned run_blocks, Clear clear) {
  if (blockIdx.y >= run_blocks) {
    clear_block<64 * kJoinWaves>(clear, int64_t(blockIdx.y - run_blocks) * gridDim.x + blockIdx.x,
                                 int64_t(gridDim.y - run_blocks) * gridDim.x);
    return;
  }
  __shared__ float share[kJoinWaves][4][64];
  const uint32_t* skey = w.key[w.sorted];
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  const SlabVec<4, MODE> at(int64_t(blockIdx.x) * 256, lane * 4, a.cols);
  const uint32_t runs = w.crossing[0];
  for (uint32_t i = blockIdx.y; i < runs; i += run_blocks) {
    const int64_t chunk = w.crossing[1 + i];
    const uint32_t key = skey[(chunk + 1) * w.chunk - 1];
    // the last chunk with a sum of the run: more than kReach of its tokens; 64 guesses at a time, near ones first
    int64_t last = chunk;
    const auto reach = [&](int64_t step) {
      const int64_t j = last + (lane + 1) * step;
      const uint64_t ok = __ballot(j * w.chunk + kReach < a.n_ids && skey[j * w.chunk + kReach] == key);
      const int cnt = ok == ~uint64_t(0) ? 64 : __builtin_ctzll(~ok);
      last += cnt * step;
      return cnt == 64;
    };
    if (reach(1)) {
      while (reach(4096)) {}
      while (reach(64)) {}
      while (reach(1)) {}
    }
    const int64_t m = last - chunk + 1, q = (m + kJoinWaves - 1) / kJoinWaves;
    const int64_t b = std::min<int64_t>(m, wave * q), e = std::min<int64_t>(m, b + q);
    float acc[4] = {};
#pragma unroll 8
    for (int64_t j = b; j < e; ++j) {
      const Pack<float, 4> p = at.load(w.part + (size_t(chunk + j) * 2 + (j == 0 ? 1 : 0)) * size_t(a.cols));
#pragma unroll
      for (int k = 0; k < 4; ++k) acc[k] += p.v[k];
    }
#pragma unroll
    for (int k = 0; k < 4; ++k) share[wave][k][lane] = acc[k];
    __syncthreads();
    if (wave == 0) {
#pragma unroll
      for (int s = 1; s < kJoinWaves; ++s)
#pragma unroll
        for (int k = 0; k < 4; ++k) acc[k] += share[s][k][lane];
      store_row<TG>(a, static_cast<TG*>(a.dtable) + int64_t(key) * a.ldt, at, acc);
    }
    __syncthreads();
  }
}

template <class F>
auto with_type(int32_t dtype, F&& f) {
  if (dtype == kF32) return f(float());
  if (dtype == kBF16) return f(bf16());
  return f(f16());
}

}  // namespace

size_t embedding_backward_bytes(int64_t n_ids, int64_t rows, int64_t cols) { return layout(nullptr, n_ids, rows, cols).bytes; }

hipError_t launch_embedding_forward(const EmbeddingForward& a, hipStream_t s) {
  if (a.n_ids == 0) return hipSuccess;
  return with_type(a.tdtype, [&](auto tt) {
    return with_type(a.odtype, [&](auto to) {
      using TT = decltype(tt);
      using TO = decltype(to);
      const int tpr = a.cols <= 64 ? 8 : 64;
      const int64_t units = a.n_ids * ((a.cols + 8 * tpr - 1) / (8 * tpr)), per = 256 / tpr;
      const dim3 grid(unsigned(std::min<int64_t>((units + per - 1) / per, 1 << 20))), block(256);
      const int mode = row_mode(a.cols, 8);
      if (mode == kTiny) k_embedding_forward<TT, TO, 8, kTiny><<<grid, block, 0, s>>>(a);
      else if (tpr == 8) k_embedding_forward<TT, TO, 8, kTail><<<grid, block, 0, s>>>(a);
      else if (mode == kWhole) k_embedding_forward<TT, TO, 64, kWhole><<<grid, block, 0, s>>>(a);
      else k_embedding_forward<TT, TO, 64, kTail><<<grid, block, 0, s>>>(a);
      return hipGetLastError();
    });
  });
}

hipError_t launch_embedding_backward(const EmbeddingBackward& a, hipStream_t s) {
  if (a.n_ids == 0 && a.accumulate) return hipSuccess;
  const Work w = layout(a.ws, a.n_ids, a.rows, a.cols);
  const bool one = a.n_ids <= kOneBlock;
  Clear clear{};
  const int64_t units = a.gdtype == kF32 ? 2 : 1;
  const bool large = a.rows * a.cols * units >= (int64_t(8) << 20);   // 16 MB to clear
  const int64_t few_waves = a.n_ids * ((a.cols + 64 * kSumVec - 1) / (64 * kSumVec));
  if (a.n_ids > 0 && a.n_ids <= kFew && (a.accumulate || !large) && few_waves <= kFewWaves) {
    return with_type(a.gdtype, [&](auto tg) {
      return with_type(a.dtype, [&](auto td) {
        using TG = decltype(tg);
        using TD = decltype(td);
        const int64_t waves = few_waves + (a.accumulate ? 0 : std::min<int64_t>(a.rows, 8192));
        const dim3 g(unsigned((waves + 3) / 4));
        if (a.cols < kSumVec) k_embedding_few<TD, TG, kTiny><<<g, dim3(256), 0, s>>>(a, few_waves);
        else k_embedding_few<TD, TG, kTail><<<g, dim3(256), 0, s>>>(a, few_waves);
        return hipGetLastError();
      });
    });
  }
  clear.to = static_cast<uint16_t*>(a.dtable);
  clear.row = a.cols * units;
  clear.ld = a.ldt * units;
  // The next launch's share of the rows to clear, in 20ths of all, and the
  // blocks of `threads` that clear them.  A short list's sort, sums and join
  // take about 10, 8 and 4 us, and clear in that proportion (50,257 x 1024: 53
  // us for everything with all of it in the sort's launch, 48 so); the sort's launch
  // clears named rows too, which are written again later.  (77 tokens of 1000
  // x 65: 13 us with all of it there, 18 otherwise.)  A long list names
  // much of the table: its first pass marks the rows, those of the later ones
  // clear the others.
  int64_t done = 0;
  const auto share = [&](int64_t twentieths, int64_t threads) {
    clear.first = a.accumulate ? 0 : a.rows * done / 20;
    done += twentieths;
    clear.last = a.accumulate ? 0 : a.rows * done / 20;
    const int64_t vectors = (clear.last - clear.first) * ((clear.row + 7) / 8);
    if (!clear.touched) return std::min<int64_t>((vectors + threads - 1) / threads, 1 << 20);
    return std::min<int64_t>((vectors + threads * 8 - 1) / (threads * 8), 1024 * 1024 / threads);
  };
  const bool joins = w.chunks >= 2;
  const bool later = one && w.marks && a.n_ids > 0 && large;
  const dim3 block(kSortBlock);
  if (one) {
    const dim3 g(unsigned(1 + share(!later ? 20 : joins ? 9 : 11, kSortBlock)));
    if (a.n_ids <= kSortBlock) k_embedding_sort<1><<<g, block, 0, s>>>(a, w, clear);
    else if (a.n_ids <= 4 * kSortBlock) k_embedding_sort<4><<<g, block, 0, s>>>(a, w, clear);
    else k_embedding_sort<8><<<g, block, 0, s>>>(a, w, clear);
  } else {
    // with one pass (below 256 rows) there is no later launch, and little to clear
    const int launches = w.passes == 1 ? 2 : 2 * (w.passes - 1);
    int launch = 0;
    const auto next = [&](int pass) {
      if (pass == 0 && w.passes > 1) return share(0, kSortBlock);
      ++launch;
      return share(20 * launch / launches - 20 * (launch - 1) / launches, kSortBlock);
    };
    if (w.passes > 1) clear.touched = w.touched;
    for (int pass = 0; pass < w.passes; ++pass) {
      dim3 g(unsigned(w.tiles + next(pass)));
      k_embedding_digits<<<g, block, 0, s>>>(a, w, pass, clear);
      g = dim3(unsigned(w.tiles + next(pass)));
      k_embedding_place<<<g, block, 0, s>>>(a, w, pass, clear);
    }
  }
  const hipError_t e = hipGetLastError();
  if (e != hipSuccess || a.n_ids == 0) return e;
  clear.touched = w.touched;
  return with_type(a.gdtype, [&](auto tg) {
    using TG = decltype(tg);
    with_type(a.dtype, [&](auto td) {
      using TD = decltype(td);
      constexpr int V = kSumVec;
      const int64_t slabs = (a.cols + 64 * V - 1) / (64 * V), blocks = std::min<int64_t>((w.chunks * slabs + 3) / 4, 1 << 20);
      const dim3 g(unsigned(blocks + share(!later ? 0 : joins ? 7 : 9, 256)));
      const int mode = row_mode(a.cols, V);
      if (mode == kTiny) k_embedding_sum<TD, TG, kTiny><<<g, dim3(256), 0, s>>>(a, w, blocks, clear);
      else if (mode == kWhole) k_embedding_sum<TD, TG, kWhole><<<g, dim3(256), 0, s>>>(a, w, blocks, clear);
      else k_embedding_sum<TD, TG, kTail><<<g, dim3(256), 0, s>>>(a, w, blocks, clear);
    });
    if (joins) {
      const int64_t x = (a.cols + 255) / 256, runs = std::min<int64_t>(w.chunks, 256), c = share(later ? 4 : 0, 64 * kJoinWaves);
      const dim3 g(unsigned(x), unsigned(runs + (c + x - 1) / x));
      if (a.cols < 4) k_embedding_join<TG, kTiny><<<g, dim3(64 * kJoinWaves), 0, s>>>(a, w, unsigned(runs), clear);
      else k_embedding_join<TG, kTail><<<g, dim3(64 * kJoinWaves), 0, s>>>(a, w, unsigned(runs), clear);
    }
    return hipGetLastError();
  });
}

}  // namespace lopt
