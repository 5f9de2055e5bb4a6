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

constexpr int kTile = 4096;       // tokens a block of the sort takes at a time
constexpr int kMaxTiles = 256;    // blocks of the sort
constexpr int kSortBlock = 1024;
constexpr int kPerWave = kTile / (kSortBlock / 64);   // tokens of a wave, in 64s
constexpr int kDigits = 256;      // 8 bits a pass

// Row of the table that an id names, `rows` if none.
__device__ __forceinline__ uint32_t row_of(const void* ids, int id_bytes, int64_t t, int64_t row0, int64_t rows) {
  const int64_t id = id_bytes == 8 ? static_cast<const int64_t*>(ids)[t] : int64_t(static_cast<const int32_t*>(ids)[t]);
  // row0 is within [0, 2^62], so the difference of any two of them is an int64_t
  if (id < row0) return uint32_t(rows);
  const int64_t v = id - row0;
  return uint32_t(v < rows ? v : rows);
}

// ---------------------------------------------------------------------------
// Forward: TPR threads write 8 TPR columns of one token.
template <class TT, class TO, int TPR>
__global__ __launch_bounds__(256) void k_embedding_forward(EmbeddingForward a) {
  constexpr int E = 8, V = kVec<TT> < E ? kVec<TT> : E;
  const int lane = threadIdx.x % TPR;
  const int64_t slabs = (a.cols + E * TPR - 1) / (E * TPR), units = a.n_ids * slabs;
  for (int64_t u = int64_t(blockIdx.x) * (256 / TPR) + threadIdx.x / TPR; u < units; u += int64_t(gridDim.x) * (256 / TPR)) {
    const int64_t t = slabs == 1 ? u : u / slabs;
    const int64_t c = (u - t * slabs) * (E * TPR) + lane * E;
    const uint32_t v = row_of(a.ids, a.id_bytes, t, a.row0, a.rows);
    const bool there = int64_t(v) < a.rows;
    const TT* w = static_cast<const TT*>(a.table) + (there ? int64_t(v) : 0) * a.ldt;
    Pack<TO, E> o;
#pragma unroll
    for (int k = 0; k < E / V; ++k) {
      Pack<TT, V> p{};
      if (there) p = load_pack<TT, V>(w, c + k * V, a.cols);
#pragma unroll
      for (int i = 0; i < V; ++i) o.v[k * V + i] = from_f32<TO>(there ? to_f32(p.v[i]) * a.scale : 0.f);
    }
    TO* out = static_cast<TO*>(a.out) + t * a.ldo;
    if constexpr (sizeof(TO) == 4) {
      Pack<TO, 4> h;
#pragma unroll
      for (int k = 0; k < 2; ++k) {
#pragma unroll
        for (int i = 0; i < 4; ++i) h.v[i] = o.v[4 * k + i];
        store_pack<TO, 4>(out, c + 4 * k, a.cols, h);
      }
    } else {
      store_pack<TO, E>(out, c, a.cols, o);
    }
  }
}

// ---------------------------------------------------------------------------
// Workspace of the gradient.
struct Work {
  uint32_t *key[2], *val[2];   // tokens' rows and positions, by turns
  uint32_t* hist;              // [tiles][256] digits of a pass
  unsigned char* touched;      // per row: some token names it
  float* part;                 // [chunks][2][cols]: sums of runs that cross a chunk's first / last token
  int64_t tiles, rounds, chunks;
  int32_t chunk;               // tokens of a chunk
  int32_t passes;
  size_t bytes;
};

size_t up(size_t x) { return (x + 255) / 256 * 256; }

Work layout(unsigned char* ws, int64_t n, int64_t rows, int64_t cols) {
  Work w{};
  const int64_t tiles = (n + kTile - 1) / kTile;
  w.rounds = std::max<int64_t>(1, (tiles + kMaxTiles - 1) / kMaxTiles);
  w.tiles = std::max<int64_t>(1, (tiles + w.rounds - 1) / w.rounds);
  w.chunk = n <= 16384 ? 8 : 32;
  w.chunks = (n + w.chunk - 1) / w.chunk;
  w.passes = 1;
  while (w.passes < 4 && (uint64_t(rows) >> (8 * w.passes)) != 0) ++w.passes;
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
  w.touched = take(size_t(rows));
  w.part = reinterpret_cast<float*>(take(size_t(w.chunks) * 2 * size_t(cols) * 4));
  w.bytes = at;
  return w;
}

// Digits of every tile; the first pass reads the ids and clears the row marks.
__global__ __launch_bounds__(kSortBlock) void k_embedding_digits(EmbeddingBackward a, Work w, int pass) {
  __shared__ uint32_t hist[kDigits];
  for (int d = threadIdx.x; d < kDigits; d += kSortBlock) hist[d] = 0;
  __syncthreads();
  const int64_t first = int64_t(blockIdx.x) * w.rounds * kTile, last = std::min<int64_t>(a.n_ids, first + w.rounds * kTile);
  for (int64_t t = first + threadIdx.x; t < last; t += kSortBlock) {
    const uint32_t key = pass == 0 ? row_of(a.ids, a.id_bytes, t, a.row0, a.rows) : w.key[pass & 1][t];
    atomicAdd(&hist[(key >> (8 * pass)) & 255], 1u);
  }
  __syncthreads();
  for (int d = threadIdx.x; d < kDigits; d += kSortBlock) w.hist[int64_t(blockIdx.x) * kDigits + d] = hist[d];
  if (pass == 0 && !a.accumulate)
    for (int64_t v = int64_t(blockIdx.x) * kSortBlock + threadIdx.x; v < a.rows; v += int64_t(gridDim.x) * kSortBlock)
      w.touched[v] = 0;
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

// The other lanes of the wave with this lane's digit (valid lanes only).
__device__ __forceinline__ uint64_t same_digit(uint32_t digit, bool valid) {
  uint64_t m = __ballot(valid);
#pragma unroll
  for (int b = 0; b < 8; ++b) {
    const bool bit = (digit >> b) & 1;
    const uint64_t set = __ballot(bit);
    m &= bit ? set : ~set;
  }
  return m;
}

// One stable pass: every token goes behind the tokens of lower digits and the
// earlier ones of its own.  Within a tile each wave holds 256 consecutive
// tokens, ranks them among its own (ballots), and the waves' counts are
// scanned in order.
__global__ __launch_bounds__(kSortBlock) void k_embedding_place(EmbeddingBackward a, Work w, int pass) {
  constexpr int WAVES = kSortBlock / 64, N = kPerWave / 64;
  __shared__ uint32_t count[WAVES][kDigits];
  __shared__ uint32_t base[kDigits];
  __shared__ uint32_t wave_total[4];
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;

  uint32_t total = 0, before = 0;
  if (threadIdx.x < kDigits)
    for (int64_t b = 0; b < w.tiles; ++b) {
      const uint32_t h = w.hist[b * kDigits + threadIdx.x];
      if (b < int64_t(blockIdx.x)) before += h;
      total += h;
    }
  const uint32_t start = scan_digits(total, wave_total);
  if (threadIdx.x < kDigits) base[threadIdx.x] = start + before;

  for (int64_t round = 0; round < w.rounds; ++round) {
    const int64_t tile = (int64_t(blockIdx.x) * w.rounds + round) * kTile;
    for (int d = threadIdx.x; d < WAVES * kDigits; d += kSortBlock) (&count[0][0])[d] = 0;
    __syncthreads();
    uint32_t key[N], val[N], rank[N];
#pragma unroll
    for (int j = 0; j < N; ++j) {
      const int64_t t = tile + wave * kPerWave + j * 64 + lane;
      const bool valid = t < a.n_ids;
      key[j] = 0;
      val[j] = uint32_t(t);
      if (valid) {
        if (pass == 0) {
          key[j] = row_of(a.ids, a.id_bytes, t, a.row0, a.rows);
          if (!a.accumulate && int64_t(key[j]) < a.rows) w.touched[key[j]] = 1;
        } else {
          key[j] = w.key[pass & 1][t];
          val[j] = w.val[pass & 1][t];
        }
      }
      const uint32_t digit = (key[j] >> (8 * pass)) & 255;
      const uint64_t same = same_digit(digit, valid), lower = same & ((uint64_t(1) << lane) - 1);
      rank[j] = 0;
      if (valid) {
        rank[j] = count[wave][digit] + __popcll(lower);
      }
      // the wave's reads of its counts come before its writes, and those before the next round's reads
      __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
      __builtin_amdgcn_wave_barrier();
      if (valid && lower == 0) count[wave][digit] += __popcll(same);
      __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
      __builtin_amdgcn_wave_barrier();
    }
    __syncthreads();
    if (threadIdx.x < kDigits) {
      uint32_t at = base[threadIdx.x];
#pragma unroll
      for (int k = 0; k < WAVES; ++k) {
        const uint32_t c = count[k][threadIdx.x];
        count[k][threadIdx.x] = at;
        at += c;
      }
      base[threadIdx.x] = at;
    }
    __syncthreads();
#pragma unroll
    for (int j = 0; j < N; ++j) {
      const int64_t t = tile + wave * kPerWave + j * 64 + lane;
      if (t < a.n_ids) {
        const uint32_t to = count[wave][(key[j] >> (8 * pass)) & 255] + rank[j];
        w.key[(pass + 1) & 1][to] = key[j];
        w.val[(pass + 1) & 1][to] = val[j];
      }
    }
    __syncthreads();
  }
}

template <class TG>
__device__ __forceinline__ void store_row(const EmbeddingBackward& a, uint32_t v, int64_t c, const float* x, int n) {
  TG* to = static_cast<TG*>(a.dtable) + int64_t(v) * a.ldt;
  constexpr int V = 4;
  for (int k = 0; k < n; k += V) {
    Pack<TG, V> p{};
    if (a.accumulate) p = load_pack<TG, V>(to, c + k, a.cols);
#pragma unroll
    for (int i = 0; i < V; ++i) p.v[i] = from_f32<TG>(to_f32(p.v[i]) + x[k + i] * a.scale);
    store_pack<TG, V>(to, c + k, a.cols, p);
  }
}

// One chunk of sorted tokens over one slab of columns (this lane's from c).
template <class TD, class TG>
__device__ __forceinline__ void sum_chunk(const EmbeddingBackward& a, const Work& w, int64_t chunk, int64_t c) {
  constexpr int V = kVec<TD>, U = 8;
  const int lane = threadIdx.x & 63;
  const uint32_t* skey = w.key[w.passes & 1];
  const uint32_t* sval = w.val[w.passes & 1];
  const uint32_t none = uint32_t(a.rows);
  const int64_t p0 = chunk * w.chunk, p1 = std::min<int64_t>(a.n_ids, p0 + w.chunk);
  const int n = int(p1 - p0);
  uint32_t lane_key = none, lane_val = 0;
  if (lane < n) {
    lane_key = skey[p0 + lane];
    lane_val = sval[p0 + lane];
  }
  const uint32_t prev = p0 > 0 ? skey[p0 - 1] : none, next = p1 < a.n_ids ? skey[p1] : none;
  uint32_t cur = __builtin_amdgcn_readlane(lane_key, 0);
  bool inside = cur != prev;   // the run began in this chunk
  float acc[V] = {};
  float* part = w.part + size_t(chunk) * 2 * size_t(a.cols);
  for (int i0 = 0; i0 < n; i0 += U) {
    Pack<TD, V> p[U];
#pragma unroll
    for (int j = 0; j < U; ++j) {
      const uint32_t k = __builtin_amdgcn_readlane(lane_key, i0 + j < 64 ? i0 + j : 63);
      const uint32_t t = __builtin_amdgcn_readlane(lane_val, i0 + j < 64 ? i0 + j : 63);
      p[j] = Pack<TD, V>{};
      if (i0 + j < n && k != none && c < a.cols) p[j] = load_pack<TD, V>(static_cast<const TD*>(a.dout) + int64_t(t) * a.ldd, c, a.cols);
    }
#pragma unroll
    for (int j = 0; j < U; ++j) {
      if (i0 + j >= n) break;
      const uint32_t k = __builtin_amdgcn_readlane(lane_key, i0 + j);
      if (k != cur) {
        if (c < a.cols) {
          if (inside) store_row<TG>(a, cur, c, acc, V);
          else
#pragma unroll
            for (int i = 0; i < V; ++i)
              if (c + i < a.cols) part[c + i] = acc[i];
        }
        inside = true;
        cur = k;
#pragma unroll
        for (int i = 0; i < V; ++i) acc[i] = 0.f;
      }
#pragma unroll
      for (int i = 0; i < V; ++i) acc[i] += to_f32(p[j].v[i]);
    }
  }
  if (cur == none || c >= a.cols) return;
  if (inside && cur != next) {
    store_row<TG>(a, cur, c, acc, V);
  } else {
    if (inside) part += a.cols;
#pragma unroll
    for (int i = 0; i < V; ++i)
      if (c + i < a.cols) part[c + i] = acc[i];
  }
}

// Sums of the sorted tokens: a wave takes `chunk` of them in order over 64
// 16-byte vectors of columns, and writes a row where its run of equal keys
// ends.  A run that crosses the chunk's border leaves its sum in the
// workspace: slot 0 if it began before the chunk, slot 1 if it began in it.
// Blocks behind those clear the rows that no token names.
template <class TD, class TG>
__global__ __launch_bounds__(256) void k_embedding_sum(EmbeddingBackward a, Work w, int64_t sum_blocks) {
  constexpr int V = kVec<TD>;
  const int lane = threadIdx.x & 63;
  if (int64_t(blockIdx.x) >= sum_blocks) {
    // rows that no token names, one wave a row
    const int64_t waves = (int64_t(gridDim.x) - sum_blocks) * 4;
    for (int64_t v = (int64_t(blockIdx.x) - sum_blocks) * 4 + (threadIdx.x >> 6); v < a.rows; v += waves) {
      if (w.touched[v]) continue;
      TG* to = static_cast<TG*>(a.dtable) + v * a.ldt;
      constexpr int VG = kVec<TG>;
      const Pack<TG, VG> zero{};
      for (int64_t c = lane * VG; c < a.cols; c += 64 * VG) store_pack<TG, VG>(to, c, a.cols, zero);
    }
    return;
  }
  const int64_t slabs = (a.cols + 64 * V - 1) / (64 * V), units = w.chunks * slabs;
  for (int64_t unit = int64_t(blockIdx.x) * 4 + (threadIdx.x >> 6); unit < units; unit += sum_blocks * 4)
    sum_chunk<TD, TG>(a, w, unit / slabs, unit % slabs * (64 * V) + lane * V);
}

// The run of equal keys that begins in `chunk` and goes on behind it, if there is one.
template <class TG>
__device__ __forceinline__ void join_run(const EmbeddingBackward& a, const Work& w, float (&quarter)[4][256], int64_t chunk,
                                         int64_t c0) {
  const uint32_t* skey = w.key[w.passes & 1];
  const int64_t p0 = chunk * w.chunk, p1 = p0 + w.chunk;
  if (p1 >= a.n_ids) return;                       // the last chunk: nothing behind it
  const uint32_t key = skey[p1 - 1];
  if (key == uint32_t(a.rows) || skey[p1] != key) return;
  if (p0 > 0 && skey[p0] == key && skey[p0 - 1] == key) return;   // began before this chunk
  // chunks behind this one whose first token belongs to the run
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  int64_t last = chunk;
  for (int64_t step = 4096; step >= 1; step /= 64) {
    int cnt;
    do {
      const int64_t j = last + (lane + 1) * step;
      const uint64_t ok = __ballot(j < w.chunks && skey[j * w.chunk] == key);
      cnt = ok == ~uint64_t(0) ? 64 : __builtin_ctzll(~ok);
      last += cnt * step;
    } while (cnt == 64);
  }
  const int64_t m = last - chunk + 1, q = (m + 3) / 4;
  const int64_t b = std::min<int64_t>(m, wave * q), e = std::min<int64_t>(m, b + q);
  const int64_t c = c0 + lane * 4;
  float acc[4] = {};
  if (c < a.cols) {
#pragma unroll 4
    for (int64_t j = b; j < e; ++j) {
      const float* part = w.part + (size_t(chunk + j) * 2 + (j == 0 ? 1 : 0)) * size_t(a.cols);
      const Pack<float, 4> p = load_pack<float, 4>(part, c, a.cols);
#pragma unroll
      for (int i = 0; i < 4; ++i) acc[i] += p.v[i];
    }
  }
#pragma unroll
  for (int i = 0; i < 4; ++i) quarter[wave][lane * 4 + i] = acc[i];
  __syncthreads();
  if (wave != 0 || c >= a.cols) return;
#pragma unroll
  for (int k = 1; k < 4; ++k)
#pragma unroll
    for (int i = 0; i < 4; ++i) acc[i] += quarter[k][lane * 4 + i];
  store_row<TG>(a, key, c, acc, 4);
}

// Rows whose run crosses chunks: the block of the chunk where the run begins
// adds up the chunks' sums, four waves a quarter each, the quarters in order.
template <class TG>
__global__ __launch_bounds__(256) void k_embedding_join(EmbeddingBackward a, Work w) {
  __shared__ float quarter[4][256];
  const int64_t slabs = (a.cols + 255) / 256, units = w.chunks * slabs;
  for (int64_t u = blockIdx.x; u < units; u += gridDim.x) {
    join_run<TG>(a, w, quarter, u / slabs, u % slabs * 256);
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
      if (tpr == 8) k_embedding_forward<TT, TO, 8><<<grid, block, 0, s>>>(a);
      else k_embedding_forward<TT, TO, 64><<<grid, block, 0, s>>>(a);
      return hipGetLastError();
    });
  });
}

hipError_t launch_embedding_backward(const EmbeddingBackward& a, hipStream_t s) {
  if (a.n_ids == 0 && a.accumulate) return hipSuccess;
  const Work w = layout(a.ws, a.n_ids, a.rows, a.cols);
  for (int pass = 0; pass < w.passes; ++pass) {
    k_embedding_digits<<<dim3(unsigned(w.tiles)), dim3(kSortBlock), 0, s>>>(a, w, pass);
    k_embedding_place<<<dim3(unsigned(w.tiles)), dim3(kSortBlock), 0, s>>>(a, w, pass);
  }
  hipError_t e = hipGetLastError();
  if (e != hipSuccess) return e;
  return with_type(a.gdtype, [&](auto tg) {
    using TG = decltype(tg);
    const hipError_t e2 = with_type(a.dtype, [&](auto td) {
      using TD = decltype(td);
      const int64_t slabs = (a.cols + 64 * kVec<TD> - 1) / (64 * kVec<TD>);
      const int64_t sum_blocks = std::min<int64_t>((w.chunks * slabs + 3) / 4, 1 << 20);
      const int64_t zero_blocks = a.accumulate ? 0 : std::min<int64_t>((a.rows + 3) / 4, 8192);
      if (sum_blocks + zero_blocks == 0) return hipSuccess;
      k_embedding_sum<TD, TG><<<dim3(unsigned(sum_blocks + zero_blocks)), dim3(256), 0, s>>>(a, w, sum_blocks);
      return hipGetLastError();
    });
    if (e2 != hipSuccess || w.chunks < 2) return e2;
    k_embedding_join<TG><<<dim3(unsigned(std::min<int64_t>(w.chunks * ((a.cols + 255) / 256), 1 << 20))), dim3(256), 0, s>>>(a, w);
    return hipGetLastError();
  });
}

}  // namespace lopt
