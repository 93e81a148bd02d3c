// embed_kernels.hip -- embedding lookup with scaling, and the table's
// gradient from tokens sorted by id, for gfx950.
//
//   out[t]     = round(scale * weight[key_t])          zero where t has no key
//   dweight[v] = round(scale * sum_{t: key_t = v} dout[t])
//
// Both are bound by memory.  The gradient never adds with atomics: the ids are
// sorted (stable), the sorted list is cut into chunks of C tokens, and a wave
// sums one chunk's rows over 64 vectors of columns, writing each run of equal
// keys that lies inside the chunk straight to its row.  A run that crosses a
// chunk's edge leaves fp32 partials, which a second launch adds in order; so
// a token that fills half the batch is spread over as many waves as its
// chunks.  Rows without a token are zeroed beside all of that: the table's
// first rows beside the sort's launches, the others by further workgroups of
// the sum and join launches, which look their rows up in the sorted list.
//
// Measured: the lookup of 30,011 x 4096 bf16, a quarter of them in the table,
// 41 us (246 MB written, 37 read, 6.9 TB/s); the gradient of 32,768 x 2048 bf16 into
// 100,003 fp32 rows 194 us, of which the sort 24 (41 with 200 MB zeroed
// beside it): 1.0 GB in all, 0.85 of it written, 5.2 TB/s, as a large copy
// does.  Its parts alone: the sums 60-75 us, all the zeroing 117 us.
#include "key_sort.hpp"
#include "launch.hpp"

namespace hc {
namespace {

constexpr uint32_t kMaxBlocks = 1u << 22;

inline uint32_t blocks_for(uint64_t waves) {
  const uint64_t b = (waves + kWaves - 1) / kWaves;
  return (uint32_t)(b < kMaxBlocks ? b : kMaxBlocks);
}

// ---------------------------------------------------------------- lookup

// A wave handles 64 >> lg rows of 1 << lg vectors (lg < 6: narrow tables), or
// a slice of U * 64 vectors of one row (lg == 6).  Plain loads: a frequent
// token's row comes out of the cache (non-temporal ones 56 against 41 us).
template <typename T, int U, bool NT>
__global__ void __launch_bounds__(kThreads) embedding_kernel(KeySource src, size_t ntokens, const void* weight,
                                                             uint32_t dim, size_t wstride, float scale, void* out,
                                                             size_t ostride, uint32_t lg, uint32_t slices,
                                                             uint64_t units) {
  const uint32_t nvec = (dim + T::kVec - 1) / T::kVec;
  const uint32_t sub = lane_id() >> lg, at = lane_id() & ((1u << lg) - 1);
  for (uint64_t u = (uint64_t)blockIdx.x * kWaves + wave_id(); u < units; u += (uint64_t)gridDim.x * kWaves) {
    const size_t t = u / slices * (64u >> lg) + sub;
    const uint32_t v0 = (uint32_t)(u % slices) * (64 * U) + at;
    if (t >= ntokens) continue;
    const uint32_t key = load_key(src, t);
    typename T::vec x[U];
#pragma unroll
    for (int i = 0; i < U; ++i) {
      const uint32_t v = v0 + 64 * i;
      x[i] = zero_vec<T>();
      if (key != kNoKey && v < nvec)
        x[i] = load_vec<T>(elem<T>(weight, (size_t)key * wstride + vec_at<T>(v * T::kVec, dim)));
    }
#pragma unroll
    for (int i = 0; i < U; ++i) {
      const uint32_t v = v0 + 64 * i;
      if (v >= nvec) continue;
      float f[T::kVec];
      T::unpack(x[i], f);
#pragma unroll
      for (int j = 0; j < T::kVec; ++j) f[j] *= scale;
      store_vec<T, NT>(elem<T>(out, t * ostride + vec_at<T>(v * T::kVec, dim)),
                       key == kNoKey ? zero_vec<T>() : T::pack(f));
    }
  }
}

// ---------------------------------------------------------------- zeroing beside the sort

// The sort's launches occupy a quarter of the GPU for a few microseconds each
// and depend on nothing but the ids; the other compute units meanwhile zero
// the first rows of the table, tokens or not (the sums come later and write
// theirs again).  Pieces of some 64 KB: of one flat range where the rows are
// contiguous, else whole rows, a wave to each; a row wider than that is a piece
// by itself (500 x 65,536 bf16 into 600 fp32 rows: 75 us contiguous, 86 apart).
// A launch of the sort takes 2-3 us longer for 25 MB of them and 5 us for 50 MB,
// which alone would take 8 (2000 tokens x 1000 fp32 into 10,007 rows, 40 MB:
// 23.4 us without, 18.3 with).
constexpr uint64_t kPieceBytes = 65536;

struct ZeroJob {
  char* base = nullptr;
  uint64_t row_bytes = 0, stride = 0;   // flat: one row of all
  uint64_t rows = 0, rows_per_piece = 0;
  uint64_t pieces = 0, done = 0;
  bool flat = false;
  bool stream = false;                  // non-temporal
};

template <bool NT>
__device__ __forceinline__ void zero_piece(const ZeroJob& z, uint64_t piece) {
  if (z.flat) {
    const uint64_t at = piece * kPieceBytes;
    zero_span<NT>(z.base + at, z.row_bytes - at < kPieceBytes ? z.row_bytes - at : kPieceBytes, threadIdx.x,
                  kSortThreads);
    return;
  }
  const uint64_t r0 = piece * z.rows_per_piece;
  for (uint64_t r = r0 + wave_id(); r < z.rows && r < r0 + z.rows_per_piece; r += kSortWaves)
    zero_span<NT>(z.base + r * z.stride, z.row_bytes, lane_id(), 64);
}
__device__ __forceinline__ void zero_piece(const ZeroJob& z, uint64_t piece) {
  if (z.stream)
    zero_piece<true>(z, piece);
  else
    zero_piece<false>(z, piece);
}

// ---------------------------------------------------------------- sorting the ids

// Ids up to this many are sorted in one launch: a workgroup places kRankIds of
// them, each of its waves comparing them with a sixteenth of all ids, a quarter
// of that sixteenth per 16 lanes.  n^2 comparisons, 3 instructions each, spread
// over all compute units, beat the launches of a radix sort while n is small.
// The whole gradient of n x 256 bf16, us, so / by digits: into 20,000 rows (two
// digits) 8000 tokens 22.7 / 28.3, 10,000 32.6 / 30.3; into 500 rows (one) 6000
// tokens 19.4 / 18.7.  With 64 ids a workgroup 4096 tokens took 17.9, not 15.3.
constexpr uint32_t kRankMax = 8192;
constexpr uint32_t kRankIds = 16;
inline bool by_rank(size_t n, size_t nkeys) { return n <= (nkeys <= kMaxRadix ? kRankMax / 2 : kRankMax); }

__global__ void __launch_bounds__(kSortThreads) rank_kernel(KeySource src, uint32_t n, uint32_t* keys, uint32_t* pos,
                                                            uint32_t groups, ZeroJob zero) {
  if (blockIdx.x >= groups) {
    zero_piece(zero, zero.done + blockIdx.x - groups);
    return;
  }
  __shared__ __attribute__((aligned(16))) uint32_t all[kRankMax];
  __shared__ uint32_t part[kSortWaves][kRankIds];
  const uint32_t padded = (n + 255) & ~255u;
  for (uint32_t i = threadIdx.x; i < padded; i += kSortThreads) {
    const uint32_t k = i < n ? load_key(src, i) : kNoKey;
    all[i] = k < src.nkeys ? k : src.nkeys;     // no key sorts last
  }
  __syncthreads();
  const uint32_t g0 = blockIdx.x * kRankIds, i = g0 + lane_id() % kRankIds;
  const uint32_t key = all[i];
  const uint32_t share = padded / (kSortWaves * 4);     // a multiple of 4
  const uint32_t lo = (wave_id() * 4 + lane_id() / kRankIds) * share;
  uint32_t c = 0;
#pragma unroll 4
  for (uint32_t j = lo; j < lo + share; j += 4) {
    const vec4 k = *reinterpret_cast<const vec4*>(&all[j]);
    const uint32_t below = key + (j < g0 ? 1 : 0);      // of earlier ids, equal ones come first too
    const uint32_t four = (k[0] < below) + (k[1] < below) + (k[2] < below) + (k[3] < below);
    c += j - g0 < kRankIds ? 0 : four;                  // the group's own: below
  }
  c += __shfl_xor(c, 16);
  c += __shfl_xor(c, 32);
  if (lane_id() < kRankIds) part[threadIdx.x >> 6][lane_id()] = c;
  __syncthreads();
  if (threadIdx.x < kRankIds && i < n) {
    uint32_t r = 0;
    for (uint32_t w = 0; w < kSortWaves; ++w) r += part[w][threadIdx.x];
#pragma unroll
    for (uint32_t q = 0; q < kRankIds; ++q) r += all[g0 + q] < key + (g0 + q < i ? 1 : 0);
    if (r < n) {
      keys[r] = key < src.nkeys ? key : kNoKey;
      pos[r] = i;
    }
  }
}

// One digit of a least-significant-digit radix sort.  The first pass reads
// the ids, later ones the pairs that the pass before wrote.
struct Pass {
  KeySource src;
  const uint32_t* keys;     // NULL: the ids of src
  const uint32_t* pos;
  uint32_t n, tile, tiles, shift, bits;
  uint32_t* hist;
  uint32_t* keys_out;
  uint32_t* pos_out;
};

__device__ __forceinline__ uint32_t pass_digit(const Pass& p, size_t i) {
  const uint32_t k = p.keys ? p.keys[i] : load_key(p.src, i);
  return k == kNoKey ? kNoKey : (k >> p.shift) & ((1u << p.bits) - 1);
}

__global__ void __launch_bounds__(kSortThreads) pass_histogram_kernel(Pass p, ZeroJob zero) {
  if (blockIdx.x >= p.tiles) {
    zero_piece(zero, zero.done + blockIdx.x - p.tiles);
    return;
  }
  __shared__ uint32_t lds[kMaxRadix];
  const uint32_t radix = 1u << p.bits;
  const size_t lo = (size_t)blockIdx.x * p.tile;
  const size_t hi = lo + p.tile < p.n ? lo + p.tile : p.n;
  tile_histogram(lds, radix, lo, hi, [&](size_t i) { return pass_digit(p, i); }, p.hist + (size_t)blockIdx.x * radix);
}

__global__ void __launch_bounds__(kSortThreads) pass_scatter_kernel(Pass p, ZeroJob zero) {
  if (blockIdx.x >= p.tiles) {
    zero_piece(zero, zero.done + blockIdx.x - p.tiles);
    return;
  }
  __shared__ uint32_t counts[kSortWaves * kMaxRadix];
  __shared__ uint32_t scan[kSortWaves];
  const uint32_t radix = 1u << p.bits;
  const size_t lo = (size_t)blockIdx.x * p.tile;
  const size_t hi = lo + p.tile < p.n ? lo + p.tile : p.n;
  auto digit = [&](size_t i) { return pass_digit(p, i); };
  const Run run = load_run(lo, hi, p.tile, digit);
  uint32_t before, total, all;
  tile_sums(p.hist, radix, p.tiles, blockIdx.x, threadIdx.x, &before, &total);
  const uint32_t first = block_scan(total, scan, &all);
  place_items(counts, radix, p.bits, run, first + before, digit,
              [&](size_t i, uint32_t d, uint32_t place) {
                if (d != kNoKey && place < p.n) {
                  p.keys_out[place] = p.keys ? p.keys[i] : load_key(p.src, i);
                  p.pos_out[place] = p.pos ? p.pos[i] : (uint32_t)i;
                }
                if (i >= all) {       // behind the last id with a key
                  p.keys_out[i] = kNoKey;
                  p.pos_out[i] = 0;
                }
              });
}

}  // namespace

constexpr size_t kHistBytes = (size_t)kMaxTiles * kMaxRadix * sizeof(uint32_t);

// Of any number of keys: fewer of them may take a longer sort.
size_t sort_ids_ws_bytes(size_t n) {
  return by_rank(n, 1) ? 0 : kHistBytes + (2 * n * sizeof(uint32_t) + 15) / 16 * 16;
}

namespace {

// Pieces that a launch of the sort zeroes beside it, 50 MB (more where rows that
// lie apart are wider than a piece: 200 MB of 256 KB rows).  The gradient with
// 25, 50, 100 and 200 MB a launch, us: 32,768 x 2048 bf16 into 100,003 fp32 rows
// 202, 196, 198 and 228; 16,000 into 40,000 rows 92, 92, 106 and 113; placed by one
// launch, 8000 into 128,000 rows 210, 210, 212 and 213, 500 into 30,000 47, 47, 49
// and 54, 2000 into 40,000 65, 63, 65 and 68.
constexpr uint64_t kPiecesBeside = 768;

hipError_t sort_ids(const KeySource& src, size_t n, uint32_t* keys, uint32_t* pos, void* ws, ZeroJob* zero,
                    hipStream_t stream) {
  if (n == 0) return hipSuccess;
  uint32_t beside = 0;
  auto next = [&] {
    zero->done += beside;
    beside = (uint32_t)(zero->pieces - zero->done < kPiecesBeside ? zero->pieces - zero->done : kPiecesBeside);
  };
  if (by_rank(n, src.nkeys)) {
    const uint32_t groups = (uint32_t)((n + kRankIds - 1) / kRankIds);
    next();
    HC_ENQUEUE(rank_kernel, groups + beside, kSortThreads, stream, src, (uint32_t)n, keys, pos, groups, *zero);
    zero->done += beside;
    return hipSuccess;
  }
  uint32_t bits = 1;
  while (bits < 32 && ((uint64_t)src.nkeys - 1) >> bits) ++bits;
  const uint32_t passes = (bits + 9) / 10, per = (bits + passes - 1) / passes;
  uint32_t* hist = static_cast<uint32_t*>(ws);
  uint32_t* tmp_keys = hist + (size_t)kMaxTiles * kMaxRadix;
  uint32_t* tmp_pos = tmp_keys + n;
  Pass p = {src, nullptr, nullptr, (uint32_t)n, sort_tile(n), sort_tiles(n), 0, per, hist, nullptr, nullptr};
  for (uint32_t k = 0; k < passes; ++k) {
    const bool last_buffer = ((passes - 1 - k) & 1) == 0;   // the last pass ends in keys/pos
    p.shift = k * per;
    p.bits = per;
    p.keys_out = last_buffer ? keys : tmp_keys;
    p.pos_out = last_buffer ? pos : tmp_pos;
    next();
    HC_ENQUEUE(pass_histogram_kernel, p.tiles + beside, kSortThreads, stream, p, *zero);
    next();
    HC_ENQUEUE(pass_scatter_kernel, p.tiles + beside, kSortThreads, stream, p, *zero);
    p.keys = p.keys_out;
    p.pos = p.pos_out;
  }
  zero->done += beside;
  return hipSuccess;
}

}  // namespace

// ---------------------------------------------------------------- the gradient

namespace {

constexpr size_t kZeroBytes = 32768;    // of table rows per zeroing workgroup, 4 to 64 rows
                                        // (64 and 128 KB: 1-3% slower)
constexpr uint32_t kJoinCols = 256;     // columns per workgroup and round of the join: 4 fp32 per lane

struct Grad {
  const uint32_t* keys;     // sorted
  const uint32_t* pos;
  uint32_t n, chunk, nchunks, dim, slices;
  uint32_t vocab;
  const void* dout;
  size_t dstride;
  float scale;
  void* dweight;
  size_t wstride;
  float* partial;           // [chunk][2][pstride]: a run that began before the chunk; one that goes on after it
  uint32_t pstride;
  uint32_t join_chunks;
  uint32_t zero_from;       // rows before it are zero already
  uint32_t zero_rows;       // table rows per zeroing workgroup
  bool zero_stream;         // zeroed non-temporal
  uint64_t sum_units;
};

// Writes N columns of a table row from `at` on; the first `skip` of them
// belong to another lane, which has the same sums for them: written all the
// same, unless the table's own values are added: that goes by elements, which
// is slow (32,768 x 2048 bf16 into 100,003 fp32 rows 286 us, where overwriting takes
// 196 and these rows read and written, 592 MB, some 114).
template <typename To, int N, bool ACC>
__device__ __forceinline__ void write_row(const Grad& g, uint32_t row, uint32_t at, uint32_t skip, const float* sum) {
  typename To::raw* p = elem<To>(g.dweight, (size_t)row * g.wstride + at);
  float f[N];
#pragma unroll
  for (int i = 0; i < N; ++i) f[i] = sum[i] * g.scale;
  if constexpr (ACC) {
#pragma unroll
    for (int i = 0; i < N; ++i)
      if ((uint32_t)i >= skip) p[i] = To::narrow(To::widen(p[i]) + f[i]);
  } else {
    store_vals<To, N>(p, f);
  }
}

template <typename Ti, typename To, bool ACC>
__device__ __forceinline__ void sum_chunk(const Grad& g, uint32_t c, uint32_t slice) {
  constexpr int N = Ti::kVec, U = 8;
  const uint32_t lane = lane_id();
  const uint32_t p0 = c * g.chunk;
  const uint32_t cnt = g.n - p0 < g.chunk ? g.n - p0 : g.chunk;
  const uint32_t key = lane < cnt ? g.keys[p0 + lane] : kNoKey;
  const uint32_t pos = lane < cnt ? g.pos[p0 + lane] : 0;
  const uint32_t prev = p0 ? g.keys[p0 - 1] : kNoKey;
  const uint32_t next = p0 + cnt < g.n ? g.keys[p0 + cnt] : kNoKey;
  const uint32_t live = (uint32_t)__popcll(__ballot(key != kNoKey));    // the keys come first
  if (!live) return;
  uint32_t after = __shfl_down(key, 1);
  if (lane == cnt - 1) after = next;
  const uint64_t ends = __ballot(lane < live && (key != after || lane == live - 1));
  const bool head = first_lane_read(key) == first_lane_read(prev);
  const bool tail = lane_read(key, live - 1) == lane_read(after, live - 1);
  const uint32_t col = slice * 64 * N + lane * N, at = vec_at<Ti>(col, g.dim);
  const bool mine = col < g.dim;
  float acc[N];
#pragma unroll
  for (int j = 0; j < N; ++j) acc[j] = 0.0f;
  bool first_run = true;
  for (uint32_t i = 0; i < live; i += U) {
    typename Ti::vec x[U];
#pragma unroll
    for (int u = 0; u < U; ++u) {
      x[u] = zero_vec<Ti>();
      if (i + u < live) {
        const uint32_t row = lane_read(pos, i + u);
        if (mine) x[u] = load_vec<Ti>(elem<Ti>(g.dout, (size_t)row * g.dstride + at));
      }
    }
#pragma unroll
    for (int u = 0; u < U; ++u) {
      if (i + u >= live) break;
      float f[N];
      Ti::unpack(x[u], f);
#pragma unroll
      for (int j = 0; j < N; ++j) acc[j] += f[j];
      if (!((ends >> (i + u)) & 1)) continue;
      const bool from_before = first_run && head;
      const bool goes_on = i + u == live - 1 && tail;
      first_run = false;
      const uint32_t table_row = lane_read(key, i + u);
      if (mine) {
        if (from_before || goes_on)
          store_vals<F32, N>(elem<F32>(g.partial, ((size_t)c * 2 + (from_before ? 0 : 1)) * g.pstride + at), acc);
        else
          write_row<To, N, ACC>(g, table_row, at, col - at, acc);
      }
#pragma unroll
      for (int j = 0; j < N; ++j) acc[j] = 0.0f;
    }
  }
}

// The first place in the sorted list whose key is not below v: 64 places are
// compared at a time, so three loads in turn search 2^18 tokens.
__device__ __forceinline__ uint32_t lower_bound(const uint32_t* keys, uint32_t n, uint32_t v) {
  uint32_t lo = 0;
  while (n) {
    const uint32_t step = (n + 63) / 64, at = lane_id() * step;
    const uint32_t below = (uint32_t)__popcll(__ballot(at < n && keys[lo + at] < v));
    if (!below) break;
    const uint32_t skip = (below - 1) * step + 1;     // the last place below v, and it
    const uint32_t rest = n - skip;
    lo += skip;
    n = rest < step - 1 ? rest : step - 1;
  }
  return lo;
}

// Which of the rows [v0, v0 + count) have tokens, count <= 64.
__device__ __forceinline__ uint64_t rows_with_tokens(const Grad& g, uint32_t v0, uint32_t count) {
  uint64_t found = 0;
  uint32_t p = lower_bound(g.keys, g.n, v0);
  for (;;) {
    const uint32_t key = p + lane_id() < g.n ? g.keys[p + lane_id()] : kNoKey;
    const uint32_t r = key - v0;
    uint64_t mine = key != kNoKey && r < count ? 1ull << r : 0;
#pragma unroll
    for (int m = 32; m; m >>= 1) mine |= __shfl_xor(mine, m);
    found |= mine;
    const uint32_t last = lane_read(key, 63);
    if (last == kNoKey || last - v0 >= count - 1) return found;
    p = lower_bound(g.keys, g.n, last + 1);           // past the run that fills the rest
  }
}

// A workgroup zeroes those of its rows that no token has: a row at a time, or
// several where a row is less than a wave's vectors.
template <typename To, bool NT>
__device__ __forceinline__ void zero_rows(const Grad& g, uint32_t v0) {
  const uint32_t count = g.vocab - v0 < g.zero_rows ? g.vocab - v0 : g.zero_rows;
  const uint64_t all = count < 64 ? (1ull << count) - 1 : ~0ull;
  uint64_t absent = all & ~rows_with_tokens(g, v0, count);
  const uint64_t bytes = (uint64_t)g.dim * sizeof(typename To::raw), nvec = (bytes + 15) / 16;
  auto row = [&](uint32_t k) { return reinterpret_cast<char*>(elem<To>(g.dweight, (size_t)(v0 + k) * g.wstride)); };
  if (nvec > 64) {
    while (absent) {
      const uint32_t k = (uint32_t)__builtin_ctzll(absent);
      absent &= absent - 1;
      zero_span<NT>(row(k), bytes, threadIdx.x, kThreads);
    }
    return;
  }
  const uint32_t lanes = nvec == 1 ? 8 : 1u << (32 - __builtin_clz((uint32_t)nvec - 1));   // of a row
  for (uint32_t k = threadIdx.x / lanes; k < count; k += kThreads / lanes)
    if (absent >> k & 1) zero_span<NT>(row(k), bytes, threadIdx.x % lanes, lanes);
}
template <typename To>
__device__ __forceinline__ void zero_rows(const Grad& g, uint32_t v0) {
  if (g.zero_stream)
    zero_rows<To, true>(g, v0);
  else
    zero_rows<To, false>(g, v0);
}

template <typename Ti, typename To, bool ACC>
__global__ void __launch_bounds__(kThreads) grad_kernel(Grad g, uint32_t sum_blocks, uint32_t zero_blocks) {
  for (uint64_t b = blockIdx.x; b < (uint64_t)sum_blocks + zero_blocks; b += gridDim.x) {
    if (b < sum_blocks) {
      const uint64_t u = b * kWaves + wave_id();
      if (u < g.sum_units) sum_chunk<Ti, To, ACC>(g, (uint32_t)(u / g.slices), (uint32_t)(u % g.slices));
    } else if constexpr (!ACC) {
      zero_rows<To>(g, g.zero_from + (uint32_t)(b - sum_blocks) * g.zero_rows);
    }
  }
}

// Adds the partials of the runs that cross chunk edges.  The chunk in which
// such a run begins owns it.  A workgroup looks at join_chunks (<= 8) chunks at
// once, one per lane, since most own none in a large batch; for one that does,
// its 4 waves take every fourth of the chunks that follow, and wave 0 adds the
// four sums in order.

template <typename To, bool ACC>
__device__ __forceinline__ void join_runs(const Grad& g, uint32_t group, uint32_t col_block, uint32_t col_blocks) {
  __shared__ float lds[kWaves][kJoinCols];
  const uint32_t lane = lane_id(), w = wave_id();
  const uint32_t mine = group * g.join_chunks + lane;
  uint32_t key = kNoKey;
  bool owner = false;
  if (lane < g.join_chunks && mine + 1 < g.nchunks) {
    const uint32_t p0 = mine * g.chunk, p1 = p0 + g.chunk;
    key = g.keys[p1 - 1];
    owner = key != kNoKey && g.keys[p1] == key && !(p0 && g.keys[p0] == key && g.keys[p0 - 1] == key);
  }
  uint64_t owners = __ballot(owner);
  while (owners) {
    const uint32_t at = (uint32_t)__builtin_ctzll(owners);
    owners &= owners - 1;
    const uint32_t c = group * g.join_chunks + at, row = lane_read(key, at);
    uint32_t more = 0;     // chunks after c that begin inside the run
    for (;;) {
      const uint32_t k = c + 1 + more + lane;
      const uint64_t same = __ballot(k < g.nchunks && g.keys[(size_t)k * g.chunk] == row);
      const uint32_t run = ~same ? (uint32_t)__builtin_ctzll(~same) : 64u;
      more += run;
      if (run < 64) break;
    }
    for (uint32_t c0 = col_block * kJoinCols; c0 < g.dim; c0 += col_blocks * kJoinCols) {
      const uint32_t col = c0 + lane * 4;
      float acc[4] = {0, 0, 0, 0};
      if (col < g.dim) {
#pragma unroll 8
        for (uint32_t i = w; i < more; i += kWaves) {
          const vec4 p = *reinterpret_cast<const vec4*>(g.partial + (size_t)(c + 1 + i) * 2 * g.pstride + col);
#pragma unroll
          for (int j = 0; j < 4; ++j) acc[j] += bits_f32(p[j]);
        }
      }
#pragma unroll
      for (int j = 0; j < 4; ++j) lds[w][lane * 4 + j] = acc[j];
      __syncthreads();
      if (w == 0 && col < g.dim) {
        const float* p = g.partial + ((size_t)c * 2 + 1) * g.pstride + col;
        float sum[4];
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          sum[j] = p[j];
          for (int k = 0; k < kWaves; ++k) sum[j] += lds[k][lane * 4 + j];
        }
        if (col + 4 <= g.dim) {
          write_row<To, 4, ACC>(g, row, col, 0, sum);
        } else {
#pragma unroll
          for (int j = 0; j < 4; ++j)
            if (col + j < g.dim) write_row<To, 1, ACC>(g, row, col + j, 0, sum + j);
        }
      }
      __syncthreads();
    }
  }
}

// The joins, and the last of the zeroing beside them.
template <typename To, bool ACC>
__global__ void __launch_bounds__(kThreads) join_kernel(Grad g, uint32_t join_blocks, uint32_t col_blocks,
                                                        uint32_t zero_done) {
  if (blockIdx.x < join_blocks) {
    const uint32_t groups = (g.nchunks - 1 + g.join_chunks - 1) / g.join_chunks;
    for (uint32_t i = blockIdx.x / col_blocks; i < groups; i += join_blocks / col_blocks)
      join_runs<To, ACC>(g, i, blockIdx.x % col_blocks, col_blocks);
    return;
  }
  if constexpr (!ACC) zero_rows<To>(g, g.zero_from + (zero_done + blockIdx.x - join_blocks) * g.zero_rows);
}

// Tokens per chunk (<= 64): short ones where the sums would not fill the GPU
// otherwise, long ones where they do, for fewer partials (the gradient of
// 60000 tokens x 4096 bf16, 32 and 64 tokens a chunk: 224 and 215 us; of 32000,
// 155 and 151; of 32768 x 2048, 205 and 207).
struct ChunkStep {
  uint32_t tokens;
  size_t work;      // from here on: tokens times slices of 256 columns
};
constexpr ChunkStep kChunkSteps[] = {{64, 4096 * 96}, {32, 4096 * 32}, {16, 4096 * 16}, {8, 0}};
uint32_t chunk_tokens(size_t n, size_t dim) {
  const size_t work = n * ((dim + 255) / 256);
  for (const ChunkStep& s : kChunkSteps)
    if (work >= s.work) return s.tokens;
  return 8;
}

// Values of the partials, at least, for every batch of up to n tokens and
// columns: not this batch's own, which are half as many wherever a chunk grows.
// A batch of n' tokens x w columns (w a multiple of 4) in chunks of c needs
// 2 * ceil(n' / c) * w <= 2 * (n' * w / c + w), and n' * w stays below 256
// times the work from which on chunks are longer.
size_t partial_values(size_t n, size_t dim) {
  const size_t width = (dim + 3) / 4 * 4;
  size_t most = 0, below = SIZE_MAX;
  for (const ChunkStep& s : kChunkSteps) {
    const size_t values = n * width < below ? n * width : below;
    const size_t v = (values + s.tokens - 1) / s.tokens;
    if (v > most) most = v;
    below = s.work * 256;
  }
  return n ? 2 * (most + width) : 0;
}

struct GradLayout {
  size_t keys, pos, sort, partial, bytes;
};
GradLayout grad_layout(size_t n, size_t dim) {
  auto up = [](size_t x) { return (x + 15) & ~(size_t)15; };
  GradLayout l;
  l.keys = 0;
  l.pos = up(n * 4);
  l.sort = l.pos + up(n * 4);
  l.partial = l.sort + up(sort_ids_ws_bytes(n));
  l.bytes = l.partial + partial_values(n, dim) * sizeof(float);
  return l;
}

template <typename Ti, typename To, bool ACC>
hipError_t run_grad(Grad g, hipStream_t stream) {
  // A quarter of the zeroing that is left runs beside the joins, which by
  // themselves are a few workgroups waiting for memory (a half or all of it
  // there: the same within 3%).
  const bool joins = g.nchunks > 1;
  g.slices = (g.dim + 64 * Ti::kVec - 1) / (64 * Ti::kVec);
  g.sum_units = (uint64_t)g.nchunks * g.slices;
  const uint32_t zero_blocks = (uint32_t)(((uint64_t)g.vocab - g.zero_from + g.zero_rows - 1) / g.zero_rows);
  uint32_t later = joins ? zero_blocks / 4 : 0;
  if (later > kMaxBlocks) later = kMaxBlocks;
  const uint32_t now = zero_blocks - later, sum_blocks = (uint32_t)((g.sum_units + kWaves - 1) / kWaves);
  const uint64_t blocks = (uint64_t)sum_blocks + now;
  if (blocks) {
    HC_ENQUEUE((grad_kernel<Ti, To, ACC>), (uint32_t)(blocks < kMaxBlocks ? blocks : kMaxBlocks), kThreads, stream, g,
               sum_blocks, now);
  }
  if (!joins) return hipSuccess;
  const uint32_t cols = (g.dim + kJoinCols - 1) / kJoinCols, col_blocks = cols < 8 ? cols : 8;
  // enough chunks per workgroup for one round of workgroups, some 2048
  const uint64_t all = (uint64_t)g.nchunks * col_blocks;
  g.join_chunks = all >= 2048 * 8 ? 8 : all <= 2048 ? 1 : (uint32_t)(all / 2048);
  const uint32_t groups = (g.nchunks - 1 + g.join_chunks - 1) / g.join_chunks;
  const uint32_t join_blocks = (groups < 65536 ? groups : 65536) * col_blocks;
  HC_ENQUEUE((join_kernel<To, ACC>), join_blocks + later, kThreads, stream, g, join_blocks, col_blocks, now);
  return hipSuccess;
}

}  // namespace

hipError_t launch_embedding(const KeySource& src, size_t ntokens, const void* weight, hc_dtype_t dtype, size_t dim,
                            size_t wstride, float scale, void* out, size_t ostride, hipStream_t stream) {
  auto run = [&](auto type) {
    typedef decltype(type) T;
    constexpr int U = 2;
    const uint32_t nvec = (uint32_t)((dim + T::kVec - 1) / T::kVec);
    uint32_t lg = 0;
    while (lg < 6 && (1u << lg) < nvec) ++lg;
    const uint32_t slices = (nvec + 64 * U - 1) / (64 * U);
    const uint64_t units = (uint64_t)((ntokens + (64u >> lg) - 1) / (64u >> lg)) * slices;
    auto launch = [&](auto kernel) {
      HC_ENQUEUE(kernel, blocks_for(units), kThreads, stream, src, ntokens, weight, (uint32_t)dim, wstride, scale, out,
                 ostride, lg, slices, units);
      return hipSuccess;
    };
    return ntokens * dim * sizeof(typename T::raw) >= kStreamStoreBytes ? launch(embedding_kernel<T, U, true>)
                                                                        : launch(embedding_kernel<T, U, false>);
  };
  if (dtype == HC_F32) return dim < F32::kVec ? run(F32S{}) : run(F32{});
  return dim < BF16::kVec ? run(BF16S{}) : run(BF16{});
}

size_t embedding_grad_ws_bytes(size_t ntokens, size_t dim) { return grad_layout(ntokens, dim).bytes; }

hipError_t launch_embedding_grad(const KeySource& src, size_t ntokens, const void* dout, hc_dtype_t dtype, size_t dim,
                                 size_t dstride, float scale, void* dweight, hc_dtype_t dwtype, size_t wstride,
                                 bool accumulate, void* ws, hipStream_t stream) {
  const GradLayout l = grad_layout(ntokens, dim);
  char* base = static_cast<char*>(ws);
  uint32_t* keys = reinterpret_cast<uint32_t*>(base + l.keys);
  uint32_t* pos = reinterpret_cast<uint32_t*>(base + l.pos);
  const size_t row_bytes = dim * (dwtype == HC_F32 ? 4 : 2), stride = wstride * (dwtype == HC_F32 ? 4 : 2);
  // A large table's zeroes are stored non-temporal: plain ones push the tokens'
  // rows out of the caches before they are summed.  Tokens x 2048 bf16 into
  // rows of fp32, plain / non-temporal, us: 2000 into 24,000 rows (197 MB) 45 / 41,
  // into 40,000 68 / 63; 16,000 into 24,000 81 / 75, into 40,000 102 / 91; 32,768
  // into 100,003 205 / 194.  Below, the gain is small (2000 into 12,000 28 / 26), and
  // the table itself stays in the caches for its next reader.  (Sums stored
  // non-temporal too: 201 where 194.)
  const bool stream_zeroes = src.nkeys * row_bytes >= kStreamStoreBytes;
  ZeroJob zero;
  zero.stream = stream_zeroes;
  if (!accumulate) {
    zero.base = static_cast<char*>(dweight);
    zero.flat = stride == row_bytes || src.nkeys == 1;
    zero.rows = zero.flat ? 1 : src.nkeys;
    zero.row_bytes = zero.flat ? row_bytes * src.nkeys : row_bytes;
    zero.stride = stride;
    zero.rows_per_piece = row_bytes < kPieceBytes ? kPieceBytes / row_bytes : 1;
    zero.pieces = zero.flat ? (zero.row_bytes + kPieceBytes - 1) / kPieceBytes
                            : (zero.rows + zero.rows_per_piece - 1) / zero.rows_per_piece;
  }
  if (hipError_t e = sort_ids(src, ntokens, keys, pos, base + l.sort, &zero, stream); e != hipSuccess) return e;
  Grad g = {};
  g.keys = keys;
  g.pos = pos;
  g.n = (uint32_t)ntokens;
  g.chunk = chunk_tokens(ntokens, dim);
  g.nchunks = (g.n + g.chunk - 1) / g.chunk;
  g.dim = (uint32_t)dim;
  g.vocab = src.nkeys;
  g.dout = dout;
  g.dstride = dstride;
  g.scale = scale;
  g.dweight = dweight;
  g.wstride = wstride;
  g.partial = reinterpret_cast<float*>(base + l.partial);
  g.pstride = (g.dim + 3) / 4 * 4;
  const uint64_t zeroed = zero.done == zero.pieces ? src.nkeys
                          : zero.flat              ? zero.done * kPieceBytes / row_bytes
                                                   : zero.done * zero.rows_per_piece;
  g.zero_stream = stream_zeroes;
  g.zero_from = accumulate ? g.vocab : (uint32_t)zeroed;
  g.zero_rows = row_bytes >= kZeroBytes / 4    ? 4
                : row_bytes <= kZeroBytes / 64 ? 64
                                               : (uint32_t)(kZeroBytes / row_bytes);
  auto run = [&](auto in, auto table) {
    typedef decltype(in) Ti;
    typedef decltype(table) To;
    return accumulate ? run_grad<Ti, To, true>(g, stream) : run_grad<Ti, To, false>(g, stream);
  };
  auto run_in = [&](auto in) { return dwtype == HC_F32 ? run(in, F32{}) : run(in, BF16{}); };
  if (dtype == HC_F32) return dim < F32::kVec ? run_in(F32S{}) : run_in(F32{});
  return dim < BF16::kVec ? run_in(BF16S{}) : run_in(BF16{});
}

}  // namespace hc
