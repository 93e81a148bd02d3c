// key_sort.hpp -- a stable counting sort by one digit, shared by the tokens
// of an embedding's gradient (one to four digits) and the slots of experts
// (one digit).
//
// The input is cut into at most kMaxTiles tiles, one per workgroup of 16
// waves.  A histogram launch counts each tile's digits; the scatter launch's
// workgroups then add up the counts of the tiles before theirs themselves
// (at most 64 x 1024 words out of the cache), so the pair needs no scan launch
// between them.  Short inputs need no histogram launch either: every workgroup
// counts all of them.  Within a tile each wave owns a contiguous run of items: it
// counts its run, the waves' counts are scanned per digit, and the wave walks
// its run 64 items at a time, ranking equal digits by ballots.  Nothing
// depends on the order in which atomics arrive.
#pragma once

#include "rows.hpp"
#include "step_launch.hpp"

namespace hc {

constexpr uint32_t kSortThreads = 1024;
constexpr uint32_t kSortWaves = kSortThreads / 64;
constexpr uint32_t kMaxRadix = 1024;
constexpr uint32_t kMaxTiles = 64;
constexpr uint32_t kMinTile = 1024;     // items

// Items per tile, a multiple of 1024 (64 per wave), for at most kMaxTiles tiles.
inline uint32_t sort_tile(size_t n) {
  const size_t per = (n + kMaxTiles - 1) / kMaxTiles;
  const size_t t = (per + kMinTile - 1) / kMinTile * kMinTile;
  return (uint32_t)(t < kMinTile ? kMinTile : t);
}
inline uint32_t sort_tiles(size_t n) { return (uint32_t)((n + sort_tile(n) - 1) / sort_tile(n)); }

__device__ __forceinline__ uint32_t load_key(const KeySource& s, size_t i) {
  const int64_t id =
      s.id_bytes == 8 ? static_cast<const int64_t*>(s.ids)[i] : (int64_t)static_cast<const int32_t*>(s.ids)[i];
  // the unsigned difference is exact for an id from start on; below it, it would
  // pass for a key where start + nkeys is past the ids' type
  const uint64_t k = (uint64_t)id - (uint64_t)s.start;
  if (id < s.start || k >= s.nkeys || (s.use_skip && id == s.skip)) return kNoKey;
  return (uint32_t)k;
}

// The lanes of the wave with this lane's digit, among those with `valid`.
__device__ __forceinline__ uint64_t same_digit(uint32_t digit, bool valid, uint32_t bits) {
  uint64_t m = __ballot(valid);
  for (uint32_t b = 0; b < bits; ++b) {
    const uint64_t s = __ballot((digit >> b) & 1u);
    m &= ((digit >> b) & 1u) ? s : ~s;
  }
  return m;
}

// Exclusive scan over the workgroup's kSortThreads values; *total: their sum.
__device__ __forceinline__ uint32_t block_scan(uint32_t v, uint32_t* lds /* kSortWaves + 1 */, uint32_t* total) {
  uint32_t x = v;
#pragma unroll
  for (int d = 1; d < 64; d <<= 1) {
    const uint32_t y = __shfl_up(x, d);
    if (lane_id() >= (uint32_t)d) x += y;
  }
  if (lane_id() == 63) lds[threadIdx.x >> 6] = x;
  __syncthreads();
  uint32_t before = 0, all = 0;
  for (uint32_t w = 0; w < kSortWaves; ++w) {
    if (w < (threadIdx.x >> 6)) before += lds[w];
    all += lds[w];
  }
  *total = all;
  __syncthreads();
  return before + x - v;
}

// One tile's histogram of digit(i) in [0, radix) over items [lo, hi);
// kNoKey counts nowhere.
template <typename Digit>
__device__ __forceinline__ void tile_histogram(uint32_t* lds, uint32_t radix, size_t lo, size_t hi, Digit digit,
                                               uint32_t* out) {
  for (uint32_t d = threadIdx.x; d < radix; d += kSortThreads) lds[d] = 0;
  __syncthreads();
  for (size_t i = lo + threadIdx.x; i < hi; i += kSortThreads) {
    const uint32_t d = digit(i);
    if (d != kNoKey) atomicAdd(&lds[d], 1u);
  }
  __syncthreads();
  for (uint32_t d = threadIdx.x; d < radix; d += kSortThreads) out[d] = lds[d];
}

// Per digit: the sum of the tiles' counts before `tile`, and over all tiles.
// All tiles' loads are in flight at once.
__device__ __forceinline__ void tile_sums(const uint32_t* hist, uint32_t radix, uint32_t tiles, uint32_t tile,
                                          uint32_t d, uint32_t* before, uint32_t* total) {
  uint32_t b = 0, a = 0;
  if (d < radix) {
    uint32_t c[kMaxTiles];
#pragma unroll
    for (uint32_t i = 0; i < kMaxTiles; ++i) c[i] = i < tiles ? hist[(size_t)i * radix + d] : 0;
    __builtin_amdgcn_sched_barrier(0);
#pragma unroll
    for (uint32_t i = 0; i < kMaxTiles; ++i) {
      b += i < tile ? c[i] : 0;
      a += c[i];
    }
  }
  *before = b;
  *total = a;
}

// A wave's items of its tile: a contiguous run, 64 at a time.  The first
// kHeld rounds' digits stay in registers, which is all of them in tiles of up
// to 4096 items; later ones are read again when they are placed.
constexpr uint32_t kHeld = 4;
struct Run {
  size_t begin, end;
  uint32_t held[kHeld];
};
template <typename Digit>
__device__ __forceinline__ Run load_run(size_t lo, size_t hi, uint32_t tile_items, Digit digit) {
  Run r;
  const uint32_t run = tile_items / kSortWaves;
  r.begin = lo + (size_t)wave_id() * run;
  r.end = r.begin + run < hi ? r.begin + run : hi;
#pragma unroll
  for (uint32_t k = 0; k < kHeld; ++k) {
    const size_t i = r.begin + k * 64 + lane_id();
    r.held[k] = i < r.end ? digit(i) : kNoKey;
  }
  return r;
}

// The same two sums, counted by the workgroup itself from all n items: up to
// kSelfCount items that is less than a histogram launch before it (sort and
// dispatch of 500 tokens x 8 slots 9.2 us so, 9.8 by two launches; of 2000 x 8,
// 13.1 and 11.2).  counts: 2 x radix words of LDS, free again afterwards.
constexpr uint32_t kSelfCount = 4096;
template <typename Digit>
__device__ __forceinline__ void self_sums(uint32_t* counts, uint32_t radix, size_t n, size_t lo, const Run& run,
                                          uint32_t d, Digit digit, uint32_t* before, uint32_t* total) {
  for (uint32_t i = threadIdx.x; i < 2 * radix; i += kSortThreads) counts[i] = 0;
  __syncthreads();
  const bool one = n <= kMinTile;       // all items are the run's first round
  if (one && run.held[0] != kNoKey) atomicAdd(&counts[radix + run.held[0]], 1u);
  for (size_t i0 = one ? n : 0; i0 < n; i0 += 8 * kSortThreads) {
    uint32_t key[8];
#pragma unroll
    for (uint32_t u = 0; u < 8; ++u) {
      const size_t i = i0 + u * kSortThreads + threadIdx.x;
      key[u] = i < n ? digit(i) : kNoKey;
    }
#pragma unroll
    for (uint32_t u = 0; u < 8; ++u)
      if (key[u] != kNoKey) atomicAdd(&counts[(i0 + u * kSortThreads < lo ? 0 : radix) + key[u]], 1u);
  }
  __syncthreads();
  *before = d < radix ? counts[d] : 0;
  *total = d < radix ? *before + counts[radix + d] : 0;
  __syncthreads();
}

// Hands each item of the run its place: put(i, digit, place) with place = the
// digit's first place for this tile (my_base, of digit threadIdx.x) + how many
// items of the tile before it have the same digit.  counts: kSortWaves x radix
// words of LDS.  Items without a key: put(i, kNoKey, 0).
template <typename Digit, typename Put>
__device__ __forceinline__ void place_items(uint32_t* counts, uint32_t radix, uint32_t bits, const Run& r,
                                            uint32_t my_base, Digit digit, Put put) {
  const uint32_t lane = lane_id();
  uint32_t* mine = counts + (size_t)wave_id() * radix;
  for (uint32_t d = threadIdx.x; d < radix * kSortWaves; d += kSortThreads) counts[d] = 0;
  __syncthreads();
#pragma unroll
  for (uint32_t k = 0; k < kHeld; ++k)
    if (r.held[k] != kNoKey) atomicAdd(&mine[r.held[k]], 1u);
  for (size_t i = r.begin + kHeld * 64 + lane; i < r.end; i += 64) {
    const uint32_t d = digit(i);
    if (d != kNoKey) atomicAdd(&mine[d], 1u);
  }
  __syncthreads();
  if (threadIdx.x < radix) {
    uint32_t c[kSortWaves], p = my_base;
#pragma unroll
    for (uint32_t v = 0; v < kSortWaves; ++v) c[v] = counts[v * radix + threadIdx.x];
#pragma unroll
    for (uint32_t v = 0; v < kSortWaves; ++v) {
      counts[v * radix + threadIdx.x] = p;
      p += c[v];
    }
  }
  __syncthreads();
  auto place64 = [&](size_t i, uint32_t d) {
    const bool valid = d != kNoKey;
    const uint64_t same = same_digit(d, valid, bits);
    uint32_t place = 0;
    if (valid) place = mine[d] + (uint32_t)__popcll(same & ((1ull << lane) - 1));
    // the counters are the wave's own: its lanes read before its lanes write
    __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
    __builtin_amdgcn_wave_barrier();
    if (valid && (same >> lane) == 1) mine[d] = place + 1;   // the digit's last lane
    __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
    __builtin_amdgcn_wave_barrier();
    if (i < r.end) put(i, d, place);
  };
#pragma unroll
  for (uint32_t k = 0; k < kHeld; ++k)
    if (r.begin + k * 64 < r.end) place64(r.begin + k * 64 + lane, r.held[k]);
  for (size_t i0 = r.begin + kHeld * 64; i0 < r.end; i0 += 64)
    place64(i0 + lane, i0 + lane < r.end ? digit(i0 + lane) : kNoKey);
}

}  // namespace hc
