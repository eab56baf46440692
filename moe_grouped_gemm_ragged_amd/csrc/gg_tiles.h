// gg_tiles.h -- the 256-row tiles of a layout that packed scales are counted
// in, for the kernels that write or read them row by row.
#pragma once
#include <hip/hip_runtime.h>
#include <stdint.h>

#include <type_traits>

#include "gg_internal.h"

namespace gg {
namespace tiles {

// RAGGED: groups = end offsets, rows in all.  MASKED_ROWS: groups = masked_m,
// rows of each expert.  WEIGHTS: rows of each expert, all of them.
enum Layout { RAGGED = 0, MASKED_ROWS = 1, WEIGHTS = 2 };

constexpr int kTileRows = 256;     // rows per packed tile
constexpr int kThreads = 256;      // of a workgroup that decodes them

// Block-wide scan of one non-negative int per thread (sum, or max): a shuffle
// scan within each wave, then the totals of the earlier waves.  Returns the
// inclusive value; *excl gets the exclusive one (0 for thread 0).
template <bool MAX>
__device__ __forceinline__ int block_scan(int v, int* wave_tot, int tid, int* excl) {
  const int lane = tid & 63, w = tid >> 6;
#pragma unroll
  for (int d = 1; d < 64; d <<= 1) {
    const int o = __shfl_up(v, (unsigned)d, 64);
    if (lane >= d) v = MAX ? (v > o ? v : o) : v + o;
  }
  int prev = __shfl_up(v, 1u, 64);
  if (lane == 0) prev = 0;
  if (lane == 63) wave_tot[w] = v;
  __syncthreads();
  int before = 0;
  for (int q = 0; q < w; ++q) {
    const int t = wave_tot[q];
    before = MAX ? (before > t ? before : t) : before + t;
  }
  __syncthreads();
  *excl = MAX ? (prev > before ? prev : before) : prev + before;
  return MAX ? (v > before ? v : before) : v + before;
}

// The ragged layout's tiles: experts' clamped monotone ends (prefix max of the
// offsets, capped at rows) and the tiles before each, as the GEMMs decode them.
struct Tiles {
  int32_t end[GG_MAX_GROUPS_DEV];
  int32_t pref[GG_MAX_GROUPS_DEV + 1];
  int32_t wave[kThreads / 64];
};
struct NoTiles {};

// Returns the number of tiles.
__device__ __forceinline__ int64_t decode_tiles(Tiles& s, const int32_t* groups, int64_t rows, int E, int tid) {
  const int per = (E + kThreads - 1) / kThreads;
  const int g0 = tid * per;
  const int g1 = g0 + per < E ? g0 + per : E;
  int run = 0;
  for (int g = g0; g < g1; ++g) {
    const int o = groups[g];
    run = o > run ? o : run;
    s.end[g] = run;
  }
  int before;
  block_scan<true>(run, s.wave, tid, &before);
  for (int g = g0; g < g1; ++g) {
    const int e = s.end[g] > before ? s.end[g] : before;
    s.end[g] = e < rows ? e : (int)rows;
  }
  __syncthreads();
  int local = 0;
  for (int g = g0; g < g1; ++g) local += (s.end[g] - (g == 0 ? 0 : s.end[g - 1]) + kTileRows - 1) / kTileRows;
  int acc;
  const int incl = block_scan<false>(local, s.wave, tid, &acc);
  for (int g = g0; g < g1; ++g) {
    s.pref[g] = acc;
    acc += (s.end[g] - (g == 0 ? 0 : s.end[g - 1]) + kTileRows - 1) / kTileRows;
  }
  if (tid == kThreads - 1) s.pref[E] = incl;
  __syncthreads();
  return s.pref[E];
}

// The first row of tile T and how many of its 256 rows are an expert's.
template <int LAYOUT, typename S>
__device__ __forceinline__ void tile_rows(const S& s, const int32_t* groups, int64_t rows, int E, int64_t T,
                                          int64_t& first, int& valid) {
  if constexpr (LAYOUT == RAGGED) {
    int lo = 0, hi = E;                 // largest g with pref[g] <= T
    while (hi - lo > 1) {
      const int mid = (lo + hi) >> 1;
      if (s.pref[mid] <= T) lo = mid; else hi = mid;
    }
    first = (lo == 0 ? 0 : s.end[lo - 1]) + (T - s.pref[lo]) * kTileRows;
    const int64_t v = s.end[lo] - first;
    valid = v < kTileRows ? (int)v : kTileRows;
  } else {
    const int64_t per = (rows + kTileRows - 1) / kTileRows;
    const int64_t e = T / per, r0 = (T - e * per) * kTileRows;
    int64_t active = rows;
    if constexpr (LAYOUT == MASKED_ROWS) {
      const int64_t a = groups[e];
      active = a < 0 ? 0 : a < rows ? a : rows;
    }
    first = e * rows + r0;
    const int64_t v = active - r0;
    valid = v < 0 ? 0 : v < kTileRows ? (int)v : kTileRows;
  }
}

}  // namespace tiles
}  // namespace gg
