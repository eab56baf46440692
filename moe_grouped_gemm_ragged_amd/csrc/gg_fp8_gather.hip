// gg_fp8_gather.hip -- e4m3 rows sorted by expert together with their scales.
//
//   dst[r] = src[row_slot[r] / topk]                    (16 bytes per lane)
//   dst_scales = the scales of those rows in the packed, tile-major layout
//                that the fp8 GEMM reads (stated in gg_fp8_scales.hip)
//
// One launch in place of two gathers and a pack step, whose scale rows would
// have to be a multiple of 16 bytes.  A padding row gets zero codes and the
// scale 1 (byte 127), tile rows past an expert's last row the byte 0, as
// gg_fp8_pack_scales writes them.
//
// Bound by memory: a token has to be read once and a row written once.  The
// first workgroups write scales, one wave for 8 blocks of a 256-row tile; the
// rest copy rows.  8195 tokens of 7168 bytes to 8 of 256 experts: 107-115 us
// (219 MB read, the tokens 3.7 times, and 490 MB written: 6.3 TB/s); 32 tokens
// of 2048 bytes to 8 of 128 experts: 5 us.
#include <hip/hip_runtime.h>
#include <stdint.h>

#include "gg_internal.h"
#include "gg_rows.h"

namespace gg {
namespace {

using namespace rows;

constexpr int kThreads = 256;
constexpr int kWaves = kThreads / 64;
constexpr int kTile = 256;      // rows of a packed scale tile
constexpr int kKb = 8;          // k-blocks a wave packs at a time
// Workgroups a compute unit at most: copying rows in order; copying by
// windows, where fewer keep closer together (8195 tokens of 7168 bytes to 8
// experts each: 108 us with 2, 114 with 4, 120 with 8); packing scales (first
// in the grid: few bytes, long latency).
constexpr int kRowBlocks = 8;
constexpr int kWindowBlocks = 2;
constexpr int kScaleBlocks = 2;
constexpr int64_t kWindowBytes = 2 << 20;      // of src in a window: half an XCD's L2
constexpr int64_t kWindowedBytes = 8 << 20;    // of src from which on rows are copied by windows

// Rows of packed tile `tile`: the first one and how many.  false if no
// expert has that tile.  Called by the whole wave: lane l looks after a run
// of consecutive experts; the end offsets become monotone and clamped to
// rows_cap as the GEMMs read them.
__device__ bool tile_rows(const int32_t* offs, int32_t E, int64_t rows_cap, int64_t tile, int64_t& first,
                          int& valid) {
  const int lane = threadIdx.x & 63;
  const int per = (E + 63) / 64;
  const int g0 = lane * per < E ? lane * per : E;
  const int g1 = g0 + per < E ? g0 + per : E;
  int before = 0;
  for (int g = g0; g < g1; ++g) before = offs[g] > before ? offs[g] : before;
  int incl = before;
#pragma unroll
  for (int d = 1; d < 64; d <<= 1) {
    const int o = __shfl_up(incl, (unsigned)d, 64);
    if (lane >= d) incl = o > incl ? o : incl;
  }
  before = __shfl_up(incl, 1u, 64);
  if (lane == 0) before = 0;
  int64_t start = before < rows_cap ? before : rows_cap;
  int64_t prev = start, count = 0;
  for (int g = g0; g < g1; ++g) {
    int64_t e = offs[g] < rows_cap ? offs[g] : rows_cap;
    e = e > prev ? e : prev;
    count += (e - prev + kTile - 1) / kTile;
    prev = e;
  }
  int upto = (int)count;
#pragma unroll
  for (int d = 1; d < 64; d <<= 1) {
    const int o = __shfl_up(upto, (unsigned)d, 64);
    if (lane >= d) upto += o;
  }
  int64_t at = upto - count;
  const bool mine = at <= tile && tile < upto;
  const uint64_t who = __ballot(mine);
  if (!who) return false;
  int64_t f = 0;
  int v = 0;
  if (mine) {
    prev = start;
    for (int g = g0; g < g1; ++g) {
      int64_t e = offs[g] < rows_cap ? offs[g] : rows_cap;
      e = e > prev ? e : prev;
      const int64_t tiles = (e - prev + kTile - 1) / kTile;
      if (tile < at + tiles) {
        f = prev + (tile - at) * kTile;
        v = (int)(e - f < kTile ? e - f : kTile);
        break;
      }
      at += tiles;
      prev = e;
    }
  }
  const int src = __builtin_ctzll(who);
  first = ((int64_t)__shfl((int)(f >> 32), src, 64) << 32) | (uint32_t)__shfl((int)(uint32_t)f, src, 64);
  valid = __shfl(v, src, 64);
  return true;
}

constexpr int kUnits = 8;       // 1 KB pieces a wave moves at a time

// Copies kUnits / CH rows (CH pieces of 1 KB each; CH = 8: any longer row, 8
// KB after 8 KB), all loads before the first store.  Lane i < R brings row i
// and its slot (row < 0: none).  NT: stores that leave the caches to src (not
// for few rows, which the GEMM then finds in the caches).
template <int CH, bool NT>
__device__ __forceinline__ void copy_rows(const uint8_t* src, int64_t row, int32_t slot, int32_t topk, int64_t tokens,
                                          int64_t k, uint8_t* dst) {
  constexpr int R = kUnits / CH;
  const int lane = threadIdx.x & 63;
  const uint8_t* from[R];
  uint8_t* to[R];
  bool there[R], live[R];
#pragma unroll
  for (int i = 0; i < R; ++i) {
    const int32_t s = __builtin_amdgcn_readlane(slot, i), r = __builtin_amdgcn_readlane((int)row, i);
    const int64_t token = s >= 0 ? s / topk : tokens;
    live[i] = r >= 0;
    there[i] = token < tokens;
    from[i] = src + (there[i] ? token * k : 0);
    to[i] = dst + (int64_t)(live[i] ? r : 0) * k;
  }
  for (int64_t c0 = 16 * lane; c0 < k; c0 += CH * 1024) {
    u32x4r v[kUnits];
#pragma unroll
    for (int u = 0; u < kUnits; ++u) {
      const int64_t c = c0 + 1024 * (u % CH);
      v[u] = u32x4r{0u, 0u, 0u, 0u};
      if (there[u / CH] && c < k) v[u] = load16(from[u / CH] + c);
    }
#pragma unroll
    for (int u = 0; u < kUnits; ++u) {
      const int64_t c = c0 + 1024 * (u % CH);
      if (live[u / CH] && c < k) {
        if constexpr (NT) store16(to[u / CH] + c, v[u]);
        else *reinterpret_cast<u32x4r*>(to[u / CH] + c) = v[u];
      }
    }
  }
}

// Rows in order, a wave's next slots on their way while it copies.
template <int CH>
__device__ __forceinline__ void copy_in_order(const uint8_t* src, const int32_t* row_slot, int32_t topk,
                                              int64_t tokens, int64_t end, int64_t k, uint8_t* dst, int64_t wave,
                                              int64_t waves) {
  constexpr int R = kUnits / CH;
  const int lane = threadIdx.x & 63;
  int64_t row = wave * R + lane;
  bool mine = lane < R && row < end;
  int32_t slot = mine ? row_slot[row] : -1;
  for (int64_t first = wave * R; first < end; first += waves * R) {
    const int64_t ahead = row + waves * R;
    const bool more = lane < R && ahead < end;
    const int32_t next = more ? row_slot[ahead] : -1;
    copy_rows<CH, false>(src, mine ? row : -1, slot, topk, tokens, k, dst);
    row = ahead;
    mine = more;
    slot = next;
  }
}

// Block-wide inclusive scan of one non-negative int per thread (sum, or
// maximum), and the value before this thread's.
template <bool MAX>
__device__ __forceinline__ int block_scan(int v, int* wave_tot, int& before) {
  const int lane = threadIdx.x & 63, w = threadIdx.x >> 6;
#pragma unroll
  for (int d = 1; d < 64; d <<= 1) {
    const int o = __shfl_up(v, (unsigned)d, 64);
    if (lane >= d) v = MAX ? (v > o ? v : o) : v + o;
  }
  before = __shfl_up(v, 1u, 64);
  if (lane == 0) before = 0;
  if (lane == 63) wave_tot[w] = v;
  __syncthreads();
  int base = 0;
  for (int q = 0; q < w; ++q) base = MAX ? (base > wave_tot[q] ? base : wave_tot[q]) : base + wave_tot[q];
  before = MAX ? (before > base ? before : base) : before + base;
  return MAX ? (v > base ? v : base) : v + base;
}

// Rows by windows of tokens.  A token is read once for each of its rows,
// which lie in as many experts; within an expert the rows ascend by token, so
// the rows of one fraction of every expert come from about the same fraction
// of the tokens.  Window i of `windows` is that fraction of every expert;
// workgroup b runs on XCD b mod 8, and each XCD takes an eighth of the windows
// one after the other, so that a window's tokens (and its neighbours', for the
// fractions fit the tokens only roughly) stay in its L2 for all their rows.
// Where a row lies is exact; how well the windows fit only decides the speed.
template <int CH>
__device__ __forceinline__ void copy_by_window(const uint8_t* src, const int32_t* row_slot, int32_t topk,
                                               int64_t tokens, const int32_t* offs, int32_t E, int64_t rows_cap,
                                               int64_t k, uint8_t* dst, int block, int blocks, int windows) {
  constexpr int R = kUnits / CH;
  __shared__ int32_t s_end[GG_MAX_GROUPS_DEV];
  __shared__ int32_t s_pref[2][GG_MAX_GROUPS_DEV + 1];
  __shared__ int32_t s_tot[2][kWaves];
  const int t = threadIdx.x, lane = t & 63;
  const int per = (E + kThreads - 1) / kThreads;
  const int g0 = t * per < E ? t * per : E;
  const int g1 = g0 + per < E ? g0 + per : E;
  // clamped monotone ends, as the GEMMs read the offsets
  int run = 0, before;
  for (int g = g0; g < g1; ++g) {
    run = offs[g] > run ? offs[g] : run;
    s_end[g] = run;
  }
  block_scan<true>(run, s_tot[0], before);
  for (int g = g0; g < g1; ++g) {
    const int e = s_end[g] > before ? s_end[g] : before;
    s_end[g] = e < rows_cap ? e : (int)rows_cap;
  }
  __syncthreads();
  int turn = 0;
  const int share = windows >> 3;       // windows is a multiple of 8
  for (int w = (block & 7) * share; w < ((block & 7) + 1) * share; ++w) {
    // rows of this window before each expert's: two buffers in turn, see
    // RowSums in gg_norm.hip for why one barrier a window is enough
    int32_t* pref = s_pref[turn];
    int local = 0;
    for (int g = g0; g < g1; ++g) {
      const int64_t rows = s_end[g] - (g ? s_end[g - 1] : 0);
      local += (int)(rows * (w + 1) / windows - rows * w / windows);
    }
    const int incl = block_scan<false>(local, s_tot[turn], before);
    for (int g = g0; g < g1; ++g) {
      pref[g] = before;
      const int64_t rows = s_end[g] - (g ? s_end[g - 1] : 0);
      before += (int)(rows * (w + 1) / windows - rows * w / windows);
    }
    if (t == kThreads - 1) pref[E] = incl;
    __syncthreads();
    turn ^= 1;
    const int total = pref[E];
    const int waves = (blocks >> 3) * kWaves;
    for (int at = ((block >> 3) * kWaves + (t >> 6)) * R; at < total; at += waves * R) {
      // lane i: row at + i of the window
      int64_t row = -1;
      int32_t slot = -1;
      if (lane < R && at + lane < total) {
        int lo = 0, hi = E;               // the last expert with pref <= at + lane
        while (hi - lo > 1) {
          const int mid = (lo + hi) >> 1;
          if (pref[mid] <= at + lane) lo = mid; else hi = mid;
        }
        const int64_t start = lo ? s_end[lo - 1] : 0;
        row = start + (s_end[lo] - start) * w / windows + (at + lane - pref[lo]);
        slot = row_slot[row];
      }
      copy_rows<CH, true>(src, row, slot, topk, tokens, k, dst);
    }
  }
}

// CH: 1 KB pieces of a row taken together.  VEC: the scales of a row are read
// 4 at a time (k-blocks a multiple of 4).  windows: 0 for rows in order.
template <int CH, bool VEC>
__global__ __launch_bounds__(kThreads) void fp8_gather_rows_kernel(const uint8_t* src, const uint8_t* src_scales,
                                                                   const int32_t* row_slot, const int32_t* offs,
                                                                   int32_t E, int32_t topk, int64_t tokens,
                                                                   int64_t rows_cap, int64_t k, int64_t tiles,
                                                                   uint8_t* dst, uint8_t* dst_scales,
                                                                   int32_t scale_blocks, int32_t windows) {
  const int lane = threadIdx.x & 63;
  const int wave = threadIdx.x >> 6;
  const int kblocks = (int)(k / kBlock);
  if ((int)blockIdx.x >= scale_blocks) {
    const int block = blockIdx.x - scale_blocks, blocks = gridDim.x - scale_blocks;
    if (windows > 0)
      copy_by_window<CH>(src, row_slot, topk, tokens, offs, E, rows_cap, k, dst, block, blocks, windows);
    else
      copy_in_order<CH>(src, row_slot, topk, tokens, owned_rows(offs, E, rows_cap), k, dst,
                        (int64_t)block * kWaves + wave, (int64_t)blocks * kWaves);
    return;
  }
  const int chunks = (kblocks + kKb - 1) / kKb;
  const int64_t items = tiles * chunks;
  for (int64_t it = (int64_t)blockIdx.x * kWaves + wave; it < items; it += (int64_t)scale_blocks * kWaves) {
    const int64_t tile = it / chunks;
    const int kb0 = (int)(it - tile * chunks) * kKb;
    int64_t first;
    int valid;
    if (!tile_rows(offs, E, rows_cap, tile, first, valid)) break;   // tiles past the last one
    // lane d writes dword d of a block's 256 bytes: the bytes of tile rows
    // 128 (d / 32) + d mod 32 + 32 b
    uint32_t word[kKb];
#pragma unroll
    for (int i = 0; i < kKb; ++i) word[i] = 0u;
#pragma unroll
    for (int b = 0; b < 4; ++b) {
      const int r = 128 * (lane >> 5) + (lane & 31) + 32 * b;
      if (r >= valid) continue;
      const int32_t s = row_slot[first + r];
      const int64_t token = s >= 0 ? s / topk : -1;
      if (token < 0 || token >= tokens) {
#pragma unroll
        for (int i = 0; i < kKb; ++i) word[i] |= 127u << (8 * b);
        continue;
      }
      const uint8_t* from = src_scales + token * kblocks + kb0;
      if constexpr (VEC) {
#pragma unroll
        for (int i = 0; i < kKb; i += 4) {
          if (kb0 + i >= kblocks) break;
          const uint32_t q = *reinterpret_cast<const uint32_t*>(from + i);
#pragma unroll
          for (int j = 0; j < 4; ++j) word[i + j] |= ((q >> (8 * j)) & 0xFFu) << (8 * b);
        }
      } else {
#pragma unroll
        for (int i = 0; i < kKb; ++i)
          if (kb0 + i < kblocks) word[i] |= (uint32_t)from[i] << (8 * b);
      }
    }
#pragma unroll
    for (int i = 0; i < kKb; ++i)
      if (kb0 + i < kblocks) reinterpret_cast<uint32_t*>(dst_scales + (tile * kblocks + kb0 + i) * kTile)[lane] = word[i];
  }
}

}  // namespace

hipError_t launch_fp8_gather_rows(const void* src, const void* src_scales, const int32_t* row_slot,
                                  const int32_t* offs, int32_t E, int32_t topk, int64_t tokens, int64_t rows_cap,
                                  int64_t k, void* dst, void* dst_scales, int num_cus, hipStream_t stream) {
  if (rows_cap == 0) return hipSuccess;
  const int64_t tiles = fp8_scale_tiles(0, rows_cap, E);
  const int64_t kib = (k + 1023) / 1024;
  const int ch = kib <= 1 ? 1 : kib <= 2 ? 2 : kib <= 4 ? 4 : 8;
  // Rows by windows where tokens are read several times and a large src would
  // come from memory each time: 8195 x 7168 to 8 of 256 experts 108 us (in
  // order 152), 8192 x 2048 to 8 of 128 28.6 us (in order 41.8).  (With fewer
  // rows than tokens most tokens are read once at most, and the windows, as
  // many as src is long, would hold next to nothing each.)
  const int64_t bytes = tokens * k;
  const bool windowed = topk > 1 && bytes > kWindowedBytes && rows_cap > tokens;
  const int windows = windowed ? (int)((bytes + 8 * kWindowBytes - 1) / (8 * kWindowBytes) * 8) : 0;
  const int64_t per = kWaves * (kUnits / ch);
  const int64_t rows_want = (rows_cap + per - 1) / per;
  const int64_t rows_most = (windows ? kWindowBlocks : kRowBlocks) * (int64_t)num_cus;
  // (multiples of 8, where a workgroup's XCD matters)
  const int row_blocks = ((int)(rows_want < rows_most ? rows_want : rows_most) + 7) / 8 * 8;
  const int64_t chunks = (k / kBlock + kKb - 1) / kKb;
  const int64_t scale_want = (tiles * chunks + kWaves - 1) / kWaves, scale_most = kScaleBlocks * (int64_t)num_cus;
  const int scale_blocks = (int)((scale_want < scale_most ? scale_want : scale_most) + 7) / 8 * 8;
  const bool vec = (k / kBlock) % 4 == 0 && (reinterpret_cast<uintptr_t>(src_scales) & 3u) == 0;
  auto run = [&](auto* kernel) {
    return launch_kernel(kernel, dim3(row_blocks + scale_blocks), dim3(kThreads), stream,
                         static_cast<const uint8_t*>(src), static_cast<const uint8_t*>(src_scales), row_slot, offs, E,
                         topk, tokens, rows_cap, k, tiles, static_cast<uint8_t*>(dst),
                         static_cast<uint8_t*>(dst_scales), scale_blocks, windows);
  };
  switch (ch) {
    case 1: return vec ? run(fp8_gather_rows_kernel<1, true>) : run(fp8_gather_rows_kernel<1, false>);
    case 2: return vec ? run(fp8_gather_rows_kernel<2, true>) : run(fp8_gather_rows_kernel<2, false>);
    case 4: return vec ? run(fp8_gather_rows_kernel<4, true>) : run(fp8_gather_rows_kernel<4, false>);
    default: return vec ? run(fp8_gather_rows_kernel<8, true>) : run(fp8_gather_rows_kernel<8, false>);
  }
}

}  // namespace gg
