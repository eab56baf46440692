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
// Bound by memory: every live row is read and written once.  The first
// workgroups copy rows, one wave a row; the rest write scales, one wave for
// 8 blocks of a 256-row tile.
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

// VEC: the scales of a row are read 4 at a time (k-blocks a multiple of 4).
template <bool VEC>
__global__ __launch_bounds__(kThreads) void fp8_gather_rows_kernel(const uint8_t* src, const uint8_t* src_scales,
                                                                   const int32_t* row_slot, const int32_t* offs,
                                                                   int32_t E, int32_t topk, int64_t tokens,
                                                                   int64_t rows_cap, int64_t k, int64_t tiles,
                                                                   uint8_t* dst, uint8_t* dst_scales,
                                                                   int32_t row_blocks) {
  const int lane = threadIdx.x & 63;
  const int wave = threadIdx.x >> 6;
  const int kblocks = (int)(k / kBlock);
  if ((int)blockIdx.x < row_blocks) {
    const int64_t end = owned_rows(offs, E, rows_cap);
    for (int64_t r = (int64_t)blockIdx.x * kWaves + wave; r < end; r += (int64_t)row_blocks * kWaves) {
      const int32_t s = row_slot[r];
      const int64_t token = s >= 0 ? s / topk : -1;
      const bool there = token >= 0 && token < tokens;
      const uint8_t* from = src + token * k;
      for (int64_t c = 16 * lane; c < k; c += 16 * 64) {
        u32x4r v = {0u, 0u, 0u, 0u};
        if (there) v = load16(from + c);
        store16(dst + r * k + c, v);
      }
    }
    return;
  }
  const int chunks = (kblocks + kKb - 1) / kKb;
  const int64_t items = tiles * chunks;
  for (int64_t it = (int64_t)(blockIdx.x - row_blocks) * kWaves + wave; it < items;
       it += (int64_t)(gridDim.x - row_blocks) * kWaves) {
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
  const int64_t most = 8 * (int64_t)num_cus;
  const int64_t rows_want = (rows_cap + kWaves - 1) / kWaves;
  const int row_blocks = (int)(rows_want < most ? rows_want : most);
  const int64_t chunks = (k / kBlock + kKb - 1) / kKb;
  const int64_t scale_want = (tiles * chunks + kWaves - 1) / kWaves;
  const int scale_blocks = (int)(scale_want < most ? scale_want : most);
  const dim3 grid(row_blocks + scale_blocks), block(kThreads);
  const bool vec = (k / kBlock) % 4 == 0 && (reinterpret_cast<uintptr_t>(src_scales) & 3u) == 0;
  auto* kernel = vec ? fp8_gather_rows_kernel<true> : fp8_gather_rows_kernel<false>;
  return launch_kernel(kernel, grid, block, stream, static_cast<const uint8_t*>(src),
                       static_cast<const uint8_t*>(src_scales), row_slot, offs, E, topk, tokens, rows_cap, k, tiles,
                       static_cast<uint8_t*>(dst), static_cast<uint8_t*>(dst_scales), row_blocks);
}

}  // namespace gg
