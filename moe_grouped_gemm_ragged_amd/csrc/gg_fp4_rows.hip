// gg_fp4_rows.hip -- bf16 rows to 4 bits and back (see gg_fp4.h for the rows
// and the packed layout of their scales).
//
//   plain    codes of x's rows
//   gather   codes of token rows sorted by expert, zero codes and the scale 1
//            for a padding row
//   silu     codes of a = silu(g) u of gate/up rows h = [g | u]
//   back     code * scale, in bf16
//   pack     scale bytes [rows, k / 32], as a checkpoint holds them, to the
//            packed layout
//
// All of them walk units of half a tile (128 rows) by two stages (256
// values): the unit's scales are then 1024 bytes of the packed layout that
// one workgroup assembles in LDS and writes whole, where rows one at a time
// would write single bytes 1 KB apart.  A row's part of a unit is 512 bytes
// of bf16 and 128 of codes, 32 lanes with 8 values each; 4 lanes hold a
// block, so its largest value is two lane exchanges away.
//
// Bound by memory: 65536 rows of 2048 values 72 us (339 MB: 4.7 TB/s; a copy 5.05),
// back 61 us (5.5 TB/s), 64 x 1536 rows of weights 99 and 96 us, silu of 65536
// rows to 768 values 53 us (229 MB).  gather, 8192 tokens of 2048 values to 8 of
// 128 experts: 47 us (33.5 MB in, 71 out, a token read for each of its rows);
// with a row's slot read by every thread as it needs it 91.
#include <hip/hip_runtime.h>
#include <stdint.h>

#include "gg_fp4.h"
#include "gg_internal.h"
#include "gg_rows.h"
#include "gg_tiles.h"

namespace gg {
namespace {

using namespace rows;
using namespace fp4;
using namespace tiles;

constexpr int kHalf = 128;           // rows of a unit
constexpr int kRowsAtOnce = 8;       // of them at a time: 32 lanes each
constexpr int kUnitStages = 2;

enum Source { PLAIN = 0, GATHER = 1, SILU = 2 };

__device__ __forceinline__ int64_t uniform64(int64_t v) {
  const uint32_t lo = (uint32_t)__builtin_amdgcn_readfirstlane((int)(uint32_t)v);
  const uint32_t hi = (uint32_t)__builtin_amdgcn_readfirstlane((int)(uint32_t)((uint64_t)v >> 32));
  return (int64_t)((uint64_t)hi << 32 | lo);
}

struct In {
  const uint16_t* x;         // plain: rows; gather: token rows; silu: gate/up rows of 2 k values
  const int32_t* row_slot;   // gather
  int32_t topk;
  int64_t tokens;
};

__device__ __forceinline__ float sigmoid(float g) { return __builtin_amdgcn_rcpf(1.0f + __expf(-g)); }

template <int LAYOUT, int SRC>
__global__ __launch_bounds__(kThreads) void to4_kernel(In in, const int32_t* groups, int64_t rows, int64_t k, int32_t E,
                                                       int64_t tiles, uint8_t* codes, uint8_t* scales) {
  __shared__ std::conditional_t<LAYOUT == RAGGED, Tiles, NoTiles> s_tiles;
  __shared__ uint32_t s_sc[kUnitStages * kStageBytes / 2 / 4];     // [stage][half tile]
  __shared__ int32_t s_token[SRC == GATHER ? kHalf : 1];
  const int tid = threadIdx.x;
  if constexpr (LAYOUT == RAGGED) tiles = decode_tiles(s_tiles, groups, rows, E, tid);
  const int64_t stages = stages4(k);
  const int64_t across = (stages + kUnitStages - 1) / kUnitStages;
  const int lane = tid & 31, rsub = tid >> 5;
  uint8_t* const my = reinterpret_cast<uint8_t*>(s_sc) + 512 * (lane >> 4);
  const int q = (lane & 15) >> 2;
  // Units in the order of their rows; gather: of their columns, an eighth of that
  // list to each XCD (workgroup b runs on XCD b mod 8), so that a token's piece
  // comes from memory once and its other rows find it in the XCD's L2.
  const int64_t units = 2 * tiles * across;
  const bool by_xcd = SRC == GATHER && gridDim.x % 8 == 0;
  const int64_t x = by_xcd ? blockIdx.x % 8 : 0, each = by_xcd ? 8 : 1;
  const int64_t end = by_xcd ? units * (x + 1) / 8 : units;
  for (int64_t u = (by_xcd ? units * x / 8 : 0) + blockIdx.x / each; u < end; u += gridDim.x / each) {
    const int64_t th = SRC == GATHER ? u % (2 * tiles) : u / across;
    const int64_t s0 = (SRC == GATHER ? u / (2 * tiles) : u - th * across) * kUnitStages;
    const int half = (int)(th & 1);
    int64_t first;
    int valid;
    tile_rows<LAYOUT>(s_tiles, groups, rows, E, th >> 1, first, valid);
    if (valid <= 0) continue;                    // (masked: a tile without rows)
    valid = __builtin_amdgcn_readfirstlane(valid) - kHalf * half;
    first = uniform64(first) + kHalf * half;
    const int64_t col = s0 * kStage4 + 8 * lane;
    // (a unit's rows span 2^29 bytes at most: 32-bit offsets from a scalar base)
    const uint32_t pitch = 2u * (uint32_t)k;
    const uint8_t* const from =
        reinterpret_cast<const uint8_t*>(in.x + (SRC == GATHER ? 0 : (SRC == SILU ? 2 : 1) * first * k)) +
        2 * s0 * kStage4;
    uint8_t* const to = codes + first * (k / 2) + s0 * kStage4 / 2;
    const uint32_t lane16 = 16u * (uint32_t)lane;
    s_sc[tid] = 0u;
    if constexpr (SRC == GATHER) {
      // the rows' tokens (-1: padding)
      if (tid < valid && tid < kHalf) {
        const int32_t slot = in.row_slot[first + tid], t = slot / in.topk;
        s_token[tid] = slot < 0 || t >= in.tokens ? -1 : t;
      }
    }
    __syncthreads();
    if (col < k) {
      constexpr int kAhead = 4;
      for (int r0 = rsub; r0 < valid && r0 < kHalf; r0 += kRowsAtOnce * kAhead) {
        u32x4r g[kAhead], up[SRC == SILU ? kAhead : 1];
#pragma unroll
        for (int a = 0; a < kAhead; ++a) {
          const int r = r0 + kRowsAtOnce * a;
          g[a] = u32x4r{0u, 0u, 0u, 0u};
          if (r < valid && r < kHalf) {
            if constexpr (SRC == PLAIN) {
              g[a] = load16(from + (lane16 + (uint32_t)r * pitch));
            } else if constexpr (SRC == SILU) {
              g[a] = load16(from + (lane16 + (uint32_t)r * 2u * pitch));
              up[a] = load16(from + (lane16 + ((uint32_t)r * 2u + 1u) * pitch));
            } else {
              const int32_t t = s_token[r];
              if (t >= 0) g[a] = load16(from + ((uint64_t)(uint32_t)t * pitch + lane16));
            }
          }
        }
#pragma unroll
        for (int a = 0; a < kAhead; ++a) {
          const int r = r0 + kRowsAtOnce * a;
          if (r < valid && r < kHalf) {
            int byte;
            uint32_t c;
            if constexpr (SRC == SILU) {
              float v[8], w[8];
              unpack8(g[a], v);
              unpack8(up[a], w);
#pragma unroll
              for (int e = 0; e < 8; ++e) v[e] = v[e] * sigmoid(v[e]) * w[e];
              c = quantise4(v, byte);
            } else {
              c = quantise4(g[a], byte);
            }
            *reinterpret_cast<uint32_t*>(to + (4u * (uint32_t)lane + (uint32_t)r * (pitch / 4))) = c;
            if ((lane & 3) == 0) my[scale_place(r, q)] = (uint8_t)byte;
          }
        }
      }
    }
    __syncthreads();
    const int64_t st = s0 + (tid >> 7);
    if (st < stages)
      reinterpret_cast<uint32_t*>(scales + ((th >> 1) * stages + st) * kStageBytes + 512 * half)[tid & 127] = s_sc[tid];
    __syncthreads();
  }
}

template <int LAYOUT>
__global__ __launch_bounds__(kThreads) void from4_kernel(const uint8_t* codes, const uint8_t* scales,
                                                         const int32_t* groups, int64_t rows, int64_t k, int32_t E,
                                                         int64_t tiles, uint16_t* out) {
  __shared__ std::conditional_t<LAYOUT == RAGGED, Tiles, NoTiles> s_tiles;
  __shared__ uint32_t s_sc[kUnitStages * kStageBytes / 2 / 4];
  const int tid = threadIdx.x;
  if constexpr (LAYOUT == RAGGED) tiles = decode_tiles(s_tiles, groups, rows, E, tid);
  const int64_t stages = stages4(k);
  const int64_t across = (stages + kUnitStages - 1) / kUnitStages;
  const int lane = tid & 31, rsub = tid >> 5;
  const uint8_t* const my = reinterpret_cast<const uint8_t*>(s_sc) + 512 * (lane >> 4);
  const int q = (lane & 15) >> 2;
  for (int64_t u = blockIdx.x; u < 2 * tiles * across; u += gridDim.x) {
    const int64_t th = u / across;
    const int64_t s0 = (u - th * across) * kUnitStages;
    const int half = (int)(th & 1);
    int64_t first;
    int valid;
    tile_rows<LAYOUT>(s_tiles, groups, rows, E, th >> 1, first, valid);
    valid -= kHalf * half;
    first += kHalf * half;
    if (valid <= 0) continue;
    const int64_t col = s0 * kStage4 + 8 * lane;
    const int64_t st = s0 + (tid >> 7);
    if (st < stages)
      s_sc[tid] =
          reinterpret_cast<const uint32_t*>(scales + ((th >> 1) * stages + st) * kStageBytes + 512 * half)[tid & 127];
    __syncthreads();
    if (col < k) {
      constexpr int kAhead = 4;
      for (int r0 = rsub; r0 < valid && r0 < kHalf; r0 += kRowsAtOnce * kAhead) {
        uint32_t c[kAhead];
#pragma unroll
        for (int a = 0; a < kAhead; ++a) {
          const int r = r0 + kRowsAtOnce * a;
          c[a] = 0u;
          if (r < valid && r < kHalf) c[a] = *reinterpret_cast<const uint32_t*>(codes + (first + r) * (k / 2) + col / 2);
        }
#pragma unroll
        for (int a = 0; a < kAhead; ++a) {
          const int r = r0 + kRowsAtOnce * a;
          if (r < valid && r < kHalf) {
            // the conversion takes the scale's exponent bits alone, as an E8M0 byte
            const float s = __builtin_bit_cast(float, (uint32_t)my[scale_place(r, q)] << 23);
            u32x4r o;
            o[0] = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(c[a], s, 0));
            o[1] = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(c[a], s, 1));
            o[2] = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(c[a], s, 2));
            o[3] = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(c[a], s, 3));
            store16(out + (first + r) * k + col, o);
          }
        }
      }
    }
    __syncthreads();
  }
}

// Thread t writes dword t of a unit: the 4 rows of its place, one block.
template <int LAYOUT>
__global__ __launch_bounds__(kThreads) void pack4_kernel(const uint8_t* src, int64_t ld_src, const int32_t* groups,
                                                         int64_t rows, int64_t k, int32_t E, int64_t tiles,
                                                         uint8_t* scales) {
  __shared__ std::conditional_t<LAYOUT == RAGGED, Tiles, NoTiles> s_tiles;
  const int tid = threadIdx.x;
  if constexpr (LAYOUT == RAGGED) tiles = decode_tiles(s_tiles, groups, rows, E, tid);
  const int64_t stages = stages4(k), blocks = k / kBlock4;
  const int64_t across = (stages + kUnitStages - 1) / kUnitStages;
  const int d = tid & 127;
  for (int64_t u = blockIdx.x; u < 2 * tiles * across; u += gridDim.x) {
    const int64_t th = u / across;
    const int64_t st = (u - th * across) * kUnitStages + (tid >> 7);
    const int half = (int)(th & 1);
    int64_t first;
    int valid;
    tile_rows<LAYOUT>(s_tiles, groups, rows, E, th >> 1, first, valid);
    if (valid <= 0 || st >= stages) continue;
    const int64_t b = 4 * st + 2 * (d & 1) + ((d >> 1) & 1);
    uint32_t word = 0;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const int r = kHalf * half + (d >> 2) + 32 * i;
      if (r < valid && b < blocks) word |= (uint32_t)src[(first + r) * ld_src + b] << (8 * i);
    }
    reinterpret_cast<uint32_t*>(scales + ((th >> 1) * stages + st) * kStageBytes + 512 * half)[d] = word;
  }
}

// Workgroups a compute unit.  To 4 bits 6, as many as its registers hold at once but
// for silu's 5 (8: the last begin when others end, and have as much to do: gather 55
// us against 47, weights 105 against 99; 4: 57 and 99).  Back 5: weights 96 us, with 8
// of them 104, with 6 105; 65536 rows 61.5, 60 and 61.
constexpr int kToGroups = 6, kFromGroups = 5;

int grid_for(int64_t tiles, int64_t k, int num_cus, int each) {
  const int64_t units = 2 * tiles * ((stages4(k) + kUnitStages - 1) / kUnitStages);
  const int64_t most = each * (int64_t)num_cus;
  return (int)(units < most ? units : most);
}

template <int LAYOUT>
hipError_t to4(const In& in, const int32_t* groups, int64_t rows, int64_t k, int32_t E, void* codes, void* scales,
               int num_cus, hipStream_t stream) {
  const int64_t tiles = fp4_scale_tiles(LAYOUT, rows, E);
  auto* kernel = to4_kernel<LAYOUT, PLAIN>;
  return launch_kernel(kernel, dim3(grid_for(tiles, k, num_cus, kToGroups)), dim3(kThreads), stream, in, groups, rows,
                       k, E, tiles, static_cast<uint8_t*>(codes), static_cast<uint8_t*>(scales));
}

}  // namespace

int64_t fp4_scale_tiles(int layout, int64_t rows, int32_t num_groups) {
  const int64_t t = (rows + kTileRows - 1) / kTileRows;
  return layout == RAGGED ? t + num_groups : t * num_groups;
}

hipError_t launch_fp4_quantize(int layout, const void* x, const int32_t* groups, int64_t rows, int64_t k, int32_t E,
                               void* codes, void* scales, int num_cus, hipStream_t stream) {
  if (rows == 0) return hipSuccess;
  const In in = {static_cast<const uint16_t*>(x), nullptr, 1, 0};
  switch (layout) {
    case RAGGED: return to4<RAGGED>(in, groups, rows, k, E, codes, scales, num_cus, stream);
    case MASKED_ROWS: return to4<MASKED_ROWS>(in, groups, rows, k, E, codes, scales, num_cus, stream);
    default: return to4<WEIGHTS>(in, groups, rows, k, E, codes, scales, num_cus, stream);
  }
}

hipError_t launch_fp4_gather_rows(const void* src, int64_t tokens, int64_t k, const int32_t* row_slot, int32_t topk,
                                  const int32_t* offs, int32_t E, int64_t rows_cap, void* codes, void* scales,
                                  int num_cus, hipStream_t stream) {
  if (rows_cap == 0) return hipSuccess;
  const In in = {static_cast<const uint16_t*>(src), row_slot, topk, tokens};
  const int64_t tiles = fp4_scale_tiles(RAGGED, rows_cap, E);
  return launch_kernel(to4_kernel<RAGGED, GATHER>, dim3(grid_for(tiles, k, num_cus, kToGroups)), dim3(kThreads),
                       stream, in, offs, rows_cap, k, E, tiles, static_cast<uint8_t*>(codes),
                       static_cast<uint8_t*>(scales));
}

hipError_t launch_fp4_silu_mul_rows(bool masked, const void* h, const int32_t* groups, int32_t E, int64_t m,
                                    int64_t width, void* codes, void* scales, int num_cus, hipStream_t stream) {
  if (m == 0) return hipSuccess;
  const In in = {static_cast<const uint16_t*>(h), nullptr, 1, 0};
  const int layout = masked ? MASKED_ROWS : RAGGED;
  const int64_t tiles = fp4_scale_tiles(layout, m, E);
  auto* kernel = masked ? to4_kernel<MASKED_ROWS, SILU> : to4_kernel<RAGGED, SILU>;
  return launch_kernel(kernel, dim3(grid_for(tiles, width, num_cus, kToGroups)), dim3(kThreads), stream, in, groups, m,
                       width, E, tiles, static_cast<uint8_t*>(codes), static_cast<uint8_t*>(scales));
}

hipError_t launch_fp4_dequantize(int layout, const void* codes, const void* scales, const int32_t* groups, int64_t rows,
                                 int64_t k, int32_t E, void* out, int num_cus, hipStream_t stream) {
  if (rows == 0) return hipSuccess;
  const int64_t tiles = fp4_scale_tiles(layout, rows, E);
  auto* kernel = layout == RAGGED        ? from4_kernel<RAGGED>
                 : layout == MASKED_ROWS ? from4_kernel<MASKED_ROWS>
                                         : from4_kernel<WEIGHTS>;
  return launch_kernel(kernel, dim3(grid_for(tiles, k, num_cus, kFromGroups)), dim3(kThreads), stream,
                       static_cast<const uint8_t*>(codes), static_cast<const uint8_t*>(scales), groups, rows, k, E,
                       tiles, static_cast<uint16_t*>(out));
}

hipError_t launch_fp4_pack_scales(int layout, const void* src, int64_t ld_src, const int32_t* groups, int64_t rows,
                                  int64_t k, int32_t E, void* dst, int num_cus, hipStream_t stream) {
  if (rows == 0) return hipSuccess;
  const int64_t tiles = fp4_scale_tiles(layout, rows, E);
  auto* kernel = layout == RAGGED        ? pack4_kernel<RAGGED>
                 : layout == MASKED_ROWS ? pack4_kernel<MASKED_ROWS>
                                         : pack4_kernel<WEIGHTS>;
  return launch_kernel(kernel, dim3(grid_for(tiles, k, num_cus, kFromGroups)), dim3(kThreads), stream,
                       static_cast<const uint8_t*>(src), ld_src, groups, rows, k, E, tiles,
                       static_cast<uint8_t*>(dst));
}

}  // namespace gg
