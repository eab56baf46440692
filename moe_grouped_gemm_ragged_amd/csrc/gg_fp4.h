// gg_fp4.h -- 4-bit rows: e2m1 codes with one power-of-two scale per 32
// values, the packed layout of those scales, and the row tiles of a layout.
//
// A code is OCP E2M1: sign, two exponent bits, one mantissa bit (0, 0.5, 1,
// 1.5, 2, 3, 4, 6); value 2 j of a row is the low half of its byte j.  A
// block is 32 consecutive values of a row.  Its scale is the smallest power
// of two s with amax / s <= 6, 1 for a block of zeros, never below 2^-126, as
// an E8M0 byte (exponent + 127); e2m1 has no infinity or NaN, so a block that
// holds one gets the byte 255 (NaN) and codes of 0.
//
// Packed scales.  The rows of an operand are cut into tiles of 256 (an
// expert's rows from its first one on), the reduction into stages of 128
// values.  Tile t, stage s takes 1024 bytes at (t * stages + s) * 1024; block
// q (0..3) of tile row r lies there at
//   512 (r / 128) + 16 (r mod 32) + 8 (q mod 2) + 4 (q / 2) + (r / 32) mod 4.
// The product's lane l reads 8 bytes for rows l mod 32 (+ 32 i, i = 0..3) and
// blocks l / 32 and 2 + l / 32: consecutive lanes' 8 bytes make up the 512 of
// a half tile, which keeps that read free of bank conflicts, and every 64
// consecutive bytes are 16 rows' scales of a whole stage, which is what a
// reader of few weight rows needs.
#pragma once
#include <hip/hip_runtime.h>
#include <stdint.h>

#include "gg_internal.h"
#include "gg_rows.h"
#include "gg_tiles.h"

namespace gg {
namespace fp4 {

constexpr int kBlock4 = 32;        // values per scale
constexpr int kStage4 = 128;       // values per stage
using tiles::kTileRows;
constexpr int kStageBytes = 1024;  // packed scales of a tile and stage

__host__ __device__ inline int64_t stages4(int64_t k) { return (k + kStage4 - 1) / kStage4; }

// Place of block q (0..3) of tile row r in a stage's 1024 bytes.
__device__ __forceinline__ int scale_place(int r, int q) {
  return 512 * (r >> 7) + 16 * (r & 31) + 8 * (q & 1) + 4 * (q >> 1) + ((r >> 5) & 3);
}

// Scale byte of a block whose largest magnitude has the bits amax (finite):
// 6 is 1.5 * 2^2.
__device__ __forceinline__ int scale_byte4(uint32_t amax) {
  int b = (int)(amax >> 23) - 2 + ((amax & 0x7FFFFFu) > 0x400000u ? 1 : 0);
  b = b < 1 ? 1 : b;
  return amax == 0u ? 127 : b;
}

// Largest of a lane's value over its group of 4 lanes.
__device__ __forceinline__ uint32_t quad_max(uint32_t v) {
  uint32_t o = (uint32_t)__builtin_amdgcn_update_dpp(0, (int)v, 0xB1, 0xf, 0xf, true);   // lane ^ 1
  v = o > v ? o : v;
  o = (uint32_t)__builtin_amdgcn_update_dpp(0, (int)v, 0x4E, 0xf, 0xf, true);            // lane ^ 2
  return o > v ? o : v;
}

// The largest magnitude of a lane's 8 values, as fp32 bits: the order of
// magnitudes is that of their bits, infinity and NaN on top.
__device__ __forceinline__ uint32_t magnitude(const rows::u32x4r& q) {      // bf16
  typedef uint16_t u16x2 __attribute__((ext_vector_type(2)));
  u16x2 m = __builtin_bit_cast(u16x2, q[0] & 0x7FFF7FFFu);
#pragma unroll
  for (int e = 1; e < 4; ++e) m = __builtin_elementwise_max(m, __builtin_bit_cast(u16x2, q[e] & 0x7FFF7FFFu));
  return (uint32_t)(m[0] > m[1] ? m[0] : m[1]) << 16;
}
__device__ __forceinline__ uint32_t magnitude(const float (&v)[8]) {
  uint32_t m = 0;
#pragma unroll
  for (int e = 0; e < 8; ++e) {
    const uint32_t a = __builtin_bit_cast(uint32_t, v[e]) & 0x7FFFFFFFu;
    m = a > m ? a : m;
  }
  return m;
}

// The conversions divide by a power of two (exact) and round once, to nearest
// even.  (They take the scale's exponent bits alone.)
__device__ __forceinline__ uint32_t codes8(const rows::u32x4r& q, float s) {
  // (pairs by shuffles: a bit cast of a vector's element takes element 0, with
  // this compiler, whichever is named)
  typedef __bf16 bf16x8 __attribute__((ext_vector_type(8)));
  const bf16x8 b = __builtin_bit_cast(bf16x8, q);
  uint32_t w = 0;
  w = __builtin_amdgcn_cvt_scalef32_pk_fp4_bf16(w, __builtin_shufflevector(b, b, 0, 1), s, 0);
  w = __builtin_amdgcn_cvt_scalef32_pk_fp4_bf16(w, __builtin_shufflevector(b, b, 2, 3), s, 1);
  w = __builtin_amdgcn_cvt_scalef32_pk_fp4_bf16(w, __builtin_shufflevector(b, b, 4, 5), s, 2);
  return __builtin_amdgcn_cvt_scalef32_pk_fp4_bf16(w, __builtin_shufflevector(b, b, 6, 7), s, 3);
}
__device__ __forceinline__ uint32_t codes8(const float (&v)[8], float s) {
  uint32_t w = 0;
  w = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(w, v[0], v[1], s, 0);
  w = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(w, v[2], v[3], s, 1);
  w = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(w, v[4], v[5], s, 2);
  return __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(w, v[6], v[7], s, 3);
}

// The codes of this lane's 8 values and its block's scale byte.  All 4 lanes
// of a quad call it together; they hold one block.
template <typename V>
__device__ __forceinline__ uint32_t quantise4(const V& v, int& byte) {
  const uint32_t m = quad_max(magnitude(v));
  const bool bad = m >= 0x7F800000u;
  byte = bad ? 255 : scale_byte4(m);
  const uint32_t c = codes8(v, __builtin_bit_cast(float, (uint32_t)byte << 23));
  return bad ? 0u : c;
}

}  // namespace fp4
}  // namespace gg
