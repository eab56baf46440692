// gg_rows.h -- device helpers shared by the row kernels (norm, SiLU-mul rows,
// 8-bit gather, combine gradient): bf16 vectors, sums and maxima across
// lanes, and e4m3 rows with one power-of-two scale per 128 values.
#pragma once
#include <hip/hip_runtime.h>
#include <stdint.h>

namespace gg {
namespace rows {

typedef uint32_t u32x4r __attribute__((ext_vector_type(4)));
typedef uint32_t u32x2r __attribute__((ext_vector_type(2)));
typedef float f32x2r __attribute__((ext_vector_type(2)));
typedef float f32x4r __attribute__((ext_vector_type(4)));
typedef __bf16 bf16x2r __attribute__((ext_vector_type(2)));

// 8 bf16 values (16 bytes) to fp32 and back, one round-to-nearest-even each.
__device__ __forceinline__ void unpack8(const u32x4r& q, float (&v)[8]) {
#pragma unroll
  for (int e = 0; e < 4; ++e) {
    v[2 * e] = __builtin_bit_cast(float, q[e] << 16);
    v[2 * e + 1] = __builtin_bit_cast(float, q[e] & 0xFFFF0000u);
  }
}

__device__ __forceinline__ u32x4r pack8(const float (&v)[8]) {
  u32x4r q;
#pragma unroll
  for (int e = 0; e < 4; ++e) {
    const f32x2r f = {v[2 * e], v[2 * e + 1]};
    q[e] = __builtin_bit_cast(uint32_t, __builtin_convertvector(f, bf16x2r));
  }
  return q;
}

__device__ __forceinline__ u32x4r load16(const void* p) { return *static_cast<const u32x4r*>(p); }

// Results go out past the L2 (non-temporal): they are larger than it in every
// call where bandwidth counts, and the operands still to be read keep their
// place.  Against ordinary stores: norm of 16384 x 7168 156 -> 153 us, its
// gradient at 8192 x 6144 88.9 -> 86.5, combine gradient 8192 x 8 x 2048 117 ->
// 115, SiLU-mul gradient of 65536 x 768 96.7 -> 93.7; rows that are no whole
// cache lines (n 1000, 2056, 7176) between 4 % faster and 6 % slower; the GEMM
// that reads them next is within 1 % either way.
__device__ __forceinline__ void store16(void* p, const u32x4r& v) {
  __builtin_nontemporal_store(v, static_cast<u32x4r*>(p));
}
__device__ __forceinline__ void store8(void* p, const u32x2r& v) {
  __builtin_nontemporal_store(v, static_cast<u32x2r*>(p));
}

// The value of the lane N places further round in the same 16-lane row.
template <int N>
__device__ __forceinline__ float row_ror(float v) {
  return __builtin_bit_cast(
      float, __builtin_amdgcn_update_dpp(0, __builtin_bit_cast(int, v), 0x120 + N, 0xf, 0xf, true));
}

// Maximum / sum over a 16-lane row, in every lane of it.
__device__ __forceinline__ float row_max(float v) {
  v = fmaxf(v, row_ror<8>(v));
  v = fmaxf(v, row_ror<4>(v));
  v = fmaxf(v, row_ror<2>(v));
  return fmaxf(v, row_ror<1>(v));
}
__device__ __forceinline__ float row_sum(float v) {
  v += row_ror<8>(v);
  v += row_ror<4>(v);
  v += row_ror<2>(v);
  return v + row_ror<1>(v);
}

__device__ __forceinline__ float lane_value(float v, int lane) {
  return __builtin_bit_cast(float, __builtin_amdgcn_readlane(__builtin_bit_cast(int, v), lane));
}

// Sum over the wave's 64 lanes (every lane active), the same in all of them.
__device__ __forceinline__ float wave_sum(float v) {
  v = row_sum(v);
  return (lane_value(v, 0) + lane_value(v, 16)) + (lane_value(v, 32) + lane_value(v, 48));
}

// ---- e4m3 with E8M0 block scales ---------------------------------------------------
//
// A block is 128 consecutive values of a row: 16 lanes with 8 values each.
// Its scale is the smallest power of two s with amax / s <= 448 (e4m3's
// largest value, 1.75 * 2^8), 1 for a block of zeros, never below 2^-126, as
// an E8M0 byte (exponent + 127).  The codes are v / s (exact: a power of
// two) rounded to nearest even.  amax is taken over the block's finite
// values; an infinity or NaN becomes the NaN code.

constexpr int kBlock = 128;

__device__ __forceinline__ int scale_byte(float amax) {
  const uint32_t a = __builtin_bit_cast(uint32_t, amax);
  int b = (int)(a >> 23) - 8 + ((a & 0x7FFFFFu) > 0x600000u ? 1 : 0);
  b = b < 1 ? 1 : b;
  return a == 0u ? 127 : b;
}

// 2^-(byte - 127); byte in [1, 253]
__device__ __forceinline__ float inverse_scale(int byte) {
  return __builtin_bit_cast(float, (uint32_t)(254 - byte) << 23);
}

// 2^(byte - 127): byte 0 is the denormal 2^-127, 255 (E8M0's NaN) is NaN
__device__ __forceinline__ float scale_value(uint32_t byte) {
  const uint32_t bits = byte == 0u ? 0x00400000u : byte == 255u ? 0x7FC00000u : byte << 23;
  return __builtin_bit_cast(float, bits);
}

__device__ __forceinline__ bool finite(float v) {
  return (__builtin_bit_cast(uint32_t, v) & 0x7F800000u) != 0x7F800000u;
}

// The codes of this lane's 8 values and its block's scale byte.  All 16
// lanes of a DPP row call it together, each row one block.
__device__ __forceinline__ u32x2r quantise8(const float (&v)[8], int& byte) {
  float m = 0.f;
#pragma unroll
  for (int e = 0; e < 8; ++e) m = fmaxf(m, fabsf(v[e]));   // fmaxf passes over NaN
  m = row_max(m);
  u32x2r q;
  if (__builtin_expect(finite(m), 1)) {
    byte = scale_byte(m);
    const float inv = inverse_scale(byte);
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      int w = __builtin_amdgcn_cvt_pk_fp8_f32(v[4 * h] * inv, v[4 * h + 1] * inv, 0, false);
      w = __builtin_amdgcn_cvt_pk_fp8_f32(v[4 * h + 2] * inv, v[4 * h + 3] * inv, w, true);
      q[h] = (uint32_t)w;
    }
    return q;
  }
  // an infinity in the block (the whole 16-lane row takes this path)
  m = 0.f;
#pragma unroll
  for (int e = 0; e < 8; ++e) m = fmaxf(m, finite(v[e]) ? fabsf(v[e]) : 0.f);
  m = row_max(m);
  byte = scale_byte(m);
  const float inv = inverse_scale(byte);
#pragma unroll
  for (int h = 0; h < 2; ++h) {
    uint32_t w = 0;
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      const float f = v[4 * h + e];
      const uint32_t c = (uint32_t)__builtin_amdgcn_cvt_pk_fp8_f32(finite(f) ? f * inv : 0.f, 0.f, 0, false) & 0xFFu;
      w |= (finite(f) ? c : 0x7Fu) << (8 * e);
    }
    q[h] = w;
  }
  return q;
}

// fp32 values of 8 codes times a scale.
__device__ __forceinline__ void dequantise8(const u32x2r& q, float scale, float (&v)[8]) {
#pragma unroll
  for (int h = 0; h < 2; ++h) {
    const f32x2r lo = __builtin_amdgcn_cvt_pk_f32_fp8((int)q[h], false);
    const f32x2r hi = __builtin_amdgcn_cvt_pk_f32_fp8((int)q[h], true);
    v[4 * h] = lo[0] * scale;
    v[4 * h + 1] = lo[1] * scale;
    v[4 * h + 2] = hi[0] * scale;
    v[4 * h + 3] = hi[1] * scale;
  }
}

// ---- rows of experts ------------------------------------------------------------------

// Rows of the ragged layout that experts own: the largest end offset,
// clamped to [0, rows] as the GEMMs clamp it.  Called by the whole wave.
__device__ __forceinline__ int64_t owned_rows(const int32_t* offs, int32_t E, int64_t rows) {
  int m = 0;
  for (int g = (int)(threadIdx.x & 63); g < E; g += 64) m = offs[g] > m ? offs[g] : m;
#pragma unroll
  for (int d = 32; d > 0; d >>= 1) {
    const int o = __shfl_xor(m, d, 64);
    m = o > m ? o : m;
  }
  return m < rows ? m : rows;
}

}  // namespace rows
}  // namespace gg
