// gg_silu_rows.hip -- SiLU-mul on grouped rows with the rows kept in 8 bits,
// and its gradient.
//
// For a gate/up row h = [g | u] of 2 I values (gate columns first), with
// s = 1 / (1 + exp(-g)):
//
//   a = g s u
//   dg = da u s (1 + g (1 - s)),   du = da g s
//
// in an order that stays in fp32 wherever the gradient does (see product).
//
// The forward step writes a (bf16, or e4m3 rows with one power-of-two scale
// per 128 values: the fp8 down projection's operand) and can keep h in 8 bits
// for the backward step: 2 I + I / 64 bytes a row instead of 4 I.  The
// backward step reads h in either form and can form a again for the down
// projection's dW.
//
// Element by element and bound by memory: each lane takes 8 gate and the 8
// matching up values; 16 lanes are one 128-value block, so a block's largest
// value is found within a 16-lane row.  Rows no expert owns (ragged: past the
// last end offset; masked: at or past masked_m[e]) are neither read nor
// written.  65536 rows, I 768: to e4m3 a and h 65.5 us (354 MB: 5.4 TB/s), the
// gradient from those rows with a again 94 us (504 MB: 5.4 TB/s); the counters
// show no other bytes.
#include <hip/hip_runtime.h>
#include <stdint.h>

#include "gg_internal.h"
#include "gg_rows.h"

namespace gg {
namespace {

using namespace rows;

constexpr int kThreads = 256;

// Walks the 8-value groups of [rows, groups] grid-stride without a division
// per step.
struct Walk {
  int64_t row;
  int group;
  int64_t row_step;
  int group_step;
  int groups;
  __device__ __forceinline__ Walk(int g) : groups(g) {
    const int64_t at = (int64_t)blockIdx.x * kThreads + threadIdx.x;
    const int64_t step = (int64_t)gridDim.x * kThreads;
    row = at / g;
    group = (int)(at - row * g);
    row_step = step / g;
    group_step = (int)(step - row_step * g);
  }
  __device__ __forceinline__ void next() {
    row += row_step;
    group += group_step;
    if (group >= groups) {
      group -= groups;
      ++row;
    }
  }
};

template <bool MASKED>
__device__ __forceinline__ bool owned(const int32_t* groups, int64_t m, int64_t end, int64_t row) {
  if constexpr (MASKED) {
    const uint32_t r = (uint32_t)row, e = r / (uint32_t)m;   // rows are below 2^31
    return (int32_t)(r - e * (uint32_t)m) < groups[e];
  } else {
    return row < end;
  }
}

__device__ __forceinline__ float sigmoid(float g) { return __builtin_amdgcn_rcpf(1.0f + __expf(-g)); }

// d u f for |f| < 1.1 (silu's derivative), where d u alone may leave fp32
// although the product does not: the larger of d and u takes f first, so that
// nothing underflows before its time, and f is halved on the way, so that
// nothing overflows either (both exact).  65536 rows, I 768: 92.8 us from kept
// rows, 92.2 with d u f from left to right, 109.1 and 110.1 from bf16 rows.
__device__ __forceinline__ float product(float d, float u, float f) {
  const bool first = fabsf(d) > fabsf(u);
  return (first ? d : u) * (0.5f * f) * (first ? u : d) * 2.0f;
}

struct SiluOut {
  uint16_t* a;        // each pair may be null
  uint8_t* a8;
  uint8_t* a8_scales;
  uint8_t* h8;
  uint8_t* h8_scales;
};

template <bool MASKED>
__global__ __launch_bounds__(kThreads) void silu_mul_rows_kernel(const uint16_t* h, const int32_t* groups, int32_t E,
                                                                 int64_t m, int64_t rows, int64_t width, SiluOut out) {
  const int64_t end = MASKED ? rows : owned_rows(groups, E, rows);
  const int64_t kb = width / kBlock;
  for (Walk w((int)(width / 8)); w.row < end; w.next()) {
    if (!owned<MASKED>(groups, m, end, w.row)) continue;
    const int64_t at = w.row * 2 * width + 8 * w.group;
    float g[8], u[8], a[8];
    unpack8(load16(h + at), g);
    unpack8(load16(h + at + width), u);
#pragma unroll
    for (int e = 0; e < 8; ++e) a[e] = g[e] * sigmoid(g[e]) * u[e];
    const int64_t to = w.row * width + 8 * w.group;
    if (out.a) store16(out.a + to, pack8(a));
    const bool lead = (w.group & 15) == 0;
    int byte;
    if (out.a8) {
      store8(out.a8 + to, quantise8(a, byte));
      if (lead) out.a8_scales[w.row * kb + w.group / 16] = (uint8_t)byte;
    }
    if (out.h8) {
      store8(out.h8 + at, quantise8(g, byte));
      if (lead) out.h8_scales[w.row * 2 * kb + w.group / 16] = (uint8_t)byte;
      store8(out.h8 + at + width, quantise8(u, byte));
      if (lead) out.h8_scales[w.row * 2 * kb + kb + w.group / 16] = (uint8_t)byte;
    }
  }
}

template <bool MASKED, bool H8>
__global__ __launch_bounds__(kThreads) void silu_mul_grad_kernel(const uint16_t* da, const void* h,
                                                                 const uint8_t* h_scales, const int32_t* groups,
                                                                 int32_t E, int64_t m, int64_t rows, int64_t width,
                                                                 uint16_t* dh, uint16_t* act) {
  // g and u of kept rows are carried halved: a value from 2^128 - 2^123 on is
  // kept as 2^128, which fp32 does not hold
  constexpr float kUnit = H8 ? 0.5f : 1.0f, kUnits = 1.0f / kUnit;
  const int64_t end = MASKED ? rows : owned_rows(groups, E, rows);
  const int64_t kb = width / kBlock;
  for (Walk w((int)(width / 8)); w.row < end; w.next()) {
    if (!owned<MASKED>(groups, m, end, w.row)) continue;
    const int64_t at = w.row * 2 * width + 8 * w.group;
    const int64_t to = w.row * width + 8 * w.group;
    float g[8], u[8], d[8];
    unpack8(load16(da + to), d);
    if constexpr (H8) {
      const uint8_t* p = static_cast<const uint8_t*>(h) + at;
      const uint8_t* s = h_scales + w.row * 2 * kb + w.group / 16;
      dequantise8(*reinterpret_cast<const u32x2r*>(p), scale_value(s[0]) * kUnit, g);
      dequantise8(*reinterpret_cast<const u32x2r*>(p + width), scale_value(s[kb]) * kUnit, u);
    } else {
      const uint16_t* p = static_cast<const uint16_t*>(h) + at;
      unpack8(load16(p), g);
      unpack8(load16(p + width), u);
    }
    float dg[8], du[8], a[8];
#pragma unroll
    for (int e = 0; e < 8; ++e) {
      const float s = sigmoid(g[e] * kUnits);
      const float gs = g[e] * s;
      a[e] = gs * u[e] * (kUnits * kUnits);
      du[e] = d[e] * gs * kUnits;
      // (g s, not g, times 1 - s: g may be infinite where s is 0)
      dg[e] = product(d[e], u[e], s + gs * (1.0f - s) * kUnits) * kUnits;
    }
    store16(dh + at, pack8(dg));
    store16(dh + at + width, pack8(du));
    if (act) store16(act + to, pack8(a));
  }
}

int grid_for(int64_t rows, int64_t width, int num_cus) {
  const int64_t want = (rows * (width / 8) + kThreads - 1) / kThreads;
  const int64_t most = 16 * (int64_t)num_cus;
  return (int)(want < most ? want : most);
}

}  // namespace

hipError_t launch_silu_mul_rows(bool masked, const void* h, const int32_t* groups, int32_t E, int64_t m,
                                int64_t width, void* a, void* a8, void* a8_scales, void* h8, void* h8_scales,
                                int num_cus, hipStream_t stream) {
  const int64_t rows = masked ? E * m : m;
  if (rows == 0) return hipSuccess;
  const SiluOut out = {static_cast<uint16_t*>(a), static_cast<uint8_t*>(a8), static_cast<uint8_t*>(a8_scales),
                       static_cast<uint8_t*>(h8), static_cast<uint8_t*>(h8_scales)};
  auto* kernel = masked ? silu_mul_rows_kernel<true> : silu_mul_rows_kernel<false>;
  return launch_kernel(kernel, dim3(grid_for(rows, width, num_cus)), dim3(kThreads), stream,
                       static_cast<const uint16_t*>(h), groups, E, m, rows, width, out);
}

hipError_t launch_silu_mul_grad(bool masked, const void* da, const void* h, const void* h_scales,
                                const int32_t* groups, int32_t E, int64_t m, int64_t width, void* dh, void* act,
                                int num_cus, hipStream_t stream) {
  const int64_t rows = masked ? E * m : m;
  if (rows == 0) return hipSuccess;
  auto* kernel = h_scales ? (masked ? silu_mul_grad_kernel<true, true> : silu_mul_grad_kernel<false, true>)
                          : (masked ? silu_mul_grad_kernel<true, false> : silu_mul_grad_kernel<false, false>);
  return launch_kernel(kernel, dim3(grid_for(rows, width, num_cus)), dim3(kThreads), stream,
                       static_cast<const uint16_t*>(da), h, static_cast<const uint8_t*>(h_scales), groups, E, m, rows,
                       width, static_cast<uint16_t*>(dh), static_cast<uint16_t*>(act));
}

}  // namespace gg
