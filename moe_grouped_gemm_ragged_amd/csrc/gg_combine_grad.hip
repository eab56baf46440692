// gg_combine_grad.hip -- the gradient of bringing expert rows back to tokens.
//
//   out[t] = sum_k w[t, k] y[row(t, k)]      (gg_combine_rows)
//
//   dy[row(t, k)] = w[t, k] dout[t]          zero on padding rows
//   dw[t, k] = <y[row(t, k)], dout[t]>       zero for a dropped slot
//
// Bound by memory: y is read and dy written once per slot, dout once per
// token.  So one workgroup takes a token: dout[t] is in registers while its
// topk rows are read and written, instead of being fetched again for every
// row (topk times the bytes, if rows were the unit of work).  Padding rows
// belong to no token; a few more workgroups look for them in row_slot.  8192
// tokens, 8 slots each, n 2048: 114 us (571 MB needed, 577 moved: 5.0 TB/s);
// 777 tokens, 5 slots, n 1016: 6.4 us.
#include <hip/hip_runtime.h>
#include <stdint.h>

#include "gg_internal.h"
#include "gg_rows.h"

namespace gg {
namespace {

using namespace rows;

constexpr int kThreads = 256;
constexpr int kWaves = kThreads / 64;
constexpr int kSlots = 8;      // slots of a token taken together

template <bool F32>
__device__ __forceinline__ void load_dout(const void* dout, int64_t at, float (&v)[8]) {
  if constexpr (F32) {
    const float* p = static_cast<const float*>(dout) + at;
    const f32x4r lo = *reinterpret_cast<const f32x4r*>(p), hi = *reinterpret_cast<const f32x4r*>(p + 4);
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      v[e] = lo[e];
      v[4 + e] = hi[e];
    }
  } else {
    unpack8(load16(static_cast<const uint16_t*>(dout) + at), v);
  }
}

// Workgroups [0, token_blocks) take tokens, the rest padding rows.
template <bool F32>
__global__ __launch_bounds__(kThreads) void combine_rows_grad_kernel(
    const void* dout, const uint16_t* y, const int32_t* slot_row, const int32_t* row_slot, const int32_t* offs,
    int32_t E, const float* w, int32_t topk, int64_t tokens, int64_t rows_cap, int64_t n, uint16_t* dy, float* dw,
    int32_t token_blocks) {
  __shared__ float red[2][kSlots][kWaves];
  const int t = threadIdx.x, T = blockDim.x;
  const int waves = T / 64;
  const int groups = (int)(n / 8);
  if ((int)blockIdx.x < token_blocks) {
    int turn = 0;
    for (int64_t token = blockIdx.x; token < tokens; token += token_blocks) {
      for (int k0 = 0; k0 < topk; k0 += kSlots) {
        int32_t row[kSlots];
        float wk[kSlots], dot[kSlots];
#pragma unroll
        for (int k = 0; k < kSlots; ++k) {
          row[k] = -1;
          wk[k] = 1.0f;
          dot[k] = 0.f;
          if (k0 + k < topk) {
            const int32_t r = slot_row[token * topk + k0 + k];
            row[k] = r < rows_cap ? r : -1;
            if (w) wk[k] = w[token * topk + k0 + k];
          }
        }
        for (int c = t; c < groups; c += T) {
          u32x4r q[kSlots];
          if (dw) {
#pragma unroll
            for (int k = 0; k < kSlots; ++k)
              if (row[k] >= 0) q[k] = load16(y + (int64_t)row[k] * n + 8 * c);
          }
          float d[8];
          load_dout<F32>(dout, token * n + 8 * c, d);
#pragma unroll
          for (int k = 0; k < kSlots; ++k) {
            if (row[k] < 0) continue;
            if (dw) {
              float v[8];
              unpack8(q[k], v);
#pragma unroll
              for (int e = 0; e < 8; ++e) dot[k] += v[e] * d[e];
            }
            float o[8];
#pragma unroll
            for (int e = 0; e < 8; ++e) o[e] = wk[k] * d[e];
            store16(dy + (int64_t)row[k] * n + 8 * c, pack8(o));
          }
        }
        if (dw) {
          // two buffers in turn: see RowSums in gg_norm.hip for why one barrier is enough
          float (*r)[kWaves] = red[turn];
          turn ^= 1;
#pragma unroll
          for (int k = 0; k < kSlots; ++k) {
            dot[k] = wave_sum(dot[k]);
            if ((t & 63) == 0) r[k][t >> 6] = dot[k];
          }
          __syncthreads();
          if (t < kSlots && k0 + t < topk) {
            float s = r[t][0];
            for (int v = 1; v < waves; ++v) s += r[t][v];
            dw[token * topk + k0 + t] = s;
          }
        }
      }
    }
    return;
  }
  // padding rows: row_slot names no slot below the last end offset
  const int64_t end = owned_rows(offs, E, rows_cap);
  const int64_t slots = tokens * topk;
  const int lane = t & 63;
  const int64_t first = ((int64_t)(blockIdx.x - token_blocks) * waves + (t >> 6)) * 64;
  for (int64_t base = first; base < end; base += (int64_t)(gridDim.x - token_blocks) * waves * 64) {
    const int64_t r = base + lane;
    int32_t s = 0;
    if (r < end) s = row_slot[r];
    uint64_t pad = __ballot(r < end && (s < 0 || s >= slots));
    while (pad) {
      const int b = __builtin_ctzll(pad);
      pad &= pad - 1;
      for (int c = lane; c < groups; c += 64) store16(dy + (base + b) * n + 8 * c, u32x4r{0u, 0u, 0u, 0u});
    }
  }
}

}  // namespace

hipError_t launch_combine_rows_grad(const void* dout, bool dout_f32, const void* y, const int32_t* slot_row,
                                    const int32_t* row_slot, const int32_t* offs, int32_t E, const float* w,
                                    int32_t topk, int64_t tokens, int64_t rows_cap, int64_t n, void* dy, float* dw,
                                    int num_cus, hipStream_t stream) {
  const int64_t groups = n / 8;
  const int threads = groups >= kThreads ? kThreads : (int)((groups + 63) / 64 * 64);
  const int64_t most = 1 << 20;
  const int token_blocks = (int)(tokens < most ? tokens : most);
  const int64_t scan = (rows_cap + threads - 1) / threads;
  const int pad_blocks = (int)(scan < num_cus ? scan : num_cus);
  if (token_blocks + pad_blocks == 0) return hipSuccess;
  const dim3 grid(token_blocks + pad_blocks), block(threads);
  const uint16_t* yp = static_cast<const uint16_t*>(y);
  uint16_t* dp = static_cast<uint16_t*>(dy);
  if (dout_f32)
    return launch_kernel(combine_rows_grad_kernel<true>, grid, block, stream, dout, yp, slot_row, row_slot, offs, E, w,
                         topk, tokens, rows_cap, n, dp, dw, token_blocks);
  return launch_kernel(combine_rows_grad_kernel<false>, grid, block, stream, dout, yp, slot_row, row_slot, offs, E, w,
                       topk, tokens, rows_cap, n, dp, dw, token_blocks);
}

}  // namespace gg
