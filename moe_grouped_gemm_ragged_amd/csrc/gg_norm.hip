// gg_norm.hip -- root-mean-square norm with the residual's addition, and its
// gradient: the step in front of a layer's grouped GEMMs.
//
//   h = x + residual,  rho = 1 / sqrt(mean(h^2) + eps),  y = h rho gamma
//
// y goes out as bf16, or as the fp8 forward's operand: e4m3 rows with one
// power-of-two scale per 128 values (gg_rows.h states the rule), or both.
// h stays in fp32 between the sum and the product; the bf16 copy written for
// the residual stream is rounded from it.
//
// Gradient, for p = dy gamma:
//
//   dx = rho (p - u mean(p u)) + dh,  u = h rho,     dgamma = sum over rows of dy u
//
// with dh the gradient that reaches h through the residual stream.  dx is
// the gradient of x and of residual alike.
//
// Both are bound by memory: one read of every operand, one write of every
// output, the row held in registers in between.  16384 x 7168 with a residual
// to h and e4m3 rows 150-160 us (5.1-5.5 TB/s; the counters show 824 MB moved,
// of 823 needed); the gradient of 8192 x 6144 with dh 74.5 + 4.8 us (5.1 TB/s;
// 409 MB of 403).  A single row of 2048 takes 2.7 us, which is one launch.
#include <hip/hip_runtime.h>
#include <stdint.h>

#include "gg_internal.h"
#include "gg_rows.h"

namespace gg {
namespace {

using namespace rows;

constexpr int kMaxThreads = 1024;
constexpr int kMaxWaves = kMaxThreads / 64;

// Sums over the T threads of a row (waves = T / 64; one wave needs no
// barrier).  red holds two buffers used in turn: a row's writes touch the one
// that the previous row did not read, and the row after it comes behind the
// next row's barrier.  A workgroup of several rows (blockDim.y) calls it
// together.
template <int N>
struct RowSums {
  float (*red)[N * kMaxWaves];
  int turn;
  __device__ __forceinline__ void operator()(float (&v)[N], int waves) {
#pragma unroll
    for (int i = 0; i < N; ++i) v[i] = wave_sum(v[i]);
    if (waves == 1) return;
    const int first = waves * threadIdx.y;
    float* r = red[turn] + first;
    turn ^= 1;
    if ((threadIdx.x & 63) == 0)
#pragma unroll
      for (int i = 0; i < N; ++i) r[i * kMaxWaves + (threadIdx.x >> 6)] = v[i];
    __syncthreads();
#pragma unroll
    for (int i = 0; i < N; ++i) v[i] = r[i * kMaxWaves];
    for (int w = 1; w < waves; ++w)
#pragma unroll
      for (int i = 0; i < N; ++i) v[i] += r[i * kMaxWaves + w];
  }
};

__device__ __forceinline__ void load_sum(const uint16_t* x, const uint16_t* res, int64_t at, float (&h)[8]) {
  unpack8(load16(x + at), h);
  if (res) {
    float r[8];
    unpack8(load16(res + at), r);
#pragma unroll
    for (int e = 0; e < 8; ++e) h[e] += r[e];
  }
}

struct NormOut {
  uint16_t* h;       // each may be null
  uint16_t* y;
  uint8_t* y8;
  uint8_t* scales;
};

// Group c (8 values at element `at`) of a row's outputs.  Where y8 is
// written, n is a multiple of 128, so 16-lane rows come here whole.
__device__ __forceinline__ void store_norm(const NormOut& out, const uint16_t* gamma, int64_t row, int64_t n, int c,
                                           const float (&h)[8], float rho) {
  const int64_t at = row * n + 8 * c;
  if (out.h) store16(out.h + at, pack8(h));
  float g[8], v[8];
  unpack8(load16(gamma + 8 * c), g);
#pragma unroll
  for (int e = 0; e < 8; ++e) v[e] = h[e] * rho * g[e];
  if (out.y) store16(out.y + at, pack8(v));
  if (out.y8) {
    int byte;
    store8(out.y8 + at, quantise8(v, byte));
    if ((c & 15) == 0) out.scales[row * (n / kBlock) + c / 16] = (uint8_t)byte;
  }
}

// One row per T = blockDim.x threads, blockDim.y rows a workgroup (more than
// one only where T is a single wave).  Thread t holds the 8-value groups t,
// t + T, ..., VPT of them.
template <int VPT>
__global__ __launch_bounds__(kMaxThreads) void rmsnorm_kernel(const uint16_t* x, const uint16_t* res,
                                                              const uint16_t* gamma, NormOut out, int64_t rows,
                                                              int64_t n, float eps) {
  __shared__ float red[2][kMaxWaves];
  RowSums<1> sums = {red, 0};
  const int T = blockDim.x;
  const int t = threadIdx.x;
  const int groups = (int)(n / 8);
  for (int64_t row = (int64_t)blockIdx.x * blockDim.y + threadIdx.y; row < rows;
       row += (int64_t)gridDim.x * blockDim.y) {
    float h[VPT][8];
    float s[1] = {0.f};
#pragma unroll
    for (int j = 0; j < VPT; ++j) {
      const int c = t + j * T;
#pragma unroll
      for (int e = 0; e < 8; ++e) h[j][e] = 0.f;
      if (c < groups) load_sum(x, res, row * n + 8 * c, h[j]);
#pragma unroll
      for (int e = 0; e < 8; ++e) s[0] += h[j][e] * h[j][e];
    }
    sums(s, T / 64);
    const float rho = 1.0f / sqrtf(s[0] / (float)n + eps);
#pragma unroll
    for (int j = 0; j < VPT; ++j)
      if (t + j * T < groups) store_norm(out, gamma, row, n, t + j * T, h[j], rho);
  }
}

// Rows too long for the registers: a workgroup reads each row twice.
__global__ __launch_bounds__(kMaxThreads) void rmsnorm_long_kernel(const uint16_t* x, const uint16_t* res,
                                                                   const uint16_t* gamma, NormOut out, int64_t rows,
                                                                   int64_t n, float eps) {
  __shared__ float red[2][kMaxWaves];
  RowSums<1> sums = {red, 0};
  const int groups = (int)(n / 8);
  for (int64_t row = blockIdx.x; row < rows; row += gridDim.x) {
    float s[1] = {0.f};
    for (int c = threadIdx.x; c < groups; c += kMaxThreads) {
      float h[8];
      load_sum(x, res, row * n + 8 * c, h);
#pragma unroll
      for (int e = 0; e < 8; ++e) s[0] += h[e] * h[e];
    }
    sums(s, kMaxWaves);
    const float rho = 1.0f / sqrtf(s[0] / (float)n + eps);
    for (int c = threadIdx.x; c < groups; c += kMaxThreads) {
      float h[8];
      load_sum(x, res, row * n + 8 * c, h);
      store_norm(out, gamma, row, n, c, h, rho);
    }
  }
}

// ---- gradient ------------------------------------------------------------------------

// A workgroup takes blockDim.y = Y rows at a time, T = blockDim.x threads
// each: workgroup b rows Y b .., Y (b + G) .., and so on.  Each slice keeps
// its share of dgamma in registers; at the end the slices are added in order
// and written to row b of the workspace: no atomics, so the sum's order is
// fixed.
template <int VPT>
__global__ __launch_bounds__(kMaxThreads) void rmsnorm_grad_kernel(const uint16_t* dy, const uint16_t* h,
                                                                   const uint16_t* gamma, const uint16_t* dh,
                                                                   uint16_t* dx, float* part, int64_t rows,
                                                                   int64_t n, float eps) {
  __shared__ float red[2][2 * kMaxWaves];
  __shared__ f32x4r slices[kMaxThreads * 2];
  RowSums<2> sums = {red, 0};
  const int T = blockDim.x, Y = blockDim.y;
  const int t = threadIdx.x, y = threadIdx.y;
  const int waves = T / 64;
  const int groups = (int)(n / 8);
  const float rn = 1.0f / (float)n;
  float dg[VPT][8];
  u32x4r gq[VPT];
#pragma unroll
  for (int j = 0; j < VPT; ++j) {
    const int c = t + j * T;
    gq[j] = u32x4r{0u, 0u, 0u, 0u};
    if (c < groups) gq[j] = load16(gamma + 8 * c);
#pragma unroll
    for (int e = 0; e < 8; ++e) dg[j][e] = 0.f;
  }
  // every slice goes through the loop equally often (the sums' barriers)
  for (int64_t first = (int64_t)blockIdx.x * Y; first < rows; first += (int64_t)gridDim.x * Y) {
    const int64_t row = first + y;
    const bool live = row < rows;
    u32x4r hq[VPT], dq[VPT], rq[VPT];
    float s[2] = {0.f, 0.f};
#pragma unroll
    for (int j = 0; j < VPT; ++j) {
      const int c = t + j * T;
      hq[j] = dq[j] = rq[j] = u32x4r{0u, 0u, 0u, 0u};
      if (live && c < groups) {
        hq[j] = load16(h + row * n + 8 * c);
        dq[j] = load16(dy + row * n + 8 * c);
        if (dh) rq[j] = load16(dh + row * n + 8 * c);
      }
    }
#pragma unroll
    for (int j = 0; j < VPT; ++j) {
      float hv[8], dv[8], gv[8];
      unpack8(hq[j], hv);
      unpack8(dq[j], dv);
      unpack8(gq[j], gv);
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        s[0] += hv[e] * hv[e];
        s[1] += dv[e] * gv[e] * hv[e];
      }
    }
    sums(s, waves);
    if (!live) continue;             // (eps may be 0: no 0 / 0 into the sums)
    const float rho = 1.0f / sqrtf(s[0] * rn + eps);
    const float m = s[1] * rn * rho;        // mean of p (h rho)
#pragma unroll
    for (int j = 0; j < VPT; ++j) {
      const int c = t + j * T;
      float hv[8], dv[8], gv[8], rv[8], o[8];
      unpack8(hq[j], hv);
      unpack8(dq[j], dv);
      unpack8(gq[j], gv);
      unpack8(rq[j], rv);
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        const float u = hv[e] * rho;
        o[e] = rho * (dv[e] * gv[e] - u * m) + rv[e];
        dg[j][e] += dv[e] * u;
      }
      if (c < groups) store16(dx + row * n + 8 * c, pack8(o));
    }
  }
#pragma unroll
  for (int j = 0; j < VPT; ++j) {
    const int c = t + j * T;
    f32x4r lo = {dg[j][0], dg[j][1], dg[j][2], dg[j][3]}, hi = {dg[j][4], dg[j][5], dg[j][6], dg[j][7]};
    if (Y > 1) {
      __syncthreads();               // the round before has been read
      slices[2 * (y * T + t)] = lo;
      slices[2 * (y * T + t) + 1] = hi;
      __syncthreads();
      if (y == 0)
        for (int z = 1; z < Y; ++z) {
          lo += slices[2 * (z * T + t)];
          hi += slices[2 * (z * T + t) + 1];
        }
    }
    if (y == 0 && c < groups) {
      float* p = part + (int64_t)blockIdx.x * n + 8 * c;
      *reinterpret_cast<f32x4r*>(p) = lo;
      *reinterpret_cast<f32x4r*>(p + 4) = hi;
    }
  }
}

// Rows too long for the registers: each row is read twice, and the
// workgroup's share of dgamma lives in its workspace row (every element is
// only ever touched by one thread).
__global__ __launch_bounds__(kMaxThreads) void rmsnorm_grad_long_kernel(const uint16_t* dy, const uint16_t* h,
                                                                        const uint16_t* gamma, const uint16_t* dh,
                                                                        uint16_t* dx, float* part, int64_t rows,
                                                                        int64_t n, float eps) {
  __shared__ float red[2][2 * kMaxWaves];
  RowSums<2> sums = {red, 0};
  const int t = threadIdx.x;
  const int groups = (int)(n / 8);
  const float rn = 1.0f / (float)n;
  float* mine = part + (int64_t)blockIdx.x * n;
  for (int64_t row = blockIdx.x; row < rows; row += gridDim.x) {
    float s[2] = {0.f, 0.f};
    for (int c = t; c < groups; c += kMaxThreads) {
      float hv[8], dv[8], gv[8];
      unpack8(load16(h + row * n + 8 * c), hv);
      unpack8(load16(dy + row * n + 8 * c), dv);
      unpack8(load16(gamma + 8 * c), gv);
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        s[0] += hv[e] * hv[e];
        s[1] += dv[e] * gv[e] * hv[e];
      }
    }
    sums(s, kMaxWaves);
    const float rho = 1.0f / sqrtf(s[0] * rn + eps);
    const float m = s[1] * rn * rho;        // mean of p (h rho)
    const bool first = row == blockIdx.x;
    for (int c = t; c < groups; c += kMaxThreads) {
      float hv[8], dv[8], gv[8], o[8];
      float rv[8] = {0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f};
      unpack8(load16(h + row * n + 8 * c), hv);
      unpack8(load16(dy + row * n + 8 * c), dv);
      unpack8(load16(gamma + 8 * c), gv);
      if (dh) unpack8(load16(dh + row * n + 8 * c), rv);
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        const float u = hv[e] * rho;
        o[e] = rho * (dv[e] * gv[e] - u * m) + rv[e];
        const float d = dv[e] * u;
        mine[8 * c + e] = first ? d : mine[8 * c + e] + d;
      }
      store16(dx + row * n + 8 * c, pack8(o));
    }
  }
}

// dgamma = the sum of the G workspace rows: 32 columns a workgroup, 32 row
// lanes of 4 columns a thread, the lanes added in order.  (G is at most 256,
// so a thread adds 8 rows: this is a matter of latency.)
__global__ __launch_bounds__(256) void rmsnorm_dgamma_kernel(const float* part, int G, int64_t n, float* dgamma) {
  __shared__ f32x4r lanes[32][8];
  const int c = threadIdx.x & 7, l = threadIdx.x >> 3;
  const int64_t col = (int64_t)blockIdx.x * 32 + 4 * c;
  f32x4r s = {0.f, 0.f, 0.f, 0.f};
  if (col < n) {
#pragma unroll 8
    for (int g = l; g < G; g += 32) s += *reinterpret_cast<const f32x4r*>(part + (int64_t)g * n + col);
  }
  lanes[l][c] = s;
  __syncthreads();
  // 32 threads: one column each
  const int64_t mine = (int64_t)blockIdx.x * 32 + threadIdx.x;
  if (threadIdx.x < 32 && mine < n) {
    float t = 0.f;
#pragma unroll
    for (int q = 0; q < 32; ++q) t += lanes[q][threadIdx.x >> 2][threadIdx.x & 3];
    dgamma[mine] = t;
  }
}

// Threads and 8-value groups per thread for a row of `groups` groups.
struct Shape {
  int threads, vpt;
};
Shape shape_of(int64_t groups) {
  int vpt = groups <= 64 ? 1 : groups <= 2048 ? 2 : 4;
  const int64_t t = ((groups + vpt - 1) / vpt + 63) / 64 * 64;
  return {(int)t, vpt};
}
// Longest rows the registers hold (the gradient, with its dgamma sums, holds
// half as much without spilling).
constexpr int64_t kLongRow = 8 * 4 * kMaxThreads;
constexpr int64_t kLongGradRow = 8 * 2 * kMaxThreads;

constexpr int64_t kMostBlocks = 1 << 20;   // a launch's threads stay below 2^32

// Threads of a workgroup of the gradient, in slices of a row each, and the
// most workgroups (workspace rows): one large workgroup a compute unit keeps
// the workspace small and still has its waves' loads in flight.  Both kernels
// together, 256 workgroups of 768 against 512 of 512 and 512 of a single slice:
// 8192 x 6144 with dh 78.0, 78.3 and 78.1 us, 16384 x 512 14.8, 15.5 and 26.8,
// 4096 x 2048 with dh 17.5, 16.0 and 18.9.
constexpr int kGradThreads = 768;
constexpr int kGradGroups = 256;
int grad_slices(int threads) { return threads >= kGradThreads ? 1 : kGradThreads / threads; }
int grad_groups(int64_t rows, int64_t n) {
  const int64_t per = n > kLongGradRow ? 1 : grad_slices(shape_of(n / 8).threads);
  const int64_t want = (rows + per - 1) / per;
  return (int)(want < kGradGroups ? want : kGradGroups);
}

}  // namespace

int64_t rmsnorm_grad_groups(int64_t rows, int64_t n) { return grad_groups(rows, n); }

hipError_t launch_rmsnorm(const void* x, const void* res, const void* gamma, void* h, void* y, void* y8,
                          void* scales, int64_t rows, int64_t n, float eps, hipStream_t stream) {
  if (rows == 0) return hipSuccess;
  const uint16_t* xp = static_cast<const uint16_t*>(x);
  const uint16_t* rp = static_cast<const uint16_t*>(res);
  const uint16_t* gp = static_cast<const uint16_t*>(gamma);
  const NormOut out = {static_cast<uint16_t*>(h), static_cast<uint16_t*>(y), static_cast<uint8_t*>(y8),
                       static_cast<uint8_t*>(scales)};
  const Shape s = shape_of(n / 8);
  const int per = s.threads == 64 ? 4 : 1;
  const int64_t want = (rows + per - 1) / per;
  const dim3 grid((unsigned)(want < kMostBlocks ? want : kMostBlocks)), block(s.threads, per);
  if (n > kLongRow)
    return launch_kernel(rmsnorm_long_kernel, grid, dim3(kMaxThreads), stream, xp, rp, gp, out, rows, n, eps);
  switch (s.vpt) {
    case 1: return launch_kernel(rmsnorm_kernel<1>, grid, block, stream, xp, rp, gp, out, rows, n, eps);
    case 2: return launch_kernel(rmsnorm_kernel<2>, grid, block, stream, xp, rp, gp, out, rows, n, eps);
    default: return launch_kernel(rmsnorm_kernel<4>, grid, block, stream, xp, rp, gp, out, rows, n, eps);
  }
}

hipError_t launch_rmsnorm_grad(const void* dy, const void* h, const void* gamma, const void* dh, void* dx,
                               float* dgamma, float* part, int64_t rows, int64_t n, float eps, hipStream_t stream) {
  const uint16_t* dp = static_cast<const uint16_t*>(dy);
  const uint16_t* hp = static_cast<const uint16_t*>(h);
  const uint16_t* gp = static_cast<const uint16_t*>(gamma);
  const uint16_t* rp = static_cast<const uint16_t*>(dh);
  uint16_t* xp = static_cast<uint16_t*>(dx);
  const int G = grad_groups(rows, n);
  if (G > 0) {
    hipError_t e;
    const Shape s = shape_of(n / 8);
    const dim3 block(s.threads, grad_slices(s.threads));
    if (n > kLongGradRow)
      e = launch_kernel(rmsnorm_grad_long_kernel, dim3(G), dim3(kMaxThreads), stream, dp, hp, gp, rp, xp, part, rows,
                        n, eps);
    else if (s.vpt == 1)
      e = launch_kernel(rmsnorm_grad_kernel<1>, dim3(G), block, stream, dp, hp, gp, rp, xp, part, rows, n,
                        eps);
    else
      e = launch_kernel(rmsnorm_grad_kernel<2>, dim3(G), block, stream, dp, hp, gp, rp, xp, part, rows, n,
                        eps);
    if (e != hipSuccess) return e;
  }
  return launch_kernel(rmsnorm_dgamma_kernel, dim3((unsigned)((n + 31) / 32)), dim3(256), stream, part, G, n, dgamma);
}

}  // namespace gg
