// gg_few_tokens.hip -- a whole expert layer for a few tokens in two kernels.
//
//   out[t] = sum over the slots s of t of weight[s] W2[e] a,   e = expert[s],
//   a = silu(W1[e] x[t]) * (W3[e] x[t])
//
// with W13[e] = [W1[e]; W3[e]] [2 I, H] and W2[e] [H, I], reduction
// contiguous, in bf16 or in 4 bits with packed scales (gg_fp4.h).
//
// With a few tokens the layer is the reading of the experts that they reach:
// nothing else counts, so nothing is sorted, padded or gathered.  Each
// workgroup reads a strip of weight rows once, straight into registers (16
// bytes a lane, the reduction split over its waves), and multiplies it with
// all rows that need it: a lane's 8 consecutive weights are a matrix
// instruction's operand as they lie in memory, the rows are its other 16
// columns.  4-bit weights become bf16 in registers (exactly).
//
//   up kernel    a workgroup takes an expert and 16 columns of I: rows c of W1
//                and W3 against x of the tokens that chose the expert; writes
//                weight * a (bf16) to the workspace
//   down kernel  a workgroup takes 16 rows of every reached expert's W2 and
//                adds all experts' shares in its registers, so out is written
//                once, with no partial sums in memory
//
// Which experts are reached, and by whom, every workgroup of the up kernel
// finds by itself from the expert ids (at most 1024 slots); the first of each
// expert leaves it in the workspace for the down kernel.
#include <hip/hip_runtime.h>
#include <stdint.h>

#include "gg_fp4.h"
#include "gg_internal.h"
#include "gg_rows.h"

namespace gg {
namespace {

using namespace fp4;
using rows::u32x4r;

constexpr int kMaxTokens = kFewTokensMax;
constexpr int kMaxSlots = kFewSlotsMax;
constexpr int kStrip = 16;                    // weight rows of a workgroup (and columns of a matrix instruction)
constexpr int kUpWaves = 8, kDownWaves = 16;
constexpr int kPitch = kStrip + 1;            // floats between a token's strips in LDS

typedef __bf16 bf16x8f __attribute__((ext_vector_type(8)));
typedef float f32x4f __attribute__((ext_vector_type(4)));

// An expert that tokens reach: its index, the workspace row of its first
// token, and the tokens (bit t).
struct Reached {
  int32_t expert;
  int32_t base;
  uint64_t tokens;
};

struct Weights {
  const uint8_t* w;        // codes or bf16
  const uint8_t* scales;   // 4 bits: packed
  int64_t rows;            // of one expert
  int64_t k;
};

__device__ __forceinline__ int wave_index() { return __builtin_amdgcn_readfirstlane((int)(threadIdx.x >> 6)); }

// One reduction step of a wave: 64 bf16 or 128 4-bit values of each of the 16
// rows, as operands of its matrix instructions.  Lane l holds row l mod 16;
// operand j covers, of l / 16 = q,
//   bf16  values 32 j + 8 q .. + 7      (two operands)
//   4 bit values 32 q + 8 j .. + 7      (four)
template <bool FOUR>
struct Step {
  static constexpr int kValues = FOUR ? 128 : 64;
  static constexpr int kOperands = FOUR ? 4 : 2;
  static __device__ __forceinline__ int at(int q, int j) { return FOUR ? 32 * q + 8 * j : 32 * j + 8 * q; }
};

template <bool FOUR>
struct Raw {
  u32x4r v[FOUR ? 1 : 2];
  uint32_t scale;
};

// This lane's row of a strip.
template <bool FOUR>
struct Row {
  const uint8_t* w;
  const uint8_t* scales;
  int k;                                   // values that may be read (0: no such row)
  __device__ __forceinline__ Row(const Weights& s, int64_t expert, int64_t row, bool there, int q) {
    k = there ? (int)s.k : 0;
    row = there ? row : 0;
    if constexpr (FOUR) {
      w = s.w + (expert * s.rows + row) * (s.k / 2);
      scales = s.scales + (expert * ((s.rows + kTileRows - 1) / kTileRows) + row / kTileRows) * stages4(s.k) * kStageBytes +
               scale_place((int)(row % kTileRows), q);
    } else {
      w = s.w + (expert * s.rows + row) * s.k * 2;
      scales = nullptr;
    }
  }
  __device__ __forceinline__ void load(int step, int q, Raw<FOUR>& r) const {
    if constexpr (FOUR) {
      const int at = 128 * step + 32 * q;
      r.v[0] = u32x4r{0u, 0u, 0u, 0u};
      r.scale = 0u;
      if (at < k) {
        r.v[0] = rows::load16(w + at / 2);
        r.scale = scales[(int64_t)step * kStageBytes];
      }
    } else {
#pragma unroll
      for (int j = 0; j < 2; ++j) {
        const int at = 64 * step + 32 * j + 8 * q;
        r.v[j] = u32x4r{0u, 0u, 0u, 0u};
        if (at < k) r.v[j] = rows::load16(w + 2 * at);
      }
    }
  }
};

template <bool FOUR>
__device__ __forceinline__ bf16x8f operand(const Raw<FOUR>& r, int j) {
  if constexpr (FOUR) {
    const float s = __builtin_bit_cast(float, r.scale << 23);     // (the conversion takes the exponent bits alone)
    u32x4r o;
    o[0] = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(r.v[0][j], s, 0));
    o[1] = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(r.v[0][j], s, 1));
    o[2] = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(r.v[0][j], s, 2));
    o[3] = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(r.v[0][j], s, 3));
    return __builtin_bit_cast(bf16x8f, o);
  } else {
    return __builtin_bit_cast(bf16x8f, r.v[j]);
  }
}

// Row of a strip's place i (0..15).  4 bits: four runs of 4 rows 32 apart,
// whose scales are 64 consecutive bytes of every stage.
template <bool FOUR>
__device__ __forceinline__ int64_t strip_row(int64_t strip, int i) {
  if constexpr (FOUR) return strip / 8 * 128 + 32 * (i & 3) + 4 * (strip % 8) + (i >> 2);
  else return strip * kStrip + i;
}

template <bool FOUR>
__host__ __device__ inline int64_t strips(int64_t rows) {
  return FOUR ? (rows + 127) / 128 * 8 : (rows + kStrip - 1) / kStrip;
}

struct Few {
  const uint16_t* x;        // [tokens, hidden]
  const int32_t* experts;   // [tokens, topk]
  const float* share;       // [tokens, topk] or null
  Weights up, down;
  int32_t tokens, topk, hidden, inter, num_groups;
  int32_t* count;           // workspace: reached experts,
  Reached* reached;         //   each of them,
  uint16_t* act;            //   and rows of weight * a [slots, inter]
  void* out;                // [tokens, hidden]
};

// BLOCKS: of 16 tokens, at most.
template <bool FOUR, int BLOCKS>
__global__ __launch_bounds__(64 * kUpWaves) void few_up_kernel(Few p) {
  __shared__ int32_t s_expert[kMaxSlots];
  __shared__ uint32_t s_bits[GG_MAX_GROUPS_DEV / 32];
  __shared__ int32_t s_token[kMaxTokens];
  __shared__ float s_share[kMaxTokens];
  __shared__ int32_t s_info[3];             // the expert's tokens, and its workspace row
  __shared__ float s_sum[kUpWaves][2][kStrip][kPitch];
  const int tid = threadIdx.x, lane = tid & 63, wave = wave_index();
  const int slots = p.tokens * p.topk;
  const int strip = blockIdx.x, d = blockIdx.y;

  for (int i = tid; i < GG_MAX_GROUPS_DEV / 32; i += 64 * kUpWaves) s_bits[i] = 0u;
  __syncthreads();
  for (int s = tid; s < slots; s += 64 * kUpWaves) {
    const int e = p.experts[s];
    s_expert[s] = e;
    if (e >= 0 && e < p.num_groups) atomicOr(&s_bits[e >> 5], 1u << (e & 31));
  }
  __syncthreads();
  // the d-th reached expert, by index
  const uint32_t word = s_bits[lane];
  int upto = __popc(word);
#pragma unroll
  for (int o = 1; o < 64; o <<= 1) {
    const int v = __shfl_up(upto, (unsigned)o, 64);
    if (lane >= o) upto += v;
  }
  const int reached = __shfl(upto, 63, 64);
  if (strip == 0 && d == 0 && tid == 0) *p.count = reached;
  if (d >= reached) return;
  const int at = __ffsll((unsigned long long)__ballot(upto > d)) - 1;
  const uint32_t bits = (uint32_t)__shfl((int)word, at, 64);
  const int nth = d - (__shfl(upto, at, 64) - __popc(bits));
  const int bit = lane & 31;
  const uint64_t hit = __ballot(((bits >> bit) & 1u) && __popc(bits & ((1u << bit) - 1u)) == nth);
  const int expert = __builtin_amdgcn_readfirstlane(32 * at + __ffsll((unsigned long long)hit) - 1);

  // its tokens (a token that names it twice counts once, with both weights)
  if (wave == 0) {
    int found = 0, before = 0;
    uint64_t who = 0;
    for (int s0 = 0; s0 < slots; s0 += 64) {
      const int s = s0 + lane;
      const int e = s < slots ? s_expert[s] : -1;
      const int t = s < slots ? s / p.topk : 0;
      bool mine = e == expert;
      float w = 0.f;
      if (mine) {
        for (int j = t * p.topk; j < (t + 1) * p.topk; ++j) {
          if (s_expert[j] != expert) continue;
          if (j < s) mine = false;
          w += p.share ? p.share[j] : 1.0f;
        }
      }
      const uint64_t m = __ballot(mine);
      before += __popcll(__ballot(e >= 0 && e < expert));
      if (mine) {
        const int i = found + __popcll(m & ((1ull << lane) - 1ull));
        s_token[i] = t;
        s_share[i] = w;
        who |= 1ull << t;
      }
      found += __popcll(m);
    }
#pragma unroll
    for (int o = 32; o > 0; o >>= 1) who |= __shfl_xor((unsigned long long)who, o, 64);
    if (lane == 0) {
      s_info[0] = found;
      s_info[1] = before;
      if (strip == 0) p.reached[d] = Reached{expert, before, who};
    }
  }
  __syncthreads();
  const int found = s_info[0], base = s_info[1];

  const int col = lane & 15, q = lane >> 4;
  const int64_t row = strip_row<FOUR>(strip, col);
  const bool there = row < p.inter;
  const Row<FOUR> gate(p.up, expert, row, there, q), up(p.up, expert, p.inter + row, there, q);
  const uint16_t* xr[BLOCKS];
#pragma unroll
  for (int b = 0; b < BLOCKS; ++b) xr[b] = 16 * b + col < found ? p.x + (int64_t)s_token[16 * b + col] * p.hidden : nullptr;
  f32x4f ag[BLOCKS], au[BLOCKS];
#pragma unroll
  for (int b = 0; b < BLOCKS; ++b) ag[b] = au[b] = f32x4f{0.f, 0.f, 0.f, 0.f};

  using S = Step<FOUR>;
  const int steps = (p.hidden + S::kValues - 1) / S::kValues;
  constexpr int kAhead = 4;
  for (int s0 = wave; s0 < steps; s0 += kUpWaves * kAhead) {
    Raw<FOUR> g[kAhead], u[kAhead];
#pragma unroll
    for (int a = 0; a < kAhead; ++a) {
      gate.load(s0 + kUpWaves * a, q, g[a]);
      up.load(s0 + kUpWaves * a, q, u[a]);
    }
#pragma unroll
    for (int a = 0; a < kAhead; ++a) {
      const int step = s0 + kUpWaves * a;
      if (step >= steps) break;
#pragma unroll
      for (int j = 0; j < S::kOperands; ++j) {
        const bf16x8f wg = operand<FOUR>(g[a], j), wu = operand<FOUR>(u[a], j);
        const int k = step * S::kValues + S::at(q, j);
#pragma unroll
        for (int b = 0; b < BLOCKS; ++b) {
          if (16 * b >= found) break;
          u32x4r xv = {0u, 0u, 0u, 0u};
          if (xr[b] && k < p.hidden) xv = rows::load16(xr[b] + k);
          const bf16x8f xo = __builtin_bit_cast(bf16x8f, xv);
          ag[b] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(wg, xo, ag[b], 0, 0, 0);
          au[b] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(wu, xo, au[b], 0, 0, 0);
        }
      }
    }
  }
  // the waves' shares of the reduction, added in order; lane l holds token l
  // mod 16, places 4 (l / 16) .. + 3
#pragma unroll
  for (int b = 0; b < BLOCKS; ++b) {
    if (16 * b >= found) break;
    if (b > 0) __syncthreads();
#pragma unroll
    for (int r = 0; r < 4; ++r) {
      s_sum[wave][0][col][4 * q + r] = ag[b][r];
      s_sum[wave][1][col][4 * q + r] = au[b][r];
    }
    __syncthreads();
    if (tid < kStrip * kStrip) {
      const int t = 16 * b + (tid >> 4), i = tid & 15;
      const int64_t c = strip_row<FOUR>(strip, i);
      if (t < found && c < p.inter) {
        float g = 0.f, u = 0.f;
#pragma unroll
        for (int w = 0; w < kUpWaves; ++w) {
          g += s_sum[w][0][tid >> 4][i];
          u += s_sum[w][1][tid >> 4][i];
        }
        const float a = g * __builtin_amdgcn_rcpf(1.0f + __expf(-g)) * u * s_share[t];
        reinterpret_cast<__bf16*>(p.act)[(int64_t)(base + t) * p.inter + c] = (__bf16)a;
      }
    }
  }
}

template <bool FOUR, int BLOCKS, bool OUT_F32>
__global__ __launch_bounds__(64 * kDownWaves) void few_down_kernel(Few p) {
  __shared__ Reached s_reached[kMaxSlots];
  __shared__ float s_sum[kDownWaves][kStrip][kPitch];
  const int tid = threadIdx.x, lane = tid & 63, wave = wave_index();
  const int reached = *p.count;
  for (int i = tid; i < reached; i += 64 * kDownWaves) s_reached[i] = p.reached[i];
  __syncthreads();
  const int col = lane & 15, q = lane >> 4;
  const int strip = blockIdx.x;
  const int64_t row = strip_row<FOUR>(strip, col);
  const bool there = row < p.hidden;
  f32x4f acc[BLOCKS];
#pragma unroll
  for (int b = 0; b < BLOCKS; ++b) acc[b] = f32x4f{0.f, 0.f, 0.f, 0.f};

  using S = Step<FOUR>;
  const int steps = (p.inter + S::kValues - 1) / S::kValues;
  const int items = reached * steps;
  constexpr int kAhead = 4;
  for (int i0 = wave; i0 < items; i0 += kDownWaves * kAhead) {
    Raw<FOUR> w[kAhead];
#pragma unroll
    for (int a = 0; a < kAhead; ++a) {
      const int i = i0 + kDownWaves * a;
      const int d = i < items ? i / steps : 0;
      const int e = __builtin_amdgcn_readfirstlane(s_reached[d].expert);
      Row<FOUR>(p.down, e, row, there && i < items, q).load(i - d * steps, q, w[a]);
    }
#pragma unroll
    for (int a = 0; a < kAhead; ++a) {
      const int i = i0 + kDownWaves * a;
      if (i >= items) break;
      const int d = i / steps, step = i - d * steps;
      const Reached r = s_reached[d];
#pragma unroll
      for (int b = 0; b < BLOCKS; ++b) {
        const uint32_t in16 = (uint32_t)__builtin_amdgcn_readfirstlane((int)((r.tokens >> (16 * b)) & 0xFFFFu));
        if (in16 == 0u) continue;
        const bool mine = (in16 >> col) & 1u;
        const int t = 16 * b + col;
        const uint16_t* from = p.act + (int64_t)(r.base + __popcll(r.tokens & ((1ull << t) - 1ull))) * p.inter;
        // a product of its own, so that a weight that is not finite reaches
        // the expert's own tokens only
        f32x4f part = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
        for (int j = 0; j < S::kOperands; ++j) {
          const int k = step * S::kValues + S::at(q, j);
          u32x4r v = {0u, 0u, 0u, 0u};
          if (mine && k < p.inter) v = rows::load16(from + k);
          part = __builtin_amdgcn_mfma_f32_16x16x32_bf16(operand<FOUR>(w[a], j), __builtin_bit_cast(bf16x8f, v), part, 0,
                                                         0, 0);
        }
#pragma unroll
        for (int e = 0; e < 4; ++e) acc[b][e] += mine ? part[e] : 0.f;
      }
    }
  }
#pragma unroll
  for (int b = 0; b < BLOCKS; ++b) {
    if (16 * b >= p.tokens) break;
    if (b > 0) __syncthreads();
#pragma unroll
    for (int r = 0; r < 4; ++r) s_sum[wave][col][4 * q + r] = acc[b][r];
    __syncthreads();
    if (tid < kStrip * kStrip) {
      const int t = 16 * b + (tid >> 4), i = tid & 15;
      const int64_t c = strip_row<FOUR>(strip, i);
      if (t < p.tokens && c < p.hidden) {
        float v = 0.f;
#pragma unroll
        for (int w = 0; w < kDownWaves; ++w) v += s_sum[w][tid >> 4][i];
        if constexpr (OUT_F32) static_cast<float*>(p.out)[(int64_t)t * p.hidden + c] = v;
        else static_cast<__bf16*>(p.out)[(int64_t)t * p.hidden + c] = (__bf16)v;
      }
    }
  }
}

template <bool FOUR, int BLOCKS>
hipError_t launch(const Few& p, bool out_f32, hipStream_t stream) {
  const int slots = p.tokens * p.topk;
  const int most = slots < p.num_groups ? slots : p.num_groups;
  hipError_t e = launch_kernel(few_up_kernel<FOUR, BLOCKS>, dim3((unsigned)strips<FOUR>(p.inter), (unsigned)most),
                               dim3(64 * kUpWaves), stream, p);
  if (e != hipSuccess) return e;
  auto* down = out_f32 ? few_down_kernel<FOUR, BLOCKS, true> : few_down_kernel<FOUR, BLOCKS, false>;
  return launch_kernel(down, dim3((unsigned)strips<FOUR>(p.hidden)), dim3(64 * kDownWaves), stream, p);
}

// The workspace: the count (16 bytes), the reached experts, the rows.
int64_t reached_bytes(int64_t slots, int32_t E) { return 16 * (slots < E ? slots : E); }

}  // namespace

int64_t few_tokens_workspace(int64_t slots, int64_t inter, int32_t E) {
  return 16 + reached_bytes(slots, E) + slots * inter * 2;
}

hipError_t launch_few_tokens(bool four, const void* x, const int32_t* experts, const float* share, const void* w13,
                             const void* s13, const void* w2, const void* s2, void* out, bool out_f32, void* workspace,
                             int64_t tokens, int32_t topk, int64_t hidden, int64_t inter, int32_t E,
                             hipStream_t stream) {
  static_assert(sizeof(Reached) == 16, "the workspace holds 16 bytes for each");
  if (tokens == 0) return hipSuccess;
  uint8_t* ws = static_cast<uint8_t*>(workspace);
  Few p;
  p.x = static_cast<const uint16_t*>(x);
  p.experts = experts;
  p.share = share;
  p.up = Weights{static_cast<const uint8_t*>(w13), static_cast<const uint8_t*>(s13), 2 * inter, hidden};
  p.down = Weights{static_cast<const uint8_t*>(w2), static_cast<const uint8_t*>(s2), hidden, inter};
  p.tokens = (int32_t)tokens;
  p.topk = topk;
  p.hidden = (int32_t)hidden;
  p.inter = (int32_t)inter;
  p.num_groups = E;
  p.count = reinterpret_cast<int32_t*>(ws);
  p.reached = reinterpret_cast<Reached*>(ws + 16);
  p.act = reinterpret_cast<uint16_t*>(ws + 16 + reached_bytes(tokens * topk, E));
  p.out = out;
  if (four) return tokens <= 16 ? launch<true, 1>(p, out_f32, stream) : launch<true, 4>(p, out_f32, stream);
  return tokens <= 16 ? launch<false, 1>(p, out_f32, stream) : launch<false, 4>(p, out_f32, stream);
}

}  // namespace gg
