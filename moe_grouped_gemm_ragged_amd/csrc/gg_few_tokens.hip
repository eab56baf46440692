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
// instruction's operand as they lie in memory, the rows are its 16 columns.
// 4-bit weights become bf16 in registers (exactly).
//
//   up kernel    a workgroup takes an expert and 16 columns of I: rows c of W1
//                and W3 against x of the tokens that chose the expert; writes
//                weight * a to the workspace, as the sum of two bf16 values (a
//                single one would double the layer's error)
//   down kernel  a workgroup takes 16 rows of every reached expert's W2 and
//                adds all experts' shares itself, so out is written once, with
//                no partial sums in memory
//
// Which experts are reached, and by whom, the up kernel's workgroups find for
// themselves from the expert ids: each wave alone where there are at most 64
// slots (no barrier, one load ahead of the weights), else in LDS.  The first
// workgroup of each expert leaves it in the workspace for the down kernel.
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
constexpr int kWaveSlots = 64;                // slots that a wave holds, one a lane
constexpr int kStrip = 16;                    // weight rows of a workgroup (and columns of a matrix instruction)
constexpr int kUpWaves = 8, kDownWaves = 16;
constexpr int kPitch = kStrip + 1;            // floats between a token's strips in LDS
constexpr int kPair = 8;                      // tokens of a down product: two columns each
constexpr uint32_t kOutside = 0x80000000u;    // an offset past every range here

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

__device__ __forceinline__ u32x4r load_range(const __amdgpu_buffer_rsrc_t& rs, uint32_t at, int base) {
  return __builtin_bit_cast(u32x4r, __builtin_amdgcn_raw_buffer_load_b128(rs, at, base, 0));
}
__device__ __forceinline__ __amdgpu_buffer_rsrc_t range(const void* base, int64_t bytes) {
  return __builtin_amdgcn_make_buffer_rsrc(const_cast<void*>(base), (short)0, (int)(uint32_t)bytes, 0x00020000);
}

// Rows row0 .. of an expert's matrix, as far as a strip reaches, as ranges that
// end with them (rows past the last read as zero).  All scalar.
template <bool FOUR>
struct Strip {
  __amdgpu_buffer_rsrc_t w, scales;
  __device__ __forceinline__ Strip(const Weights& m, int64_t expert, int64_t row0, int64_t rows) {
    constexpr int kSpan = FOUR ? 128 : kStrip;
    const int64_t span = rows < kSpan ? rows : kSpan;
    const int64_t pitch = FOUR ? m.k / 2 : m.k * 2;
    w = range(m.w + (expert * m.rows + row0) * pitch, span * pitch);
    // (the span may begin anywhere in a tile of scales, and reach into the next)
    if constexpr (FOUR) {
      const int64_t tile = stages4(m.k) * kStageBytes, tiles = (m.rows + kTileRows - 1) / kTileRows;
      const int64_t first = row0 / kTileRows;
      scales = range(m.scales + (expert * tiles + first) * tile, (tiles - first < 2 ? tiles - first : 2) * tile);
    }
  }
};

// This lane's place in a strip: the offsets of its row's first values and of
// their scales.
template <bool FOUR>
struct Lane {
  uint32_t w, scale;
  __device__ __forceinline__ Lane(const Weights& m, int64_t row0, int place, int q) {
    const uint32_t pitch = (uint32_t)(FOUR ? m.k / 2 : m.k * 2);
    w = (uint32_t)place * pitch + 16u * (uint32_t)q;
    if constexpr (FOUR) {
      const int64_t row = row0 + place;
      scale = (uint32_t)((row / kTileRows - row0 / kTileRows) * stages4(m.k) * kStageBytes) +
              (uint32_t)scale_place((int)(row % kTileRows), q);
    }
  }
};

// Values that a lane's operand j of a step covers and that a row of k has.
template <bool FOUR>
__device__ __forceinline__ bool inside(int step, int q, int j, int k) {
  return step * Step<FOUR>::kValues + Step<FOUR>::at(q, FOUR ? 0 : j) < k;
}

template <bool FOUR>
__device__ __forceinline__ void load_weights(const Strip<FOUR>& s, const Lane<FOUR>& l, int step, int q, int k,
                                             Raw<FOUR>& r) {
  if constexpr (FOUR) {
    const bool in = inside<FOUR>(step, q, 0, k);
    r.v[0] = load_range(s.w, in ? l.w : kOutside, 64 * step);
    r.scale = __builtin_amdgcn_raw_buffer_load_b8(s.scales, in ? l.scale : kOutside, kStageBytes * step, 0);
  } else {
#pragma unroll
    for (int j = 0; j < 2; ++j) r.v[j] = load_range(s.w, inside<FOUR>(step, q, j, k) ? l.w + 64 * j : kOutside, 128 * step);
  }
}

// The rows' operands: bf16 rows from `at` on (this lane's first value's offset,
// or kOutside).
template <bool FOUR>
__device__ __forceinline__ void load_rows(const __amdgpu_buffer_rsrc_t& rs, uint32_t at, int base, int step, int q, int k,
                                          u32x4r (&v)[Step<FOUR>::kOperands]) {
#pragma unroll
  for (int j = 0; j < Step<FOUR>::kOperands; ++j)
    v[j] = load_range(rs, inside<FOUR>(step, q, j, k) ? at + (uint32_t)(2 * (Step<FOUR>::at(0, j))) : kOutside,
                      base + 2 * Step<FOUR>::kValues * step);
}

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

// First row of a strip's span, and the row in it of the strip's place i (0..15).
// 4 bits: four runs of 4 rows 32 apart, whose scales are 64 consecutive bytes
// of every stage.
template <bool FOUR>
__device__ __forceinline__ int64_t strip_first(int strip) {
  return FOUR ? strip / 8 * 128 : (int64_t)strip * kStrip;
}
template <bool FOUR>
__device__ __forceinline__ int strip_place(int strip, int i) {
  return FOUR ? 32 * (i & 3) + 4 * (strip % 8) + (i >> 2) : i;
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
  uint16_t* act;            //   and rows of weight * a [slots, 2, inter]: its bf16 value, and what that left
  void* out;                // [tokens, hidden]
  bool out_f32;
};

__device__ __forceinline__ uint64_t lanes_before(int lane) { return (1ull << lane) - 1ull; }

__device__ __forceinline__ uint64_t lane_value64(uint64_t v, int lane) {
  const uint32_t lo = (uint32_t)__builtin_amdgcn_readlane((int)(uint32_t)v, lane);
  const uint32_t hi = (uint32_t)__builtin_amdgcn_readlane((int)(uint32_t)(v >> 32), lane);
  return (uint64_t)hi << 32 | lo;
}

// The reduction of one expert's gate and up strip over this wave's steps, for
// up to 16 BLOCKS tokens.
template <bool FOUR, int BLOCKS>
__device__ __forceinline__ void up_steps(const Few& p, const Strip<FOUR>& gate, const Strip<FOUR>& up, const Lane<FOUR>& lg,
                                         const Lane<FOUR>& lu, const int32_t* tokens, int found, int wave, int col, int q,
                                         f32x4f (&ag)[4], f32x4f (&au)[4]) {
  using S = Step<FOUR>;
  constexpr int kAhead = BLOCKS == 1 ? (FOUR ? 3 : 4) : BLOCKS == 2 ? 2 : 1;
  const int k = p.hidden, steps = (k + S::kValues - 1) / S::kValues;
  const __amdgpu_buffer_rsrc_t xs = range(p.x, (int64_t)p.tokens * k * 2);
  uint32_t xat[BLOCKS];
#pragma unroll
  for (int b = 0; b < BLOCKS; ++b)
    xat[b] = 16 * b + col < found ? (uint32_t)(tokens[16 * b + col] * k + S::at(q, 0)) * 2u : kOutside;
  Raw<FOUR> g[kAhead], u[kAhead];
  u32x4r x[kAhead][BLOCKS][S::kOperands];
  auto issue = [&](int a, int step) __attribute__((always_inline)) {
#pragma unroll
    for (int b = 0; b < BLOCKS; ++b) load_rows<FOUR>(xs, xat[b], 0, step, q, k, x[a][b]);
    load_weights<FOUR>(gate, lg, step, q, k, g[a]);
    load_weights<FOUR>(up, lu, step, q, k, u[a]);
  };
#pragma unroll
  for (int a = 0; a < kAhead; ++a) issue(a, wave + kUpWaves * a);
  for (int s0 = wave; s0 < steps; s0 += kUpWaves * kAhead) {
#pragma unroll
    for (int a = 0; a < kAhead; ++a) {
      // (steps past the last are zeros)
#pragma unroll
      for (int j = 0; j < S::kOperands; ++j) {
        const bf16x8f wg = operand<FOUR>(g[a], j), wu = operand<FOUR>(u[a], j);
#pragma unroll
        for (int b = 0; b < BLOCKS; ++b) {
          const bf16x8f xo = __builtin_bit_cast(bf16x8f, x[a][b][j]);
          ag[b] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(wg, xo, ag[b], 0, 0, 0);
          au[b] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(wu, xo, au[b], 0, 0, 0);
        }
      }
      issue(a, s0 + kUpWaves * (kAhead + a));
    }
  }
}

// SMALL: at most 64 slots.
template <bool FOUR, bool SMALL>
__global__ __launch_bounds__(64 * kUpWaves, 4) void few_up_kernel(Few p) {
  __shared__ int32_t s_expert[SMALL ? 1 : kMaxSlots];
  __shared__ uint32_t s_bits[SMALL ? 1 : GG_MAX_GROUPS_DEV / 32];
  __shared__ int32_t s_token[SMALL ? kUpWaves : 1][kMaxTokens];
  __shared__ float s_share[SMALL ? kUpWaves : 1][kMaxTokens];
  __shared__ int32_t s_info[2];             // the expert's tokens, and its workspace row
  __shared__ float s_sum[kUpWaves][2][kStrip][kPitch];
  const int tid = threadIdx.x, lane = tid & 63, wave = wave_index();
  const int own = SMALL ? wave : 0;         // SMALL: every wave has its copy of the lists
  const int slots = p.tokens * p.topk;
  const int strip = blockIdx.x, d = blockIdx.y;
  int expert, found, base;

  if constexpr (SMALL) {
    int e = lane < slots ? p.experts[lane] : -1;
    const float w = p.share && lane < slots ? p.share[lane] : 1.0f;
    e = e < p.num_groups ? e : -1;
    // experts in the order of their first slots; each leaves as many workspace
    // rows as it has slots
    uint64_t left = __ballot(e >= 0), mine = 0;
    int n = 0;
    base = 0;
    expert = 0;
    while (left != 0ull) {
      const int at = __builtin_amdgcn_readlane(e, __ffsll((unsigned long long)left) - 1);
      const uint64_t same = __ballot(e == at);
      left &= ~same;
      if (n == d) {
        mine = same;
        expert = at;
        if (strip != 0 || d != 0) break;        // (the first workgroup counts them all)
      } else if (n < d) {
        base += __popcll(same);
      }
      ++n;
    }
    if (strip == 0 && d == 0 && tid == 0) *p.count = n;
    if (mine == 0ull) return;
    // its tokens, by slot: a token that names it twice counts once, with both
    // shares
    uint64_t who = 0;
    found = 0;
    int last = -1;
    float sum = 0.f;
    for (uint64_t m = mine; m != 0ull; m &= m - 1ull) {
      const int s = __ffsll((unsigned long long)m) - 1, t = s / p.topk;
      const float v = rows::lane_value(w, s);
      if (t != last) {
        if (lane == found) {
          s_token[own][found] = t;
        }
        ++found;
        sum = 0.f;
        last = t;
        who |= 1ull << t;
      }
      sum += v;
      if (lane == 0) s_share[own][found - 1] = sum;
    }
    if (strip == 0 && tid == 0) p.reached[d] = Reached{expert, base, who};
  } else {
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
    expert = __builtin_amdgcn_readfirstlane(32 * at + __ffsll((unsigned long long)hit) - 1);
    if (wave == 0) {
      int count = 0, before = 0;
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
          const int i = count + __popcll(m & lanes_before(lane));
          s_token[0][i] = t;
          s_share[0][i] = w;
          who |= 1ull << t;
        }
        count += __popcll(m);
      }
#pragma unroll
      for (int o = 32; o > 0; o >>= 1) who |= __shfl_xor((unsigned long long)who, o, 64);
      if (lane == 0) {
        s_info[0] = count;
        s_info[1] = before;
        if (strip == 0) p.reached[d] = Reached{expert, before, who};
      }
    }
    __syncthreads();
    found = __builtin_amdgcn_readfirstlane(s_info[0]);
    base = s_info[1];
  }

  const int col = lane & 15, q = lane >> 4;
  const int64_t row0 = strip_first<FOUR>(strip);
  const int place = strip_place<FOUR>(strip, col);
  const Strip<FOUR> gate(p.up, expert, row0, p.inter - row0), up(p.up, expert, p.inter + row0, p.inter - row0);
  const Lane<FOUR> lg(p.up, row0, place, q), lu(p.up, p.inter + row0, place, q);
  f32x4f ag[4], au[4];
#pragma unroll
  for (int b = 0; b < 4; ++b) ag[b] = au[b] = f32x4f{0.f, 0.f, 0.f, 0.f};
  if (found <= 16) up_steps<FOUR, 1>(p, gate, up, lg, lu, s_token[own], found, wave, col, q, ag, au);
  else if (found <= 32) up_steps<FOUR, 2>(p, gate, up, lg, lu, s_token[own], found, wave, col, q, ag, au);
  else up_steps<FOUR, 4>(p, gate, up, lg, lu, s_token[own], found, wave, col, q, ag, au);
  // the waves' shares of the reduction, added in order; lane l holds token l
  // mod 16, places 4 (l / 16) .. + 3
#pragma unroll
  for (int b = 0; b < 4; ++b) {
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
      const int64_t c = row0 + strip_place<FOUR>(strip, i);
      if (t < found && c < p.inter) {
        float g = 0.f, u = 0.f;
#pragma unroll
        for (int w = 0; w < kUpWaves; ++w) {
          g += s_sum[w][0][tid >> 4][i];
          u += s_sum[w][1][tid >> 4][i];
        }
        const float a = g * __builtin_amdgcn_rcpf(1.0f + __expf(-g)) * u * s_share[own][t];
        __bf16* to = reinterpret_cast<__bf16*>(p.act) + (int64_t)(base + t) * 2 * p.inter + c;
        const __bf16 high = (__bf16)a;
        const float left = a - (float)high;
        to[0] = high;
        // (an infinity or NaN is its own value, with nothing left)
        to[p.inter] = (__bf16)(rows::finite(left) ? left : 0.f);
      }
    }
  }
}

// TOKENS: at most.
template <bool FOUR, int TOKENS>
__global__ __launch_bounds__(64 * kDownWaves) void few_down_kernel(Few p) {
  __shared__ __attribute__((aligned(16))) float s_out[kDownWaves][TOKENS][kStrip];     // each wave's sums
  const int tid = threadIdx.x, lane = tid & 63, wave = wave_index();
  const int slots = p.tokens * p.topk;
  const int most = slots < p.num_groups ? slots : p.num_groups;
  // Reached experts, one a lane (loaded before their number is known), the next
  // 64 when a wave gets there.
  Reached mine = {0, 0, 0};
  int have = 0;
  auto fetch = [&](int first) {
    have = first;
    if (first + lane < most) mine = p.reached[first + lane];
  };
  const int strip = blockIdx.x;
  const int col = lane & 15, q = lane >> 4;

  using S = Step<FOUR>;
  const int k = p.inter, steps = (k + S::kValues - 1) / S::kValues;
  const int64_t row0 = strip_first<FOUR>(strip);
  const Lane<FOUR> ll(p.down, row0, strip_place<FOUR>(strip, col), q);
  const __amdgpu_buffer_rsrc_t acts = range(p.act, (int64_t)slots * 4 * k);
  // columns 0..7 are the bf16 values of 8 of an expert's tokens, 8..15 what
  // those left
  const int member = col & (kPair - 1);
  const uint32_t act_at = (uint32_t)((2 * member + (col >> 3)) * k + S::at(q, 0)) * 2u;
  for (int i = lane; i < TOKENS * kStrip / 4; i += 64)
    reinterpret_cast<f32x4f*>(&s_out[wave][0][0])[i] = f32x4f{0.f, 0.f, 0.f, 0.f};
  fetch(0);
  const int reached = __builtin_amdgcn_readfirstlane(*p.count);

  // The reached experts' steps, one expert after the other; a wave takes an
  // equal run of them.
  const int items = reached * steps;
  const int end = (int)((int64_t)items * (wave + 1) / kDownWaves);
  struct Item {
    int expert, base, step;
    uint64_t tokens;
  };
  int at = (int)((int64_t)items * wave / kDownWaves);
  int d = at / steps, step = at - d * steps;
  auto next = [&]() {
    Item i = {0, 0, 0, 0ull};                    // (past the wave's last item: no rows)
    if (at < end) {
      if (d - have >= 64) fetch(d & ~63);
      i.expert = __builtin_amdgcn_readlane(mine.expert, d & 63);
      i.base = __builtin_amdgcn_readlane(mine.base, d & 63);
      i.tokens = lane_value64(mine.tokens, d & 63);
      i.step = step;
      ++at;
      if (++step == steps) {
        step = 0;
        ++d;
      }
    }
    return i;
  };
  constexpr int kAhead = FOUR ? 4 : 6;
  Raw<FOUR> w[kAhead];
  u32x4r v[kAhead][S::kOperands];
  Item items_ahead[kAhead];
  auto issue = [&](int a) __attribute__((always_inline)) {
    const Item i = items_ahead[a] = next();
    const int found = __popcll(i.tokens);
    load_rows<FOUR>(acts, member < found ? act_at : kOutside, 4 * i.base * k, i.step, q, k, v[a]);
    const Strip<FOUR> s(p.down, i.expert, row0, i.tokens ? p.hidden - row0 : 0);
    load_weights<FOUR>(s, ll, i.step, q, k, w[a]);
  };
  auto multiply = [&](const Raw<FOUR>& wr, const u32x4r (&vr)[S::kOperands], f32x4f c) __attribute__((always_inline)) {
#pragma unroll
    for (int j = 0; j < S::kOperands; ++j)
      c = __builtin_amdgcn_mfma_f32_16x16x32_bf16(operand<FOUR>(wr, j), __builtin_bit_cast(bf16x8f, vr[j]), c, 0, 0, 0);
    return c;
  };
  // Adds tokens 8 b .. of an expert's product to the wave's sums.  (Each
  // expert's product is one of its own, so that a weight that is not finite
  // reaches the expert's own tokens only.)
  auto add = [&](f32x4f part, uint64_t tokens, int b) {
#pragma unroll
    for (int e = 0; e < 4; ++e) part[e] += rows::row_ror<kPair>(part[e]);
    const int i = kPair * b + col;
    if (col < kPair && i < __popcll(tokens)) {
      uint64_t left = tokens;
      for (int z = 0; z < i; ++z) left &= left - 1ull;
      f32x4f* to = reinterpret_cast<f32x4f*>(&s_out[wave][__ffsll((unsigned long long)left) - 1][4 * q]);
      *to = *to + part;
    }
  };
  if (at < end) {
    int left = end - at;
    f32x4f part = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
    for (int a = 0; a < kAhead; ++a) issue(a);
    int expert = items_ahead[0].expert;
    uint64_t tokens = items_ahead[0].tokens;
    for (; left > 0; left -= kAhead) {
#pragma unroll
      for (int a = 0; a < kAhead; ++a) {
        const Item i = items_ahead[a];
        if (i.tokens && i.expert != expert) {
          add(part, tokens, 0);
          part = f32x4f{0.f, 0.f, 0.f, 0.f};
          expert = i.expert;
          tokens = i.tokens;
        }
        part = multiply(w[a], v[a], part);
        const int found = __popcll(i.tokens);
        for (int b = 1; kPair * b < found; ++b) {
          u32x4r more[S::kOperands];
          load_rows<FOUR>(acts, kPair * b + member < found ? act_at : kOutside, 4 * (i.base + kPair * b) * k, i.step, q, k,
                          more);
          add(multiply(w[a], more, f32x4f{0.f, 0.f, 0.f, 0.f}), i.tokens, b);
        }
        issue(a);
      }
    }
    add(part, tokens, 0);
  }
  __syncthreads();
  for (int o = tid; o < p.tokens * kStrip; o += 64 * kDownWaves) {
    const int t = o / kStrip, i = o % kStrip;
    const int64_t c = row0 + strip_place<FOUR>(strip, i);
    if (c >= p.hidden) continue;
    float sum = 0.f;
#pragma unroll
    for (int z = 0; z < kDownWaves; ++z) sum += s_out[z][t][i];
    if (p.out_f32) static_cast<float*>(p.out)[(int64_t)t * p.hidden + c] = sum;
    else static_cast<__bf16*>(p.out)[(int64_t)t * p.hidden + c] = (__bf16)sum;
  }
}

template <bool FOUR>
hipError_t launch_four(const Few& p, hipStream_t stream) {
  const int slots = p.tokens * p.topk;
  const int most = slots < p.num_groups ? slots : p.num_groups;
  auto* up = slots <= kWaveSlots ? few_up_kernel<FOUR, true> : few_up_kernel<FOUR, false>;
  const hipError_t e = launch_kernel(up, dim3((unsigned)strips<FOUR>(p.inter), (unsigned)most), dim3(64 * kUpWaves),
                                     stream, p);
  if (e != hipSuccess) return e;
  auto* down = p.tokens <= 16 ? few_down_kernel<FOUR, 16> : few_down_kernel<FOUR, kMaxTokens>;
  return launch_kernel(down, dim3((unsigned)strips<FOUR>(p.hidden)), dim3(64 * kDownWaves), stream, p);
}

// The workspace: the count (16 bytes), the reached experts, the rows.
int64_t reached_bytes(int64_t slots, int32_t E) { return 16 * (slots < E ? slots : E); }

}  // namespace

int64_t few_tokens_workspace(int64_t slots, int64_t inter, int32_t E) {
  return 16 + reached_bytes(slots, E) + slots * inter * 4;
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
  p.out_f32 = out_f32;
  return four ? launch_four<true>(p, stream) : launch_four<false>(p, stream);
}

}  // namespace gg
