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
//   up kernel    a workgroup takes an expert and strips of 8 columns of I: an
//                instruction's 16 rows are the 8 of W1 and the 8 of W3.  Writes
//                weight * a to the workspace, as the sum of two bf16 values (a
//                single one would add half as much again to the layer's error)
//   down kernel  a workgroup takes 8 rows of every reached expert's W2 and adds
//                all experts' shares itself, so out is written once, with no
//                partial sums in memory.  Places 8..15 of an instruction are the
//                same 8 rows at the next values of the reduction, and so are
//                its columns 8..15: two of its four quarters count
//
// A compute unit takes in about 25 GB/s of weights from memory, whatever it has
// in flight, so what counts is that all 256 have the same share: hence strips of
// 8 rows (128 experts, hidden 2048, inter 768, bf16, 23 tokens to 8 each: down
// 61 us, with strips of 16 rows 99; one token 6.9 against 12.2).  The address
// unit takes 16 bytes of 4 lanes a cycle, used or not: x goes through LDS in the
// up kernel (4 tokens, 64 experts, 7168 x 2048 in 4 bits: 114 us, loaded by
// every lane 151), and no load is issued past a wave's last step (one token:
// up 14.4 us against 16.7, down 6.8 against 8.8).  Small workgroups, 4 of up and
// 2 of down a compute unit, fill each other's beginnings and ends (up with 8
// waves 120, 15.0 and 11.8 us where 4 take 113, 13.0 and 7.7; down with 16
// waves 77 us where 8 take 69).
//
// Reached, one token 13.0 + 6.9 us (75 MB, 20.0 in a row of passes, 22.7 with weights
// that no cache holds; 4 bits 7.7 + 5.3, 20 MB, 11.6 and 13.5), 23 tokens
// 111 + 60 us (921 MB: 5.4 TB/s), 4 tokens of the wide 4-bit layer 98 + 55 us
// (620 MB: 4.1 TB/s; the conversions hide behind the loads, strips of half the
// bytes have the same beginnings and ends).  Between the two kernels lies 1.1 us.
//
// An expert of many tokens costs more than its weights: one operand holds 16 of them
// in the up kernel and 4 in the down kernel, and every strip loads their rows (8
// experts of 2048 x 768, bf16, 75 MB: 16 tokens each 45 us, 32 88, 33, where the up
// kernel begins to read its weights twice, 106, and 64 215).
//
// Which experts are reached, and by whom, a workgroup's first wave finds from
// the expert ids; the first workgroup of each expert leaves it in the workspace
// for the down kernel.
#include <hip/hip_runtime.h>
#include <stdint.h>

#include <type_traits>

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
constexpr int kStrip = 8;                     // weight rows of a strip
constexpr int kUpWaves = 4, kDownWaves = 8;
constexpr int kPitch = 2 * kStrip + 1;        // floats between a token's sums in LDS
constexpr int kRowBytes = 30 << 10;           // x rows of an up workgroup's tokens in LDS, where they fit
constexpr int kUpGroups = 4096;               // up workgroups for each strip that one takes,
constexpr int kUpStrips = 4;                  //   and the most strips (measured beside launch_four)
constexpr unsigned kDownAlone = 256;          // 4-bit down strips up to which each has a workgroup of its own,
constexpr int kDownCrowd = 8;                 //   and slots an expert on average from which on it has too
constexpr int kQuad = 4;                      // tokens of a down product: four columns each
constexpr uint32_t kOutside = 0x80000000u;    // an offset past every range here
constexpr float kMaxBf16 = 0x1.fep127f;

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

// One reduction step of an instruction's row: 64 bf16 or 128 4-bit values, as
// operands of matrix instructions.  Operand j of lane l covers, of q = l / 16,
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

// Rows row0 .. row0 + rows - 1 of an expert's matrix and the tiles of scales
// that hold them, as ranges that end with them (what lies past reads as zero).
// All scalar.
template <bool FOUR>
struct Strip {
  __amdgpu_buffer_rsrc_t w, scales;
  __device__ __forceinline__ Strip(const Weights& m, int64_t expert, int64_t row0, int64_t rows) {
    const int64_t pitch = FOUR ? m.k / 2 : m.k * 2;
    w = range(m.w + (expert * m.rows + row0) * pitch, rows * pitch);
    if constexpr (FOUR) {
      const int64_t tile = stages4(m.k) * kStageBytes, tiles = (m.rows + kTileRows - 1) / kTileRows;
      const int64_t first = row0 / kTileRows;
      scales = range(m.scales + (expert * tiles + first) * tile, (tiles - first) * tile);
    }
  }
};

// The offsets of this lane's row's first values and of their scales, from a
// strip's first row on.
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

// HALVES 2: lanes of columns 8..15 take the step after the given one (a step
// then is two).
template <bool FOUR, int HALVES>
struct Reader {
  static constexpr int kOperands = Step<FOUR>::kOperands;
  static constexpr int kValues = HALVES * Step<FOUR>::kValues;
  int k, first;            // values of a row; this lane's first one of step 0
  __device__ __forceinline__ Reader(int64_t row_values, int col, int q)
      : k((int)row_values), first((HALVES == 2 && col >= 8 ? Step<FOUR>::kValues : 0) + Step<FOUR>::at(q, 0)) {}
  __device__ __forceinline__ int steps() const { return (k + kValues - 1) / kValues; }
  __device__ __forceinline__ bool inside(int step, int j) const {
    return step * kValues + first + (FOUR ? 0 : Step<FOUR>::at(0, j)) < k;
  }
  __device__ __forceinline__ void weights(const Strip<FOUR>& s, const Lane<FOUR>& l, bool second, int step,
                                          Raw<FOUR>& r) const {
    const uint32_t half = HALVES == 2 && second ? 1u : 0u;
    if constexpr (FOUR) {
      const bool in = inside(step, 0);
      r.v[0] = load_range(s.w, in ? l.w + 64u * half : kOutside, kValues / 2 * step);
      r.scale = __builtin_amdgcn_raw_buffer_load_b8(s.scales, in ? l.scale + kStageBytes * half : kOutside,
                                                    HALVES * kStageBytes * step, 0);
    } else {
#pragma unroll
      for (int j = 0; j < 2; ++j)
        r.v[j] = load_range(s.w, (inside(step, j) ? l.w + 128u * half : kOutside) + 64u * j, 2 * kValues * step);
    }
  }
  // The rows' operands: bf16 rows; `at` is the offset of this lane's row's
  // first value of step 0 (first, that is), or kOutside.
  __device__ __forceinline__ void rows(const __amdgpu_buffer_rsrc_t& rs, uint32_t at, int base, int step,
                                       u32x4r (&v)[kOperands]) const {
#pragma unroll
    for (int j = 0; j < kOperands; ++j)
      v[j] = load_range(rs, (inside(step, j) ? at : kOutside) + 2u * (uint32_t)Step<FOUR>::at(0, j),
                        base + 2 * kValues * step);
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

// Strips' first rows, and the row of a strip's place i (0..7) from there.  4
// bits: strips share spans of 128 rows, each two runs of 4 rows 32 apart, whose
// scales are 32 consecutive bytes of every stage.
template <bool FOUR>
__host__ __device__ inline int64_t strips(int64_t rows) {
  return FOUR ? (rows + 127) / 128 * 16 : (rows + kStrip - 1) / kStrip;
}
template <bool FOUR>
__device__ __forceinline__ int64_t strip_first(int strip) {
  return FOUR ? strip / 16 * 128 : (int64_t)strip * kStrip;
}
template <bool FOUR>
__device__ __forceinline__ int strip_place(int strip, int i) {
  return FOUR ? 32 * (i & 3) + 2 * (strip % 16) + (i >> 2) : i;
}

// Workgroup b of n runs on XCD b mod 8: neighbouring strips, which share cache
// lines of scales, to one XCD, 4 in a row (4 tokens of the wide 4-bit layer: up
// reads 438 MB in 98 us, with lines shared across XCDs 510 in 102).  What is left
// of n after whole 32s as it comes.
__device__ __forceinline__ int strip_of(int b, int n) {
  return b >= n / 32 * 32 ? b : b / 32 * 32 + b % 8 * 4 + b / 8 % 4;
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
  int32_t strips_each;      // strips of an up workgroup
};

__device__ __forceinline__ uint64_t lanes_before(int lane) { return (1ull << lane) - 1ull; }

__device__ __forceinline__ uint64_t lane_value64(uint64_t v, int lane) {
  const uint32_t lo = (uint32_t)__builtin_amdgcn_readlane((int)(uint32_t)v, lane);
  const uint32_t hi = (uint32_t)__builtin_amdgcn_readlane((int)(uint32_t)(v >> 32), lane);
  return (uint64_t)hi << 32 | lo;
}

// use(a, i) on items i = 0 .. n - 1 with issue(a, i) kAhead of them ahead, a
// their place.  Whole rounds in the loop, the rest after it: an issue that may
// be skipped in the loop would make the compiler wait for all loads on every
// path, and a load out of range costs as much of the address unit's time as
// any other.  start() comes between the first issues and the first use.
template <int kAhead, typename Issue, typename Use, typename Start>
__device__ __forceinline__ void pipelined(int n, const Issue& issue, const Use& use, const Start& start) {
#pragma unroll
  for (int a = 0; a < kAhead; ++a)
    if (a < n) issue(a, a);
  start();
  int i = 0;
  for (; i + 2 * kAhead <= n; i += kAhead) {
#pragma unroll
    for (int a = 0; a < kAhead; ++a) {
      use(a, i + a);
      issue(a, i + kAhead + a);
    }
  }
#pragma unroll
  for (int a = 0; a < kAhead; ++a) {
    if (i + a < n) use(a, i + a);
    if (i + kAhead + a < n) issue(a, i + kAhead + a);
  }
#pragma unroll
  for (int a = 0; a < kAhead; ++a)
    if (i + kAhead + a < n) use(a, i + kAhead + a);
}

// The reduction of one strip over this wave's steps, for up to 16 tokens whose
// rows are in LDS: row i at pitch i, zeros from p.hidden on to the last step's
// end.  fill() puts them there (and waits for all waves), once the first weights
// are on their way.  Columns without a token repeat the last one's.
template <bool FOUR, typename Fill>
__device__ __forceinline__ void up_steps_lds(const Few& p, const Strip<FOUR>& s, const Lane<FOUR>& l, const uint8_t* x,
                                             uint32_t pitch, int found, int wave, int col, int q, f32x4f& acc,
                                             const Fill& fill) {
  constexpr int kAhead = FOUR ? 6 : 4;
  const Reader<FOUR, 1> rd(p.hidden, col, q);
  const uint8_t* const row = x + (uint32_t)(col < found ? col : found - 1) * pitch + 2 * rd.first;
  Raw<FOUR> w[kAhead];
  auto issue = [&](int a, int i) __attribute__((always_inline)) {
    rd.weights(s, l, false, wave + kUpWaves * i, w[a]);
  };
  auto use = [&](int a, int i) __attribute__((always_inline)) {
    const uint8_t* const from = row + (uint32_t)(2 * Reader<FOUR, 1>::kValues) * (uint32_t)(wave + kUpWaves * i);
#pragma unroll
    for (int j = 0; j < Step<FOUR>::kOperands; ++j) {
      const u32x4r v = *reinterpret_cast<const u32x4r*>(from + 2 * Step<FOUR>::at(0, j));
      acc = __builtin_amdgcn_mfma_f32_16x16x32_bf16(operand<FOUR>(w[a], j), __builtin_bit_cast(bf16x8f, v), acc, 0, 0, 0);
    }
  };
  pipelined<kAhead>((rd.steps() - wave + kUpWaves - 1) / kUpWaves, issue, use, fill);
}

// The same for up to 32 tokens, whose rows are loaded with the weights.
template <bool FOUR, int BLOCKS>
__device__ __forceinline__ void up_steps(const Few& p, const Strip<FOUR>& s, const Lane<FOUR>& l, const int32_t* tokens,
                                         int found, int wave, int col, int q, f32x4f* acc) {
  constexpr int kAhead = BLOCKS == 1 ? 2 : 1;
  const Reader<FOUR, 1> rd(p.hidden, col, q);
  const __amdgpu_buffer_rsrc_t xs = range(p.x, (int64_t)p.tokens * p.hidden * 2);
  uint32_t xat[BLOCKS];
#pragma unroll
  for (int b = 0; b < BLOCKS; ++b)
    xat[b] = 16 * b + col < found ? (uint32_t)(tokens[16 * b + col] * p.hidden + rd.first) * 2u : kOutside;
  Raw<FOUR> w[kAhead];
  u32x4r x[kAhead][BLOCKS][Step<FOUR>::kOperands];
  auto issue = [&](int a, int i) __attribute__((always_inline)) {
    const int step = wave + kUpWaves * i;
#pragma unroll
    for (int b = 0; b < BLOCKS; ++b) rd.rows(xs, xat[b], 0, step, x[a][b]);
    rd.weights(s, l, false, step, w[a]);
  };
  auto use = [&](int a, int) __attribute__((always_inline)) {
#pragma unroll
    for (int j = 0; j < Step<FOUR>::kOperands; ++j) {
      const bf16x8f wo = operand<FOUR>(w[a], j);
#pragma unroll
      for (int b = 0; b < BLOCKS; ++b)
        acc[b] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(wo, __builtin_bit_cast(bf16x8f, x[a][b][j]), acc[b], 0, 0, 0);
    }
  };
  pipelined<kAhead>((rd.steps() - wave + kUpWaves - 1) / kUpWaves, issue, use, [] {});
}

// SMALL: at most 64 slots.
template <bool FOUR, bool SMALL>
__global__ __launch_bounds__(64 * kUpWaves, 4) void few_up_kernel(Few p) {
  __shared__ int32_t s_expert[SMALL ? 1 : kMaxSlots];
  __shared__ uint32_t s_bits[SMALL ? 1 : GG_MAX_GROUPS_DEV / 32];
  __shared__ int32_t s_token[kMaxTokens];   // the expert's tokens,
  __shared__ int32_t s_slot[kMaxTokens];    //   the slots that name it,
  __shared__ int32_t s_more[kMaxTokens];    //   and how many more of the token's do
  __shared__ float s_share[kMaxTokens];
  __shared__ int32_t s_info[3];             // their number, the first one's workspace row, the expert
  __shared__ float s_sum[kUpWaves][16][kPitch];
  __shared__ __attribute__((aligned(16))) uint8_t s_x[kRowBytes];
  const int tid = threadIdx.x, lane = tid & 63, wave = wave_index();
  const int slots = p.tokens * p.topk;
  const int d = blockIdx.y;
  const bool leader = blockIdx.x == 0;      // of the expert's workgroups

  // Wave 0 finds the d-th reached expert and its tokens (one that names it
  // twice counts once, with both shares).  An expert has as many workspace rows
  // as it has slots.
  if constexpr (SMALL) {
    if (wave == 0) {
      int e = lane < slots ? p.experts[lane] : -1;
      e = e < p.num_groups ? e : -1;
      // experts in the order of their first slots
      uint64_t left = __ballot(e >= 0), mine = 0;
      int n = 0, base = 0, expert = 0;
      while (left != 0ull) {
        const int at = __builtin_amdgcn_readlane(e, __ffsll((unsigned long long)left) - 1);
        const uint64_t same = __ballot(e == at);
        left &= ~same;
        if (n == d) {
          mine = same;
          expert = at;
          if (!leader || d != 0) break;         // (the first workgroup counts them all)
        } else if (n < d) {
          base += __popcll(same);
        }
        ++n;
      }
      const int t = lane / p.topk, start = t * p.topk, end = start + p.topk;
      const uint64_t token = mine & ~lanes_before(start < 64 ? start : 63) & (end < 64 ? lanes_before(end) : ~0ull);
      const bool first = ((mine >> lane) & 1ull) && (token & lanes_before(lane)) == 0ull;
      const uint64_t firsts = __ballot(first);
      if (first) {
        const int i = __popcll(firsts & lanes_before(lane));
        s_token[i] = t;
        s_slot[i] = lane;
        s_more[i] = __popcll(token) - 1;
      }
      if (lane == 0) {
        s_info[0] = __popcll(firsts);
        s_info[1] = base;
        s_info[2] = expert;
      }
      if (leader) {
        uint64_t who = 0;
        for (uint64_t m = firsts; m != 0ull; m &= m - 1ull)
          who |= 1ull << __builtin_amdgcn_readlane(t, __ffsll((unsigned long long)m) - 1);
        if (lane == 0 && mine != 0ull) p.reached[d] = Reached{expert, base, who};
        if (lane == 0 && d == 0) *p.count = n;
      }
    }
  } else {
    for (int i = tid; i < GG_MAX_GROUPS_DEV / 32; i += 64 * kUpWaves) s_bits[i] = 0u;
    __syncthreads();
    for (int s = tid; s < slots; s += 64 * kUpWaves) {
      const int e = p.experts[s];
      s_expert[s] = e;
      if (e >= 0 && e < p.num_groups) atomicOr(&s_bits[e >> 5], 1u << (e & 31));
    }
    __syncthreads();
    if (wave == 0) {
      // experts by index
      const uint32_t word = s_bits[lane];
      int upto = __popc(word);
#pragma unroll
      for (int o = 1; o < 64; o <<= 1) {
        const int v = __shfl_up(upto, (unsigned)o, 64);
        if (lane >= o) upto += v;
      }
      const int reached = __shfl(upto, 63, 64);
      if (leader && d == 0 && lane == 0) *p.count = reached;
      int found = 0;
      if (d < reached) {
        const int at = __ffsll((unsigned long long)__ballot(upto > d)) - 1;
        const uint32_t bits = (uint32_t)__shfl((int)word, at, 64);
        const int nth = d - (__shfl(upto, at, 64) - __popc(bits));
        const int bit = lane & 31;
        const uint64_t hit = __ballot(((bits >> bit) & 1u) && __popc(bits & ((1u << bit) - 1u)) == nth);
        const int expert = __builtin_amdgcn_readfirstlane(32 * at + __ffsll((unsigned long long)hit) - 1);
        int base = 0;
        uint64_t who = 0;
        for (int s0 = 0; s0 < slots; s0 += 64) {
          const int s = s0 + lane;
          const int e = s < slots ? s_expert[s] : -1;
          base += __popcll(__ballot(e >= 0 && e < expert));
          if (__ballot(e == expert) == 0ull) continue;
          const int t = s / p.topk;
          bool first = e == expert;
          int more = 0;
          if (first) {
            for (int j = t * p.topk; j < s; ++j) first = first && s_expert[j] != expert;
            for (int j = s + 1; j < (t + 1) * p.topk; ++j) more += s_expert[j] == expert ? 1 : 0;
          }
          const uint64_t firsts = __ballot(first);
          if (first) {
            const int i = found + __popcll(firsts & lanes_before(lane));
            s_token[i] = t;
            s_slot[i] = s;
            s_more[i] = more;
          }
          found += __popcll(firsts);
          for (uint64_t m = firsts; m != 0ull; m &= m - 1ull)
            who |= 1ull << __builtin_amdgcn_readlane(t, __ffsll((unsigned long long)m) - 1);
        }
        if (lane == 0) {
          s_info[1] = base;
          s_info[2] = expert;
          if (leader) p.reached[d] = Reached{expert, base, who};
        }
      }
      if (lane == 0) s_info[0] = found;
    }
  }
  __syncthreads();
  const int found = __builtin_amdgcn_readfirstlane(s_info[0]);
  if (found == 0) return;
  const int base = __builtin_amdgcn_readfirstlane(s_info[1]);
  const int expert = __builtin_amdgcn_readfirstlane(s_info[2]);
  // its tokens' shares: on their way while the weights are read
  float share = 1.0f;
  if (tid < found && p.share) share = p.share[s_slot[tid]];

  const int col = lane & 15, q = lane >> 4;
  // x's rows: 16 bytes a load, zeros after them
  constexpr int kRowLoads = 2;                 // of each thread, ahead of the weights (the rest after them)
  const uint32_t per = (uint32_t)(Reader<FOUR, 1>(p.hidden, col, q).steps() * Reader<FOUR, 1>::kValues / 8);
  const uint32_t pitch = 16u * per + 64u;      // (rows a quarter of the banks apart)
  const uint32_t all = per * (uint32_t)found;
  const bool in_lds = found <= 16 && (uint64_t)pitch * (uint32_t)found <= (uint64_t)kRowBytes;
  u32x4r xv[kRowLoads];
  auto get_x = [&](int m) {
    const uint32_t c = (uint32_t)(tid + 64 * kUpWaves * m);
    u32x4r v = {0u, 0u, 0u, 0u};
    if (c < all && 8u * (c % per) < (uint32_t)p.hidden)
      v = rows::load16(p.x + (int64_t)s_token[c / per] * p.hidden + 8u * (c % per));
    return v;
  };
  auto put_x = [&](int m, const u32x4r& v) {
    const uint32_t c = (uint32_t)(tid + 64 * kUpWaves * m);
    if (c < all) *reinterpret_cast<u32x4r*>(s_x + c / per * pitch + 16u * (c % per)) = v;
  };
  if (in_lds) {
#pragma unroll
    for (int m = 0; m < kRowLoads; ++m) xv[m] = get_x(m);
  }
  const int n = (int)strips<FOUR>(p.inter);
  // strips a grid apart, so that neighbours are read at the same time
  const int block = strip_of(blockIdx.x, gridDim.x);
  for (int z = 0; z < p.strips_each; ++z) {
    const int strip = block + z * (int)gridDim.x;
    if (strip >= n) break;
    const int64_t row0 = strip_first<FOUR>(strip);
    // places 0..7 rows of W1, 8..15 the same rows of W3
    const Strip<FOUR> s(p.up, expert, row0, 2 * (int64_t)p.inter - row0);
    const Lane<FOUR> l(p.up, row0, strip_place<FOUR>(strip, col & 7) + (col >= 8 ? p.inter : 0), q);
    f32x4f acc[4];
#pragma unroll
    for (int b = 0; b < 4; ++b) acc[b] = f32x4f{0.f, 0.f, 0.f, 0.f};
    if (in_lds) {
      up_steps_lds<FOUR>(p, s, l, s_x, pitch, found, wave, col, q, acc[0], [&] {
        if (z > 0) return;
#pragma unroll
        for (int m = 0; m < kRowLoads; ++m) put_x(m, xv[m]);
        for (int m = kRowLoads; 64u * kUpWaves * m < all; ++m) put_x(m, get_x(m));
        // (the weights stay in flight)
        asm volatile("s_waitcnt lgkmcnt(0)\n\ts_barrier" ::: "memory");
      });
    } else if (found <= 16) {
      up_steps<FOUR, 1>(p, s, l, s_token, found, wave, col, q, acc);
    } else {
      up_steps<FOUR, 2>(p, s, l, s_token, found, wave, col, q, acc);
      // (beyond 32 the weights are read twice)
      if (found > 32) up_steps<FOUR, 2>(p, s, l, s_token + 32, found - 32, wave, col, q, acc + 2);
    }
    if (z == 0 && tid < found) {
      if (s_more[tid] && p.share) {              // the token's other slots that name the expert
        for (int j = s_slot[tid] + 1; j < (s_token[tid] + 1) * p.topk; ++j)
          if (p.experts[j] == expert) share += p.share[j];
      } else {
        share += (float)s_more[tid];
      }
      s_share[tid] = share;
    }
    // the waves' parts of the reduction, added in order; lane l holds token l
    // mod 16, places 4 (l / 16) .. + 3
#pragma unroll
    for (int b = 0; b < 4; ++b) {
      if (16 * b >= found) break;
      if (b > 0 || z > 0) __syncthreads();
#pragma unroll
      for (int r = 0; r < 4; ++r) s_sum[wave][col][4 * q + r] = acc[b][r];
      __syncthreads();
      if (tid < 16 * kStrip) {
        const int i = tid & (kStrip - 1), t = 16 * b + tid / kStrip;
        const int64_t c = row0 + strip_place<FOUR>(strip, i);
        if (t < found && c < p.inter) {
          float g = 0.f, u = 0.f;
#pragma unroll
          for (int w = 0; w < kUpWaves; ++w) {
            g += s_sum[w][tid / kStrip][i];
            u += s_sum[w][tid / kStrip][kStrip + i];
          }
          const float a = g * __builtin_amdgcn_rcpf(1.0f + __expf(-g)) * u * s_share[t];
          __bf16* to = reinterpret_cast<__bf16*>(p.act) + (int64_t)(base + t) * 2 * p.inter + c;
          // (a finite value above bf16's largest is that and what it left)
          const __bf16 high = (__bf16)(rows::finite(a) ? __builtin_amdgcn_fmed3f(a, -kMaxBf16, kMaxBf16) : a);
          const float left = a - (float)high;
          to[0] = high;
          // (an infinity or NaN is its own value, with nothing left)
          to[p.inter] = (__bf16)(rows::finite(left) ? left : 0.f);
        }
      }
    }
  }
}

// The value of the lane opposite in its half of a 16-lane row (7 - i for i).
__device__ __forceinline__ float half_mirror(float v) {
  return __builtin_bit_cast(float,
                            __builtin_amdgcn_update_dpp(0, __builtin_bit_cast(int, v), 0x141, 0xf, 0xf, true));
}

// The value of the lane 40 on (lanes 0..7 of each of the first two rows of 16):
// columns 8..15 of the row two on.
__device__ __forceinline__ float second_half(float v) {
  const uint32_t x = __builtin_bit_cast(uint32_t, rows::row_ror<8>(v));
  return __builtin_bit_cast(float, (uint32_t)__builtin_amdgcn_permlane32_swap(x, x, false, false)[1]);
}

// TOKENS: at most.  SUB: strips of a workgroup, side by side in their span (4
// bits): a step's four loads of rows then serve two of weights.  With both and
// their scales a strip's step costs the address unit 64 clocks instead of 96: some 25
// experts of 7168 x 2048 69 -> 55 us, 8 of them 23.5 -> 21.6.  Up to one strip for each
// compute unit they stay alone, and where experts have so many tokens that their
// rows, not the weights, take the time (I 768, 16 experts, 320 strips: 8 slots an
// expert 56.2 us alone and 54.2 in pairs, 32 slots 170 and 200; 640 strips 92 and 99,
// 292 and 368; I 512, 16 slots, 61.5 and 64.7; I 1024, 8 experts, 12 slots, 47.9 and
// 49.6).  The layer in us, 64 experts for 1 and 4 tokens to 8 each, 128 for more, one
// strip a workgroup and two:
//   strips  1 token, I 768   4 tokens, I 2048   23 tokens, I 768   64 tokens, I 768
//     128     11.6   12.6       51.6   57.9        70.6   81.0       136    157
//     256     12.6   13.6       59.8   66.1        81.9   92.0       153    174
//     272     14.1   13.9       78.1   70.0       114.4   97.6       222    182
//     368     14.9   14.5       86.3   77.6       127.0  108.8       244    202
//     512     16.7   16.3      100.2   91.9       149.2  130.8       283    242
//     640     20.6   22.1      131.8  132.1       198.7  195.3       382    372
//     896     24.7   24.7      167.8  153.9       262.2  233.8       509    440
template <bool FOUR, int TOKENS, int SUB>
__global__ __launch_bounds__(64 * kDownWaves) void few_down_kernel(Few p) {
  static_assert(SUB == 1 || FOUR, "bf16 strips do not share a span");
  __shared__ __attribute__((aligned(16))) float s_out[kDownWaves][SUB * TOKENS][kStrip];     // each wave's sums
  const int tid = threadIdx.x, lane = tid & 63, wave = wave_index();
  const int slots = p.tokens * p.topk;
  const int most = slots < p.num_groups ? slots : p.num_groups;
  // Reached experts, one a lane: the first 64 before their number is known, and
  // where that is not enough the wave's own.  (None is loaded in the loop: a load
  // that may be skipped there would make it wait for all.)
  Reached mine = {0, 0, 0};
  if (lane < most) mine = p.reached[lane];
  const int strip = SUB * strip_of(blockIdx.x, gridDim.x);
  const int col = lane & 15, q = lane >> 4;
  const bool second = col >= 8;
  const Reader<FOUR, 2> rd(p.inter, col, q);
  const int k = p.inter, steps = rd.steps();
  const int64_t row0 = strip_first<FOUR>(strip);
  const Lane<FOUR> l0(p.down, row0, strip_place<FOUR>(strip, col & 7), q);
  const Lane<FOUR> l1(p.down, row0, strip_place<FOUR>(strip + SUB - 1, col & 7), q);
  const __amdgpu_buffer_rsrc_t acts = range(p.act, (int64_t)slots * 4 * k);
  // columns 0..3 are the bf16 values of 4 of an expert's tokens, 7..4 what those
  // left; 8..15 the same at the step's second half
  const int member = (col & 4) ? 3 - (col & 3) : col & 3;
  const uint32_t act_at = (uint32_t)((2 * member + ((col >> 2) & 1)) * k + rd.first) * 2u;
  for (int i = lane; i < SUB * TOKENS * kStrip / 4; i += 64)
    reinterpret_cast<f32x4f*>(&s_out[wave][0][0])[i] = f32x4f{0.f, 0.f, 0.f, 0.f};
  const int reached = __builtin_amdgcn_readfirstlane(*p.count);

  // The reached experts' steps, one expert after the other; a wave takes an
  // equal run of them (of whole experts where there are many: at most 64).
  static_assert(kMaxSlots <= 64 * kDownWaves, "a wave holds its experts one a lane");
  const bool whole = reached >= 256;
  const int units = whole ? reached : reached * steps, unit = whole ? steps : 1;
  const int begin = units * wave / kDownWaves * unit, end = units * (wave + 1) / kDownWaves * unit;
  int d = begin / steps, step = begin - d * steps;
  if (reached > 64) {
    if (d + lane < reached) mine = p.reached[d + lane];
    d = 0;
  }
  constexpr int kAhead = FOUR ? 3 : 4;
  Raw<FOUR> w[kAhead][SUB];
  u32x4r v[kAhead][Step<FOUR>::kOperands];
  int ahead[kAhead];          // the lane of the item's expert
  // What the next item is loaded with; only the steps change from item to item of
  // an expert.
  Strip<FOUR> strip_w(p.down, 0, row0, p.hidden - row0);
  uint32_t act_lane = kOutside;
  int act_base = 0, from = -1, issue_d = d, issue_step = step;
  auto issue = [&](int a, int) __attribute__((always_inline)) {
    if (issue_d != from) {
      from = issue_d;
      strip_w = Strip<FOUR>(p.down, __builtin_amdgcn_readlane(mine.expert, from), row0, p.hidden - row0);
      act_base = 4 * __builtin_amdgcn_readlane(mine.base, from) * k;
      act_lane = member < __popcll(lane_value64(mine.tokens, from)) ? act_at : kOutside;
    }
    ahead[a] = from;
    rd.rows(acts, act_lane, act_base, issue_step, v[a]);
    rd.weights(strip_w, l0, second, issue_step, w[a][0]);
    if constexpr (SUB == 2) rd.weights(strip_w, l1, second, issue_step, w[a][1]);
    if (++issue_step == steps) {
      issue_step = 0;
      ++issue_d;
    }
  };
  auto multiply = [&](const Raw<FOUR>& wr, const u32x4r (&vr)[Step<FOUR>::kOperands], f32x4f c)
      __attribute__((always_inline)) {
#pragma unroll
    for (int j = 0; j < Step<FOUR>::kOperands; ++j)
      c = __builtin_amdgcn_mfma_f32_16x16x32_bf16(operand<FOUR>(wr, j), __builtin_bit_cast(bf16x8f, vr[j]), c, 0, 0, 0);
    return c;
  };
  // Adds tokens 4 b .. of an expert's product to the wave's sums.  (Each
  // expert's product is one of its own, so that a weight that is not finite
  // reaches the expert's own tokens only.)  Lanes 0..31 hold the first half's
  // rows in columns 0..7, lanes 32..63 the second's in 8..15: one lane adds both
  // (two lanes in turn, under conditions that exclude each other, may become one
  // instruction, which would lose one of the two).
  auto add = [&](f32x4f part, uint64_t tokens, int b, int sub) {
    f32x4f other;
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      // (an infinite weight times what the bf16 value left is NaN, or of the other sign)
      const float left = half_mirror(part[e]);
      part[e] += rows::finite(part[e]) ? left : 0.f;
      other[e] = second_half(part[e]);
    }
    const int i = kQuad * b + (col & 3);
    if ((col & 4) == 0 && q < 2 && !second && i < __popcll(tokens)) {
      uint64_t left = tokens;
      for (int z = 0; z < i; ++z) left &= left - 1ull;
      f32x4f* to = reinterpret_cast<f32x4f*>(&s_out[wave][sub * TOKENS + __ffsll((unsigned long long)left) - 1][4 * (q & 1)]);
      *to = *to + part + other;
    }
  };
  f32x4f part[SUB];
#pragma unroll
  for (int z = 0; z < SUB; ++z) part[z] = f32x4f{0.f, 0.f, 0.f, 0.f};
  int current = d;
  uint64_t tokens = end > begin ? lane_value64(mine.tokens, d) : 0ull;
  auto use = [&](auto many, int a, int i) __attribute__((always_inline)) {
    if (ahead[a] != current) {
#pragma unroll
      for (int z = 0; z < SUB; ++z) {
        add(part[z], tokens, 0, z);
        part[z] = f32x4f{0.f, 0.f, 0.f, 0.f};
      }
      current = ahead[a];
      tokens = lane_value64(mine.tokens, current);
    }
#pragma unroll
    for (int z = 0; z < SUB; ++z) part[z] = multiply(w[a][z], v[a], part[z]);
    if constexpr (decltype(many)::value) {
      const int found = __popcll(tokens), base = __builtin_amdgcn_readlane(mine.base, current);
      for (int b = 1; kQuad * b < found; ++b) {
        u32x4r more[Step<FOUR>::kOperands];
        rd.rows(acts, kQuad * b + member < found ? act_at : kOutside, 4 * (base + kQuad * b) * k, (step + i) % steps, more);
#pragma unroll
        for (int z = 0; z < SUB; ++z) add(multiply(w[a][z], more, f32x4f{0.f, 0.f, 0.f, 0.f}), tokens, b, z);
      }
    }
  };
  // (without an expert of more tokens the loop holds no loads under a condition)
  const int last = d + (step + end - begin - 1) / steps;
  if (__ballot(lane >= d && lane <= last && __popcll(mine.tokens) > kQuad) == 0ull)
    pipelined<kAhead>(end - begin, issue, [&](int a, int i) { use(std::false_type(), a, i); }, [] {});
  else
    pipelined<kAhead>(end - begin, issue, [&](int a, int i) { use(std::true_type(), a, i); }, [] {});
#pragma unroll
  for (int z = 0; z < SUB; ++z) add(part[z], tokens, 0, z);
  __syncthreads();
  for (int o = tid; o < SUB * p.tokens * kStrip; o += 64 * kDownWaves) {
    const int sub = o / kStrip % SUB, t = o / (SUB * kStrip), i = o % kStrip;
    const int64_t c = row0 + strip_place<FOUR>(strip + sub, i);
    if (c >= p.hidden) continue;
    float sum = 0.f;
#pragma unroll
    for (int z = 0; z < kDownWaves; ++z) sum += s_out[z][sub * TOKENS + t][i];
    if (p.out_f32) static_cast<float*>(p.out)[(int64_t)t * p.hidden + c] = sum;
    else static_cast<__bf16*>(p.out)[(int64_t)t * p.hidden + c] = (__bf16)sum;
  }
}

template <bool FOUR>
hipError_t launch_four(Few p, hipStream_t stream) {
  const int slots = p.tokens * p.topk;
  const int64_t most = slots < p.num_groups ? slots : p.num_groups, n = strips<FOUR>(p.inter);
  // Several strips a workgroup where there are plenty of workgroups.  The layer in us,
  // by strips a workgroup (tokens of 8 slots, experts, hidden x inter; * the rule's):
  //                                 1     2     3     4     6     8
  //   bf16 23, 128, 2048 x  704   163   159*  162   165   165   174
  //        23, 128, 2048 x  800   180   178   181*  183   187   194
  //        64, 512,  512 x  256   128   106   102    99*   95   102
  //        32, 256, 2048 x 1024   365   348   353   357*  363   368
  //   4 b   4,  64, 7168 x 2048   162   155*  153   156   163   162
  //        23, 128, 2048 x  768   106    87    82*   82    82    86
  //        64, 512,  512 x  256   104    78    71    67*   64    66
  //        32, 128, 7168 x 2048   741   712   699   715*  715   734
  const int64_t full = n * most / kUpGroups;
  const int64_t each = full < 1 ? 1 : full > kUpStrips ? kUpStrips : full;
  p.strips_each = (int32_t)each;
  const int64_t across = (n + each - 1) / each;
  auto* up = slots <= 64 ? few_up_kernel<FOUR, true> : few_up_kernel<FOUR, false>;
  const hipError_t e = launch_kernel(up, dim3((unsigned)across, (unsigned)most), dim3(64 * kUpWaves),
                                     stream, p);
  if (e != hipSuccess) return e;
  auto* down = p.tokens <= 16 ? few_down_kernel<FOUR, 16, 1> : few_down_kernel<FOUR, kMaxTokens, 1>;
  unsigned groups = (unsigned)strips<FOUR>(p.hidden);
  if constexpr (FOUR) {
    if (groups > kDownAlone && slots <= (int64_t)kDownCrowd * p.num_groups) {
      down = p.tokens <= 16 ? few_down_kernel<FOUR, 16, 2> : few_down_kernel<FOUR, kMaxTokens, 2>;
      groups /= 2;
    }
  }
  return launch_kernel(down, dim3(groups), dim3(64 * kDownWaves), stream, p);
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
