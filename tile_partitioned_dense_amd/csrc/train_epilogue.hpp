// train_epilogue.hpp -- the stores of the tile and stream kernels that belong
// to the gated block's backward pass and to the cross entropy of a projection.
//
// Each is a dense product whose owned tile is not written as C but turned, in
// the owning workgroup, into what the operator needs of it:
//
//   kEpiStats     logits l = x W^T of a large vocabulary: per row and segment
//                 of columns the running maximum m and sum of e^(l - m), the
//                 logit of the row's target, and (label smoothing) the sum of
//                 the logits. The logits themselves are never written.
//   kEpiXentGrad  the same logits computed again, turned into
//                 G = a e^(l - lse) - u - b [column is the target]
//                 (a, b, u: per row, see xent_rows_kernel).
//   kEpiGluGrad   gate and up pre-activations z = x W^T + bias turned, with
//                 the output gradient dh, into dz_gate = dh z_up act'(z_gate)
//                 and dz_up = dh act(z_gate).
//   kEpiGlu       the gated block's forward result act(z_gate) z_up, for the
//                 gates that the plain kernels' store does not know.
//   kEpiPartial   a gradient's product with K cut into `splits` parts: fp32
//                 partial results of each part, or (one part) the bf16 result
//                 times a device scalar.
//   kEpiPair      kEpiPartial in the first workgroups of a launch, the weight
//                 gradient over few tokens (outer_kernel.hpp) in the others.
//
// G and dz feed two products each: dx contracts their columns, dW their rows.
// Both want the contracted axis contiguous, so they are written twice, as
// rows and transposed: one more write of 2 bytes a value, where a transposing
// product would need a second LDS layout and twice the LDS reads for A. Both
// copies are the round-to-nearest-even bf16 of the same fp32 value, the form
// the MFMA takes; the two gradients therefore carry one rounding of G besides
// their own (both about 2^-9 of a value, independent).
//
// Everything is formed from the accumulator registers of one wave: lane l of
// a 16-row block holds row l % 16, columns 16 j + 4 (l / 16) .. + 3 of block
// j, so a row's maximum and sum are a loop over registers and two exchanges
// across the lanes. No LDS traffic for kEpiStats; the gradients stage 16 (or
// 32) rows of bf16 in a strip of LDS that is private to the wave.
#pragma once

#include <type_traits>

#include "tile_kernel.hpp"

namespace tg {

constexpr int kEpiNone = 0, kEpiStats = 1, kEpiXentGrad = 2, kEpiGluGrad = 3, kEpiPartial = 4, kEpiGlu = 5,
              kEpiPair = 6;
constexpr bool epi_partial(int epi) { return epi == kEpiPartial || epi == kEpiPair; }

// A gated store can have its gate compiled in, EPI = kind + 16 (gate + 1): the
// one-wave-per-SIMD kernel's 256 accumulators stay where the MFMAs left them
// only if a single code path reads them (five of them made the compiler move
// accumulators inside the K loop). The others take it from the arguments.
constexpr int epi_kind(int epi) { return epi & 15; }
constexpr int epi_gate(int epi) { return (epi >> 4) - 1; }
constexpr int with_gate(int kind, int gate) { return kind + 16 * (gate + 1); }
constexpr bool epi_gated(int epi) { return epi_kind(epi) == kEpiGluGrad || epi_kind(epi) == kEpiGlu; }

// Per-row constants of kEpiXentGrad (xent_rows_kernel): the log-sum-exp, a, b
// and the target's column (-1: none).
struct XentRow {
  float lse, a, b;
  int32_t target;
};

struct TrainArgs : TileArgs {
  // kEpiStats
  const void* target;  // M targets, int32 or int64
  int32_t target64;
  float2* part;     // [segment][M]: maximum, sum
  float* part_sum;  // [segment][M]: sum of the logits, or NULL
  float* hit;       // [M]: the target's logit (rows without one are not written)
  // kEpiXentGrad
  const XentRow* rows;   // NULL (at most 64 rows, stream kernel): formed from the fields below
  const float* lse;
  const float* dloss;
  int64_t ignore, vocab;
  float z_loss;
  float* row_scale;      // where the largest |dloss| goes
  int32_t first;  // vocabulary column of this launch's column 0 (kEpiStats too)
  float smooth;   // u = b * smooth (label smoothing over the vocabulary size)
  float keep;     // the target's share: b * keep is subtracted there
  // kEpiXentGrad, kEpiGluGrad: the result as rows and transposed (either NULL)
  uint16_t* Z;
  int64_t ldz;
  uint16_t* Zt;
  int64_t ldzt;
  // kEpiGluGrad
  const uint16_t* dC;
  int64_t lddc;
  float* dbias_part;  // [tile row, wave row][2 F] column sums, or NULL
  int32_t gate;
  // kEpiPartial
  int32_t splits, k_per;
  int64_t part_stride;  // elements between the partial results
  const float* scale;   // bf16 result: one fp32 value, or NULL
};

struct PairArgs;  // outer_kernel.hpp
template <int EPI>
using EpiArgs = std::conditional_t<EPI == kEpiNone, TileArgs, std::conditional_t<EPI == kEpiPair, PairArgs, TrainArgs>>;

constexpr float kLog2e = 1.44269504088896341f;

__device__ __forceinline__ float lane_xor(float v, int m) { return __shfl_xor(v, m, 64); }

// The value of the lane 16 (SPAN = 16) or 32 lanes away joined with the
// lane's own: both halves of an exchange of a register with itself. These run
// in the vector ALU, where a cross-lane move through LDS would cost its
// latency with no other wave on the SIMD to fill it.
template <int SPAN, class Op>
__device__ __forceinline__ float join_lanes(float v, Op op) {
  const uint32_t u = __float_as_uint(v);
  if constexpr (SPAN == 16) {
    const auto r = __builtin_amdgcn_permlane16_swap(u, u, false, false);
    return op(__uint_as_float(r[0]), __uint_as_float(r[1]));
  } else {
    const auto r = __builtin_amdgcn_permlane32_swap(u, u, false, false);
    return op(__uint_as_float(r[0]), __uint_as_float(r[1]));
  }
}

__device__ __forceinline__ int64_t target_of(const void* target, int is64, int64_t row) {
  return is64 ? static_cast<const int64_t*>(target)[row] : (int64_t) static_cast<const int32_t*>(target)[row];
}

// Constants of the loss gradient of one row: target t, log-sum-exp, dloss / c
// (see xent_rows_kernel).
__device__ __forceinline__ XentRow xent_row(int64_t t, int64_t ignore, int64_t vocab, float lse, float dloss,
                                            float c, float z_loss) {
  XentRow r{lse, 0.0f, 0.0f, -1};
  if (t != ignore) {
    const bool known = t >= 0 && t < vocab;
    r.b = known ? dloss / c : NAN;
    r.a = r.b * fmaf(2.0f * z_loss, lse, 1.0f);
    r.target = known ? (int32_t)t : -1;
  }
  return r;
}
// The common factor of the loss gradients from their largest absolute value.
__device__ __forceinline__ float xent_scale(float c) { return c > 0.0f && c < INFINITY ? c : 1.0f; }

// Column of row `row`'s target, relative to column `first` of this launch; -1
// where the row or its target is outside.
__device__ __forceinline__ int target_col(const TrainArgs& p, int row, int first) {
  if (row >= p.M) return -1;
  const uint64_t c = (uint64_t)target_of(p.target, p.target64, row) - (uint64_t)((int64_t)p.first + first);
  return c < (uint64_t)(int64_t)(p.N - first) ? (int)c : -1;
}

// Maximum, sum of exponentials, (sum) and target of one row held as NJ groups
// of four consecutive columns, group j at column step * j + 4 lg of a segment
// that starts at column col0 (col0 < N). The lanes of a row differ in lg (two
// or, with FOUR, four of them). c: the target's column in the segment.
template <int NJ, bool FOUR>
__device__ __forceinline__ void stats_row(floatx4 (&v)[NJ], int step, int lg, int col0, int row, int c,
                                          int64_t seg, const TrainArgs& p) {
  const auto add = [](float x, float y) { return x + y; };
  const auto most = [](float x, float y) { return fmaxf(x, y); };
  auto join = [&](float x, auto op) {
    if constexpr (FOUR) x = join_lanes<16>(x, op);
    return join_lanes<32>(x, op);
  };
  const int left = p.N - col0 - 4 * lg;  // columns of this lane's groups inside the vocabulary
  float sum = 0.0f;
  if (p.part_sum) {
#pragma unroll
    for (int j = 0; j < NJ; ++j)
#pragma unroll
      for (int e = 0; e < 4; ++e) sum += (step * j + e < left) ? v[j][e] : 0.0f;
  }
  if (p.N - col0 < step * NJ) {
#pragma unroll
    for (int j = 0; j < NJ; ++j)
#pragma unroll
      for (int e = 0; e < 4; ++e) v[j][e] = (step * j + e < left) ? v[j][e] : -INFINITY;
  }
  float m = -INFINITY;
#pragma unroll
  for (int j = 0; j < NJ; ++j)
#pragma unroll
    for (int e = 0; e < 4; ++e) m = fmaxf(m, v[j][e]);
  m = join(m, most);
  // An infinite maximum is not subtracted: a segment of logits that are all
  // -inf has the sum 0 (not the NaN of inf - inf), one with an inf the sum inf.
  // Subtracted before the scaling, not with it in one fma: the maximum's own
  // exponential is then exactly 1. The rounding of its multiple would be a
  // common factor of the sum: 5e-6 at 100, the whole loss of a nearly certain
  // token; inf from 1e10 on, and so NaN where columns are masked by a large
  // negative value. (Loss and gradients of 3001 x 2048 x 50257: 2189 to 2201 us.)
  const float ref = fabsf(m) < INFINITY ? m : 0.0f;
  // written as passes over independent values: the exponential's latency
  // would otherwise be paid once per value, with no other wave to hide it
  float x[4 * NJ];
#pragma unroll
  for (int j = 0; j < NJ; ++j)
#pragma unroll
    for (int e = 0; e < 4; ++e) x[4 * j + e] = (v[j][e] - ref) * kLog2e;
#pragma unroll
  for (int k = 0; k < 4 * NJ; ++k) x[k] = __builtin_amdgcn_exp2f(x[k]);
  float part4[4] = {x[0], x[1], x[2], x[3]};
#pragma unroll
  for (int k = 4; k < 4 * NJ; ++k) part4[k & 3] += x[k];
  float s = (part4[0] + part4[1]) + (part4[2] + part4[3]);
  s = join(s, add);
  if (c >= 0 && c < step * NJ) {
    // few rows have their target in this segment: the search is skipped by
    // every other wave
#pragma unroll
    for (int j = 0; j < NJ; ++j)
#pragma unroll
      for (int e = 0; e < 4; ++e)
        if (c == step * j + 4 * lg + e) p.hit[row] = v[j][e];
  }
  if (p.part_sum) sum = join(sum, add);
  if (lg == 0 && row < p.M) {
    p.part[seg * p.M + row] = make_float2(m, s);
    if (p.part_sum) p.part_sum[seg * p.M + row] = sum;
  }
}

// G of NV logits of one row, value k being column col(k) of the wave's segment
// (XentRow's constants, its target relative to the segment). Rows that count
// for nothing (b = 0) give exact zeros whatever their logits are. `near`:
// whether any row of the wave has its target in the segment; few do, and the
// others skip the comparisons. (The subtraction comes before the scaling, as in
// stats_row: a multiple of the log-sum-exp is off by more than any exponent
// where that is large.)
template <int NV, class Get, class Col>
__device__ __forceinline__ void xent_grad(float (&g)[NV], Get logit, Col col, const XentRow& r, bool near,
                                          const TrainArgs& p) {
#pragma unroll
  for (int k = 0; k < NV; ++k) g[k] = (logit(k) - r.lse) * kLog2e;
#pragma unroll
  for (int k = 0; k < NV; ++k) g[k] = __builtin_amdgcn_exp2f(g[k]);
#pragma unroll
  for (int k = 0; k < NV; ++k) g[k] = r.b == 0.0f ? 0.0f : r.a * g[k];
  if (p.smooth != 0.0f) {
    const float u = r.b * p.smooth;
#pragma unroll
    for (int k = 0; k < NV; ++k) g[k] -= u;
  }
  if (near) {
    const float hit = r.b * p.keep;
#pragma unroll
    for (int k = 0; k < NV; ++k) g[k] -= col(k) == r.target ? hit : 0.0f;
  }
}

// act(z) and act'(z).
//   silu     z s, s (1 + z (1 - s)) with s = 1 / (1 + e^-z)
//   gelu     z P, P + z p with P the normal distribution function, p its
//            density; P from the rational approximation of erfc(x) e^(x^2) by
//            Hastings (Abramowitz and Stegun 7.1.26, error of erfc at most
//            1.5e-7), which shares its exponential with p
//   gelu_tanh  z (1 + t) / 2, t = tanh(y), y = c (z + 0.044715 z^3), written
//            with s = 1 / (1 + e^-2y) = (1 + t) / 2: z s and
//            s + z s (1 - s) 2 c (1 + 0.134145 z^2); in both this and silu
//            the rounding of 1 - s near s = 1 is small against the slope of
//            about 1 there
//   relu     z, 1 for z > 0, else 0 (also of -inf; NaN stays)
//   sigmoid  s, s (1 - s), 1 - s from its own exponential (it is the value)
constexpr int kGateSilu = 0, kGateGelu = 1, kGateGeluTanh = 2, kGateRelu = 3, kGateSigmoid = 4;

template <int GATE>
__device__ __forceinline__ void gate_both(float z, float& act, float& slope) {
  if constexpr (GATE == kGateSilu) {
    const float s = sigmoid_hw(z);
    act = z * s;
    slope = s * fmaf(z, 1.0f - s, 1.0f);
  } else if constexpr (GATE == kGateGelu) {
    const float x = fabsf(z) * 0.70710678118654752f, ex = exp_hw(-x * x);
    const float t = __builtin_amdgcn_rcpf(fmaf(0.3275911f, x, 1.0f));
    float q = fmaf(1.061405429f, t, -1.453152027f);
    q = fmaf(q, t, 1.421413741f);
    q = fmaf(q, t, -0.284496736f);
    q = fmaf(q, t, 0.254829592f);
    q *= 0.5f * t * ex;  // erfc(x) / 2
    const float P = z < 0.0f ? q : 1.0f - q;
    act = z * P;
    slope = fmaf(z * 0.39894228040143268f, ex, P);
  } else if constexpr (GATE == kGateGeluTanh) {
    const float y2 = 1.5957691216057308f * z * fmaf(0.044715f * z, z, 1.0f);
    const float s = sigmoid_hw(y2);
    act = z * s;
    // (1 - s is 0 long before the square is cut off)
    const float sq = fminf(z * z, 1e30f);
    slope = fmaf(z * s, (1.0f - s) * (1.5957691216057308f * fmaf(0.134145f, sq, 1.0f)), s);
  } else if constexpr (GATE == kGateRelu) {
    slope = z > 0.0f ? 1.0f : 0.0f;
    act = z < 0.0f ? 0.0f : z;
  } else {
    const float s = sigmoid_hw(z);
    act = s;
    slope = s * sigmoid_hw(-z);
  }
}

typedef uint32_t u32x2s __attribute__((ext_vector_type(2)));
typedef uint32_t u32x4s __attribute__((ext_vector_type(4)));

__device__ __forceinline__ void lds_store_u32x2(uint32_t addr, uint32_t a, uint32_t b) {
  *(__attribute__((address_space(3))) u32x2s*)(uintptr_t)addr = u32x2s{a, b};
}
__device__ __forceinline__ uint32_t lds_load_u32(uint32_t addr) {
  return *(const __attribute__((address_space(3))) uint32_t*)(uintptr_t)addr;
}

// Write a wave's strip of ROWS x COLS bf16 values (LDS address `strip`, row
// pitch COLS * 2 + 16 bytes; rows grow0 ..) as rows of p.Z and transposed into
// p.Zt. col_of(c) gives the output column of strip column c (a multiple of
// 8's worth of columns stays together), or -1 where it is outside. Both
// leading dimensions are padded (ldz to 8 columns, ldzt to 16 rows), so whole
// chunks are written wherever their first value is inside, with zeros past the
// last column or row: the products that follow load whole chunks. No waits are written between the strip's writes, its reads and
// the next writes: a wave's LDS operations run in order.
template <int ROWS, int COLS, class ColOf>
__device__ __forceinline__ void store_both(uint32_t strip, int lane, int grow0, const TrainArgs& p,
                                           ColOf col_of) {
  constexpr int PITCH = COLS * 2 + 16;
  if (p.Z) {
    constexpr int CH = COLS / 8;
#pragma unroll
    for (int c0 = 0; c0 < ROWS * CH; c0 += 64) {
      const int c = c0 + lane;
      if (ROWS * CH % 64 != 0 && c >= ROWS * CH) break;
      const int r = c / CH, ch = c - (c / CH) * CH;
      u32x4s v =
          *(const __attribute__((address_space(3))) u32x4s*)(uintptr_t)(strip + (uint32_t)(r * PITCH + ch * 16));
      const int col = col_of(ch * 8), row = grow0 + r;
      if (row < p.M && col >= 0) {
        if (col + 8 > p.N) {
#pragma unroll
          for (int w = 0; w < 4; ++w)
            v[w] &= col + 2 * w + 2 <= p.N ? 0xffffffffu : col + 2 * w < p.N ? 0xffffu : 0u;
        }
        *reinterpret_cast<u32x4s*>(p.Z + (int64_t)row * p.ldz + col) = v;
      }
    }
  }
  if (p.Zt) {
    if constexpr (ROWS == 16) {
      // Transposing 8-byte reads: within 16 lanes, lane 4 j + q names row j,
      // columns 4 q .. + 3 of a 4 x 16 block and receives the four rows of
      // column lane % 16. Each 16 lanes take another 16-column block, four
      // reads the sixteen rows: 32 consecutive bytes of one column per lane.
      constexpr int NB = COLS / 16;
      const int g = lane >> 4, l16 = lane & 15;
      const uint32_t src = strip + (uint32_t)((l16 >> 2) * PITCH + (l16 & 3) * 8);
#pragma unroll
      for (int b0 = 0; b0 < NB; b0 += 4) {
        const int b = b0 + g < NB ? b0 + g : NB - 1;  // idle lanes repeat the last block
        i16x4 t[4];
#pragma unroll
        for (int q = 0; q < 4; ++q)
          t[q] = __builtin_amdgcn_ds_read_tr16_b64_v4i16(
              (__attribute__((address_space(3))) i16x4*)(uintptr_t)(src + (uint32_t)(4 * q * PITCH + b * 32)));
        const int cs = 16 * b + l16, col8 = col_of(cs & ~7);
        const int c = col8 + (cs & 7);
        if (b0 + g < NB && grow0 < p.M && col8 >= 0 && c < p.N) {
          u32x4s* z = reinterpret_cast<u32x4s*>(p.Zt + (int64_t)c * p.ldzt + grow0);
          const u32x2s w[4] = {__builtin_bit_cast(u32x2s, t[0]), __builtin_bit_cast(u32x2s, t[1]),
                               __builtin_bit_cast(u32x2s, t[2]), __builtin_bit_cast(u32x2s, t[3])};
          z[0] = u32x4s{w[0].x, w[0].y, w[1].x, w[1].y};
          z[1] = u32x4s{w[2].x, w[2].y, w[3].x, w[3].y};
        }
      }
    } else {
      // 32 x 32 (the stream kernel): a lane takes two columns and eight rows
      static_assert(ROWS == 32 && COLS == 32, "one lane per column pair and eight rows");
      const int pr = lane & 15, rg = lane >> 4;
      const int col = col_of((2 * pr) & ~7);
      uint32_t d[8];
#pragma unroll
      for (int r = 0; r < 8; ++r) d[r] = lds_load_u32(strip + (uint32_t)((rg * 8 + r) * PITCH + pr * 4));
      const int row = grow0 + rg * 8;
      if (row < p.M && col >= 0) {
        const int c = col + ((2 * pr) & 7);
        u32x4s lo, hi;
#pragma unroll
        for (int r = 0; r < 4; ++r) {
          lo[r] = pack_halves(d[2 * r], d[2 * r + 1], false);
          hi[r] = pack_halves(d[2 * r], d[2 * r + 1], true);
        }
        uint16_t* z0 = p.Zt + (int64_t)c * p.ldzt + row;
        if (c < p.N) *reinterpret_cast<u32x4s*>(z0) = lo;
        if (c + 1 < p.N) *reinterpret_cast<u32x4s*>(z0 + p.ldzt) = hi;
      }
    }
  }
}

// Gated stores: every 16-column block of the tile is 8 gate columns and the
// matching 8 up columns (b_col of the kernels), so lanes 0-31 hold gate and
// lanes 32-63 up pre-activations. Exchanging the upper half of block j with
// the lower half of block j + 1 leaves each lane with the gate (g) and up (u)
// values of four consecutive outputs, lanes 0-31 of block j and lanes 32-63 of
// block j + 1; the last block of an odd number is paired with itself, its
// upper lanes then count for nothing (glu_live). Any width of 16 columns works.
template <int J, int FN>
__device__ __forceinline__ void glu_pair(const floatx4 (&row)[FN], float (&g)[4], float (&u)[4]) {
  constexpr int J1 = 2 * J + 1 < FN ? 2 * J + 1 : 2 * J;
#pragma unroll
  for (int e = 0; e < 4; ++e) {
    const auto r = __builtin_amdgcn_permlane32_swap(__float_as_uint(row[2 * J][e]), __float_as_uint(row[J1][e]),
                                                    false, false);
    g[e] = __uint_as_float(r[0]);
    u[e] = __uint_as_float(r[1]);
  }
}
// First output column (relative to the wave's first) of a lane's pair J, and
// whether the pair is there at all.
template <int J>
__device__ __forceinline__ int glu_col(int lg) {
  return 8 * (2 * J + (lg >> 1)) + 4 * (lg & 1);
}
template <int J, int FN>
__device__ __forceinline__ bool glu_live(int lg) {
  return 2 * J + 1 < FN || lg < 2;
}

// The bias of a lane's gate and up columns, one load for all block rows.
template <int NP>
__device__ __forceinline__ void glu_bias(floatx4 (&bg)[NP], floatx4 (&bu)[NP], int lg, int col0,
                                         const TrainArgs& p) {
#pragma unroll
  for (int j = 0; j < NP; ++j) {
    const int c = col0 + 8 * (2 * j + (lg >> 1)) + 4 * (lg & 1);
    bg[j] = bu[j] = floatx4{};
    if (p.bias && c < p.glu_half) {
      bg[j] = *reinterpret_cast<const floatx4*>(p.bias + c);
      bu[j] = *reinterpret_cast<const floatx4*>(p.bias + p.glu_half + c);
    }
  }
}

// kEpiGluGrad for one gate; see train_store.
template <int GATE, int FM, int FN, class Pin>
__device__ __forceinline__ void glu_grad_store(floatx4 (&acc)[FM][FN], uint32_t strip, int lane, int row0,
                                               int col0, int wave_row, const TrainArgs& p, Pin pin) {
  constexpr int NP = (FN + 1) / 2;
  constexpr int PITCH = FN * 32 + 16;
  const int l16 = lane & 15, lg = lane >> 4;
  const int F = p.glu_half;
  float db[NP][2][4];
#pragma unroll
  for (int j = 0; j < NP; ++j)
#pragma unroll
    for (int e = 0; e < 4; ++e) db[j][0][e] = db[j][1][e] = 0.0f;
  floatx4 bg[NP], bu[NP];
  glu_bias(bg, bu, lg, col0, p);
  // dh of a block row is loaded one block row ahead
  u32x2s dn[NP];
  auto load_dh = [&](int i) {
    const int row = row0 + 16 * i + l16;
#pragma unroll
    for (int j = 0; j < NP; ++j) {
      const int c = col0 + 8 * (2 * j + (lg >> 1)) + 4 * (lg & 1);
      dn[j] = u32x2s{0u, 0u};
      if (row < p.M && c < F) dn[j] = *reinterpret_cast<const u32x2s*>(p.dC + (int64_t)row * p.lddc + c);
    }
  };
  load_dh(0);
  static_for<0, FM>([&](auto i_c) {
    constexpr int i = decltype(i_c)::value;
    pin(acc[i]);
    u32x2s dc[NP];
#pragma unroll
    for (int j = 0; j < NP; ++j) dc[j] = dn[j];
    if constexpr (i + 1 < FM) load_dh(i + 1);
    static_for<0, NP>([&](auto j_c) {
      constexpr int j = decltype(j_c)::value;
      float g[4], u[4];
      glu_pair<j>(acc[i], g, u);
      const int cw = glu_col<j>(lg);
      if (glu_live<j, FN>(lg)) {
        // rows and columns outside have dh = 0; what their pre-activations are
        // (rows past M are zero, columns past F those of another half) must
        // not matter, so their results are set, not multiplied
        const bool live = row0 + 16 * i + l16 < p.M && col0 + cw < F;
        const float dh[4] = {__uint_as_float(dc[j].x << 16), __uint_as_float(dc[j].x & 0xffff0000u),
                             __uint_as_float(dc[j].y << 16), __uint_as_float(dc[j].y & 0xffff0000u)};
        float dg[4], du[4];
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          float act, slope;
          gate_both<GATE>(g[e] + bg[j][e], act, slope);
          dg[e] = live ? dh[e] * (u[e] + bu[j][e]) * slope : 0.0f;
          du[e] = live ? dh[e] * act : 0.0f;
          db[j][0][e] += dg[e];
          db[j][1][e] += du[e];
        }
        const uint32_t a = strip + (uint32_t)(l16 * PITCH + cw * 2);
        lds_store_u32x2(a, pack_bf16x2(dg[0], dg[1]), pack_bf16x2(dg[2], dg[3]));
        lds_store_u32x2(a + FN * 16, pack_bf16x2(du[0], du[1]), pack_bf16x2(du[2], du[3]));
      }
    });
    store_both<16, FN * 16>(strip, lane, row0 + 16 * i, p, [&](int c) {
      const int h = c >= FN * 8, k = col0 + c - h * FN * 8;
      return k < F ? k + h * F : -1;
    });
    __builtin_amdgcn_sched_barrier(0);  // block rows in turn: interleaved, they spill
  });
  if (!p.dbias_part) return;
  // column sums of the wave's rows, in fp32 before the rounding of dz
  static_for<0, NP>([&](auto j_c) {
    constexpr int j = decltype(j_c)::value;
    const int c = col0 + glu_col<j>(lg);
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      float t[4];
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        t[e] = db[j][h][e];
        t[e] += lane_xor(t[e], 1);
        t[e] += lane_xor(t[e], 2);
        t[e] += lane_xor(t[e], 4);
        t[e] += lane_xor(t[e], 8);
      }
      if (l16 == 0 && glu_live<j, FN>(lg) && c < F)
        *reinterpret_cast<float4*>(p.dbias_part + (int64_t)wave_row * (2 * F) + h * F + c) =
            make_float4(t[0], t[1], t[2], t[3]);
    }
  });
}

// kEpiGlu for one gate: the results of 16 rows at a time are staged and stored
// as 16-byte row chunks.
template <int GATE, bool OUT_BF16, int FM, int FN, class Pin>
__device__ __forceinline__ void glu_store(floatx4 (&acc)[FM][FN], uint32_t strip, int lane, int row0,
                                          int col0, const TrainArgs& p, Pin pin) {
  constexpr int NP = (FN + 1) / 2;
  constexpr int ESZ = OUT_BF16 ? 2 : 4;
  constexpr int PITCH = FN * 8 * ESZ + 16;
  constexpr int CH = FN * 8 * ESZ / 16, EPC = 16 / ESZ;
  const int l16 = lane & 15, lg = lane >> 4;
  const int F = p.glu_half;
  floatx4 bg[NP], bu[NP];
  glu_bias(bg, bu, lg, col0, p);
  static_for<0, FM>([&](auto i_c) {
    constexpr int i = decltype(i_c)::value;
    pin(acc[i]);
    static_for<0, NP>([&](auto j_c) {
      constexpr int j = decltype(j_c)::value;
      float g[4], u[4];
      glu_pair<j>(acc[i], g, u);
      floatx4 v;
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        float act, slope;
        gate_both<GATE>(g[e] + bg[j][e], act, slope);
        v[e] = act * (u[e] + bu[j][e]);
      }
      if (glu_live<j, FN>(lg)) {
        const uint32_t a = strip + (uint32_t)(l16 * PITCH + glu_col<j>(lg) * ESZ);
        if constexpr (OUT_BF16)
          lds_store_u32x2(a, pack_bf16x2(v[0], v[1]), pack_bf16x2(v[2], v[3]));
        else
          lds_store_f4(a, v);
      }
    });
#pragma unroll
    for (int c0 = 0; c0 < 16 * CH; c0 += 64) {
      const int c = c0 + lane;
      if (16 * CH % 64 != 0 && c >= 16 * CH) break;
      const int r = c / CH, ch = c - (c / CH) * CH;
      const u32x4s v =
          *(const __attribute__((address_space(3))) u32x4s*)(uintptr_t)(strip + (uint32_t)(r * PITCH + ch * 16));
      const int row = row0 + 16 * i + r, col = col0 + ch * EPC;
      // F is a multiple of 8: a chunk is inside or outside as a whole
      if (row < p.M && col < F)
        *reinterpret_cast<u32x4s*>(static_cast<char*>(p.C) + ((int64_t)row * p.ldc + col) * ESZ) = v;
    }
  });
}

// Calls f(integral_constant<int, gate>) for a gate known only at run time.
template <class F>
__device__ __forceinline__ void for_gate(int gate, F f) {
  switch (gate) {
    case kGateGelu: f(std::integral_constant<int, kGateGelu>{}); break;
    case kGateGeluTanh: f(std::integral_constant<int, kGateGeluTanh>{}); break;
    case kGateRelu: f(std::integral_constant<int, kGateRelu>{}); break;
    case kGateSigmoid: f(std::integral_constant<int, kGateSigmoid>{}); break;
    default: f(std::integral_constant<int, kGateSilu>{});
  }
}

// The store of a wave's FM x FN blocks (16 x 16 each) of its tile, rows
// row0 .. and columns col0 .. (gated: 8 FN output columns from col0). `strip`
// is LDS private to the wave;
// `pin` ties block row i's accumulators to this point of the program.
template <int EPI, bool OUT_BF16, int FM, int FN, class Pin>
__device__ __forceinline__ void train_store(floatx4 (&acc)[FM][FN], uint32_t strip, int lane, int row0,
                                            int col0, int64_t seg, int wave_row, const TrainArgs& p,
                                            Pin pin) {
  const int l16 = lane & 15, lg = lane >> 4;
  constexpr int KIND = epi_kind(EPI);
  if constexpr (KIND == kEpiStats) {
    if (col0 >= p.N) return;
    int c[FM];  // loaded together: one latency, not one for each block row
#pragma unroll
    for (int i = 0; i < FM; ++i) c[i] = target_col(p, row0 + 16 * i + l16, col0);
    static_for<0, FM>([&](auto i_c) {
      constexpr int i = decltype(i_c)::value;
      pin(acc[i]);
      stats_row<FN, true>(acc[i], 16, lg, col0, row0 + 16 * i + l16, c[i], seg, p);
    });
  } else if constexpr (KIND == kEpiXentGrad) {
    constexpr int PITCH = FN * 32 + 16;
    if (col0 >= p.N) return;
    XentRow r[FM];
#pragma unroll
    for (int i = 0; i < FM; ++i) {
      const int row = row0 + 16 * i + l16;
      r[i] = row < p.M ? p.rows[row] : XentRow{0.0f, 0.0f, 0.0f, -1};
      r[i].target -= p.first + col0;
    }
    static_for<0, FM>([&](auto i_c) {
      constexpr int i = decltype(i_c)::value;
      pin(acc[i]);
      float g[4 * FN];
      xent_grad(g, [&](int k) { return acc[i][k >> 2][k & 3]; },
                [&](int k) { return 16 * (k >> 2) + 4 * lg + (k & 3); }, r[i],
                __any(r[i].target >= 0 && r[i].target < 16 * FN), p);
#pragma unroll
      for (int j = 0; j < FN; ++j)
        lds_store_u32x2(strip + (uint32_t)(l16 * PITCH + (16 * j + 4 * lg) * 2),
                        pack_bf16x2(g[4 * j], g[4 * j + 1]), pack_bf16x2(g[4 * j + 2], g[4 * j + 3]));
      store_both<16, FN * 16>(strip, lane, row0 + 16 * i, p,
                              [&](int c) { return col0 + c < p.N ? col0 + c : -1; });
    });
  } else {
    if (col0 >= p.glu_half) return;
    auto run = [&](auto gate) {
      constexpr int GATE = decltype(gate)::value;
      if constexpr (KIND == kEpiGluGrad)
        glu_grad_store<GATE>(acc, strip, lane, row0, col0, wave_row, p, pin);
      else
        glu_store<GATE, OUT_BF16>(acc, strip, lane, row0, col0, p, pin);
    };
    if constexpr (epi_gate(EPI) >= 0)
      run(std::integral_constant<int, epi_gate(EPI)>{});
    else
      for_gate(p.gate, run);
  }
}

// The same stores for the stream kernel's 32 x 32 blocks, FM of them down one
// 32-column block: lane l holds row l % 32, columns 8 q + 4 (l / 32) .. + 3 in
// elements 4 q .. + 3.
constexpr int kStrip32 = 32 * 2 + 16;  // bytes of a strip row

template <int EPI, int FM>
__device__ __forceinline__ void train_store_32(floatx16 (&acc)[FM], uint32_t strip, int lane, int row0,
                                               int col0, int64_t seg, const TrainArgs& p) {
  static_assert(EPI == kEpiStats || EPI == kEpiXentGrad, "logits only; kEpiGlu has its own");
  const int lrow = lane & 31, lgrp = lane >> 5;
  if (col0 >= p.N) return;
  // At most 64 rows and few tiles: each wave finds the largest |dloss| and its
  // rows' constants itself, a lane a row, which spares a launch
  // (24 rows of 1024 against 8191 columns: 3.5 of 47 us with its issue).
  [[maybe_unused]] float scale = 1.0f;
  if constexpr (EPI == kEpiXentGrad) {
    if (!p.rows) {
      float c = 0.0f;
      if (lane < p.M && target_of(p.target, p.target64, lane) != p.ignore) c = fabsf(p.dloss[lane]);
#pragma unroll
      for (int h = 32; h > 0; h /= 2) c = fmaxf(c, lane_xor(c, h));
      scale = xent_scale(c);
      if (lane == 0 && row0 == 0 && col0 == 0) *p.row_scale = scale;
    }
  }
#pragma unroll
  for (int i = 0; i < FM; ++i) {
    const int row = row0 + 32 * i + lrow;
    if constexpr (EPI == kEpiStats) {
      floatx4 v[4];
#pragma unroll
      for (int q = 0; q < 4; ++q)
        v[q] = floatx4{acc[i][4 * q], acc[i][4 * q + 1], acc[i][4 * q + 2], acc[i][4 * q + 3]};
      stats_row<4, false>(v, 8, lgrp, col0, row, target_col(p, row, col0), seg, p);
    } else {
      XentRow r{0.0f, 0.0f, 0.0f, -1};
      if (row < p.M)
        r = p.rows ? p.rows[row]
                   : xent_row(target_of(p.target, p.target64, row), p.ignore, p.vocab, p.lse[row], p.dloss[row],
                              scale, p.z_loss);
      r.target -= p.first + col0;
      float g[16];
      xent_grad(g, [&](int k) { return acc[i][k]; },
                [&](int k) { return 8 * (k >> 2) + 4 * lgrp + (k & 3); }, r,
                __any(r.target >= 0 && r.target < 32), p);
#pragma unroll
      for (int q = 0; q < 4; ++q)
        lds_store_u32x2(strip + (uint32_t)(lrow * kStrip32 + (8 * q + 4 * lgrp) * 2),
                        pack_bf16x2(g[4 * q], g[4 * q + 1]), pack_bf16x2(g[4 * q + 2], g[4 * q + 3]));
      store_both<32, 32>(strip, lane, row0 + 32 * i, p,
                         [&](int c) { return col0 + c < p.N ? col0 + c : -1; });
    }
  }
}

// kEpiGlu of the stream kernel. The gate and up columns of an output are in
// different 32-column blocks, so a block-wide strip holds ROWS x (COLS gate,
// COLS up) fp32 pre-activations (row pitch in bytes) and all threads form one
// 16-byte output chunk each at a time.
template <bool OUT_BF16, int ROWS, int COLS>
__device__ __forceinline__ void glu_strip(uint32_t src, int pitch, int row0, int col0, int tid, int nthr,
                                          const TrainArgs& p) {
  constexpr int EPC = OUT_BF16 ? 8 : 4;
  constexpr int ESZ = OUT_BF16 ? 2 : 4;
  constexpr int CH = COLS / EPC;
  const int F = p.glu_half;
  for_gate(p.gate, [&](auto gate) {
    for (int c = tid; c < ROWS * CH; c += nthr) {
      const int r = c / CH, ch = c - (c / CH) * CH;
      const int row = row0 + r, col = col0 + ch * EPC;
      if (row >= p.M || col >= F) continue;
      float v[EPC];
#pragma unroll
      for (int h = 0; h < EPC / 4; ++h) {
        const uint32_t a = src + (uint32_t)(r * pitch + (ch * EPC + 4 * h) * 4);
        floatx4 g = lds_load_f4(a), u = lds_load_f4(a + (uint32_t)(COLS * 4));
        if (p.bias) {
          g += *reinterpret_cast<const floatx4*>(p.bias + col + 4 * h);
          u += *reinterpret_cast<const floatx4*>(p.bias + F + col + 4 * h);
        }
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          float act, slope;
          gate_both<decltype(gate)::value>(g[e], act, slope);
          v[4 * h + e] = act * u[e];
        }
      }
      char* out = static_cast<char*>(p.C) + ((int64_t)row * p.ldc + col) * ESZ;
      if constexpr (OUT_BF16)
        *reinterpret_cast<u32x4s*>(out) = u32x4s{pack_bf16x2(v[0], v[1]), pack_bf16x2(v[2], v[3]),
                                                 pack_bf16x2(v[4], v[5]), pack_bf16x2(v[6], v[7])};
      else
        *reinterpret_cast<floatx4*>(out) = floatx4{v[0], v[1], v[2], v[3]};
    }
  });
}

// kEpiGluGrad of the stream kernel, from the same block-wide strip of ROWS x
// (COLS gate, COLS up) fp32 pre-activations. A thread takes one output column
// and eight rows of it: one 16-byte chunk of each transposed row, and single
// values of the rows (consecutive lanes write consecutive columns). The
// strips are small (outputs with few tiles), so the narrow stores do not
// count. `sums` is LDS for the column sums of the row groups.
template <int ROWS, int COLS>
__device__ __forceinline__ void glu_grad_strip(uint32_t src, int pitch, uint32_t sums, int row0, int col0,
                                               int strip_row, int tid, int nthr, const TrainArgs& p) {
  constexpr int RG = ROWS / 8;
  const int F = p.glu_half;
  for_gate(p.gate, [&](auto gate) {
    for (int k = tid; k < RG * COLS; k += nthr) {
      const int rg = k / COLS, cc = k - (k / COLS) * COLS;
      const int c = col0 + cc, r0 = row0 + 8 * rg;
      float bg = 0.0f, bu = 0.0f, sg = 0.0f, su = 0.0f;
      uint32_t wg[4], wu[4];
      if (c < F && p.bias) {
        bg = p.bias[c];
        bu = p.bias[F + c];
      }
      float dh[8];
#pragma unroll
      for (int r = 0; r < 8; ++r)
        dh[r] = (c < F && r0 + r < p.M)
                    ? __uint_as_float((uint32_t)p.dC[(int64_t)(r0 + r) * p.lddc + c] << 16)
                    : 0.0f;
#pragma unroll
      for (int r = 0; r < 8; r += 2) {
        float dg[2], du[2];
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          const uint32_t a = src + (uint32_t)((8 * rg + r + h) * pitch + cc * 4);
          const float g = __uint_as_float(lds_load_u32(a)) + bg;
          const float u = __uint_as_float(lds_load_u32(a + (uint32_t)(COLS * 4))) + bu;
          float act, slope;
          gate_both<decltype(gate)::value>(g, act, slope);
          const bool live = c < F && r0 + r + h < p.M;
          dg[h] = live ? dh[r + h] * u * slope : 0.0f;
          du[h] = live ? dh[r + h] * act : 0.0f;
          sg += dg[h];
          su += du[h];
        }
        wg[r / 2] = pack_bf16x2(dg[0], dg[1]);
        wu[r / 2] = pack_bf16x2(du[0], du[1]);
      }
      if (c < F && r0 < p.M) {
        if (p.Zt) {
          *reinterpret_cast<u32x4s*>(p.Zt + (int64_t)c * p.ldzt + r0) = u32x4s{wg[0], wg[1], wg[2], wg[3]};
          *reinterpret_cast<u32x4s*>(p.Zt + (int64_t)(F + c) * p.ldzt + r0) = u32x4s{wu[0], wu[1], wu[2], wu[3]};
        }
        if (p.Z) {
#pragma unroll
          for (int r = 0; r < 8; ++r) {
            if (r0 + r < p.M) {
              uint16_t* z = p.Z + (int64_t)(r0 + r) * p.ldz + c;
              z[0] = (uint16_t)(wg[r / 2] >> (16 * (r & 1)));
              z[F] = (uint16_t)(wu[r / 2] >> (16 * (r & 1)));
            }
          }
        }
      }
      if (p.dbias_part) {
        lds_store_u32x2(sums + (uint32_t)(k * 8), __float_as_uint(sg), __float_as_uint(su));
      }
    }
  });
  if (!p.dbias_part) return;
  wait_lgkmcnt0();
  block_barrier();
  for (int cc = tid; cc < COLS; cc += nthr) {
    const int c = col0 + cc;
    float s[2] = {0.0f, 0.0f};
#pragma unroll
    for (int rg = 0; rg < RG; ++rg)
#pragma unroll
      for (int h = 0; h < 2; ++h) s[h] += __uint_as_float(lds_load_u32(sums + (uint32_t)((rg * COLS + cc) * 8 + h * 4)));
    if (c < F) {
      float* d = p.dbias_part + (int64_t)strip_row * (2 * F) + c;
      d[0] = s[0];
      d[F] = s[1];
    }
  }
}

}  // namespace tg
