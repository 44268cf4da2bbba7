// outer_kernel.hpp -- a weight gradient over few tokens, dW = scale * G^T x.
//
// With T <= 128 tokens the contraction is one to four MFMA steps and the
// product is its output: V x K bf16 values written once, bound by HBM writes.
// The tile kernel would spend a tile's load latency, barriers and staged store
// on one or two slabs. Here a wave keeps the x values of its 64 columns (all
// T tokens) in registers and walks down G^T, 16 rows at a time: one 16-byte
// load per lane and 32 tokens, four MFMAs for them, two 16-byte stores per
// lane. Many waves per SIMD hide the latencies (seven with one MFMA step, two
// with four: eight steps, up to 256 tokens, leave one and measured 1.1 to 1.9
// times slower than the tile kernel).
//
// MFMA operands as in tile16_kernel.hpp: the x fragment is the row operand, so
// lane l receives row l % 16 of a block, four consecutive columns 4 (l / 16) ..
// of it. The wave's 16 x 64 results pass through a strip of LDS private to it
// (no barrier), so that every store instruction writes whole 128-byte lines.
#pragma once

#include "train_epilogue.hpp"

namespace tg {

constexpr int kOuterMaxT = 128;
constexpr int kOuterCols = 256;  // columns of a workgroup: four waves of 64

struct OuterArgs {
  const uint16_t* gt;  // V rows of T values (whole chunks of 8; zeros past T in the last)
  int64_t ldg;
  const uint16_t* x;  // T rows of K values
  int64_t ldx;
  uint16_t* out;  // V rows of K values
  int64_t ldo;
  const float* scale;  // one fp32 value, or NULL
  int32_t T, V, K;
  int32_t col_groups;      // workgroups across the columns
  int32_t rows_per_group;  // rows of a workgroup, a multiple of 16
};

// A gradient's product in the first `n_first` workgroups of a launch, and the
// weight gradient of the same G in the others. Neither needs the other, and at
// few tokens each is mostly latency: side by side they take the longer's time.
struct PairArgs : TrainArgs {
  OuterArgs outer;
  int32_t n_first;
};

// Workgroup `group` of the product, with 4 * 16 * kOuterPitch bytes of LDS.
constexpr int kOuterPitch = 64 * 2 + 16;
template <int STEPS, bool WAIT>
__device__ __forceinline__ void outer_group(const OuterArgs& p, int group, const void* smem) {
  constexpr int kPitch = kOuterPitch;
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  const uint32_t strip = (uint32_t)(uintptr_t)smem + (uint32_t)(wave * 16 * kPitch);
  const int l16 = lane & 15, lg = lane >> 4;
  const int cg = group % p.col_groups, rg = group / p.col_groups;
  const int col0 = cg * kOuterCols + wave * 64;
  if (col0 >= p.K) return;
  const float scale = p.scale ? *p.scale : 1.0f;

  bf16x8 xf[STEPS][4];
#pragma unroll
  for (int s = 0; s < STEPS; ++s)
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const int col = col0 + 16 * j + l16;
      uint32_t w[4] = {0u, 0u, 0u, 0u};
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        const int t = 32 * s + 8 * lg + e;
        const uint32_t v = (t < p.T && col < p.K) ? (uint32_t)p.x[(int64_t)t * p.ldx + col] : 0u;
        w[e >> 1] |= v << (16 * (e & 1));
      }
      xf[s][j] = as_bf16x8(make_uint4(w[0], w[1], w[2], w[3]));
    }

  const int r_begin = rg * p.rows_per_group;
  const int r_end = tg_min(r_begin + p.rows_per_group, p.V);
  auto load = [&](int r0, uint4 (&g)[STEPS]) {
    const int row = r0 + l16;
#pragma unroll
    for (int s = 0; s < STEPS; ++s) {
      const int t = 32 * s + 8 * lg;
      g[s] = make_uint4(0, 0, 0, 0);
      if (row < r_end && t < p.T) g[s] = *reinterpret_cast<const uint4*>(p.gt + (int64_t)row * p.ldg + t);
    }
  };
  // U blocks of 16 rows at a time, the next U's values on their way meanwhile
  constexpr int U = STEPS == 4 ? 2 : 4;
  uint4 g[U][STEPS];
#pragma unroll
  for (int b = 0; b < U; ++b) load(r_begin + 16 * b, g[b]);
  for (int r1 = r_begin; r1 < r_end; r1 += 16 * U) {
    uint4 gn[U][STEPS];
#pragma unroll
    for (int b = 0; b < U; ++b) load(r1 + 16 * (U + b), gn[b]);
#pragma unroll
    for (int b = 0; b < U; ++b) {
      const int r0 = r1 + 16 * b;
      floatx4 acc[4];
#pragma unroll
      for (int j = 0; j < 4; ++j) acc[j] = floatx4{};
#pragma unroll
      for (int s = 0; s < STEPS; ++s)
#pragma unroll
        for (int j = 0; j < 4; ++j) acc[j] = mfma16(xf[s][j], as_bf16x8(g[b][s]), acc[j]);
      // In the pair, whose kernel bears the tile kernels' name, the results are
      // left alone for 19 wait states (the hazard check's rule for MFMAs written
      // out). Alone it costs 5% where the writes are the bound.
      if constexpr (WAIT)
        asm volatile("s_nop 7\n\ts_nop 7\n\ts_nop 2" : "+v"(acc[0]), "+v"(acc[1]), "+v"(acc[2]), "+v"(acc[3]));
#pragma unroll
      for (int j = 0; j < 4; ++j)
        lds_store_u32x2(strip + (uint32_t)(l16 * kPitch + (16 * j + 4 * lg) * 2),
                        pack_bf16x2(acc[j][0] * scale, acc[j][1] * scale),
                        pack_bf16x2(acc[j][2] * scale, acc[j][3] * scale));
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        const int r = 8 * h + (lane >> 3), row = r0 + r, col = col0 + 8 * (lane & 7);
        const u32x4s v = *(const __attribute__((address_space(3))) u32x4s*)(uintptr_t)(
            strip + (uint32_t)(r * kPitch + (lane & 7) * 16));
        if (row >= r_end) continue;
        uint16_t* o = p.out + (int64_t)row * p.ldo + col;
        if (col + 8 <= p.K) {
          *reinterpret_cast<u32x4s*>(o) = v;
        } else {
#pragma unroll
          for (int e = 0; e < 8; ++e)
            if (col + e < p.K) o[e] = (uint16_t)(v[e >> 1] >> (16 * (e & 1)));
        }
      }
    }
#pragma unroll
    for (int b = 0; b < U; ++b)
#pragma unroll
      for (int s = 0; s < STEPS; ++s) g[b][s] = gn[b][s];
  }
}

template <int STEPS>
__global__ __launch_bounds__(256) void outer_kernel(OuterArgs p) {
  __shared__ __attribute__((aligned(16))) uint8_t smem[4 * 16 * kOuterPitch];
  outer_group<STEPS, false>(p, blockIdx.x, smem);
}

}  // namespace tg
