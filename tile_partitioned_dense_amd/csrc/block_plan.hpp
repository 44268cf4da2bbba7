// block_plan.hpp -- launch plan of the E4M3 products with block scales
// (tile_gemm_run_fp8, tile_gemm_run_fp8_experts). Host and device.
#pragma once

#include "plan.hpp"

namespace tg {

constexpr int kScaleBlock = 128;      // values of K that share a scale (and rows of B)
constexpr int kBlockMaxGroups = 1024;  // experts of one call

// Compiled configurations: tiles of bm x bn, wm x wn waves on it times ks that
// share every stage's K, stages of sb bytes of K per row. `tile`: those of
// block_tile_kernel.hpp, the others of block_kernel.hpp.
struct BlockConfig {
  int bm, bn, wm, wn, ks, sb, stages;
  int occ;     // workgroups that fit on one compute unit at once
  bool tile;
  // Microseconds of a launch, for bf16 and for fp32 outputs: c0 + rounds (a +
  // stages b), with b going to b2 as a round's tiles come to fill the chip (two
  // tiles a compute unit where occ is 2). Fitted to 267 shapes of 1 to 6100 rows,
  // 48 to 28672 columns and K of 128 to 8192: the configuration it picks takes
  // 1.9% longer than the fastest on average (8% or less on 95 of 100).
  float cost[2][4];
};
constexpr int kNumBlockConfigs = 12;
constexpr BlockConfig kBlockConfigs[kNumBlockConfigs] = {
    {256, 256, 2, 4, 1, 128, 2, 1, true, {{0.83f, 7.80f, 1.01f, 1.83f}, {}}},  // 0: 8 waves of 128x64 (bf16 outputs)
    {192, 256, 2, 4, 1, 128, 2, 1, true, {{0.94f, 5.56f, 0.91f, 1.45f}, {0.00f, 8.25f, 1.67f, 2.56f}}},  // 1: 8 waves of 96x64
    {256, 128, 4, 2, 1, 128, 2, 1, true, {{1.57f, 3.94f, 0.71f, 1.09f}, {0.00f, 6.79f, 1.05f, 1.75f}}},  // 2: 8 waves of 64x64
    {128, 128, 2, 2, 1, 128, 2, 2, true, {{0.89f, 3.95f, 0.63f, 1.07f}, {0.00f, 5.77f, 0.96f, 1.80f}}},  // 3: 4 waves of 64x64
    {16, 128, 1, 4, 2, 256, 3, 1, false, {{2.57f, 1.63f, 0.68f, 0.71f}, {2.62f, 1.74f, 0.81f, 0.84f}}},  // 4
    {32, 128, 1, 4, 2, 256, 3, 1, false, {{2.55f, 1.99f, 0.77f, 0.81f}, {2.48f, 2.41f, 1.01f, 1.06f}}},  // 5
    {64, 128, 1, 4, 2, 256, 3, 1, false, {{2.57f, 3.03f, 1.07f, 1.16f}, {2.41f, 3.37f, 1.46f, 1.55f}}},  // 6
    {16, 64, 1, 2, 4, 512, 3, 1, false, {{2.58f, 1.64f, 0.67f, 0.72f}, {2.57f, 1.69f, 0.82f, 0.87f}}},  // 7
    {32, 64, 1, 2, 4, 512, 3, 1, false, {{2.67f, 2.05f, 0.83f, 0.90f}, {2.56f, 2.43f, 1.06f, 1.13f}}},  // 8
    {64, 64, 2, 2, 4, 512, 2, 1, false, {{3.08f, 2.33f, 1.04f, 1.18f}, {2.97f, 2.69f, 1.42f, 1.54f}}},  // 9
    {16, 32, 1, 1, 8, 1024, 3, 1, false, {{2.60f, 1.72f, 0.80f, 0.88f}, {2.67f, 1.66f, 0.95f, 1.05f}}},  // 10
    {32, 32, 1, 1, 8, 1024, 2, 1, false, {{2.80f, 1.79f, 0.98f, 1.11f}, {2.81f, 1.98f, 1.20f, 1.32f}}},  // 11
};

inline int block_lds_bytes(const BlockConfig& c) {
  const int rows = (c.bm + 63) / 64 * 64;  // of scales
  return c.stages * ((c.bm + c.bn) * c.sb + rows * (c.sb / kScaleBlock) * 4 + 256);
}

inline Plan plan_block_for(int config, int64_t M, int64_t N, int cu_count) {
  Plan p{};
  const BlockConfig& c = kBlockConfigs[config];
  p.variant = 1;
  p.config = config;
  p.bm = c.bm;
  p.bn = c.bn;
  p.bk = c.sb;
  p.threads = c.wm * c.wn * c.ks * 64;
  p.lds_bytes = block_lds_bytes(c);
  p.k_split = c.ks;
  p.map.tiles_m = (int32_t)ceil_div(M, c.bm);
  p.map.tiles_n = (int32_t)ceil_div(N, c.bn);
  p.map.group_m = pick_group_m(p.map.tiles_m, p.map.tiles_n);
  p.map.xcds = kXcds;
  p.tiles = (int64_t)p.map.tiles_m * p.map.tiles_n;
  const int64_t all = (int64_t)cu_count * c.occ;
  p.grid = c.occ > 1 ? (p.tiles < all ? p.tiles : all) : persistent_grid(p.tiles, cu_count);
  return p;
}

// The launch's estimated microseconds for `tiles` tiles (see BlockConfig::cost).
inline double block_cost(int config, bool fp32, int64_t tiles, int64_t K, int cu_count) {
  const BlockConfig& c = kBlockConfigs[config];
  const float* f = c.cost[fp32];
  const double st = (double)ceil_div(K, c.sb), a = f[1], b = f[2], b2 = f[3];
  if (c.occ > 1) {
    const int64_t full = tiles / (2 * cu_count), rest = tiles - full * 2 * cu_count;
    double t = f[0] + (double)full * (a + b2 * st);
    if (rest > cu_count) t += a + b2 * st;
    else if (rest > 0) t += a + b * st;
    return t;
  }
  const int64_t rounds = ceil_div(tiles, cu_count);
  const double fill = (double)ceil_div(tiles, rounds) / cu_count;
  return f[0] + (double)rounds * (a + (b + (b2 - b) * (fill < 1.0 ? fill : 1.0)) * st);
}

// fp32: outputs of that type, whose products run on bf16 instructions
// (block_kernel.hpp): their operands take twice the registers, so they have no
// 256 x 256 tiles.
template <class Tiles>
int pick_block_config(bool fp32, int64_t K, int cu_count, Tiles tiles) {
  int best = -1;
  double best_cost = 0.0;
  for (int i = fp32 ? 1 : 0; i < kNumBlockConfigs; ++i) {
    const double cost = block_cost(i, fp32, tiles(kBlockConfigs[i]), K, cu_count);
    if (best < 0 || cost < best_cost) {
      best = i;
      best_cost = cost;
    }
  }
  return best;
}

inline Plan make_plan_block(int64_t M, int64_t N, int64_t K, bool fp32, int cu_count) {
  if (M <= 0 || N <= 0) return plan_for(0, 0, M, N, cu_count);
  const int config = pick_block_config(fp32, K, cu_count, [&](const BlockConfig& c) {
    return ceil_div(M, c.bm) * ceil_div(N, c.bn);
  });
  return plan_block_for(config, M, N, cu_count);
}

// Rows sorted by expert: a tile is bm rows of one expert. Which rows are whose
// is known on the device only, so the configuration goes by the tiles to be
// expected (live experts of e rows on average end half a tile short) and the
// grid by the most there can be.
inline Plan make_plan_experts(int64_t M, int64_t N, int64_t K, int64_t groups, bool fp32, int cu_count) {
  if (M <= 0 || N <= 0 || groups <= 0) return plan_for(0, 0, M, N, cu_count);
  const int64_t live = groups < M ? groups : M;
  const int config = pick_block_config(fp32, K, cu_count, [&](const BlockConfig& c) {
    const int64_t rows = M / c.bm + (live + 1) / 2;
    return (rows > live ? rows : live) * ceil_div(N, c.bn);
  });
  Plan p = plan_block_for(config, M, N, cu_count);
  p.tiles = (ceil_div(M, p.bm) + live) * p.map.tiles_n;
  const int64_t all = (int64_t)cu_count * kBlockConfigs[config].occ;
  p.grid = p.tiles < all ? p.tiles : all;
  return p;
}

}  // namespace tg
