// block_plan.hpp -- launch plan of the E4M3 products with block scales
// (tile_gemm_run_fp8, tile_gemm_run_fp8_experts). Host and device.
#pragma once

#include "plan.hpp"

namespace tg {

constexpr int kScaleBlock = 128;      // values of K that share a scale (and rows of B)
constexpr int kBlockMaxGroups = 1024;  // experts of one call
constexpr int kExpertLds = 2 * (kBlockMaxGroups + 4) * 4;  // bytes of their tables in LDS

// Compiled configurations: tiles of bm x bn, wm x wn waves on it times ks that
// share every stage's K, stages of sb bytes of K per row. `tile`: those of
// block_tile_kernel.hpp, the others of block_kernel.hpp.
struct BlockConfig {
  int bm, bn, wm, wn, ks, sb, stages;
  int occ;     // workgroups that fit on one compute unit at once
  bool tile;
  // Microseconds of a launch, for bf16 and for fp32 outputs: c0 + rounds (a +
  // stages b), with b going to b2 as a round's tiles come to fill the chip (two
  // tiles a compute unit where occ is 2). Fitted to 411 shapes of 1 to 6100 rows,
  // 48 to 131072 columns and K of 128 to 8192: the configuration it picks takes
  // 0.6% longer than the fastest on average (4% or less on 95 of 100).
  float cost[2][4];
};
constexpr int kNumBlockConfigs = 15;
constexpr BlockConfig kBlockConfigs[kNumBlockConfigs] = {
    {256, 256, 2, 4, 1, 128, 2, 1, true, {{1.53f, 6.30f, 1.09f, 1.75f}, {}}},  // 0: 8 waves of 128x64 (bf16 outputs)
    {192, 256, 2, 4, 1, 128, 2, 1, true, {{0.54f, 5.31f, 0.98f, 1.43f}, {0.00f, 7.61f, 1.74f, 2.35f}}},  // 1: 8 waves of 96x64
    {256, 128, 4, 2, 1, 128, 2, 1, true, {{2.72f, 2.39f, 0.76f, 1.10f}, {0.73f, 5.36f, 1.09f, 1.63f}}},  // 2: 8 waves of 64x64
    {128, 128, 2, 2, 1, 128, 2, 2, true, {{0.76f, 3.93f, 0.68f, 1.10f}, {0.00f, 5.53f, 0.98f, 1.73f}}},  // 3: 4 waves of 64x64
    {16, 128, 1, 4, 2, 256, 3, 1, false, {{2.42f, 1.43f, 0.66f, 0.71f}, {2.42f, 1.57f, 0.81f, 0.86f}}},  // 4
    {32, 128, 1, 4, 2, 256, 3, 1, false, {{2.49f, 1.84f, 0.74f, 0.81f}, {2.47f, 2.02f, 0.97f, 1.05f}}},  // 5
    {64, 128, 2, 2, 2, 256, 3, 1, false, {{2.26f, 2.55f, 0.88f, 1.00f}, {1.98f, 3.27f, 1.32f, 1.46f}}},  // 6
    {96, 128, 2, 2, 2, 256, 2, 1, false, {{2.20f, 3.05f, 1.10f, 1.25f}, {1.86f, 4.01f, 1.64f, 1.78f}}},  // 7
    {96, 64, 2, 2, 2, 256, 3, 1, false, {{2.39f, 2.47f, 0.77f, 0.81f}, {2.39f, 2.78f, 1.16f, 1.21f}}},  // 8
    {16, 64, 1, 2, 4, 512, 3, 1, false, {{2.43f, 1.51f, 0.67f, 0.70f}, {2.45f, 1.55f, 0.86f, 0.89f}}},  // 9
    {32, 64, 1, 2, 4, 512, 3, 1, false, {{2.47f, 1.95f, 0.77f, 0.86f}, {2.40f, 2.35f, 1.00f, 1.11f}}},  // 10
    {48, 64, 1, 2, 4, 512, 2, 1, false, {{2.40f, 2.26f, 0.97f, 1.10f}, {2.33f, 2.76f, 1.21f, 1.34f}}},  // 11
    {64, 64, 2, 2, 4, 512, 2, 1, false, {{2.98f, 2.47f, 1.11f, 1.27f}, {2.92f, 2.98f, 1.40f, 1.55f}}},  // 12
    {16, 32, 1, 1, 8, 1024, 3, 1, false, {{2.36f, 1.66f, 0.79f, 0.88f}, {2.24f, 1.69f, 0.92f, 1.02f}}},  // 13
    {32, 32, 1, 1, 8, 1024, 2, 1, false, {{2.57f, 1.82f, 1.00f, 1.18f}, {2.49f, 2.07f, 1.20f, 1.36f}}},  // 14
};

// The ring of stages, and the store's own part where it fits beside it and the
// experts' tables (block_kernel.hpp).
inline int block_lds_bytes(const BlockConfig& c) {
  const int rows = (c.bm + 63) / 64 * 64;  // of scales
  const int ring = c.stages * ((c.bm + c.bn) * c.sb + rows * (c.sb / kScaleBlock) * 4 + 256);
  const int store = (c.ks - 1) * c.bm * c.bn * 4 + c.wm * c.wn * 16 * (c.bn / c.wn * 4 + 16);
  return ring + (!c.tile && ring + kExpertLds + store <= 160 * 1024 ? store : 0);
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
