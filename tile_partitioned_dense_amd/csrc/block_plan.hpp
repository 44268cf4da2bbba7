// block_plan.hpp -- launch plan of the E4M3 products with block scales
// (tile_gemm_run_fp8, tile_gemm_run_fp8_experts). Host and device.
#pragma once

#include "plan.hpp"

namespace tg {

constexpr int kScaleBlock = 128;      // values of K that share a scale (and rows of B)
constexpr int kBlockMaxGroups = 1024;  // experts of one call

// Compiled configurations of block_kernel.hpp: tiles of bm x bn, wm x wn waves
// on it times ks that share every stage's K, stages of sb bytes of K per row.
struct BlockConfig {
  int bm, bn, wm, wn, ks, sb, stages;
  int occ;    // workgroups that fit on one compute unit at once
  float eff;  // rate relative to configuration 0; 0: a stream configuration
};
constexpr int kNumBlockConfigs = 5;
constexpr BlockConfig kBlockConfigs[kNumBlockConfigs] = {
    {256, 256, 2, 4, 1, 128, 2, 1, 1.00f},  // 0: 8 waves of 128x64
    {128, 128, 2, 2, 1, 128, 2, 2, 0.70f},  // 1: 4 waves of 64x64
    {16, 64, 1, 2, 4, 512, 3, 1, 0.0f},     // 2: up to 16 rows
    {32, 64, 1, 2, 4, 512, 3, 1, 0.0f},     // 3: up to 32 rows
    {64, 128, 1, 4, 2, 256, 3, 1, 0.0f},    // 4: up to 64 rows
};

inline int block_lds_bytes(const BlockConfig& c) {
  return c.stages * ((c.bm + c.bn) * c.sb + c.bm * (c.sb / kScaleBlock) * 4 + 256);
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
  p.grid = persistent_grid(p.tiles, cu_count * c.occ);
  return p;
}

// fp32: outputs of that type, whose products run on bf16 instructions
// (block_kernel.hpp): their operands take twice the registers, so they have the
// 64 x 64 wave tiles.
inline int pick_block_config(int64_t M, int64_t N, bool fp32, int cu_count) {
  if (M <= 16) return 2;
  if (M <= 32) return 3;
  if (M <= 64) return 4;
  if (fp32) return 1;
  const int64_t big = ceil_div(M, 256) * ceil_div(N, 256);
  const int64_t small = ceil_div(M, 128) * ceil_div(N, 128);
  const double t0 = (double)ceil_div(big, cu_count) * 4.0 / kBlockConfigs[0].eff;
  const double t1 = (double)ceil_div(small, 2 * cu_count) * 2.0 / kBlockConfigs[1].eff;
  return t1 < t0 ? 1 : 0;
}

inline Plan make_plan_block(int64_t M, int64_t N, bool fp32, int cu_count) {
  if (M <= 0 || N <= 0) return plan_for(0, 0, M, N, cu_count);
  return plan_block_for(pick_block_config(M, N, fp32, cu_count), M, N, cu_count);
}

// Rows sorted by expert: a tile is bm rows of one expert. Which rows are whose
// is known on the device only, so the configuration goes by the rows an expert
// has on average, and the grid by the most tiles there can be.
inline Plan make_plan_experts(int64_t M, int64_t N, int64_t groups, bool fp32, int cu_count) {
  if (M <= 0 || N <= 0 || groups <= 0) return plan_for(0, 0, M, N, cu_count);
  const int64_t avg = ceil_div(M, groups);
  const int config = avg <= 8 ? 2 : avg <= 24 ? 3 : avg <= 64 ? 4 : avg <= 384 || fp32 ? 1 : 0;
  Plan p = plan_block_for(config, M, N, cu_count);
  const int64_t most = ceil_div(M, p.bm) + (groups < M ? groups : M);
  p.tiles = most * p.map.tiles_n;
  const int64_t all = (int64_t)cu_count * kBlockConfigs[config].occ;
  p.grid = p.tiles < all ? p.tiles : all;
  return p;
}

}  // namespace tg
