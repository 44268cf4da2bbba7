// train_launch.hpp -- launchers of the training kernels (kernels_train.hip)
// and of the small kernels around them (kernels_train_rows.hip).
#pragma once

#include "launch.hpp"
#include "outer_kernel.hpp"
#include "train_plan.hpp"

namespace tg {

template <int ID>
hipError_t launch_train(const TrainArgs& a, int64_t grid, hipStream_t stream);

struct FinishArgs {
  const float2* part;
  const float* part_sum;  // NULL without label smoothing
  const float* hit;
  const void* target;
  int32_t target64;
  int64_t ignore;
  int32_t M, segs;
  int64_t N;
  float smoothing, z_loss;
  float* loss;  // either may be NULL
  float* lse;
};
hipError_t launch_xent_finish(const FinishArgs& a, hipStream_t stream);

struct RowsArgs {
  const void* target;
  int32_t target64;
  int64_t ignore;
  int32_t M;
  int64_t N;
  const float* lse;
  const float* dloss;
  float z_loss;
  XentRow* rows;
  float* scale;
};
hipError_t launch_xent_rows(const RowsArgs& a, hipStream_t stream);

// out[i][j] = scale * sum over parts of part[s][i][j] (scale: NULL for 1).
struct AddArgs {
  const float* part;
  int64_t part_stride;  // elements
  int32_t parts;
  int32_t M, N;
  int64_t ldp;
  const float* scale;
  uint16_t* out;
  int64_t ldo;
};
hipError_t launch_add_parts(const AddArgs& a, hipStream_t stream);

// The weight gradient over at most kOuterMaxT tokens (outer_kernel.hpp).
hipError_t launch_outer(OuterArgs a, int cu_count, hipStream_t stream);

// A gradient's product on the small tile (plan_product's kSmallTile; bf16: its
// result rather than the partial ones) and that weight gradient in one launch.
hipError_t launch_pair(const TrainArgs& product, int64_t grid, bool bf16, const OuterArgs& outer, int cu_count,
                       hipStream_t stream);

// out[c] = sum over rows of part[r][c], fp32.
hipError_t launch_add_rows(const float* part, int64_t rows, int64_t cols, float* out, hipStream_t stream);

// rows x bytes of zeros, `pitch` bytes apart.
hipError_t launch_zero(void* p, int64_t rows, int64_t bytes, int64_t pitch, hipStream_t stream);

}  // namespace tg
