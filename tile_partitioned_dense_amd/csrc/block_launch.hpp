// block_launch.hpp -- launchers of the E4M3 products with block scales
// (kernels_block.hip), of the quantization (kernels_quant.hip) and of the
// routing to experts (kernels_route.hip).
#pragma once

#include "block_tile_kernel.hpp"
#include "launch.hpp"

namespace tg {

template <int CFG>
hipError_t launch_block(const BlockArgs& a, bool experts, bool out_bf16, int64_t grid, hipStream_t stream);

struct QuantArgs {
  const uint16_t* X;
  uint8_t* Q;
  float* scale;
  const int32_t* rows;  // row of X of each row of Q, or NULL: its own
  int32_t M, K;
  int32_t x_rows;       // rows of X
  int64_t ldx, ldq, lds;
};
// gate: kGate*, or -1 for X's values themselves
hipError_t launch_quant_rows(const QuantArgs& a, int gate, hipStream_t stream);
hipError_t launch_quant_blocks(const QuantArgs& a, hipStream_t stream);

struct RouteArgs {
  const void* logits;
  int64_t ld;
  const float* bias;
  int32_t* ids;
  float* weights;
  int32_t T, E, k;
  int32_t groups, top_groups, group_top;
  int32_t sigmoid, renorm;
  int32_t wide;        // rows of whole 16 bytes, they and the bias 16-byte aligned
  float scale;
  // gradient
  const float* dweights;
  void* dlogits;
  int64_t ldd;
};
hipError_t launch_route(const RouteArgs& a, bool bf16, hipStream_t stream);
hipError_t launch_route_backward(const RouteArgs& a, bool bf16, hipStream_t stream);

struct PlaceArgs {
  const int32_t* ids;
  int32_t n, k;        // entries, entries of one token
  int32_t first, E;    // experts first .. first + E - 1
  int32_t* offsets;
  int32_t* rows;       // may be NULL
  int32_t* places;     // may be NULL
  int32_t* hist;       // chunks x E
  int32_t chunks, rounds;
};
hipError_t launch_place(const PlaceArgs& a, hipStream_t stream);

struct CombineArgs {
  const uint16_t* Z;
  const int32_t* places;
  const float* weights;  // NULL: ones
  void* Y;
  int32_t T, N, k, z_rows;
  int64_t ldz, ldy;
};
hipError_t launch_combine(const CombineArgs& a, bool bf16, hipStream_t stream);

}  // namespace tg
