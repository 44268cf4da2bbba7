// block_run.hpp -- the launches and C entry points of the E4M3 products with
// block scales, of the quantization, of the routing to experts and of the
// experts' sums. Included by the library's one host translation unit
// (tile_gemm.hip) after train_run.hpp.
#pragma once

#include "block_abi.hpp"
#include "block_launch.hpp"

namespace {

template <int CFG>
hipError_t dispatch_block(int cfg, const tg::BlockArgs& a, bool experts, bool bf16, int64_t grid, hipStream_t st) {
  if constexpr (CFG < tg::kNumBlockConfigs) {
    if (cfg == CFG) return tg::launch_block<CFG>(a, experts, bf16, grid, st);
    return dispatch_block<CFG + 1>(cfg, a, experts, bf16, grid, st);
  } else {
    return hipErrorInvalidValue;
  }
}

tile_gemm_status_t run_fp8(tile_gemm_t h, const void* A, const void* B, void* C, int64_t M, int64_t N, int64_t K,
                           int64_t experts, const int32_t* offsets, const tile_gemm_fp8_strides_t* s,
                           const float* sa, const float* sb, int dtype, const float* bias, int act, void* stream) {
  if (!h) return fail(TILE_GEMM_ERR_NULL_ARG, "handle: NULL");
  TG_TRY(check_fp8(A, B, C, M, N, K, experts, offsets, s, sa, sb, dtype, bias, act));
  if (M == 0 || N == 0) return TILE_GEMM_OK;
  TG_TRY(check_device(h));
  const tg::Plan p = experts < 0 ? tg::make_plan_block(M, N, K, dtype == TILE_GEMM_BF16_TO_F32, h->cu_count)
                                 : tg::make_plan_experts(M, N, K, experts, dtype == TILE_GEMM_BF16_TO_F32, h->cu_count);
  tg::BlockArgs a{};
  a.A = static_cast<const uint8_t*>(A);
  a.B = static_cast<const uint8_t*>(B);
  a.sA = sa;
  a.sB = sb;
  a.C = C;
  a.M = (int32_t)M;
  a.N = (int32_t)N;
  a.K = (int32_t)K;
  // (the stride of a single row or block is any: the kernels form offsets of a tile's other ones from it)
  a.lda = M > 1 ? s->a_stride : K;
  a.ldb = N > 1 ? s->b_stride : K;
  a.ldc = M > 1 ? s->c_stride : N;
  a.lsa = K > tg::kScaleBlock ? s->a_scale_stride : M;
  a.lsb = N > tg::kScaleBlock ? s->b_scale_stride : 0;
  a.map = p.map;
  a.bias = bias;
  a.act = act;
  a.offsets = offsets;
  a.groups = (int32_t)experts;
  a.eb = s->b_expert_stride;
  a.esb = s->b_scale_expert_stride;
  // (experts: whose rows mostly fit one tile.) Past the caches, against the plain
  // loads: weights of 17 to 235 MB that come in turn take 9 to 14% less time for up
  // to 16 rows (16 x 8192 x 4096 10.4 and 12.1 us, 16 x 28672 x 8192 40.5 and 46.0; 64
  // experts of 4096 x 2048 with 3 rows each 78 and 90), the same for 96; one weight
  // again and again the same up to 67 MB, at 134 MB 3% and at 235 MB, which the
  // last-level cache would just hold, 25% more.
  a.once = experts < 0 ? p.map.tiles_m == 1 : 2 * M <= experts * p.bm;
  log_plan(h, experts < 0 ? "run_fp8" : "run_fp8_experts", M, N, K, 1, dtype, act, p);
  return hip_status(dispatch_block<0>(p.config, a, experts >= 0, dtype == TILE_GEMM_BF16_TO_BF16, p.grid,
                                      static_cast<hipStream_t>(stream)));
}

tg::RouteArgs route_args(const void* logits, const float* bias, int64_t T, int64_t E, int64_t k, int64_t ld,
                         const tile_gemm_route_t* o) {
  tg::RouteArgs a{};
  a.logits = logits;
  a.bias = bias;
  a.ld = ld;
  a.T = (int32_t)T;
  a.E = (int32_t)E;
  a.k = (int32_t)k;
  a.groups = o->groups;
  a.top_groups = o->top_groups;
  a.group_top = o->group_top;
  a.sigmoid = o->score == TILE_GEMM_SCORE_SIGMOID;
  a.renorm = o->renormalize != 0;
  a.wide = (uintptr_t)logits % 16 == 0 && (uintptr_t)bias % 16 == 0 && ld * (o->logits_type == TILE_GEMM_LOGITS_BF16 ? 2 : 4) % 16 == 0;
  a.scale = o->scale;
  return a;
}

}  // namespace

extern "C" {

tile_gemm_status_t tile_gemm_run_fp8(tile_gemm_t h, const void* A, const void* B, void* C, int64_t M, int64_t N,
                                     int64_t K, const tile_gemm_fp8_strides_t* strides, const float* a_scale,
                                     const float* b_scale, tile_gemm_dtype_t dtype, const float* bias,
                                     tile_gemm_act_t act, void* stream) {
  return run_fp8(h, A, B, C, M, N, K, -1, nullptr, strides, a_scale, b_scale, (int)dtype, bias, (int)act, stream);
}

tile_gemm_status_t tile_gemm_run_fp8_experts(tile_gemm_t h, const void* A, const void* B, void* C, int64_t M,
                                             int64_t N, int64_t K, int64_t E, const int32_t* offsets,
                                             const tile_gemm_fp8_strides_t* strides, const float* a_scale,
                                             const float* b_scale, tile_gemm_dtype_t dtype, void* stream) {
  return run_fp8(h, A, B, C, M, N, K, E < 0 ? 0 : E, offsets, strides, a_scale, b_scale, (int)dtype, nullptr,
                 TILE_GEMM_ACT_NONE, stream);
}

tile_gemm_status_t tile_gemm_run_quantize(tile_gemm_t h, const void* X, void* Q, float* scale, int64_t M, int64_t K,
                                          int64_t x_stride, int64_t q_stride, int64_t scale_stride,
                                          tile_gemm_quant_t form, tile_gemm_gate_t gate, const int32_t* rows,
                                          int64_t x_rows, void* stream) {
  if (!h) return fail(TILE_GEMM_ERR_NULL_ARG, "handle: NULL");
  TG_TRY(check_quantize(X, Q, scale, M, K, x_stride, q_stride, scale_stride, (int)form, (int)gate, rows, x_rows));
  if (M == 0 || K == 0) return TILE_GEMM_OK;
  TG_TRY(check_device(h));
  tg::QuantArgs a{};
  a.X = static_cast<const uint16_t*>(X);
  a.Q = static_cast<uint8_t*>(Q);
  a.scale = scale;
  a.rows = rows;
  a.M = (int32_t)M;
  a.K = (int32_t)K;
  a.x_rows = (int32_t)x_rows;
  a.ldx = x_stride;
  a.ldq = q_stride;
  a.lds = scale_stride;
  const hipStream_t st = static_cast<hipStream_t>(stream);
  if (form == TILE_GEMM_QUANT_BLOCKS) return hip_status(tg::launch_quant_blocks(a, st));
  return hip_status(tg::launch_quant_rows(a, form == TILE_GEMM_QUANT_GATED_ROWS ? (int)gate : -1, st));
}

tile_gemm_status_t tile_gemm_run_route(tile_gemm_t h, const void* logits, const float* bias, int32_t* ids,
                                       float* weights, int64_t T, int64_t E, int64_t k, int64_t logit_stride,
                                       const tile_gemm_route_t* options, void* stream) {
  if (!h) return fail(TILE_GEMM_ERR_NULL_ARG, "handle: NULL");
  TG_TRY(check_route(logits, bias, ids, weights, T, E, k, logit_stride, options));
  if (T == 0) return TILE_GEMM_OK;
  TG_TRY(check_device(h));
  tg::RouteArgs a = route_args(logits, bias, T, E, k, logit_stride, options);
  a.ids = ids;
  a.weights = weights;
  return hip_status(tg::launch_route(a, options->logits_type == TILE_GEMM_LOGITS_BF16,
                                     static_cast<hipStream_t>(stream)));
}

tile_gemm_status_t tile_gemm_run_route_backward(tile_gemm_t h, const void* logits, const int32_t* ids,
                                                const float* dweights, void* dlogits, int64_t T, int64_t E,
                                                int64_t k, int64_t logit_stride, int64_t dlogit_stride,
                                                const tile_gemm_route_t* options, void* stream) {
  if (!h) return fail(TILE_GEMM_ERR_NULL_ARG, "handle: NULL");
  TG_TRY(check_route_backward(logits, ids, dweights, dlogits, T, E, k, logit_stride, dlogit_stride, options));
  if (T == 0) return TILE_GEMM_OK;
  TG_TRY(check_device(h));
  tg::RouteArgs a = route_args(logits, nullptr, T, E, k, logit_stride, options);
  a.ids = const_cast<int32_t*>(ids);
  a.dweights = dweights;
  a.dlogits = dlogits;
  a.ldd = dlogit_stride;
  a.wide = a.wide && (uintptr_t)dlogits % 16 == 0 &&
           dlogit_stride * (options->logits_type == TILE_GEMM_LOGITS_BF16 ? 2 : 4) % 16 == 0;
  return hip_status(tg::launch_route_backward(a, options->logits_type == TILE_GEMM_LOGITS_BF16,
                                              static_cast<hipStream_t>(stream)));
}

tile_gemm_status_t tile_gemm_run_place(tile_gemm_t h, const int32_t* ids, int64_t T, int64_t k, int64_t first,
                                       int64_t E, int32_t* offsets, int32_t* rows, int32_t* places,
                                       void* workspace, int64_t workspace_bytes, void* stream) {
  if (!h) return fail(TILE_GEMM_ERR_NULL_ARG, "handle: NULL");
  PlacePlan plan;
  TG_TRY(check_place(ids, T, k, first, E, offsets, rows, places, workspace, workspace_bytes, &plan));
  TG_TRY(check_device(h));
  tg::PlaceArgs a{};
  a.ids = ids;
  a.n = (int32_t)(T * k);
  a.k = (int32_t)k;
  a.first = (int32_t)first;
  a.E = (int32_t)E;
  a.offsets = offsets;
  a.rows = rows;
  a.places = places;
  a.hist = static_cast<int32_t*>(workspace);
  a.chunks = (int32_t)plan.chunks;
  a.rounds = (int32_t)plan.rounds;
  return hip_status(tg::launch_place(a, static_cast<hipStream_t>(stream)));
}

tile_gemm_status_t tile_gemm_run_combine(tile_gemm_t h, const void* Z, const int32_t* places, const float* weights,
                                         void* Y, int64_t T, int64_t N, int64_t k, int64_t z_rows, int64_t z_stride,
                                         int64_t y_stride, tile_gemm_dtype_t dtype, void* stream) {
  if (!h) return fail(TILE_GEMM_ERR_NULL_ARG, "handle: NULL");
  TG_TRY(check_combine(Z, places, weights, Y, T, N, k, z_rows, z_stride, y_stride, (int)dtype));
  if (T == 0 || N == 0) return TILE_GEMM_OK;
  TG_TRY(check_device(h));
  tg::CombineArgs a{};
  a.Z = static_cast<const uint16_t*>(Z);
  a.places = places;
  a.weights = weights;
  a.Y = Y;
  a.T = (int32_t)T;
  a.N = (int32_t)N;
  a.k = (int32_t)k;
  a.z_rows = (int32_t)z_rows;
  a.ldz = z_stride;
  a.ldy = y_stride;
  return hip_status(tg::launch_combine(a, dtype == TILE_GEMM_BF16_TO_BF16, static_cast<hipStream_t>(stream)));
}

}  // extern "C"
