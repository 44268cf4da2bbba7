// block_abi.hpp -- argument checks, plans and workspace sizes of the E4M3
// products with block scales, of the quantization, of the routing to experts
// and of the experts' sums (include/tile_gemm.h). Host only; included after
// train_abi.hpp by the library's one translation unit.
#pragma once

#include "block_plan.hpp"
#include "train_abi.hpp"

namespace {

constexpr int64_t kMax22 = (int64_t)1 << 22;
constexpr int64_t kPlaceRound = 1024;       // entries a workgroup places at a time
constexpr int64_t kPlaceMaxChunks = 128;    // workgroups of a call
constexpr int64_t kMaxRouteT = (int64_t)1 << 25;  // up to 64 threads each, a launch has less than 2^32
constexpr int64_t kMaxRouteK = 32, kMaxCombineK = 64, kMaxGroups = 64;

tile_gemm_status_t check_dtype(int dtype) {
  if (dtype != TILE_GEMM_BF16_TO_F32 && dtype != TILE_GEMM_BF16_TO_BF16)
    return fail(TILE_GEMM_ERR_DTYPE, "dtype: unknown value %d", dtype);
  return TILE_GEMM_OK;
}
tile_gemm_status_t check_range(const char* name, int64_t v, int64_t lo, int64_t below) {
  if (v < lo || v >= below)
    return fail(TILE_GEMM_ERR_BAD_SHAPE, "%s=%lld, must be in [%lld, %lld)", name, (long long)v, (long long)lo,
                (long long)below);
  return TILE_GEMM_OK;
}
tile_gemm_status_t check_stride(const char* name, int64_t v, int64_t least, int64_t below, int64_t rows) {
  if (rows > 1 && (v < least || v >= below))
    return fail(TILE_GEMM_ERR_BAD_STRIDE, "%s=%lld, must be in [%lld, %lld)", name, (long long)v, (long long)least,
                (long long)below);
  return TILE_GEMM_OK;
}
Arg scales(const char* name, const float* p, int64_t rows, int64_t cols, int64_t ld, bool written = false) {
  return Arg{name, p, rows, cols, ld, 4, 4, written, true};
}
Arg wide_matrix(const char* name, const void* p, int64_t rows, int64_t cols, int64_t ld, int64_t esz,
                bool written = false) {
  return matrix(name, p, rows, cols, ld, esz, written, true);
}

// experts < 0: one B for all rows
tile_gemm_status_t check_fp8(const void* A, const void* B, const void* C, int64_t M, int64_t N, int64_t K,
                             int64_t experts, const int32_t* offsets, const tile_gemm_fp8_strides_t* s,
                             const float* sa, const float* sb, int dtype, const float* bias, int act) {
  g_detail[0] = '\0';
  TG_TRY(check_dtype(dtype));
  TG_TRY(check_range("M", M, 0, kMax22));
  TG_TRY(check_range("N", N, 0, kMax22));
  TG_TRY(check_range("K", K, 0, kMax22));
  if (experts >= 0) TG_TRY(check_range("E", experts, 1, tg::kBlockMaxGroups + 1));
  if (K % 16) return fail(TILE_GEMM_ERR_BAD_SHAPE, "K=%lld: must be a multiple of 16", (long long)K);
  if (!s) return fail(TILE_GEMM_ERR_NULL_ARG, "strides: NULL");
  if (act < TILE_GEMM_ACT_NONE || act > TILE_GEMM_ACT_SILU)
    return fail(TILE_GEMM_ERR_EPILOGUE, "act: %d is not available for the E4M3 product", act);
  if (M == 0 || N == 0) return TILE_GEMM_OK;
  // the kernels number tiles (16 x 32 at the smallest, and a part of one for
  // each expert) in 32 bits
  if ((tg::ceil_div(M, 16) + (experts > 0 ? experts : 0)) * tg::ceil_div(N, 32) >= kMaxDim)
    return fail(TILE_GEMM_ERR_BAD_SHAPE, "shape: M=%lld N=%lld, too many tiles for one call", (long long)M,
                (long long)N);
  const int64_t kb = tg::ceil_div(K, tg::kScaleBlock), nb = tg::ceil_div(N, tg::kScaleBlock);
  TG_TRY(check_stride("a_stride", s->a_stride, K, kMax22, M));
  TG_TRY(check_stride("b_stride", s->b_stride, K, kMax22, N));
  TG_TRY(check_stride("c_stride", s->c_stride, N, kMax22, M));
  TG_TRY(check_stride("a_scale_stride", s->a_scale_stride, M, kMaxDim, kb));
  TG_TRY(check_stride("b_scale_stride", s->b_scale_stride, kb, kMax22, nb));
  const int64_t esz = dtype == TILE_GEMM_BF16_TO_F32 ? 4 : 2;
  Arg a[8];
  int n = 0;
  a[n++] = wide_matrix("C", C, M, N, s->c_stride, esz, true);
  if (K > 0) {
    a[n++] = wide_matrix("A", A, M, K, s->a_stride, 1);
    a[n++] = scales("a_scale", sa, kb, M, s->a_scale_stride);
    if (experts < 0) {
      a[n++] = wide_matrix("B", B, N, K, s->b_stride, 1);
      a[n++] = scales("b_scale", sb, nb, kb, s->b_scale_stride);
    } else {
      const int64_t one = span_bytes(N, N > 1 ? s->b_stride : 0, K, 1);
      const int64_t one_s = span_bytes(nb, nb > 1 ? s->b_scale_stride : 0, kb, 1);
      if (one >= kMaxDim) return fail(TILE_GEMM_ERR_BAD_SHAPE, "B: an expert's matrix spans 2 GiB or more");
      a[n++] = wide_matrix("B", B, experts, one, s->b_expert_stride, 1);
      a[n++] = scales("b_scale", sb, experts, one_s, s->b_scale_expert_stride);
      if (N > 1 && s->b_stride % 16)
        return fail(TILE_GEMM_ERR_MISALIGNED, "B: b_stride %lld is not a multiple of 16 bytes",
                    (long long)s->b_stride);
    }
  }
  if (experts >= 0) a[n++] = vec("offsets", offsets, experts + 1, 4);
  if (bias) {
    a[n] = vec("bias", bias, N, 4);
    a[n++].align = 16;
  }
  return check_arg_list(a, n);
}

tile_gemm_status_t check_quantize(const void* X, const void* Q, const float* scale, int64_t M, int64_t K, int64_t ldx,
                                  int64_t ldq, int64_t lds, int form, int gate, const int32_t* rows,
                                  int64_t x_rows) {
  g_detail[0] = '\0';
  if (form < TILE_GEMM_QUANT_ROWS || form > TILE_GEMM_QUANT_BLOCKS)
    return fail(TILE_GEMM_ERR_DTYPE, "form: unknown value %d", form);
  const bool gated = form == TILE_GEMM_QUANT_GATED_ROWS, blocks = form == TILE_GEMM_QUANT_BLOCKS;
  if (gated) TG_TRY(check_gate(gate));
  TG_TRY(check_range("M", M, 0, kMax22));
  TG_TRY(check_range("K", K, 0, kMax22));
  if (K % 16) return fail(TILE_GEMM_ERR_BAD_SHAPE, "K=%lld: must be a multiple of 16", (long long)K);
  if (rows && blocks) return fail(TILE_GEMM_ERR_BAD_SHAPE, "rows: not with blocks of 128 x 128");
  if (rows) TG_TRY(check_range("x_rows", x_rows, 0, kMaxDim));
  if (M == 0 || K == 0) return TILE_GEMM_OK;
  const int64_t xr = rows ? x_rows : M, xc = gated ? 2 * K : K;
  TG_TRY(check_stride("x_stride", ldx, xc, kMax22, xr));
  TG_TRY(check_stride("q_stride", ldq, K, kMax22, M));
  const int64_t kb = tg::ceil_div(K, tg::kScaleBlock);
  Arg a[4];
  int n = 0;
  a[n++] = wide_matrix("X", X, xr, xc, ldx, 2);
  a[n++] = wide_matrix("Q", Q, M, K, ldq, 1, true);
  a[n++] = blocks ? scales("scale", scale, tg::ceil_div(M, tg::kScaleBlock), kb, lds, true)
                  : scales("scale", scale, kb, M, lds, true);
  if (rows) a[n++] = vec("rows", rows, M, 4);
  return check_arg_list(a, n);
}

tile_gemm_status_t check_route_common(int64_t T, int64_t E, int64_t k, int64_t ld, const tile_gemm_route_t* o) {
  g_detail[0] = '\0';
  if (!o) return fail(TILE_GEMM_ERR_NULL_ARG, "options: NULL");
  if (o->score != TILE_GEMM_SCORE_SOFTMAX && o->score != TILE_GEMM_SCORE_SIGMOID)
    return fail(TILE_GEMM_ERR_DTYPE, "score: unknown value %d", (int)o->score);
  if (o->logits_type != TILE_GEMM_LOGITS_F32 && o->logits_type != TILE_GEMM_LOGITS_BF16)
    return fail(TILE_GEMM_ERR_DTYPE, "logits_type: unknown value %d", (int)o->logits_type);
  if (!(o->scale > -INFINITY && o->scale < INFINITY))
    return fail(TILE_GEMM_ERR_BAD_SHAPE, "scale: %g, must be finite", (double)o->scale);
  TG_TRY(check_range("T", T, 0, kMaxRouteT));
  TG_TRY(check_range("E", E, 1, tg::kBlockMaxGroups + 1));
  TG_TRY(check_range("k", k, 1, kMaxRouteK + 1));
  return check_stride("logit_stride", ld, E, kMaxDim, T);
}
Arg logits_arg(const char* name, const void* p, int64_t T, int64_t E, int64_t ld, const tile_gemm_route_t* o,
               bool written = false) {
  const int esz = o->logits_type == TILE_GEMM_LOGITS_BF16 ? 2 : 4;
  return Arg{name, p, T, E, ld, esz, esz, written, true};
}

tile_gemm_status_t check_route(const void* logits, const float* bias, const int32_t* ids, const float* weights,
                               int64_t T, int64_t E, int64_t k, int64_t ld, const tile_gemm_route_t* o) {
  TG_TRY(check_route_common(T, E, k, ld, o));
  if (o->groups < 1 || o->groups > kMaxGroups || E % o->groups)
    return fail(TILE_GEMM_ERR_BAD_SHAPE, "groups=%d: must be in [1, %d] and divide E=%lld", (int)o->groups,
                (int)kMaxGroups, (long long)E);
  if (o->top_groups < 1 || o->top_groups > o->groups)
    return fail(TILE_GEMM_ERR_BAD_SHAPE, "top_groups=%d: must be in [1, groups=%d]", (int)o->top_groups,
                (int)o->groups);
  if (o->group_top != 1 && o->group_top != 2)
    return fail(TILE_GEMM_ERR_BAD_SHAPE, "group_top=%d: must be 1 or 2", (int)o->group_top);
  if (k > o->top_groups * (E / o->groups))
    return fail(TILE_GEMM_ERR_BAD_SHAPE, "k=%lld: only %lld experts can be chosen", (long long)k,
                (long long)(o->top_groups * (E / o->groups)));
  Arg a[4];
  int n = 0;
  a[n++] = logits_arg("logits", logits, T, E, ld, o);
  if (bias) a[n++] = vec("bias", bias, T ? E : 0, 4);
  a[n++] = vec("ids", ids, T * k, 4, true);
  a[n++] = vec("weights", weights, T * k, 4, true);
  return check_arg_list(a, n);
}

tile_gemm_status_t check_route_backward(const void* logits, const int32_t* ids, const float* dweights,
                                        const void* dlogits, int64_t T, int64_t E, int64_t k, int64_t ld,
                                        int64_t ldd, const tile_gemm_route_t* o) {
  TG_TRY(check_route_common(T, E, k, ld, o));
  TG_TRY(check_stride("dlogit_stride", ldd, E, kMaxDim, T));
  const Arg a[4] = {logits_arg("logits", logits, T, E, ld, o), vec("ids", ids, T * k, 4),
                    vec("dweights", dweights, T * k, 4), logits_arg("dlogits", dlogits, T, E, ldd, o, true)};
  return check_arg_list(a, 4);
}

struct PlacePlan {
  int64_t chunks, rounds, bytes;
};
// One workgroup up to 4096 entries (a second launch costs more than its three
// further rounds), then 1024 entries each and at most 128 of them.
PlacePlan plan_place(int64_t n, int64_t E) {
  PlacePlan p;
  p.rounds = n <= 4 * kPlaceRound ? tg::ceil_div(n, kPlaceRound) : tg::ceil_div(n, kPlaceRound * kPlaceMaxChunks);
  if (p.rounds < 1) p.rounds = 1;
  p.chunks = tg::ceil_div(n, p.rounds * kPlaceRound);
  if (p.chunks < 1) p.chunks = 1;
  p.bytes = p.chunks > 1 ? p.chunks * E * 4 : 0;
  return p;
}
tile_gemm_status_t check_place_shape(int64_t T, int64_t k, int64_t E) {
  g_detail[0] = '\0';
  TG_TRY(check_range("T", T, 0, kMaxDim));
  TG_TRY(check_range("k", k, 1, kMaxDim));
  TG_TRY(check_range("E", E, 1, tg::kBlockMaxGroups + 1));
  if (T * k >= kMaxDim) return fail(TILE_GEMM_ERR_BAD_SHAPE, "T k=%lld: must be below 2^31", (long long)(T * k));
  return TILE_GEMM_OK;
}
tile_gemm_status_t check_place(const int32_t* ids, int64_t T, int64_t k, int64_t first, int64_t E,
                               const int32_t* offsets, const int32_t* rows, const int32_t* places, const void* ws,
                               int64_t ws_bytes, PlacePlan* plan) {
  TG_TRY(check_place_shape(T, k, E));
  TG_TRY(check_range("first", first, 0, kMaxDim));
  *plan = plan_place(T * k, E);
  TG_TRY(check_workspace(ws, ws_bytes, plan->bytes));
  Arg a[5];
  int n = 0;
  a[n++] = vec("ids", ids, T * k, 4);
  a[n++] = vec("offsets", offsets, E + 1, 4, true);
  if (rows) a[n++] = vec("rows", rows, T * k, 4, true);
  if (places) a[n++] = vec("places", places, T * k, 4, true);
  if (plan->bytes) a[n++] = vec("workspace", ws, plan->bytes, 1, true);
  return check_arg_list(a, n);
}

tile_gemm_status_t check_combine(const void* Z, const int32_t* places, const float* weights, const void* Y,
                                 int64_t T, int64_t N, int64_t k, int64_t z_rows, int64_t ldz, int64_t ldy,
                                 int dtype) {
  g_detail[0] = '\0';
  TG_TRY(check_dtype(dtype));
  TG_TRY(check_range("T", T, 0, kMax22));
  TG_TRY(check_range("N", N, 0, kMax22));
  TG_TRY(check_range("k", k, 1, kMaxCombineK + 1));
  TG_TRY(check_range("z_rows", z_rows, 0, kMaxDim));
  if (T == 0 || N == 0) return TILE_GEMM_OK;
  // (threads of 8 columns each, in workgroups of 256: a launch has less than 2^32)
  if (T * tg::ceil_div(N, 8) > 2 * kMaxDim - 512)
    return fail(TILE_GEMM_ERR_BAD_SHAPE, "shape: T=%lld N=%lld, too many values for one call", (long long)T,
                (long long)N);
  Arg a[4];
  int n = 0;
  a[n++] = wide_matrix("Z", Z, z_rows, N, ldz, 2);
  a[n++] = vec("places", places, T * k, 4);
  if (weights) a[n++] = vec("weights", weights, T * k, 4);
  a[n++] = wide_matrix("Y", Y, T, N, ldy, dtype == TILE_GEMM_BF16_TO_F32 ? 4 : 2, true);
  return check_arg_list(a, n);
}

}  // namespace

extern "C" {

tile_gemm_status_t tile_gemm_check_fp8(const void* A, const void* B, const void* C, int64_t M, int64_t N, int64_t K,
                                       const tile_gemm_fp8_strides_t* strides, const float* a_scale,
                                       const float* b_scale, tile_gemm_dtype_t dtype, const float* bias,
                                       tile_gemm_act_t act) {
  return check_fp8(A, B, C, M, N, K, -1, nullptr, strides, a_scale, b_scale, (int)dtype, bias, (int)act);
}

tile_gemm_status_t tile_gemm_check_fp8_experts(const void* A, const void* B, const void* C, int64_t M, int64_t N,
                                               int64_t K, int64_t E, const int32_t* offsets,
                                               const tile_gemm_fp8_strides_t* strides, const float* a_scale,
                                               const float* b_scale, tile_gemm_dtype_t dtype) {
  return check_fp8(A, B, C, M, N, K, E < 0 ? 0 : E, offsets, strides, a_scale, b_scale, (int)dtype, nullptr,
                   TILE_GEMM_ACT_NONE);
}

tile_gemm_status_t tile_gemm_check_quantize(const void* X, const void* Q, const float* scale, int64_t M, int64_t K,
                                            int64_t x_stride, int64_t q_stride, int64_t scale_stride,
                                            tile_gemm_quant_t form, tile_gemm_gate_t gate, const int32_t* rows,
                                            int64_t x_rows) {
  return check_quantize(X, Q, scale, M, K, x_stride, q_stride, scale_stride, (int)form, (int)gate, rows, x_rows);
}

tile_gemm_status_t tile_gemm_check_route(const void* logits, const float* bias, const int32_t* ids,
                                         const float* weights, int64_t T, int64_t E, int64_t k,
                                         int64_t logit_stride, const tile_gemm_route_t* options) {
  return check_route(logits, bias, ids, weights, T, E, k, logit_stride, options);
}

tile_gemm_status_t tile_gemm_check_route_backward(const void* logits, const int32_t* ids, const float* dweights,
                                                  const void* dlogits, int64_t T, int64_t E, int64_t k,
                                                  int64_t logit_stride, int64_t dlogit_stride,
                                                  const tile_gemm_route_t* options) {
  return check_route_backward(logits, ids, dweights, dlogits, T, E, k, logit_stride, dlogit_stride, options);
}

tile_gemm_status_t tile_gemm_check_place(const int32_t* ids, int64_t T, int64_t k, int64_t first, int64_t E,
                                         const int32_t* offsets, const int32_t* rows, const int32_t* places,
                                         const void* workspace, int64_t workspace_bytes) {
  PlacePlan p;
  return check_place(ids, T, k, first, E, offsets, rows, places, workspace, workspace_bytes, &p);
}

tile_gemm_status_t tile_gemm_place_workspace(int64_t T, int64_t k, int64_t E, int64_t* bytes) {
  if (!bytes) return fail(TILE_GEMM_ERR_NULL_ARG, "bytes: NULL");
  TG_TRY(check_place_shape(T, k, E));
  *bytes = plan_place(T * k, E).bytes;
  return TILE_GEMM_OK;
}

tile_gemm_status_t tile_gemm_check_combine(const void* Z, const int32_t* places, const float* weights, const void* Y,
                                           int64_t T, int64_t N, int64_t k, int64_t z_rows, int64_t z_stride,
                                           int64_t y_stride, tile_gemm_dtype_t dtype) {
  return check_combine(Z, places, weights, Y, T, N, k, z_rows, z_stride, y_stride, (int)dtype);
}

tile_gemm_status_t tile_gemm_plan_fp8(int64_t M, int64_t N, int64_t K, int64_t E, tile_gemm_dtype_t dtype,
                                      int cu_count, tile_gemm_plan_t* out) {
  g_detail[0] = '\0';
  TG_TRY(check_dtype((int)dtype));
  const bool fp32 = dtype == TILE_GEMM_BF16_TO_F32;
  if (!out) return fail(TILE_GEMM_ERR_NULL_ARG, "out: NULL");
  TG_TRY(check_range("M", M, 0, kMax22));
  TG_TRY(check_range("N", N, 0, kMax22));
  TG_TRY(check_range("K", K, 0, kMax22));
  TG_TRY(check_range("E", E, 0, tg::kBlockMaxGroups + 1));
  if ((tg::ceil_div(M, 16) + E) * tg::ceil_div(N, 32) >= kMaxDim)
    return fail(TILE_GEMM_ERR_BAD_SHAPE, "shape: too many tiles");
  if (cu_count <= 0) return fail(TILE_GEMM_ERR_DEVICE, "cu_count: %d", cu_count);
  fill_plan(E ? tg::make_plan_experts(M, N, K, E, fp32, cu_count) : tg::make_plan_block(M, N, K, fp32, cu_count), out);
  return TILE_GEMM_OK;
}

}  // extern "C"
