// train_abi.hpp -- argument checks and workspace sizes of the gated block's
// backward pass and of the cross entropy of a projection (include/tile_gemm.h).
// Host only; included after host_abi.hpp by the library's one translation unit.
#pragma once

#include <math.h>

#include "host_abi.hpp"
#include "train_plan.hpp"

namespace {

constexpr int kDefaultCus = 256;  // an MI355X, where no handle says otherwise

// One argument of a call: `rows` rows of `cols` elements of `esz` bytes, `ld`
// elements apart, unit column stride; a vector is one row.
struct Arg {
  const char* name;
  const void* p;
  int64_t rows, cols, ld, esz;
  int align;      // bytes: of the base and of the leading dimension
  bool written;
  bool wide;      // may span 4 GiB or more
};

Arg matrix(const char* name, const void* p, int64_t rows, int64_t cols, int64_t ld, int64_t esz,
           bool written = false, bool wide = false) {
  return Arg{name, p, rows, cols, ld, esz, 16, written, wide};
}
Arg vec(const char* name, const void* p, int64_t n, int64_t esz, bool written = false) {
  return Arg{name, p, 1, n, n, esz, (int)esz, written, true};
}

// Every argument's pointer, stride, alignment and extent, then that no
// written argument overlaps any other (arguments left out are NULL and
// dropped by the caller).
tile_gemm_status_t check_arg_list(const Arg* a, int n) {
  uintptr_t lo[16], hi[16];
  for (int i = 0; i < n; ++i) {
    const Arg& x = a[i];
    lo[i] = hi[i] = 0;
    if (x.rows == 0 || x.cols == 0) continue;
    if (!x.p) return fail(TILE_GEMM_ERR_NULL_ARG, "%s: NULL", x.name);
    if (x.rows > 1 && x.ld < x.cols)
      return fail(TILE_GEMM_ERR_BAD_STRIDE, "%s: leading dimension %lld, must be >= %lld", x.name,
                  (long long)x.ld, (long long)x.cols);
    if (x.rows > 1 && x.ld >= kMaxDim)
      return fail(TILE_GEMM_ERR_BAD_STRIDE, "%s: leading dimension %lld, must be < 2^31", x.name,
                  (long long)x.ld);
    if ((uintptr_t)x.p % x.align)
      return fail(TILE_GEMM_ERR_MISALIGNED, "%s: pointer not %d-byte aligned", x.name, x.align);
    if (x.rows > 1 && (x.ld * x.esz) % x.align)
      return fail(TILE_GEMM_ERR_MISALIGNED, "%s: leading dimension %lld is not a multiple of %d bytes",
                  x.name, (long long)x.ld, x.align);
    const int64_t span = span_bytes(x.rows, x.rows > 1 ? x.ld : 0, x.cols, x.esz);
    if (span < 0 || (!x.wide && span >= ((int64_t)1 << 32)))
      return fail(TILE_GEMM_ERR_BAD_SHAPE, "%s: spans %lld bytes, must be below 4 GiB", x.name,
                  (long long)span);
    lo[i] = (uintptr_t)x.p;
    hi[i] = lo[i] + (uintptr_t)span;
    if (hi[i] < lo[i])
      return fail(TILE_GEMM_ERR_BAD_SHAPE, "%s: its byte range overflows the address space", x.name);
  }
  for (int i = 0; i < n; ++i)
    for (int j = 0; j < i; ++j)
      if ((a[i].written || a[j].written) && overlap(lo[i], hi[i], lo[j], hi[j]))
        return fail(TILE_GEMM_ERR_ALIAS, "%s overlaps %s (%s is written)", a[i].name, a[j].name,
                    a[i].written ? a[i].name : a[j].name);
  return TILE_GEMM_OK;
}

// Rows (tokens) and columns these operators take in one call: a 256-row panel
// of either axis, 2 bytes a value, stays below 4 GiB.
constexpr int64_t kTrainMaxRows = (int64_t)1 << 22;

tile_gemm_status_t check_train_shape(int64_t M, int64_t N, int64_t K, int64_t max_n) {
  g_detail[0] = '\0';
  if (M < 0 || N < 0 || K < 1)
    return fail(TILE_GEMM_ERR_BAD_SHAPE, "shape: M=%lld N=%lld K=%lld, need M, N >= 0 and K >= 1",
                (long long)M, (long long)N, (long long)K);
  if (M >= kTrainMaxRows || N >= max_n || K >= kTrainMaxRows)
    return fail(TILE_GEMM_ERR_BAD_SHAPE,
                "shape: M=%lld N=%lld K=%lld, need M and K < 2^22 and N < %lld", (long long)M,
                (long long)N, (long long)K, (long long)max_n);
  // the kernels number tiles (32 x 64 at the smallest) in 32 bits, those of
  // the gradients M x K and N x K too
  const int64_t cols = tg::ceil_div(K, 64);
  if (tg::ceil_div(M, 32) * tg::ceil_div(N, 64) >= kMaxDim || tg::ceil_div(M, 32) * cols >= kMaxDim ||
      tg::ceil_div(N, 32) * cols >= kMaxDim)
    return fail(TILE_GEMM_ERR_BAD_SHAPE, "shape: M=%lld N=%lld K=%lld, too many tiles for one call",
                (long long)M, (long long)N, (long long)K);
  return TILE_GEMM_OK;
}

// W (B) is taken as it is stored: N rows of K consecutive values.
tile_gemm_status_t check_col_major(const char* name, const tile_gemm_strides_t* s, int64_t K) {
  if (s->b_k != 1 || s->b_n < K || s->b_n >= kTrainMaxRows)
    return fail(TILE_GEMM_ERR_BAD_STRIDE,
                "%s strides (b_k=%lld, b_n=%lld): need b_k == 1 and K=%lld <= b_n < 2^22 (column-major)",
                name, (long long)s->b_k, (long long)s->b_n, (long long)K);
  return TILE_GEMM_OK;
}
tile_gemm_status_t check_unit(const char* name, int64_t stride, const char* which) {
  if (stride != 1)
    return fail(TILE_GEMM_ERR_BAD_STRIDE, "%s: %s=%lld, must be 1", name, which, (long long)stride);
  return TILE_GEMM_OK;
}

tile_gemm_status_t check_workspace(const void* ws, int64_t have, int64_t need) {
  if (need == 0) return TILE_GEMM_OK;
  if (!ws) return fail(TILE_GEMM_ERR_WORKSPACE, "workspace: NULL, needs %lld bytes", (long long)need);
  if ((uintptr_t)ws % 256) return fail(TILE_GEMM_ERR_WORKSPACE, "workspace: not 256-byte aligned");
  if (have < need)
    return fail(TILE_GEMM_ERR_WORKSPACE, "workspace: %lld bytes, needs %lld", (long long)have,
                (long long)need);
  return TILE_GEMM_OK;
}

#define TG_TRY(x)                                \
  do {                                           \
    const tile_gemm_status_t st_ = (x);          \
    if (st_ != TILE_GEMM_OK) return st_;         \
  } while (0)

// --------------------------------------------------- gated block, backward

tile_gemm_status_t check_gate(int gate) {
  if (gate < TILE_GEMM_GATE_SILU || gate > TILE_GEMM_GATE_SIGMOID)
    return fail(TILE_GEMM_ERR_EPILOGUE, "gate: unknown activation %d", gate);
  return TILE_GEMM_OK;
}

// Checks and, in *plan, the launch plan.
tile_gemm_status_t check_glu_backward(const void* A, const void* B, const void* dC, const void* dA,
                                      const void* dB, int64_t M, int64_t N, int64_t K,
                                      const tile_gemm_strides_t* s, const tile_gemm_strides_t* g,
                                      const float* bias, const float* dbias, int gate, const void* ws,
                                      int64_t ws_bytes, int cu, tg::GluGradPlan* plan) {
  TG_TRY(check_train_shape(M, N, K, kTrainMaxRows));
  if (N % 16)
    return fail(TILE_GEMM_ERR_BAD_SHAPE,
                "N=%lld: a gated block needs B's column count (gate + up) a multiple of 16", (long long)N);
  TG_TRY(check_gate(gate));
  if (!s || !g) return fail(TILE_GEMM_ERR_NULL_ARG, "strides: NULL");
  // (an empty gradient has no address either)
  if (M && N && !dA && !dB && !dbias) return fail(TILE_GEMM_ERR_NULL_ARG, "dA, dB and dbias: all NULL");
  TG_TRY(check_unit("A", s->a_k, "a_k"));
  TG_TRY(check_col_major("B", s, K));
  TG_TRY(check_unit("dC", g->c_n, "c_n"));
  if (dA) TG_TRY(check_unit("dA", g->a_k, "a_k"));
  if (dB) TG_TRY(check_col_major("dB", g, K));
  *plan = tg::plan_glu_grad(M, N, K, dA != nullptr, dB != nullptr, dbias != nullptr, cu);
  Arg a[9];
  int n = 0;
  a[n++] = matrix("A", A, N ? M : 0, K, s->a_m, 2);
  a[n++] = matrix("B", B, M ? N : 0, K, s->b_n, 2);
  a[n++] = matrix("dC", dC, M, N / 2, g->c_m, 2);
  if (dA) a[n++] = matrix("dA", dA, M, K, g->a_m, 2, true);
  if (dB) a[n++] = matrix("dB", dB, N, K, g->b_n, 2, true);
  if (bias) {
    a[n] = vec("bias", bias, N, 4);
    a[n++].align = 16;
  }
  if (dbias) a[n++] = vec("dbias", dbias, N, 4, true);
  TG_TRY(check_workspace(ws, ws_bytes, plan->bytes));
  if (plan->bytes) a[n++] = vec("workspace", ws, plan->bytes, 1, true);
  return check_arg_list(a, n);
}

// ---------------------------------------------------------- cross entropy

tile_gemm_status_t check_xent_common(const void* target, int64_t M, int64_t N, int64_t K,
                                     const tile_gemm_strides_t* s, const tile_gemm_xent_t* o) {
  TG_TRY(check_train_shape(M, N, K, kMaxDim));
  if (N < 1) return fail(TILE_GEMM_ERR_BAD_SHAPE, "N=%lld: the vocabulary must not be empty", (long long)N);
  if (!s) return fail(TILE_GEMM_ERR_NULL_ARG, "strides: NULL");
  if (!o) return fail(TILE_GEMM_ERR_NULL_ARG, "options: NULL");
  if (o->target_type != TILE_GEMM_INDEX_I32 && o->target_type != TILE_GEMM_INDEX_I64)
    return fail(TILE_GEMM_ERR_DTYPE, "target_type: unknown value %d", (int)o->target_type);
  if (!(o->label_smoothing >= 0.0f && o->label_smoothing <= 1.0f))
    return fail(TILE_GEMM_ERR_BAD_SHAPE, "label_smoothing: %g, must be in [0, 1]", (double)o->label_smoothing);
  if (!(o->z_loss >= 0.0f && o->z_loss < INFINITY))
    return fail(TILE_GEMM_ERR_BAD_SHAPE, "z_loss: %g, must be finite and >= 0", (double)o->z_loss);
  if (o->piece < 0) return fail(TILE_GEMM_ERR_BAD_SHAPE, "piece: %lld, must be >= 0", (long long)o->piece);
  TG_TRY(check_unit("A", s->a_k, "a_k"));
  TG_TRY(check_col_major("B", s, K));
  (void)target;
  return TILE_GEMM_OK;
}
Arg target_arg(const void* target, int64_t M, const tile_gemm_xent_t* o) {
  return vec("target", target, M, o->target_type == TILE_GEMM_INDEX_I64 ? 8 : 4);
}

tile_gemm_status_t check_xent(const void* A, const void* B, const void* target, const float* loss,
                              const float* lse, int64_t M, int64_t N, int64_t K,
                              const tile_gemm_strides_t* s, const tile_gemm_xent_t* o, const void* ws,
                              int64_t ws_bytes, int cu, tg::XentPlan* plan) {
  TG_TRY(check_xent_common(target, M, N, K, s, o));
  if (M && !loss && !lse) return fail(TILE_GEMM_ERR_NULL_ARG, "loss and lse: both NULL");
  *plan = tg::plan_xent(M, N, K, o->label_smoothing > 0.0f, cu);
  if (M == 0) return TILE_GEMM_OK;
  Arg a[6];
  int n = 0;
  a[n++] = matrix("A", A, M, K, s->a_m, 2);
  a[n++] = matrix("B", B, N, K, s->b_n, 2, false, true);
  a[n++] = target_arg(target, M, o);
  if (loss) a[n++] = vec("loss", loss, M, 4, true);
  if (lse) a[n++] = vec("lse", lse, M, 4, true);
  TG_TRY(check_workspace(ws, ws_bytes, plan->bytes));
  a[n++] = vec("workspace", ws, plan->bytes, 1, true);
  return check_arg_list(a, n);
}

tile_gemm_status_t check_xent_backward(const void* A, const void* B, const void* target, const float* lse,
                                       const float* dloss, const void* dA, const void* dB, int64_t M,
                                       int64_t N, int64_t K, const tile_gemm_strides_t* s,
                                       const tile_gemm_strides_t* g, const tile_gemm_xent_t* o,
                                       const void* ws, int64_t ws_bytes, int cu, tg::XentGradPlan* plan) {
  TG_TRY(check_xent_common(target, M, N, K, s, o));
  if (!g) return fail(TILE_GEMM_ERR_NULL_ARG, "grad_strides: NULL");
  if (M && !dA && !dB) return fail(TILE_GEMM_ERR_NULL_ARG, "dA and dB: both NULL");
  if (dA) TG_TRY(check_unit("dA", g->a_k, "a_k"));
  if (dB) TG_TRY(check_col_major("dB", g, K));
  *plan = tg::plan_xent_grad(M, N, K, s->b_n, o->piece, dA != nullptr, dB != nullptr, cu);
  Arg a[8];
  int n = 0;
  a[n++] = matrix("A", A, M, K, s->a_m, 2);
  a[n++] = matrix("B", B, M ? N : 0, K, s->b_n, 2, false, true);
  a[n++] = target_arg(target, M, o);
  a[n++] = vec("lse", lse, M, 4);
  a[n++] = vec("dloss", dloss, M, 4);
  if (dA) a[n++] = matrix("dA", dA, M, K, g->a_m, 2, true);
  if (dB) a[n++] = matrix("dB", dB, N, K, g->b_n, 2, true, true);
  TG_TRY(check_workspace(ws, ws_bytes, plan->bytes));
  if (plan->bytes) a[n++] = vec("workspace", ws, plan->bytes, 1, true);
  return check_arg_list(a, n);
}

}  // namespace

extern "C" {

tile_gemm_status_t tile_gemm_check_glu_backward(const void* A, const void* B, const void* dC, const void* dA,
                                                const void* dB, int64_t M, int64_t N, int64_t K,
                                                const tile_gemm_strides_t* strides,
                                                const tile_gemm_strides_t* grad_strides, const float* bias,
                                                const float* dbias, tile_gemm_gate_t gate,
                                                const void* workspace, int64_t workspace_bytes) {
  tg::GluGradPlan p;
  return check_glu_backward(A, B, dC, dA, dB, M, N, K, strides, grad_strides, bias, dbias, (int)gate, workspace,
                            workspace_bytes, kDefaultCus, &p);
}

tile_gemm_status_t tile_gemm_check_xent(const void* A, const void* B, const void* target, const float* loss,
                                        const float* lse, int64_t M, int64_t N, int64_t K,
                                        const tile_gemm_strides_t* strides, const tile_gemm_xent_t* options,
                                        const void* workspace, int64_t workspace_bytes) {
  tg::XentPlan p;
  return check_xent(A, B, target, loss, lse, M, N, K, strides, options, workspace, workspace_bytes, kDefaultCus,
                    &p);
}

tile_gemm_status_t tile_gemm_check_xent_backward(const void* A, const void* B, const void* target,
                                                 const float* lse, const float* dloss, const void* dA,
                                                 const void* dB, int64_t M, int64_t N, int64_t K,
                                                 const tile_gemm_strides_t* strides,
                                                 const tile_gemm_strides_t* grad_strides,
                                                 const tile_gemm_xent_t* options, const void* workspace,
                                                 int64_t workspace_bytes) {
  tg::XentGradPlan p;
  return check_xent_backward(A, B, target, lse, dloss, dA, dB, M, N, K, strides, grad_strides, options, workspace,
                             workspace_bytes, kDefaultCus, &p);
}

tile_gemm_status_t tile_gemm_plan_train(int64_t M, int64_t N, int64_t K, tile_gemm_train_product_t product,
                                        int cu_count, tile_gemm_plan_t* out) {
  g_detail[0] = '\0';
  if (!out) return fail(TILE_GEMM_ERR_NULL_ARG, "out: NULL");
  if (M < 1 || N < 1 || K < 1 || M >= kMaxDim || N >= kMaxDim || K >= kMaxDim)
    return fail(TILE_GEMM_ERR_BAD_SHAPE, "shape: M, N and K must be in [1, 2^31)");
  if (product < TILE_GEMM_TRAIN_LOGITS || product > TILE_GEMM_TRAIN_GRADIENT)
    return fail(TILE_GEMM_ERR_BAD_SHAPE, "product: unknown value %d", (int)product);
  if (tg::ceil_div(M, 32) * tg::ceil_div(N, 64) >= kMaxDim)
    return fail(TILE_GEMM_ERR_BAD_SHAPE, "shape: too many tiles");
  if (cu_count <= 0) return fail(TILE_GEMM_ERR_DEVICE, "cu_count: %d", cu_count);
  const tg::TrainProduct q = product == TILE_GEMM_TRAIN_GRADIENT
                                 ? tg::plan_product(M, N, K, tg::kMaxSplits, cu_count)
                                 : tg::plan_forward(M, N, K, cu_count, product == TILE_GEMM_TRAIN_GATED).z;
  fill_plan(tg::train_plan(q), out);
  return TILE_GEMM_OK;
}

}  // extern "C"
