// train_run.hpp -- the launches of the gated block's backward pass and of the
// cross entropy of a projection, and their C entry points. Included by the
// library's one host translation unit (tile_gemm.hip) after the handle.
#pragma once

#include "train_abi.hpp"
#include "train_launch.hpp"

namespace {

template <int ID>
hipError_t dispatch_train_from(int id, const tg::TrainArgs& a, int64_t grid, hipStream_t st) {
  if constexpr (ID < tg::kNumTrainKernels) {
    if (id == ID) return tg::launch_train<ID>(a, grid, st);
    return dispatch_train_from<ID + 1>(id, a, grid, st);
  } else {
    return hipErrorInvalidValue;
  }
}

hipError_t launch_product(const tg::TrainProduct& q, int store, tg::TrainArgs& a, hipStream_t st,
                          bool bcol = true, bool bf16 = true) {
  a.map = q.map;
  a.splits = q.splits;
  a.k_per = (int32_t)q.k_per;
  return dispatch_train_from<0>(tg::train_kernel(store, q.tile, a.gate, bcol, bf16), a, q.grid, st);
}

// A gradient's product over a row-major right operand, `with` a few-token
// weight gradient in the same launch.
hipError_t launch_gradient(const tg::TrainProduct& q, tg::TrainArgs& a, bool bf16, const tg::OuterArgs* with,
                           int cu, hipStream_t st) {
  if (!with) return launch_product(q, bf16 ? tg::kStoreBf16 : tg::kStoreParts, a, st, false, bf16);
  a.map = q.map;
  a.splits = q.splits;
  a.k_per = (int32_t)q.k_per;
  return tg::launch_pair(a, q.grid, bf16, *with, cu, st);
}

tile_gemm_status_t hip_status(hipError_t e) {
  if (e == hipSuccess) return TILE_GEMM_OK;
  return fail(TILE_GEMM_ERR_HIP, "launch: %s", hipGetErrorString(e));
}
#define TG_LAUNCH(x) TG_TRY(hip_status(x))

tile_gemm_status_t check_device(tile_gemm_t h) {
  int cur = -1;
  if (hipGetDevice(&cur) != hipSuccess || cur != h->device)
    return fail(TILE_GEMM_ERR_DEVICE, "current device %d is not the handle's device %d", cur, h->device);
  return TILE_GEMM_OK;
}

void log_product(tile_gemm_handle* h, const char* kind, int64_t M, int64_t N, int64_t K,
                 const tg::TrainProduct& q) {
  if (h->log) log_plan(h, kind, M, N, K, 1, 1, 0, tg::train_plan(q));
}

// Whether the weight gradient (rows x cols over `tokens`) takes the few-token
// kernel. Up to 32 tokens it runs near the rate of its writes (the whole
// backward pass of 1 token, 14000 x 8192, 144 us for the 164 with the tile
// kernel). Past them its registers leave too few waves for that, and the tile
// kernel is faster unless the result is small and the launch that the pair
// saves counts: 64 tokens, 8000 x 512 42.9 and 45.0, 16000 x 1024 66.2 and
// 64.6, 10000 x 4096 86.9 and 76.9; 100 tokens, 272 x 264 20.5 and 23.3, 8000 x
// 1024 45.2 and 41.3; 128 tokens, 32000 x 1024 137 and 107.
bool few_tokens(int64_t tokens, int64_t rows, int64_t cols) {
  return tokens <= 32 || (tokens <= tg::kOuterMaxT && rows * cols * 2 <= ((int64_t)8 << 20));
}
// Whether it then rides along with the launch of the other gradient's product
// q. On the small tile both are mostly latency (40 tokens, 2736 x 1024: 29.8 to
// 24.1 us for the whole backward pass). Few workgroups of the pair fit a
// compute unit, though, and from 64 MiB on the weight gradient alone is faster
// (24 tokens: 32000 x 1024 80 to 78 us, 8 tokens: 10000 x 4096 63 to 66).
bool pairs(const tg::TrainProduct& q, int64_t tokens, int64_t rows, int64_t cols) {
  return q.tile == tg::kSmallTile && few_tokens(tokens, rows, cols) && rows * cols * 2 <= ((int64_t)64 << 20);
}

// The row stride the kernels take for x: a single row may come with any, but
// the offsets of a tile's other rows are formed from it, and whole chunks
// loaded there need them to be multiples of 16 bytes.
int64_t row_stride(int64_t rows, int64_t ld, int64_t cols) { return rows > 1 ? ld : tg::ceil_div(cols, 8) * 8; }

// One gradient: out (bf16) = scale * (left [rows x len]) . (right [len x cols],
// row-major), by parts of the contraction when the plan says so. left is G or
// dz as a store wrote it: its rows are zero past len up to a multiple of 8.
tile_gemm_status_t run_gradient(const tg::TrainProduct& q, const uint16_t* left, int64_t ldl,
                                const uint16_t* right, int64_t ldr, int64_t rows, int64_t cols, int64_t len,
                                uint16_t* out, int64_t ldo, const float* scale, float* part,
                                hipStream_t st, const tg::OuterArgs* with = nullptr, int cu = 0) {
  tg::TrainArgs a{};
  a.A = left;
  a.B = right;
  a.M = (int32_t)rows;
  a.N = (int32_t)cols;
  a.K = (int32_t)len;
  a.lda = ldl;
  a.ldb = ldr;
  if (q.splits == 1) {
    a.C = out;
    a.ldc = ldo;
    a.scale = scale;
    return hip_status(launch_gradient(q, a, true, with, cu, st));
  }
  a.C = part;
  a.ldc = tg::ceil_div(cols, 4) * 4;
  a.part_stride = rows * a.ldc;
  TG_LAUNCH(launch_gradient(q, a, false, with, cu, st));
  return hip_status(tg::launch_add_parts(tg::AddArgs{part, a.part_stride, q.splits, (int32_t)rows, (int32_t)cols,
                                                     a.ldc, scale, out, ldo},
                                         st));
}

// The gated forward product. With a row-major B, silu is the plain kernels'
// SwiGLU store (which have a few-row kernel for that layout).
tile_gemm_status_t run_glu(tile_gemm_t h, const void* A, const void* B, void* C, int64_t M, int64_t N,
                           int64_t K, const tile_gemm_strides_t* s, int dtype, const float* bias, int gate,
                           void* stream) {
  if (!h) return fail(TILE_GEMM_ERR_NULL_ARG, "handle: NULL");
  TG_TRY(check_args(A, B, C, M, N, K, s, dtype, N / 2));
  TG_TRY(check_epilogue(C, M, N, s, dtype, bias, TILE_GEMM_ACT_SWIGLU));
  if (M == 0 || N == 0) return TILE_GEMM_OK;
  TG_TRY(check_device(h));
  const bool bcol = K > 0 && !b_is_row_major(s, N);
  const tg::TrainProduct q =
      bcol ? tg::plan_forward(M, N, K, h->cu_count, true).z
                                  : tg::plan_product(M, N, K, 1, h->cu_count, true);
  if (q.grid > 0x7fffffff) return fail(TILE_GEMM_ERR_BAD_SHAPE, "shape: too many workgroups");
  tg::TrainArgs a{};
  a.A = static_cast<const uint16_t*>(A);
  a.B = static_cast<const uint16_t*>(B);
  a.C = C;
  a.M = (int32_t)M;
  a.N = (int32_t)N;
  a.K = (int32_t)K;
  a.lda = s->a_m;
  a.ldb = bcol ? s->b_n : s->b_k;
  a.ldc = s->c_m;
  a.bias = bias;
  a.glu_half = (int32_t)(N / 2);
  a.gate = gate;
  log_product(h, "run_glu", M, N, K, q);
  return hip_status(launch_product(q, tg::kStoreGlu, a, static_cast<hipStream_t>(stream), bcol,
                                   dtype == TILE_GEMM_BF16_TO_BF16));
}

// The weight gradient dW = scale * left . right with left V x T (G or dz
// transposed) and right the T x K activations.
tile_gemm_status_t run_weight_gradient(const tg::TrainProduct& q, const uint16_t* left, int64_t ldl,
                                       const uint16_t* right, int64_t ldr, int64_t rows, int64_t cols,
                                       int64_t len, uint16_t* out, int64_t ldo, const float* scale, float* part,
                                       int cu, hipStream_t st) {
  if (few_tokens(len, rows, cols))
    return hip_status(tg::launch_outer(tg::OuterArgs{left, ldl, right, ldr, out, ldo, scale, (int32_t)len,
                                                     (int32_t)rows, (int32_t)cols, 0, 0},
                                       cu, st));
  const int64_t head = q.splits == 1 ? tg::head_rows(rows, cols, len, cu) : rows;
  if (head == rows) return run_gradient(q, left, ldl, right, ldr, rows, cols, len, out, ldo, scale, part, st);
  TG_TRY(run_gradient(tg::plan_product(head, cols, len, 1, cu), left, ldl, right, ldr, head, cols, len, out, ldo,
                      scale, nullptr, st));
  return run_gradient(tg::plan_product(rows - head, cols, len, 1, cu), left + head * ldl, ldl, right, ldr, rows - head,
                      cols, len, out + head * ldo, ldo, scale, nullptr, st);
}

tile_gemm_status_t run_glu_backward(tile_gemm_t h, const void* A, const void* B, const void* dC, void* dA,
                                    void* dB, int64_t M, int64_t N, int64_t K, const tile_gemm_strides_t* s,
                                    const tile_gemm_strides_t* g, const float* bias, float* dbias, int gate,
                                    void* workspace, int64_t ws_bytes, void* stream) {
  if (!h) return fail(TILE_GEMM_ERR_NULL_ARG, "handle: NULL");
  tg::GluGradPlan p;
  TG_TRY(check_glu_backward(A, B, dC, dA, dB, M, N, K, s, g, bias, dbias, gate, workspace, ws_bytes,
                            h->cu_count, &p));
  TG_TRY(check_device(h));
  const hipStream_t st = static_cast<hipStream_t>(stream);
  if (M == 0 || N == 0) {  // empty sums
    if (dA && M) TG_LAUNCH(tg::launch_zero(dA, M, 2 * K, 2 * g->a_m, st));
    if (dB && N) TG_LAUNCH(tg::launch_zero(dB, N, 2 * K, 2 * g->b_n, st));
    if (dbias && N) TG_LAUNCH(tg::launch_zero(dbias, 1, 4 * N, 4 * N, st));
    return TILE_GEMM_OK;
  }
  char* ws = static_cast<char*>(workspace);
  uint16_t* z = dA ? reinterpret_cast<uint16_t*>(ws + p.off_z) : nullptr;
  uint16_t* zt = dB ? reinterpret_cast<uint16_t*>(ws + p.off_zt) : nullptr;
  float* part = reinterpret_cast<float*>(ws + p.off_part);
  tg::TrainArgs a{};
  a.A = static_cast<const uint16_t*>(A);
  a.B = static_cast<const uint16_t*>(B);
  a.M = (int32_t)M;
  a.N = (int32_t)N;
  a.K = (int32_t)K;
  a.lda = row_stride(M, s->a_m, K);
  a.ldb = s->b_n;
  a.bias = bias;
  a.glu_half = (int32_t)(N / 2);
  a.Z = z;
  a.ldz = p.ldz;
  a.Zt = zt;
  a.ldzt = p.ldzt;
  a.dC = static_cast<const uint16_t*>(dC);
  a.lddc = g->c_m;
  a.dbias_part = dbias ? reinterpret_cast<float*>(ws + p.off_bias) : nullptr;
  a.gate = gate;
  log_product(h, "run_glu_backward", M, N, K, p.z);
  TG_LAUNCH(launch_product(p.z, tg::kStoreGluGrad, a, st));
  if (dbias) TG_LAUNCH(tg::launch_add_rows(a.dbias_part, p.bias_rows, N, dbias, st));
  const tg::OuterArgs outer{zt, p.ldzt, a.A, a.lda, static_cast<uint16_t*>(dB), g->b_n, nullptr, (int32_t)M,
                            (int32_t)N, (int32_t)K, 0, 0};
  const bool pair = dA && dB && pairs(p.dx, M, N, K);
  if (dA)
    TG_TRY(run_gradient(p.dx, z, p.ldz, a.B, a.ldb, M, K, N, static_cast<uint16_t*>(dA), g->a_m, nullptr, part, st,
                        pair ? &outer : nullptr, h->cu_count));
  if (dB && !pair)
    TG_TRY(run_weight_gradient(p.dw, zt, p.ldzt, a.A, a.lda, N, K, M, static_cast<uint16_t*>(dB), g->b_n, nullptr,
                               part, h->cu_count, st));
  return TILE_GEMM_OK;
}

tile_gemm_status_t run_xent(tile_gemm_t h, const void* A, const void* B, const void* target, float* loss,
                            float* lse, int64_t M, int64_t N, int64_t K, const tile_gemm_strides_t* s,
                            const tile_gemm_xent_t* o, void* workspace, int64_t ws_bytes, void* stream) {
  if (!h) return fail(TILE_GEMM_ERR_NULL_ARG, "handle: NULL");
  tg::XentPlan p;
  TG_TRY(check_xent(A, B, target, loss, lse, M, N, K, s, o, workspace, ws_bytes, h->cu_count, &p));
  TG_TRY(check_device(h));
  if (M == 0) return TILE_GEMM_OK;
  const hipStream_t st = static_cast<hipStream_t>(stream);
  char* ws = static_cast<char*>(workspace);
  const bool smooth = o->label_smoothing > 0.0f;
  tg::TrainArgs a{};
  a.A = static_cast<const uint16_t*>(A);
  a.B = static_cast<const uint16_t*>(B);
  a.M = (int32_t)M;
  a.K = (int32_t)K;
  a.lda = row_stride(M, s->a_m, K);
  a.ldb = s->b_n;
  a.target = target;
  a.target64 = o->target_type == TILE_GEMM_INDEX_I64;
  a.part = reinterpret_cast<float2*>(ws + p.off_part);
  a.part_sum = smooth ? reinterpret_cast<float*>(ws + p.off_sum) : nullptr;
  a.hit = reinterpret_cast<float*>(ws + p.off_hit);
  a.N = (int32_t)p.head;
  log_product(h, "run_xent", M, p.head, K, p.l.z);
  TG_LAUNCH(launch_product(p.l.z, tg::kStoreStats, a, st));
  if (p.head < N) {
    tg::TrainArgs b = a;
    b.N = (int32_t)(N - p.head);
    b.B += p.head * b.ldb;
    b.first = (int32_t)p.head;
    b.part += (p.segs - p.rest_segs) * M;
    if (smooth) b.part_sum += (p.segs - p.rest_segs) * M;
    log_product(h, "run_xent", M, N - p.head, K, p.rest.z);
    TG_LAUNCH(launch_product(p.rest.z, tg::kStoreStats, b, st));
  }
  tg::FinishArgs f{a.part,    a.part_sum, a.hit, target, a.target64, o->ignore_index, (int32_t)M,
                   (int32_t)p.segs, N, o->label_smoothing, o->z_loss, loss, lse};
  return hip_status(tg::launch_xent_finish(f, st));
}

tile_gemm_status_t run_xent_backward(tile_gemm_t h, const void* A, const void* B, const void* target,
                                     const float* lse, const float* dloss, void* dA, void* dB, int64_t M,
                                     int64_t N, int64_t K, const tile_gemm_strides_t* s,
                                     const tile_gemm_strides_t* g, const tile_gemm_xent_t* o, void* workspace,
                                     int64_t ws_bytes, void* stream) {
  if (!h) return fail(TILE_GEMM_ERR_NULL_ARG, "handle: NULL");
  tg::XentGradPlan p;
  const int cu = h->cu_count;
  TG_TRY(check_xent_backward(A, B, target, lse, dloss, dA, dB, M, N, K, s, g, o, workspace, ws_bytes, cu, &p));
  TG_TRY(check_device(h));
  const hipStream_t st = static_cast<hipStream_t>(stream);
  if (M == 0) return dB ? hip_status(tg::launch_zero(dB, N, 2 * K, 2 * g->b_n, st)) : TILE_GEMM_OK;
  char* ws = static_cast<char*>(workspace);
  tg::XentRow* rows = reinterpret_cast<tg::XentRow*>(ws + p.off_rows);
  float* scale = reinterpret_cast<float*>(ws + p.off_scale);
  float* dx_part = reinterpret_cast<float*>(ws + p.off_dx);
  const int target64 = o->target_type == TILE_GEMM_INDEX_I64;
  // The stream kernel's waves can form the row constants of up to 64 rows
  // themselves. Each tile then costs about 0.7 us more and the launch of
  // xent_rows_kernel 3 to 5 us: worth it up to two tiles a workgroup (24 rows,
  // 32000 x 4096 231 to 225 us; 50 rows, 131072 x 512, eight tiles, 160 to 163).
  auto streams = [&](int64_t cols) {
    const tg::TrainProduct z = tg::plan_forward(M, cols, K, cu).z;
    return z.tile >= tg::kNumTrainTiles && (int64_t)z.map.tiles_m * z.map.tiles_n <= 2 * cu;
  };
  const bool few = M <= 64 && streams(p.piece) && streams(N - (p.n_pieces - 1) * p.piece);
  if (!few)
    TG_LAUNCH(tg::launch_xent_rows(
        tg::RowsArgs{target, target64, o->ignore_index, (int32_t)M, N, lse, dloss, o->z_loss, rows, scale}, st));
  const int64_t part_ld = tg::ceil_div(K, 4) * 4;
  int slot = 0;
  for (int64_t v = 0; v < N; v += p.piece) {
    const int64_t cols = N - v < p.piece ? N - v : p.piece;
    const uint16_t* w = static_cast<const uint16_t*>(B) + v * s->b_n;
    tg::TrainArgs a{};
    a.A = static_cast<const uint16_t*>(A);
    a.B = w;
    a.M = (int32_t)M;
    a.N = (int32_t)cols;
    a.K = (int32_t)K;
    a.lda = row_stride(M, s->a_m, K);
    a.ldb = s->b_n;
    if (few) {
      a.target = target;
      a.target64 = target64;
      a.lse = lse;
      a.dloss = dloss;
      a.ignore = o->ignore_index;
      a.vocab = N;
      a.z_loss = o->z_loss;
      a.row_scale = scale;
    } else {
      a.rows = rows;
    }
    a.first = (int32_t)v;
    a.smooth = o->label_smoothing / (float)N;
    a.keep = 1.0f - o->label_smoothing;
    a.Z = dA ? reinterpret_cast<uint16_t*>(ws + p.off_z) : nullptr;
    a.ldz = p.ldz;
    a.Zt = dB ? reinterpret_cast<uint16_t*>(ws + p.off_zt) : nullptr;
    a.ldzt = p.ldzt;
    const int64_t head = few ? cols : tg::head_logits(M, cols, K, cu);
    for (int64_t c = 0; c < cols; c += head) {
      tg::TrainArgs b = a;
      b.N = (int32_t)(c ? cols - head : head);
      b.B += c * b.ldb;
      b.first += (int32_t)c;
      if (b.Z) b.Z += c;
      if (b.Zt) b.Zt += c * b.ldzt;
      const tg::TrainProduct l = tg::plan_forward(M, b.N, K, cu).z;
      log_product(h, "run_xent_backward", M, b.N, K, l);
      TG_LAUNCH(launch_product(l, tg::kStoreXentGrad, b, st));
      if (c) break;
    }
    const tg::TrainProduct q = tg::plan_xent_dx(M, K, cols, cu);
    uint16_t* dw = dB ? static_cast<uint16_t*>(dB) + v * g->b_n : nullptr;
    const tg::OuterArgs outer{a.Zt,  p.ldzt, a.A, a.lda, dw, g->b_n, scale, (int32_t)M, (int32_t)cols, (int32_t)K,
                              0, 0};
    const bool pair = dA && dB && pairs(q, M, cols, K);
    if (dA) {
      if (p.slots == 0) {
        TG_TRY(run_gradient(q, a.Z, p.ldz, w, s->b_n, M, K, cols, static_cast<uint16_t*>(dA), g->a_m, scale,
                            nullptr, st, pair ? &outer : nullptr, cu));
      } else {
        tg::TrainArgs d{};
        d.A = a.Z;
        d.B = w;
        d.M = (int32_t)M;
        d.N = (int32_t)K;
        d.K = (int32_t)cols;
        d.lda = p.ldz;
        d.ldb = s->b_n;
        d.C = dx_part + slot * M * part_ld;
        d.ldc = part_ld;
        d.part_stride = M * part_ld;
        TG_LAUNCH(launch_gradient(q, d, false, pair ? &outer : nullptr, cu, st));
        slot += q.splits;
      }
    }
    if (dB && !pair)
      TG_TRY(run_weight_gradient(tg::plan_xent_dw(M, K, cols, cu), a.Zt, p.ldzt, a.A, a.lda, cols, K, M,
                                 dw, g->b_n, scale,
                                 reinterpret_cast<float*>(ws + p.off_dw), cu, st));
  }
  if (dA && p.slots)
    TG_LAUNCH(tg::launch_add_parts(tg::AddArgs{dx_part, M * part_ld, p.slots, (int32_t)M, (int32_t)K, part_ld,
                                               scale, static_cast<uint16_t*>(dA), g->a_m},
                                   st));
  return TILE_GEMM_OK;
}

int handle_cus(tile_gemm_t h) { return h ? h->cu_count : kDefaultCus; }

}  // namespace

extern "C" {

tile_gemm_status_t tile_gemm_run_glu(tile_gemm_t h, const void* A, const void* B, void* C, int64_t M,
                                     int64_t N, int64_t K, const tile_gemm_strides_t* strides,
                                     tile_gemm_dtype_t dtype, const float* bias, tile_gemm_gate_t gate,
                                     void* stream) {
  g_detail[0] = '\0';
  TG_TRY(check_gate((int)gate));
  if (gate == TILE_GEMM_GATE_SILU && (!strides || K <= 0 || b_is_row_major(strides, N)))
    return run_impl(h, A, B, C, M, N, K, strides, dtype, stream, nullptr, 0, bias, TILE_GEMM_ACT_SWIGLU);
  return run_glu(h, A, B, C, M, N, K, strides, (int)dtype, bias, (int)gate, stream);
}

tile_gemm_status_t tile_gemm_run_glu_backward(tile_gemm_t h, const void* A, const void* B, const void* dC,
                                              void* dA, void* dB, int64_t M, int64_t N, int64_t K,
                                              const tile_gemm_strides_t* strides,
                                              const tile_gemm_strides_t* grad_strides, const float* bias,
                                              float* dbias, tile_gemm_gate_t gate, void* workspace,
                                              int64_t workspace_bytes, void* stream) {
  return run_glu_backward(h, A, B, dC, dA, dB, M, N, K, strides, grad_strides, bias, dbias, (int)gate,
                          workspace, workspace_bytes, stream);
}

tile_gemm_status_t tile_gemm_glu_backward_workspace(tile_gemm_t h, int64_t M, int64_t N, int64_t K,
                                                    int64_t* bytes) {
  if (!bytes) return fail(TILE_GEMM_ERR_NULL_ARG, "bytes: NULL");
  TG_TRY(check_train_shape(M, N, K, kTrainMaxRows));
  *bytes = tg::plan_glu_grad(M, N, K, true, true, true, handle_cus(h)).bytes;
  return TILE_GEMM_OK;
}

tile_gemm_status_t tile_gemm_run_xent(tile_gemm_t h, const void* A, const void* B, const void* target,
                                      float* loss, float* lse, int64_t M, int64_t N, int64_t K,
                                      const tile_gemm_strides_t* strides, const tile_gemm_xent_t* options,
                                      void* workspace, int64_t workspace_bytes, void* stream) {
  return run_xent(h, A, B, target, loss, lse, M, N, K, strides, options, workspace, workspace_bytes, stream);
}

tile_gemm_status_t tile_gemm_xent_workspace(tile_gemm_t h, int64_t M, int64_t N, int64_t K,
                                            const tile_gemm_xent_t* options, int64_t* bytes) {
  if (!bytes || !options) return fail(TILE_GEMM_ERR_NULL_ARG, "bytes or options: NULL");
  TG_TRY(check_train_shape(M, N, K, kMaxDim));
  *bytes = tg::plan_xent(M, N, K, options->label_smoothing > 0.0f, handle_cus(h)).bytes;
  return TILE_GEMM_OK;
}

tile_gemm_status_t tile_gemm_run_xent_backward(tile_gemm_t h, const void* A, const void* B,
                                               const void* target, const float* lse, const float* dloss,
                                               void* dA, void* dB, int64_t M, int64_t N, int64_t K,
                                               const tile_gemm_strides_t* strides,
                                               const tile_gemm_strides_t* grad_strides,
                                               const tile_gemm_xent_t* options, void* workspace,
                                               int64_t workspace_bytes, void* stream) {
  return run_xent_backward(h, A, B, target, lse, dloss, dA, dB, M, N, K, strides, grad_strides, options,
                           workspace, workspace_bytes, stream);
}

tile_gemm_status_t tile_gemm_xent_backward_workspace(tile_gemm_t h, int64_t M, int64_t N, int64_t K,
                                                     const tile_gemm_strides_t* strides,
                                                     const tile_gemm_xent_t* options, int64_t* bytes) {
  if (!bytes || !options || !strides) return fail(TILE_GEMM_ERR_NULL_ARG, "bytes, strides or options: NULL");
  TG_TRY(check_train_shape(M, N, K, kMaxDim));
  TG_TRY(check_col_major("B", strides, K));
  *bytes = tg::plan_xent_grad(M, N, K, strides->b_n, options->piece, true, true, handle_cus(h)).bytes;
  return TILE_GEMM_OK;
}

}  // extern "C"
