// train_abi_checks.cpp -- drives the host-only half of the gated block's and
// the cross entropy's entry points (argument checks, planners, workspace
// layout; csrc/train_abi.hpp) over ordinary, edge and hostile inputs, built
// with g++ under the address and undefined-behaviour sanitizers by
// tests/test_train_sanitize.py. The driver checks that every status is a
// defined one, that an accepted call's plan fits its kernels' 32-bit counts
// and that a workspace's regions lie inside it, in order.
#include <stdint.h>
#include <stdio.h>
#include <stdlib.h>

#include <initializer_list>

#include "train_abi.hpp"

namespace {

long g_calls = 0;

void require(bool ok, const char* what, long long a = 0, long long b = 0, long long c = 0) {
  if (!ok) {
    fprintf(stderr, "FAILED: %s (%lld, %lld, %lld)\n", what, a, b, c);
    exit(1);
  }
}

bool known(tile_gemm_status_t s) { return s >= TILE_GEMM_OK && s <= TILE_GEMM_ERR_WORKSPACE; }

const int64_t kDims[] = {0, 1, 2, 16, 17, 31, 32, 64, 65, 128, 129, 256, 1000, 4096, 8192, 50257, 131072,
                         ((int64_t)1 << 22) - 16, ((int64_t)1 << 22) - 1, (int64_t)1 << 22,
                         ((int64_t)1 << 31) - 1, (int64_t)1 << 31, -1, INT64_MAX, INT64_MIN};
const int64_t kStrides[] = {0, 1, -1, 64, 8192, ((int64_t)1 << 22) - 8, (int64_t)1 << 22, ((int64_t)1 << 31) - 16,
                            (int64_t)1 << 40, INT64_MAX, INT64_MIN};

void check_product(const tg::TrainProduct& q, int64_t M, int64_t N, int64_t K) {
  require(q.splits >= 1 && q.grid >= 1 && q.grid < ((int64_t)1 << 31), "product: grid", q.splits, q.grid);
  require((int64_t)q.map.tiles_m * q.map.tiles_n * q.splits < ((int64_t)1 << 31), "product: tiles", M, N, K);
  require(q.splits == 1 || (q.k_per % 64 == 0 && q.k_per * (q.splits - 1) < K && q.k_per * q.splits >= K),
          "product: parts cover K", q.k_per, q.splits, K);
}

void plans() {
  for (int cu : {1, 8, 224, 256})
    for (int64_t M : kDims)
      for (int64_t N : kDims)
        for (int64_t K : kDims) {
          for (int kind = -1; kind < 4; ++kind) {
            tile_gemm_plan_t p;
            const tile_gemm_status_t s = tile_gemm_plan_train(M, N, K, (tile_gemm_train_product_t)kind, cu, &p);
            ++g_calls;
            require(known(s), "plan: unknown status", M, N, K);
            if (s == TILE_GEMM_OK)
              require(p.tiles == (int64_t)p.tiles_m * p.tiles_n && p.grid >= 1 && p.grid <= p.tiles * p.k_split,
                      "plan: grid", M, N, K);
          }
          if (check_train_shape(M, N, K, kMaxDim) != TILE_GEMM_OK || M == 0 || N == 0) continue;
          const tg::XentPlan x = tg::plan_xent(M, N, K, true, cu);
          ++g_calls;
          require(x.head >= 1 && x.head <= N && (x.head == N || x.head % 32 == 0), "loss: first launch", M, N, K);
          check_product(x.l.z, M, x.head, K);
          if (x.head < N) check_product(x.rest.z, M, N - x.head, K);
          require(x.off_part == 0 && x.off_sum >= tg::bytes_of(x.segs, M * 8) && x.off_hit >= x.off_sum + x.segs * M * 4 &&
                      x.bytes >= x.off_hit + M * 4,
                  "loss: workspace regions", M, N, K);
          for (int64_t piece : {(int64_t)0, (int64_t)1, (int64_t)300, INT64_MAX}) {
            const int64_t ld = (K + 7) / 8 * 8;
            if (ld >= kTrainMaxRows) continue;
            const tg::XentGradPlan g = tg::plan_xent_grad(M, N, K, ld, piece, true, true, cu);
            ++g_calls;
            require(g.piece >= 1 && g.piece <= N && g.n_pieces == tg::ceil_div(N, g.piece), "pieces", M, N, K);
            require(g.piece * ld * 2 < ((int64_t)1 << 32), "a piece of W fits 32-bit offsets", M, N, K);
            require(256 * g.ldz * 2 < ((int64_t)1 << 31), "256 rows of G fit 32-bit offsets", M, N, K);
            require(g.off_rows == 0 && g.off_scale >= M * 16 && g.off_z >= g.off_scale + 4 &&
                        g.off_dx >= g.off_z + tg::bytes_of(M, g.ldz * 2) &&
                        g.off_zt >= g.off_dx + tg::bytes_of(g.slots, tg::slot_bytes(M, K)) &&
                        g.off_dw >= g.off_zt + tg::bytes_of(g.piece, g.ldzt * 2) && g.bytes >= g.off_dw,
                    "gradient: workspace regions", M, N, K);
          }
          if (N < kTrainMaxRows) {
            const tg::GluGradPlan g = tg::plan_glu_grad(M, N, K, true, true, true, cu);
            ++g_calls;
            check_product(g.z, M, N, K);
            check_product(g.dx, M, K, N);
            check_product(g.dw, N, K, M);
            require(g.off_zt >= tg::bytes_of(M, g.ldz * 2) && g.off_part >= g.off_zt + tg::bytes_of(N, g.ldzt * 2) &&
                        g.bytes >= g.off_bias + tg::bytes_of(g.bias_rows, N * 4),
                    "gated: workspace regions", M, N, K);
          }
        }
}

void checks() {
  unsigned r = 12345;
  auto next = [&](int n) { return (int)((r = r * 1664525u + 1013904223u) >> 8) % n; };
  auto dim = [&] { return kDims[next(sizeof kDims / sizeof *kDims)]; };
  auto stride = [&](int64_t good) { return next(3) ? good : kStrides[next(sizeof kStrides / sizeof *kStrides)]; };
  auto ptr = [&](int i) -> const void* {
    switch (next(12)) {
      case 0: return nullptr;
      case 1: return (const void*)(uintptr_t)(((uintptr_t)i << 40) + 8);
      case 2: return (const void*)(UINTPTR_MAX - 255);
      case 3: return (const void*)((uintptr_t)(i + 1) << 40);
      default: return (const void*)((uintptr_t)i << 44);
    }
  };
  for (int i = 0; i < 400000; ++i) {
    const int64_t M = dim(), N = dim(), K = dim();
    const int64_t ld = K > 0 && K < ((int64_t)1 << 40) ? (K + 7) / 8 * 8 : 64;
    const tile_gemm_strides_t s{stride(ld), stride(1), stride(1), stride(ld), 0, 0};
    const tile_gemm_strides_t g{stride(ld), stride(1), stride(1), stride(ld), stride(ld), stride(1)};
    const tile_gemm_xent_t o{stride(-100), next(9) ? 0.1f : -1.0f, next(9) ? 0.0f : 1.0f / 0.0f, stride(0),
                             next(9) ? 1 : 7};
    const int64_t ws = next(4) ? INT64_MAX : stride(0);
    require(known(tile_gemm_check_glu_backward(ptr(1), ptr(2), ptr(3), ptr(4), ptr(5), M, N, K, next(20) ? &s : nullptr,
                                               next(20) ? &g : nullptr, (const float*)ptr(6), (const float*)ptr(7),
                                               (tile_gemm_gate_t)(next(7) - 1), ptr(8), ws)),
            "glu status", M, N, K);
    require(known(tile_gemm_check_xent(ptr(1), ptr(2), ptr(3), (const float*)ptr(4), (const float*)ptr(5), M, N, K,
                                       next(20) ? &s : nullptr, next(20) ? &o : nullptr, ptr(8), ws)),
            "xent status", M, N, K);
    require(known(tile_gemm_check_xent_backward(ptr(1), ptr(2), ptr(3), (const float*)ptr(4), (const float*)ptr(5),
                                                ptr(6), ptr(7), M, N, K, next(20) ? &s : nullptr,
                                                next(20) ? &g : nullptr, next(20) ? &o : nullptr, ptr(8), ws)),
            "xent backward status", M, N, K);
    g_calls += 3;
  }
}

}  // namespace

int main() {
  plans();
  checks();
  printf("ok %ld calls\n", g_calls);
  return 0;
}
