// block_abi_checks.cpp -- drives the host-only half of the E4M3 products with
// block scales, of the quantization, of the routing and of the experts' sums
// (argument checks, plans, workspace sizes; csrc/block_abi.hpp) over ordinary,
// edge and hostile inputs, built with g++ under the address and
// undefined-behaviour sanitizers by tests/test_block_sanitize.py. The driver
// checks that every status is a defined one, that an accepted product's plan
// covers the output and fits the kernels' 32-bit counts and offsets, and that
// the places' chunks cover their entries.
#include <stdint.h>
#include <stdio.h>
#include <stdlib.h>

#include <initializer_list>

#include "block_abi.hpp"

namespace {

long g_calls = 0;

void require(bool ok, const char* what, long long a = 0, long long b = 0, long long c = 0) {
  if (!ok) {
    fprintf(stderr, "FAILED: %s (%lld, %lld, %lld)\n", what, a, b, c);
    exit(1);
  }
}

bool known(tile_gemm_status_t s) { return s >= TILE_GEMM_OK && s <= TILE_GEMM_ERR_WORKSPACE; }

const int64_t k31 = (int64_t)1 << 31, k22 = (int64_t)1 << 22;
const int64_t kDims[] = {0, 1, 2, 16, 17, 31, 32, 48, 64, 65, 128, 129, 256, 1000, 1024, 4096, 8192, 50257, 131072,
                         k22 - 16, k22 - 1, k22, k31 - 1, k31, -1, INT64_MAX, INT64_MIN};
const int64_t kStrides[] = {0, 1, -1, 64, 8192, k22 - 16, k22, k31 - 16, (int64_t)1 << 40, INT64_MAX, INT64_MIN};

void plans() {
  for (int cu : {1, 8, 224, 256})
    for (int64_t M : kDims)
      for (int64_t N : kDims)
        for (int64_t K : kDims)
          for (int64_t E : {(int64_t)0, (int64_t)1, (int64_t)6, (int64_t)256, (int64_t)1024, (int64_t)1025, (int64_t)-1})
            for (int dtype = -1; dtype < 3; ++dtype) {
              tile_gemm_plan_t p;
              const tile_gemm_status_t s = tile_gemm_plan_fp8(M, N, K, E, (tile_gemm_dtype_t)dtype, cu, &p);
              ++g_calls;
              require(known(s), "plan: unknown status", M, N, K);
              if (s != TILE_GEMM_OK || M == 0 || N == 0) continue;
              require(p.config >= (dtype == TILE_GEMM_BF16_TO_F32 ? 1 : 0) && p.config < tg::kNumBlockConfigs,
                      "plan: configuration", p.config);
              require((int64_t)p.tiles_n * p.bn >= N && (int64_t)p.tiles_m * p.bm >= M, "plan: covers", M, N);
              require(p.tiles >= (int64_t)p.tiles_m * p.tiles_n && p.tiles < k31 && p.grid >= 1 && p.grid <= p.tiles,
                      "plan: tiles", p.tiles, p.grid);
              // rows of a tile from its first, as far apart as they may be
              require((int64_t)(p.bm > p.bn ? p.bm : p.bn) * (k22 - 1) < k31, "plan: 32-bit offsets", p.bm, p.bn);
              require(p.lds_bytes + (E ? tg::kExpertLds : 0) <= 160 * 1024, "plan: LDS", p.lds_bytes);
            }
}

void places() {
  for (int64_t T : kDims)
    for (int64_t k : kDims)
      for (int64_t E : kDims) {
        int64_t bytes = -1;
        const tile_gemm_status_t s = tile_gemm_place_workspace(T, k, E, &bytes);
        ++g_calls;
        require(known(s), "workspace: unknown status", T, k, E);
        if (s != TILE_GEMM_OK) continue;
        const PlacePlan p = plan_place(T * k, E);
        require(p.chunks >= 1 && p.chunks <= kPlaceMaxChunks && p.rounds >= 1, "places: chunks", p.chunks, p.rounds);
        require(p.chunks * p.rounds * kPlaceRound >= T * k && (p.chunks - 1) * p.rounds * kPlaceRound <= T * k,
                "places: cover the entries", T, k);
        require(bytes == (p.chunks > 1 ? p.chunks * E * 4 : 0), "places: workspace", bytes);
      }
  require(tile_gemm_place_workspace(1, 1, 1, nullptr) == TILE_GEMM_ERR_NULL_ARG, "workspace: null");
}

void checks() {
  unsigned r = 54321;
  auto next = [&](int n) { return (int)((r = r * 1664525u + 1013904223u) >> 8) % n; };
  auto dim = [&] { return kDims[next(sizeof kDims / sizeof *kDims)]; };
  auto small = [&] { return next(9) ? (int64_t)next(40) : dim(); };
  auto stride = [&](int64_t good) { return next(4) ? good : kStrides[next(sizeof kStrides / sizeof *kStrides)]; };
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
    const int64_t M = dim(), N = dim(), K = next(3) ? dim() : 16 * (int64_t)next(600), E = small();
    const bool sane = M >= 0 && M <= k22 && N >= 0 && N <= k22 && K >= 0 && K <= k22;
    const int64_t kb = sane ? (K + 127) / 128 : 1, ld = sane ? (K + 15) / 16 * 16 : 64, ldn = sane ? (N + 15) / 16 * 16 : 64;
    const tile_gemm_fp8_strides_t s{stride(ld), stride(ld), stride(ldn), stride(sane ? M : 1),
                                    stride(kb), stride(sane ? N * ld : 1), stride(sane ? kb * ((N + 127) / 128) : 1)};
    const int dtype = next(4) - 1, act = next(9) - 1;
    require(known(tile_gemm_check_fp8(ptr(1), ptr(2), ptr(3), M, N, K, next(20) ? &s : nullptr, (const float*)ptr(4),
                                      (const float*)ptr(5), (tile_gemm_dtype_t)dtype, (const float*)ptr(6),
                                      (tile_gemm_act_t)act)),
            "fp8 status", M, N, K);
    const tile_gemm_status_t e = tile_gemm_check_fp8_experts(
        ptr(1), ptr(2), ptr(3), M, N, K, E, (const int32_t*)ptr(6), next(20) ? &s : nullptr, (const float*)ptr(4),
        (const float*)ptr(5), (tile_gemm_dtype_t)dtype);
    require(known(e), "experts status", M, N, E);
    if (e == TILE_GEMM_OK) require(E >= 1 && E <= tg::kBlockMaxGroups, "experts: number", E);
    require(known(tile_gemm_check_quantize(ptr(1), ptr(2), (const float*)ptr(3), M, K, stride(next(2) ? ld : 2 * ld),
                                           stride(ld), stride(next(2) ? kb : sane ? M : 1),
                                           (tile_gemm_quant_t)(next(5) - 1), (tile_gemm_gate_t)(next(7) - 1),
                                           next(2) ? (const int32_t*)ptr(4) : nullptr, dim())),
            "quantize status", M, K);
    const tile_gemm_route_t o{next(4) - 1, next(4) - 1, (int32_t)small(), (int32_t)small(), next(4), next(2),
                              next(9) ? 1.0f : 1.0f / 0.0f};
    const int64_t T = dim(), X = small(), k = small();
    require(known(tile_gemm_check_route(ptr(1), (const float*)ptr(2), (const int32_t*)ptr(3), (const float*)ptr(4), T, X,
                                        k, stride(X), next(20) ? &o : nullptr)),
            "route status", T, X, k);
    require(known(tile_gemm_check_route_backward(ptr(1), (const int32_t*)ptr(2), (const float*)ptr(3), ptr(4), T, X, k,
                                                 stride(X), stride(X), next(20) ? &o : nullptr)),
            "route backward status", T, X, k);
    require(known(tile_gemm_check_place((const int32_t*)ptr(1), T, k, dim(), X, (const int32_t*)ptr(2),
                                        (const int32_t*)ptr(3), (const int32_t*)ptr(4), ptr(5),
                                        next(4) ? INT64_MAX : stride(0))),
            "place status", T, X, k);
    require(known(tile_gemm_check_combine(ptr(1), (const int32_t*)ptr(2), (const float*)ptr(3), ptr(4), M, N, k, dim(),
                                          stride(ldn), stride(ldn), (tile_gemm_dtype_t)dtype)),
            "combine status", M, N, k);
    g_calls += 7;
  }
}

}  // namespace

int main() {
  plans();
  places();
  checks();
  printf("ok %ld calls\n", g_calls);
  return 0;
}
