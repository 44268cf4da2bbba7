// train_plan_checks.cpp -- the planners of the gated block and of the cross
// entropy (csrc/train_plan.hpp) over contractions of no and few values, built
// with g++ under the address and undefined-behaviour sanitizers by
// tests/test_train_plan_sanitize.py. A gated product over K = 0 (the block of
// its biases alone) has a plan like any other, one whose part of K is not 0.
#include <stdint.h>
#include <stdio.h>
#include <stdlib.h>

#include "train_plan.hpp"

namespace {

void require(bool ok, const char* what, long long a, long long b, long long c) {
  if (!ok) {
    fprintf(stderr, "FAILED: %s (%lld, %lld, %lld)\n", what, a, b, c);
    exit(1);
  }
}

}  // namespace

int main() {
  long calls = 0;
  for (int cu : {1, 224, 256})
    for (int64_t M : {1, 5, 16, 300, 8192, 1 << 20})
      for (int64_t N : {16, 48, 64, 528, 7168, 131072})
        for (int64_t K : {0, 1, 7, 63, 64, 65, 255, 256, 257, 513}) {
          for (int splits : {1, 2, tg::kMaxSplits})
            for (bool gated : {false, true}) {
              const tg::TrainProduct q = tg::plan_product(M, N, K, splits, cu, gated);
              require(q.splits >= 1 && q.splits <= splits && q.grid >= 1, "parts and workgroups", M, N, K);
              require(q.splits == 1 || (q.k_per * (q.splits - 1) < K && q.k_per * q.splits >= K), "parts cover K", M,
                      N, K);
              require(tg::train_plan(q).grid == q.grid, "launch plan", M, N, K);
              ++calls;
            }
          const tg::ForwardPlan f = tg::plan_forward(M, N, K, cu, true);
          require(f.z.splits == 1 && f.z.grid >= 1 && f.seg_cols >= 32, "forward", M, N, K);
          require(tg::head_rows(N, M, K, cu) >= 1 && tg::head_logits(M, N, K, cu) >= 1, "first launch", M, N, K);
          ++calls;
        }
  printf("ok %ld calls\n", calls);
  return 0;
}
