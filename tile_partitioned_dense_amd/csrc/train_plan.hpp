// train_plan.hpp -- launch geometry and workspace layout of the gated block's
// backward pass and of the cross entropy of a projection. Host only, no HIP
// dependency, pure functions of the shape and the compute-unit count.
#pragma once

#include <initializer_list>
#include "plan.hpp"

namespace tg {

// The tile kernels these operators are compiled for: 256-row tiles of the
// 64-deep one-wave-per-SIMD kernel in four widths (which one leaves the fewest
// compute units idle depends on the output) and 128 x 128 tiles of the 32-deep
// kernel, two of which share a compute unit, for shapes with few tiles.
//
// A round of tiles, one on every compute unit (two of the small ones), was
// measured to take us_k microseconds per 1000 values of K and us_tile for the
// rest (first loads, last slabs, store); with few compute units busy the chip
// clocks higher and us_k falls by about 15%. us_k1: a small tile alone on its
// compute unit. `gated`: compiled with the gated block's stores too. us_tile is
// that of the loss's stores for every product: the gated backward's store takes
// longer (1501 x 5488 over 4104, one round of 210 tiles of 256 x 160: 62 us by
// these figures, 87 to 94 under the profiler).
struct TrainTile {
  int bm, bn, wm, wn;
  double us_k, us_tile, us_k1;
  int occ;
  bool gated;
};
constexpr int kNumTrainTiles = 5;
constexpr int kSmallTile = 4;
constexpr TrainTile kTrainTiles[kNumTrainTiles] = {
    {256, 256, 2, 2, 19.5, 10.0, 19.5, 1, true}, {256, 224, 2, 2, 17.6, 9.5, 17.6, 1, true},
    {256, 192, 2, 2, 15.6, 9.0, 15.6, 1, false}, {256, 160, 2, 2, 13.3, 8.5, 13.3, 1, true},
    {128, 128, 2, 2, 17.5, 5.0, 12.0, 2, true},
};
// The stream kernel's configurations here, in the same terms: for few rows or
// few tiles, where a tile's K loop is latency and long stages shared by many
// waves win. (Four waves on each 32-column block instead of the two of the
// plain configurations: 64 x 64 tiles 7.2 to 4.2 us per 1000 of K, 32 x 64
// tiles 3.9 to 3.3.) The 32 x 32 tiles are for one round of them: the loss of
// 24 rows, 8191 x 1024 10.5 to 9.6 us, 8191 x 4096 19.7 to 17.6, the gated block
// of 27 rows, 6000 x 3696 16.0 to 13.3; in two rounds (12000 x 1024, the loss)
// they take 14.2 for the 10.9 of 32 x 64.
struct TrainStream {
  int bm, bn, sb, stages, ks;
  double us_k, us_tile;
};
constexpr int kNumTrainStreams = 4;
constexpr TrainStream kTrainStreams[kNumTrainStreams] = {
    {32, 64, 512, 3, 4, 3.3, 2.0},
    {64, 128, 256, 3, 2, 8.0, 2.5},
    {64, 64, 512, 2, 4, 4.2, 2.5},
    {32, 32, 512, 3, 4, 2.4, 2.0},
};

// What a product is turned into (train_epilogue.hpp; a gradient's bf16 result
// or the fp32 partial results of its parts are both kEpiPartial there).
enum TrainStore { kStoreStats = 0, kStoreXentGrad, kStoreBf16, kStoreParts, kStoreGluGrad, kStoreGlu };

// The compiled kernels: on the tiles above or the stream kernel's
// configurations (tile kNumTrainTiles + configuration), gate < 0 where it is an argument.
// Logits and pre-activations take W as it is stored (column-major B) and the
// gated forward product either layout; gradients contract over W's rows (dx)
// or over the tokens (dW), where the second operand is row-major.
struct TrainKernel {
  int store, tile, gate;
  bool bcol, bf16;
};
constexpr int kNumTrainKernels = 114;
struct TrainKernels {
  TrainKernel k[kNumTrainKernels] = {};
  int n = 0;
  constexpr void add(int store, int tile, int gate, bool bcol, bool bf16) {
    k[n].store = store;
    k[n].tile = tile;
    k[n].gate = gate;
    k[n].bcol = bcol;
    k[n].bf16 = bf16;
    ++n;
  }
  constexpr TrainKernels() {
    for (int t = 0; t < kNumTrainTiles; ++t) {
      add(kStoreStats, t, -1, true, true);
      add(kStoreXentGrad, t, -1, true, true);
      add(kStoreBf16, t, -1, false, true);
      add(kStoreParts, t, -1, false, false);
    }
    for (int c = kNumTrainTiles; c < kNumTrainTiles + kNumTrainStreams; ++c) {
      add(kStoreStats, c, -1, true, true);
      add(kStoreXentGrad, c, -1, true, true);
      add(kStoreGlu, c, -1, true, true);
      add(kStoreGlu, c, -1, true, false);
      add(kStoreGluGrad, c, -1, true, true);
    }
    for (int t = 0; t < kSmallTile; ++t) {
      if (!kTrainTiles[t].gated) continue;
      for (int g = 0; g < 5; ++g) add(kStoreGluGrad, t, g, true, true);
      for (int l = 0; l < 4; ++l)
        for (int g = (l & 1) ? 0 : 1; g < 5; ++g) add(kStoreGlu, t, g, l & 1, l & 2);
    }
    add(kStoreGluGrad, kSmallTile, -1, true, true);
    for (int l = 0; l < 4; ++l) add(kStoreGlu, kSmallTile, -1, l & 1, l & 2);
  }
};
constexpr TrainKernels kTrainKernels{};
static_assert(kTrainKernels.n == kNumTrainKernels, "the table is as long as it says");

// Index of a compiled kernel, -1 if there is none.
inline int train_kernel(int store, int tile, int gate, bool bcol, bool bf16) {
  for (int i = 0; i < kNumTrainKernels; ++i) {
    const TrainKernel& k = kTrainKernels.k[i];
    if (k.store == store && k.tile == tile && (k.gate < 0 || k.gate == gate) && k.bcol == bcol &&
        k.bf16 == bf16)
      return i;
  }
  return -1;
}

// A product cut into tiles and, for gradients whose output has few tiles but
// a long contraction (dx over the vocabulary, dW over the tokens), into
// `splits` parts of k_per along K whose fp32 results are added in a fixed
// order afterwards.
struct TrainProduct {
  int tile;
  int splits;
  int64_t k_per;
  TileMap map;
  int64_t grid;
};

// Microseconds a product takes, roughly: the rounds of its tiles, and the pass
// that adds the parts of K (the bytes it reads and writes at 4 TB/s and a
// launch). A row-major right operand (the gradients) takes two transposing
// LDS reads per fragment, measured 12% longer per value of K.
inline double rounds_us(int64_t tiles, int occ, double us_k, double us_k1, double us_tile, double k, int cu) {
  if (tiles <= cu) {
    const double busy = (double)tiles / cu;
    return k * 1e-3 * us_k1 * (0.85 + 0.15 * busy) + us_tile;
  }
  return (double)ceil_div(tiles, (int64_t)cu * occ) * (k * 1e-3 * us_k + us_tile);
}
inline double product_us(const TrainTile& t, int64_t M, int64_t N, int64_t k_per, int splits, bool row_major,
                         int cu) {
  const int64_t tiles = ceil_div(M, t.bm) * ceil_div(N, t.bn) * splits;
  const double f = row_major ? 1.12 : 1.0;
  double us = rounds_us(tiles, t.occ, f * t.us_k, f * t.us_k1, t.us_tile, (double)k_per, cu);
  if (splits > 1) us += 4.0 + (double)M * (double)N * (4.0 * splits + 2.0) / 4.0e6;
  return us;
}

inline TileMap tile_map(int64_t M, int64_t N, int bm, int bn) {
  TileMap m{};
  m.tiles_m = (int32_t)ceil_div(M, bm);
  m.tiles_n = (int32_t)ceil_div(N, bn);
  m.group_m = pick_group_m(m.tiles_m, m.tiles_n);
  m.xcds = kXcds;
  return m;
}

// max_splits > 1: a gradient.
inline TrainProduct plan_product(int64_t M, int64_t N, int64_t K, int max_splits, int cu,
                                 bool gated = false, double* us_out = nullptr) {
  TrainProduct best{};
  double best_us = 0.0;
  for (int c = 0; c < kNumTrainTiles; ++c) {
    const TrainTile& t = kTrainTiles[c];
    if (gated && !t.gated) continue;
    const int64_t tiles = ceil_div(M, t.bm) * ceil_div(N, t.bn);
    for (int s = 1; s <= max_splits; ++s) {
      const int64_t k_per = ceil_div(ceil_div(K, s), 64) * 64;
      // parts of at least 256 keep the load pipeline longer than its ramp; past
      // four rounds of tiles more parts even nothing out
      if (s > 1 && (k_per < 256 || tiles * (s - 1) >= 4 * (int64_t)cu * t.occ)) break;
      if (s > 1 && ceil_div(K, k_per) != s) continue;
      const double us = product_us(t, M, N, s == 1 ? K : k_per, s, max_splits > 1, cu);
      if (best_us == 0.0 || us < best_us * 0.999) {
        best_us = us;
        best.tile = c;
        best.splits = s;
        best.k_per = k_per;
      }
    }
  }
  if (us_out) *us_out = best_us;
  const TrainTile& t = kTrainTiles[best.tile];
  best.map = tile_map(M, N, t.bm, t.bn);
  best.grid = persistent_grid((int64_t)best.map.tiles_m * best.map.tiles_n * best.splits, cu * t.occ);
  return best;
}
constexpr int kMaxSplits = 64;

// A gradient's product with its workspace: `slots` fp32 partial results of
// M x N (0: the product writes its bf16 result itself).
inline int64_t slot_bytes(int64_t M, int64_t N) { return M * ceil_div(N, 4) * 16; }

// A product of two sizes, at most kManyBytes (more than any memory holds, and
// a sum of eight of them still fits): the sizes of a shape that no workspace
// can serve stay comparable.
constexpr int64_t kManyBytes = (int64_t)1 << 59;
inline int64_t bytes_of(int64_t n, int64_t each) {
  const __int128 b = (__int128)n * each;
  return b < kManyBytes ? (int64_t)b : kManyBytes;
}

// Bytes of one workspace region, and the running offset past it: regions
// start at multiples of 256 bytes.
inline int64_t region(int64_t& at, int64_t bytes) {
  const int64_t p = at;
  at += ceil_div(bytes, 256) * 256;
  return p;
}

// The product over W as it is stored (logits, gated pre-activations): a tile
// kernel or, with an even K, a configuration of the stream kernel, whichever
// is expected to be shorter; neither is shorter than the stream of W's bytes,
// which decides between them for few rows. `seg_cols`: the columns whose
// logits one wave joins; `row_groups`: the groups of a tile's rows whose
// column sums are stored apart.
struct ForwardPlan {
  TrainProduct z;
  int seg_cols, row_groups;
};

inline ForwardPlan plan_forward(int64_t M, int64_t N, int64_t K, int cu, bool gated = false,
                                double* us_out = nullptr) {
  ForwardPlan f{};
  double us = 0.0;
  f.z = plan_product(M, N, K, 1, cu, gated, &us);
  const TrainTile& t = kTrainTiles[f.z.tile];
  f.seg_cols = t.bn / t.wn;
  f.row_groups = t.wm;
  if (us_out) *us_out = us;
  if (K % 2 != 0) return f;
  const double bytes_us = (double)N * (double)K * 2.0 / 6.0e6;
  if (us < bytes_us) us = bytes_us;
  int best = -1;
  for (int c = 0; c < kNumTrainStreams; ++c) {
    const TrainStream& sc = kTrainStreams[c];
    const int64_t tiles = ceil_div(M, sc.bm) * ceil_div(N, sc.bn);
    double s = rounds_us(tiles, 1, sc.us_k, sc.us_k, sc.us_tile, (double)K, cu);
    if (s < bytes_us) s = bytes_us;
    // level with a tile kernel (both at the rate of W's bytes): the stream
    if (s < us || (best < 0 && s <= us)) {
      best = c;
      us = s;
    }
  }
  if (us_out) *us_out = us;
  if (best < 0) return f;
  const TrainStream& sc = kTrainStreams[best];
  f.z.tile = kNumTrainTiles + best;
  f.z.map = tile_map(M, N, sc.bm, sc.bn);
  f.z.grid = persistent_grid((int64_t)f.z.map.tiles_m * f.z.map.tiles_n, cu);
  f.z.splits = 1;
  f.seg_cols = 32;
  f.row_groups = sc.bm / 32;
  return f;
}

// Outputs of several rounds of tiles, the last one nearly empty, are cut in
// two launches: whole rounds of some tile, and what is left on a plan of its
// own (smaller tiles, more of the compute units). The axis of length N is cut,
// in steps of a tile's `step(t)`; `across(t)` tiles lie side by side over it;
// `plan(n, &us)` plans n of it. Returns the first launch's share; N where one
// launch is expected to be as fast. kLaunchUs: what the second launch costs.
constexpr double kLaunchUs = 4.0;
template <class Step, class Across, class Plan>
int64_t head_of(int64_t N, int cu, Step step, Across across, Plan plan) {
  double us = 0.0;
  if (plan(N, &us).tile >= kNumTrainTiles) return N;
  int64_t best = N;
  us *= 0.98;
  for (const TrainTile& t : kTrainTiles) {
    const int64_t side = across(t), slots = (int64_t)cu * t.occ;
    const int64_t rounds = side * ceil_div(N, (int64_t)step(t)) / slots;
    const int64_t n = rounds * slots / side * step(t);
    if (n <= 0 || n >= N) continue;
    double head = 0.0, rest = 0.0;
    plan(n, &head);
    plan(N - n, &rest);
    if (head + rest + kLaunchUs < us) {
      us = head + rest + kLaunchUs;
      best = n;
    }
  }
  return best;
}
// Columns of the logits M x N in their first launch.
inline int64_t head_logits(int64_t M, int64_t N, int64_t K, int cu) {
  return head_of(N, cu, [](const TrainTile& t) { return t.bn; },
                 [&](const TrainTile& t) { return ceil_div(M, t.bm); },
                 [&](int64_t n, double* us) { return plan_forward(M, n, K, cu, false, us).z; });
}
// Rows of the weight gradient N x K over M tokens in its first launch (no
// parts of the contraction in either).
inline int64_t head_rows(int64_t N, int64_t K, int64_t M, int cu) {
  return head_of(N, cu, [](const TrainTile& t) { return t.bm; },
                 [&](const TrainTile& t) { return ceil_div(K, t.bn); },
                 [&](int64_t n, double* us) { return plan_product(n, K, M, 1, cu, false, us); });
}

// A training product as a launch plan (log lines, introspection).
inline Plan train_plan(const TrainProduct& q) {
  Plan p{};
  p.variant = 1;
  p.config = q.tile;
  if (q.tile < kNumTrainTiles) {
    const TrainTile& t = kTrainTiles[q.tile];
    p.bm = t.bm;
    p.bn = t.bn;
    p.bk = t.bm == 256 ? 64 : 32;
    p.threads = t.wm * t.wn * 64;
    p.lds_bytes = (t.bm == 256 ? 2 : 4) * (t.bm + t.bn) * p.bk * 2;
  } else {
    const TrainStream& c = kTrainStreams[q.tile - kNumTrainTiles];
    p.bm = c.bm;
    p.bn = c.bn;
    p.bk = c.sb / 2;
    p.threads = c.bn / 32 * c.ks * 64;
    p.lds_bytes = c.stages * (c.bm + c.bn) * c.sb;
  }
  p.map = q.map;
  p.k_split = q.splits;
  p.tiles = (int64_t)q.map.tiles_m * q.map.tiles_n;
  p.grid = q.grid;
  return p;
}

// ------------------------------------------------------------ gated block

struct GluGradPlan {
  TrainProduct z, dx, dw;
  int64_t ldz, ldzt;
  int64_t off_z, off_zt, off_part, off_bias;
  int64_t bias_rows;
  int64_t bytes;
};

// z is M x N (N = 2 F columns, tiled F columns of gate and up at a time), dx
// M x K over N, dW N x K over M.
inline GluGradPlan plan_glu_grad(int64_t M, int64_t N, int64_t K, bool want_dx, bool want_dw,
                                 bool want_bias, int cu) {
  GluGradPlan p{};
  if (M <= 0 || N <= 0) return p;
  const ForwardPlan f = plan_forward(M, N, K, cu, true);
  p.z = f.z;
  p.dx = plan_product(M, K, N, kMaxSplits, cu);
  p.dw = plan_product(N, K, M, kMaxSplits, cu);
  p.ldz = ceil_div(N, 8) * 8;
  p.ldzt = ceil_div(M, 16) * 16;
  int64_t at = 0;
  if (want_dx) p.off_z = region(at, bytes_of(M, p.ldz * 2));
  if (want_dw) p.off_zt = region(at, bytes_of(N, p.ldzt * 2));
  int64_t part = 0;
  if (want_dx && p.dx.splits > 1) part = bytes_of(p.dx.splits, slot_bytes(M, K));
  if (want_dw && p.dw.splits > 1) {
    const int64_t b = bytes_of(p.dw.splits, slot_bytes(N, K));
    if (b > part) part = b;  // the two products run one after the other
  }
  p.off_part = region(at, part);
  p.bias_rows = (int64_t)p.z.map.tiles_m * f.row_groups;
  p.off_bias = region(at, want_bias ? bytes_of(p.bias_rows, N * 4) : 0);
  p.bytes = at;
  return p;
}

// ----------------------------------------------- cross entropy of a product

struct XentPlan {
  ForwardPlan l, rest;  // of the first `head` columns and of the others
  int64_t head;
  int64_t segs, rest_segs;
  int64_t off_part, off_sum, off_hit;
  int64_t bytes;
};

inline XentPlan plan_xent(int64_t M, int64_t N, int64_t K, bool smooth, int cu) {
  XentPlan p{};
  if (M <= 0) return p;
  p.head = head_logits(M, N, K, cu);
  p.l = plan_forward(M, p.head, K, cu);
  if (p.head < N) {
    p.rest = plan_forward(M, N - p.head, K, cu);
    p.rest_segs = ceil_div(N - p.head, p.rest.seg_cols);
  }
  p.segs = ceil_div(p.head, p.l.seg_cols) + p.rest_segs;
  int64_t at = 0;
  p.off_part = region(at, bytes_of(p.segs, M * 8));
  p.off_sum = region(at, smooth ? bytes_of(p.segs, M * 4) : 0);
  p.off_hit = region(at, M * 4);
  p.bytes = at;
  return p;
}

struct XentGradPlan {
  int64_t piece, n_pieces;
  int64_t ldz, ldzt;
  int slots;  // fp32 partial results of dx over all pieces (0: written at once)
  int64_t off_rows, off_scale, off_z, off_zt, off_dx, off_dw;
  int64_t bytes;
};

// Columns of a vocabulary piece: both copies of its G (2 bytes a value) stay
// within 1 GiB. Fewer, larger pieces need fewer partial results of dx and
// leave fewer ragged rounds of tiles.
constexpr int64_t kXentPieceBytes = (int64_t)1 << 30;
constexpr int64_t kXentPieceMax = ((int64_t)1 << 22) - 256;

inline TrainProduct plan_xent_dx(int64_t M, int64_t K, int64_t cols, int cu) {
  return plan_product(M, K, cols, kMaxSplits, cu);
}
inline TrainProduct plan_xent_dw(int64_t M, int64_t K, int64_t cols, int cu) {
  return plan_product(cols, K, M, kMaxSplits, cu);
}

inline XentGradPlan plan_xent_grad(int64_t M, int64_t N, int64_t K, int64_t ldw, int64_t piece,
                                   bool want_dx, bool want_dw, int cu) {
  XentGradPlan p{};
  if (M <= 0 || N <= 0) return p;
  p.ldzt = ceil_div(M, 16) * 16;
  // the dx product reads a piece of W, and 256 rows of its G, through 32-bit
  // offsets
  int64_t rows = ((int64_t)1 << 31) / (2 * ldw);
  if (rows > kXentPieceMax) rows = kXentPieceMax;
  if (piece <= 0) {
    piece = kXentPieceBytes / (4 * p.ldzt) / 256 * 256;
    if (piece < 256) piece = 256;
    if (piece > rows) piece = rows;
    const int64_t n = ceil_div(N, piece);
    const int64_t even = ceil_div(ceil_div(N, n), 256) * 256;  // pieces of equal size
    if (even < piece) piece = even;
  }
  if (piece > rows) piece = rows;
  if (piece > N) piece = N;
  p.piece = piece;
  p.n_pieces = ceil_div(N, piece);
  p.ldz = ceil_div(piece, 8) * 8;
  // every piece but the last has the same plan
  const int64_t last = N - (p.n_pieces - 1) * piece;
  int64_t at = 0;
  p.off_rows = region(at, M * 16);
  p.off_scale = region(at, 4);
  if (want_dx) {
    p.off_z = region(at, bytes_of(M, p.ldz * 2));
    p.slots = plan_xent_dx(M, K, last, cu).splits;
    if (p.n_pieces > 1) p.slots += (p.n_pieces - 1) * plan_xent_dx(M, K, piece, cu).splits;
    if (p.slots == 1) p.slots = 0;
    p.off_dx = region(at, bytes_of(p.slots, slot_bytes(M, K)));
  }
  if (want_dw) {
    p.off_zt = region(at, bytes_of(piece, p.ldzt * 2));
    int64_t part = 0;
    for (const int64_t cols : {piece, last}) {
      const TrainProduct q = plan_xent_dw(M, K, cols, cu);
      const int64_t b = q.splits > 1 ? bytes_of(q.splits, slot_bytes(cols, K)) : 0;
      if (b > part) part = b;
    }
    p.off_dw = region(at, part);
  }
  p.bytes = at;
  return p;
}

}  // namespace tg
