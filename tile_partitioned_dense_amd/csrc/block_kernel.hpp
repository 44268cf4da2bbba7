// block_kernel.hpp -- E4M3 products with float32 scales for blocks of 128.
//
//   C[i][j] = sum_b sA[b][i] sB[j / 128][b] * sum_{k in block b} A[i][k] B[j][k]
//
// The inner sum is one matrix instruction's (16 x 16 x 128); its fp32 result is
// scaled and added to the accumulators by an FMA an element: 2 K / 128 VALU
// operations a value of C against 2 K products, which fit beside the matrix
// instructions of another wave.
//
// This kernel is for outputs of few rows or columns: such a call is bound by
// reading B once, or by its operands' way into LDS (55 to 60 GB/s a compute
// unit) where a few hundred rows read B again. Tiles of 16 to 96 rows and 32 to
// 128 columns; the waves of a workgroup share K as well (KS of them, two to
// eight) where the tile is too small for eight waves, each taking every KS-th
// block, and the first adds the others' sums through LDS in a fixed order.
// Operands, the blocks' scales among them, arrive by direct loads to LDS, NST - 1
// stages of 36 to 64 KB ahead: with 256 units about 16 MB are under way, what the
// memory's latency times its rate asks for. Chunks of 16 bytes are kept at
// positions XORed with their row, so that the 16 rows of a fragment read come
// from all banks. Rows and chunks past an operand's end are sent past their
// resource's and arrive as zeros; no load or store depends on a branch.
//
// Measured: 16 x 28672 x 8192 36 us (6.5 TB/s; the launch and the first loads
// are 5 of them); 64 experts of 4096 x 2048 with 3 rows each 80 us (6.8 TB/s;
// one read of many large pieces reaches 7.1). Not faster: tiles cut so that 256
// instead of 224 units have one (the memory is as busy with either); the sc0 and
// sc1 cache hints instead of nt.
#pragma once

#include "mx_kernel.hpp"  // first: the HIP runtime headers plan.hpp relies on under hipcc
#include "block_plan.hpp"

namespace tg {

struct BlockArgs {
  const uint8_t* A;   // M x K E4M3, lda bytes between rows
  const uint8_t* B;   // N x K E4M3, ldb bytes between rows (one such matrix per expert)
  const float* sA;    // K-block b of row i at sA[b * lsa + i]
  const float* sB;    // K-block b of rows 128 r .. at sB[r * lsb + b]
  void* C;
  int32_t M, N, K;
  int64_t lda, ldb, ldc, lsa, lsb;
  TileMap map;
  const float* bias;
  int32_t act;
  // experts: expert e owns rows [offsets[e], offsets[e + 1]) of A and C, and
  // the matrix and scales `eb` bytes and `esb` floats after expert e - 1's
  const int32_t* offsets;
  int32_t groups;
  int64_t eb, esb;
  int32_t once;  // B's bytes are read by one tile only
};

// (an unscaled product: with both scale operands a constant 0 the plain form
// of the instruction is selected)
__device__ __forceinline__ floatx4 mma_fp8(const i32x8& a_frag, const i32x8& b_frag) {
  return __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(b_frag, a_frag, floatx4{}, 0, 0, 0, 0, 0, 0);
}

// The same with bf16 instructions: E4M3 values are bf16 values, and the bf16
// instruction adds their products in fp32, where the E4M3 ones cut each run of
// 8 products at 2^-14 of its largest (probed; 1.5e-5 of the result in the
// 2-norm, whichever of them). Byte 8 q + e of a lane's 32 is value e of step q
// of both operands.
typedef bf16x8 bf16x32[4];
__device__ __forceinline__ void widen_e4m3(const i32x8& v, bf16x32& out) {
#pragma unroll
  for (int q = 0; q < 4; ++q) {
    uint4 w;
    w.x = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8((unsigned)v[2 * q], 1.0f, false));
    w.y = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8((unsigned)v[2 * q], 1.0f, true));
    w.z = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8((unsigned)v[2 * q + 1], 1.0f, false));
    w.w = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8((unsigned)v[2 * q + 1], 1.0f, true));
    out[q] = as_bf16x8(w);
  }
}

// Buffer resource over [base, base + bytes), at most 2 GiB of it: a tile's
// rows lie within that (leading dimensions are below 2^22).
__device__ __forceinline__ i32x4 panel_rsrc(const void* base, int64_t bytes) {
  return make_rsrc(base, bytes > 0x7fffffffll ? 0x7fffffffll : bytes);
}

// dma16 past the caches, for bytes that are read once
#pragma clang diagnostic push
#pragma clang diagnostic ignored "-Winline-asm"
__device__ __forceinline__ void dma16_once(uint32_t lds, const i32x4& rsrc_in, uint32_t voff) {
  const i32x4 rsrc = uniform_rsrc(rsrc_in);
  lds = __builtin_amdgcn_readfirstlane(lds);
  asm volatile(
      "s_mov_b32 m0, %0\n\t"
      "buffer_load_dwordx4 %1, %2, 0 offen nt lds"
      :
      : "s"(lds), "v"(voff), "s"(rsrc)
      : "memory", "m0");
}
#pragma clang diagnostic pop

// --- owned tiles
struct BlockTile {
  int m0, n0, m_end;  // first row and column, end of the rows it may store
  const uint8_t* B;
  const float* sB;
};

__device__ __forceinline__ int32_t lds_load_i32(uint32_t addr) {
  return *(const __attribute__((address_space(3))) int32_t*)(uintptr_t)addr;
}
__device__ __forceinline__ void lds_store_i32(uint32_t addr, int32_t v) {
  *(__attribute__((address_space(3))) int32_t*)(uintptr_t)addr = v;
}
__device__ __forceinline__ float lds_load_f32(uint32_t addr) {
  return *(const __attribute__((address_space(3))) float*)(uintptr_t)addr;
}

// Experts, in LDS: the row tiles before each expert, and each one's first row cut
// to [0, M] (groups + 1 values of both).
struct ExpertTables {
  uint32_t pre, row;  // addresses
  int last;           // expert of the last tile asked for
};

// Fills the tables at `at`; the tiles there are. Ascending offsets give at most
// M / BM + groups row tiles, the number that is checked to fit 32 bits: the rest
// is cut off.
template <int BM>
__device__ __forceinline__ int expert_tiles(const BlockArgs& p, uint32_t at, int wave, int lane, ExpertTables& tab) {
  tab.pre = at;
  tab.row = at + kExpertLds / 2;
  tab.last = 0;
  if (wave == 0) {
    int base = 0;
    for (int g0 = 0; g0 < p.groups; g0 += 64) {
      const int g = g0 + lane;
      int t = 0;
      if (g < p.groups) {
        const int lo = min(max(p.offsets[g], 0), p.M);
        const int hi = min(max(p.offsets[g + 1], 0), p.M);
        t = (max(hi - lo, 0) + BM - 1) / BM;
        lds_store_i32(tab.row + 4u * g, lo);
        if (g == p.groups - 1) lds_store_i32(tab.row + 4u * g + 4u, hi);
      }
      int incl = t;
#pragma unroll
      for (int d = 1; d < 64; d *= 2) {
        const int up = __shfl_up(incl, d, 64);
        if (lane >= d) incl += up;
      }
      if (g < p.groups) lds_store_i32(tab.pre + 4u * g, base + incl - t);
      base += __shfl(incl, 63, 64);
    }
    if (lane == 0) lds_store_i32(tab.pre + 4u * p.groups, base);
  }
  __syncthreads();
  const int most = (p.M + BM - 1) / BM + p.groups;
  return __builtin_amdgcn_readfirstlane(min(lds_load_i32(tab.pre + 4u * p.groups), most)) * p.map.tiles_n;
}

// The tile of index wg: of the output, or (experts) of one expert's rows, 8 row
// tiles of it at a time before the next columns; consecutive tiles on one XCD.
template <int BM, int BN, bool EXPERTS>
__device__ __forceinline__ BlockTile block_tile(const BlockArgs& p, ExpertTables& tab, int wg, int n_tiles) {
  BlockTile at;
  at.B = p.B;
  at.sB = p.sB;
  if constexpr (EXPERTS) {
    const int q = n_tiles / kXcds, r = n_tiles % kXcds, x = wg % kXcds;
    const int t = x * q + min(x, r) + wg / kXcds;
    const int row_tile = t / p.map.tiles_n;
    // the last expert whose first row tile is not past this one: mostly that of
    // the tile before or the next
    int lo = tab.last, hi = min(lo + 1, p.groups - 1);
    if (lds_load_i32(tab.pre + 4u * lo) > row_tile || lds_load_i32(tab.pre + 4u * hi + 4u) <= row_tile) {
      lo = 0;
      hi = p.groups - 1;
    }
    while (lo < hi) {
      const int mid = (lo + hi + 1) / 2;
      if (lds_load_i32(tab.pre + 4u * mid) <= row_tile) lo = mid;
      else hi = mid - 1;
    }
    const int e = tab.last = __builtin_amdgcn_readfirstlane(lo);
    const int first = __builtin_amdgcn_readfirstlane(lds_load_i32(tab.pre + 4u * e));
    const int next = __builtin_amdgcn_readfirstlane(lds_load_i32(tab.pre + 4u * e + 4u));
    const int e_lo = __builtin_amdgcn_readfirstlane(lds_load_i32(tab.row + 4u * e));
    at.m_end = __builtin_amdgcn_readfirstlane(lds_load_i32(tab.row + 4u * e + 4u));
    const int local = t - first * p.map.tiles_n;
    const int per = 8 * p.map.tiles_n;
    const int grp = local / per;
    const int gsz = min(8, next - first - 8 * grp);
    const int in = local - grp * per;
    at.m0 = e_lo + (8 * grp + in % gsz) * BM;
    at.n0 = (in / gsz) * BN;
    at.B += (int64_t)e * p.eb;
    at.sB += (int64_t)e * p.esb;
  } else {
    int32_t tm, tn;
    tile_of(p.map, wg, tm, tn);
    at.m0 = tm * BM;
    at.n0 = tn * BN;
    at.m_end = p.M;
  }
  return at;
}

template <int BM, int BN, int WM, int WN, int KS, int SB, int NST, bool EXPERTS, bool OUT_BF16>
__global__ __launch_bounds__(WM * WN * KS * 64, 2) void block_gemm_kernel(BlockArgs p) {
  static_assert(NST >= 2, "a stage is read behind the loads of the next");
  constexpr int NW = WM * WN * KS;
  constexpr int WTM = BM / WM, WTN = BN / WN;
  constexpr int FM = WTM / 16, FN = WTN / 16;
  constexpr int KBS = SB / kScaleBlock;   // scale blocks of K per stage
  static_assert(WTM % 16 == 0 && WTN % 16 == 0 && 128 % WTN == 0, "wave tiles within one block of B's rows");
  static_assert(KBS % KS == 0, "waves share a stage's blocks evenly");
  constexpr int CPR = SB / 16;            // 16-byte chunks per stage row
  constexpr int RPI = 1024 / SB;          // rows per load instruction
  constexpr int A_BYTES = BM * SB, B_BYTES = BN * SB;
  constexpr int A_DMA = A_BYTES / 1024, B_DMA = B_BYTES / 1024;
  constexpr int SROW = (BM + 63) / 64 * 64;  // floats of one block's A scales in LDS
  constexpr int S_DMA = KBS * (SROW / 64) + 1;
  constexpr int S_BYTES = S_DMA * 256;
  constexpr int STAGE = A_BYTES + B_BYTES + S_BYTES;
  static_assert(B_DMA % NW == 0, "B stages split evenly over the waves");
  constexpr int A_PER = (A_DMA + NW - 1) / NW, B_PER = B_DMA / NW, S_PER = (S_DMA + NW - 1) / NW;
  constexpr int NDMA = A_PER + B_PER + S_PER;
  static_assert((NST - 1) * NDMA <= 63, "loads in flight fit the counter");
  constexpr int RING = NST * STAGE;
  constexpr int LDS_EXTRA = EXPERTS ? kExpertLds : 0;
  // the store's LDS: partial sums, then a strip of 16 rows a wave; beside the
  // ring where that fits, and the next tile's first stages are loaded during the
  // store (131072 columns, K = 1024: 28.4 to 24.8 us)
  constexpr int WT = WM * WN;
  constexpr int PART = (KS - 1) * WT * FM * FN * 1024;
  constexpr int OPF = WTN * 4 + 16;
  constexpr int EPI = PART + WT * 16 * OPF;
  static_assert(EPI <= RING, "partial sums and strips fit the ring");
  constexpr bool AHEAD = RING + kExpertLds + EPI <= 160 * 1024;
  constexpr int LDS = RING + LDS_EXTRA + (AHEAD ? EPI : 0);
  static_assert(LDS <= 160 * 1024, "LDS");

  __shared__ __attribute__((aligned(1024))) uint4 smem[LDS / 16];
  const uint32_t lds0 = (uint32_t)(uintptr_t)smem;
  const uint32_t epi0 = lds0 + (AHEAD ? RING + LDS_EXTRA : 0);
  const int tid = threadIdx.x;
  const int lane = tid & 63;
  const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int ks = wave / (WM * WN);
  const int wm = (wave / WN) % WM, wn = wave % WN;
  const int l16 = lane & 15, lg = lane >> 4;
  const int N = p.N, K = p.K;
  const int nkb = (K + kScaleBlock - 1) / kScaleBlock;
  const int nst = (nkb + KBS - 1) / KBS;
  const int kch = K / 16;                 // whole chunks in a row (K is a multiple of 16)

  auto swz = [](int r) { return SB >= 256 ? (r & 15) : ((r >> 1) & 7); };
  // load sources: instruction u covers rows RPI u ..; lane l fills position
  // l % CPR of row RPI u + l / CPR, i.e. fetches chunk (l % CPR) ^ swz(row)
  uint32_t voA[A_PER], voB[B_PER];
  int chA[A_PER], chB[B_PER];
#pragma unroll
  for (int t = 0; t < A_PER; ++t) {
    const int u = wave + NW * t < A_DMA ? wave + NW * t : A_DMA - 1;
    const int r = RPI * u + lane / CPR;
    chA[t] = (lane % CPR) ^ swz(r);
    voA[t] = (uint32_t)(r * (int)p.lda) + (uint32_t)(chA[t] << 4);
  }
#pragma unroll
  for (int t = 0; t < B_PER; ++t) {
    const int r = RPI * (wave + NW * t) + lane / CPR;
    chB[t] = (lane % CPR) ^ swz(r);
    voB[t] = (uint32_t)(r * (int)p.ldb) + (uint32_t)(chB[t] << 4);
  }
  // fragment reads: row l16 of the wave's first block, chunks lg and 4 + lg of
  // each 128 bytes
  const int sw = swz(l16);
  const uint32_t rowA = lds0 + (uint32_t)((wm * WTM + l16) * SB);
  const uint32_t rowB = lds0 + A_BYTES + (uint32_t)((wn * WTN + l16) * SB);
  const uint32_t scA = lds0 + A_BYTES + B_BYTES + (uint32_t)((wm * WTM + l16) * 4);
  const uint32_t scB = lds0 + A_BYTES + B_BYTES + (uint32_t)((S_DMA - 1) * 256);

  ExpertTables tab{};
  const int n_tiles = EXPERTS ? expert_tiles<BM>(p, lds0 + RING, wave, lane, tab) : p.map.tiles_m * p.map.tiles_n;
  // the tile whose loads are issued
  int m0;
  const uint8_t *a_panel, *b_panel;
  const float* sb_row;
  int64_t a_bytes, b_bytes, sa_left, sb_left;
  // where the tiles in use, with stages loaded and next to be loaded go, the
  // oldest first (of single stages, with NST - 1 of them ahead, that is NST + 1)
  constexpr int QUEUE = AHEAD ? NST + 1 : 1;
  struct Place {
    int m0, n0, m_end;
  } under_way[QUEUE] = {};
  int n_under_way = 0;
  auto take = [&](const BlockTile& at) {
    m0 = at.m0;
    a_panel = p.A + (int64_t)m0 * p.lda;
    b_panel = at.B + (int64_t)at.n0 * p.ldb;
    a_bytes = (int64_t)(p.M - 1 - m0) * p.lda + K;
    b_bytes = (int64_t)(N - 1 - at.n0) * p.ldb + K;
    const int nb0 = at.n0 / kScaleBlock;
    sb_row = at.sB + (int64_t)nb0 * p.lsb;
    sb_left = ((int64_t)((N - 1) / kScaleBlock - nb0) * p.lsb + nkb) * 4;
    sa_left = ((int64_t)(nkb - 1) * p.lsa + (p.M - m0)) * 4;
#pragma unroll
    for (int i = 0; i < QUEUE; ++i)
      if (i == n_under_way) under_way[i] = {at.m0, at.n0, at.m_end};
    ++n_under_way;
  };
  auto issue = [&](int s, int buf) {
    const uint32_t st = lds0 + (uint32_t)(buf * STAGE);
    const int64_t kbyte = (int64_t)s * SB;
    const i32x4 rsA = panel_rsrc(a_panel + kbyte, a_bytes - kbyte);
    const i32x4 rsB = panel_rsrc(b_panel + kbyte, b_bytes - kbyte);
    const int left = kch - s * CPR;  // whole chunks of this stage's rows
#pragma unroll
    for (int t = 0; t < A_PER; ++t) {
      const int u = wave + NW * t < A_DMA ? wave + NW * t : A_DMA - 1;
      dma16(st + 1024 * u, rsA, chA[t] < left ? voA[t] : kDmaPast, 0u);
    }
    if (p.once) {
#pragma unroll
      for (int t = 0; t < B_PER; ++t)
        dma16_once(st + A_BYTES + 1024 * (wave + NW * t), rsB, chB[t] < left ? voB[t] : kDmaPast);
    } else {
#pragma unroll
      for (int t = 0; t < B_PER; ++t)
        dma16(st + A_BYTES + 1024 * (wave + NW * t), rsB, chB[t] < left ? voB[t] : kDmaPast, 0u);
    }
    const int kb = s * KBS;
#pragma unroll
    for (int t = 0; t < S_PER; ++t) {
      const int u = wave + NW * t < S_DMA ? wave + NW * t : S_DMA - 1;
      const uint32_t dst = st + A_BYTES + B_BYTES + 256 * u;
      if (u < S_DMA - 1) {
        const int b = kb + u / (SROW / 64), r0 = 64 * (u % (SROW / 64));
        const int64_t off = ((int64_t)b * p.lsa + r0) * 4;
        dma4(dst, make_rsrc(reinterpret_cast<const char*>(p.sA + m0) + off, sa_left - off), 4u * lane, 0u);
      } else {
        // lane 2 j + i: block kb + j of the tile's i-th 128 rows of B
        const int i = lane & 1, j = lane >> 1;
        const bool ok = j < KBS && kb + j < nkb && (BN > kScaleBlock || i == 0);
        const int64_t off = ((int64_t)kb) * 4;
        dma4(dst, panel_rsrc(reinterpret_cast<const char*>(sb_row) + off, sb_left - off),
             ok ? (uint32_t)(i * (int)p.lsb + j) * 4u : kDmaPast, 0u);
      }
    }
  };
  if ((int)blockIdx.x >= n_tiles) return;
  // The stages of all this workgroup's tiles go through the ring one after the
  // other, NST - 1 of them ahead (without AHEAD, those of a tile).
  int wg_next = blockIdx.x;                 // of the tile whose stages are loaded
  int s_next = nst > 0 ? 0 : -1, buf_next = 0;  // the next stage to load (-1: none), its place
  int ahead = 0;                            // stages loaded and not used yet
  take(block_tile<BM, BN, EXPERTS>(p, tab, blockIdx.x, n_tiles));
  auto tile_behind = [&] {
    wg_next += gridDim.x;
    return block_tile<BM, BN, EXPERTS>(p, tab, wg_next, n_tiles);
  };
  auto issue_next = [&] {
    if (s_next < 0) return;
    issue(s_next, buf_next);
    buf_next = buf_next + 1 == NST ? 0 : buf_next + 1;
    ++ahead;
    if (++s_next == nst) {
      s_next = -1;
      if (AHEAD && wg_next + (int)gridDim.x < n_tiles) {  // (loads are under way)
        s_next = 0;
        take(tile_behind());
      }
    }
  };
  int buf = 0;  // of the stage in use
  for (int i = 0; i < NST - 1; ++i) issue_next();
  for (int wg = blockIdx.x; wg < n_tiles; wg += gridDim.x) {
    auto frag = [&](uint32_t row_base, int kb, int blk) -> i32x8 {
      const uint32_t b = row_base + (uint32_t)(blk * 16 * SB);
      const uint4 x = __builtin_bit_cast(uint4, lds_read16(b + (uint32_t)(((8 * kb + lg) ^ sw) << 4)));
      const uint4 y = __builtin_bit_cast(uint4, lds_read16(b + (uint32_t)(((8 * kb + 4 + lg) ^ sw) << 4)));
      return i32x8{(int)x.x, (int)x.y, (int)x.z, (int)x.w, (int)y.x, (int)y.y, (int)y.z, (int)y.w};
    };

    floatx4 acc[FM][FN];
#pragma unroll
    for (int i = 0; i < FM; ++i)
#pragma unroll
      for (int j = 0; j < FN; ++j) acc[i][j] = floatx4{};

    for (int s = 0; s < nst; ++s) {
      // stage s has landed: `ahead` - 1 were issued after it (and the stores of the
      // tile before, which only make this wait longer)
      --ahead;
      static_for<0, NST - 1>([&](auto a_c) {
        if (ahead == decltype(a_c)::value) wait_vmcnt<decltype(a_c)::value * NDMA>();
      });
      wait_lgkmcnt0();
      block_barrier();
      issue_next();
      const uint32_t so = (uint32_t)(buf * STAGE);
      buf = buf + 1 == NST ? 0 : buf + 1;
      static_for<0, KBS / KS>([&](auto q_c) {
        const int kb = ks + KS * decltype(q_c)::value;
        if (KBS == 1 || s * KBS + kb < nkb) {
          const float sb = lds_load_f32(scB + so + (uint32_t)(8 * kb + (BN > kScaleBlock ? 4 * ((wn * WTN) / kScaleBlock) : 0)));
          i32x8 bq[FN], aq[FM];
          bf16x32 bw[OUT_BF16 ? 1 : FN];
          float sc[FM];
          // (all of them under way before the first is waited for: 64 x 128 tiles of
          // 200 x 8000 x 8192 48.6 to 39.0 us)
#pragma unroll
          for (int j = 0; j < FN; ++j) bq[j] = frag(rowB + so, kb, j);
#pragma unroll
          for (int i = 0; i < FM; ++i) aq[i] = frag(rowA + so, kb, i);
#pragma unroll
          for (int i = 0; i < FM; ++i) sc[i] = lds_load_f32(scA + so + (uint32_t)(kb * SROW * 4 + i * 64)) * sb;
          __builtin_amdgcn_sched_barrier(0);
          if constexpr (!OUT_BF16) {
#pragma unroll
            for (int j = 0; j < FN; ++j) widen_e4m3(bq[j], bw[j]);
          }
#pragma unroll
          for (int i = 0; i < FM; ++i) {
            floatx4 d[FN];
            if constexpr (OUT_BF16) {
#pragma unroll
              for (int j = 0; j < FN; ++j) d[j] = mma_fp8(aq[i], bq[j]);
            } else {
              bf16x32 aw;
              widen_e4m3(aq[i], aw);
#pragma unroll
              for (int j = 0; j < FN; ++j) d[j] = floatx4{};
#pragma unroll
              for (int q = 0; q < 4; ++q)
#pragma unroll
                for (int j = 0; j < FN; ++j) d[j] = mfma16(bw[j][q], aw[q], d[j]);
            }
#pragma unroll
            for (int j = 0; j < FN; ++j)
#pragma unroll
              for (int e = 0; e < 4; ++e) acc[i][j][e] = __builtin_fmaf(d[j][e], sc[i], acc[i][j][e]);
          }
        }
      });
    }

    // store: waves that share K pass their sums through LDS in a fixed order;
    // then 16-row strips staged as fp32
    wait_lgkmcnt0();
    block_barrier();  // the ring is free
    const int row0 = under_way[0].m0, col0 = under_way[0].n0, end = under_way[0].m_end;
#pragma unroll
    for (int i = 0; i + 1 < QUEUE; ++i) under_way[i] = under_way[i + 1];
    --n_under_way;
    if constexpr (KS > 1) {
      if (ks > 0) {
        const uint32_t at = epi0 + (uint32_t)((((ks - 1) * WT + wave % WT) * FM * FN) * 1024 + lane * 16);
#pragma unroll
        for (int i = 0; i < FM; ++i)
#pragma unroll
          for (int j = 0; j < FN; ++j) lds_store_f4(at + 1024u * (i * FN + j), acc[i][j]);
      }
      wait_lgkmcnt0();
      block_barrier();
      if (ks == 0) {
#pragma unroll
        for (int h = 1; h < KS; ++h) {
          const uint32_t at = epi0 + (uint32_t)((((h - 1) * WT + wave) * FM * FN) * 1024 + lane * 16);
#pragma unroll
          for (int i = 0; i < FM; ++i)
#pragma unroll
            for (int j = 0; j < FN; ++j) {
              const floatx4 v = lds_load_f4(at + 1024u * (i * FN + j));
#pragma unroll
              for (int e = 0; e < 4; ++e) acc[i][j][e] += v[e];
            }
        }
      }
    }
    if (KS == 1 || ks == 0) {
      const uint32_t stf = epi0 + (uint32_t)(PART + (wave % WT) * 16 * OPF);
      const EpiOut eo{p.C, p.ldc, end, N, EXPERTS ? nullptr : p.bias, EXPERTS ? kActNone : p.act, nullptr, 0};
#pragma unroll
      for (int i = 0; i < FM; ++i) {
#pragma unroll
        for (int j = 0; j < FN; ++j) lds_store_f4(stf + (uint32_t)(l16 * OPF + (16 * j + 4 * lg) * 4), acc[i][j]);
        wave_lds_sync();
        store_staged_fused<OUT_BF16, false, kActReluNan>(stf, OPF, 16, WTN, row0 + wm * WTM + 16 * i, col0 + wn * WTN,
                                                         lane, 64, eo);
        wave_lds_sync();
      }
    }
    if (wg + (int)gridDim.x >= n_tiles) break;
    if (!AHEAD || nst == 0) {
      wait_vmcnt<0>();
      wait_lgkmcnt0();
      block_barrier();
      take(tile_behind());
      s_next = nst > 0 ? 0 : -1;
      for (int i = 0; i < NST - 1; ++i) issue_next();
    }
  }
}

}  // namespace tg
