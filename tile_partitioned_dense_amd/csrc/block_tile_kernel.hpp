// block_tile_kernel.hpp -- E4M3 products with block scales for outputs of many
// rows and columns (the operands, formula, scales and owned tiles of
// block_kernel.hpp).
//
// One persistent workgroup a compute unit (two of the 128 x 128 ones) takes
// tiles of one XCD's run, 256 x 256 where the output fills the chip with them.
// Two stages of 128 bytes of K are in LDS (131 KB). A stage is one pass over the
// wave's blocks, row by row: a matrix instruction, the fragment reads that later
// ones need, a part of the loads of the stage after next and the scaling of the
// sum formed two instructions ago, pinned in this order (left to itself the
// compiler moves them together and spills). One barrier a stage, before the last
// two rows of blocks: these are worked column by column, so that B of the next
// stage takes the place of each column as its last use is through and the loads
// go out over half a stage. A tile's last two stages load the next one's first
// (16396 rows of 16 experts, 7168 x 2048: 273 to 268 us; 8192 of 64, 4096 x 1024:
// 76.9 to 74.6), while its sums leave from registers.
//
// Bound by power (the clock falls to 1.9 to 2.0 GHz; the bare instructions do
// 3.9 PFLOP/s under load, the bf16 ones 2.1) and by the loads' path into LDS (10
// to 11 TB/s): without loads it is 18 to 20% faster, without the FMAs 10%,
// without fragment reads 9%. Measured: 8192 x 7168 x 8192 to bf16 420 us (2.29
// PFLOP/s; the library's product with one scale 388); 16396 rows of 16 experts,
// 7168 x 2048, 264 us; to fp32 8192 x 7168 x 8192 755 us (1.27 PFLOP/s, bf16
// instructions; the library's bf16 8192^3 reaches 1.45). Not faster: a second barrier that frees B early (7% slower), three
// stages of a 256 x 128 tile, loads over 8, 12, 20 and 24 instead of 16
// instructions, wave priorities, waves of 64 x 128 (9% slower), runs of 4 and 16
// row tiles, smaller tiles for the last round.
#pragma once

#include "block_kernel.hpp"

// The kernel's lambdas: one that is not inlined holds its captures, the operands'
// addresses among them, in memory (the 128 x 128 tile took nine times as long).
#define TG_INLINE __attribute__((always_inline))

namespace tg {

// The fused epilogue on the accumulators: column col + 16 j + e in acc[][j][e].
template <int FM, int FN, int ACT>
__device__ __forceinline__ void finish_act(floatx4 (&acc)[FM][FN], const BlockArgs& p, int col) {
#pragma unroll
  for (int j = 0; j < FN; ++j) {
    floatx4 b = floatx4{};
    if (p.bias) {
#pragma unroll
      for (int e = 0; e < 4; ++e) b[e] = p.bias[min(col + 16 * j + e, p.N - 1)];
    }
#pragma unroll
    for (int i = 0; i < FM; ++i)
#pragma unroll
      for (int e = 0; e < 4; ++e) acc[i][j][e] = act_fn<ACT>(acc[i][j][e] + b[e]);
    __builtin_amdgcn_sched_barrier(0);
  }
}
template <int FM, int FN>
__device__ __forceinline__ void finish(floatx4 (&acc)[FM][FN], const BlockArgs& p, int col) {
  switch (p.act) {
    case kActRelu: finish_act<FM, FN, kActReluNan>(acc, p, col); break;
    case kActSigmoid: finish_act<FM, FN, kActSigmoid>(acc, p, col); break;
    case kActTanh: finish_act<FM, FN, kActTanh>(acc, p, col); break;
    case kActSilu: finish_act<FM, FN, kActSilu>(acc, p, col); break;
    default: finish_act<FM, FN, kActNone>(acc, p, col);
  }
}

// WIDE: an fp32 output, its products on bf16 instructions (widen_e4m3). The
// conversions are 2% of its time.
template <int BM, int BN, int WM, int WN, bool EXPERTS, bool WIDE>
__global__ __launch_bounds__(WM * WN * 64, 2) void block_tile_kernel(BlockArgs p) {
  constexpr int NW = WM * WN;
  constexpr int WTM = BM / WM, WTN = BN / WN;
  constexpr int FM = WTM / 16, FN = WTN / 16;
  static_assert(FM % 2 == 0 && FM >= 4 && FN % 2 == 0 && FN >= 4 && 128 % WTN == 0, "row parity; one block of B's rows a wave");
  constexpr int RB = kScaleBlock;         // bytes of a row and stage
  constexpr int A_BYTES = BM * RB, B_BYTES = BN * RB;
  constexpr int A_DMA = A_BYTES / 1024, B_DMA = B_BYTES / 1024;
  static_assert(A_DMA % NW == 0 && B_DMA % NW == 0 && BM % 64 == 0 && NW % 2 == 0, "loads split evenly over the waves");
  constexpr int A_PER = A_DMA / NW, B_PER = B_DMA / NW;
  constexpr int S_DMA = BM / 64 + 1;
  static_assert(S_DMA <= NW, "a scale load each at most");
  constexpr int STAGE = A_BYTES + B_BYTES + S_DMA * 256;
  constexpr int RING = 2 * STAGE;
  constexpr int LDS_EXTRA = EXPERTS ? kExpertLds : 0;
  static_assert(RING + LDS_EXTRA <= 160 * 1024, "LDS");
  constexpr int NU = A_PER + B_PER + 1;   // a wave's loads of a stage
  // MFMA n of a stage: row by row of blocks, the last two rows together, column
  // by column
  constexpr int PAIR = (FM - 2) * FN;
  constexpr auto mfma_row = [](int n) { return n < PAIR ? n / FN : FM - 2 + (n - PAIR) % 2; };
  constexpr auto mfma_col = [](int n) { return n < PAIR ? n % FN : (n - PAIR) / 2; };
  // where load u goes out: MFMAs after the barrier
  constexpr int LD = FM * FN / 2;
  constexpr auto load_pos = [](int u) { return ((2 * u + 1) * LD) / (2 * NU); };
  constexpr int NU1 = [] {  // loads before the end of the stage
    int n = 0;
    while (n < NU && ((2 * n + 1) * LD) / (2 * NU) < 2 * FN) ++n;
    return n;
  }();

  constexpr bool LAST = FM * FN < 32;     // an odd last stage by itself (below)
  constexpr int STORES = WIDE ? FM * FN : FM * (FN / 2);  // of a tile, per wave
  constexpr int ESZ = WIDE ? 4 : 2;       // bytes of an output
  static_assert(FN % 2 == 0 && NU1 + STORES <= 63, "pairs of blocks; the counter");

  __shared__ __attribute__((aligned(1024))) uint4 smem[(RING + LDS_EXTRA) / 16];
  const uint32_t lds0 = (uint32_t)(uintptr_t)smem;
  const int tid = threadIdx.x;
  const int lane = tid & 63;
  const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int wm = wave / WN, wn = wave % WN;
  const int l16 = lane & 15, lg = lane >> 4;
  const int N = p.N, K = p.K;
  const int nst = (K + RB - 1) / RB;

  // load sources: instruction u = wave + NW t covers rows 8 u ..; lane l fills
  // position l % 8 of row 8 u + l / 8, i.e. fetches chunk (l % 8) ^ ((row >> 1) & 7)
  // (the same for all t: NW is even)
  const int row0 = 8 * wave + (lane >> 3);
  const int chunk = (lane & 7) ^ ((row0 >> 1) & 7);
  const uint32_t voA = (uint32_t)(row0 * (int)p.lda + 16 * chunk), voB = (uint32_t)(row0 * (int)p.ldb + 16 * chunk);
  const uint32_t stepA = (uint32_t)(8 * NW * (int)p.lda), stepB = (uint32_t)(8 * NW * (int)p.ldb);
  const uint32_t ldsw = __builtin_amdgcn_readfirstlane(lds0 + 1024 * wave);
  // fragment reads: row l16 of the wave's first block, chunks lg and 4 + lg
  const int sw = (l16 >> 1) & 7;
  const uint32_t ch0 = (uint32_t)((lg ^ sw) << 4), ch1 = (uint32_t)(((4 + lg) ^ sw) << 4);
  uint32_t fA[2][2], fB[2][2];  // of buffer and chunk
#pragma unroll
  for (int st = 0; st < 2; ++st)
#pragma unroll
    for (int c = 0; c < 2; ++c) {
      fA[st][c] = lds0 + (uint32_t)(st * STAGE + (wm * WTM + l16) * RB) + (c ? ch1 : ch0);
      fB[st][c] = lds0 + (uint32_t)(st * STAGE + A_BYTES + (wn * WTN + l16) * RB) + (c ? ch1 : ch0);
      asm volatile("" : "+v"(fA[st][c]), "+v"(fB[st][c]));  // (blocks by immediate offsets from these)
    }
  const uint32_t scA = lds0 + A_BYTES + B_BYTES + (uint32_t)((wm * WTM + l16) * 4);
  const uint32_t scB = lds0 + A_BYTES + B_BYTES + (uint32_t)((S_DMA - 1) * 256 + ((wn * WTN) / kScaleBlock) * 4);

  ExpertTables tab{};
  const int n_tiles = EXPERTS ? expert_tiles<BM>(p, lds0 + RING, wave, lane, tab) : p.map.tiles_m * p.map.tiles_n;
  if ((int)blockIdx.x >= n_tiles) return;
  const bool far = p.ldc * ESZ * BM > 0x7fffffffll;  // a tile of C spans more than a resource

  // the tile whose loads are issued: its operands, and the stages' number from
  // its first (`past`: the stages of the tile before, when its last ones load this
  // one's first)
  struct Source {
    const uint8_t *a_panel, *b_panel;
    const char* s_base;
    int64_t a_bytes, b_bytes, s_bytes;
  } src;
  int past = 0;
  // this wave's scales: 64 rows of A, or (one wave) the tile's blocks of B
  // (lane i < BN / 128); the other waves repeat the last of these
  const int su = wave < S_DMA ? wave : S_DMA - 1;
  const bool sA_wave = su < S_DMA - 1;
  const int64_t s_step = sA_wave ? p.lsa * 4 : 4;
  const uint32_t voS = sA_wave ? 4u * lane : lane < BN / kScaleBlock ? (uint32_t)(lane * (int)p.lsb) * 4u : kDmaPast;
  auto source = [&](const BlockTile& at) TG_INLINE {
    const int nb0 = at.n0 / kScaleBlock;
    return Source{p.A + (int64_t)at.m0 * p.lda, at.B + (int64_t)at.n0 * p.ldb,
                  sA_wave ? reinterpret_cast<const char*>(p.sA + at.m0 + 64 * su)
                          : reinterpret_cast<const char*>(at.sB + (int64_t)nb0 * p.lsb),
                  (int64_t)(p.M - 1 - at.m0) * p.lda + K, (int64_t)(N - 1 - at.n0) * p.ldb + K,
                  sA_wave ? ((int64_t)(nst - 1) * p.lsa + (p.M - at.m0 - 64 * su)) * 4
                          : ((int64_t)((N - 1) / kScaleBlock - nb0) * p.lsb + nst) * 4};
  };
  // load n of stage s into buffer ST = s % 2: A's, B's, then the scales. Chunks
  // past K are sent to an offset past their resource's end (2 GiB at most),
  // where they arrive as zeros.
  auto load = [&](auto st_c, int s_all, int n) TG_INLINE {
    const int s = s_all - past;
    constexpr uint32_t st = (uint32_t)(decltype(st_c)::value * STAGE);
    const bool in = chunk * 16 < K - s * RB;
    if (n < A_PER)
      dma16(ldsw + st + 1024 * NW * n, panel_rsrc(src.a_panel + (int64_t)s * RB, src.a_bytes - (int64_t)s * RB),
            (in ? voA : 0x80000000u) + n * stepA, 0u);
    else if (n < A_PER + B_PER)
      dma16(ldsw + st + A_BYTES + 1024 * NW * (n - A_PER),
            panel_rsrc(src.b_panel + (int64_t)s * RB, src.b_bytes - (int64_t)s * RB),
            (in ? voB : 0x80000000u) + (n - A_PER) * stepB, 0u);
    else
      dma4(lds0 + st + A_BYTES + B_BYTES + 256 * su, panel_rsrc(src.s_base + s * s_step, s < nst ? src.s_bytes - s * s_step : 0), voS, 0u);
  };
  auto frag = [&](const uint32_t (&f)[2][2], int st, int blk) -> i32x8 {
    const uint4 x = __builtin_bit_cast(uint4, lds_read16(f[st][0] + (uint32_t)(blk * 16 * RB)));
    const uint4 y = __builtin_bit_cast(uint4, lds_read16(f[st][1] + (uint32_t)(blk * 16 * RB)));
    return i32x8{(int)x.x, (int)x.y, (int)x.z, (int)x.w, (int)y.x, (int)y.y, (int)y.z, (int)y.w};
  };

  auto first_loads = [&]() TG_INLINE {
    static_for<0, NU>([&](auto u_c) TG_INLINE { load(std::integral_constant<int, 0>{}, 0, decltype(u_c)::value); });
    static_for<0, NU1>([&](auto u_c) TG_INLINE { load(std::integral_constant<int, 1>{}, 1, decltype(u_c)::value); });
  };

  // The last two stages of a tile load the next one's first (`cross`), unless
  // their number is odd and the buffers would change places. Past the last tile,
  // and past the last stage without that, zeros arrive, without traffic.
  const int nst2 = LAST ? nst : (nst + 1) / 2 * 2;
  const bool cross = nst2 > 0 && nst2 % 2 == 0;
  BlockTile now = block_tile<BM, BN, EXPERTS>(p, tab, blockIdx.x, n_tiles), next = now;
  src = source(now);
  first_loads();
  wait_vmcnt<NU1>();
  block_barrier();
  for (int wg = blockIdx.x; wg < n_tiles;) {
    // (stage 0 has landed)
    wg += gridDim.x;
    const int m0 = now.m0, n0 = now.n0, m_end = now.m_end;
    Source ahead{};
    if (wg < n_tiles) {
      next = block_tile<BM, BN, EXPERTS>(p, tab, wg, n_tiles);
      ahead = source(next);
    }
    past = 0;
    // at the barrier of stage s
    auto change = [&](int s) TG_INLINE {
      const bool at = cross && s == nst2 - 2;
      src.a_panel = at ? ahead.a_panel : src.a_panel;
      src.b_panel = at ? ahead.b_panel : src.b_panel;
      src.s_base = at ? ahead.s_base : src.s_base;
      src.a_bytes = at ? ahead.a_bytes : src.a_bytes;
      src.b_bytes = at ? ahead.b_bytes : src.b_bytes;
      src.s_bytes = at ? ahead.s_bytes : src.s_bytes;
      past = at ? nst2 : past;
    };

    // a wave whose rows are all past the tile's last (an expert's last tile)
    // only takes part in the loads
    if (m0 + wm * WTM >= m_end) {
      // a stage's loads and barrier alone
      auto idle = [&](auto st_c, int s) TG_INLINE {
        constexpr int ST = decltype(st_c)::value;
        static_for<NU1, NU>([&](auto u_c) TG_INLINE { load(std::integral_constant<int, ST ^ 1>{}, s + 1, decltype(u_c)::value); });
        wait_vmcnt<0>();
        block_barrier();
        if constexpr (ST == 0) change(s);
        static_for<0, NU1>([&](auto u_c) TG_INLINE { load(std::integral_constant<int, ST>{}, s + 2, decltype(u_c)::value); });
      };

      int s = 0;
      for (; LAST ? s + 1 < nst : s < nst; s += 2) {
        idle(std::integral_constant<int, 0>{}, s);
        idle(std::integral_constant<int, 1>{}, s + 1);
      }
      if (LAST && s < nst) idle(std::integral_constant<int, 0>{}, s);
      if (!cross) {
        wait_vmcnt<0>();
        block_barrier();
        src = ahead;
        if (wg < n_tiles) first_loads();
        wait_vmcnt<NU1>();
        block_barrier();
      }
      now = next;
      continue;
    }

    floatx4 acc[FM][FN];
#pragma unroll
    for (int i = 0; i < FM; ++i)
#pragma unroll
      for (int j = 0; j < FN; ++j) {
        acc[i][j] = floatx4{};
        asm volatile("" : "+v"(acc[i][j]));  // (not folded into a first stage of its own)
      }

    // B of the stage; A: rows r < FM - 1 alternate between two sets, which the
    // stages take in turn, row FM - 1 has the third
    i32x8 bq[FN], a[3];
    bf16x32 aw[WIDE ? 2 : 1], bw[WIDE ? FN : 1];  // WIDE: of the row's parity; of the stage
    floatx4 d[4];            // sums of the last MFMAs, scaled and added two later
    float raw[2], sc[2], sb; // A's scales as read, and times B's, by the row's parity
#pragma unroll
    for (int j = 0; j < FN; ++j) bq[j] = frag(fB, 0, j);
    a[0] = frag(fA, 0, 0);
    raw[0] = lds_load_f32(scA);
    sb = lds_load_f32(scB);
    sc[0] = sc[1] = raw[1] = 0.0f;
    d[2] = d[3] = floatx4{};
    auto add = [&](auto m_c) TG_INLINE {
      constexpr int m = decltype(m_c)::value, i = mfma_row(m), j = mfma_col(m);
      asm volatile("" : "+v"(d[m % 4]));
#pragma unroll
      for (int e = 0; e < 4; ++e) acc[i][j][e] = __builtin_fmaf(d[m % 4][e], sc[i & 1], acc[i][j][e]);
      asm volatile("" : "+v"(acc[i][j]));
    };

    // One stage, in buffer ST. Its last phase and the next stage's first one
    // load stage s + 2; one past the last arrives as zeros, without traffic.
    auto step = [&](auto st_c, int s) TG_INLINE {
      constexpr int ST = decltype(st_c)::value;
      static_for<0, FM * FN>([&](auto n_c) TG_INLINE {
        constexpr int n = decltype(n_c)::value;
        constexpr int i = mfma_row(n), j = mfma_col(n);
        constexpr int q = n - PAIR;       // MFMA of the last two rows
        constexpr int slot = i == FM - 1 ? 2 : (i + ST) & 1;
        if constexpr (q == 0) {
          // stage s + 1 has landed, every wave has read this stage's last rows
          wait_vmcnt<0>();
          wait_lgkmcnt0();
          block_barrier();
          if constexpr (ST == 0) change(s);
        }
        if constexpr (WIDE) {
          if constexpr (j == 0) widen_e4m3(a[slot], aw[i & 1]);
          if constexpr (i == 0) widen_e4m3(bq[j], bw[j]);
          floatx4 c = floatx4{};
#pragma unroll
          for (int k = 0; k < 4; ++k) {
            asm volatile("" : "+v"(aw[i & 1][k]), "+v"(bw[j][k]));
            c = mfma16(bw[j][k], aw[i & 1][k], c);
          }
          d[n % 4] = c;
        } else {
          asm volatile("" : "+v"(a[slot]), "+v"(bq[j]));
          d[n % 4] = mma_fp8(a[slot], bq[j]);
        }
        // reads: the next row of A and its scale; in the last two rows the next
        // stage's first one, and its blocks of B as this stage's are done with
        if constexpr (q < 0) {
          if constexpr (j == 0) a[(i + 1 + ST) & 1] = frag(fA, ST, i + 1);
          if constexpr (j == 0 && i == FM - 3) a[2] = frag(fA, ST, FM - 1);
          if constexpr (j == 1) raw[(i + 1) & 1] = lds_load_f32(scA + (uint32_t)(ST * STAGE + (i + 1) * 64));
          if constexpr (j == FN - 1 && i == FM - 3) raw[1] = lds_load_f32(scA + (uint32_t)(ST * STAGE + (FM - 1) * 64));
        } else {
          if constexpr (q == 0) a[ST ^ 1] = frag(fA, ST ^ 1, 0);
          if constexpr (i == FM - 1) bq[j] = frag(fB, ST ^ 1, j);
          if constexpr (q == 4) {
            raw[0] = lds_load_f32(scA + (uint32_t)((ST ^ 1) * STAGE));
            sb = lds_load_f32(scB + (uint32_t)((ST ^ 1) * STAGE));
          }
        }
        // loads of stage s + 2 (from the barrier on) and of s + 1 (the rest)
        static_for<0, NU>([&](auto u_c) TG_INLINE {
          constexpr int u = decltype(u_c)::value;
          if constexpr (q >= 0 && load_pos(u) == q) load(std::integral_constant<int, ST>{}, s + 2, u);
          if constexpr (q < 0 && load_pos(u) == FM * FN - PAIR + n) load(std::integral_constant<int, ST ^ 1>{}, s + 1, u);
        });
        // the scale of a row before its first sum is added; the sums of the MFMA
        // two before this one
        constexpr int m = (n + FM * FN - 2) % (FM * FN), mi = mfma_row(m);
        if constexpr (mfma_col(m) == 0) sc[mi & 1] = raw[mi & 1] * sb;
        add(std::integral_constant<int, m>{});
        __builtin_amdgcn_sched_barrier(0);
      });
    };
    // (two at a time, so that the buffers are fixed. An odd last one is done by
    // itself, 3 to 7% on 33 and 11 of them; on the largest tile that kept a copy
    // of the accumulators, and one of zeros makes the number even)
    int s = 0;
    for (; LAST ? s + 1 < nst : s < nst; s += 2) {
      step(std::integral_constant<int, 0>{}, s);
      step(std::integral_constant<int, 1>{}, s + 1);
    }
    if (LAST && s < nst) step(std::integral_constant<int, 0>{}, s);
    add(std::integral_constant<int, FM * FN - 2>{});
    add(std::integral_constant<int, FM * FN - 1>{});
    if (!cross) {
      wait_vmcnt<0>();  // (zeros past the last stage)
      wait_lgkmcnt0();
      block_barrier();  // the ring is free
      src = ahead;
      if (wg < n_tiles) first_loads();
    }

    // the store, from registers
    const int row0_c = m0, col0_c = n0, end_c = m_end;
    const bool edge = n0 + BN > N || far;
    // (The experts' product has no epilogue. On the 256 x 256 tile it spills 143
    // registers, 192 bytes of scratch a lane, 9 MB of writes beside 117 for 8192 x
    // 7168; the experts' form takes the same time with and without.)
    if constexpr (!EXPERTS) {
      if (p.bias || p.act != kActNone) finish(acc, p, n0 + wn * WTN + 4 * lg);
    }
    // v_permlane exchanges of the packed blocks j and j + 1 leave a lane 8
    // consecutive columns: of block j + lg / 2, columns 8 (lg % 2) ..
    int row = wm * WTM + l16, col = wn * WTN + (WIDE ? 4 * lg : 16 * (lg >> 1) + 8 * (lg & 1));
    asm volatile("" : "+v"(row), "+v"(col));  // (formed here: held over the stages they spilled)
    const int64_t c_bytes = ((int64_t)(end_c - 1 - row0_c) * p.ldc + (N - col0_c)) * ESZ;
    char* const c_tile = static_cast<char*>(p.C) + ((int64_t)row0_c * p.ldc + col0_c) * ESZ;
    const auto rsC = __builtin_amdgcn_make_buffer_rsrc(c_tile, 0, c_bytes > 0x7fffffffll ? 0x7fffffff : (int)c_bytes,
                                                       0x00020000);
    static_for<0, FM>([&](auto i_c) TG_INLINE {
      constexpr int i = decltype(i_c)::value;
      static_for<0, WIDE ? FN : FN / 2>([&](auto h_c) TG_INLINE {
        constexpr int j = (WIDE ? 1 : 2) * decltype(h_c)::value;
        u32x4v v;
        if constexpr (WIDE) {
          v = __builtin_bit_cast(u32x4v, acc[i][j]);
        } else {
#pragma unroll
          for (int e = 0; e < 2; ++e) {
            const auto r = __builtin_amdgcn_permlane32_swap(
                pack_bf16x2(acc[i][j][2 * e], acc[i][j][2 * e + 1]),
                pack_bf16x2(acc[i][j + 1][2 * e], acc[i][j + 1][2 * e + 1]), false, false);
            const auto t = __builtin_amdgcn_permlane16_swap(r[0], r[1], false, false);
            v[e] = t[0];
            v[2 + e] = t[1];
          }
        }
        if (!edge) {
          // rows past the last lie past the end of the resource
          __builtin_amdgcn_raw_buffer_store_b128(v, rsC, (int)(((row + 16 * i) * (int)p.ldc + col + 16 * j) * ESZ), 0, 0);
        } else if (row0_c + row + 16 * i < end_c) {
          constexpr int EPC = 16 / ESZ;
          const int c = col0_c + col + 16 * j;
          char* o = c_tile + ((int64_t)(row + 16 * i) * p.ldc + col + 16 * j) * ESZ;
          if (c + EPC <= N) *reinterpret_cast<u32x4v*>(o) = v;
          else
#pragma unroll
            for (int e = 0; e < EPC; ++e)
              if (c + e < N) {
                if constexpr (WIDE) reinterpret_cast<uint32_t*>(o)[e] = v[e];
                else reinterpret_cast<uint16_t*>(o)[e] = (uint16_t)(v[e / 2] >> (16 * (e & 1)));
              }
        }
      });
    });
    if (!cross) {
      // (memory operations count down in order: the stores came after the loads)
      if (edge) wait_vmcnt<0>();  // (any number of stores)
      wait_vmcnt<NU1 + STORES>();
      block_barrier();
    }
    now = next;
  }
  wait_vmcnt<0>();  // (zeros on their way into LDS)
}

}  // namespace tg

#undef TG_INLINE
