// kernels_route.hip -- routing to experts: scores, choice and weights of each
// token, their gradient, the order of the tokens by expert, and the weighted
// sum of the experts' rows.
#include "block_launch.hpp"

namespace tg {

namespace {

constexpr int kRouteMaxE = 1024, kRouteMaxK = 32;

template <bool BF16>
__device__ __forceinline__ float load_value(const void* p, int64_t i) {
  if constexpr (BF16) return __uint_as_float((uint32_t) static_cast<const uint16_t*>(p)[i] << 16);
  else return static_cast<const float*>(p)[i];
}

// --- scores and choice
// L lanes work on a token, lane l of them on the experts l PL .. l PL + PL - 1, so
// that the lowest lane and then the lowest slot is the lowest index. Measured on
// 8191 tokens of 256 experts, 8 of them (sigmoid, bias, 8 groups), with scores in
// 64 bits: a whole wave a token, its steps by LDS exchanges, 34 us; this form
// 13.5 us (with the two-half keys and the groups below).

// v of the lane STEP before in its row of 16
template <int STEP>
__device__ __forceinline__ uint32_t lane_step(uint32_t v) {
  return (uint32_t)__builtin_amdgcn_update_dpp(0, (int)v, 0x120 + STEP, 0xf, 0xf, false);  // row_ror:STEP
}
// both values of lanes 16 (32) apart, the same pair in both
template <int STEP>
__device__ __forceinline__ void lane_pair(uint32_t v, uint32_t& x, uint32_t& y) {
  if constexpr (STEP == 16) {
    const auto r = __builtin_amdgcn_permlane16_swap(v, v, false, false);
    x = r[0];
    y = r[1];
  } else {
    const auto r = __builtin_amdgcn_permlane32_swap(v, v, false, false);
    x = r[0];
    y = r[1];
  }
}
template <int STEP>
__device__ __forceinline__ void lane_pair64(uint64_t v, uint64_t& x, uint64_t& y) {
  if constexpr (STEP < 16) {
    x = v;
    y = (uint64_t)lane_step<STEP>((uint32_t)(v >> 32)) << 32 | lane_step<STEP>((uint32_t)v);
  } else {
    uint32_t xl, yl, xh, yh;
    lane_pair<STEP>((uint32_t)v, xl, yl);
    lane_pair<STEP>((uint32_t)(v >> 32), xh, yh);
    x = (uint64_t)xh << 32 | xl;
    y = (uint64_t)yh << 32 | yl;
  }
}
// f over a token's lanes, the same in all of them (f commutes)
template <int L, class F>
__device__ __forceinline__ uint64_t join_token64(uint64_t v, F f) {
  uint64_t x, y;
  lane_pair64<8>(v, x, y);
  v = f(x, y);
  lane_pair64<4>(v, x, y);
  v = f(x, y);
  lane_pair64<2>(v, x, y);
  v = f(x, y);
  lane_pair64<1>(v, x, y);
  v = f(x, y);
  if constexpr (L > 16) {
    lane_pair64<16>(v, x, y);
    v = f(x, y);
  }
  if constexpr (L > 32) {
    lane_pair64<32>(v, x, y);
    v = f(x, y);
  }
  return v;
}
template <int L>
__device__ __forceinline__ float max_token(float v) {
  v = fmaxf(v, __uint_as_float(lane_step<8>(__float_as_uint(v))));
  v = fmaxf(v, __uint_as_float(lane_step<4>(__float_as_uint(v))));
  v = fmaxf(v, __uint_as_float(lane_step<2>(__float_as_uint(v))));
  v = fmaxf(v, __uint_as_float(lane_step<1>(__float_as_uint(v))));
  uint32_t x, y;
  if constexpr (L > 16) {
    lane_pair<16>(__float_as_uint(v), x, y);
    v = fmaxf(__uint_as_float(x), __uint_as_float(y));
  }
  if constexpr (L > 32) {
    lane_pair<32>(__float_as_uint(v), x, y);
    v = fmaxf(__uint_as_float(x), __uint_as_float(y));
  }
  return v;
}
template <int L>
__device__ __forceinline__ double sum_token(double v) {
  return __builtin_bit_cast(double, join_token64<L>(__builtin_bit_cast(uint64_t, v), [](uint64_t x, uint64_t y) {
    return __builtin_bit_cast(uint64_t, __builtin_bit_cast(double, x) + __builtin_bit_cast(double, y));
  }));
}
// An unsigned integer of the same order; 0 is below every value's.
__device__ __forceinline__ uint64_t order_key(double v) {
  const uint64_t b = __builtin_bit_cast(uint64_t, v);
  return (int64_t)b < 0 ? ~b : b | (1ull << 63);
}

template <int CTRL>
__device__ __forceinline__ double dpp_f64(double v) {
  const uint64_t u = __builtin_bit_cast(uint64_t, v);
  const uint32_t l = (uint32_t)__builtin_amdgcn_update_dpp(0, (int)(uint32_t)u, CTRL, 0xf, 0xf, false);
  const uint32_t h = (uint32_t)__builtin_amdgcn_update_dpp(0, (int)(uint32_t)(u >> 32), CTRL, 0xf, 0xf, false);
  return __builtin_bit_cast(double, (uint64_t)h << 32 | l);
}
template <int L>
__device__ __forceinline__ uint32_t max_token_u32(uint32_t v) {
  v = max(v, lane_step<8>(v));
  v = max(v, lane_step<4>(v));
  v = max(v, lane_step<2>(v));
  v = max(v, lane_step<1>(v));
  uint32_t x, y;
  if constexpr (L > 16) {
    lane_pair<16>(v, x, y);
    v = max(x, y);
  }
  if constexpr (L > 32) {
    lane_pair<32>(v, x, y);
    v = max(x, y);
  }
  return v;
}

// Logits of the experts e0 .. e0 + PL - 1; -inf for a NaN (an expert that is not
// there) and past the last. No branch around a load: each would be waited for by
// itself; experts past the last read the last one's.
template <int PL, bool BF16>
__device__ __forceinline__ void load_logits(const RouteArgs& p, int64_t row, int e0, float (&l)[PL]) {
  constexpr int V = BF16 ? 8 : 4;  // logits of 16 bytes
  if (PL % V == 0 && p.wide && e0 + PL <= p.E) {
    if constexpr (PL % V == 0) {
      uint4 w[PL / V];
#pragma unroll
      for (int i = 0; i < PL / V; ++i)
        w[i] = reinterpret_cast<const uint4*>(static_cast<const char*>(p.logits) + (row + e0) * (BF16 ? 2 : 4))[i];
#pragma unroll
      for (int i = 0; i < PL; ++i) {
        const uint32_t d[4] = {w[i / V].x, w[i / V].y, w[i / V].z, w[i / V].w};
        const uint32_t u = BF16 ? (i & 1 ? d[i % V / 2] & 0xffff0000u : d[i % V / 2] << 16) : d[i % V % 4];
        l[i] = __uint_as_float(u);
      }
    }
  } else {
#pragma unroll
    for (int i = 0; i < PL; ++i) l[i] = load_value<BF16>(p.logits, row + min(e0 + i, p.E - 1));
  }
#pragma unroll
  for (int i = 0; i < PL; ++i) l[i] = e0 + i < p.E && l[i] == l[i] ? l[i] : -INFINITY;
}

// e^(x - m), m the largest logit: an infinite one's experts share the weight,
// and with no finite logit at all every score is 0.
__device__ __forceinline__ double score_part(float x, float m) {
  return x == m ? (m == -INFINITY ? 0.0 : 1.0) : exp((double)x - (double)m);
}
__device__ __forceinline__ double sigmoid64(float x) { return 1.0 / (1.0 + exp(-(double)x)); }
// s (1 - s) from the exponential, in which 1 - s does not round away as s comes near 1.
__device__ __forceinline__ double sigmoid_slope64(float x) {
  const double t = exp(-fabs((double)x));
  return t / ((1.0 + t) * (1.0 + t));
}

// Scores of a token's experts in 64 bits (in 32 neighbouring ones would round to
// equal ones and the choice hang on them), with the largest logit m and one over
// the sum of their parts.
template <int L, int PL>
__device__ __forceinline__ void scores_of(const float (&l)[PL], bool sigmoid, double (&s)[PL], float& m, double& inv) {
  m = -INFINITY;
  inv = 0.0;
  double part = 0.0;
  if (sigmoid) {
#pragma unroll
    for (int i = 0; i < PL; ++i) s[i] = sigmoid64(l[i]);
    return;
  }
#pragma unroll
  for (int i = 0; i < PL; ++i) m = fmaxf(m, l[i]);
  m = max_token<L>(m);
#pragma unroll
  for (int i = 0; i < PL; ++i) {
    s[i] = score_part(l[i], m);
    part += s[i];
  }
  const double sum = sum_token<L>(part);
  inv = sum > 0.0 ? 1.0 / sum : 0.0;
#pragma unroll
  for (int i = 0; i < PL; ++i) s[i] *= inv;
}
// The same of one logit.
__device__ __forceinline__ double score_of(float x, bool sigmoid, float m, double inv) {
  x = x == x ? x : -INFINITY;
  return sigmoid ? sigmoid64(x) : score_part(x, m) * inv;
}

template <int L, int PL, bool BF16>
__global__ __launch_bounds__(256) void route_kernel(RouteArgs p) {
  constexpr int TPW = 64 / L, TPG = 256 / L;  // tokens of a wave and of the workgroup
  __shared__ int32_t chosen[TPG][kRouteMaxK];
  extern __shared__ double groups_lds[];      // with groups: E values and `groups` of them a token
  const int lane = threadIdx.x & 63, sub = lane % L, q = lane / L;
  const int slot = threadIdx.x / L;
  const int64_t t = (int64_t)blockIdx.x * TPG + slot;
  const bool live = t < p.T;  // (no barrier below: a wave works alone)
  const int e0 = sub * PL;
  float l[PL], bias[PL];
  const int64_t row = (live ? t : p.T - 1) * p.ld;
  if (!p.bias) {
#pragma unroll
    for (int i = 0; i < PL; ++i) bias[i] = 0.0f;
  } else if (p.wide && e0 + PL <= p.E) {
#pragma unroll
    for (int i = 0; i < PL; i += 4) {
      const float4 b = *reinterpret_cast<const float4*>(p.bias + e0 + i);
      bias[i] = b.x;
      bias[i + 1] = b.y;
      bias[i + 2] = b.z;
      bias[i + 3] = b.w;
    }
  } else {
#pragma unroll
    for (int i = 0; i < PL; ++i) bias[i] = p.bias[min(e0 + i, p.E - 1)];
  }
  load_logits<PL, BF16>(p, row, e0, l);
  float m;
  double inv;
  double s[PL];
  scores_of<L, PL>(l, p.sigmoid, s, m, inv);
#pragma unroll
  for (int i = 0; i < PL; ++i) {  // values from here on
    s[i] += (double)bias[i];
    if (!(s[i] == s[i])) s[i] = -INFINITY;
  }
  bool open = true;      // whether this lane's experts may be chosen, all of them
  uint64_t groups_open = ~0ull;  // or those of these groups
  const int size = p.E / p.groups;
  const int per = size / PL;  // lanes of a group
  if (p.groups > 1) {
    double* const value = groups_lds + slot * (p.E + p.groups);
    double* const best = value + p.E;
    // whole lanes, 1, 2, 4, 8 or 16 of them, to a group: its two largest by lane
    // exchanges (8191 tokens of 256 experts in 8 groups: 2.5 us less than
    // through LDS)
    if (size % PL == 0 && (per & (per - 1)) == 0 && per <= 16) {
      double a = -INFINITY, b = -INFINITY;
#pragma unroll
      for (int i = 0; i < PL; ++i) {
        b = fmax(b, fmin(a, s[i]));
        a = fmax(a, s[i]);
      }
      auto both = [&](auto step) {
        const double x = step(a), y = step(b);
        b = fmax(fmin(a, x), fmax(b, y));
        a = fmax(a, x);
      };
      // (each step's lanes hold one pair in every 1, 2, 4, 8: mirrors exchange them)
      if (per > 1) both([](double v) { return dpp_f64<0xb1>(v); });    // quad_perm 1 0 3 2
      if (per > 2) both([](double v) { return dpp_f64<0x4e>(v); });    // quad_perm 2 3 0 1
      if (per > 4) both([](double v) { return dpp_f64<0x141>(v); });   // row_half_mirror
      if (per > 8) both([](double v) { return dpp_f64<0x140>(v); });   // row_mirror
      double v = p.group_top > 1 && size > 1 ? a + b : a;
      if (!(v == v)) v = -INFINITY;
      const int g = e0 / size;
      if (g < p.groups && sub % per == 0) best[g] = v;
      wave_lds_sync();
      int before = 0;
      for (int h0 = 0; h0 < p.groups; h0 += 8) {
        double x[8];
#pragma unroll
        for (int h = 0; h < 8; ++h) x[h] = best[min(h0 + h, p.groups - 1)];
#pragma unroll
        for (int h = 0; h < 8; ++h)
          before += h0 + h < p.groups && (x[h] > v || (x[h] == v && h0 + h < g));
      }
      open = before < p.top_groups;
    } else {
#pragma unroll
      for (int i = 0; i < PL; ++i)
        if (e0 + i < p.E) value[e0 + i] = s[i];
      wave_lds_sync();
      for (int g = sub; g < p.groups; g += L) {
        double a = -INFINITY, b = -INFINITY;  // the group's two largest
        int j = g % size;                     // (groups start at different banks)
        for (int n = 0; n < size; ++n) {
          const double x = value[g * size + j];
          if (++j == size) j = 0;
          b = fmax(b, fmin(a, x));
          a = fmax(a, x);
        }
        double v = p.group_top > 1 && size > 1 ? a + b : a;
        if (!(v == v)) v = -INFINITY;
        best[g] = v;
      }
      wave_lds_sync();
      groups_open = 0;
      for (int g0 = 0; g0 < p.groups; g0 += L) {
        const int g = g0 + sub;
        int before = 0;  // groups before this one
        if (g < p.groups) {
          const double v = best[g];
          for (int h = 0; h < p.groups; ++h) {
            const double x = best[h];
            before += x > v || (x == v && h < g);
          }
        }
        uint64_t on = __ballot(g < p.groups && before < p.top_groups);
        if constexpr (L < 64) on = on >> (q * L) & ((1ull << L) - 1);
        groups_open |= on << g0;
      }
    }
  }
  // order keys in two halves; 0 where an expert cannot be chosen (any more)
  uint32_t hi[PL], lo[PL];
  {
    int g = e0 / size, left = size - (e0 - g * size);
#pragma unroll
    for (int i = 0; i < PL; ++i) {
      const uint64_t k = order_key(s[i]);
      const bool on = e0 + i < p.E && open && (groups_open >> min(g, 63) & 1);
      hi[i] = on ? (uint32_t)(k >> 32) : 0u;
      lo[i] = on ? (uint32_t)k : 0u;
      if (--left == 0) {
        left = size;
        ++g;
      }
    }
  }
  for (int j = 0; j < p.k; ++j) {
    uint32_t top = 0;
#pragma unroll
    for (int i = 0; i < PL; ++i) top = max(top, hi[i]);
    top = max_token_u32<L>(top);
    // the experts with that upper half: nearly always one of each token, which
    // is then the largest value's
    int at = -1, n = 0;
#pragma unroll
    for (int i = PL - 1; i >= 0; --i) {
      const bool same = hi[i] == top;
      n += same;
      at = same ? i : at;
    }
    const uint64_t lanes = __ballot(n > 0);
    bool one = __ballot(n > 1) == 0;
#pragma unroll
    for (int x = 0; x < TPW; ++x) {
      const uint64_t m = L < 64 ? lanes >> (x * (L % 64)) & ((1ull << (L % 64)) - 1) : lanes;
      one = one && (m & (m - 1)) == 0;
    }
    if (!one) {  // by the lower halves, then the lowest index
      uint32_t low = 0;
      at = -1;
#pragma unroll
      for (int i = PL - 1; i >= 0; --i) {
        const bool more = hi[i] == top && lo[i] >= low;
        low = more ? lo[i] : low;
        at = more ? i : at;
      }
      const uint32_t best = max_token_u32<L>(low);
      uint64_t equal = __ballot(at >= 0 && low == best);
      if constexpr (L < 64) equal = equal >> (q * L) & ((1ull << L) - 1);
      if (sub != __builtin_ctzll(equal)) at = -1;
    }
    if (at >= 0) {
#pragma unroll
      for (int i = 0; i < PL; ++i) hi[i] = i == at ? 0u : hi[i];
      chosen[slot][j] = e0 + at;
    }
  }
  wave_lds_sync();
  if (!live) return;
  // each lane the weights of places sub, sub + L, ..: from the logits again
  double w[(kRouteMaxK + L - 1) / L], total = 0.0;
  int id[(kRouteMaxK + L - 1) / L];
#pragma unroll
  for (int r = 0; r < (kRouteMaxK + L - 1) / L; ++r) {
    const int j = sub + r * L;
    w[r] = 0.0;
    if (j < p.k) {
      id[r] = chosen[slot][j];
      const float x = load_value<BF16>(p.logits, row + id[r]);
      w[r] = score_of(x, p.sigmoid, m, inv);
    }
    total += w[r];
  }
  if (p.renorm) {
    total = sum_token<L>(total);
#pragma unroll
    for (int r = 0; r < (kRouteMaxK + L - 1) / L; ++r) w[r] = total > 0.0 ? w[r] / total : 0.0;
  }
#pragma unroll
  for (int r = 0; r < (kRouteMaxK + L - 1) / L; ++r) {
    const int j = sub + r * L;
    if (j < p.k) {
      p.ids[t * p.k + j] = id[r];
      p.weights[t * p.k + j] = (float)(w[r] * (double)p.scale);
    }
  }
}

// With x the scores, d = scale dweights (renormalised: (d - sum x d / sum x) / sum
// x over the chosen ones) and g an expert's d, or 0:
//   dlogits = g x (1 - x)  (sigmoid),  x (g - sum x d)  (softmax; the sum is 0
//   where the weights are renormalised)
// The lanes of a token as above; the chosen experts' d go through LDS to the lanes
// that hold them. 65536 tokens of 64 experts (bf16, 4 of them) 17 us, 4096 of 160
// 6.0 us; with a whole wave a token, its exchanges through LDS, 42 and 8.6 us.
// Without the exponentials in 64 bits it would be 5.3 and 1.5 us less, without the
// loop over the chosen 2.2 and 1.0; the 17 MB are 3.9 us.
template <int L, int PL, bool BF16>
__global__ __launch_bounds__(256) void route_backward_kernel(RouteArgs p) {
  constexpr int TPG = 256 / L, PER = (kRouteMaxK + L - 1) / L;
  __shared__ __attribute__((aligned(16))) double chosen[TPG][kRouteMaxK][2];  // d, and the id's bits
  const int sub = threadIdx.x % L, slot = threadIdx.x / L;
  const int64_t t = (int64_t)blockIdx.x * TPG + slot;
  const bool live = t < p.T;  // (no barrier below: a wave works alone)
  const int64_t tok = live ? t : p.T - 1;
  const int e0 = sub * PL;
  // places sub, sub + L, ..: ids and gradients; then the logits
  int id[PER];
  double d[PER], x[PER];
#pragma unroll
  for (int r = 0; r < PER; ++r) {
    const int j = min(sub + r * L, p.k - 1);
    id[r] = p.ids[tok * p.k + j];
    d[r] = (double)p.dweights[tok * p.k + j] * (double)p.scale;
    if (sub + r * L >= p.k || (uint32_t)id[r] >= (uint32_t)p.E) id[r] = -1;
  }
  float l[PL];
  const int64_t row = tok * p.ld;
  load_logits<PL, BF16>(p, row, e0, l);
  float at[PER];
#pragma unroll
  for (int r = 0; r < PER; ++r) at[r] = load_value<BF16>(p.logits, row + max(id[r], 0));
  float m = 0.0f;
  double inv = 0.0;
  double s[PL];  // scores, of sigmoid their slopes
  if (p.sigmoid) {
#pragma unroll
    for (int i = 0; i < PL; ++i) s[i] = sigmoid_slope64(l[i]);
  } else {
    scores_of<L, PL>(l, false, s, m, inv);
  }
  double total = 0.0, dot = 0.0;
#pragma unroll
  for (int r = 0; r < PER; ++r) {
    x[r] = 0.0;
    if (id[r] < 0) d[r] = 0.0;
    else x[r] = score_of(at[r], p.sigmoid, m, inv);
    total += x[r];
    dot += x[r] * d[r];
  }
  dot = sum_token<L>(dot);
  if (p.renorm) {
    total = sum_token<L>(total);
#pragma unroll
    for (int r = 0; r < PER; ++r) d[r] = total > 0.0 ? (d[r] - dot / total) / total : 0.0;
    dot = 0.0;
  }
#pragma unroll
  for (int r = 0; r < PER; ++r)
    if (sub + r * L < p.k) {
      chosen[slot][sub + r * L][0] = d[r];
      chosen[slot][sub + r * L][1] = __builtin_bit_cast(double, (int64_t)id[r]);
    }
  wave_lds_sync();
  double g[PL];
#pragma unroll
  for (int i = 0; i < PL; ++i) g[i] = 0.0;
  for (int j = 0; j < p.k; ++j) {  // (in the order of j: an id that comes twice counts twice)
    const double v = chosen[slot][j][0];
    const int e = (int)__builtin_bit_cast(int64_t, chosen[slot][j][1]) - e0;
#pragma unroll
    for (int i = 0; i < PL; ++i)
      if (e == i) g[i] += v;
  }
  float out[PL];
#pragma unroll
  for (int i = 0; i < PL; ++i) out[i] = (float)(p.sigmoid ? g[i] * s[i] : s[i] * (g[i] - dot));
  if (!live) return;
  constexpr int V = BF16 ? 8 : 4;
  char* const o = static_cast<char*>(p.dlogits) + (t * p.ldd + e0) * (BF16 ? 2 : 4);
  if (PL % V == 0 && p.wide && e0 + PL <= p.E) {
    if constexpr (PL % V == 0) {
#pragma unroll
      for (int i = 0; i < PL; i += V) {
        if constexpr (BF16)
          *reinterpret_cast<uint4*>(o + 2 * i) =
              make_uint4(pack_bf16x2(out[i], out[i + 1]), pack_bf16x2(out[i + 2], out[i + 3]),
                         pack_bf16x2(out[i + 4], out[i + 5]), pack_bf16x2(out[i + 6], out[i + 7]));
        else *reinterpret_cast<float4*>(o + 4 * i) = make_float4(out[i], out[i + 1], out[i + 2], out[i + 3]);
      }
    }
  } else {
#pragma unroll
    for (int i = 0; i < PL; ++i)
      if (e0 + i < p.E) {
        if constexpr (BF16) reinterpret_cast<uint16_t*>(o)[i] = f32_to_bf16(out[i]);
        else reinterpret_cast<float*>(o)[i] = out[i];
      }
  }
}

// --- places
// A counting sort that is stable, so that results are the same every run: 1024
// entries a workgroup and round, first their counts by expert (place_count_kernel;
// a single workgroup counts for itself), then the places. Bound by latency: 2 to
// 5 us and 6.5 us for 65536 entries of 256 experts, of which the bytes are 0.2 us.

// Entries of the workgroup's chunk by expert.
__global__ __launch_bounds__(1024) void place_count_kernel(PlaceArgs p) {
  __shared__ int32_t count[kRouteMaxE];
  for (int e = threadIdx.x; e < p.E; e += 1024) count[e] = 0;
  __syncthreads();
  const int64_t n0 = (int64_t)blockIdx.x * p.rounds * 1024;
  for (int r = 0; r < p.rounds; ++r) {
    const int64_t n = n0 + r * 1024 + threadIdx.x;
    if (n < p.n) {
      const int64_t e = (int64_t)p.ids[n] - p.first;
      if (e >= 0 && e < p.E) atomicAdd(&count[e], 1);
    }
  }
  __syncthreads();
  for (int e = threadIdx.x; e < p.E; e += 1024) p.hist[(int64_t)blockIdx.x * p.E + e] = count[e];
}

// Each entry's place: entries of earlier experts, of its expert in earlier
// chunks, and of its expert before it in this chunk (1024 at a time: in
// earlier waves, in earlier lanes). Lanes of one expert find each other by a
// ballot for each bit of its number.
__global__ __launch_bounds__(1024) void place_kernel(PlaceArgs p) {
  __shared__ int32_t cnt[16][kRouteMaxE];
  __shared__ int32_t next[kRouteMaxE];  // first free place of each expert in this chunk
  __shared__ int32_t wave_sum[16];
  const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
  const int64_t n0 = (int64_t)blockIdx.x * p.rounds * 1024;
  int before = 0, all = 0;
  int id = n0 + tid < p.n ? p.ids[n0 + tid] : -1;  // of the first round
  if (p.chunks > 1) {
    // the threads of a power of two at least E take the chunks in turn, 16
    // loads in flight each
    const int bits = max(6, 32 - __builtin_clz(max(p.E - 1, 1))), parts = 1024 >> bits;
    const int e = tid & ((1 << bits) - 1);
    if (e < p.E)
      for (int c0 = tid >> bits; c0 < p.chunks; c0 += 16 * parts) {
        int h[16];
#pragma unroll
        for (int i = 0; i < 16; ++i) {
          const int c = c0 + parts * i;
          h[i] = c < p.chunks ? p.hist[(int64_t)c * p.E + e] : 0;
        }
#pragma unroll
        for (int i = 0; i < 16; ++i) {
          before += c0 + parts * i < (int)blockIdx.x ? h[i] : 0;
          all += h[i];
        }
      }
    cnt[0][tid] = before;
    cnt[1][tid] = all;
    __syncthreads();
    before = all = 0;
    if (tid < p.E)
      for (int q = 0; q < parts; ++q) {
        before += cnt[0][(q << bits) + tid];
        all += cnt[1][(q << bits) + tid];
      }
    __syncthreads();
  } else {
    next[tid] = 0;
    __syncthreads();
    for (int r = 0; r < p.rounds; ++r) {
      const int64_t n = n0 + r * 1024 + tid;
      if (n < p.n) {
        const int64_t e = (int64_t)p.ids[n] - p.first;
        if (e >= 0 && e < p.E) atomicAdd(&next[e], 1);
      }
    }
    __syncthreads();
    all = tid < p.E ? next[tid] : 0;
    __syncthreads();
  }
  int incl = all;
#pragma unroll
  for (int d = 1; d < 64; d *= 2) {
    const int up = __shfl_up(incl, d, 64);
    if (lane >= d) incl += up;
  }
  if (lane == 63) wave_sum[wave] = incl;
  __syncthreads();
  int base = 0, live = 0;
  for (int w = 0; w < 16; ++w) {
    base += w < wave ? wave_sum[w] : 0;
    live += wave_sum[w];
  }
  const int start = base + incl - all;
  if (tid < p.E) next[tid] = start + before;
  if (blockIdx.x == 0) {
    if (tid < p.E) p.offsets[tid] = start;
    if (tid == 0) p.offsets[p.E] = live;
  }
  for (int r = 0; r < p.rounds; ++r) {
    const int64_t n = n0 + r * 1024 + tid;
    const int64_t x = (int64_t)id - p.first;
    const int e = n < p.n && x >= 0 && x < p.E ? (int)x : -1;
    if (n + 1024 < p.n) id = p.ids[n + 1024];
    for (int i = lane; i < p.E; i += 64) cnt[wave][i] = 0;
    __syncthreads();
    uint64_t same = __ballot(e >= 0);  // lanes of this wave with this expert
#pragma unroll
    for (int b = 0; b < 10; ++b) {
      const uint64_t on = __ballot((e >> b) & 1);
      same &= (e >> b) & 1 ? on : ~on;
    }
    const int rank = __popcll(same & ((1ull << lane) - 1));
    if (e >= 0 && rank == 0) cnt[wave][e] = __popcll(same);
    __syncthreads();
    if (tid < p.E) {
      int at = next[tid], c[16];
#pragma unroll
      for (int w = 0; w < 16; ++w) c[w] = cnt[w][tid];
#pragma unroll
      for (int w = 0; w < 16; ++w) {
        cnt[w][tid] = at;
        at += c[w];
      }
      next[tid] = at;
    }
    __syncthreads();
    if (n < p.n) {
      const int at = e >= 0 ? cnt[wave][e] + rank : -1;
      if (p.places) p.places[n] = at;
      if (p.rows) {
        if (e >= 0) p.rows[at] = (int)(n / p.k);
        if (n >= live) p.rows[n] = -1;
      }
    }
    __syncthreads();
  }
}

// --- sums of the experts' rows
// Bound by reading Z once: eight columns of a token per thread, eight of its rows
// in flight at a time (two: 98 us, all eight: 88 us for 8191 tokens of 8 rows of
// 4096, a quarter of them absent, 5.4 TB/s), past the caches, since no row is
// read twice.
template <bool BF16>
__global__ __launch_bounds__(256) void combine_kernel(CombineArgs p) {
  const int per = (p.N + 7) / 8;
  const int64_t at = (int64_t)blockIdx.x * 256 + threadIdx.x;
  const int64_t t = at / per;
  const int c = (int)(at - t * per) * 8;
  if (t >= p.T) return;
  const bool full = c + 8 <= p.N;
  float y[8];
#pragma unroll
  for (int e = 0; e < 8; ++e) y[e] = 0.0f;
  for (int j0 = 0; j0 < p.k; j0 += 8) {
    uint4 v[8];
    float w[8];
    bool on[8];
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      const int row = j0 + j < p.k ? p.places[t * p.k + j0 + j] : -1;
      on[j] = (uint32_t)row < (uint32_t)p.z_rows;
      w[j] = on[j] && p.weights ? p.weights[t * p.k + j0 + j] : 1.0f;
      v[j] = make_uint4(0, 0, 0, 0);
      if (on[j]) {
        const uint16_t* z = p.Z + (int64_t)row * p.ldz;
        v[j] = full ? load16_stream(z + c) : load8_masked(z, c, p.N);
      }
    }
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      if (!on[j]) continue;  // (a weight that is not finite counts for its place only)
      const uint32_t d[4] = {v[j].x, v[j].y, v[j].z, v[j].w};
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        y[2 * e] = fmaf(w[j], __uint_as_float(d[e] << 16), y[2 * e]);
        y[2 * e + 1] = fmaf(w[j], __uint_as_float(d[e] & 0xffff0000u), y[2 * e + 1]);
      }
    }
  }
  if constexpr (BF16) {
    uint16_t* o = static_cast<uint16_t*>(p.Y) + t * p.ldy + c;
    if (full)
      *reinterpret_cast<uint4*>(o) = make_uint4(pack_bf16x2(y[0], y[1]), pack_bf16x2(y[2], y[3]),
                                                pack_bf16x2(y[4], y[5]), pack_bf16x2(y[6], y[7]));
    else
      for (int e = 0; e < 8; ++e)
        if (c + e < p.N) o[e] = f32_to_bf16(y[e]);
  } else {
    float* o = static_cast<float*>(p.Y) + t * p.ldy + c;
    if (full) {
      *reinterpret_cast<float4*>(o) = make_float4(y[0], y[1], y[2], y[3]);
      *reinterpret_cast<float4*>(o + 4) = make_float4(y[4], y[5], y[6], y[7]);
    } else {
      for (int e = 0; e < 8; ++e)
        if (c + e < p.N) o[e] = y[e];
    }
  }
}

// The kernel for E experts and the tokens of a workgroup.
template <bool BF16>
const void* route_of(int E, bool backward, int* tokens) {
#define TG_ROUTE(L, PL)                                                                 \
  {                                                                                     \
    *tokens = 256 / L;                                                                  \
    return backward ? reinterpret_cast<const void*>(&route_backward_kernel<L, PL, BF16>) \
                    : reinterpret_cast<const void*>(&route_kernel<L, PL, BF16>);        \
  }
  if (E <= 64) TG_ROUTE(16, 4);
  if (E <= 128) TG_ROUTE(16, 8);
  if (E <= 256) TG_ROUTE(32, 8);
  if (E <= 512) TG_ROUTE(64, 8);
  TG_ROUTE(64, 16);
#undef TG_ROUTE
}

template <typename Args>
hipError_t launch_with_lds(const void* fn, dim3 grid, dim3 block, size_t lds, const Args& args, hipStream_t stream) {
  void* argv[] = {const_cast<Args*>(&args)};
  return hipLaunchKernel(fn, grid, block, argv, lds, stream);
}

}  // namespace

hipError_t launch_route(const RouteArgs& a, bool bf16, hipStream_t stream) {
  int tokens;
  const void* fn = bf16 ? route_of<true>(a.E, false, &tokens) : route_of<false>(a.E, false, &tokens);
  const size_t lds = a.groups > 1 ? (size_t)tokens * (a.E + a.groups) * sizeof(double) : 0;
  return launch_with_lds(fn, dim3((unsigned)ceil_div(a.T, tokens)), dim3(256), lds, a, stream);
}

hipError_t launch_route_backward(const RouteArgs& a, bool bf16, hipStream_t stream) {
  int tokens;
  const void* fn = bf16 ? route_of<true>(a.E, true, &tokens) : route_of<false>(a.E, true, &tokens);
  return launch_raw(fn, dim3((unsigned)ceil_div(a.T, tokens)), dim3(256), a, stream);
}

hipError_t launch_place(const PlaceArgs& a, hipStream_t stream) {
  if (a.chunks > 1) {
    const hipError_t e = launch_raw(reinterpret_cast<const void*>(&place_count_kernel), dim3((unsigned)a.chunks),
                                    dim3(1024), a, stream);
    if (e != hipSuccess) return e;
  }
  return launch_raw(reinterpret_cast<const void*>(&place_kernel), dim3((unsigned)a.chunks), dim3(1024), a, stream);
}

hipError_t launch_combine(const CombineArgs& a, bool bf16, hipStream_t stream) {
  const int64_t threads = (int64_t)a.T * ceil_div(a.N, 8);
  const void* fn = bf16 ? reinterpret_cast<const void*>(&combine_kernel<true>)
                        : reinterpret_cast<const void*>(&combine_kernel<false>);
  return launch_raw(fn, dim3((unsigned)ceil_div(threads, 256)), dim3(256), a, stream);
}

}  // namespace tg
