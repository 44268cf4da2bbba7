// kernels_quant.hip -- bf16 values to E4M3 with a float32 scale for every 128
// values of a row, or for every 128 x 128 block.
#include "block_launch.hpp"
#include "train_epilogue.hpp"

namespace tg {

namespace {

constexpr float kE4m3Max = 448.0f;
// magnitudes below this count as it: scales stay normal numbers and a block
// of zeros has one too
constexpr uint32_t kLeastBits = 0x0d800000u;  // 2^-100

// The largest of the 16 lanes of a row of lanes, in all of them.
__device__ __forceinline__ uint32_t max_row16(uint32_t v) {
  v = max(v, (uint32_t)__builtin_amdgcn_update_dpp(0, (int)v, 0x128, 0xf, 0xf, false));  // row_ror:8
  v = max(v, (uint32_t)__builtin_amdgcn_update_dpp(0, (int)v, 0x124, 0xf, 0xf, false));
  v = max(v, (uint32_t)__builtin_amdgcn_update_dpp(0, (int)v, 0x122, 0xf, 0xf, false));
  v = max(v, (uint32_t)__builtin_amdgcn_update_dpp(0, (int)v, 0x121, 0xf, 0xf, false));
  return v;
}

__device__ __forceinline__ void unpack8(const uint4& v, float (&x)[8]) {
  const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
  for (int e = 0; e < 4; ++e) {
    x[2 * e] = __builtin_bit_cast(float, w[e] << 16);
    x[2 * e + 1] = __builtin_bit_cast(float, w[e] & 0xffff0000u);
  }
}

// The largest magnitude's bits: as integers, infinity and NaN are above every number.
__device__ __forceinline__ uint32_t max_bits(const float (&x)[8]) {
  uint32_t m = 0;
#pragma unroll
  for (int e = 0; e < 8; ++e) m = max(m, __builtin_bit_cast(uint32_t, x[e]) & 0x7fffffffu);
  return m;
}

__device__ __forceinline__ uint2 codes8(const float (&x)[8], float r) {
  uint32_t w[2];
#pragma unroll
  for (int h = 0; h < 2; ++h) {
    int v = __builtin_amdgcn_cvt_pk_fp8_f32(x[4 * h] * r, x[4 * h + 1] * r, 0, false);
    v = __builtin_amdgcn_cvt_pk_fp8_f32(x[4 * h + 2] * r, x[4 * h + 3] * r, v, true);
    w[h] = (uint32_t)v;
  }
  return make_uint2(w[0], w[1]);
}

// act(z) of a bf16 value. gelu is z Q(-z), Q the normal distribution's upper tail,
// Q(z) = e^(-z^2 / 2) R(z / sqrt 2) / 2 for z >= 0 with R(x) = e^(x^2) erfc(x): a
// block's scale may hang on values far out on the tail, which have to be right
// relative to themselves (gate_both's are off by up to 1e-7 of 1, 1.5% of the value
// at -9). R is a polynomial of degree 7 in t =
// 1 / (1 + 0.45 x) times t, fitted for the least relative error (3e-7, for x up
// to 9.5) to 64-bit values; z^2 is exact. 8192 x 3584 34 us, 33 with gate_both's.
template <int GATE>
__device__ __forceinline__ float gate_of(float z) {
  if constexpr (GATE == kGateGelu) {
    const float t = __builtin_amdgcn_rcpf(fmaf(0.31819805153394637f, fabsf(z), 1.0f));
    float r = 0.5f * 0.06631969151f;
    r = fmaf(r, t, 0.5f * -0.2378895656f);
    r = fmaf(r, t, 0.5f * 0.2045545914f);
    r = fmaf(r, t, 0.5f * 0.04441020492f);
    r = fmaf(r, t, 0.5f * 0.1863791616f);
    r = fmaf(r, t, 0.5f * 0.2287909009f);
    r = fmaf(r, t, 0.5f * 0.253518495f);
    r = fmaf(r, t, 0.5f * 0.2539168146f);
    const float q = r * (t * __builtin_amdgcn_exp2f(z * z * -0.72134752044448171f));
    return z * (z < 0.0f ? q : 1.0f - q);
  } else {
    float act, slope;
    gate_both<GATE>(z, act, slope);
    return act;
  }
}

// q = x (448 / a), scale = a / 448, a the block's largest magnitude: one pass, the
// values held in registers between the maximum and the codes. Bound by memory.
// 16 lanes hold one block of a row, 8 values each, their maximum by four lane
// exchanges; a wave takes 4 rows, whose loads are all out before the first is
// used, a workgroup 16 rows x 512 columns, so that the scales of its 16 rows leave
// as 64 bytes together. 8192 x 7168 bf16 32 us (5.5 TB/s, a large copy reaches
// 4.8); gated 8192 x 3584 28 us (5.3 TB/s), the first half of the pair never
// written as bf16.
template <int GATE>
__global__ __launch_bounds__(256) void quant_rows_kernel(QuantArgs p) {
  __shared__ float sc[4][16];
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  const int col = (int)blockIdx.x * 512 + lane * 8;
  const int row0 = (int)blockIdx.y * 16 + wave * 4;
  const bool in = col < p.K;
  int src[4];
  bool live[4];
#pragma unroll
  for (int r = 0; r < 4; ++r) {
    const int row = row0 + r;
    src[r] = row;
    live[r] = row < p.M;
    if (p.rows && live[r]) {
      src[r] = p.rows[row];
      live[r] = (uint32_t)src[r] < (uint32_t)p.x_rows;
    }
  }
  uint4 v[4], u[4];
#pragma unroll
  for (int r = 0; r < 4; ++r) {
    v[r] = u[r] = make_uint4(0, 0, 0, 0);
    if (live[r] && in) {
      const uint16_t* x = p.X + (int64_t)src[r] * p.ldx + col;
      v[r] = *reinterpret_cast<const uint4*>(x);
      if constexpr (GATE >= 0) u[r] = *reinterpret_cast<const uint4*>(x + p.K);
    }
  }
#pragma unroll
  for (int r = 0; r < 4; ++r) {
    float x[8];
    unpack8(v[r], x);
    if constexpr (GATE >= 0) {
      float y[8];
      unpack8(u[r], y);
#pragma unroll
      for (int e = 0; e < 8; ++e) x[e] = gate_of<GATE>(x[e]) * y[e];
    }
    const uint32_t top = max(max_row16(max_bits(x)), kLeastBits);
    const float t = __builtin_bit_cast(float, top);
    const uint2 c = codes8(x, kE4m3Max / t);
    if (live[r] && in) *reinterpret_cast<uint2*>(p.Q + (int64_t)(row0 + r) * p.ldq + col) = c;
    if ((lane & 15) == 0) sc[lane >> 4][wave * 4 + r] = live[r] ? t / kE4m3Max : -1.0f;
  }
  __syncthreads();
  if (threadIdx.x < 64) {
    const int b = (int)blockIdx.x * 4 + (threadIdx.x >> 4), row = (int)blockIdx.y * 16 + (threadIdx.x & 15);
    const float s = sc[threadIdx.x >> 4][threadIdx.x & 15];
    // (a row that is not written keeps its scales: no scale is negative)
    if (b * kScaleBlock < p.K && row < p.M && !(s < 0.0f)) p.scale[(int64_t)b * p.lds + row] = s;
  }
}

// A workgroup takes one 128 x 128 block, held in registers: 16 lanes a row,
// 16 rows at a time, 8 loads in flight each. 7168 x 8192 35 us (5.1 TB/s): done
// once for a weight.
__global__ __launch_bounds__(256) void quant_blocks_kernel(QuantArgs p) {
  __shared__ uint32_t tops[4];
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  const int col = (int)blockIdx.x * 128 + (lane & 15) * 8;
  const int row0 = (int)blockIdx.y * 128 + (int)(threadIdx.x >> 4);
  const bool in = col < p.K;
  uint4 v[8];
#pragma unroll
  for (int r = 0; r < 8; ++r) {
    const int row = row0 + 16 * r;
    v[r] = make_uint4(0, 0, 0, 0);
    if (in && row < p.M) v[r] = *reinterpret_cast<const uint4*>(p.X + (int64_t)row * p.ldx + col);
  }
  uint32_t top = kLeastBits;
#pragma unroll
  for (int r = 0; r < 8; ++r) {
    float x[8];
    unpack8(v[r], x);
    top = max(top, max_bits(x));
  }
  top = max_row16(top);
  top = max(top, (uint32_t)__shfl_xor((int)top, 16, 64));
  top = max(top, (uint32_t)__shfl_xor((int)top, 32, 64));
  if (lane == 0) tops[wave] = top;
  __syncthreads();
  top = max(max(tops[0], tops[1]), max(tops[2], tops[3]));
  const float t = __builtin_bit_cast(float, top), inv = kE4m3Max / t;
#pragma unroll
  for (int r = 0; r < 8; ++r) {
    float x[8];
    unpack8(v[r], x);
    const int row = row0 + 16 * r;
    if (in && row < p.M) *reinterpret_cast<uint2*>(p.Q + (int64_t)row * p.ldq + col) = codes8(x, inv);
  }
  if (threadIdx.x == 0) p.scale[(int64_t)blockIdx.y * p.lds + blockIdx.x] = t / kE4m3Max;
}

}  // namespace

hipError_t launch_quant_rows(const QuantArgs& a, int gate, hipStream_t stream) {
  const dim3 grid((unsigned)ceil_div(a.K, 512), (unsigned)ceil_div(a.M, 16));
  const void* fn = reinterpret_cast<const void*>(&quant_rows_kernel<-1>);
  switch (gate) {
    case kGateSilu: fn = reinterpret_cast<const void*>(&quant_rows_kernel<kGateSilu>); break;
    case kGateGelu: fn = reinterpret_cast<const void*>(&quant_rows_kernel<kGateGelu>); break;
    case kGateGeluTanh: fn = reinterpret_cast<const void*>(&quant_rows_kernel<kGateGeluTanh>); break;
    case kGateRelu: fn = reinterpret_cast<const void*>(&quant_rows_kernel<kGateRelu>); break;
    case kGateSigmoid: fn = reinterpret_cast<const void*>(&quant_rows_kernel<kGateSigmoid>); break;
  }
  return launch_raw(fn, grid, dim3(256), a, stream);
}

hipError_t launch_quant_blocks(const QuantArgs& a, hipStream_t stream) {
  const dim3 grid((unsigned)ceil_div(a.K, 128), (unsigned)ceil_div(a.M, 128));
  return launch_raw(reinterpret_cast<const void*>(&quant_blocks_kernel), grid, dim3(256), a, stream);
}

}  // namespace tg
