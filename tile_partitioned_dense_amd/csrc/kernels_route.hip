// kernels_route.hip -- routing to experts: scores, choice and weights of each
// token, their gradient, the order of the tokens by expert, and the weighted
// sum of the experts' rows.
#include "block_launch.hpp"

namespace tg {

namespace {

constexpr int kRouteMaxE = 1024;

template <bool BF16>
__device__ __forceinline__ float load_logit(const void* p, int64_t i) {
  float v;
  if constexpr (BF16) v = __builtin_bit_cast(float, (uint32_t) static_cast<const uint16_t*>(p)[i] << 16);
  else v = static_cast<const float*>(p)[i];
  return v == v ? v : -INFINITY;  // NaN: an expert that is not there
}

__device__ __forceinline__ double shfl_xor_f64(double v, int m) { return __shfl_xor(v, m, 64); }

// Scores of a wave's token in 64 bits; expert lane + 64 i in s[i]. In 32 bits
// neighbouring scores would round to equal ones and the choice hang on them.
template <int PL>
__device__ __forceinline__ void scores_of(const float (&l)[PL], int E, int lane, bool sigmoid, double (&s)[PL]) {
  if (sigmoid) {
#pragma unroll
    for (int i = 0; i < PL; ++i) s[i] = 1.0 / (1.0 + exp(-(double)l[i]));
    return;
  }
  float m = -INFINITY;
#pragma unroll
  for (int i = 0; i < PL; ++i) m = fmaxf(m, l[i]);
#pragma unroll
  for (int d = 32; d > 0; d /= 2) m = fmaxf(m, __shfl_xor(m, d, 64));
  double sum = 0.0;
#pragma unroll
  for (int i = 0; i < PL; ++i) {
    // (an infinite largest logit: those experts share the weight; no finite
    // logit at all: every score is 0)
    s[i] = l[i] == m ? (m == -INFINITY ? 0.0 : 1.0) : exp((double)l[i] - (double)m);
    sum += s[i];
  }
#pragma unroll
  for (int d = 32; d > 0; d /= 2) sum += shfl_xor_f64(sum, d);
#pragma unroll
  for (int i = 0; i < PL; ++i) s[i] = sum > 0.0 ? s[i] / sum : 0.0;
}

template <int PL, bool BF16>
__global__ __launch_bounds__(256) void route_kernel(RouteArgs p) {
  extern __shared__ double val[];  // with groups: E values per wave
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  const int t = (int)blockIdx.x * 4 + wave;
  if (t >= p.T) return;  // (no barrier below: a wave works alone)
  float l[PL];
#pragma unroll
  for (int i = 0; i < PL; ++i) {
    const int e = lane + 64 * i;
    l[i] = e < p.E ? load_logit<BF16>(p.logits, (int64_t)t * p.ld + e) : -INFINITY;
  }
  double s[PL], v[PL];
  scores_of<PL>(l, p.E, lane, p.sigmoid, s);
  uint32_t open = 0;  // experts of this lane that may still be chosen
#pragma unroll
  for (int i = 0; i < PL; ++i) {
    const int e = lane + 64 * i;
    v[i] = s[i];
    if (e < p.E) {
      open |= 1u << i;
      if (p.bias) v[i] += (double)p.bias[e];
      if (!(v[i] == v[i])) v[i] = -INFINITY;
    }
  }
  if (p.groups > 1) {
    double* mine = val + wave * p.E;
    const int size = p.E / p.groups;
#pragma unroll
    for (int i = 0; i < PL; ++i)
      if (lane + 64 * i < p.E) mine[lane + 64 * i] = v[i];
    __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");  // (other lanes read them)
    __builtin_amdgcn_wave_barrier();
    double a = -INFINITY, b = -INFINITY;  // the group's two largest
    if (lane < p.groups)
      for (int j = 0; j < size; ++j) {
        const double x = mine[lane * size + j];
        if (x > a) { b = a; a = x; }
        else if (x > b) b = x;
      }
    double best = p.group_top > 1 && size > 1 ? a + b : a;
    if (!(best == best)) best = -INFINITY;
    int better = 0;  // groups before this one
    for (int g = 0; g < p.groups; ++g) {
      const double x = __shfl(best, g, 64);
      better += x > best || (x == best && g < lane);
    }
    const uint64_t chosen = __ballot(lane < p.groups && better < p.top_groups);
#pragma unroll
    for (int i = 0; i < PL; ++i)
      if (!((chosen >> ((lane + 64 * i) / size)) & 1)) open &= ~(1u << i);
  }
  double total = 0.0, w = 0.0;
  int id = 0;
  for (int j = 0; j < p.k; ++j) {
    double bv = -INFINITY, bs = 0.0;
    int be = 0x7fffffff;
#pragma unroll
    for (int i = 0; i < PL; ++i) {
      const int e = lane + 64 * i;
      if ((open >> i & 1) && (be == 0x7fffffff || v[i] > bv)) {
        bv = v[i];
        bs = s[i];
        be = e;
      }
    }
#pragma unroll
    for (int d = 32; d > 0; d /= 2) {
      const double ov = shfl_xor_f64(bv, d), os = shfl_xor_f64(bs, d);
      const int oe = __shfl_xor(be, d, 64);
      if (ov > bv || (ov == bv && oe < be)) {
        bv = ov;
        bs = os;
        be = oe;
      }
    }
    if ((be & 63) == lane) open &= ~(1u << (be >> 6));
    total += bs;
    if (lane == j) {
      w = bs;
      id = be;
    }
  }
  if (lane < p.k) {
    if (p.renorm) w = total > 0.0 ? w / total : 0.0;
    p.ids[(int64_t)t * p.k + lane] = id;
    p.weights[(int64_t)t * p.k + lane] = (float)(w * (double)p.scale);
  }
}

template <int PL, bool BF16>
__global__ __launch_bounds__(256) void route_backward_kernel(RouteArgs p) {
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  const int t = (int)blockIdx.x * 4 + wave;
  if (t >= p.T) return;
  float l[PL];
#pragma unroll
  for (int i = 0; i < PL; ++i) {
    const int e = lane + 64 * i;
    l[i] = e < p.E ? load_logit<BF16>(p.logits, (int64_t)t * p.ld + e) : -INFINITY;
  }
  double s[PL];
  scores_of<PL>(l, p.E, lane, p.sigmoid, s);
  int id = -1;
  double d = 0.0;
  if (lane < p.k) {
    id = p.ids[(int64_t)t * p.k + lane];
    if ((uint32_t)id >= (uint32_t)p.E) id = -1;
    else d = (double)p.dweights[(int64_t)t * p.k + lane] * (double)p.scale;
  }
  // the chosen scores, and with renormalised weights the gradient through their sum
  double total = 0.0, dot = 0.0;
  for (int j = 0; j < p.k; ++j) {
    const int e = __shfl(id, j, 64);
    if (e < 0) continue;
    double x = 0.0;
#pragma unroll
    for (int i = 0; i < PL; ++i)
      if (i == (e >> 6)) x = s[i];
    x = __shfl(x, e & 63, 64);
    total += x;
    dot += x * __shfl(d, j, 64);
  }
  if (p.renorm) {
    d = total > 0.0 ? (d - dot / total) / total : 0.0;
    dot = 0.0;  // (of the new gradients and the scores: their mean is taken out)
  }
  double g[PL];
#pragma unroll
  for (int i = 0; i < PL; ++i) g[i] = 0.0;
  for (int j = 0; j < p.k; ++j) {
    const int e = __shfl(id, j, 64);
    const double x = __shfl(d, j, 64);
    if (e < 0) continue;
#pragma unroll
    for (int i = 0; i < PL; ++i)
      if (e == lane + 64 * i) g[i] += x;
  }
#pragma unroll
  for (int i = 0; i < PL; ++i) {
    const int e = lane + 64 * i;
    if (e >= p.E) continue;
    const double r = p.sigmoid ? g[i] * s[i] * (1.0 - s[i]) : s[i] * (g[i] - dot);
    if constexpr (BF16) static_cast<uint16_t*>(p.dlogits)[(int64_t)t * p.ldd + e] = f32_to_bf16((float)r);
    else static_cast<float*>(p.dlogits)[(int64_t)t * p.ldd + e] = (float)r;
  }
}

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
// earlier waves, in earlier lanes).
__global__ __launch_bounds__(1024) void place_kernel(PlaceArgs p) {
  __shared__ int32_t cnt[16][kRouteMaxE];
  __shared__ int32_t next[kRouteMaxE];  // first free place of each expert in this chunk
  __shared__ int32_t wave_sum[16];
  const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
  const int64_t n0 = (int64_t)blockIdx.x * p.rounds * 1024;
  int before = 0, all = 0;
  if (p.chunks > 1) {
    if (tid < p.E)
      for (int c = 0; c < p.chunks; ++c) {
        const int h = p.hist[(int64_t)c * p.E + tid];
        before += c < (int)blockIdx.x ? h : 0;
        all += h;
      }
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
    for (int w = 0; w < 16; ++w)
      if (tid < p.E) cnt[w][tid] = 0;
    __syncthreads();
    const int64_t n = n0 + r * 1024 + tid;
    int e = -1;
    if (n < p.n) {
      const int64_t x = (int64_t)p.ids[n] - p.first;
      if (x >= 0 && x < p.E) e = (int)x;
    }
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
      int at = next[tid];
      for (int w = 0; w < 16; ++w) {
        const int c = cnt[w][tid];
        cnt[w][tid] = at;
        at += c;
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

// Eight columns of a token per thread.
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
#pragma unroll 4
  for (int j = 0; j < p.k; ++j) {
    const int at_j = p.places[t * p.k + j];
    if ((uint32_t)at_j >= (uint32_t)p.z_rows) continue;
    const float w = p.weights ? p.weights[t * p.k + j] : 1.0f;
    const uint16_t* z = p.Z + (int64_t)at_j * p.ldz + c;
    uint4 v;
    if (full) v = *reinterpret_cast<const uint4*>(z);
    else v = load8_masked(z - c, c, p.N);
    const uint32_t d[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      y[2 * e] = fmaf(w, __builtin_bit_cast(float, d[e] << 16), y[2 * e]);
      y[2 * e + 1] = fmaf(w, __builtin_bit_cast(float, d[e] & 0xffff0000u), y[2 * e + 1]);
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

template <bool BF16>
const void* route_of(int E, bool backward) {
#define TG_ROUTE(PL)                                                                  \
  return backward ? reinterpret_cast<const void*>(&route_backward_kernel<PL, BF16>) \
                  : reinterpret_cast<const void*>(&route_kernel<PL, BF16>)
  if (E <= 64) TG_ROUTE(1);
  if (E <= 128) TG_ROUTE(2);
  if (E <= 256) TG_ROUTE(4);
  if (E <= 512) TG_ROUTE(8);
  TG_ROUTE(16);
#undef TG_ROUTE
}

template <typename Args>
hipError_t launch_with_lds(const void* fn, dim3 grid, dim3 block, size_t lds, const Args& args, hipStream_t stream) {
  void* argv[] = {const_cast<Args*>(&args)};
  return hipLaunchKernel(fn, grid, block, argv, lds, stream);
}

}  // namespace

hipError_t launch_route(const RouteArgs& a, bool bf16, hipStream_t stream) {
  const size_t lds = a.groups > 1 ? (size_t)a.E * 4 * sizeof(double) : 0;
  return launch_with_lds(bf16 ? route_of<true>(a.E, false) : route_of<false>(a.E, false),
                         dim3((unsigned)ceil_div(a.T, 4)), dim3(256), lds, a, stream);
}

hipError_t launch_route_backward(const RouteArgs& a, bool bf16, hipStream_t stream) {
  return launch_raw(bf16 ? route_of<true>(a.E, true) : route_of<false>(a.E, true), dim3((unsigned)ceil_div(a.T, 4)),
                    dim3(256), a, stream);
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
