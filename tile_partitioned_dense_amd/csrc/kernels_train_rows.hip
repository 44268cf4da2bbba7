// kernels_train_rows.hip -- the small kernels around the training products:
// joining the segments of a softmax, per-row constants of its gradient, sums
// of partial results. All sums run in a fixed order.
#include "outer_kernel.hpp"
#include "train_launch.hpp"

namespace tg {

namespace {

// (m, s) of two disjoint sets of columns: s counts e^(l - m).
__device__ __forceinline__ void join(float& m, float& s, float m1, float s1) {
  const float hi = fmaxf(m, m1);
  // an empty side has m = -inf, s = 0: its factor is 0, unless both are empty
  const float a = m == hi ? 1.0f : __builtin_amdgcn_exp2f((m - hi) * kLog2e);
  const float b = m1 == hi ? 1.0f : __builtin_amdgcn_exp2f((m1 - hi) * kLog2e);
  s = s * a + s1 * b;
  m = hi;
}

// RB rows per workgroup, 256 / RB threads each walking a row's segments in
// steps, then a tree over the threads. RB = 16 reads whole 128-byte lines of
// the [segment][row] partials; RB = 1 gives few rows enough threads.
template <int RB>
__global__ __launch_bounds__(256) void xent_finish_kernel(FinishArgs p) {
  constexpr int Q = 256 / RB;
  __shared__ float sm[256], ss[256], st[256];
  const int r = threadIdx.x % RB, q = threadIdx.x / RB;
  const int64_t row = (int64_t)blockIdx.x * RB + r;
  float m = -INFINITY, s = 0.0f, total = 0.0f;
  if (row < p.M) {
#pragma unroll 8
    for (int g = q; g < p.segs; g += Q) {
      const float2 v = p.part[(int64_t)g * p.M + row];
      join(m, s, v.x, v.y);
    }
    if (p.part_sum)
      for (int g = q; g < p.segs; g += Q) total += p.part_sum[(int64_t)g * p.M + row];
  }
  sm[threadIdx.x] = m;
  ss[threadIdx.x] = s;
  st[threadIdx.x] = total;
  __syncthreads();
#pragma unroll
  for (int h = Q / 2; h > 0; h /= 2) {
    if (q < h) {
      join(m, s, sm[threadIdx.x + h * RB], ss[threadIdx.x + h * RB]);
      total += st[threadIdx.x + h * RB];
      sm[threadIdx.x] = m;
      ss[threadIdx.x] = s;
      st[threadIdx.x] = total;
    }
    __syncthreads();
  }
  if (q != 0 || row >= p.M) return;
  const float lse = m + logf(s);
  if (p.lse) p.lse[row] = lse;
  if (!p.loss) return;
  const int64_t t = target_of(p.target, p.target64, row);
  float loss = 0.0f;
  if (t != p.ignore) {
    if (t < 0 || t >= p.N) {
      loss = NAN;  // a target that is no column of the vocabulary
    } else {
      // m - hit first: both are near each other where the target is likely
      loss = (m - p.hit[row]) + logf(s);
      if (p.part_sum) loss += p.smoothing * (p.hit[row] - total / (float)p.N);
      loss += p.z_loss * lse * lse;
    }
  }
  p.loss[row] = loss;
}

// Constants of the gradient of every row, and the common factor of the loss
// gradients. G is held in bf16, where a loss gradient of, say, 1 / 1000 on
// every row would put one and the same rounding error on all of them; so the
// largest |dloss| is taken out (exactly 1 stays where they are equal) and
// multiplied onto the finished gradients in fp32 instead. Every workgroup
// finds that maximum itself: dloss is small and stays in the caches. (1024
// threads: 3001 rows take three rounds of loads.)
constexpr int kRowsThreads = 1024;
__global__ __launch_bounds__(kRowsThreads) void xent_rows_kernel(RowsArgs p) {
  __shared__ float sm[kRowsThreads / 64];
  float c = 0.0f;
#pragma unroll 4
  for (int i = threadIdx.x; i < p.M; i += kRowsThreads) {
    // both loads at once: one latency for each round of the threads, not two
    const float d = fabsf(p.dloss[i]);
    c = fmaxf(c, target_of(p.target, p.target64, i) != p.ignore ? d : 0.0f);
  }
#pragma unroll
  for (int h = 32; h > 0; h /= 2) c = fmaxf(c, lane_xor(c, h));
  if ((threadIdx.x & 63) == 0) sm[threadIdx.x >> 6] = c;
  __syncthreads();
#pragma unroll
  for (int w = 0; w < kRowsThreads / 64; ++w) c = fmaxf(c, sm[w]);
  c = xent_scale(c);
  if (blockIdx.x == 0 && threadIdx.x == 0) *p.scale = c;
  const int64_t row = (int64_t)blockIdx.x * kRowsThreads + threadIdx.x;
  if (row >= p.M) return;
  p.rows[row] = xent_row(target_of(p.target, p.target64, row), p.ignore, p.N, p.lse[row], p.dloss[row], c, p.z_loss);
}

__global__ __launch_bounds__(256) void add_parts_kernel(AddArgs p) {
  const int64_t chunks = (p.N + 3) / 4;
  const float scale = p.scale ? *p.scale : 1.0f;
  for (int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x; i < p.M * chunks; i += (int64_t)gridDim.x * 256) {
    const int64_t row = i / chunks, col = 4 * (i - row * chunks);
    const float* src = p.part + row * p.ldp + col;
    float4 v = *reinterpret_cast<const float4*>(src);
#pragma unroll 4
    for (int s = 1; s < p.parts; ++s) {
      const float4 w = *reinterpret_cast<const float4*>(src + s * p.part_stride);
      v.x += w.x; v.y += w.y; v.z += w.z; v.w += w.w;
    }
    uint16_t* dst = p.out + row * p.ldo + col;
    const uint32_t lo = pack_bf16x2(v.x * scale, v.y * scale), hi = pack_bf16x2(v.z * scale, v.w * scale);
    if (col + 4 <= p.N) {
      *reinterpret_cast<uint2*>(dst) = make_uint2(lo, hi);
    } else {
      const uint32_t w[2] = {lo, hi};
      for (int e = 0; col + e < p.N; ++e) dst[e] = (uint16_t)(w[e >> 1] >> (16 * (e & 1)));
    }
  }
}

__global__ __launch_bounds__(256) void add_rows_kernel(const float* part, int64_t rows, int64_t cols, float* out) {
  // 64 columns per workgroup, four waves sharing the rows
  __shared__ float sm[256];
  const int64_t c = (int64_t)blockIdx.x * 64 + (threadIdx.x & 63);
  float s = 0.0f;
  if (c < cols) {
#pragma unroll 4
    for (int64_t r = threadIdx.x >> 6; r < rows; r += 4) s += part[r * cols + c];
  }
  sm[threadIdx.x] = s;
  __syncthreads();
  if (threadIdx.x < 64 && c < cols)
    out[c] = (sm[threadIdx.x] + sm[threadIdx.x + 64]) + (sm[threadIdx.x + 128] + sm[threadIdx.x + 192]);
}

__global__ __launch_bounds__(256) void zero_kernel(uint16_t* p, int64_t rows, int64_t cols, int64_t pitch) {
  for (int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x; i < rows * cols; i += (int64_t)gridDim.x * 256)
    p[i / cols * pitch + i % cols] = 0;
}

// Workgroups of the outer product, and their share of the rows: about eight
// per compute unit (their waves fill its SIMDs), but at least 64 rows each, so
// that the x fragments are read for several blocks.
unsigned outer_groups(OuterArgs& a, int cu_count) {
  a.col_groups = (int32_t)ceil_div(a.K, kOuterCols);
  int64_t rows = ceil_div((int64_t)a.V * a.col_groups, 8 * cu_count);
  rows = ceil_div(rows < 64 ? 64 : rows, 16) * 16;
  a.rows_per_group = (int32_t)rows;
  return (unsigned)(a.col_groups * ceil_div(a.V, rows));
}

unsigned blocks_for(int64_t items) {
  const int64_t b = ceil_div(items, 256);
  return (unsigned)(b < 1 ? 1 : b > 4096 ? 4096 : b);
}

}  // namespace

hipError_t launch_xent_finish(const FinishArgs& a, hipStream_t stream) {
  // 16 rows a workgroup once that still gives half of the compute units one
  if (a.M >= 2048)
    return launch_raw(reinterpret_cast<const void*>(&xent_finish_kernel<16>), dim3((unsigned)ceil_div(a.M, 16)),
                      dim3(256), a, stream);
  return launch_raw(reinterpret_cast<const void*>(&xent_finish_kernel<1>), dim3((unsigned)a.M), dim3(256), a,
                    stream);
}

hipError_t launch_xent_rows(const RowsArgs& a, hipStream_t stream) {
  return launch_raw(reinterpret_cast<const void*>(&xent_rows_kernel), dim3((unsigned)ceil_div(a.M, kRowsThreads)),
                    dim3(kRowsThreads), a, stream);
}

hipError_t launch_add_parts(const AddArgs& a, hipStream_t stream) {
  return launch_raw(reinterpret_cast<const void*>(&add_parts_kernel),
                    dim3(blocks_for((int64_t)a.M * ceil_div(a.N, 4))), dim3(256), a, stream);
}

hipError_t launch_add_rows(const float* part, int64_t rows, int64_t cols, float* out, hipStream_t stream) {
  void* argv[] = {&part, &rows, &cols, &out};
  return hipLaunchKernel(reinterpret_cast<const void*>(&add_rows_kernel), dim3((unsigned)ceil_div(cols, 64)),
                         dim3(256), argv, 0, stream);
}

hipError_t launch_outer(OuterArgs a, int cu_count, hipStream_t stream) {
  const dim3 grid(outer_groups(a, cu_count));
  const void* fn = a.T <= 32   ? reinterpret_cast<const void*>(&outer_kernel<1>)
                   : a.T <= 64 ? reinterpret_cast<const void*>(&outer_kernel<2>)
                               : reinterpret_cast<const void*>(&outer_kernel<4>);
  return launch_raw(fn, grid, dim3(256), a, stream);
}

hipError_t launch_pair(const TrainArgs& product, int64_t grid, bool bf16, const OuterArgs& outer, int cu_count,
                       hipStream_t stream) {
  constexpr TrainTile t = kTrainTiles[kSmallTile];
  static_assert(t.wm * t.wn * 64 == 256, "the threads of both kernels");
  PairArgs a{};
  static_cast<TrainArgs&>(a) = product;
  a.outer = outer;
  a.n_first = (int32_t)grid;
  const unsigned groups = outer_groups(a.outer, cu_count);
  const void* fn =
      bf16 ? reinterpret_cast<const void*>(&tile16_gemm_kernel<t.bm, t.bn, t.wm, t.wn, 4, false, true, false, kEpiPair>)
           : reinterpret_cast<const void*>(
                 &tile16_gemm_kernel<t.bm, t.bn, t.wm, t.wn, 4, false, false, false, kEpiPair>);
  return launch_raw(fn, dim3((unsigned)grid + groups), dim3(256), a, stream);
}

hipError_t launch_zero(void* p, int64_t rows, int64_t bytes, int64_t pitch, hipStream_t stream) {
  uint16_t* q = static_cast<uint16_t*>(p);
  int64_t cols = bytes / 2, ld = pitch / 2;
  void* argv[] = {&q, &rows, &cols, &ld};
  return hipLaunchKernel(reinterpret_cast<const void*>(&zero_kernel), dim3(blocks_for(rows * cols)), dim3(256), argv,
                         0, stream);
}

}  // namespace tg
