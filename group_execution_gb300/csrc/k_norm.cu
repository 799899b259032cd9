// Layer norm forward:
//   m = sum(x) / n,  v = sum((x - m)^2) / n,  r = 1 / sqrt(v + eps),
//   h = (x - m) r,   y = gamma h + beta,
// with h optionally saved as an 8-bit checkpoint in the same pass.
//
// Two passes over values that stay in registers: the variance is taken about
// the mean that was found, so it neither cancels nor goes negative.  Bound by
// memory where rows are wide types, else by the two reductions a row between
// its loads and its stores: 8192 x 4096 takes 45 us in f32 (88 % of the copy
// rate), 33 in bf16 (60 %), 44 from f32 to bf16 with the checkpoint (79 %);
// 64 x 1024 f32 3.7, of which a launch is 2 to 3.
#include <algorithm>
#include <atomic>

#include "launch.h"
#include "ts_device.cuh"

namespace fg {
namespace {

// Sum over the NW warps that share a row, in warp order; every thread gets it.
template <int NW>
__device__ __forceinline__ float row_sum(float v, float* red, int warp, int lane) {
  v = warp_sum(v);
  if (NW == 1) return v;
  if (lane == 0) red[warp] = v;
  __syncthreads();
  float s = 0.f;
#pragma unroll
  for (int w = 0; w < NW; ++w) s += red[w];
  return s;
}

// NW warps hold one row, NC groups of 256 columns a warp; blocks (of four rows
// when a row is one warp's) walk the rows, with the next row's loads in flight
// while one is worked on.  (With a block to a row, loads are in flight for a
// third of a block's life only: 45 us instead of 33 at 8192 x 4096 in bf16, 50
// instead of 44 from float32 to bf16 with the checkpoint, where memory's copy
// rate allows 35.)
template <class TX, class TY, bool VEC, int NW, int NC>
__global__ void __launch_bounds__(NW == 1 ? 128 : NW * 32, NW == 1 ? 5 : NW == 8 ? 4 : NC == 2 ? 2 : 1)
    ts_norm_kernel(const NormArgs a) {
  constexpr int kRows = NW == 1 ? 4 : 1;   // rows a block works on at a time
  __shared__ float red[2][NW];
  __shared__ __align__(16) float scratch[VEC ? 1 : kRows * NW][kGroupCols];
  pdl_launch_dependents();
  pdl_wait();
  const int lane = threadIdx.x & 31, warp = NW == 1 ? 0 : threadIdx.x >> 5;
  const int rows = (int)a.rows, step = gridDim.x * kRows;
  int row = blockIdx.x * kRows + (NW == 1 ? threadIdx.x >> 5 : 0);
  const TX* x = static_cast<const TX*>(a.x.p) + (int64_t)row * a.x.ld;
  TY* y = static_cast<TY*>(a.y.p) + (int64_t)row * a.y.ld;
  const int64_t x_step = (int64_t)step * a.x.ld, y_step = (int64_t)step * a.y.ld;
  const float n = (float)a.cols;
  RawGroup<TX, VEC> raw[NC];
  auto fetch = [&]() {
#pragma unroll
    for (int i = 0; i < NC; ++i) raw[i].load(x, (i * NW + warp) * kGroupCols, a.cols, lane);
    x += x_step;
  };
  if (row < rows) fetch();
  for (; row < rows; row += step, y += y_step) {
    F2 v[NC][4], s = 0;
#pragma unroll
    for (int i = 0; i < NC; ++i) {
      float e[8];
      raw[i].get(e);
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        v[i][j] = pack2f(e[2 * j], e[2 * j + 1]);
        s = add2(s, v[i][j]);
      }
    }
    if (row + step < rows) fetch();
    const float mean = row_sum<NW>(sum2(s), red[0], warp, lane) / n;
    const F2 minus = pack2f(-mean, -mean);
    s = 0;
#pragma unroll
    for (int i = 0; i < NC; ++i) {
      const int c0 = (i * NW + warp) * kGroupCols;
#pragma unroll
      for (int j = 0; j < 4; ++j) v[i][j] = add2(v[i][j], minus);
      if (c0 + kGroupCols > a.cols) {   // columns past the last do not count
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          float e[2];
          unpack2f(v[i][j], e[0], e[1]);
#pragma unroll
          for (int k = 0; k < 2; ++k)
            if (c0 + group_col<VEC>(lane, 2 * j + k) >= a.cols) e[k] = 0.f;
          v[i][j] = pack2f(e[0], e[1]);
        }
      }
#pragma unroll
      for (int j = 0; j < 4; ++j) s = fma2(v[i][j], v[i][j], s);
    }
    const float rstd = 1.f / sqrtf(row_sum<NW>(sum2(s), red[1], warp, lane) / n + a.eps);
    if (warp == 0 && lane == 0) {
      if (a.mean) a.mean[row] = mean;
      if (a.rstd) a.rstd[row] = rstd;
    }
    const F2 scale = pack2f(rstd, rstd);
#pragma unroll
    for (int i = 0; i < NC; ++i) {
      const int c0 = (i * NW + warp) * kGroupCols;
      if (c0 >= a.cols) break;
      float h[8], g[8], b[8];
#pragma unroll
      for (int j = 0; j < 4; ++j) unpack2f(mul2(v[i][j], scale), h[2 * j], h[2 * j + 1]);
      if (a.ckpt.q) ckpt_store_group<VEC>(a.ckpt, row, c0, lane, h, scratch[VEC ? 0 : threadIdx.x >> 5]);
      if (a.gamma) {
        load_group<VEC>(a.gamma, c0, a.cols, lane, g);
#pragma unroll
        for (int j = 0; j < 8; ++j) h[j] *= g[j];
      }
      if (a.beta) {
        load_group<VEC>(a.beta, c0, a.cols, lane, b);
#pragma unroll
        for (int j = 0; j < 8; ++j) h[j] += b[j];
      }
      store_group<VEC>(y, c0, a.cols, lane, h);
    }
  }
}

// Rows too long for registers: one block a row, which reads it three times
// (the later two from L2).  1024 x 32768 bf16 takes 68 us, where one reading
// and the store at the copy rate take 20.
template <class TX, class TY, bool VEC>
__global__ void __launch_bounds__(1024) ts_norm_long_kernel(const NormArgs a) {
  __shared__ float red[2][32];
  __shared__ __align__(16) float scratch[VEC ? 1 : 32][kGroupCols];
  pdl_launch_dependents();
  pdl_wait();
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int64_t row = blockIdx.x;
  const TX* x = static_cast<const TX*>(a.x.p) + row * a.x.ld;
  const float n = (float)a.cols;
  float s = 0.f, v[8];
  const int step = 32 * kGroupCols;
  for (int64_t c0 = warp * kGroupCols; c0 < a.cols; c0 += step) {
    load_group<VEC>(x, (int)c0, a.cols, lane, v);
    s += ((v[0] + v[1]) + (v[2] + v[3])) + ((v[4] + v[5]) + (v[6] + v[7]));
  }
  const float mean = row_sum<32>(s, red[0], warp, lane) / n;
  s = 0.f;
  for (int64_t c0 = warp * kGroupCols; c0 < a.cols; c0 += step) {
    load_group<VEC>(x, (int)c0, a.cols, lane, v);
    float q = 0.f;
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      const float d = (int)c0 + group_col<VEC>(lane, j) < a.cols ? v[j] - mean : 0.f;
      q += d * d;
    }
    s += q;
  }
  const float rstd = 1.f / sqrtf(row_sum<32>(s, red[1], warp, lane) / n + a.eps);
  if (threadIdx.x == 0) {
    if (a.mean) a.mean[row] = mean;
    if (a.rstd) a.rstd[row] = rstd;
  }
  TY* y = static_cast<TY*>(a.y.p) + row * a.y.ld;
  for (int64_t cc = warp * kGroupCols; cc < a.cols; cc += step) {
    const int c0 = (int)cc;
    float g[8];
    load_group<VEC>(x, c0, a.cols, lane, v);
#pragma unroll
    for (int j = 0; j < 8; ++j) v[j] = c0 + group_col<VEC>(lane, j) < a.cols ? (v[j] - mean) * rstd : 0.f;
    if (a.ckpt.q) ckpt_store_group<VEC>(a.ckpt, row, c0, lane, v, scratch[VEC ? 0 : threadIdx.x >> 5]);
    if (a.gamma) {
      load_group<VEC>(a.gamma, c0, a.cols, lane, g);
#pragma unroll
      for (int j = 0; j < 8; ++j) v[j] *= g[j];
    }
    if (a.beta) {
      load_group<VEC>(a.beta, c0, a.cols, lane, g);
#pragma unroll
      for (int j = 0; j < 8; ++j) v[j] += g[j];
    }
    store_group<VEC>(y, c0, a.cols, lane, v);
  }
}

// As many blocks as the device holds at once, at most one to every kRows rows.
template <class TX, class TY, bool VEC, int NW, int NC>
cudaError_t norm_walk(const ts_ops& h, const NormArgs& a, cudaStream_t st) {
  constexpr int kRows = NW == 1 ? 4 : 1, kThreads = NW == 1 ? 128 : NW * 32;
  static std::atomic<int> per_sm{0};   // the same on every device this is built for
  int k = per_sm.load(std::memory_order_relaxed);
  if (!k) {
    cudaError_t e = cudaOccupancyMaxActiveBlocksPerMultiprocessor(&k, ts_norm_kernel<TX, TY, VEC, NW, NC>, kThreads, 0);
    if (e != cudaSuccess) return e;
    if (k < 1) return cudaErrorLaunchOutOfResources;
    per_sm.store(k, std::memory_order_relaxed);
  }
  const int64_t grid = std::min<int64_t>((a.rows + kRows - 1) / kRows, (int64_t)k * h.nsm);
  cudaLaunchConfig_t cfg = pdl_config((int)grid, kThreads, 0, st);
  cudaLaunchAttribute at[1];
  pdl_attr(cfg, at);
  return cudaLaunchKernelEx(&cfg, ts_norm_kernel<TX, TY, VEC, NW, NC>, a);
}

template <class TX, class TY, bool VEC>
cudaError_t norm_rows(const ts_ops& h, const NormArgs& a, cudaStream_t st) {
  const int groups = (a.cols + kGroupCols - 1) / kGroupCols;
  // a warp to a row while four groups hold it (no barrier), then the fewest
  // warps whose registers do
  if (groups <= 4) return norm_walk<TX, TY, VEC, 1, 4>(h, a, st);
  if (groups <= 16) return norm_walk<TX, TY, VEC, 8, 2>(h, a, st);
  if (groups <= 32) return norm_walk<TX, TY, VEC, 16, 2>(h, a, st);
  if (groups <= 64) return norm_walk<TX, TY, VEC, 16, 4>(h, a, st);
  cudaLaunchAttribute at[1];
  cudaLaunchConfig_t cfg = pdl_config((int)a.rows, 1024, 0, st);
  pdl_attr(cfg, at);
  return cudaLaunchKernelEx(&cfg, ts_norm_long_kernel<TX, TY, VEC>, a);
}

template <class TX, class TY>
cudaError_t norm_types(const ts_ops& h, const NormArgs& a, cudaStream_t st) {
  return rows_aligned(a.x) && rows_aligned(a.y) && aligned16(a.gamma) && aligned16(a.beta)
             ? norm_rows<TX, TY, true>(h, a, st)
             : norm_rows<TX, TY, false>(h, a, st);
}

}  // namespace

cudaError_t launch_layer_norm(const ts_ops& h, const NormArgs& a, cudaStream_t st) {
  if (a.x.bf16)
    return a.y.bf16 ? norm_types<__nv_bfloat16, __nv_bfloat16>(h, a, st) : norm_types<__nv_bfloat16, float>(h, a, st);
  return a.y.bf16 ? norm_types<float, __nv_bfloat16>(h, a, st) : norm_types<float, float>(h, a, st);
}

}  // namespace fg
