// Layer norm forward:
//   m = sum(x) / n,  v = sum((x - m)^2) / n,  r = 1 / sqrt(v + eps),
//   h = (x - m) r,   y = gamma h + beta,
// with h optionally saved as an 8-bit checkpoint in the same pass.
//
// Two passes over values that stay in registers: the variance is taken about
// the mean that was found, so it neither cancels nor goes negative.
#include <algorithm>

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

// NW warps hold one row, NC groups of 256 columns a warp; a block of
// kRowsPerBlock rows when a row is one warp's.
template <class TX, class TY, bool VEC, int NW, int NC>
__global__ void __launch_bounds__(NW == 1 ? 128 : NW * 32) ts_norm_kernel(const NormArgs a) {
  __shared__ float red[2][NW];
  pdl_launch_dependents();
  pdl_wait();
  const int lane = threadIdx.x & 31, warp = NW == 1 ? 0 : threadIdx.x >> 5;
  const int64_t row = NW == 1 ? (int64_t)blockIdx.x * 4 + (threadIdx.x >> 5) : blockIdx.x;
  if (row >= a.rows) return;
  const TX* x = static_cast<const TX*>(a.x.p) + row * a.x.ld;
  float v[NC][8];
  float s = 0.f;
#pragma unroll
  for (int i = 0; i < NC; ++i) load_group<VEC>(x, (i * NW + warp) * kGroupCols, a.cols, lane, v[i]);
#pragma unroll
  for (int i = 0; i < NC; ++i)
    s += ((v[i][0] + v[i][1]) + (v[i][2] + v[i][3])) + ((v[i][4] + v[i][5]) + (v[i][6] + v[i][7]));
  const float n = (float)a.cols;
  const float mean = row_sum<NW>(s, red[0], warp, lane) / n;
  s = 0.f;
#pragma unroll
  for (int i = 0; i < NC; ++i)
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      const int c = (i * NW + warp) * kGroupCols + group_col<VEC>(lane, j);
      v[i][j] = c < a.cols ? v[i][j] - mean : 0.f;
      s += v[i][j] * v[i][j];
    }
  const float rstd = 1.f / sqrtf(row_sum<NW>(s, red[1], warp, lane) / n + a.eps);
  if (warp == 0 && lane == 0) {
    if (a.mean) a.mean[row] = mean;
    if (a.rstd) a.rstd[row] = rstd;
  }
  TY* y = static_cast<TY*>(a.y.p) + row * a.y.ld;
#pragma unroll
  for (int i = 0; i < NC; ++i) {
    const int c0 = (i * NW + warp) * kGroupCols;
    if (c0 >= a.cols) break;
    float g[8], b[8];
#pragma unroll
    for (int j = 0; j < 8; ++j) v[i][j] *= rstd;
    if (a.ckpt.q) ckpt_store_group<VEC>(a.ckpt, row, c0, lane, v[i]);
    if (a.gamma) {
      load_group<VEC>(a.gamma, c0, a.cols, lane, g);
#pragma unroll
      for (int j = 0; j < 8; ++j) v[i][j] *= g[j];
    }
    if (a.beta) {
      load_group<VEC>(a.beta, c0, a.cols, lane, b);
#pragma unroll
      for (int j = 0; j < 8; ++j) v[i][j] += b[j];
    }
    store_group<VEC>(y, c0, a.cols, lane, v[i]);
  }
}

// Rows too long for registers: one block a row, which reads it three times
// (the later two from L2).
template <class TX, class TY, bool VEC>
__global__ void __launch_bounds__(1024) ts_norm_long_kernel(const NormArgs a) {
  __shared__ float red[2][32];
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
    if (a.ckpt.q) ckpt_store_group<VEC>(a.ckpt, row, c0, lane, v);
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

template <class TX, class TY, bool VEC>
cudaError_t norm_rows(const NormArgs& a, cudaStream_t st) {
  cudaLaunchAttribute at[1];
  const int groups = (a.cols + kGroupCols - 1) / kGroupCols;
  if (groups <= 4) {
    cudaLaunchConfig_t cfg = pdl_config((int)((a.rows + 3) / 4), 128, 0, st);
    pdl_attr(cfg, at);
    return cudaLaunchKernelEx(&cfg, ts_norm_kernel<TX, TY, VEC, 1, 4>, a);
  }
  if (groups <= 16) {
    cudaLaunchConfig_t cfg = pdl_config((int)a.rows, 256, 0, st);
    pdl_attr(cfg, at);
    return cudaLaunchKernelEx(&cfg, ts_norm_kernel<TX, TY, VEC, 8, 2>, a);
  }
  if (groups <= 64) {
    cudaLaunchConfig_t cfg = pdl_config((int)a.rows, 512, 0, st);
    pdl_attr(cfg, at);
    return cudaLaunchKernelEx(&cfg, ts_norm_kernel<TX, TY, VEC, 16, 4>, a);
  }
  cudaLaunchConfig_t cfg = pdl_config((int)a.rows, 1024, 0, st);
  pdl_attr(cfg, at);
  return cudaLaunchKernelEx(&cfg, ts_norm_long_kernel<TX, TY, VEC>, a);
}

template <class TX, class TY>
cudaError_t norm_types(const NormArgs& a, cudaStream_t st) {
  return rows_aligned(a.x) && rows_aligned(a.y) && aligned16(a.gamma) && aligned16(a.beta)
             ? norm_rows<TX, TY, true>(a, st)
             : norm_rows<TX, TY, false>(a, st);
}

}  // namespace

cudaError_t launch_layer_norm(const ts_ops&, const NormArgs& a, cudaStream_t st) {
  if (a.x.bf16)
    return a.y.bf16 ? norm_types<__nv_bfloat16, __nv_bfloat16>(a, st) : norm_types<__nv_bfloat16, float>(a, st);
  return a.y.bf16 ? norm_types<float, __nv_bfloat16>(a, st) : norm_types<float, float>(a, st);
}

}  // namespace fg
