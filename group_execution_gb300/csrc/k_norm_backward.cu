// Layer norm backward.  With h the normalised row (from x, mean and rstd, or
// from its 8-bit checkpoint) and u = dy gamma,
//   dx = r (u - mean(u) - h mean(u h)),
//   dgamma_j = sum over rows of dy h,  dbeta_j = sum over rows of dy.
//
// The column sums are taken in two steps without atomics: each block adds the
// rows it walks in order into registers and writes one partial row to the
// workspace, then a second kernel adds the partials in block order.  The
// result depends on the sizes alone, not on scheduling.
#include <algorithm>

#include "launch.h"
#include "ts_device.cuh"

namespace fg {
namespace {

// Where h comes from.
template <class TX>
struct FromX {
  using Dx = TX;
  template <bool VEC>
  __device__ __forceinline__ static void load(const NormArgs& a, int64_t row, int c0, int lane, float mean, float rstd,
                                              float (&h)[8]) {
    load_group<VEC>(static_cast<const TX*>(a.x.p) + row * a.x.ld, c0, a.cols, lane, h);
#pragma unroll
    for (int j = 0; j < 8; ++j) h[j] = (h[j] - mean) * rstd;
  }
  __device__ __forceinline__ static float mean(const NormArgs& a, int64_t row) { return a.mean[row]; }
};
template <class TDX>
struct FromCkpt {
  using Dx = TDX;
  template <bool VEC>
  __device__ __forceinline__ static void load(const NormArgs& a, int64_t row, int c0, int lane, float, float,
                                              float (&h)[8]) {
    ckpt_load_group<VEC>(a.ckpt, row, c0, lane, h);
  }
  __device__ __forceinline__ static float mean(const NormArgs&, int64_t) { return 0.f; }
};

// dx alone: one block a row, any length.
template <class TDY, class Src, bool VEC>
__global__ void __launch_bounds__(256) ts_norm_dx_kernel(const NormArgs a) {
  __shared__ float red[2][8];
  pdl_launch_dependents();
  pdl_wait();
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int64_t row = blockIdx.x;
  const TDY* dy = static_cast<const TDY*>(a.dy.p) + row * a.dy.ld;
  const float mean = Src::mean(a, row), rstd = a.rstd[row];
  float s1 = 0.f, s2 = 0.f;
  for (int64_t cc = warp * kGroupCols; cc < a.cols; cc += 8 * kGroupCols) {
    const int c0 = (int)cc;
    float u[8], h[8], g[8];
    load_group<VEC>(dy, c0, a.cols, lane, u);
    Src::template load<VEC>(a, row, c0, lane, mean, rstd, h);
    if (a.gamma) {
      load_group<VEC>(a.gamma, c0, a.cols, lane, g);
#pragma unroll
      for (int j = 0; j < 8; ++j) u[j] *= g[j];
    }
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      if (c0 + group_col<VEC>(lane, j) < a.cols) {
        s1 += u[j];
        s2 += u[j] * h[j];
      }
    }
  }
  s1 = warp_sum(s1);
  s2 = warp_sum(s2);
  if (lane == 0) {
    red[0][warp] = s1;
    red[1][warp] = s2;
  }
  __syncthreads();
  s1 = s2 = 0.f;
#pragma unroll
  for (int w = 0; w < 8; ++w) {
    s1 += red[0][w];
    s2 += red[1][w];
  }
  const float m1 = s1 / (float)a.cols, m2 = s2 / (float)a.cols;
  typename Src::Dx* dx = static_cast<typename Src::Dx*>(a.dx.p) + row * a.dx.ld;
  for (int64_t cc = warp * kGroupCols; cc < a.cols; cc += 8 * kGroupCols) {
    const int c0 = (int)cc;
    float u[8], h[8], g[8];
    load_group<VEC>(dy, c0, a.cols, lane, u);
    Src::template load<VEC>(a, row, c0, lane, mean, rstd, h);
    if (a.gamma) {
      load_group<VEC>(a.gamma, c0, a.cols, lane, g);
#pragma unroll
      for (int j = 0; j < 8; ++j) u[j] *= g[j];
    }
#pragma unroll
    for (int j = 0; j < 8; ++j) u[j] = rstd * (u[j] - m1 - h[j] * m2);
    store_group<VEC>(dx, c0, a.cols, lane, u);
  }
}

// Partial column sums: block (bx, by) takes 256 columns and every gridDim.y-th
// run of 8 rows, a warp a row; the block's warps are added in order.  part:
// [gridDim.y][2][cols], dy's sums and then, with a Src, dy h's.
template <class TDY, class Src, bool VEC>
__global__ void __launch_bounds__(256) ts_column_kernel(const NormArgs a, float* part) {
  __shared__ float sm[8][2][kGroupCols];
  pdl_launch_dependents();
  pdl_wait();
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int c0 = blockIdx.x * kGroupCols;
  float sb[8] = {}, sg[8] = {};
  for (int64_t row = (int64_t)blockIdx.y * 8 + warp; row < a.rows; row += (int64_t)gridDim.y * 8) {
    float d[8];
    load_group<VEC>(static_cast<const TDY*>(a.dy.p) + row * a.dy.ld, c0, a.cols, lane, d);
#pragma unroll
    for (int j = 0; j < 8; ++j) sb[j] += d[j];
    if constexpr (!std::is_void<Src>::value) {
      float h[8];
      Src::template load<VEC>(a, row, c0, lane, Src::mean(a, row), a.rstd[row], h);
#pragma unroll
      for (int j = 0; j < 8; ++j) sg[j] += d[j] * h[j];
    }
  }
#pragma unroll
  for (int j = 0; j < 8; ++j) {
    sm[warp][0][group_col<VEC>(lane, j)] = sb[j];
    sm[warp][1][group_col<VEC>(lane, j)] = sg[j];
  }
  __syncthreads();
  const int c = c0 + threadIdx.x;
  if (c < a.cols) {
    float b = 0.f, g = 0.f;
#pragma unroll
    for (int w = 0; w < 8; ++w) {
      b += sm[w][0][threadIdx.x];
      g += sm[w][1][threadIdx.x];
    }
    part[((int64_t)blockIdx.y * 2 + 0) * a.cols + c] = b;
    part[((int64_t)blockIdx.y * 2 + 1) * a.cols + c] = g;
  }
}

// The partials' sums in order: a block takes 32 columns of dbeta or dgamma,
// its eight warps every eighth partial.  fresh, if not null, also receives
// dbeta's sums of this call alone.
__global__ void __launch_bounds__(256) ts_column_finish_kernel(const float* part, int parts, int cols, float* dbeta,
                                                               float* dgamma, int accumulate, float* fresh) {
  __shared__ float sm[8][32];
  pdl_launch_dependents();
  pdl_wait();
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int c = blockIdx.x * 32 + lane;
  float* out = blockIdx.y ? dgamma : dbeta;
  if (!out && (blockIdx.y || !fresh)) return;
  float s = 0.f;
  if (c < cols)
    for (int p = warp; p < parts; p += 8) s += part[((int64_t)p * 2 + blockIdx.y) * cols + c];
  sm[warp][lane] = s;
  __syncthreads();
  if (warp == 0 && c < cols) {
    s = 0.f;
#pragma unroll
    for (int w = 0; w < 8; ++w) s += sm[w][lane];
    if (blockIdx.y == 0 && fresh) fresh[c] = s;
    if (out) out[c] = accumulate ? out[c] + s : s;
  }
}

cudaError_t finish_columns(const float* part, int parts, int cols, float* dbeta, float* dgamma, int accumulate,
                           float* fresh, cudaStream_t st) {
  cudaLaunchConfig_t cfg = pdl_config(1, 256, 0, st);
  cfg.gridDim = dim3((cols + 31) / 32, 2);
  cudaLaunchAttribute at[1];
  pdl_attr(cfg, at);
  return cudaLaunchKernelEx(&cfg, ts_column_finish_kernel, part, parts, cols, dbeta, dgamma, accumulate, fresh);
}

// Row splits of a column sum: enough blocks for the device, 64 rows a block
// at least, partials that fit the workspace (less its last 8 bytes a column,
// kept for a call's own sums).
int column_parts(const ts_ops& h, int64_t rows, int cols) {
  const int64_t tiles = (cols + kGroupCols - 1) / kGroupCols;
  int64_t p = (8 * (int64_t)h.nsm + tiles - 1) / tiles;
  p = std::min(p, (rows + 63) / 64);
  p = std::min(p, (h.ws_bytes - 8 * (int64_t)cols) / (8 * (int64_t)cols));
  return (int)std::max<int64_t>(std::min<int64_t>(p, 65535), 1);
}

template <class TDY, class Src, bool VEC>
cudaError_t columns(const ts_ops& h, const NormArgs& a, float* fresh, cudaStream_t st) {
  const int parts = column_parts(h, a.rows, a.cols);
  cudaLaunchConfig_t cfg = pdl_config(1, 256, 0, st);
  cfg.gridDim = dim3((a.cols + kGroupCols - 1) / kGroupCols, parts);
  cudaLaunchAttribute at[1];
  pdl_attr(cfg, at);
  float* part = reinterpret_cast<float*>(h.ws);
  cudaError_t e = cudaLaunchKernelEx(&cfg, ts_column_kernel<TDY, Src, VEC>, a, part);
  if (e != cudaSuccess) return e;
  return finish_columns(part, parts, a.cols, a.dbeta, a.dgamma, a.accumulate, fresh, st);
}

template <class TDY, class Src, bool VEC>
cudaError_t backward_rows(const ts_ops& h, const NormArgs& a, cudaStream_t st) {
  if (a.rows > 0) {
    cudaLaunchConfig_t cfg = pdl_config((int)a.rows, 256, 0, st);
    cudaLaunchAttribute at[1];
    pdl_attr(cfg, at);
    cudaError_t e = cudaLaunchKernelEx(&cfg, ts_norm_dx_kernel<TDY, Src, VEC>, a);
    if (e != cudaSuccess) return e;
  }
  if (!a.dgamma && !a.dbeta) return cudaSuccess;
  return columns<TDY, Src, VEC>(h, a, nullptr, st);
}

template <class TDY, class Src>
cudaError_t backward_types(const ts_ops& h, const NormArgs& a, cudaStream_t st) {
  const bool vec = rows_aligned(a.dy) && rows_aligned(a.dx) && aligned16(a.gamma) && (!a.x.p || rows_aligned(a.x));
  return vec ? backward_rows<TDY, Src, true>(h, a, st) : backward_rows<TDY, Src, false>(h, a, st);
}

}  // namespace

cudaError_t launch_layer_norm_backward(const ts_ops& h, const NormArgs& a, cudaStream_t st) {
  using B = __nv_bfloat16;
  if (a.ckpt.q) {
    if (a.dy.bf16)
      return a.dx.bf16 ? backward_types<B, FromCkpt<B>>(h, a, st) : backward_types<B, FromCkpt<float>>(h, a, st);
    return a.dx.bf16 ? backward_types<float, FromCkpt<B>>(h, a, st) : backward_types<float, FromCkpt<float>>(h, a, st);
  }
  if (a.dy.bf16) return a.x.bf16 ? backward_types<B, FromX<B>>(h, a, st) : backward_types<B, FromX<float>>(h, a, st);
  return a.x.bf16 ? backward_types<float, FromX<B>>(h, a, st) : backward_types<float, FromX<float>>(h, a, st);
}

cudaError_t launch_column_sums(const ts_ops& h, const TsMat& dy, int64_t rows, int cols, float* fresh, float* db,
                               int accumulate, cudaStream_t st) {
  NormArgs a;
  a.dy = dy;
  a.rows = rows;
  a.cols = cols;
  a.dbeta = db;
  a.accumulate = accumulate;
  if (dy.bf16)
    return rows_aligned(dy) ? columns<__nv_bfloat16, void, true>(h, a, fresh, st)
                            : columns<__nv_bfloat16, void, false>(h, a, fresh, st);
  return rows_aligned(dy) ? columns<float, void, true>(h, a, fresh, st) : columns<float, void, false>(h, a, fresh, st);
}

}  // namespace fg
