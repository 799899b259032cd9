// 8-bit activation checkpoints (the OCP microscaling format with int8
// elements: blocks of 32 columns of a row share a power-of-two step): saving,
// loading, and the derivative of an activation from its saved output.
//
// A checkpoint's values are exact in bf16 (8 bits of significand) and the
// step's division is exact, so rounding to the nearest step is the only
// rounding on the way.  Each kernel is one pass, a warp to each group of 256
// columns; device memory bounds them.
#include <algorithm>

#include "launch.h"
#include "ts_device.cuh"

namespace fg {
namespace {

// Groups of 256 columns, row by row; blocks stride over them.
struct Groups {
  int64_t rows;
  int cols, per_row;
};

template <class F>
__device__ __forceinline__ void for_groups(const Groups& g, F f) {
  const int64_t total = g.rows * g.per_row, step = (int64_t)gridDim.x * 8;
  for (int64_t i = (int64_t)blockIdx.x * 8 + (threadIdx.x >> 5); i < total; i += step) {
    const int64_t r = i / g.per_row;
    f(r, (int)(i - r * g.per_row) * kGroupCols);
  }
}

template <class TX, bool VEC>
__global__ void __launch_bounds__(256) ts_save_kernel(const TsMat x, const Groups g, const TsCkpt c) {
  pdl_launch_dependents();
  pdl_wait();
  const int lane = threadIdx.x & 31;
  for_groups(g, [&](int64_t r, int c0) {
    float v[8];
    load_group<VEC>(static_cast<const TX*>(x.p) + r * x.ld, c0, g.cols, lane, v);
    ckpt_store_group<VEC>(c, r, c0, lane, v);
  });
}

template <class TY, bool VEC>
__global__ void __launch_bounds__(256) ts_load_kernel(const TsCkpt c, const Groups g, const TsOut y) {
  pdl_launch_dependents();
  pdl_wait();
  const int lane = threadIdx.x & 31;
  for_groups(g, [&](int64_t r, int c0) {
    float v[8];
    ckpt_load_group<VEC>(c, r, c0, lane, v);
    store_group<VEC>(static_cast<TY*>(y.p) + r * y.ld, c0, g.cols, lane, v);
  });
}

// f' from a = f(x): relu's is 1 where a > 0, sigmoid's a (1 - a), tanh's 1 - a^2.
template <int ACT>
__device__ __forceinline__ float act_slope(float a) {
  if (ACT == 0) return a > 0.f ? 1.f : a != a ? a : 0.f;
  if (ACT == 1) return a * (1.f - a);
  return 1.f - a * a;
}

template <class TDY, class TDX, int ACT, bool VEC>
__global__ void __launch_bounds__(256) ts_act_kernel(const TsMat dy, const TsCkpt c, const Groups g, const TsOut dx) {
  pdl_launch_dependents();
  pdl_wait();
  const int lane = threadIdx.x & 31;
  for_groups(g, [&](int64_t r, int c0) {
    float v[8], a[8];
    load_group<VEC>(static_cast<const TDY*>(dy.p) + r * dy.ld, c0, g.cols, lane, v);
    ckpt_load_group<VEC>(c, r, c0, lane, a);
#pragma unroll
    for (int j = 0; j < 8; ++j) v[j] *= act_slope<ACT>(a[j]);
    store_group<VEC>(static_cast<TDX*>(dx.p) + r * dx.ld, c0, g.cols, lane, v);
  });
}

Groups groups_of(int64_t rows, int cols) { return Groups{rows, cols, (cols + kGroupCols - 1) / kGroupCols}; }
int grid_for(const ts_ops& h, const Groups& g) {
  return (int)std::min<int64_t>((g.rows * g.per_row + 7) / 8, (int64_t)h.nsm * 8);
}

template <class... A, class... B>
cudaError_t start(void (*kernel)(A...), int grid, cudaStream_t st, const B&... args) {
  cudaLaunchConfig_t cfg = pdl_config(grid, 256, 0, st);
  cudaLaunchAttribute at[1];
  pdl_attr(cfg, at);
  return cudaLaunchKernelEx(&cfg, kernel, args...);
}

template <class TDY, class TDX, bool VEC>
cudaError_t act_of(int act, int grid, const TsMat& dy, const TsCkpt& c, const Groups& g, const TsOut& dx,
                   cudaStream_t st) {
  return act == 0   ? start(ts_act_kernel<TDY, TDX, 0, VEC>, grid, st, dy, c, g, dx)
         : act == 1 ? start(ts_act_kernel<TDY, TDX, 1, VEC>, grid, st, dy, c, g, dx)
                    : start(ts_act_kernel<TDY, TDX, 2, VEC>, grid, st, dy, c, g, dx);
}
template <class TDY, class TDX>
cudaError_t act_types(int act, int grid, const TsMat& dy, const TsCkpt& c, const Groups& g, const TsOut& dx,
                      cudaStream_t st) {
  return rows_aligned(dy) && rows_aligned(dx) ? act_of<TDY, TDX, true>(act, grid, dy, c, g, dx, st)
                                              : act_of<TDY, TDX, false>(act, grid, dy, c, g, dx, st);
}

}  // namespace

cudaError_t launch_checkpoint_save(const ts_ops& h, const TsMat& x, int64_t rows, int cols, const TsCkpt& c,
                                   cudaStream_t st) {
  const Groups g = groups_of(rows, cols);
  const int grid = grid_for(h, g);
  const bool vec = rows_aligned(x);
  if (x.bf16)
    return vec ? start(ts_save_kernel<__nv_bfloat16, true>, grid, st, x, g, c)
               : start(ts_save_kernel<__nv_bfloat16, false>, grid, st, x, g, c);
  return vec ? start(ts_save_kernel<float, true>, grid, st, x, g, c)
             : start(ts_save_kernel<float, false>, grid, st, x, g, c);
}

cudaError_t launch_checkpoint_load(const ts_ops& h, const TsCkpt& c, int64_t rows, int cols, const TsOut& y,
                                   cudaStream_t st) {
  const Groups g = groups_of(rows, cols);
  const int grid = grid_for(h, g);
  const bool vec = rows_aligned(y);
  if (y.bf16)
    return vec ? start(ts_load_kernel<__nv_bfloat16, true>, grid, st, c, g, y)
               : start(ts_load_kernel<__nv_bfloat16, false>, grid, st, c, g, y);
  return vec ? start(ts_load_kernel<float, true>, grid, st, c, g, y)
             : start(ts_load_kernel<float, false>, grid, st, c, g, y);
}

cudaError_t launch_activation_backward(const ts_ops& h, int act, const TsMat& dy, const TsCkpt& c, int64_t rows,
                                       int cols, const TsOut& dx, cudaStream_t st) {
  using B = __nv_bfloat16;
  const Groups g = groups_of(rows, cols);
  const int grid = grid_for(h, g);
  if (dy.bf16)
    return dx.bf16 ? act_types<B, B>(act, grid, dy, c, g, dx, st) : act_types<B, float>(act, grid, dy, c, g, dx, st);
  return dx.bf16 ? act_types<float, B>(act, grid, dy, c, g, dx, st)
                 : act_types<float, float>(act, grid, dy, c, g, dx, st);
}

}  // namespace fg
