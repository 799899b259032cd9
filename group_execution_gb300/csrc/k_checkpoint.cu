// 8-bit activation checkpoints (the OCP microscaling format with int8
// elements: blocks of 32 columns of a row share a power-of-two step): saving,
// loading, and the derivative of an activation from its saved output.
//
// A checkpoint's values are exact in bf16 (8 bits of significand) and the
// step's division is exact, so rounding to the nearest step is the only
// rounding on the way.  Each kernel is one pass, bound by device memory: at 8192
// x 4096 saving f32 takes 27 us (93 % of the copy rate), bf16 22 (67 %: the
// blocks' maxima and roundings are instructions a column, whatever its type),
// loading to bf16 16 (91 %), to f32 26 (95 %), relu's derivative in bf16 27
// (92 %), tanh's in f32 45 (99 %).
#include <algorithm>

#include "launch.h"
#include "ts_device.cuh"

namespace fg {
namespace {

// The matrix in pieces of one row, row by row: 128 columns to half a warp
// (aligned rows; a checkpoint's pitch is a multiple of that) or 256 to a warp.
// Each takes N consecutive pieces and loads all of them before it works on
// the first (one division to find its place).  us with N = 1, 2, 4: saving
// 8192 x 4096 in bf16 27, 22, 24; loading it to bf16 20, -, 16; the tanh
// derivative at 4097 x 4100 in bf16 18, -, 15.  With rows at odd elements, which
// move by single ones, N = 1 is fastest (more are too many registers): at 8192 x
// 4096 in bf16 saving takes 31 us, loading 28, the tanh derivative 35 (26
// aligned).
struct Pieces {
  int64_t rows;
  int cols, per_row;
};
template <bool VEC>
constexpr int kAtOnce = VEC ? 4 : 1;
template <bool VEC>
constexpr int kSaveAtOnce = VEC ? 2 : 1;

template <bool VEC>
constexpr int kPieceCols = VEC ? 128 : kGroupCols;

template <bool VEC, int N, class Load, class Use>
__device__ __forceinline__ void for_pieces(const Pieces& g, Load load, Use use) {
  constexpr int kLanes = VEC ? 16 : 32;
  const int64_t i = ((int64_t)blockIdx.x * (256 / kLanes) + threadIdx.x / kLanes) * N;
  int64_t row = i / g.per_row;
  int at = (int)(i - row * g.per_row);
  int64_t r[N];
  int c0[N];
#pragma unroll
  for (int u = 0; u < N; ++u) {
    r[u] = row;
    c0[u] = at * kPieceCols<VEC>;
    if (++at == g.per_row) {
      at = 0;
      ++row;
    }
  }
#pragma unroll
  for (int u = 0; u < N; ++u)
    if (r[u] < g.rows) load(u, r[u], c0[u]);
#pragma unroll
  for (int u = 0; u < N; ++u) {
    // (a warp's halves may end in different rows; the saved block's maximum
    // is taken across its four lanes)
    if (r[u] < g.rows) use(u, r[u], c0[u]);
  }
}

template <class TX, bool VEC>
__global__ void __launch_bounds__(256) ts_save_kernel(const TsMat x, const Pieces g, const TsCkpt c) {
  pdl_launch_dependents();
  pdl_wait();
  const int lane = threadIdx.x & (VEC ? 15 : 31);
  RawGroup<TX, VEC> raw[kSaveAtOnce<VEC>];
  __shared__ __align__(16) float scratch[VEC ? 1 : 8][kGroupCols];
  for_pieces<VEC, kSaveAtOnce<VEC>>(
      g,
      [&](int u, int64_t r, int c0) { raw[u].load(static_cast<const TX*>(x.p) + r * x.ld, c0, g.cols, lane); },
      [&](int u, int64_t r, int c0) {
        float v[8];
        raw[u].get(v);
        ckpt_store_group<VEC>(c, r, c0, lane, v, scratch[VEC ? 0 : threadIdx.x >> 5]);
      });
}

template <class TY, bool VEC>
__global__ void __launch_bounds__(256) ts_load_kernel(const TsCkpt c, const Pieces g, const TsOut y) {
  pdl_launch_dependents();
  pdl_wait();
  const int lane = threadIdx.x & (VEC ? 15 : 31);
  RawCkpt<VEC> raw[kAtOnce<VEC>];
  __shared__ __align__(8) CkptScratch<!VEC, 8> scratch;
  for_pieces<VEC, kAtOnce<VEC>>(
      g, [&](int u, int64_t r, int c0) { raw[u].load(c, r, c0, lane); },
      [&](int u, int64_t r, int c0) {
        float v[8];
        raw[u].get(v, lane, scratch.mine());
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
__global__ void __launch_bounds__(256) ts_act_kernel(const TsMat dy, const TsCkpt c, const Pieces g, const TsOut dx) {
  pdl_launch_dependents();
  pdl_wait();
  const int lane = threadIdx.x & (VEC ? 15 : 31);
  RawGroup<TDY, VEC> d[kAtOnce<VEC>];
  RawCkpt<VEC> raw[kAtOnce<VEC>];
  __shared__ __align__(8) CkptScratch<!VEC, 8> scratch;
  for_pieces<VEC, kAtOnce<VEC>>(
      g,
      [&](int u, int64_t r, int c0) {
        d[u].load(static_cast<const TDY*>(dy.p) + r * dy.ld, c0, g.cols, lane);
        raw[u].load(c, r, c0, lane);
      },
      [&](int u, int64_t r, int c0) {
        float v[8], a[8];
        d[u].get(v);
        raw[u].get(a, lane, scratch.mine());
#pragma unroll
        for (int j = 0; j < 8; ++j) v[j] *= act_slope<ACT>(a[j]);
        store_group<VEC>(static_cast<TDX*>(dx.p) + r * dx.ld, c0, g.cols, lane, v);
      });
}

Pieces pieces_of(int64_t rows, int cols, bool vec) {
  const int w = vec ? kPieceCols<true> : kPieceCols<false>;
  return Pieces{rows, cols, (cols + w - 1) / w};
}
int64_t grid_for(const Pieces& g, bool vec, int at_once) {
  const int64_t n = (256 / (vec ? 16 : 32)) * at_once;
  return (g.rows * g.per_row + n - 1) / n;
}

template <class... A, class... B>
cudaError_t start(void (*kernel)(A...), int64_t grid, cudaStream_t st, const B&... args) {
  if (grid > 0x7fffffff) return cudaErrorInvalidConfiguration;
  cudaLaunchConfig_t cfg = pdl_config((int)grid, 256, 0, st);
  cudaLaunchAttribute at[1];
  pdl_attr(cfg, at);
  return cudaLaunchKernelEx(&cfg, kernel, args...);
}

template <class TDY, class TDX, bool VEC>
cudaError_t act_of(int act, int64_t grid, const TsMat& dy, const TsCkpt& c, const Pieces& g, const TsOut& dx,
                   cudaStream_t st) {
  return act == 0   ? start(ts_act_kernel<TDY, TDX, 0, VEC>, grid, st, dy, c, g, dx)
         : act == 1 ? start(ts_act_kernel<TDY, TDX, 1, VEC>, grid, st, dy, c, g, dx)
                    : start(ts_act_kernel<TDY, TDX, 2, VEC>, grid, st, dy, c, g, dx);
}
template <class TDY, class TDX>
cudaError_t act_types(int act, bool vec, int64_t grid, const TsMat& dy, const TsCkpt& c, const Pieces& g, const TsOut& dx,
                      cudaStream_t st) {
  return vec ? act_of<TDY, TDX, true>(act, grid, dy, c, g, dx, st) : act_of<TDY, TDX, false>(act, grid, dy, c, g, dx, st);
}

}  // namespace

cudaError_t launch_checkpoint_save(const ts_ops&, const TsMat& x, int64_t rows, int cols, const TsCkpt& c,
                                   cudaStream_t st) {
  const bool vec = rows_aligned(x);
  const Pieces g = pieces_of(rows, cols, vec);
  const int64_t grid = grid_for(g, vec, vec ? kSaveAtOnce<true> : kSaveAtOnce<false>);
  if (x.bf16)
    return vec ? start(ts_save_kernel<__nv_bfloat16, true>, grid, st, x, g, c)
               : start(ts_save_kernel<__nv_bfloat16, false>, grid, st, x, g, c);
  return vec ? start(ts_save_kernel<float, true>, grid, st, x, g, c)
             : start(ts_save_kernel<float, false>, grid, st, x, g, c);
}

cudaError_t launch_checkpoint_load(const ts_ops&, const TsCkpt& c, int64_t rows, int cols, const TsOut& y,
                                   cudaStream_t st) {
  const bool vec = rows_aligned(y);
  const Pieces g = pieces_of(rows, cols, vec);
  const int64_t grid = grid_for(g, vec, vec ? kAtOnce<true> : kAtOnce<false>);
  if (y.bf16)
    return vec ? start(ts_load_kernel<__nv_bfloat16, true>, grid, st, c, g, y)
               : start(ts_load_kernel<__nv_bfloat16, false>, grid, st, c, g, y);
  return vec ? start(ts_load_kernel<float, true>, grid, st, c, g, y)
             : start(ts_load_kernel<float, false>, grid, st, c, g, y);
}

cudaError_t launch_activation_backward(const ts_ops&, int act, const TsMat& dy, const TsCkpt& c, int64_t rows,
                                       int cols, const TsOut& dx, cudaStream_t st) {
  using B = __nv_bfloat16;
  const bool vec = rows_aligned(dy) && rows_aligned(dx);
  const Pieces g = pieces_of(rows, cols, vec);
  const int64_t grid = grid_for(g, vec, vec ? kAtOnce<true> : kAtOnce<false>);
  if (dy.bf16)
    return dx.bf16 ? act_types<B, B>(act, vec, grid, dy, c, g, dx, st) : act_types<B, float>(act, vec, grid, dy, c, g, dx, st);
  return dx.bf16 ? act_types<float, B>(act, vec, grid, dy, c, g, dx, st)
                 : act_types<float, float>(act, vec, grid, dy, c, g, dx, st);
}

}  // namespace fg
