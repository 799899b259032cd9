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
#include <type_traits>

#include "launch.h"
#include "ts_device.cuh"

namespace fg {
namespace {

// Where the normalised row h comes from: x, or the checkpoint.
template <class TX>
struct FromX {
  using Dx = TX;
  template <bool VEC>
  struct Raw {
    static constexpr int kRegs = VEC ? (int)sizeof(TX) * 2 : 8;
    RawGroup<TX, VEC> x;
    __device__ __forceinline__ void load(const NormArgs& a, int64_t row, int c0, int lane) {
      x.load(static_cast<const TX*>(a.x.p) + row * a.x.ld, c0, a.cols, lane);
    }
    __device__ __forceinline__ void get(float mean, float rstd, float (&h)[8]) const {
      x.get(h);
#pragma unroll
      for (int j = 0; j < 8; ++j) h[j] = (h[j] - mean) * rstd;
    }
  };
  __device__ __forceinline__ static float mean(const NormArgs& a, int64_t row) { return a.mean[row]; }
};
template <class TDX>
struct FromCkpt {
  using Dx = TDX;
  template <bool VEC>
  struct Raw {
    static constexpr int kRegs = VEC ? 3 : 16;
    RawCkpt<VEC> c;
    __device__ __forceinline__ void load(const NormArgs& a, int64_t row, int c0, int lane) {
      c.load(a.ckpt, row, c0, lane);
    }
    __device__ __forceinline__ void get(float, float, float (&h)[8]) const { c.get(h); }
  };
  __device__ __forceinline__ static float mean(const NormArgs&, int64_t) { return 0.f; }
};
template <class Src, bool VEC>
__device__ __forceinline__ void load_h(const NormArgs& a, int64_t row, int c0, int lane, float mean, float rstd,
                                       float (&h)[8]) {
  typename Src::template Raw<VEC> r;
  r.load(a, row, c0, lane);
  r.get(mean, rstd, h);
}

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
    load_h<Src, VEC>(a, row, c0, lane, mean, rstd, h);
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
    load_h<Src, VEC>(a, row, c0, lane, mean, rstd, h);
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
// run of 8 rows, a warp a row, four runs in flight; the block's warps are
// added in order.  part: [gridDim.y][2][cols], dy's sums and then, with a
// Src, dy h's.
template <class TDY, class Src, bool VEC>
__global__ void __launch_bounds__(256) ts_column_kernel(const NormArgs a, float* part) {
  __shared__ float sm[8][2][kGroupCols];
  pdl_launch_dependents();
  pdl_wait();
  constexpr bool kH = !std::is_void<Src>::value;
  constexpr int kU = 4;
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int c0 = blockIdx.x * kGroupCols;
  float sb[8] = {}, sg[8] = {};
  const int64_t step = (int64_t)gridDim.y * 8;
  for (int64_t row = (int64_t)blockIdx.y * 8 + warp; row < a.rows; row += step * kU) {
    RawGroup<TDY, VEC> d[kU];
#pragma unroll
    for (int u = 0; u < kU; ++u)
      if (row + u * step < a.rows)
        d[u].load(static_cast<const TDY*>(a.dy.p) + (row + u * step) * a.dy.ld, c0, a.cols, lane);
#pragma unroll
    for (int u = 0; u < kU; ++u) {
      const int64_t rr = row + u * step;
      if (rr >= a.rows) break;
      float v[8];
      d[u].get(v);
#pragma unroll
      for (int j = 0; j < 8; ++j) sb[j] += v[j];
      if constexpr (kH) {
        float h[8];
        typename Src::template Raw<VEC> raw;
        raw.load(a, rr, c0, lane);
        raw.get(Src::mean(a, rr), a.rstd[rr], h);
#pragma unroll
        for (int j = 0; j < 8; ++j) sg[j] += v[j] * h[j];
      }
    }
  }
#pragma unroll
  for (int j = 0; j < 8; ++j) {
    sm[warp][0][group_col<VEC>(lane, j)] = sb[j];
    if (kH) sm[warp][1][group_col<VEC>(lane, j)] = sg[j];
  }
  __syncthreads();
  const int c = c0 + threadIdx.x;
  if (c < a.cols) {
    float b = 0.f, g = 0.f;
#pragma unroll
    for (int w = 0; w < 8; ++w) {
      b += sm[w][0][threadIdx.x];
      if (kH) g += sm[w][1][threadIdx.x];
    }
    part[((int64_t)blockIdx.y * 2 + 0) * a.cols + c] = b;
    if (kH) part[((int64_t)blockIdx.y * 2 + 1) * a.cols + c] = g;
  }
}

// Rows of at most 256 * G * W columns, W = 1, 2, 4, 8 or 16: dx and the
// partial column sums in one pass.  A block of 16 warps has 16 / W row slots,
// W warps a slot, G groups of 256 columns a warp.  A slot works on R rows at
// once (one barrier and one chain of shuffles for all of them) and walks its
// rows with the next D in flight in registers (one block an SM: with two, 64
// registers a thread do not hold this).  A thread meets the same columns in
// every row, so gamma (G = 1) and both column sums stay in its registers; at
// the end the block adds its slots in order and writes one partial.
template <class TDY, class Src, bool VEC, int G, int D, int R>
__global__ void __launch_bounds__(512, 1) ts_norm_backward_kernel(const NormArgs a, int W, float* part) {
  static_assert(D % R == 0, "whole sets of rows in flight");
  __shared__ float red[2][2 * R][16];
  __shared__ float sums[G == 1 ? 2 * 16 * kGroupCols : 1];   // the slots' column sums (G = 1, W < 16)
  pdl_launch_dependents();
  pdl_wait();
  const int lane = threadIdx.x & 31, slot = (threadIdx.x >> 5) / W, warp = (threadIdx.x >> 5) % W;
  const int slots = 16 / W;
  F2 gamma[4], sb[G][4] = {}, sg[G][4] = {};
  auto load_gamma = [&](int g) {
    float v[8] = {1.f, 1.f, 1.f, 1.f, 1.f, 1.f, 1.f, 1.f};
    if (a.gamma) load_group<VEC>(a.gamma, (g * W + warp) * kGroupCols, a.cols, lane, v);
#pragma unroll
    for (int j = 0; j < 4; ++j) gamma[j] = pack2f(v[2 * j], v[2 * j + 1]);
  };
  load_gamma(0);
  const float n = 1.f / (float)a.cols;
  const int64_t step = (int64_t)gridDim.x * slots;
  int64_t row = (int64_t)blockIdx.x * slots + slot;
  RawGroup<TDY, VEC> dy[D][G];
  typename Src::template Raw<VEC> x[D][G];
  float mean[D], rstd[D];
  auto fetch = [&](int d, int64_t r) {
    if (r >= a.rows) return;
#pragma unroll
    for (int g = 0; g < G; ++g) {
      const int c0 = (g * W + warp) * kGroupCols;
      dy[d][g].load(static_cast<const TDY*>(a.dy.p) + r * a.dy.ld, c0, a.cols, lane);
      x[d][g].load(a, r, c0, lane);
    }
    mean[d] = Src::mean(a, r);
    rstd[d] = a.rstd[r];
  };
#pragma unroll
  for (int d = 0; d < D; ++d) fetch(d, row + d * step);
  int buf = 0;
  while (row < a.rows) {
#pragma unroll
    for (int d = 0; d < D; d += R) {
      if (row >= a.rows) break;
      F2 u[R][G][4], h[R][G][4];
      float rs[R], s[2 * R];
#pragma unroll
      for (int k = 0; k < R; ++k) {
        F2 s1 = 0, s2 = 0;
        rs[k] = 0.f;
        if (k == 0 || row + k * step < a.rows) {
          rs[k] = rstd[d + k];
#pragma unroll
          for (int g = 0; g < G; ++g) {
            float du[8], dh[8];
            dy[d + k][g].get(du);
            x[d + k][g].get(mean[d + k], rs[k], dh);
            if (G > 1) load_gamma(g);   // (from L1)
#pragma unroll
            for (int j = 0; j < 4; ++j) {
              const F2 v = pack2f(du[2 * j], du[2 * j + 1]);
              h[k][g][j] = pack2f(dh[2 * j], dh[2 * j + 1]);
              sb[g][j] = add2(sb[g][j], v);
              sg[g][j] = fma2(v, h[k][g][j], sg[g][j]);
              u[k][g][j] = mul2(v, gamma[j]);
              s1 = add2(s1, u[k][g][j]);
              s2 = fma2(u[k][g][j], h[k][g][j], s2);
            }
          }
        }
        s[2 * k] = sum2(s1);
        s[2 * k + 1] = sum2(s2);
      }
#pragma unroll
      for (int k = 0; k < R; ++k) fetch(d + k, row + (D + k) * step);
#pragma unroll
      for (int o = 16; o > 0; o >>= 1)
#pragma unroll
        for (int k = 0; k < 2 * R; ++k) s[k] += __shfl_xor_sync(0xffffffffu, s[k], o);
      if (W > 1) {
        if (lane == 0) {
#pragma unroll
          for (int k = 0; k < 2 * R; ++k) red[buf][k][slot * W + warp] = s[k];
        }
        named_bar_sync(1 + slot, W * 32);
        // lanes 0-15 add the rows' first sums, 16-31 the second ones, in a
        // fixed tree
#pragma unroll
        for (int k = 0; k < R; ++k) {
          float v = (lane & 15) < W ? red[buf][2 * k + (lane >> 4)][slot * W + (lane & 15)] : 0.f;
#pragma unroll
          for (int o = 8; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
          s[2 * k] = __shfl_sync(0xffffffffu, v, 0);
          s[2 * k + 1] = __shfl_sync(0xffffffffu, v, 16);
        }
        buf ^= 1;   // (the next sums go to the other half, so one barrier is enough)
      }
#pragma unroll
      for (int k = 0; k < R; ++k) {
        if (k && row >= a.rows) break;
        // dx = r u - r m1 - h r m2
        const float m1 = -rs[k] * (s[2 * k] * n), m2 = -rs[k] * (s[2 * k + 1] * n);
        const F2 rr = pack2f(rs[k], rs[k]), mm1 = pack2f(m1, m1), mm2 = pack2f(m2, m2);
#pragma unroll
        for (int g = 0; g < G; ++g) {
          float o[8];
#pragma unroll
          for (int j = 0; j < 4; ++j)
            unpack2f(fma2(h[k][g][j], mm2, fma2(u[k][g][j], rr, mm1)), o[2 * j], o[2 * j + 1]);
          store_group<VEC>(static_cast<typename Src::Dx*>(a.dx.p) + row * a.dx.ld, (g * W + warp) * kGroupCols, a.cols,
                           lane, o);
        }
        row += step;
      }
    }
  }
  if (!part) return;
  float* p = part + (int64_t)blockIdx.x * 2 * a.cols;
  const int width = W * kGroupCols;
#pragma unroll
  for (int g = 0; g < G; ++g)
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      const int c = (g * W + warp) * kGroupCols + group_col<VEC>(lane, j);
      float b[2], q[2];
      unpack2f(sb[g][j / 2], b[0], b[1]);
      unpack2f(sg[g][j / 2], q[0], q[1]);
      if (G == 1 && slots > 1) {
        sums[(slot * 2 + 0) * width + c] = b[j & 1];
        sums[(slot * 2 + 1) * width + c] = q[j & 1];
      } else if (c < a.cols) {
        p[c] = b[j & 1];
        p[a.cols + c] = q[j & 1];
      }
    }
  if (G == 1 && slots > 1) {
    __syncthreads();
    for (int i = threadIdx.x; i < 2 * width; i += 512) {
      const int c = i % width, which = i / width;
      if (c >= a.cols) continue;
      float v = 0.f;
      for (int k = 0; k < slots; ++k) v += sums[(k * 2 + which) * width + c];
      p[which * a.cols + c] = v;
    }
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

template <class TDY, class Src, bool VEC, int G, int D, int R>
cudaError_t backward_fused(const ts_ops& h, const NormArgs& a, int W, cudaStream_t st) {
  // one block an SM, a partial a block
  const int slots = 16 / W;
  int64_t grid = std::min<int64_t>((a.rows + slots - 1) / slots, h.nsm);
  grid = std::max<int64_t>(1, std::min(grid, (h.ws_bytes - 8 * (int64_t)a.cols) / (8 * (int64_t)a.cols)));
  float* part = a.dgamma || a.dbeta ? reinterpret_cast<float*>(h.ws) : nullptr;
  cudaLaunchConfig_t cfg = pdl_config((int)grid, 512, 0, st);
  cudaLaunchAttribute at[1];
  pdl_attr(cfg, at);
  cudaError_t e = cudaLaunchKernelEx(&cfg, ts_norm_backward_kernel<TDY, Src, VEC, G, D, R>, a, W, part);
  if (e != cudaSuccess || !part) return e;
  return finish_columns(part, (int)grid, a.cols, a.dbeta, a.dgamma, a.accumulate, nullptr, st);
}

template <class TDY, class Src, bool VEC>
cudaError_t backward_rows(const ts_ops& h, const NormArgs& a, cudaStream_t st) {
  // rows in flight: what about 32 registers hold
  constexpr int kRegs = (VEC ? (int)sizeof(TDY) * 2 : 8) + Src::template Raw<VEC>::kRegs;
  constexpr int D = kRegs <= 8 ? 4 : kRegs <= 16 ? 2 : 1, R = D > 1 ? 2 : 1;
  if (a.rows > 0 && a.cols <= 16 * kGroupCols) {
    int W = 1;
    while (W * kGroupCols < a.cols) W *= 2;
    return backward_fused<TDY, Src, VEC, 1, D, R>(h, a, W, st);
  }
  if (a.rows > 0 && a.cols <= 32 * kGroupCols) return backward_fused<TDY, Src, VEC, 2, 1, 1>(h, a, 16, st);
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
