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
#include <atomic>
#include <type_traits>

#include "launch.h"
#include "ts_device.cuh"

namespace fg {
namespace {

// A row of a block of 1024 threads, on its way to L2.
__device__ __forceinline__ void prefetch_row(const void* p, int bytes) {
  for (int i = threadIdx.x * 128; i < bytes; i += 1024 * 128)
    asm volatile("prefetch.global.L2 [%0];" ::"l"(static_cast<const char*>(p) + i));
}

// Where the normalised row h comes from: x, or the checkpoint.  An object is a
// cursor on a row; Raw holds a group of it as it lies in memory.
template <class TX>
struct FromX {
  using Dx = TX;
  static constexpr bool kCkpt = false;
  const TX* row;
  __device__ __forceinline__ FromX(const NormArgs& a, int64_t r) : row(static_cast<const TX*>(a.x.p) + r * a.x.ld) {}
  __device__ __forceinline__ void advance(const NormArgs& a, int64_t rows) { row += rows * a.x.ld; }
  template <bool VEC>
  struct Raw {
    RawGroup<TX, VEC> x;
    __device__ __forceinline__ void load(const NormArgs& a, const FromX& s, int c0, int lane) {
      x.load(s.row, c0, a.cols, lane);
    }
    __device__ __forceinline__ void get(float (&v)[8], int, int8_t*) const { x.get(v); }   // x itself
  };
  __device__ __forceinline__ static float mean(const NormArgs& a, int64_t row) { return a.mean[row]; }
  __device__ __forceinline__ static void prefetch(const NormArgs& a, int64_t row) {
    prefetch_row(static_cast<const TX*>(a.x.p) + row * a.x.ld, a.cols * (int)sizeof(TX));
  }
};
template <class TDX>
struct FromCkpt {
  using Dx = TDX;
  static constexpr bool kCkpt = true;
  TsCkpt row;   // a view of this one row
  __device__ __forceinline__ FromCkpt(const NormArgs& a, int64_t r) : row(a.ckpt) { move(r); }
  __device__ __forceinline__ void move(int64_t rows) {
    row.q += rows * row.pitch;
    row.scale += rows * (row.pitch / kCkptBlock);
  }
  __device__ __forceinline__ void advance(const NormArgs&, int64_t rows) { move(rows); }
  template <bool VEC>
  struct Raw {
    RawCkpt<VEC> c;
    __device__ __forceinline__ void load(const NormArgs&, const FromCkpt& s, int c0, int lane) {
      c.load(s.row, 0, c0, lane);
    }
    __device__ __forceinline__ void get(float (&v)[8], int lane, int8_t* scratch) const {
      c.get(v, lane, scratch);   // h
    }
  };
  __device__ __forceinline__ static float mean(const NormArgs&, int64_t) { return 0.f; }
  __device__ __forceinline__ static void prefetch(const NormArgs& a, int64_t row) {
    prefetch_row(a.ckpt.q + row * a.ckpt.pitch, (int)a.ckpt.pitch);
    prefetch_row(a.ckpt.scale + row * (a.ckpt.pitch / kCkptBlock), (int)(a.ckpt.pitch / kCkptBlock));
  }
};
template <class Src, bool VEC>
__device__ __forceinline__ void load_h(const NormArgs& a, int64_t row, int c0, int lane, float mean, float rstd,
                                       float (&h)[8], int8_t* scratch) {
  typename Src::template Raw<VEC> r;
  r.load(a, Src(a, row), c0, lane);
  r.get(h, lane, scratch);
  if (!Src::kCkpt) {
#pragma unroll
    for (int j = 0; j < 8; ++j) h[j] = (h[j] - mean) * rstd;
  }
}

// dx alone: one block a row, any length.  With the column sums' kernel below,
// which reads the operands again, it takes the rows that no block's registers
// hold, beyond 16384 columns.
template <class TDY, class Src, bool VEC>
__global__ void __launch_bounds__(256) ts_norm_dx_kernel(const NormArgs a) {
  __shared__ float red[2][8];
  __shared__ __align__(8) CkptScratch<Src::kCkpt && !VEC, 8> scratch;
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
    load_h<Src, VEC>(a, row, c0, lane, mean, rstd, h, scratch.mine());
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
    load_h<Src, VEC>(a, row, c0, lane, mean, rstd, h, scratch.mine());
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
// Src, dy h's; null with one block to a column, which then finishes it (fresh
// as below).
template <class TDY, class Src, bool VEC>
__global__ void __launch_bounds__(256) ts_column_kernel(const NormArgs a, float* part, float* fresh) {
  __shared__ float sm[8][2][kGroupCols];
  constexpr bool kH = !std::is_void<Src>::value;
  __shared__ __align__(8) CkptScratch<kH && !VEC, 8> scratch;
  pdl_launch_dependents();
  pdl_wait();
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
        load_h<Src, VEC>(a, rr, c0, lane, Src::mean(a, rr), a.rstd[rr], h, scratch.mine());
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
    if (!part) {
      if (fresh) fresh[c] = b;
      if (a.dbeta) a.dbeta[c] = a.accumulate ? a.dbeta[c] + b : b;
      if (kH && a.dgamma) a.dgamma[c] = a.accumulate ? a.dgamma[c] + g : g;
      return;
    }
    part[((int64_t)blockIdx.y * 2 + 0) * a.cols + c] = b;
    if (kH) part[((int64_t)blockIdx.y * 2 + 1) * a.cols + c] = g;
  }
}

// Two values a row, of K = 1 or 2 rows, summed over a warp: each step halves
// what a lane still carries, so five or six shuffles do it.  Lanes 0 .. 16 / K
// - 1 end with the sum of the first value, the next 16 / K with the second,
// and so on.
template <int K>
__device__ __forceinline__ float warp_sums(const float (&s)[2 * K], int lane) {
  float v;
  if constexpr (K == 2) {
    const bool hi = lane & 16, mid = lane & 8;
    float x = hi ? s[2] : s[0], y = hi ? s[3] : s[1];
    x += __shfl_xor_sync(0xffffffffu, hi ? s[0] : s[2], 16);
    y += __shfl_xor_sync(0xffffffffu, hi ? s[1] : s[3], 16);
    v = mid ? y : x;
    v += __shfl_xor_sync(0xffffffffu, mid ? x : y, 8);
  } else {
    const bool hi = lane & 16;
    v = hi ? s[1] : s[0];
    v += __shfl_xor_sync(0xffffffffu, hi ? s[0] : s[1], 16);
    v += __shfl_xor_sync(0xffffffffu, v, 8);
  }
#pragma unroll
  for (int o = 4; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
  return v;
}

// Rows of at most 256 * G * W columns, W = 1, 2, 4, 8 or 16: dx and the
// partial column sums in one pass.  A block of 16 warps has 16 / W row slots,
// W warps a slot, G groups of 256 columns a warp.  A slot works on K rows at
// once (one barrier and one chain of shuffles for both) and walks its rows
// with the next K D in flight in registers (one block an SM: with two, 64
// registers a thread do not hold this).  A thread meets the same columns in
// every row, so gamma (G = 1) and both column sums stay in its registers; at
// the end the block adds its slots in order and writes one partial.
//
// Bound by latency before memory in bf16: a warp's 152 instructions for 256
// columns of a row (pairs of float32 operations in one, addresses advanced by
// addition) keep the schedulers busy in 46 % of the cycles, and the SM's 16
// warps wait for shuffles, shared memory, loads and the barrier of each pair of
// rows.  8192 x 4096 takes 44 us in bf16 (67 % of the copy rate), 64 in f32 (92
// %); G = 2 at 4096 x 8192 bf16 takes 48 and f32 72 (84 with the choice of
// stores).  (A partial written by single elements, 32 bytes apart across a warp,
// cost 3 to 7 us.)  1021 x 5003 f32 from the checkpoint, whose rows of dy and dx
// start at odd elements and move by single ones, and whose second group of
// columns most warps lack, takes 21 us (32 %).  About 4 us of each is the kernel
// that adds the partials.
template <class TDY, class Src, bool VEC, int G, int D, int K>
__global__ void __launch_bounds__(512, 1) ts_norm_backward_kernel(const NormArgs a, int W, float* part) {
  __shared__ float red[2][16][4];   // [warp][value]
  __shared__ __align__(8) CkptScratch<Src::kCkpt && !VEC, 16> scratch;
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
  const int rows = (int)a.rows, step = gridDim.x * slots, first = blockIdx.x * slots + slot;
  RawGroup<TDY, VEC> dy[D][K][G];
  typename Src::template Raw<VEC> x[D][K][G];
  float mean[D][K], rstd[D][K];
  // the row that is fetched next
  int at = first;
  const TDY* dyp = static_cast<const TDY*>(a.dy.p) + (int64_t)first * a.dy.ld;
  Src src(a, first);
  const int64_t dy_step = (int64_t)step * a.dy.ld;
  auto fetch = [&](int d, int k) {
    if (at < rows) {
#pragma unroll
      for (int g = 0; g < G; ++g) {
        const int c0 = (g * W + warp) * kGroupCols;
        dy[d][k][g].load(dyp, c0, a.cols, lane);
        x[d][k][g].load(a, src, c0, lane);
      }
      mean[d][k] = Src::mean(a, at);
      rstd[d][k] = a.rstd[at];
    }
    at += step;
    dyp += dy_step;
    src.advance(a, step);
  };
#pragma unroll
  for (int d = 0; d < D; ++d)
#pragma unroll
    for (int k = 0; k < K; ++k) fetch(d, k);
  int buf = 0;
  typename Src::Dx* dx = static_cast<typename Src::Dx*>(a.dx.p) + (int64_t)first * a.dx.ld;
  const int64_t dx_step = (int64_t)step * a.dx.ld;
  for (int row = first; row < rows;) {
#pragma unroll
    for (int d = 0; d < D; ++d) {
      if (row >= rows) break;
      const bool two = K == 2 && row + step < rows;
      F2 u[K][G][4], h[K][G][4];
      float rs[K], s[2 * K];
#pragma unroll
      for (int k = 0; k < K; ++k) {
        F2 s1 = 0, s2 = 0;
        rs[k] = 0.f;
        if (k == 0 || two) {
          rs[k] = rstd[d][k];
          const F2 scale = pack2f(rs[k], rs[k]), shift = pack2f(-mean[d][k], -mean[d][k]);
#pragma unroll
          for (int g = 0; g < G; ++g) {
            float du[8], dh[8];
            dy[d][k][g].get(du);
            x[d][k][g].get(dh, lane, scratch.mine());
            if (G > 1) load_gamma(g);   // (from L1)
#pragma unroll
            for (int j = 0; j < 4; ++j) {
              const F2 v = pack2f(du[2 * j], du[2 * j + 1]);
              F2 hh = pack2f(dh[2 * j], dh[2 * j + 1]);
              if (!Src::kCkpt) hh = mul2(add2(hh, shift), scale);
              h[k][g][j] = hh;
              sb[g][j] = add2(sb[g][j], v);
              sg[g][j] = fma2(v, hh, sg[g][j]);
              u[k][g][j] = mul2(v, gamma[j]);
              s1 = add2(s1, u[k][g][j]);
              s2 = fma2(u[k][g][j], hh, s2);
            }
          }
        }
        s[2 * k] = sum2(s1);
        s[2 * k + 1] = sum2(s2);
      }
#pragma unroll
      for (int k = 0; k < K; ++k) fetch(d, k);
      constexpr int kLanes = 16 / K;   // that share a value
      float v = warp_sums<K>(s, lane);
      if (W > 1) {
        if (lane % kLanes == 0) red[buf][slot * W + warp][lane / kLanes] = v;
        named_bar_sync(1 + slot, W * 32);
        // the lanes that share a value add the warps', K each, in a fixed tree
        const int w = (lane % kLanes) * K;
        v = 0.f;
        if (w < W) {
          v = red[buf][slot * W + w][lane / kLanes];
          if (K == 2) v += red[buf][slot * W + w + 1][lane / kLanes];
        }
#pragma unroll
        for (int o = kLanes / 2; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
        buf ^= 1;   // (the next sums go to the other half, so one barrier is enough)
      }
      v *= n;
#pragma unroll
      for (int k = 0; k < K; ++k) {
        const float m1 = -rs[k] * __shfl_sync(0xffffffffu, v, 2 * kLanes * k);
        const float m2 = -rs[k] * __shfl_sync(0xffffffffu, v, 2 * kLanes * k + kLanes);
        if (k && !two) break;
        // dx = r u - r m1 - h r m2
        const F2 rr = pack2f(rs[k], rs[k]), a1 = pack2f(m1, m1), a2 = pack2f(m2, m2);
#pragma unroll
        for (int g = 0; g < G; ++g) {
          float o[8];
#pragma unroll
          for (int j = 0; j < 4; ++j)
            unpack2f(fma2(h[k][g][j], a2, fma2(u[k][g][j], rr, a1)), o[2 * j], o[2 * j + 1]);
          store_group<VEC, G == 2>(dx, (g * W + warp) * kGroupCols, a.cols, lane, o);
        }
        dx += dx_step;
      }
      row += K * step;
    }
  }
  if (!part) return;
  float* p = part + (int64_t)blockIdx.x * 2 * a.cols;
  const int width = W * kGroupCols;
#pragma unroll
  for (int g = 0; g < G; ++g) {
    float b[8], q[8];
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      unpack2f(sb[g][j], b[2 * j], b[2 * j + 1]);
      unpack2f(sg[g][j], q[2 * j], q[2 * j + 1]);
    }
    const int c0 = (g * W + warp) * kGroupCols;
    if (VEC && slots == 1 && a.cols % 4 == 0 && c0 + lane * 8 + 8 <= a.cols) {
      store8(p + c0 + lane * 8, b);   // (a partial's rows start on 16 bytes)
      store8(p + a.cols + c0 + lane * 8, q);
      continue;
    }
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      const int c = c0 + group_col<VEC>(lane, j);
      if (G == 1 && slots > 1) {
        sums[(slot * 2 + 0) * width + c] = b[j];
        sums[(slot * 2 + 1) * width + c] = q[j];
      } else if (c < a.cols) {
        p[c] = b[j];
        p[a.cols + c] = q[j];
      }
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

// Rows of up to 16384 columns: dx and the partial column sums in one pass, a
// block of 32 warps to an SM, two groups of 256 columns a warp.  gamma and the
// column sums live in shared memory (192 KB), where a thread meets its own
// columns alone, four at a time; the registers hold the row, and the next one
// is on its way to L2.  2048 x 16384 bf16 takes 50 us (59 % of the copy rate;
// by the two kernels that longer rows take, 99), 2388 x 10336 f32 68 (129).  Up
// to 8192 columns, where column sums fit the registers above, those are
// faster: 4096 x 8192 bf16 48 us, here 82.
constexpr int kWideGroups = 2, kWidePlane = kWideGroups * 2 * 1024;   // float4s of one value a column
constexpr int kWideSmem = 3 * kWidePlane * 16;

template <class TDY, class Src, bool VEC>
__global__ void __launch_bounds__(1024, 1) ts_norm_backward_wide_kernel(const NormArgs a, float* part) {
  extern __shared__ float4 wide[];
  __shared__ float red[2][2][32];   // [value][warp]
  __shared__ __align__(8) CkptScratch<Src::kCkpt && !VEC, 32> scratch;
  pdl_launch_dependents();
  pdl_wait();
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  float4* const gamma = wide + threadIdx.x;   // [group][half][thread]
  float4* const sb = gamma + kWidePlane;
  float4* const sg = sb + kWidePlane;
#pragma unroll
  for (int g = 0; g < kWideGroups; ++g) {
    float v[8] = {1.f, 1.f, 1.f, 1.f, 1.f, 1.f, 1.f, 1.f};
    if (a.gamma) load_group<VEC>(a.gamma, (g * 32 + warp) * kGroupCols, a.cols, lane, v);
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      gamma[(g * 2 + i) * 1024] = make_float4(v[4 * i], v[4 * i + 1], v[4 * i + 2], v[4 * i + 3]);
      sb[(g * 2 + i) * 1024] = sg[(g * 2 + i) * 1024] = make_float4(0.f, 0.f, 0.f, 0.f);
    }
  }
  const float n = 1.f / (float)a.cols;
  int buf = 0;
  for (int64_t row = blockIdx.x; row < a.rows; row += gridDim.x) {
    const TDY* dyp = static_cast<const TDY*>(a.dy.p) + row * a.dy.ld;
    const Src src(a, row);
    RawGroup<TDY, VEC> dy[kWideGroups];
    typename Src::template Raw<VEC> x[kWideGroups];
#pragma unroll
    for (int g = 0; g < kWideGroups; ++g) {
      dy[g].load(dyp, (g * 32 + warp) * kGroupCols, a.cols, lane);
      x[g].load(a, src, (g * 32 + warp) * kGroupCols, lane);
    }
    const float rs = a.rstd[row], mean = Src::mean(a, row);
    if (row + gridDim.x < a.rows) {
      prefetch_row(dyp + gridDim.x * a.dy.ld, a.cols * (int)sizeof(TDY));
      Src::prefetch(a, row + gridDim.x);
    }
    const F2 scale = pack2f(rs, rs), shift = pack2f(-mean, -mean);
    F2 u[kWideGroups][4], h[kWideGroups][4], s1 = 0, s2 = 0;
#pragma unroll
    for (int g = 0; g < kWideGroups; ++g) {
      float du[8], dh[8];
      dy[g].get(du);
      x[g].get(dh, lane, scratch.mine());
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        const int at = (g * 2 + i) * 1024;
        const float4 gm = gamma[at];
        float4 b = sb[at], q = sg[at];
        const F2 g2[2] = {pack2f(gm.x, gm.y), pack2f(gm.z, gm.w)};
        F2 b2[2] = {pack2f(b.x, b.y), pack2f(b.z, b.w)}, q2[2] = {pack2f(q.x, q.y), pack2f(q.z, q.w)};
#pragma unroll
        for (int j = 0; j < 2; ++j) {
          const int e = i * 4 + j * 2;
          const F2 v = pack2f(du[e], du[e + 1]);
          F2 hh = pack2f(dh[e], dh[e + 1]);
          if (!Src::kCkpt) hh = mul2(add2(hh, shift), scale);
          b2[j] = add2(b2[j], v);
          q2[j] = fma2(v, hh, q2[j]);
          const F2 w = mul2(v, g2[j]);
          s1 = add2(s1, w);
          s2 = fma2(w, hh, s2);
          u[g][i * 2 + j] = w;
          h[g][i * 2 + j] = hh;
        }
        unpack2f(b2[0], b.x, b.y);
        unpack2f(b2[1], b.z, b.w);
        unpack2f(q2[0], q.x, q.y);
        unpack2f(q2[1], q.z, q.w);
        sb[at] = b;
        sg[at] = q;
      }
    }
    const float s[2] = {sum2(s1), sum2(s2)};
    float v = warp_sums<1>(s, lane);
    if (lane % 16 == 0) red[buf][lane / 16][warp] = v;
    __syncthreads();
    // sixteen lanes to a value, two warps' sums each
    v = red[buf][lane / 16][lane % 16 * 2] + red[buf][lane / 16][lane % 16 * 2 + 1];
#pragma unroll
    for (int o = 8; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
    buf ^= 1;   // (the next sums go to the other half, so one barrier is enough)
    v *= -rs * n;
    const float m1 = __shfl_sync(0xffffffffu, v, 0), m2 = __shfl_sync(0xffffffffu, v, 16);
    const F2 a1 = pack2f(m1, m1), a2 = pack2f(m2, m2);
    typename Src::Dx* dx = static_cast<typename Src::Dx*>(a.dx.p) + row * a.dx.ld;
#pragma unroll
    for (int g = 0; g < kWideGroups; ++g) {
      float o[8];
#pragma unroll
      for (int j = 0; j < 4; ++j)
        unpack2f(fma2(h[g][j], a2, fma2(u[g][j], scale, a1)), o[2 * j], o[2 * j + 1]);
      store_group<VEC>(dx, (g * 32 + warp) * kGroupCols, a.cols, lane, o);
    }
  }
  if (!part) return;
  __syncthreads();
  float* p = part + (int64_t)blockIdx.x * 2 * a.cols;
  const float* sums = reinterpret_cast<const float*>(wide + kWidePlane);
  for (int c = threadIdx.x; c < a.cols; c += 1024) {
    const int group = c / kGroupCols, in = c % kGroupCols, l = VEC ? in / 8 : in % 32, j = VEC ? in % 8 : in / 32;
    const int at = ((group / 32 * 2 + j / 4) * 1024 + group % 32 * 32 + l) * 4 + j % 4;
    p[c] = sums[at];
    p[a.cols + c] = sums[kWidePlane * 4 + at];
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
// at least (one block spares the second kernel: the bias gradient beside a
// weight gradient of 3 x 511 x 264 takes 1.0 us more in place of 2.0; at 120
// rows the longer block takes what it spares), partials that fit the workspace (less its last 8 bytes a column,
// kept for a call's own sums).
int column_parts(const ts_ops& h, int64_t rows, int cols) {
  const int64_t tiles = (cols + kGroupCols - 1) / kGroupCols;
  int64_t p = (8 * (int64_t)h.nsm + tiles - 1) / tiles;
  p = std::min(p, (rows + 63) / 64);
  p = std::min(p, (h.ws_bytes - 8 * (int64_t)cols - 256) / (8 * (int64_t)cols));
  return (int)std::max<int64_t>(std::min<int64_t>(p, 65535), 1);
}

template <class TDY, class Src, bool VEC>
cudaError_t columns(const ts_ops& h, const NormArgs& a, float* fresh, cudaStream_t st) {
  const int parts = column_parts(h, a.rows, a.cols);
  cudaLaunchConfig_t cfg = pdl_config(1, 256, 0, st);
  cfg.gridDim = dim3((a.cols + kGroupCols - 1) / kGroupCols, parts);
  cudaLaunchAttribute at[1];
  pdl_attr(cfg, at);
  float* part = parts > 1 ? reinterpret_cast<float*>(h.ws) : nullptr;
  cudaError_t e = cudaLaunchKernelEx(&cfg, ts_column_kernel<TDY, Src, VEC>, a, part, fresh);
  if (e != cudaSuccess || !part) return e;
  return finish_columns(part, parts, a.cols, a.dbeta, a.dgamma, a.accumulate, fresh, st);
}

template <class TDY, class Src, bool VEC, int G, int D, int K>
cudaError_t backward_fused(const ts_ops& h, const NormArgs& a, int W, cudaStream_t st) {
  // one block an SM, a partial a block
  const int slots = 16 / W;
  int64_t grid = std::min<int64_t>((a.rows + slots - 1) / slots, h.nsm);
  grid = std::max<int64_t>(1, std::min(grid, (h.ws_bytes - 8 * (int64_t)a.cols) / (8 * (int64_t)a.cols)));
  float* part = a.dgamma || a.dbeta ? reinterpret_cast<float*>(h.ws) : nullptr;
  cudaLaunchConfig_t cfg = pdl_config((int)grid, 512, 0, st);
  cudaLaunchAttribute at[1];
  pdl_attr(cfg, at);
  cudaError_t e = cudaLaunchKernelEx(&cfg, ts_norm_backward_kernel<TDY, Src, VEC, G, D, K>, a, W, part);
  if (e != cudaSuccess || !part) return e;
  return finish_columns(part, (int)grid, a.cols, a.dbeta, a.dgamma, a.accumulate, nullptr, st);
}

template <class TDY, class Src, bool VEC>
cudaError_t backward_wide(const ts_ops& h, const NormArgs& a, cudaStream_t st) {
  static std::atomic<uint64_t> ready{0};   // devices whose shared memory is opted in
  const uint64_t bit = h.device < 64 ? 1ull << h.device : 0;
  if (!bit || !(ready.load(std::memory_order_acquire) & bit)) {
    cudaError_t e = cudaFuncSetAttribute(ts_norm_backward_wide_kernel<TDY, Src, VEC>,
                                         cudaFuncAttributeMaxDynamicSharedMemorySize, kWideSmem);
    if (e != cudaSuccess) return e;
    ready.fetch_or(bit, std::memory_order_release);
  }
  int64_t grid = std::min<int64_t>(a.rows, h.nsm);
  grid = std::max<int64_t>(1, std::min(grid, (h.ws_bytes - 8 * (int64_t)a.cols) / (8 * (int64_t)a.cols)));
  float* part = a.dgamma || a.dbeta ? reinterpret_cast<float*>(h.ws) : nullptr;
  cudaLaunchConfig_t cfg = pdl_config((int)grid, 1024, kWideSmem, st);
  cudaLaunchAttribute at[1];
  pdl_attr(cfg, at);
  cudaError_t e = cudaLaunchKernelEx(&cfg, ts_norm_backward_wide_kernel<TDY, Src, VEC>, a, part);
  if (e != cudaSuccess || !part) return e;
  return finish_columns(part, (int)grid, a.cols, a.dbeta, a.dgamma, a.accumulate, nullptr, st);
}

template <class TDY, class Src, bool VEC>
cudaError_t backward_rows(const ts_ops& h, const NormArgs& a, cudaStream_t st) {
  // Up to 4096 columns the next pair of rows in flight; 8192 x 4096 bf16 took
  // 52 us by single rows.
  if (a.rows > 0 && a.cols <= 16 * kGroupCols) {
    int W = 1;
    while (W * kGroupCols < a.cols) W *= 2;
    return backward_fused<TDY, Src, VEC, 1, 1, 2>(h, a, W, st);
  }
  if (a.rows > 0 && a.cols <= 32 * kGroupCols) return backward_fused<TDY, Src, VEC, 2, 1, 1>(h, a, 16, st);
  if (a.rows > 0 && a.cols <= kWideGroups * 32 * kGroupCols) return backward_wide<TDY, Src, VEC>(h, a, st);
  // The sums first: dx may be dy.
  if (a.dgamma || a.dbeta) {
    cudaError_t e = columns<TDY, Src, VEC>(h, a, nullptr, st);
    if (e != cudaSuccess) return e;
  }
  if (a.rows == 0) return cudaSuccess;
  cudaLaunchConfig_t cfg = pdl_config((int)a.rows, 256, 0, st);
  cudaLaunchAttribute at[1];
  pdl_attr(cfg, at);
  return cudaLaunchKernelEx(&cfg, ts_norm_dx_kernel<TDY, Src, VEC>, a);
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
