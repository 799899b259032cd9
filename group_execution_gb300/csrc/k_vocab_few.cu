// The logits of at most 16 rows over a small vocabulary, for the cross entropy and
// its gradient (k_vocab_loss.cu has the formulas).
//
// For so small a product the latency of a launch and of a chain of loads is what
// counts.  So the weight's rows go from memory straight into the registers of
// mma.sync.m16n8k16, 16 bytes a lane, and nothing is staged: a warp takes 16 rows
// of w (two n8 tiles) against the 16 rows of x, whose pieces come from L1.  The k
// index of a fragment is permuted, the same way for both operands, so that a
// lane's eight consecutive elements serve two MMAs.  Where there are fewer tiles
// than warps, a tile's K is cut over the warps of a block, and their sums meet in
// shared memory.
//
// 1 x 1024 x 4000 takes 7 us in a graph, where tiles on the tensor cores' own
// memory take 11; a step of 16 x 1024 x 8000 or more is faster there.
//
// Forward, each block keeps a maximum and a sum of exponentials for every row;
// the block that finishes last joins all of them in block order, so that the
// whole pass is one launch.
#include <algorithm>

#include "launch.h"
#include "ts_device.cuh"
#include "vocab.cuh"

namespace fg {
namespace {

constexpr int kWarps = 8, kThreads = kWarps * 32;
constexpr int kTileV = 16;     // rows of w a warp takes at a time
constexpr int kBatch = 2;      // steps of 32 of K that are loaded while as many are multiplied
constexpr int kChainSteps = 32;   // of 32 of K that one accumulator sums (the tensor core truncates as it adds)

struct FewKernel {
  const __nv_bfloat16* x;
  const __nv_bfloat16* w;
  int64_t ldx, ldw;
  int rows, cols, vocab;
  int vec;         // all rows on 16 bytes, and whole pieces of 16 bytes
  int ksplit;      // warps that share a tile
  int tiles;
  const int64_t* targets;
  // forward
  float* tlogit;
  float2* part;    // [blocks][kFewRows]
  float* loss;
  float* lse;
  int32_t* arrived;
  // backward
  const float* lse_in;
  const float* g_loss;
  const float* g_lse;
  __nv_bfloat16* d;
  int64_t dpitch;
  CopyRows copy;
};

__device__ __forceinline__ void mma_bf16(float (&c)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0,
                                         uint32_t b1) {
  asm(
      "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, {%0, %1, %2, "
      "%3};"
      : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}
// (volatile: it stays behind the wait for the grid before)
__device__ __forceinline__ uint4 stream16(const __nv_bfloat16* p) {
  uint4 v;
  asm volatile("ld.global.nc.L1::no_allocate.v4.u32 {%0, %1, %2, %3}, [%4];"
               : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w)
               : "l"(p));
  return v;
}

// What other blocks have written in this launch.
__device__ __forceinline__ float2 load_shared(const float2* p) {
  float2 v;
  asm volatile("ld.relaxed.gpu.global.v2.f32 {%0, %1}, [%2];" : "=f"(v.x), "=f"(v.y) : "l"(p) : "memory");
  return v;
}
__device__ __forceinline__ float load_shared(const float* p) {
  float v;
  asm volatile("ld.relaxed.gpu.global.f32 %0, [%1];" : "=f"(v) : "l"(p) : "memory");
  return v;
}

template <bool BACK>
__global__ void __launch_bounds__(kThreads, 2) ts_few_kernel(const __grid_constant__ FewKernel P) {
  __shared__ float sums[kWarps][2][32][4];   // K's parts
  __shared__ float2 rows_sm[kWarps][kFewRows];
  __shared__ int last;
  pdl_launch_dependents();
  pdl_wait();
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, g = lane >> 2, q = lane & 3;
  if constexpr (BACK) copy_rows<2>(P.copy, (int64_t)blockIdx.x * kThreads + threadIdx.x, (int64_t)gridDim.x * kThreads);
  const int per_block = kWarps / P.ksplit, kp = warp % P.ksplit, group = warp / P.ksplit;
  const int steps = (P.cols + 31) / 32, s0 = steps * kp / P.ksplit, s1 = steps * (kp + 1) / P.ksplit;
  // this thread's rows: g and g + 8
  float m[2], sum[2], lse[2], coef[2], gl[2];
  int target[2];
#pragma unroll
  for (int r = 0; r < 2; ++r) {
    const int row = r * 8 + g;
    m[r] = -INFINITY;
    sum[r] = lse[r] = coef[r] = gl[r] = 0.f;
    target[r] = -1;
    if (row < P.rows && P.targets) {
      const int64_t i = P.targets[row];
      if (i >= 0 && i < P.vocab) target[r] = (int)i;
    }
    if constexpr (BACK) {
      if (row < P.rows) {
        // (a row of -inf logits takes no gradient)
        const float l = P.lse_in[row];
        const bool none = l == -INFINITY;
        lse[r] = none ? 0.f : l;
        gl[r] = target[r] >= 0 && !none ? P.g_loss[row] : 0.f;
        coef[r] = gl[r] + (P.g_lse && !none ? P.g_lse[row] : 0.f);
      }
    }
  }
  for (int tile0 = blockIdx.x * per_block; tile0 < P.tiles; tile0 += gridDim.x * per_block) {   // (uniform)
    const int tile = tile0 + group, v0 = tile * kTileV;
    float tot[2][4] = {};
    if (tile < P.tiles) {
      const __nv_bfloat16* wrow[2];
      const __nv_bfloat16* xrow[2];
      bool win[2], xin[2];
#pragma unroll
      for (int n = 0; n < 2; ++n) {
        win[n] = v0 + n * 8 + g < P.vocab;
        wrow[n] = P.w + (int64_t)(win[n] ? v0 + n * 8 + g : 0) * P.ldw;
      }
#pragma unroll
      for (int r = 0; r < 2; ++r) {
        const int row = r * 8 + g;
        xin[r] = row < P.rows;
        xrow[r] = P.x + (int64_t)(xin[r] ? row : 0) * P.ldx;
      }
      struct Batch {
        uint4 w[kBatch][2];
      };
      auto load = [&](Batch& o, int st) {
#pragma unroll
        for (int u = 0; u < kBatch; ++u)
#pragma unroll
          for (int n = 0; n < 2; ++n) {
            const int j = (st + u) * 32 + q * 8;
            o.w[u][n] = make_uint4(0, 0, 0, 0);
            if (win[n] && st + u < s1 && j < P.cols)
              o.w[u][n] = P.vec ? stream16(wrow[n] + j) : row_piece(wrow[n], j, P.cols);
          }
      };
      float acc[2][4] = {};
      auto use = [&](const Batch& o, int st) {
#pragma unroll
        for (int u = 0; u < kBatch; ++u) {
          const int j = (st + u) * 32 + q * 8;
          uint4 xv[2];
#pragma unroll
          for (int r = 0; r < 2; ++r) {
            xv[r] = make_uint4(0, 0, 0, 0);
            if (xin[r] && st + u < s1 && j < P.cols)
              xv[r] = P.vec ? *reinterpret_cast<const uint4*>(xrow[r] + j) : row_piece(xrow[r], j, P.cols);
          }
#pragma unroll
          for (int n = 0; n < 2; ++n) {
            mma_bf16(acc[n], xv[0].x, xv[1].x, xv[0].y, xv[1].y, o.w[u][n].x, o.w[u][n].y);
            mma_bf16(acc[n], xv[0].z, xv[1].z, xv[0].w, xv[1].w, o.w[u][n].z, o.w[u][n].w);
          }
        }
      };
      auto flush = [&]() {
#pragma unroll
        for (int n = 0; n < 2; ++n)
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            tot[n][i] += acc[n][i];
            acc[n][i] = 0.f;
          }
      };
      Batch b0, b1;
      load(b0, s0);
      int chain = 0;
      for (int st = s0; st < s1; st += 2 * kBatch) {
        load(b1, st + kBatch);
        use(b0, st);
        load(b0, st + 2 * kBatch);
        use(b1, st + kBatch);
        if ((chain += 2 * kBatch) >= kChainSteps) {
          flush();
          chain = 0;
        }
      }
      flush();
    }
    if (P.ksplit > 1) {
      if (kp) {
#pragma unroll
        for (int n = 0; n < 2; ++n)
#pragma unroll
          for (int i = 0; i < 4; ++i) sums[warp][n][lane][i] = tot[n][i];
      }
      __syncthreads();
      if (kp == 0) {
        for (int k = 1; k < P.ksplit; ++k)
#pragma unroll
          for (int n = 0; n < 2; ++n)
#pragma unroll
            for (int i = 0; i < 4; ++i) tot[n][i] += sums[warp + k][n][lane][i];
      }
      __syncthreads();
    }
    if (kp || tile >= P.tiles) continue;
    // a thread holds columns v0 + n * 8 + 2 q, + 1 of its rows
#pragma unroll
    for (int r = 0; r < 2; ++r) {
      const int row = r * 8 + g;
      float l[4] = {tot[0][2 * r], tot[0][2 * r + 1], tot[1][2 * r], tot[1][2 * r + 1]};
      if constexpr (BACK) {
        const bool none = coef[r] == 0.f && gl[r] == 0.f;
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const int v = v0 + (i >> 1) * 8 + 2 * q + (i & 1);
          l[i] = coef[r] * exp2_approx((l[i] - lse[r]) * kLog2e);
          if (v == target[r]) l[i] -= gl[r];
          if (none || v >= P.vocab) l[i] = 0.f;
        }
        if (row < P.rows) {
          __nv_bfloat16* d = P.d + row * P.dpitch + v0 + 2 * q;
          *reinterpret_cast<uint32_t*>(d) = bf16x2(l[0], l[1]);
          *reinterpret_cast<uint32_t*>(d + 8) = bf16x2(l[2], l[3]);
        }
      } else {
        float top = -INFINITY;
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const int v = v0 + (i >> 1) * 8 + 2 * q + (i & 1);
          if (v >= P.vocab) l[i] = -INFINITY;
          else if (v == target[r]) P.tlogit[row] = l[i];
          top = fmaxf(top, l[i]);
        }
        const float next = fmaxf(m[r], top), ref = next == -INFINITY ? 0.f : next;
        float s = 0.f;
#pragma unroll
        for (int i = 0; i < 4; ++i) s += exp2_approx((l[i] - ref) * kLog2e);
        sum[r] = sum[r] * exp2_approx((m[r] - ref) * kLog2e) + s;
        m[r] = next;
      }
    }
  }
  if constexpr (!BACK) {
#pragma unroll
    for (int r = 0; r < 2; ++r) {
#pragma unroll
      for (int o = 1; o < 4; o <<= 1) {
        const float om = __shfl_xor_sync(0xffffffffu, m[r], o), os = __shfl_xor_sync(0xffffffffu, sum[r], o);
        join_sums(m[r], sum[r], om, os);
      }
      if (q == 0) rows_sm[warp][r * 8 + g] = make_float2(m[r], sum[r]);
    }
    __syncthreads();
    if ((int)threadIdx.x < P.rows) {
      float bm = -INFINITY, bs = 0.f;
      for (int w = 0; w < kWarps; ++w) join_sums(bm, bs, rows_sm[w][threadIdx.x].x, rows_sm[w][threadIdx.x].y);
      P.part[blockIdx.x * kFewRows + threadIdx.x] = make_float2(bm, bs);
    }
    __threadfence();
    __syncthreads();
    if (threadIdx.x == 0) last = atom_add_acq_rel_gpu(P.arrived, 1) + 1 == (int)gridDim.x;
    __syncthreads();
    if (!last) return;
    __threadfence();
    for (int row = warp; row < P.rows; row += kWarps) {
      // a lane's blocks in order, then the lanes'
      float bm = -INFINITY, bs = 0.f;
      for (int b0 = lane; b0 < (int)gridDim.x; b0 += 8 * 32) {
        float2 v[8];
#pragma unroll
        for (int k = 0; k < 8; ++k) {
          v[k] = make_float2(-INFINITY, 0.f);
          if (b0 + k * 32 < (int)gridDim.x) v[k] = load_shared(P.part + (b0 + k * 32) * kFewRows + row);
        }
#pragma unroll
        for (int k = 0; k < 8; ++k) join_sums(bm, bs, v[k].x, v[k].y);
      }
#pragma unroll
      for (int o = 16; o > 0; o >>= 1) {
        const float om = __shfl_xor_sync(0xffffffffu, bm, o), os = __shfl_xor_sync(0xffffffffu, bs, o);
        join_sums(bm, bs, om, os);
      }
      if (lane == 0) {
        if (P.lse) P.lse[row] = lse_of(bm, bs);
        if (P.loss) {
          const int64_t t = P.targets[row];
          P.loss[row] = t < 0 || t >= P.vocab ? 0.f : loss_of(bm, bs, load_shared(P.tlogit + row));
        }
      }
    }
    if (threadIdx.x == 0) *P.arrived = 0;   // for the next call
  }
}

int most_blocks(int nsm) { return 2 * nsm; }

FewKernel few_kernel(const ts_ops& h, const VocabLossArgs& a, int& grid) {
  FewKernel P = {};
  P.x = static_cast<const __nv_bfloat16*>(a.x.p);
  P.w = static_cast<const __nv_bfloat16*>(a.w.p);
  P.ldx = a.x.ld;
  P.ldw = a.w.ld;
  P.rows = (int)a.rows;
  P.cols = a.cols;
  P.vocab = (int)a.vocab;
  P.vec = rows_aligned(a.x) && rows_aligned(a.w) && a.cols % 8 == 0;
  P.tiles = (P.vocab + kTileV - 1) / kTileV;
  // as many warps to a tile as leave every warp one, none with less than four
  // steps of K
  const int most = most_blocks(h.nsm), steps = (a.cols + 31) / 32;
  P.ksplit = 1;
  while (P.ksplit < kWarps && (int64_t)P.tiles * P.ksplit * 2 <= (int64_t)most * kWarps && steps >= P.ksplit * 8)
    P.ksplit *= 2;
  const int per_block = kWarps / P.ksplit;
  grid = std::min(most, (P.tiles + per_block - 1) / per_block);
  return P;
}

}  // namespace

cudaError_t launch_few_loss(const ts_ops& h, const VocabLossArgs& a, cudaStream_t st) {
  int grid = 0;
  FewKernel P = few_kernel(h, a, grid);
  P.targets = a.loss ? a.targets : nullptr;
  P.loss = a.loss;
  P.lse = a.lse;
  P.tlogit = reinterpret_cast<float*>(h.ws);
  P.part = reinterpret_cast<float2*>(h.ws + 256);
  P.arrived = h.err + 16;   // (zero between calls)
  cudaLaunchConfig_t cfg = pdl_config(grid, kThreads, 0, st);
  cudaLaunchAttribute at[1];
  pdl_attr(cfg, at);
  return cudaLaunchKernelEx(&cfg, ts_few_kernel<false>, P);
}

cudaError_t launch_few_dlogits(const ts_ops& h, const VocabLossArgs& a, const CopyRows& C, __nv_bfloat16* d,
                               int64_t dpitch, cudaStream_t st) {
  int grid = 0;
  FewKernel P = few_kernel(h, a, grid);
  P.targets = a.targets;
  P.lse_in = a.lse;
  P.g_loss = a.g_loss;
  P.g_lse = a.g_lse;
  P.d = d;
  P.dpitch = dpitch;
  P.copy = C;
  cudaLaunchConfig_t cfg = pdl_config(grid, kThreads, 0, st);
  cudaLaunchAttribute at[1];
  pdl_attr(cfg, at);
  return cudaLaunchKernelEx(&cfg, ts_few_kernel<true>, P);
}

}  // namespace fg
