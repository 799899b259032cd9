// A matmul's weight gradient from its 8-bit saved input: dW = X^T dY over the
// rows (tokens).  With an affine input X = gamma h + beta by column, h the
// checkpoint,
//   dW_cj = gamma_c sum_t h_tc dY_tj + beta_c db_j,   db_j = sum_t dY_tj.
#include <algorithm>

#include "launch.h"
#include "ts_device.cuh"

namespace fg {
namespace {

// The simplest form: a 32 x 32 tile of dW a block, 32 tokens at a time
// through shared memory.
__global__ void __launch_bounds__(256) ts_wgrad_kernel(const WgradArgs a, const float* colsum) {
  __shared__ float xs[32][33], ys[32][33];
  pdl_launch_dependents();
  pdl_wait();
  const int tx = threadIdx.x & 31, ty = threadIdx.x >> 5;
  const int c0 = blockIdx.x * 32, j0 = blockIdx.y * 32;
  float acc[4] = {};
  for (int64_t t0 = 0; t0 < a.rows; t0 += 32) {
    for (int i = ty; i < 32; i += 8) {
      const int64_t t = t0 + i;
      const int c = c0 + tx, j = j0 + tx;
      xs[i][tx] = t < a.rows && c < a.cols
                      ? (float)a.x.q[t * a.x.pitch + c] * ckpt_step(a.x.scale[(t * a.x.pitch + c) / kCkptBlock])
                      : 0.f;
      ys[i][tx] = t < a.rows && j < a.n
                      ? __bfloat162float(static_cast<const __nv_bfloat16*>(a.dy.p)[t * a.dy.ld + j])
                      : 0.f;
    }
    __syncthreads();
#pragma unroll
    for (int k = 0; k < 4; ++k)
      for (int i = 0; i < 32; ++i) acc[k] += xs[i][ty + 8 * k] * ys[i][tx];
    __syncthreads();
  }
  const int j = j0 + tx;
#pragma unroll
  for (int k = 0; k < 4; ++k) {
    const int c = c0 + ty + 8 * k;
    if (c < a.cols && j < a.n) {
      float v = acc[k];
      if (a.gamma) v *= a.gamma[c];
      if (a.beta) v += a.beta[c] * colsum[j];
      float* d = a.dw + (int64_t)c * a.lddw + j;
      *d = a.accumulate ? *d + v : v;
    }
  }
}

}  // namespace

cudaError_t launch_weight_grad(const ts_ops& h, const WgradArgs& a, cudaStream_t st) {
  // dy's column sums: this call's own at the workspace's end, for beta
  float* colsum = a.beta ? reinterpret_cast<float*>(h.ws + h.ws_bytes) - (a.n + 3) / 4 * 4 : nullptr;
  if (colsum || a.db) {
    cudaError_t e = launch_column_sums(h, a.dy, a.rows, a.n, colsum, a.db, a.accumulate, st);
    if (e != cudaSuccess) return e;
  }
  cudaLaunchConfig_t cfg = pdl_config(1, 256, 0, st);
  cfg.gridDim = dim3((a.cols + 31) / 32, (a.n + 31) / 32);
  cudaLaunchAttribute at[1];
  pdl_attr(cfg, at);
  return cudaLaunchKernelEx(&cfg, ts_wgrad_kernel, a, (const float*)colsum);
}

}  // namespace fg
