// Log probabilities of given tokens under rows of logits, with the entropy
// and the k most likely alternatives, and their gradient.  With L = log sum
// exp(x):
//   logprob = x_tok - L,  H = log sum e - sum e (x - max) / sum e,
// and for output gradients g (logprob) and w (entropy)
//   dx_v = g (1[v = tok] - p_v) - w p_v (log p_v + H).
// A row whose every logit is -inf has no distribution: L and the log
// probabilities are -inf, the entropy and the gradient 0.  A row that holds a
// NaN or +inf gives NaN.
#include <algorithm>

#include "launch.h"
#include "ts_device.cuh"

namespace fg {
namespace {

// Logits in an order for unsigned comparison: larger value, larger key; -0
// and +0 alike; a NaN above everything.
__device__ __forceinline__ uint32_t order_key(float x) {
  const uint32_t u = __float_as_uint(x + 0.f);
  if (x != x) return 0xfffffffeu;   // (all ones stays free: "no bound yet")
  return u & 0x80000000u ? ~u : u | 0x80000000u;
}

// Running maximum m, sum s of e^(x - m) and sum t of (x - m) e^(x - m).
struct Softmax {
  float m, s, t;
};
__device__ __forceinline__ Softmax merge(const Softmax& a, const Softmax& b) {
  Softmax r;
  r.m = fmaxf(a.m, b.m);
  const float da = a.m == r.m ? 0.f : fmaxf(a.m - r.m, -200.f), db = b.m == r.m ? 0.f : fmaxf(b.m - r.m, -200.f);
  const float ea = expf(da), eb = expf(db);
  r.s = a.s * ea + b.s * eb;
  r.t = (a.t + da * a.s) * ea + (b.t + db * b.s) * eb;
  return r;
}

template <class T>
__global__ void __launch_bounds__(256) ts_logprob_kernel(const LogprobArgs a) {
  __shared__ Softmax sm[8];
  __shared__ unsigned long long best[8];
  pdl_launch_dependents();
  pdl_wait();
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int64_t row = blockIdx.x;
  const T* x = static_cast<const T*>(a.logits.p) + row * a.logits.ld;
  float m = -INFINITY;
  for (int64_t c = threadIdx.x; c < a.vocab; c += 256) m = fmaxf(m, to_f32(x[c]));
  const float base = m == -INFINITY ? 0.f : m;
  Softmax r{m, 0.f, 0.f};
  for (int64_t c = threadIdx.x; c < a.vocab; c += 256) {
    const float d = to_f32(x[c]) - base, e = expf(d);
    r.s += e;
    r.t += e * fmaxf(d, -200.f);
  }
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) {
    const Softmax p{__shfl_xor_sync(0xffffffffu, r.m, o), __shfl_xor_sync(0xffffffffu, r.s, o),
                    __shfl_xor_sync(0xffffffffu, r.t, o)};
    r = lane & o ? merge(p, r) : merge(r, p);
  }
  if (lane == 0) sm[warp] = r;
  __syncthreads();
  r = sm[0];
  for (int w = 1; w < 8; ++w) r = merge(r, sm[w]);
  const bool none = r.m == -INFINITY && r.s == 0.f;
  const float lse = none ? -INFINITY : r.m + logf(r.s);
  if (threadIdx.x == 0) {
    if (a.lse) a.lse[row] = lse;
    if (a.entropy) a.entropy[row] = none ? 0.f : logf(r.s) - r.t / r.s;
    if (a.logprob) {
      const int64_t tok = a.tokens[row];
      a.logprob[row] = tok < 0 || tok >= a.vocab ? 0.f : none ? -INFINITY : to_f32(x[tok]) - lse;
    }
  }
  unsigned long long last = ~0ull;
  for (int k = 0; k < a.k; ++k) {
    unsigned long long b = 0;
    for (int64_t c = threadIdx.x; c < a.vocab; c += 256) {
      const unsigned long long v = (unsigned long long)order_key(to_f32(x[c])) << 32 | (0xffffffffu - (uint32_t)c);
      if (v < last && v > b) b = v;
    }
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) b = max(b, __shfl_xor_sync(0xffffffffu, b, o));
    __syncthreads();
    if (lane == 0) best[warp] = b;
    __syncthreads();
    for (int w = 0; w < 8; ++w) b = max(b, best[w]);
    last = b;
    if (threadIdx.x == 0) {
      const int id = (int)(0xffffffffu - (uint32_t)b);
      a.top_id[row * a.k + k] = id;
      a.top_logprob[row * a.k + k] = none ? -INFINITY : to_f32(x[id]) - lse;
    }
  }
}

template <class TX, class TD, bool VEC>
__global__ void __launch_bounds__(256) ts_logprob_backward_kernel(const LogprobArgs a) {
  pdl_launch_dependents();
  pdl_wait();
  const int lane = threadIdx.x & 31;
  const int per_row = (a.vocab + kGroupCols - 1) / kGroupCols;
  const int64_t total = a.rows * per_row, step = (int64_t)gridDim.x * 8;
  for (int64_t i = (int64_t)blockIdx.x * 8 + (threadIdx.x >> 5); i < total; i += step) {
    const int64_t row = i / per_row;
    const int c0 = (int)(i - row * per_row) * kGroupCols;
    const TX* x = static_cast<const TX*>(a.logits.p) + row * a.logits.ld;
    TD* d = static_cast<TD*>(a.dlogits.p) + row * a.dlogits.ld;
    const float lse = a.lse[row];
    const int64_t tok = a.tokens[row];
    const bool scored = tok >= 0 && tok < a.vocab;
    const float g = scored ? a.g_logprob[row] : 0.f;
    const float w = a.g_entropy ? a.g_entropy[row] : 0.f, h = a.g_entropy ? a.entropy[row] : 0.f;
    float v[8];
    load_group<VEC>(x, c0, a.vocab, lane, v);
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      const float lp = v[j] - lse;
      const float p = lse == -INFINITY ? 0.f : expf(lp);
      float o = scored ? -g * p : 0.f;
      if (w != 0.f) o -= w * p * (fmaxf(lp, -200.f) + h);
      if (c0 + group_col<VEC>(lane, j) == tok && lse != -INFINITY) o += g;
      v[j] = o;
    }
    store_group<VEC>(d, c0, a.vocab, lane, v);
  }
}

template <class TX, class TD>
cudaError_t backward_types(const ts_ops& h, const LogprobArgs& a, cudaStream_t st) {
  const int64_t groups = a.rows * ((a.vocab + kGroupCols - 1) / kGroupCols);
  cudaLaunchConfig_t cfg = pdl_config((int)std::min<int64_t>((groups + 7) / 8, (int64_t)h.nsm * 8), 256, 0, st);
  cudaLaunchAttribute at[1];
  pdl_attr(cfg, at);
  return rows_aligned(a.logits) && rows_aligned(a.dlogits)
             ? cudaLaunchKernelEx(&cfg, ts_logprob_backward_kernel<TX, TD, true>, a)
             : cudaLaunchKernelEx(&cfg, ts_logprob_backward_kernel<TX, TD, false>, a);
}

}  // namespace

cudaError_t launch_token_logprobs(const ts_ops&, const LogprobArgs& a, cudaStream_t st) {
  cudaLaunchConfig_t cfg = pdl_config((int)a.rows, 256, 0, st);
  cudaLaunchAttribute at[1];
  pdl_attr(cfg, at);
  return a.logits.bf16 ? cudaLaunchKernelEx(&cfg, ts_logprob_kernel<__nv_bfloat16>, a)
                       : cudaLaunchKernelEx(&cfg, ts_logprob_kernel<float>, a);
}

cudaError_t launch_token_logprobs_backward(const ts_ops& h, const LogprobArgs& a, cudaStream_t st) {
  using B = __nv_bfloat16;
  if (a.logits.bf16) return a.dlogits.bf16 ? backward_types<B, B>(h, a, st) : backward_types<B, float>(h, a, st);
  return a.dlogits.bf16 ? backward_types<float, B>(h, a, st) : backward_types<float, float>(h, a, st);
}

}  // namespace fg
