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

// Sums over some logits about a reference m: s of e^(x - m), t of the same
// times (x - m) log2(e).  m = -inf: nothing but -inf logits so far (s = 0).
struct Softmax {
  float m, s, t;
};
constexpr float kLog2e = 1.44269504f, kLn2 = 0.693147181f;

__device__ __forceinline__ float max_nan(float a, float b) {
  float r;
  asm("max.NaN.f32 %0, %1, %2;" : "=f"(r) : "f"(a), "f"(b));
  return r;
}
__device__ __forceinline__ float ex2(float x) {
  float r;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(x));
  return r;
}
__device__ __forceinline__ uint64_t pack2f(float a, float b) {
  uint64_t r;
  asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "f"(a), "f"(b));
  return r;
}
__device__ __forceinline__ void unpack2f(uint64_t v, float& a, float& b) {
  asm("mov.b64 {%0, %1}, %2;" : "=f"(a), "=f"(b) : "l"(v));
}
__device__ __forceinline__ uint64_t fma2(uint64_t a, uint64_t b, uint64_t c) {
  uint64_t r;
  asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r) : "l"(a), "l"(b), "l"(c));
  return r;
}
__device__ __forceinline__ uint64_t mul2(uint64_t a, uint64_t b) {
  uint64_t r;
  asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
  return r;
}
__device__ __forceinline__ uint64_t add2(uint64_t a, uint64_t b) {
  uint64_t r;
  asm("add.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
  return r;
}

// Moves sums to the reference m.
__device__ __forceinline__ void move_reference(Softmax& a, float m) {
  if (a.m == -INFINITY) {
    a.m = m;
    return;
  }
  const float d = max_nan((a.m - m) * kLog2e, -200.f), f = ex2(d);
  a.t = (a.t + d * a.s) * f;
  a.s *= f;
  a.m = m;
}
__device__ __forceinline__ Softmax merge(Softmax a, Softmax b) {
  const float m = fmaxf(a.m, b.m);
  if (m == a.m && m == b.m) return Softmax{m, a.s + b.s, a.t + b.t};   // (both -inf: all sums are 0)
  if (a.m != m) move_reference(a, m);
  if (b.m != m) move_reference(b, m);
  return Softmax{m, a.s + b.s, a.t + b.t};
}

// Eight logits as they were loaded.
template <class T>
struct Chunk;
template <>
struct Chunk<float> {
  float4 a, b;
  __device__ __forceinline__ void load(const float* p) {
    a = __ldcs(reinterpret_cast<const float4*>(p));
    b = __ldcs(reinterpret_cast<const float4*>(p) + 1);
  }
  __device__ __forceinline__ void get(float (&v)[8]) const {
    v[0] = a.x; v[1] = a.y; v[2] = a.z; v[3] = a.w;
    v[4] = b.x; v[5] = b.y; v[6] = b.z; v[7] = b.w;
  }
  __device__ __forceinline__ float top() const {   // a NaN if there is one
    return max_nan(max_nan(max_nan(a.x, a.y), max_nan(a.z, a.w)), max_nan(max_nan(b.x, b.y), max_nan(b.z, b.w)));
  }
};
template <>
struct Chunk<__nv_bfloat16> {
  uint4 w;
  __device__ __forceinline__ void load(const __nv_bfloat16* p) { w = __ldcs(reinterpret_cast<const uint4*>(p)); }
  __device__ __forceinline__ void get(float (&v)[8]) const {
    const uint32_t u[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      v[2 * i] = __uint_as_float(u[i] << 16);
      v[2 * i + 1] = __uint_as_float(u[i] & 0xffff0000u);
    }
  }
  __device__ __forceinline__ static __nv_bfloat162 pair(uint32_t u) {
    return *reinterpret_cast<const __nv_bfloat162*>(&u);
  }
  __device__ __forceinline__ float top() const {
    const __nv_bfloat162 m = __hmax2_nan(__hmax2_nan(pair(w.x), pair(w.y)), __hmax2_nan(pair(w.z), pair(w.w)));
    return max_nan(__low2float(m), __high2float(m));
  }
};

constexpr int kLpThreads = 512, kLpWarps = kLpThreads / 32;
constexpr int kCandidates = 1024;
constexpr int kMaxTop = 32, kMaxCluster = 8;

struct LpShared {
  unsigned long long cand[kCandidates];
  unsigned long long top[kMaxTop];
  // what the cluster's CTAs leave with its first one
  unsigned long long tops[kMaxCluster * kMaxTop];
  Softmax part[kMaxCluster];
  Softmax warp[kLpWarps];
  uint32_t bound[kLpWarps];
  float ref[kLpWarps];
  int count;
};

__device__ __forceinline__ unsigned long long composite(float v, int c) {
  return (unsigned long long)order_key(v) << 32 | (0xffffffffu - (uint32_t)c);
}
__device__ __forceinline__ void offer(LpShared& sh, float v, int c, unsigned long long tau) {
  const unsigned long long k = composite(v, c);
  if (k >= tau) {
    const int i = atomicAdd(&sh.count, 1);
    if (i < kCandidates) sh.cand[i] = k;
  }
}

// The k largest of n composites, in order, into out (0 where there are fewer):
// a composite's place is the number of larger ones (all are distinct, but for
// the zeros that stand for none).
__device__ void select_top(const unsigned long long* in, int n, unsigned long long* out, int k) {
  for (int i = threadIdx.x; i < k; i += kLpThreads) out[i] = 0;
  __syncthreads();
  for (int i = threadIdx.x; i < n; i += kLpThreads) {
    const unsigned long long v = in[i];
    if (!v) continue;
    int place = 0;
    for (int j = 0; j < n; ++j) place += in[j] > v;
    if (place < k) out[place] = v;
  }
  __syncthreads();
}

// One row, or one of a cluster's equal segments of a row, a CTA.  One pass:
//
// Each thread first loads U chunks of eight logits.  Their maximum over the
// CTA is the reference of every thread's sums; a thread moves its own only
// when a chunk exceeds it by 2^5, which keeps the exponentials in range
// without a running maximum per logit.  From the same chunks comes a lower
// bound of the k-th largest logit: every warp takes the r-th largest of its
// lanes' maxima, and the q-th largest of these, q r >= k, has at least k
// logits at or above it.  Chunks below the bound, nearly all, cost one
// comparison; logits at or above it go to a list in shared memory, from which
// the k largest are picked at the end.  Should the list overflow (logits in
// rising order, or many equal ones), its own k-th largest is the next bound
// and the row is read again for the list alone; the bound rises every time.
template <class T, int U>
__global__ void __launch_bounds__(kLpThreads, 2) ts_logprob_kernel(const LogprobArgs a) {
  __shared__ LpShared sh;
  pdl_launch_dependents();
  pdl_wait();
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  uint32_t ncl;
  asm("mov.u32 %0, %%cluster_nctaid.x;" : "=r"(ncl));
  const uint32_t rank = ncl > 1 ? cluster_ctarank() : 0;
  if (ncl > 1) asm volatile("barrier.cluster.arrive.aligned;" ::: "memory");
  const int64_t row = blockIdx.x / ncl;
  const T* x = static_cast<const T*>(a.logits.p) + row * a.logits.ld;
  // this CTA's logits, [begin, end), as loose ones before a 16-byte boundary,
  // whole chunks from it on, and loose ones after them
  const int begin = (int)((int64_t)a.vocab * rank / ncl), end = (int)((int64_t)a.vocab * (rank + 1) / ncl);
  const int off = (int)(reinterpret_cast<uintptr_t>(x + begin) % 16 / sizeof(T));
  const int head = min(end - begin, off ? (int)(16 / sizeof(T)) - off : 0);
  const int first = begin + head, chunks = (end - first) / 8, tail = first + chunks * 8;
  const int loose = head + (end - tail);   // at most 14
  const int my_loose = (int)threadIdx.x < loose ? (int)threadIdx.x < head ? begin + (int)threadIdx.x
                                                                          : tail + (int)threadIdx.x - head
                                                : -1;
  float tok_logit = 0.f;
  int64_t tok = -1;
  if (threadIdx.x == 0 && rank == 0 && a.logprob) {
    tok = a.tokens[row];
    if (tok >= 0 && tok < a.vocab) tok_logit = to_f32(x[tok]);
  }
  if (threadIdx.x == 0) sh.count = 0;

  Chunk<T> c[U];
  float loose_v = -INFINITY, seed = -INFINITY;
  if (my_loose >= 0) loose_v = to_f32(x[my_loose]);
#pragma unroll
  for (int u = 0; u < U; ++u)
    if (threadIdx.x + u * kLpThreads < chunks) c[u].load(x + first + (threadIdx.x + u * kLpThreads) * 8);
  uint32_t lane_key = 0;   // 0: no logit
#pragma unroll
  for (int u = 0; u < U; ++u)
    if (threadIdx.x + u * kLpThreads < chunks) {
      const float m = c[u].top();
      seed = fmaxf(seed, m);
      lane_key = max(lane_key, order_key(m));
    }
  if (my_loose >= 0) {
    seed = fmaxf(seed, loose_v);
    lane_key = max(lane_key, order_key(loose_v));
  }
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) seed = fmaxf(seed, __shfl_xor_sync(0xffffffffu, seed, o));
  const int r = (2 * a.k + kLpWarps - 1) / kLpWarps;
  const int q = a.k ? (a.k + r - 1) / r : 0;
  uint32_t nth = 0;
  for (int i = 0; i < r; ++i) {
    nth = __reduce_max_sync(0xffffffffu, lane_key);
    if (lane == __ffs(__ballot_sync(0xffffffffu, lane_key == nth)) - 1) lane_key = 0;
  }
  if (lane == 0) {
    sh.ref[warp] = seed;
    sh.bound[warp] = nth;
  }
  __syncthreads();
  seed = lane < kLpWarps ? sh.ref[lane] : -INFINITY;
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) seed = fmaxf(seed, __shfl_xor_sync(0xffffffffu, seed, o));
  uint32_t key = lane < kLpWarps ? sh.bound[lane] : 0, bound = 0;
  for (int i = 0; i < q; ++i) {
    bound = __reduce_max_sync(0xffffffffu, key);
    if (lane == __ffs(__ballot_sync(0xffffffffu, key == bound)) - 1) key = 0;
  }
  // the bound as a float: a chunk whose largest logit is below it has no
  // candidate (a NaN compares as not below)
  unsigned long long tau = a.k ? (unsigned long long)bound << 32 : ~0ull;
  const float tau_f = !a.k      ? INFINITY
                      : !bound  ? -INFINITY
                                : __uint_as_float(bound & 0x80000000u ? bound & 0x7fffffffu : ~bound);
  const bool want = a.k > 0;

  Softmax acc{seed, 0.f, 0.f};
  uint64_t s2 = 0, t2 = 0;
  float minus_m = seed == -INFINITY ? 0.f : -seed;
  float limit = seed + 32.f;
  auto sums = [&](const float (&v)[8]) {
    const uint64_t l2 = pack2f(kLog2e, kLog2e), m2 = pack2f(minus_m, minus_m);
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      float d0, d1;
      // (the difference first: m log2(e) alone may overflow)
      unpack2f(mul2(add2(pack2f(v[2 * i], v[2 * i + 1]), m2), l2), d0, d1);
      d0 = max_nan(d0, -200.f);   // (-inf times the exponential's 0 would be NaN)
      d1 = max_nan(d1, -200.f);
      const uint64_t e2 = pack2f(ex2(d0), ex2(d1));
      s2 = add2(s2, e2);
      t2 = fma2(e2, pack2f(d0, d1), t2);
    }
  };
  auto raise = [&](float m) {
    float sa, sb, ta, tb;
    unpack2f(s2, sa, sb);
    unpack2f(t2, ta, tb);
    acc.s = sa + sb;
    acc.t = ta + tb;
    move_reference(acc, m);
    s2 = pack2f(acc.s, 0.f);
    t2 = pack2f(acc.t, 0.f);
    minus_m = -m;
    limit = m + 32.f;
  };
  auto take = [&](const Chunk<T>& ch, int i) {
    const float m = ch.top();
    float v[8];
    ch.get(v);
    if (m > limit) raise(m);
    sums(v);
    if (want && !(m < tau_f)) {
#pragma unroll
      for (int j = 0; j < 8; ++j) offer(sh, v[j], first + i * 8 + j, tau);
    }
  };
  if (my_loose >= 0) {
    float v[8] = {loose_v, -INFINITY, -INFINITY, -INFINITY, -INFINITY, -INFINITY, -INFINITY, -INFINITY};
    if (loose_v > limit) raise(loose_v);
    sums(v);
    if (want) offer(sh, loose_v, my_loose, tau);
  }
  for (int i0 = threadIdx.x; i0 < chunks; i0 += U * kLpThreads) {
    // the next chunks are in flight while these are worked on
    Chunk<T> n[U];
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const int i = i0 + (u + U) * kLpThreads;
      if (i < chunks) n[u].load(x + first + (int64_t)i * 8);
    }
#pragma unroll
    for (int u = 0; u < U; ++u)
      if (i0 + u * kLpThreads < chunks) take(c[u], i0 + u * kLpThreads);
#pragma unroll
    for (int u = 0; u < U; ++u) c[u] = n[u];
  }
  {
    float sa, sb, ta, tb;
    unpack2f(s2, sa, sb);
    unpack2f(t2, ta, tb);
    acc.s = sa + sb;
    acc.t = ta + tb;
  }
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) {
    const Softmax p{__shfl_xor_sync(0xffffffffu, acc.m, o), __shfl_xor_sync(0xffffffffu, acc.s, o),
                    __shfl_xor_sync(0xffffffffu, acc.t, o)};
    acc = merge(acc, p);
  }
  if (lane == 0) sh.warp[warp] = acc;
  __syncthreads();
  if (want) {
    int n = sh.count;
    while (n > kCandidates) {
      select_top(sh.cand, kCandidates, sh.top, a.k);
      tau = sh.top[a.k - 1];
      if (threadIdx.x == 0) sh.count = 0;
      __syncthreads();
      for (int i = threadIdx.x; i < chunks; i += kLpThreads) {
        float v[8];
        Chunk<T> ch;
        ch.load(x + first + (int64_t)i * 8);
        ch.get(v);
#pragma unroll
        for (int j = 0; j < 8; ++j) offer(sh, v[j], first + i * 8 + j, tau);
      }
      if (my_loose >= 0) offer(sh, loose_v, my_loose, tau);
      __syncthreads();
      n = sh.count;
    }
    select_top(sh.cand, n, sh.top, a.k);
  }
  if (warp == 0) {
    acc = sh.warp[0];
    for (int w = 1; w < kLpWarps; ++w) acc = merge(acc, sh.warp[w]);
  }
  const unsigned long long* top = sh.top;
  if (ncl > 1) {
    // the first CTA (which has started) gathers the segments' sums and lists
    asm volatile("barrier.cluster.wait.aligned;" ::: "memory");
    if (warp == 0) {
      const uint32_t dst = cluster_addr(smem_u32(&sh.part[rank]), 0);
      if (lane == 0)
        asm volatile("st.shared::cluster.f32 [%0], %1;\n st.shared::cluster.f32 [%0 + 4], %2;\n"
                     " st.shared::cluster.f32 [%0 + 8], %3;" ::"r"(dst),
                     "f"(acc.m), "f"(acc.s), "f"(acc.t)
                     : "memory");
      if (lane < a.k)
        asm volatile("st.shared::cluster.b64 [%0], %1;" ::"r"(
                         cluster_addr(smem_u32(&sh.tops[rank * a.k + lane]), 0)),
                     "l"(sh.top[lane])
                     : "memory");
    }
    cluster_sync();   // releases the stores, acquires them in the first CTA
    if (rank) return;
    if (warp == 0) {
      acc = sh.part[0];
      for (uint32_t w = 1; w < ncl; ++w) acc = merge(acc, sh.part[w]);
    }
    if (want) select_top(sh.tops, (int)ncl * a.k, sh.top, a.k);
  }
  if (warp == 0) {
    const bool none = acc.s == 0.f;
    const float ln = logf(acc.s), lse = none ? -INFINITY : acc.m + ln;
    if (lane == 0) {
      if (a.lse) a.lse[row] = lse;
      if (a.entropy) a.entropy[row] = none ? 0.f : ln - kLn2 * (acc.t / acc.s);
      if (a.logprob)
        a.logprob[row] = tok < 0 || tok >= a.vocab ? 0.f : none ? -INFINITY : tok_logit - lse;
    }
    if (lane < a.k) {
      const unsigned long long k = top[lane];
      const int id = (int)(0xffffffffu - (uint32_t)k);
      a.top_id[row * a.k + lane] = id;
      a.top_logprob[row * a.k + lane] = none ? -INFINITY : to_f32(x[id]) - lse;
    }
  }
}

// Segments a row: as many as keep about two CTAs on every SM, each of at
// least two chunks a thread.
template <class T, int U>
cudaError_t logprob_rows(const ts_ops& h, const LogprobArgs& a, cudaStream_t st) {
  int ncl = 1;
  while (ncl < kMaxCluster && a.rows * ncl * 2 <= 2 * (int64_t)h.nsm && a.vocab / (ncl * 2) >= kLpThreads * 8) ncl *= 2;
  cudaLaunchConfig_t cfg = pdl_config((int)(a.rows * ncl), kLpThreads, 0, st);
  cudaLaunchAttribute at[2];
  at[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  at[0].val.programmaticStreamSerializationAllowed = 1;
  at[1].id = cudaLaunchAttributeClusterDimension;
  at[1].val.clusterDim.x = ncl;
  at[1].val.clusterDim.y = at[1].val.clusterDim.z = 1;
  cfg.attrs = at;
  cfg.numAttrs = 2;
  return cudaLaunchKernelEx(&cfg, ts_logprob_kernel<T, U>, a);
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

cudaError_t launch_token_logprobs(const ts_ops& h, const LogprobArgs& a, cudaStream_t st) {
  return a.logits.bf16 ? logprob_rows<__nv_bfloat16, 4>(h, a, st) : logprob_rows<float, 2>(h, a, st);
}

cudaError_t launch_token_logprobs_backward(const ts_ops& h, const LogprobArgs& a, cudaStream_t st) {
  using B = __nv_bfloat16;
  if (a.logits.bf16) return a.dlogits.bf16 ? backward_types<B, B>(h, a, st) : backward_types<B, float>(h, a, st);
  return a.dlogits.bf16 ? backward_types<float, B>(h, a, st) : backward_types<float, float>(h, a, st);
}

}  // namespace fg
