// Log probabilities of given tokens under rows of logits, with the entropy
// and the k most likely alternatives, and their gradient.  With L = log sum
// exp(x):
//   logprob = x_tok - L,  H = log s - sum e^(x - m) (x - m) / s,  s = sum e^(x - m),
// for any reference m, here one at most kLag below the row's largest logit: the
// two terms of H cancel the further, the further m is below it.  For output gradients g (logprob) and w (entropy)
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
// How far a logit may lie above the reference of its sums.  The entropy is then
// off by the roundings of numbers of that size (with 32, which float32's range
// allows, confident rows were 1e-5 off and their entropy negative).  With 0
// each larger logit of a rising row moves the sums, and each move costs an
// exponential's error.  4096 x 50001 bf16 without alternatives takes 73.6 us
// with 32, 73.9 with 2, 74.2 with 1, 74.6 with 0.
constexpr float kLag = 1.f;

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

constexpr int kCandidates = 1024;
constexpr int kMaxTop = 32, kMaxCluster = 8;

// W warps share a row.
template <int W>
struct LpShared {
  unsigned long long cand[W == 1 ? 288 : kCandidates];
  unsigned long long top[kMaxTop];
  // lists of the row's warps, and what the cluster's CTAs leave with its
  // first one
  unsigned long long lists[W == 1 ? 1 : W * 32];
  unsigned long long tops[W == 1 ? 1 : kMaxCluster * kMaxTop];
  Softmax part[kMaxCluster];
  Softmax warp[W];
  uint32_t bound[W];
  uint32_t ref[W];
  int count;
};
template <int W>
__device__ __forceinline__ void row_sync() {
  if (W == 1)
    __syncwarp();
  else
    __syncthreads();
}

// A logit, or a chunk by its largest, with its (first) column: larger logits
// first, then lower columns.  Never 0.
__device__ __forceinline__ unsigned long long composite(float v, int c) {
  return (unsigned long long)order_key(v) << 32 | (0xffffffffu - (uint32_t)c);
}
__device__ __forceinline__ int composite_col(unsigned long long k) { return (int)(0xffffffffu - (uint32_t)k); }

// The larger (keep_max) or smaller of this lane's entry and lane ^ o's.
__device__ __forceinline__ unsigned long long exchange(unsigned long long v, int o, bool keep_max) {
  const unsigned long long w = __shfl_xor_sync(0xffffffffu, v, o);
  return (w > v) == keep_max ? w : v;
}
// 32 entries in falling order across the lanes (a bitonic network).
__device__ __forceinline__ unsigned long long sort32(unsigned long long v, int lane) {
#pragma unroll
  for (int k = 2; k <= 32; k *= 2)
#pragma unroll
    for (int o = k / 2; o > 0; o /= 2) v = exchange(v, o, ((lane & o) == 0) == ((lane & k) == 0 || k == 32));
  return v;
}
// The 32 largest, in falling order, of two lists in falling order.
__device__ __forceinline__ unsigned long long merge32(unsigned long long a, unsigned long long b, int lane) {
  const unsigned long long r = __shfl_sync(0xffffffffu, b, 31 - lane);
  a = max(a, r);
#pragma unroll
  for (int o = 16; o > 0; o /= 2) a = exchange(a, o, (lane & o) == 0);
  return a;
}
// The 32 largest of n composites in falling order, one to a lane of every
// warp that calls (0 where there are fewer): warp w of W sorts every W-th
// batch of 32, then the warps' lists are merged pairwise through `lists`.
// All W warps call it; the result is warp 0's.
template <int W>
__device__ __forceinline__ unsigned long long largest32(const unsigned long long* in, int n, unsigned long long* lists,
                                                        int warp, int lane) {
  unsigned long long v = 0;
  for (int i = warp * 32; i < n; i += W * 32) {
    const unsigned long long s = sort32(i + lane < n ? in[i + lane] : 0, lane);
    v = i == warp * 32 ? s : merge32(v, s, lane);
  }
  int lists_left = min(W, (n + 31) / 32);
  while (lists_left > 1) {
    const int half = (lists_left + 1) / 2;
    if (warp >= half && warp < lists_left) lists[warp * 32 + lane] = v;
    __syncthreads();
    if (warp + half < lists_left) v = merge32(v, lists[(warp + half) * 32 + lane], lane);
    lists_left = half;
  }
  return v;
}

// Notes k in the row's list if it is at or above tau.  The i-th note takes any of
// i + 1 places, of which the list has the first: a full one holds a sample of
// all notes, evenly spread over them.  (Stores to one place may meet; either
// note will do.)
template <int W>
__device__ __forceinline__ void note_sample(LpShared<W>& sh, unsigned long long k, unsigned long long tau) {
  constexpr uint32_t kRoom = sizeof(sh.cand) / 8;
  if (k < tau) return;
  uint32_t i = atomicAdd(&sh.count, 1);
  if (i >= kRoom) i = __umulhi(i * 2654435769u, i + 1);
  if (i < kRoom) *static_cast<volatile unsigned long long*>(&sh.cand[i]) = k;
}

// One row, or one of a cluster's equal segments of a row, to W warps.  One
// pass:
//
// Each thread first loads U chunks of eight logits.  Their maximum over the
// row's threads is the reference of every thread's sums; a thread moves its
// own when a chunk exceeds it by kLag (few do, after the first ones), so
// there is no running maximum per logit.  From the same chunks comes a
// lower bound of the k-th largest logit: every warp takes the r-th largest of
// its lanes' maxima, and the q-th largest of these, q r >= k, has at least k
// logits at or above it.  A chunk below the bound costs one comparison; one
// at or above it is noted in shared memory by its maximum and column.  The k
// largest logits lie in the k chunks with the largest maxima (ties by
// column), so at the end those are picked from the list, read again (L2) and
// their logits picked from.  Should the list overflow (logits in rising
// order), its own k-th largest is the next bound and the row is read again
// for the list alone; should it overflow again, it then holds a sample of all
// notes, whose k-th largest leaves about k / 1024 of them, whatever their order.
// Rising rows are thus read twice more up to 2^15 chunks (700 x 131072 f32 takes
// 170 us, random logits 70 to 125), three times up to 2^20.
//
// 4096 x 50001 bf16 (rows at odd elements) takes 106 us with k = 20, 92 with
// k = 8 and 74 with k = 0, where the logits' bytes at the copy rate take 60;
// 2048 x 65536 f32 with k = 20 takes 95 of 79.  Instruction issue bounds the
// bf16 rows: 87 instructions to a warp's 32 chunks, 17.0 thousand a row with k =
// 0 (77 % of the issue slots), 25.5 thousand with k = 20 (81 %), by the noting
// and by a row's end, where the bound, two selections and the second reading
// are chains of latency too.  Other forms of that end, at k = 20: k passes over
// the row 3407 us, a selection by counting 210, a block's ninth warp that
// finishes rows for the others 126, one selection from the logits at or above a
// bound of the whole row 110, the chunks' maxima in shared memory in place of
// the list 97, but the short rows 12 % slower.
template <class T, int U, int W, int BLOCKS>
__global__ void __launch_bounds__(W == 1 ? 128 : W * 32, BLOCKS) ts_logprob_kernel(const LogprobArgs a) {
  constexpr int kRows = W == 1 ? 4 : 1, kN = W * 32;   // rows a block, threads a row
  __shared__ LpShared<W> shared[kRows];
  pdl_launch_dependents();
  pdl_wait();
  const int lane = threadIdx.x & 31, warp = W == 1 ? 0 : threadIdx.x >> 5, tid = W == 1 ? lane : threadIdx.x;
  LpShared<W>& sh = shared[W == 1 ? threadIdx.x >> 5 : 0];
  uint32_t ncl = 1, rank = 0;
  if (W > 1) {
    asm("mov.u32 %0, %%cluster_nctaid.x;" : "=r"(ncl));
    if (ncl > 1) {
      rank = cluster_ctarank();
      asm volatile("barrier.cluster.arrive.aligned;" ::: "memory");
    }
  }
  const int64_t row = W == 1 ? (int64_t)blockIdx.x * kRows + (threadIdx.x >> 5) : blockIdx.x / ncl;
  if (row >= a.rows) return;   // (a whole warp of the last block, W = 1)
  const T* x = static_cast<const T*>(a.logits.p) + row * a.logits.ld;
  // these threads' logits, [begin, end), as loose ones before a 16-byte
  // boundary, whole chunks from it on, and loose ones after them
  const int begin = (int)((int64_t)a.vocab * rank / ncl), end = (int)((int64_t)a.vocab * (rank + 1) / ncl);
  const int off = (int)(reinterpret_cast<uintptr_t>(x + begin) % 16 / sizeof(T));
  const int head = min(end - begin, off ? (int)(16 / sizeof(T)) - off : 0);
  const int first = begin + head, chunks = (end - first) / 8, tail = first + chunks * 8;
  const int my_loose = tid < head ? begin + tid : tail + tid - head < end ? tail + tid - head : -1;   // at most 14
  const T* body = x + first + tid * 8;   // this thread's first chunk; the next are kN chunks apart
  float tok_logit = 0.f;
  int64_t tok = -1;
  if (tid == 0 && rank == 0 && a.logprob) {
    tok = a.tokens[row];
    if (tok >= 0 && tok < a.vocab) tok_logit = to_f32(x[tok]);
  }
  if (tid == 0) sh.count = 0;

  Chunk<T> c[U];
  float loose_v = -INFINITY, seed = -INFINITY;
  if (my_loose >= 0) loose_v = to_f32(x[my_loose]);
#pragma unroll
  for (int u = 0; u < U; ++u)
    if (tid + u * kN < chunks) c[u].load(body + u * kN * 8);
  uint32_t lane_key = 0;   // 0: no logit
#pragma unroll
  for (int u = 0; u < U; ++u)
    if (tid + u * kN < chunks) {
      const float m = c[u].top();
      seed = fmaxf(seed, m);
      lane_key = max(lane_key, order_key(m));
    }
  if (my_loose >= 0) {
    seed = fmaxf(seed, loose_v);
    lane_key = max(lane_key, order_key(loose_v));
  }
  const uint32_t seed_key = __reduce_max_sync(0xffffffffu, order_key(seed));   // (fmaxf passed over any NaN)
  const int r = W == 1 ? a.k : (2 * a.k + W - 1) / W;
  const int q = W == 1 ? 0 : a.k ? (a.k + r - 1) / r : 0;
  uint32_t bound = 0, ref_key = seed_key;
  for (int i = 0; i < r; ++i) {
    bound = __reduce_max_sync(0xffffffffu, lane_key);
    if (lane == __ffs(__ballot_sync(0xffffffffu, lane_key == bound)) - 1) lane_key = 0;
  }
  if (W > 1) {
    if (lane == 0) {
      sh.ref[warp] = seed_key;
      sh.bound[warp] = bound;
    }
    __syncthreads();
    ref_key = __reduce_max_sync(0xffffffffu, lane < W ? sh.ref[lane] : 0u);
    uint32_t key = lane < W ? sh.bound[lane] : 0;
    bound = 0;
    for (int i = 0; i < q; ++i) {
      bound = __reduce_max_sync(0xffffffffu, key);
      if (lane == __ffs(__ballot_sync(0xffffffffu, key == bound)) - 1) key = 0;
    }
  } else {
    __syncwarp();
  }
  auto key_value = [](uint32_t k) { return __uint_as_float(k & 0x80000000u ? k & 0x7fffffffu : ~k); };
  seed = key_value(ref_key);
  // a chunk whose largest logit is below the bound has no candidate (a NaN
  // compares as not below)
  const bool want = a.k > 0;
  unsigned long long tau = (unsigned long long)bound << 32;
  const float tau_f = !want ? INFINITY : !bound ? -INFINITY : key_value(bound);

  Softmax acc{seed, 0.f, 0.f};
  uint64_t s2 = 0, t2 = 0;
  float minus_m = seed == -INFINITY ? 0.f : -seed;
  float limit = seed + kLag;
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
  auto settle = [&]() {
    float sa, sb, ta, tb;
    unpack2f(s2, sa, sb);
    unpack2f(t2, ta, tb);
    acc.s = sa + sb;
    acc.t = ta + tb;
  };
  auto raise = [&](float m) {
    settle();
    move_reference(acc, m);
    s2 = pack2f(acc.s, 0.f);
    t2 = pack2f(acc.t, 0.f);
    minus_m = -m;
    limit = m + kLag;
  };
  auto note = [&](float m, int col) {
    const unsigned long long k = composite(m, col);
    if (k >= tau) {
      const int i = atomicAdd(&sh.count, 1);
      if (i < (int)(sizeof(sh.cand) / 8)) sh.cand[i] = k;
    }
  };
  int col = first + tid * 8;   // the column of c[0]
  auto take = [&](const Chunk<T>& ch, int at) {
    const float m = ch.top();
    float v[8];
    ch.get(v);
    if (m > limit) raise(m);
    sums(v);
    if (!(m < tau_f)) {
      if (want) note(m, at);
    }
  };
  if (my_loose >= 0) {
    float v[8] = {loose_v, -INFINITY, -INFINITY, -INFINITY, -INFINITY, -INFINITY, -INFINITY, -INFINITY};
    if (loose_v > limit) raise(loose_v);
    sums(v);
    if (want) note(loose_v, my_loose);
  }
  // whole rounds of U chunks a thread, the next round's loads in flight
  // while one is worked on, and the rest
  const int rounds = chunks / (U * kN);
  for (int i = 0; i < rounds; ++i) {
    Chunk<T> n[U];
    body += U * kN * 8;
    if (i + 1 < rounds) {
#pragma unroll
      for (int u = 0; u < U; ++u) n[u].load(body + u * kN * 8);
    } else {
#pragma unroll
      for (int u = 0; u < U; ++u)
        if (rounds * U * kN + tid + u * kN < chunks) n[u].load(body + u * kN * 8);
    }
#pragma unroll
    for (int u = 0; u < U; ++u) take(c[u], col + u * kN * 8);
    col += U * kN * 8;
#pragma unroll
    for (int u = 0; u < U; ++u) c[u] = n[u];
  }
#pragma unroll
  for (int u = 0; u < U; ++u)
    if (rounds * U * kN + tid + u * kN < chunks) take(c[u], col + u * kN * 8);

  settle();
  // a warp's sums, about its lanes' largest reference
  const float top_m = key_value(__reduce_max_sync(0xffffffffu, order_key(acc.m)));
  if (acc.m != top_m) move_reference(acc, top_m);
  acc.s = warp_sum(acc.s);
  acc.t = warp_sum(acc.t);
  if (W > 1 && lane == 0) sh.warp[warp] = acc;
  row_sync<W>();
  unsigned long long mine = 0;   // the lane-th largest, in the row's first warp
  if (want) {
    constexpr int kRoom = (int)(sizeof(sh.cand) / 8);
    int n = sh.count;
    while (W > 1 && n > kRoom) {
      mine = largest32<W>(sh.cand, kRoom, sh.lists, warp, lane);
      if (warp == 0) sh.top[lane] = mine;
      row_sync<W>();
      tau = sh.top[a.k - 1];
      if (tid == 0) sh.count = 0;
      row_sync<W>();
      int i = tid;
      for (; i + 3 * kN < chunks; i += 4 * kN) {
        Chunk<T> ch[4];
#pragma unroll
        for (int u = 0; u < 4; ++u) ch[u].load(x + first + (int64_t)(i + u * kN) * 8);
#pragma unroll
        for (int u = 0; u < 4; ++u) note_sample(sh, composite(ch[u].top(), first + (i + u * kN) * 8), tau);
      }
      for (; i < chunks; i += kN) {
        Chunk<T> ch;
        ch.load(x + first + (int64_t)i * 8);
        note_sample(sh, composite(ch.top(), first + i * 8), tau);
      }
      if (my_loose >= 0) note_sample(sh, composite(loose_v, my_loose), tau);
      row_sync<W>();
      n = sh.count;
    }
    // the k chunks, then their logits
    mine = largest32<W>(sh.cand, n, sh.lists, warp, lane);
    if (warp == 0) sh.top[lane] = mine;
    row_sync<W>();
    if (tid == 0) sh.count = 0;
    row_sync<W>();
    const uint32_t least = (uint32_t)(sh.top[a.k - 1] >> 32);
    for (int i = tid; i < a.k * 8; i += kN) {
      const unsigned long long e = sh.top[i / 8];
      if (!e) continue;
      const int at = composite_col(e), j = i % 8;
      if (j && (at < first || at >= tail)) continue;   // a loose one
      const unsigned long long k = composite(to_f32(x[at + j]), at + j);
      if ((uint32_t)(k >> 32) >= least) sh.cand[atomicAdd(&sh.count, 1)] = k;   // 256 at most
    }
    row_sync<W>();
    mine = largest32<W>(sh.cand, sh.count, sh.lists, warp, lane);
  }
  if (warp) {
    if (W > 1 && ncl > 1) {
      asm volatile("barrier.cluster.wait.aligned;" ::: "memory");
      cluster_sync();
    }
    return;
  }
  // the row's first warp finishes
  if (W > 1) {
    acc = sh.warp[0];
    for (int w = 1; w < W; ++w) acc = merge(acc, sh.warp[w]);
  }
  __syncwarp();
  if (W > 1 && ncl > 1) {
    // the first CTA (which has started) gathers the segments' sums and lists
    asm volatile("barrier.cluster.wait.aligned;" ::: "memory");
    const uint32_t dst = cluster_addr(smem_u32(&sh.part[rank]), 0);
    if (lane == 0)
      asm volatile("st.shared::cluster.f32 [%0], %1;\n st.shared::cluster.f32 [%0 + 4], %2;\n"
                   " st.shared::cluster.f32 [%0 + 8], %3;" ::"r"(dst),
                   "f"(acc.m), "f"(acc.s), "f"(acc.t)
                   : "memory");
    if (lane < a.k)
      asm volatile("st.shared::cluster.b64 [%0], %1;" ::"r"(cluster_addr(smem_u32(&sh.tops[rank * a.k + lane]), 0)),
                   "l"(mine)
                   : "memory");
    cluster_sync();   // releases the stores, acquires them in the first CTA
    if (rank) return;
    acc = sh.part[0];
    for (uint32_t w = 1; w < ncl; ++w) acc = merge(acc, sh.part[w]);
    for (uint32_t w = 1; w < ncl && want; ++w) mine = merge32(mine, lane < a.k ? sh.tops[w * a.k + lane] : 0, lane);
  }
  const bool none = acc.s == 0.f;
  const float ln = logf(acc.s), lse = none ? -INFINITY : acc.m + ln;
  if (lane == 0) {
    if (a.lse) a.lse[row] = lse;
    if (a.entropy) a.entropy[row] = none ? 0.f : max_nan(ln - kLn2 * (acc.t / acc.s), 0.f);
    if (a.logprob) a.logprob[row] = tok < 0 || tok >= a.vocab ? 0.f : none ? -INFINITY : tok_logit - lse;
  }
  if (lane < a.k) {
    a.top_id[row * a.k + lane] = composite_col(mine);
    a.top_logprob[row * a.k + lane] = none ? -INFINITY : to_f32(x[composite_col(mine)]) - lse;
  }
}

// Which rows get how many warps, measured at k = 8:
// - up to 2048 columns one (its list holds every chunk): 16384 x 2000 bf16
//   takes 30 us, with four warps a row 77;
// - with at most four rows a SM eight, and the row cut into segments for a
//   cluster's CTAs while that leaves two blocks on every SM and two chunks a
//   thread: 600 x 50000 bf16 takes 18 us, with the four warps below 23;
// - else up to 16384 columns four, whose many short rows hide each other's
//   barriers: 4096 x 4000 bf16 takes 24 us, with eight 37, 4096 x 16000 f32 54
//   against 61;
// - beyond, eight at five blocks a SM rather than four, with a few registers
//   spilled: 2048 x 65536 f32 (k = 20) takes 95 us against 100, with four
//   warps 151.
constexpr int kWarpRow = 2048, kQuarterRow = 16384;

template <class T, int U, int W, int BLOCKS>
cudaError_t logprob_launch(const LogprobArgs& a, int64_t blocks, int cluster, cudaStream_t st) {
  cudaLaunchConfig_t cfg = pdl_config((int)blocks, W == 1 ? 128 : W * 32, 0, st);
  cudaLaunchAttribute at[2];
  at[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  at[0].val.programmaticStreamSerializationAllowed = 1;
  at[1].id = cudaLaunchAttributeClusterDimension;
  at[1].val.clusterDim.x = cluster;
  at[1].val.clusterDim.y = at[1].val.clusterDim.z = 1;
  cfg.attrs = at;
  cfg.numAttrs = cluster > 1 ? 2 : 1;
  return cudaLaunchKernelEx(&cfg, ts_logprob_kernel<T, U, W, BLOCKS>, a);
}

template <class T, int U>
cudaError_t logprob_rows(const ts_ops& h, const LogprobArgs& a, cudaStream_t st) {
  if (a.vocab <= kWarpRow) return logprob_launch<T, U, 1, 8>(a, (a.rows + 3) / 4, 1, st);
  if (a.rows <= 4 * (int64_t)h.nsm) {
    int ncl = 1;
    while (ncl < kMaxCluster && a.rows * ncl * 2 <= 2 * (int64_t)h.nsm && a.vocab / (ncl * 2) >= 256 * 16) ncl *= 2;
    return logprob_launch<T, U, 8, 4>(a, a.rows * ncl, ncl, st);
  }
  if (a.vocab <= kQuarterRow) return logprob_launch<T, U, 4, 8>(a, a.rows, 1, st);
  return logprob_launch<T, U, 8, 5>(a, a.rows, 1, st);
}

// One row's constants: dlogits = p (a - w log p) plus g at the token.  p is 2 to
// the rounded (x - lse) log2(e): off by 2^-22 of itself and |log p| 2^-23 more
// (2.4e-6 at p = e^-20), which a sum over a row's gradient does not see.
struct RowGrad {
  float lse, a, w, g;
  int tok;      // -1: the row is not scored
  bool zero;    // nothing to add up
  __device__ __forceinline__ RowGrad(const LogprobArgs& p, int64_t row) {
    lse = p.lse[row];
    const int64_t t = p.tokens[row];
    tok = t >= 0 && t < p.vocab ? (int)t : -1;
    g = tok >= 0 ? p.g_logprob[row] : 0.f;
    w = p.g_entropy ? p.g_entropy[row] : 0.f;
    zero = lse == -INFINITY || (tok < 0 && w == 0.f);
    a = -g;
    if (w != 0.f) a -= w * p.entropy[row];
  }
  // Eight logits from column c on.
  __device__ __forceinline__ void apply(float (&v)[8]) const {
    const F2 m2 = pack2f(-lse, -lse), l2 = pack2f(kLog2e, kLog2e), a2 = pack2f(a, a), w2 = pack2f(-w, -w);
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const F2 d = add2(pack2f(v[2 * i], v[2 * i + 1]), m2);
      float d0, d1;
      unpack2f(mul2(d, l2), d0, d1);
      const F2 e = pack2f(ex2(d0), ex2(d1));
      F2 o = a2;
      if (w != 0.f) {
        unpack2f(d, d0, d1);   // (where p is 0 the product must be too)
        o = fma2(w2, pack2f(max_nan(d0, -200.f), max_nan(d1, -200.f)), a2);
      }
      unpack2f(mul2(e, o), v[2 * i], v[2 * i + 1]);
    }
    if (zero) {
#pragma unroll
      for (int i = 0; i < 8; ++i) v[i] = 0.f;
    }
  }
};

// VEC: logits and gradient lie alike against 16-byte boundaries (the same
// type and pitch, or rows that start on one): a row's aligned chunks of eight
// are one lane's each, what is left at its ends single lanes'.  A warp takes
// kLpGroups consecutive groups of 32 chunks of a row, loaded together.
//
// One pass, bound by memory: 2048 x 65536 f32 takes 155 us with the entropy's
// gradient (the copy's rate; by single groups a warp, and 16 bytes a store, 167), 4096 x 50001
// bf16 at odd elements 150 us (80 %, by single elements 315).
constexpr int kLpGroups = 2;

template <class TX, class TD, bool VEC>
__global__ void __launch_bounds__(256) ts_logprob_backward_kernel(const LogprobArgs a, int per_row) {
  pdl_launch_dependents();
  pdl_wait();
  const int lane = threadIdx.x & 31;
  const int64_t i = (int64_t)blockIdx.x * 8 + (threadIdx.x >> 5);
  const int64_t row = i / per_row;
  if (row >= a.rows) return;
  const int g0 = (int)(i - row * per_row) * kLpGroups;
  const TX* x = static_cast<const TX*>(a.logits.p) + row * a.logits.ld;
  TD* d = static_cast<TD*>(a.dlogits.p) + row * a.dlogits.ld;
  int first = 0, whole = a.vocab / kGroupCols * 32;   // the first whole chunk's column, and their number
  if (VEC) {
    const int off = (int)(reinterpret_cast<uintptr_t>(x) % 16 / sizeof(TX));
    first = min(a.vocab, off ? (int)(16 / sizeof(TX)) - off : 0);
    whole = (a.vocab - first) / 8;
  }
  float v[kLpGroups][8];
#pragma unroll
  for (int u = 0; u < kLpGroups; ++u) {
    if (VEC) {
      const int c = (g0 + u) * 32 + lane;
      if (c < whole) load8(x + first + c * 8, v[u]);
    } else {
      load_group<false>(x, (g0 + u) * kGroupCols, a.vocab, lane, v[u]);
    }
  }
  const RowGrad r(a, row);
#pragma unroll
  for (int u = 0; u < kLpGroups; ++u) {
    r.apply(v[u]);
    if (VEC) {
      const int c = (g0 + u) * 32 + lane, col = first + c * 8;
      if (c >= whole) continue;
      if (!r.zero && (unsigned)(r.tok - col) < 8u) {
#pragma unroll
        for (int j = 0; j < 8; ++j)
          if (col + j == r.tok) v[u][j] += r.g;
      }
      store8(d + col, v[u]);
    } else {
#pragma unroll
      for (int j = 0; j < 8; ++j)
        if (!r.zero && (g0 + u) * kGroupCols + j * 32 + lane == r.tok) v[u][j] += r.g;
      store_group<false>(d, (g0 + u) * kGroupCols, a.vocab, lane, v[u]);
    }
  }
  if (VEC && g0 == 0) {
    // the ends of the row, at most 14 logits
    const int tail = first + whole * 8, c = lane < first ? lane : tail + lane - first;
    if (c < a.vocab) {
      float e[8] = {to_f32(x[c]), 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f};
      r.apply(e);
      d[c] = from_f32<TD>(!r.zero && c == r.tok ? e[0] + r.g : e[0]);
    }
  }
}

template <class TX, class TD>
cudaError_t backward_types(const LogprobArgs& a, cudaStream_t st) {
  const auto off = [](const void* p) { return reinterpret_cast<uintptr_t>(p) % 16; };
  const bool alike = sizeof(TX) == sizeof(TD) && off(a.logits.p) == off(a.dlogits.p) &&
                     a.logits.ld * (int64_t)sizeof(TX) % 16 == a.dlogits.ld * (int64_t)sizeof(TD) % 16;
  const bool vec = alike || (rows_aligned(a.logits) && rows_aligned(a.dlogits));
  const int per_row = (a.vocab + kGroupCols * kLpGroups - 1) / (kGroupCols * kLpGroups);
  const int64_t blocks = (a.rows * per_row + 7) / 8;
  if (blocks > 0x7fffffff) return cudaErrorInvalidConfiguration;
  cudaLaunchConfig_t cfg = pdl_config((int)blocks, 256, 0, st);
  cudaLaunchAttribute at[1];
  pdl_attr(cfg, at);
  return vec ? cudaLaunchKernelEx(&cfg, ts_logprob_backward_kernel<TX, TD, true>, a, per_row)
             : cudaLaunchKernelEx(&cfg, ts_logprob_backward_kernel<TX, TD, false>, a, per_row);
}

}  // namespace

cudaError_t launch_token_logprobs(const ts_ops& h, const LogprobArgs& a, cudaStream_t st) {
  return a.logits.bf16 ? logprob_rows<__nv_bfloat16, 4>(h, a, st) : logprob_rows<float, 2>(h, a, st);
}

cudaError_t launch_token_logprobs_backward(const ts_ops&, const LogprobArgs& a, cudaStream_t st) {
  using B = __nv_bfloat16;
  if (a.logits.bf16) return a.dlogits.bf16 ? backward_types<B, B>(a, st) : backward_types<B, float>(a, st);
  return a.dlogits.bf16 ? backward_types<float, B>(a, st) : backward_types<float, float>(a, st);
}

}  // namespace fg
