// Embedding of tokens, y_t = scale * table[id_t], and the table's gradient,
// dtable_v = scale * sum of dy_t over the tokens t with id_t = v.
//
// The lookup is bound by memory: a warp takes 256 columns of a token's row at
// a time, four such pieces in flight where there are enough of them.
//
// The gradient sums in an order that the ids and the sizes fix, so that it is the
// same every time: the tokens are sorted by id (a stable radix sort, up to 9 bits
// a pass), and the sorted list is cut into chunks of equal length, however often a
// token occurs.  A warp sums one chunk's rows over 256 columns in registers, a
// batch of rows loaded while one is added, and writes each id's row once.  An id
// whose tokens lie in more than one chunk leaves a float32 partial in the
// workspace for each, which a second kernel adds in order.  Rows of the table that
// no token uses are zeroed by later blocks of the same launch.
//
// At 8192 x 4096 bf16 into a float32 gradient of 50001 rows this takes 145 us (89 %
// of the copy rate; 130 of it the sums and zeros, 9 the sort), added to what is
// there 45 us (95 %); 65536 x 1003 float32 added to 50001 rows 99 us (87 %).
#include <algorithm>
#include <atomic>
#include <type_traits>

#include "launch.h"
#include "ts_device.cuh"

namespace fg {
namespace {

constexpr int kWarps = 8;
constexpr int kThreads = kWarps * 32;

// ---- lookup -------------------------------------------------------------------

struct EmbedKernel {
  const int64_t* ids;
  const void* table;
  void* y;
  int64_t vocab, ldt, ldy, units;
  int cols, packs;   // a unit is GROUPS groups of columns of one token, `packs` of them a token
  float scale;
};

template <class T, class U, bool VEC, int GROUPS>
__global__ void __launch_bounds__(kThreads) ts_embed_kernel(const __grid_constant__ EmbedKernel P) {
  pdl_launch_dependents();
  pdl_wait();
  const int lane = threadIdx.x & 31;
  const int64_t u = (int64_t)blockIdx.x * kWarps + (threadIdx.x >> 5);
  if (u >= P.units) return;
  const int64_t t = u / P.packs;
  const int c0 = (int)(u - t * P.packs) * GROUPS * kGroupCols;
  const int64_t id = P.ids[t];
  const bool there = id >= 0 && id < P.vocab;
  const T* src = static_cast<const T*>(P.table) + (there ? id : 0) * P.ldt;
  U* dst = static_cast<U*>(P.y) + t * P.ldy;
  RawGroup<T, VEC> raw[GROUPS];
#pragma unroll
  for (int g = 0; g < GROUPS; ++g) raw[g].load(src, c0 + g * kGroupCols, there ? P.cols : 0, lane);
#pragma unroll
  for (int g = 0; g < GROUPS; ++g) {
    if (c0 + g * kGroupCols >= P.cols) break;
    float v[8];
    raw[g].get(v);
#pragma unroll
    for (int j = 0; j < 8; ++j) v[j] = there ? v[j] * P.scale : 0.f;
    store_group<VEC>(dst, c0 + g * kGroupCols, P.cols, lane, v);
  }
}

// ---- tokens sorted by id ----------------------------------------------------------

constexpr int kSortThreads = 1024, kSortWarps = 32;
constexpr int kMaxBits = 9, kMaxBins = 1 << kMaxBits;
// Lists that one cluster sorts in one launch, every CTA holding a part of it.
constexpr int kClusterCtas = 8, kClusterPer = 2;   // CTAs, and 32-token rounds a warp, at most
constexpr int kClusterList = kClusterCtas * kClusterPer * kSortThreads;
// 32-token rounds that a warp takes of a longer list's tile: a shorter one is
// spread over more blocks, a long one has fewer counts that every block adds up.
constexpr int kShortPer = 2, kLongPer = 8;
constexpr int64_t kShortList = 1 << 18;

struct SortKernel {
  const int64_t* ids;
  int64_t vocab;
  int rows, passes, bits;
  uint2* out;            // (key, token) sorted by key, tokens of a key in order
  uint32_t* joins;       // set to 0; see EmbedBackKernel
  uint8_t* present;      // [vocab], whether an id has tokens; null: not wanted
  // one pass over a longer list
  const uint2* in;       // null: the ids
  uint32_t* counts;      // [tiles][bins]
  int shift, tiles;
};

// Zeros, 16 bytes at a time, by thread `t` of `n`; the array's place is rounded up
// to 256 bytes.
__device__ __forceinline__ void clear_present(uint8_t* p, int64_t vocab, int64_t t, int64_t n) {
  for (int64_t i = t * 16; p && i < vocab; i += n * 16) *reinterpret_cast<uint4*>(p + i) = make_uint4(0, 0, 0, 0);
}
// An id as a key: ids outside the table sort last.
__device__ __forceinline__ uint32_t id_key(int64_t id, int64_t vocab) {
  return id >= 0 && id < vocab ? (uint32_t)id : (uint32_t)vocab;
}

// Exclusive sum of v over the block's threads; every thread takes part.
__device__ __forceinline__ uint32_t block_exclusive(uint32_t v, uint32_t* warp_sums) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  uint32_t s = v;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const uint32_t n = __shfl_up_sync(0xffffffffu, s, o);
    if (lane >= o) s += n;
  }
  if (lane == 31) warp_sums[warp] = s;
  __syncthreads();
  if (warp == 0) {
    const uint32_t w = warp_sums[lane];
    uint32_t x = w;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const uint32_t n = __shfl_up_sync(0xffffffffu, x, o);
      if (lane >= o) x += n;
    }
    warp_sums[lane] = x - w;
  }
  __syncthreads();
  return warp_sums[warp] + s - v;
}

// The ranks of a warp's rounds of 32 keys among the warp's keys of the same
// digit, in order, and the counts in hist[digit] (a row of this warp's own).
// Rounds past `n` keys take no part.  Keys of the same digit find each other by
// a vote for each bit.
template <int PER>
__device__ __forceinline__ void warp_ranks(const uint32_t (&digit)[PER], int first, int n, int bits, uint32_t* hist,
                                           uint32_t (&rank)[PER]) {
  const int lane = threadIdx.x & 31;
  for (int d = lane; d < 1 << bits; d += 32) hist[d] = 0;
  __syncwarp();
#pragma unroll
  for (int r = 0; r < PER; ++r) {
    if (first + r * 32 >= n) break;
    const bool in = first + r * 32 + lane < n;
    const uint32_t d = digit[r];
    uint32_t peers = __ballot_sync(0xffffffffu, in);
#pragma unroll
    for (int b = 0; b < kMaxBits; ++b) {
      const uint32_t set = __ballot_sync(0xffffffffu, d >> b & 1);   // (digits have no bits past `bits`)
      peers &= d >> b & 1 ? set : ~set;
    }
    const uint32_t base = in ? hist[d] : 0;
    __syncwarp();
    if (in && (peers & ((1u << lane) - 1)) == 0) hist[d] = base + __popc(peers);
    __syncwarp();
    rank[r] = base + __popc(peers & ((1u << lane) - 1));
  }
}
// Turns the warps' counts of each digit into the sums of the warps before, and
// returns the digit's total (thread d < bins).
__device__ __forceinline__ uint32_t warp_offsets(uint32_t* hist, int bins) {
  uint32_t sum = 0;
  if ((int)threadIdx.x < bins) {
#pragma unroll 8
    for (int w = 0; w < kSortWarps; ++w) {
      const uint32_t c = hist[w * kMaxBins + threadIdx.x];
      hist[w * kMaxBins + threadIdx.x] = sum;
      sum += c;
    }
  }
  return sum;
}

// Up to kClusterList tokens in one launch: the list lies in the shared memory of
// a cluster's CTAs, PER * 1024 tokens each, and every pass scatters it there.
// One CTA by itself took 18 us for 8192 tokens, 16 of it instruction issue, this
// 10.  65536 tokens in eight CTAs took 29 us; passes in launches of their own (a
// count and a scatter each, below) 21.
template <int PER>
constexpr int kClusterSmem = (2 * PER * kSortThreads + kSortWarps * kMaxBins + 2 * kMaxBins + 32) * 4;

template <int PER>
__global__ void __launch_bounds__(kSortThreads, 1) ts_sort_cluster_kernel(const __grid_constant__ SortKernel P) {
  extern __shared__ __align__(16) uint32_t smem[];
  constexpr int kPart = PER * kSortThreads;
  uint2* buf = reinterpret_cast<uint2*>(smem);
  uint32_t* hist = smem + 2 * kPart;
  uint32_t* base = hist + kSortWarps * kMaxBins;
  uint32_t* totals = base + kMaxBins;
  uint32_t* sums = totals + kMaxBins;
  pdl_launch_dependents();
  pdl_wait();
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, bins = 1 << P.bits;
  const int cta = (int)cluster_ctarank();
  // a warp's rounds follow each other in the list, so that ranks keep its order
  const int part0 = cta * kPart, first = warp * PER * 32, n = min(P.rows - part0, first + PER * 32);
  uint2 e[PER];
#pragma unroll
  for (int r = 0; r < PER; ++r) {
    const int i = first + r * 32 + lane;
    e[r] = make_uint2(i < n ? id_key(P.ids[part0 + i], P.vocab) : 0, part0 + i);
  }
  if (cta == 0 && threadIdx.x == 0) *P.joins = 0;
  clear_present(P.present, P.vocab, cta * kSortThreads + threadIdx.x, kClusterCtas * kSortThreads);
  for (int pass = 0; pass < P.passes; ++pass) {
    uint32_t digit[PER], rank[PER];
#pragma unroll
    for (int r = 0; r < PER; ++r) digit[r] = (e[r].x >> (pass * P.bits)) & (bins - 1);
    warp_ranks(digit, first, n, P.bits, hist + warp * kMaxBins, rank);
    __syncthreads();
    const uint32_t mine = warp_offsets(hist, bins);
    if ((int)threadIdx.x < bins) totals[threadIdx.x] = mine;
    __threadfence();
    cluster_sync();   // (every CTA has its tokens in registers now, and `present` is clear)
    if (pass == 0 && P.present) {
#pragma unroll
      for (int r = 0; r < PER; ++r)
        if (first + r * 32 + lane < n && e[r].x < (uint32_t)P.vocab) P.present[e[r].x] = 1;
    }
    uint32_t before = 0, total = 0;
    if ((int)threadIdx.x < bins) {
      const uint32_t at = smem_u32(totals + threadIdx.x);
#pragma unroll
      for (int c = 0; c < kClusterCtas; ++c) {
        uint32_t v;
        asm volatile("ld.shared::cluster.u32 %0, [%1];" : "=r"(v) : "r"(cluster_addr(at, c)) : "memory");
        total += v;
        if (c < cta) before += v;
      }
    }
    const uint32_t at = block_exclusive(total, sums);
    if ((int)threadIdx.x < bins) base[threadIdx.x] = at + before;
    __syncthreads();
#pragma unroll
    for (int r = 0; r < PER; ++r) {
      if (first + r * 32 + lane < n) {
        const uint32_t pos = base[digit[r]] + hist[warp * kMaxBins + digit[r]] + rank[r];
        asm volatile("st.shared::cluster.v2.u32 [%0], {%1, %2};" ::"r"(
                         cluster_addr(smem_u32(buf + pos % kPart), pos / kPart)),
                     "r"(e[r].x), "r"(e[r].y)
                     : "memory");
      }
    }
    cluster_sync();
    if (pass + 1 < P.passes) {
#pragma unroll
      for (int r = 0; r < PER; ++r) {
        const int i = first + r * 32 + lane;
        if (i < n) e[r] = buf[i];
      }
    }
  }
  for (int i = threadIdx.x; i < min(P.rows - part0, kPart); i += kSortThreads) P.out[part0 + i] = buf[i];
}

// Longer lists: a pass's counts by tile, and the pass.
template <int PER>
__global__ void __launch_bounds__(kSortThreads) ts_sort_count_kernel(const __grid_constant__ SortKernel P) {
  __shared__ uint32_t hist[kMaxBins];
  pdl_launch_dependents();
  pdl_wait();
  const int bins = 1 << P.bits;
  if ((int)threadIdx.x < bins) hist[threadIdx.x] = 0;
  __syncthreads();
#pragma unroll
  for (int r = 0; r < PER; ++r) {
    const int64_t i = ((int64_t)blockIdx.x * PER + r) * kSortThreads + threadIdx.x;
    if (i < P.rows)
      atomicAdd(&hist[(P.in ? P.in[i].x : id_key(P.ids[i], P.vocab)) >> P.shift & (bins - 1)], 1u);
  }
  if (blockIdx.x == 0 && threadIdx.x == 0) *P.joins = 0;
  if (!P.in)
    clear_present(P.present, P.vocab, (int64_t)blockIdx.x * kSortThreads + threadIdx.x,
                  (int64_t)gridDim.x * kSortThreads);
  __syncthreads();
  if ((int)threadIdx.x < bins) P.counts[(int64_t)blockIdx.x * bins + threadIdx.x] = hist[threadIdx.x];
}

template <int PER>
__global__ void __launch_bounds__(kSortThreads) ts_sort_pass_kernel(const __grid_constant__ SortKernel P) {
  extern __shared__ uint32_t smem[];
  uint32_t* hist = smem;
  uint32_t* base = hist + kSortWarps * kMaxBins;
  uint32_t* sums = base + kMaxBins;
  pdl_launch_dependents();
  pdl_wait();
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, bins = 1 << P.bits;
  const int tile0 = blockIdx.x * PER * kSortThreads, first = warp * PER * 32;
  const int n = min(P.rows - tile0, first + PER * 32);
  uint2 e[PER];
  uint32_t digit[PER], rank[PER];
#pragma unroll
  for (int r = 0; r < PER; ++r) {
    const int i = first + r * 32 + lane;
    e[r] = make_uint2(0, 0);
    if (i < n) e[r] = P.in ? P.in[tile0 + i] : make_uint2(id_key(P.ids[tile0 + i], P.vocab), tile0 + i);
    digit[r] = (e[r].x >> P.shift) & (bins - 1);
  }
  uint32_t before = 0, total = 0;
  if ((int)threadIdx.x < bins) {
    const uint32_t* c = P.counts + threadIdx.x;
#pragma unroll 8
    for (int b = 0; b < P.tiles; ++b) {
      const uint32_t v = c[(int64_t)b * bins];
      total += v;
      if (b < (int)blockIdx.x) before += v;
    }
  }
  warp_ranks(digit, first, n, P.bits, hist + warp * kMaxBins, rank);
  __syncthreads();
  warp_offsets(hist, bins);
  const uint32_t at = block_exclusive(total, sums);
  if ((int)threadIdx.x < bins) base[threadIdx.x] = at + before;
  __syncthreads();
#pragma unroll
  for (int r = 0; r < PER; ++r) {
    if (first + r * 32 + lane < n) {
      P.out[base[digit[r]] + hist[warp * kMaxBins + digit[r]] + rank[r]] = e[r];
      if (!P.in && P.present && e[r].x < (uint32_t)P.vocab) P.present[e[r].x] = 1;
    }
  }
}

// ---- sums of the sorted tokens' rows ------------------------------------------------

struct EmbedBackKernel {
  const uint2* list;     // (key, token), sorted
  const void* dy;
  void* d;
  float* part;           // [chunks][2][part_cols]: a chunk's first id's, its last id's
  uint32_t* joins;       // how many ids lie in more than one chunk, and the chunks where they begin
  const uint8_t* present;
  int64_t lddy, ldd, part_cols, units, unit_blocks, vocab;
  int rows, cols, groups, chunk, chunks;
  float scale;
};

constexpr int kFillRows = 8;   // rows of the table a warp looks up at a time
constexpr int kChunk = 64;     // tokens of a chunk, at most

__device__ __forceinline__ float* part_at(const EmbedBackKernel& P, int chunk, int slot, int group, int lane) {
  return P.part + ((int64_t)chunk * 2 + slot) * P.part_cols + group * kGroupCols + lane * 8;
}

// A warp's 256 columns, eight to a lane: with VEC (all rows on 16 bytes) twice four
// that lie together, 128 apart, so that each access of the warp covers whole lines
// of either type (eight together, two accesses with gaps of 16 bytes for float32,
// took 65536 x 1003 117 us in place of 99).
template <bool VEC>
__device__ __forceinline__ int quad_col(int lane, int j) {
  return VEC ? (j >> 2) * 128 + lane * 4 + (j & 3) : j * 32 + lane;
}
// Four values of a row as they lie in memory.
template <class T>
struct alignas(4 * sizeof(T)) Quad {
  uint32_t w[sizeof(T)];
  // the last ones of a row, zeros past its `n` (< 4) columns
  __device__ __forceinline__ void edge(const T* p, int n) {
#pragma unroll
    for (int i = 0; i < (int)sizeof(T); ++i) {
      if constexpr (sizeof(T) == 4) {
        w[i] = i < n ? __float_as_uint(p[i]) : 0u;
      } else {
        w[i] = bf16x2(2 * i < n ? to_f32(p[2 * i]) : 0.f, 2 * i + 1 < n ? to_f32(p[2 * i + 1]) : 0.f);
      }
    }
  }
  __device__ __forceinline__ float get(int j) const {
    if constexpr (sizeof(T) == 4) return __uint_as_float(w[j]);
    else return __uint_as_float(j & 1 ? w[j >> 1] & 0xffff0000u : w[j >> 1] << 16);
  }
  __device__ __forceinline__ void set(const float* v) {
#pragma unroll
    for (int i = 0; i < (int)sizeof(T); ++i) {
      if constexpr (sizeof(T) == 4) w[i] = __float_as_uint(v[i]);
      else w[i] = bf16x2(v[2 * i], v[2 * i + 1]);
    }
  }
};
template <class T, bool VEC>
struct RawQuads : RawGroup<T, false> {};
template <class T>
struct RawQuads<T, true> {
  Quad<T> q[2];
  __device__ __forceinline__ void load(const T* p, int c0, int cols, int lane) {
#pragma unroll
    for (int k = 0; k < 2; ++k) {
      const int c = c0 + quad_col<true>(lane, 4 * k);
      if (c + 4 <= cols) q[k] = *reinterpret_cast<const Quad<T>*>(p + c);
      else q[k].edge(p + c, cols - c);
    }
  }
  __device__ __forceinline__ void get(float (&v)[8]) const {
#pragma unroll
    for (int j = 0; j < 8; ++j) v[j] = q[j >> 2].get(j & 3);
  }
};
template <bool VEC, class T>
__device__ __forceinline__ void store_quads(T* p, int c0, int cols, int lane, const float (&v)[8]) {
#pragma unroll
  for (int k = 0; k < 2; ++k) {
    if (VEC && c0 + quad_col<VEC>(lane, 4 * k) + 4 <= cols) {
      Quad<T> q;
      q.set(v + 4 * k);
      *reinterpret_cast<Quad<T>*>(p + c0 + quad_col<VEC>(lane, 4 * k)) = q;
    } else {
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const int c = c0 + quad_col<VEC>(lane, 4 * k + j);
        if (c < cols) p[c] = from_f32<T>(v[4 * k + j]);
      }
    }
  }
}

// Whether the sum is added in memory: float32 rows, each value by one reduction
// of one launch, so that it does not matter when.  (Reading them first took
// 65536 x 1003 into 50001 131 us in place of 111.)
template <class U, bool ACC>
constexpr bool kAddInMemory = ACC && std::is_same<U, float>::value;

// Adds the values to a float32 row.
template <bool VEC>
__device__ __forceinline__ void add_quads(float* p, int c0, int cols, int lane, const float (&v)[8]) {
#pragma unroll
  for (int k = 0; k < 2; ++k) {
    float* q = p + c0 + quad_col<VEC>(lane, 4 * k);
    if (VEC && c0 + quad_col<VEC>(lane, 4 * k) + 4 <= cols) {
      asm volatile("red.relaxed.gpu.global.add.v4.f32 [%0], {%1, %2, %3, %4};" ::"l"(q), "f"(v[4 * k]), "f"(v[4 * k + 1]),
                   "f"(v[4 * k + 2]), "f"(v[4 * k + 3])
                   : "memory");
    } else {
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const int c = c0 + quad_col<VEC>(lane, 4 * k + j);
        if (c < cols) atomicAdd(p + c, v[4 * k + j]);
      }
    }
  }
}

// scale * sum, or (ACC, in 16 bits) old + scale * sum, into a row.
template <bool VEC, bool ACC, class U>
__device__ __forceinline__ void finish(U* row, float scale, const float (&acc)[8], const float (&old)[8], int c0,
                                       int cols, int lane) {
  float v[8];
  if constexpr (kAddInMemory<U, ACC>) {
#pragma unroll
    for (int j = 0; j < 8; ++j) v[j] = scale * acc[j];
    add_quads<VEC>(row, c0, cols, lane, v);
  } else {
#pragma unroll
    for (int j = 0; j < 8; ++j) v[j] = ACC ? fmaf(scale, acc[j], old[j]) : scale * acc[j];
    store_quads<VEC>(row, c0, cols, lane, v);
  }
}

// T: dy's type, U: dtable's; ACC adds to what dtable holds.
template <class T, class U, bool VEC, bool ACC>
__global__ void __launch_bounds__(kThreads, 2) ts_embed_sum_kernel(const __grid_constant__ EmbedBackKernel P) {
  pdl_launch_dependents();
  pdl_wait();
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  U* d = static_cast<U*>(P.d);
  if (blockIdx.x >= P.unit_blocks) {
    // rows that no token uses
    const int64_t r0 = ((blockIdx.x - P.unit_blocks) * kWarps + warp) * kFillRows, v = r0 + lane;
    const bool absent = lane < kFillRows && v < P.vocab && !P.present[v];
    const float zero[8] = {};
    for (uint32_t m = __ballot_sync(0xffffffffu, absent); m; m &= m - 1) {
      U* row = d + (r0 + __ffs(m) - 1) * P.ldd;
      for (int c = 0; c < P.cols; c += kGroupCols) store_group<VEC>(row, c, P.cols, lane, zero);
    }
    return;
  }
  const int64_t u = (int64_t)blockIdx.x * kWarps + warp;
  if (u >= P.units) return;
  const int chunk = (int)(u / P.groups), group = (int)(u - (int64_t)chunk * P.groups), c0 = group * kGroupCols;
  const int p0 = chunk * P.chunk, p1 = min(P.rows, p0 + P.chunk);
  const T* dy = static_cast<const T*>(P.dy);
  const uint32_t vocab = (uint32_t)P.vocab;
  constexpr bool kOld = ACC && !kAddInMemory<U, ACC>;   // what dtable holds is read
  // rows of a batch; one is loaded while one is added
  constexpr int kU = kOld ? 2 : VEC && sizeof(T) == 2 ? 8 : 4;
  struct Batch {
    RawQuads<T, VEC> raw[kU];
    RawQuads<U, VEC> old[kOld ? kU : 1];
  };
  bool open = false;
  F2 acc[4] = {};
  for (int q = p0; q < p1; q += 32) {
    // lane j: token j, and whether it is its id's last of the chunk (`cuts`) or of
    // all (`ends`); padded places sort last and are left out
    const int at = q + lane;
    const uint2 e = at < p1 ? P.list[at] : make_uint2(vocab, 0);
    const uint32_t next = at < p1 && at + 1 < P.rows ? P.list[at + 1].x : 0xffffffffu;
    const int n = __popc(__ballot_sync(0xffffffffu, e.x < vocab));
    if (n == 0) return;
    const uint32_t ends = __ballot_sync(0xffffffffu, next != e.x);
    const uint32_t cuts = ends | (p1 - q <= 32 ? 1u << (p1 - q - 1) : 0);
    // the first id may have tokens in the chunk before
    if (q == p0) open = p0 > 0 && P.list[p0 - 1].x == __shfl_sync(0xffffffffu, e.x, 0);
    auto load = [&](Batch& b, int j) {
#pragma unroll
      for (int i = 0; i < kU; ++i) {
        const int t = min(j + i, n - 1);   // (past the last one it is loaded again)
        const uint32_t xi = __shfl_sync(0xffffffffu, e.y, t);
        b.raw[i].load(dy + (int64_t)xi * P.lddy, c0, P.cols, lane);
        if constexpr (kOld) {
          const uint32_t ki = __shfl_sync(0xffffffffu, e.x, t);
          b.old[i].load(d + (int64_t)ki * P.ldd, c0, ends >> t & 1 ? P.cols : 0, lane);
        }
      }
    };
    auto add = [&](const Batch& b, int j) {
#pragma unroll
      for (int i = 0; i < kU; ++i) {
        if (j + i >= n) return;
        float v[8];
        b.raw[i].get(v);
#pragma unroll
        for (int m = 0; m < 4; ++m) acc[m] = add2(acc[m], pack2f(v[2 * m], v[2 * m + 1]));
        if (!(cuts >> (j + i) & 1)) continue;
        const bool whole = !open && (ends >> (j + i) & 1);
#pragma unroll
        for (int m = 0; m < 4; ++m) unpack2f(acc[m], v[2 * m], v[2 * m + 1]);
        if (whole) {
          float was[8] = {};
          if constexpr (kOld) b.old[i].get(was);
          const uint32_t ki = __shfl_sync(0xffffffffu, e.x, j + i);
          finish<VEC, ACC>(d + (int64_t)ki * P.ldd, P.scale, v, was, c0, P.cols, lane);
        } else {
          float* o = part_at(P, chunk, open ? 0 : 1, group, lane);
          reinterpret_cast<float4*>(o)[0] = make_float4(v[0], v[1], v[2], v[3]);
          reinterpret_cast<float4*>(o)[1] = make_float4(v[4], v[5], v[6], v[7]);
          if (!open && group == 0 && lane == 0) P.joins[1 + atomicAdd(P.joins, 1u)] = chunk;
        }
        open = false;
#pragma unroll
        for (int m = 0; m < 4; ++m) acc[m] = 0;
      }
    };
    Batch b0, b1;
    load(b0, 0);
    for (int j = 0; j < n; j += 2 * kU) {
      load(b1, j + kU);
      add(b0, j);
      load(b0, j + 2 * kU);
      add(b1, j + kU);
    }
  }
}

// The ids whose tokens lie in more than one chunk, as the kernel before has
// noted them (in any order: each is summed by itself, its chunks in order).  A
// warp takes 64 columns, so that an id of many chunks has many warps: at 65536
// tokens the most frequent id has about 75 chunks.
constexpr int kJoinCols = 64;

template <class U, bool VEC, bool ACC>
__global__ void __launch_bounds__(kThreads) ts_embed_join_kernel(const __grid_constant__ EmbedBackKernel P) {
  pdl_launch_dependents();
  pdl_wait();
  const int lane = threadIdx.x & 31, pieces = (int)(P.part_cols / kJoinCols);
  const int64_t items = (int64_t)*P.joins * pieces;
  for (int64_t u = (int64_t)blockIdx.x * kWarps + (threadIdx.x >> 5); u < items; u += (int64_t)gridDim.x * kWarps) {
    const int piece = (int)(u % pieces), chunk = (int)P.joins[1 + u / pieces];
    const int64_t p1 = (int64_t)(chunk + 1) * P.chunk;
    const uint32_t k = P.list[p1].x;
    // a lane's two places among a group's, and their columns
    const int pos = piece * kJoinCols % kGroupCols + lane * 2;
    const float* part = part_at(P, chunk, 0, piece * kJoinCols / kGroupCols, 0) + pos;
    const int64_t step = 2 * P.part_cols;   // to the next chunk's
    float2 acc = *reinterpret_cast<const float2*>(part + P.part_cols);
    for (int64_t e = chunk + 1;; e += 32) {
      // lane i: whether the id goes on past chunk e + i
      const int64_t after = (e + lane + 1) * P.chunk;
      const uint32_t stops = __ballot_sync(0xffffffffu, !(after < P.rows && P.list[after].x == k));
      const int n = stops ? __ffs(stops) : 32;
      const float* o = part + (e - chunk) * step;
      for (int j = 0; j < n; j += 16) {
        float2 x[16];
#pragma unroll
        for (int i = 0; i < 16; ++i)
          if (j + i < n) x[i] = *reinterpret_cast<const float2*>(o + (j + i) * step);
#pragma unroll
        for (int i = 0; i < 16; ++i) {
          if (j + i < n) {
            acc.x += x[i].x;
            acc.y += x[i].y;
          }
        }
      }
      if (stops) break;
    }
    U* row = static_cast<U*>(P.d) + (int64_t)k * P.ldd;
    const float v[2] = {acc.x, acc.y};
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      const int c = piece * kJoinCols / kGroupCols * kGroupCols + quad_col<VEC>((pos + i) / 8, (pos + i) % 8);
      if (c < P.cols) row[c] = from_f32<U>(ACC ? fmaf(P.scale, v[i], to_f32(row[c])) : P.scale * v[i]);
    }
  }
}

// ---- few tokens ------------------------------------------------------------------------

// Up to kFewTokens tokens in one launch.  Every block sorts the tokens for itself
// (one a thread) and then takes 64 columns of all of them, its warps a part of the
// sorted list each; the parts of an id meet in shared memory.  Later blocks zero
// the rows that no token uses.  (512 tokens of 256 columns: 8.1 us, by the three
// kernels above, one after the other, 11.7.)
constexpr int kFewTokens = kSortThreads;
constexpr int kFewCols = 64;
constexpr int kFewSmem =
    (kSortWarps * kMaxBins + kMaxBins + 32 + 2 * kFewTokens + kSortWarps * 2 * kFewCols) * 4;

struct EmbedFewKernel {
  const int64_t* ids;
  const void* dy;
  void* d;
  int64_t vocab, lddy, ldd;
  int rows, cols, passes, bits, pieces;   // pieces of kFewCols columns, a block each
  int fill;                               // rows of the table that a later block's warp looks up
  float scale;
};

// A lane's two columns of 64: side by side (VEC: rows on 16 bytes), or 32 apart.
template <bool VEC>
__device__ __forceinline__ int few_col(int lane, int i) {
  return VEC ? 2 * lane + i : lane + 32 * i;
}
template <bool VEC, class T>
__device__ __forceinline__ float2 load_pair(const T* p, int c0, int cols, int lane) {
  if (VEC && c0 + 2 * lane + 2 <= cols) {
    if constexpr (sizeof(T) == 4) return *reinterpret_cast<const float2*>(p + c0 + 2 * lane);
    else return __bfloat1622float2(*reinterpret_cast<const __nv_bfloat162*>(p + c0 + 2 * lane));
  }
  float2 v = make_float2(0.f, 0.f);
  if (c0 + few_col<VEC>(lane, 0) < cols) v.x = to_f32(p[c0 + few_col<VEC>(lane, 0)]);
  if (c0 + few_col<VEC>(lane, 1) < cols) v.y = to_f32(p[c0 + few_col<VEC>(lane, 1)]);
  return v;
}
template <bool VEC, class T>
__device__ __forceinline__ void store_pair(T* p, int c0, int cols, int lane, float2 v) {
  if (VEC && c0 + 2 * lane + 2 <= cols) {
    if constexpr (sizeof(T) == 4) *reinterpret_cast<float2*>(p + c0 + 2 * lane) = v;
    else *reinterpret_cast<__nv_bfloat162*>(p + c0 + 2 * lane) = __floats2bfloat162_rn(v.x, v.y);
    return;
  }
  if (c0 + few_col<VEC>(lane, 0) < cols) p[c0 + few_col<VEC>(lane, 0)] = from_f32<T>(v.x);
  if (c0 + few_col<VEC>(lane, 1) < cols) p[c0 + few_col<VEC>(lane, 1)] = from_f32<T>(v.y);
}

template <class T, class U, bool VEC, bool ACC>
__global__ void __launch_bounds__(kSortThreads) ts_embed_few_kernel(const __grid_constant__ EmbedFewKernel P) {
  extern __shared__ __align__(16) uint32_t smem[];
  uint2* list = reinterpret_cast<uint2*>(smem);
  float2* part = reinterpret_cast<float2*>(smem + 2 * kFewTokens);   // [warps][2][32]
  uint32_t* hist = smem + 2 * kFewTokens + kSortWarps * 2 * kFewCols;
  uint32_t* base = hist + kSortWarps * kMaxBins;
  uint32_t* sums = base + kMaxBins;
  pdl_launch_dependents();
  pdl_wait();
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, bins = 1 << P.bits;
  const uint32_t vocab = (uint32_t)P.vocab;
  {
    const int i = threadIdx.x;
    uint2 e = make_uint2(i < P.rows ? id_key(P.ids[i], P.vocab) : 0, i);
    for (int pass = 0; pass < P.passes; ++pass) {
      const uint32_t digit[1] = {(e.x >> (pass * P.bits)) & (bins - 1)};
      uint32_t rank[1];
      warp_ranks(digit, warp * 32, P.rows, P.bits, hist + warp * kMaxBins, rank);
      __syncthreads();
      const uint32_t at = block_exclusive(warp_offsets(hist, bins), sums);
      if ((int)threadIdx.x < bins) base[threadIdx.x] = at;
      __syncthreads();
      if (i < P.rows) list[base[digit[0]] + hist[warp * kMaxBins + digit[0]] + rank[0]] = e;
      __syncthreads();
      if (i < P.rows) e = list[i];
      __syncthreads();
    }
  }
  U* d = static_cast<U*>(P.d);
  if ((int)blockIdx.x >= P.pieces) {
    // rows that no token uses
    const int64_t r0 = ((int64_t)(blockIdx.x - P.pieces) * kSortWarps + warp) * P.fill, v = r0 + lane;
    bool absent = lane < P.fill && v < P.vocab;
    if (absent) {
      int lo = 0, hi = P.rows;
      while (lo < hi) {
        const int mid = (lo + hi) >> 1;
        if ((int64_t)list[mid].x < v) lo = mid + 1;
        else hi = mid;
      }
      absent = !(lo < P.rows && (int64_t)list[lo].x == v);
    }
    const float zero[8] = {};
    for (uint32_t m = __ballot_sync(0xffffffffu, absent); m; m &= m - 1) {
      U* row = d + (r0 + __ffs(m) - 1) * P.ldd;
      for (int c = 0; c < P.cols; c += kGroupCols) store_group<VEC>(row, c, P.cols, lane, zero);
    }
    return;
  }
  const int c0 = blockIdx.x * kFewCols, per = (P.rows + kSortWarps - 1) / kSortWarps;   // tokens a warp, at most 32
  const int p0 = warp * per, n = max(0, min(P.rows - p0, per));
  const T* dy = static_cast<const T*>(P.dy);
  // lane j: token j of the warp's part, and the id after it
  const uint2 e = lane < n ? list[p0 + lane] : make_uint2(vocab, 0);
  const uint32_t next = lane < n && p0 + lane + 1 < P.rows ? list[p0 + lane + 1].x : 0xffffffffu;
  const uint32_t first = __shfl_sync(0xffffffffu, e.x, 0);
  bool open = n > 0 && p0 > 0 && list[p0 - 1].x == first;   // the first id has tokens in the part before
  bool goes_on = false;                                       // an id that begins here has some in the next
  auto out = [&](uint32_t k, float2 acc, float2 old) {
    acc.x = ACC ? fmaf(P.scale, acc.x, old.x) : P.scale * acc.x;
    acc.y = ACC ? fmaf(P.scale, acc.y, old.y) : P.scale * acc.y;
    store_pair<VEC>(d + (int64_t)k * P.ldd, c0, P.cols, lane, acc);
  };
  constexpr int kU = 8;   // rows in flight
  float2 acc = make_float2(0.f, 0.f);
  for (int j = 0; j < n; j += kU) {
    float2 x[kU], old[ACC ? kU : 1];
#pragma unroll
    for (int i = 0; i < kU; ++i) {
      const uint32_t ki = __shfl_sync(0xffffffffu, e.x, (j + i) & 31), xi = __shfl_sync(0xffffffffu, e.y, (j + i) & 31);
      const bool in = j + i < n && ki < vocab;
      x[i] = load_pair<VEC>(dy + (int64_t)(in ? xi : 0) * P.lddy, c0, in ? P.cols : 0, lane);
      if constexpr (ACC) {
        const bool ends = in && __shfl_sync(0xffffffffu, next, (j + i) & 31) != ki;
        old[i] = load_pair<VEC>(d + (int64_t)(ends ? ki : 0) * P.ldd, c0, ends ? P.cols : 0, lane);
      }
    }
#pragma unroll
    for (int i = 0; i < kU; ++i) {
      const uint32_t ki = __shfl_sync(0xffffffffu, e.x, (j + i) & 31), ni = __shfl_sync(0xffffffffu, next, (j + i) & 31);
      if (j + i >= n || ki >= vocab) break;   // (padded places sort last)
      acc.x += x[i].x;
      acc.y += x[i].y;
      const bool ends = ni != ki;
      if (!ends && j + i + 1 < n) continue;
      if (open || !ends) {
        part[(warp * 2 + !open) * 32 + lane] = acc;
        goes_on = !open;
      } else {
        out(ki, acc, old[ACC ? i : 0]);
      }
      open = false;
      acc = make_float2(0.f, 0.f);
    }
  }
  __syncthreads();
  if (!goes_on) return;
  // the id of this part's last token: the parts after it, in order
  const uint32_t k = __shfl_sync(0xffffffffu, e.x, n - 1);
  float2 old = make_float2(0.f, 0.f);
  if constexpr (ACC) old = load_pair<VEC>(d + (int64_t)k * P.ldd, c0, P.cols, lane);
  acc = part[(warp * 2 + 1) * 32 + lane];
  for (int w = warp + 1;; ++w) {
    const float2 v = part[w * 2 * 32 + lane];
    acc.x += v.x;
    acc.y += v.y;
    const int after = (w + 1) * per;
    if (after >= P.rows || list[after].x != k) break;
  }
  out(k, acc, old);
}

template <class K, class A>
cudaError_t launch(K kernel, int64_t grid, int block, int smem, const A& args, cudaStream_t st) {
  cudaLaunchConfig_t cfg = pdl_config((int)grid, block, smem, st);
  cudaLaunchAttribute at[1];
  pdl_attr(cfg, at);
  return cudaLaunchKernelEx(&cfg, kernel, args);
}

// Calls f with the types of two matrices and whether all their rows are on 16 bytes.
template <class A, class B, class F>
cudaError_t by_type(const A& a, const B& b, F f) {
  const bool vec = rows_aligned(a) && rows_aligned(b);
  auto second = [&](auto x) {
    using X = decltype(x);
    if (b.bf16) return vec ? f(X(), __nv_bfloat16(), std::true_type()) : f(X(), __nv_bfloat16(), std::false_type());
    return vec ? f(X(), float(), std::true_type()) : f(X(), float(), std::false_type());
  };
  return a.bf16 ? second(__nv_bfloat16()) : second(float());
}

constexpr int64_t kMaxGrid = (int64_t(1) << 31) - 1;

// Allows a kernel its shared memory, once a device.
template <auto Kernel>
cudaError_t opt_in(int device, int smem) {
  static std::atomic<uint64_t> done;
  if (device < 64 && done.load(std::memory_order_acquire) >> device & 1) return cudaSuccess;
  const cudaError_t e = cudaFuncSetAttribute(Kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
  if (e == cudaSuccess && device < 64) done.fetch_or(uint64_t(1) << device, std::memory_order_release);
  return e;
}

}  // namespace

cudaError_t launch_embedding(const ts_ops& h, const EmbedArgs& a, cudaStream_t st) {
  EmbedKernel P = {};
  P.ids = a.ids;
  P.table = a.table.p;
  P.y = a.y.p;
  P.vocab = a.vocab;
  P.ldt = a.table.ld;
  P.ldy = a.y.ld;
  P.cols = a.cols;
  P.scale = a.scale;
  const int groups = (a.cols + kGroupCols - 1) / kGroupCols;
  // four pieces a warp, once that leaves every SM a few warps
  const int pack = a.rows * groups >= (int64_t)h.nsm * 64 && groups >= 4 ? 4 : 1;
  P.packs = (groups + pack - 1) / pack;
  P.units = a.rows * P.packs;
  const int64_t grid = (P.units + kWarps - 1) / kWarps;
  if (grid > kMaxGrid) return cudaErrorInvalidConfiguration;
  return by_type(a.table, a.y, [&](auto t, auto u, auto vec) {
    using T = decltype(t);
    using U = decltype(u);
    constexpr bool V = decltype(vec)::value;
    return launch(pack == 4 ? ts_embed_kernel<T, U, V, 4> : ts_embed_kernel<T, U, V, 1>, grid, kThreads, 0, P, st);
  });
}

// The workspace of a sorted list of `rows` tokens, with the counts of a list
// that more than one block sorts.
namespace {
struct SortPlan {
  int passes, bits, tiles;
  int64_t counts_bytes, present_bytes, bytes;
};
SortPlan sort_plan(int64_t rows, int64_t vocab) {
  SortPlan s = {};
  int key_bits = 1;
  while (key_bits < 32 && (vocab >> key_bits)) ++key_bits;   // (the key of a padded place is `vocab`)
  s.passes = (key_bits + kMaxBits - 1) / kMaxBits;
  s.bits = (key_bits + s.passes - 1) / s.passes;
  const int64_t tile = (rows <= kShortList ? kShortPer : kLongPer) * kSortThreads;
  s.tiles = (int)((rows + tile - 1) / tile);
  const bool alone = rows <= kClusterList;
  s.counts_bytes = alone ? 0 : ((int64_t)s.tiles << s.bits) * 4;
  s.present_bytes = (vocab + 255) / 256 * 256;
  s.bytes = (rows * 8 + 255) / 256 * 256 * (alone ? 1 : 2) + (s.counts_bytes + 255) / 256 * 256 + s.present_bytes;
  return s;
}
template <int PER>
cudaError_t sort_cluster(const ts_ops& h, const SortKernel& S, cudaStream_t st) {
  cudaError_t e = opt_in<ts_sort_cluster_kernel<PER>>(h.device, kClusterSmem<PER>);
  if (e != cudaSuccess) return e;
  cudaLaunchConfig_t cfg = pdl_config(kClusterCtas, kSortThreads, kClusterSmem<PER>, st);
  cudaLaunchAttribute at[2];
  at[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  at[0].val.programmaticStreamSerializationAllowed = 1;
  at[1].id = cudaLaunchAttributeClusterDimension;
  at[1].val.clusterDim.x = kClusterCtas;
  at[1].val.clusterDim.y = at[1].val.clusterDim.z = 1;
  cfg.attrs = at;
  cfg.numAttrs = 2;
  return cudaLaunchKernelEx(&cfg, ts_sort_cluster_kernel<PER>, S);
}
template <int PER>
cudaError_t sort_pass(const ts_ops& h, const SortKernel& S, cudaStream_t st) {
  constexpr int smem = (kSortWarps * kMaxBins + kMaxBins + 32) * 4;
  cudaError_t e = opt_in<ts_sort_pass_kernel<PER>>(h.device, smem);
  if (e == cudaSuccess) e = launch(ts_sort_count_kernel<PER>, S.tiles, kSortThreads, 0, S, st);
  if (e == cudaSuccess) e = launch(ts_sort_pass_kernel<PER>, S.tiles, kSortThreads, smem, S, st);
  return e;
}
}  // namespace

namespace {
cudaError_t launch_few(const ts_ops& h, const EmbedArgs& a, const SortPlan& s, cudaStream_t st) {
  EmbedFewKernel P = {};
  P.ids = a.ids;
  P.dy = a.dy.p;
  P.d = a.d.p;
  P.vocab = a.vocab;
  P.lddy = a.dy.ld;
  P.ldd = a.d.ld;
  P.rows = (int)a.rows;
  P.cols = a.cols;
  P.passes = s.passes;
  P.bits = s.bits;
  P.pieces = a.rows ? (a.cols + kFewCols - 1) / kFewCols : 0;
  P.scale = a.scale;
  // (a block an SM, or several: each sorts first)
  P.fill = (int)std::min<int64_t>(kFillRows, std::max<int64_t>(1, a.vocab / (h.nsm * kSortWarps)));
  const int64_t fill = a.accumulate ? 0 : (a.vocab + kSortWarps * P.fill - 1) / (kSortWarps * P.fill);
  if (P.pieces + fill > kMaxGrid) return cudaErrorInvalidConfiguration;
  if (P.pieces + fill == 0) return cudaSuccess;
  return by_type(a.dy, a.d, [&](auto t, auto u, auto vec) {
    using T = decltype(t);
    using U = decltype(u);
    constexpr bool V = decltype(vec)::value;
    cudaError_t e = a.accumulate ? opt_in<ts_embed_few_kernel<T, U, V, true>>(h.device, kFewSmem)
                                 : opt_in<ts_embed_few_kernel<T, U, V, false>>(h.device, kFewSmem);
    if (e != cudaSuccess) return e;
    return launch(a.accumulate ? ts_embed_few_kernel<T, U, V, true> : ts_embed_few_kernel<T, U, V, false>,
                  P.pieces + fill, kSortThreads, kFewSmem, P, st);
  });
}
}  // namespace

int64_t embedding_backward_workspace(int64_t rows, int64_t vocab) {
  return rows <= kFewTokens ? 0 : sort_plan(rows, vocab).bytes + 512;
}

cudaError_t launch_embedding_backward(const ts_ops& h, const EmbedArgs& a, cudaStream_t st) {
  EmbedBackKernel P = {};
  const SortPlan s = sort_plan(a.rows, a.vocab);
  if (a.rows <= kFewTokens) return launch_few(h, a, s, st);
  const int64_t list = (a.rows * 8 + 255) / 256 * 256;
  uint2* at[2] = {reinterpret_cast<uint2*>(h.ws), reinterpret_cast<uint2*>(h.ws + list)};
  SortKernel S = {};
  S.ids = a.ids;
  S.vocab = a.vocab;
  S.rows = (int)a.rows;
  S.passes = s.passes;
  S.bits = s.bits;
  S.tiles = s.tiles;
  S.out = at[0];
  S.joins = reinterpret_cast<uint32_t*>(h.ws + s.bytes);
  S.present = a.accumulate ? nullptr : h.ws + s.bytes - s.present_bytes;
  cudaError_t e = cudaSuccess;
  if (a.rows <= kClusterList) {
    e = a.rows <= kClusterCtas * kSortThreads ? sort_cluster<1>(h, S, st) : sort_cluster<kClusterPer>(h, S, st);
  } else {
    S.counts = reinterpret_cast<uint32_t*>(h.ws + 2 * list);
    for (int p = 0; p < s.passes && e == cudaSuccess; ++p) {
      const int out = (s.passes - 1 - p) & 1;   // the last pass ends in the first list
      S.out = at[out];
      S.in = p ? at[1 - out] : nullptr;
      S.shift = p * s.bits;
      e = a.rows <= kShortList ? sort_pass<kShortPer>(h, S, st) : sort_pass<kLongPer>(h, S, st);
    }
  }
  if (e != cudaSuccess) return e;
  P.list = at[0];
  P.joins = S.joins;
  P.present = S.present;
  P.dy = a.dy.p;
  P.d = a.d.p;
  P.lddy = a.dy.ld;
  P.ldd = a.d.ld;
  P.vocab = a.vocab;
  P.rows = (int)a.rows;
  P.cols = a.cols;
  P.scale = a.scale;
  P.groups = (a.cols + kGroupCols - 1) / kGroupCols;
  P.part_cols = (int64_t)P.groups * kGroupCols;
  // as many warps as are resident at once (two blocks an SM), or that many several
  // times over, so that no SM idles at the end: 4 to 64 tokens a chunk; fewer,
  // longer ones where the workspace has no room for so many partials
  const int64_t all = a.rows * P.groups, resident = (int64_t)h.nsm * 2 * kWarps;
  const int64_t times = (all + resident * kChunk - 1) / (resident * kChunk);
  const int64_t want = (all + resident * times - 1) / (resident * times);
  const int64_t room = (h.ws_bytes - s.bytes - 512) / (P.part_cols * 8 + 4);
  P.chunk = (int)std::min<int64_t>(kChunk, std::max<int64_t>(4, want));
  if ((a.rows + P.chunk - 1) / P.chunk > std::max<int64_t>(room, 1))
    P.chunk = room < 2 ? (int)a.rows : (int)((a.rows + room - 1) / room);
  P.chunks = (int)((a.rows + P.chunk - 1) / P.chunk);
  P.part = reinterpret_cast<float*>(h.ws + s.bytes + ((int64_t)P.chunks * 4 + 4 + 255) / 256 * 256);
  P.units = (int64_t)P.chunks * P.groups;
  P.unit_blocks = (P.units + kWarps - 1) / kWarps;
  const int64_t fill = a.accumulate ? 0 : (a.vocab + kWarps * kFillRows - 1) / (kWarps * kFillRows);
  if (P.unit_blocks + fill > kMaxGrid) return cudaErrorInvalidConfiguration;
  return by_type(a.dy, a.d, [&](auto t, auto u, auto vec) {
    using T = decltype(t);
    using U = decltype(u);
    constexpr bool V = decltype(vec)::value;
    cudaError_t e = launch(a.accumulate ? ts_embed_sum_kernel<T, U, V, true> : ts_embed_sum_kernel<T, U, V, false>,
                           P.unit_blocks + fill, kThreads, 0, P, st);
    if (e != cudaSuccess || P.chunks < 2) return e;
    return launch(a.accumulate ? ts_embed_join_kernel<U, V, true> : ts_embed_join_kernel<U, V, false>,
                  std::min<int64_t>(4 * h.nsm, (P.chunks * (P.part_cols / kJoinCols) + kWarps - 1) / kWarps), kThreads,
                  0, P, st);
  });
}

}  // namespace fg
