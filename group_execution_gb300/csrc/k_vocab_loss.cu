// Softmax cross entropy of a linear layer over a vocabulary, l = x w^T, and its
// gradients.  The logits [rows, vocab] are never kept; the gradient keeps d, in
// bf16, of as much of the vocabulary as the workspace holds.
//
//   lse_t = log sum_v exp l_tv, loss_t = lse_t - l_t,target
//   d_tv = (g_t + h_t) exp(l_tv - lse_t) - g_t [v = target_t]
//   dx = d w, dw = d^T x
//
// Everything large is a product on the 5th-generation tensor cores.  Forward:
// one product whose epilogue reduces each row of a tile's 128 columns to a
// maximum and a sum of exponentials (8 bytes for 128 logits), which a small
// kernel joins (k_vocab_few.cu has few rows of small weights).  Backward, for each
// piece of the vocabulary: the logits again, turned by the epilogue into d,
// rounded to bf16 (the tensor cores' operand) in the workspace; then, in one
// launch, the piece's dw and its part of dx, which float32 sums in the workspace
// collect (one piece that is not cut is dx itself).
//
// The product kernel is persistent: CTA pairs walk 256 x 256 tiles (2-SM
// tcgen05.mma, cta_group::2), K 128 at a time; each CTA stages half of the
// tile's rows of A and half of its columns of B in a ring of shared-memory
// slots (128-byte swizzled TMA boxes of 64 x 128 elements, whichever way the
// operand lies; fewer rows and more slots where there are not 128).  Warps, in
// each CTA:
//   warp 0      TMA producer of the A half,
//   warp 1      allocates TMEM (two accumulators) and, in the even CTA, issues
//               the MMAs from one thread,
//   warp 2      TMA producer of the B half,
//   warp 3      copies x for dw beside the first piece's logits, where that hides it,
//   warps 4-11  epilogue: a thread owns half of one row of the CTA's 128 x 256
//               accumulator; it overlaps the next tile's MMAs.
// At 4096 x 1024 x 50001 the tensor pipe is active in 96 % of the cycles of the
// loss (213 us, 1.97 PFLOP/s in a single run; 245 to 253 in a series of calls, at the
// power limit), 83 % of the gradient's logits, 91 % of dx and dw (790 us together).
// 8192 x 4096 x 50001 takes 1850 to 1905 and 5900 to 6005 us, 1.76 to 1.81 and 1.68
// to 1.71 PFLOP/s, d of the whole vocabulary (822 MB) in the workspace.  Few rows are
// bound by the weight's bytes: 64 x 4096 x 32000 50 us forward (5.3 TB/s), 161
// backward.  Models of 256 columns or fewer are bound by the epilogue.
//
// Every wait is bounded; on expiry the CTA records the error, the pair waits
// for the copies that either CTA has in flight, frees its TMEM and returns.
#include <cuda.h>

#include <algorithm>
#include <atomic>
#include <mutex>

#include "launch.h"
#include "ts_device.cuh"
#include "vocab.cuh"

namespace fg {
namespace {

constexpr int kTile = 256;                       // rows and columns of a pair's tile
constexpr int kHalf = kTile / 2;                 // ... and one CTA stages of each operand
constexpr int kKB = 128;                         // of K in a ring slot
constexpr int kRowBytes = 64 * 2;                // a TMA box is 64 columns wide
constexpr int kRingBytes = 192 << 10;
constexpr int kMaxSlots = 8;                     // (three of 128 rows of each operand)
constexpr int kStageBytes = 32 * 128;            // an epilogue warp's rows on their way out
constexpr int kThreads = 12 * 32;
constexpr int kSmem = kRingBytes + 8 * kStageBytes + 1024;

enum Mode { kLoss, kDlogits, kGrad };

// Where a gradient goes.
struct Out {
  CUtensorMap map;   // [depth, rows, cols]
  void* p;
  int64_t ld;
  int bf16, tma;     // by TMA, or by threads
  int whole;         // rows end on 16 bytes, the unit that TMA writes
  int add;           // to what it holds
};

struct VocabKernel {
  CUtensorMap x, w, d;       // loads: x [rows, cols], w's piece [vocab, cols], d [rows, dpitch]
  CUtensorMap store_d;       // d, in boxes of 64 x 32
  Out out[2];                // dx (its sums [splits, rows, cols] float32, or itself), dw's piece
  CopyRows copy;             // x for dw, copied beside the first piece's logits
  int rows, cols, vocab;     // vocab: of the piece
  int v0;                    // its first row of w
  int64_t total;             // the whole vocabulary's size
  int tile_n;                // columns of a tile of the logits
  int box_rows;              // rows of x's and d's boxes: 128, or as many 16s as there are rows
  int slots, slot_bytes;     // of the ring
  int tiles_t, tiles_v, tiles_c;
  // forward
  float2* part;              // [column parts][rows]: largest logit, and the sum of exp(l - it)
  float* tlogit;             // the target's logit
  const int64_t* targets;
  // backward
  const float* lse;
  const float* g_loss;
  const float* g_lse;
  int splits;                // of dx's K
  int nx, nw;                // dx and dw items
  int dw_first, late, extra; // which are longer, and how the others follow; see item_of
  int32_t* err;
  int64_t wait_limit_ns;
  int inject;
};

// The tensor core truncates as it adds, so that a float32 accumulator's error
// grows with its products, to one side: 2e-6 of 4096, 1.4e-3 of 524288 of one
// sign.  So a sum runs over a chain of at most 8 blocks of K for the logits (5e-7)
// and 16 for the gradients, which sum over all rows or the whole vocabulary (of
// operands in bf16); the epilogue's threads add what the chains came to in
// registers, during the next one's MMAs.  The loss and the gradient cut alike, so
// that their logits are the same to the bit: a confident row's exp(l - lse) - 1 is
// as small as it should be, whatever the sums have lost.  (Where all items are a
// chain at most, the gradient's kernels do without the registers that several
// take: 16 x 1024 x 4000 16.8 us, with them 17.9.)
constexpr int kLossChain = 8, kGradChain = 16;
template <int MODE, bool CHAINS>
__device__ __forceinline__ int chain_end(int kb0, int kb1) {
  constexpr int kChain = MODE == kGrad ? kGradChain : kLossChain;
  return CHAINS && kb1 - kb0 > kChain ? kb0 + kChain : kb1;
}

// What a pair works on: a tile at (m0, n0) of a product, over blocks [kb0, kb1)
// of kKB.
struct Item {
  int kind;   // 0 logits, 1 dx, 2 dw, -1 none
  int m0, n0, kb0, kb1, K, split;
};

constexpr int kRowGroup = 16;   // row tiles that walk the vocabulary together (their rows of x stay in L2)

template <int MODE>
__device__ __forceinline__ Item item_of(const VocabKernel& P, int pair, int npair, int k) {
  Item w = {};
  if constexpr (MODE != kGrad) {
    const int64_t x = pair + (int64_t)k * npair;
    if (x >= (int64_t)P.tiles_t * P.tiles_v) return Item{-1};
    const int per = kRowGroup * P.tiles_v, g = (int)(x / per), r = (int)(x - (int64_t)g * per);
    const int gm = min(kRowGroup, P.tiles_t - g * kRowGroup);
    w.m0 = (g * kRowGroup + r % gm) * kTile;
    w.n0 = r / gm * P.tile_n;
    w.K = P.cols;
    w.kb1 = (P.cols + kKB - 1) / kKB;
    return w;
  } else {
    // the longer kind's items first, one after the other over all pairs; where
    // their last round leaves pairs free, those take `extra` items of the other
    // kind before the rest join them
    const int n1 = P.dw_first ? P.nw : P.nx, n2 = P.dw_first ? P.nx : P.nw;
    const int mine = pair < n1 ? (n1 - pair + npair - 1) / npair : 0;
    const bool second = k >= mine;
    int x = pair + k * npair;
    if (second) {
      const int j = k - mine, early = npair - P.late;
      if (pair >= P.late && j < P.extra) x = pair - P.late + j * early;
      else x = P.extra * early + pair + (pair >= P.late ? j - P.extra : j) * npair;
      if (x >= n2) return Item{-1};
    }
    if (second == (P.dw_first != 0)) {
      const int per = P.tiles_t * P.tiles_c, r = x % per;
      w.kind = 1;
      w.split = x / per;
      w.m0 = r / P.tiles_c * kTile;
      w.n0 = r % P.tiles_c * kTile;
      const int nkb = (P.vocab + kKB - 1) / kKB;
      w.kb0 = (int)((int64_t)nkb * w.split / P.splits);
      w.kb1 = (int)((int64_t)nkb * (w.split + 1) / P.splits);
      w.K = P.vocab;
      return w;
    }
    w.kind = 2;
    w.m0 = x / P.tiles_c * kTile;
    w.n0 = x % P.tiles_c * kTile;
    w.kb1 = (P.rows + kKB - 1) / kKB;
    w.K = P.rows;
    return w;
  }
}

__device__ __forceinline__ bool wait_bar(uint32_t bar, uint32_t parity, int64_t limit, volatile int* abort_flag) {
  if (mbar_try_wait(bar, parity)) return true;
  const uint64_t t0 = global_ns();
  while (!mbar_try_wait(bar, parity))
    if (*abort_flag || (int64_t)(global_ns() - t0) > limit) return false;
  return true;
}
__device__ __forceinline__ void st_cluster(uint32_t addr, int v) {
  asm volatile("st.shared::cluster.u32 [%0], %1;" ::"r"(addr), "r"(v) : "memory");
}
// 16 consecutive f32 columns of this warp's 32 lanes of tensor memory.
__device__ __forceinline__ void tmem_ld16(uint32_t taddr, float (&v)[16]) {
  uint32_t r[16];
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x16.b32 {%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15}, "
      "[%16];"
      : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]), "=r"(r[8]),
        "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15])
      : "r"(taddr));
  asm volatile("tcgen05.wait::ld.sync.aligned;" ::: "memory");
#pragma unroll
  for (int i = 0; i < 16; ++i) v[i] = __uint_as_float(r[i]);
}
__device__ __forceinline__ void tma_store_3d(const CUtensorMap* m, int x, int y, int z, uint32_t src) {
  asm volatile("cp.async.bulk.tensor.3d.global.shared::cta.tile.bulk_group [%0, {%1, %2, %3}], [%4];" ::"l"(
                   reinterpret_cast<uint64_t>(m)),
               "r"(x), "r"(y), "r"(z), "r"(src)
               : "memory");
}
__device__ __forceinline__ void tma_add_3d(const CUtensorMap* m, int x, int y, int z, uint32_t src) {
  asm volatile("cp.reduce.async.bulk.tensor.3d.global.shared::cta.add.tile.bulk_group [%0, {%1, %2, %3}], [%4];" ::"l"(
                   reinterpret_cast<uint64_t>(m)),
               "r"(x), "r"(y), "r"(z), "r"(src)
               : "memory");
}
// An epilogue warp's 32 rows x 128 bytes on their way out, 128-byte swizzled.
struct Stage {
  uint8_t* p;
  __device__ __forceinline__ void put(int row, int chunk, uint4 v) const {
    *reinterpret_cast<uint4*>(p + row * 128 + ((chunk ^ (row & 7)) << 4)) = v;
  }
  // Column `col` (float32) of a row.
  __device__ __forceinline__ float get(int row, int col) const {
    return *reinterpret_cast<const float*>(p + row * 128 + (((col >> 2) ^ (row & 7)) << 4) + (col & 3) * 4);
  }
  // 32 float32 columns
  __device__ __forceinline__ void put_f32(int row, const float (&v)[32]) const {
#pragma unroll
    for (int c = 0; c < 8; ++c)
      put(row, c, make_uint4(__float_as_uint(v[4 * c]), __float_as_uint(v[4 * c + 1]), __float_as_uint(v[4 * c + 2]),
                             __float_as_uint(v[4 * c + 3])));
  }
  // 32 columns in bf16, the first or second half of the 128 bytes; signs flipped
  // and values masked as asked
  __device__ __forceinline__ void put_bf16(int row, int half, const float (&v)[32], uint32_t flip = 0,
                                           uint32_t keep = 0xffffffffu) const {
#pragma unroll
    for (int c = 0; c < 4; ++c) {
      uint32_t u[4];
#pragma unroll
      for (int i = 0; i < 4; ++i) u[i] = (bf16x2(v[8 * c + 2 * i], v[8 * c + 2 * i + 1]) ^ flip) & keep;
      put(row, half * 4 + c, make_uint4(u[0], u[1], u[2], u[3]));
    }
  }
};

// A lane's column of the stage's first n rows, to rows `ld` apart.  float32 rows are
// added to in memory, as TMA does it; bf16 ones are read, four at a time.
__device__ __forceinline__ void to_rows(const Stage& stage, float* d, int64_t ld, int n, bool add) {
  const int lane = threadIdx.x & 31;
#pragma unroll 1
  for (int r = 0; r < 32; r += 4, d += 4 * ld) {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      if (r + i >= n) break;
      if (add) atomicAdd(d + i * ld, stage.get(r + i, lane));
      else d[i * ld] = stage.get(r + i, lane);
    }
  }
}
__device__ __forceinline__ void to_rows(const Stage& stage, __nv_bfloat16* d, int64_t ld, int n, bool add) {
  const int lane = threadIdx.x & 31;
#pragma unroll 1
  for (int r = 0; r < 32; r += 4, d += 4 * ld) {
    float old[4] = {};
    if (add) {
#pragma unroll
      for (int i = 0; i < 4; ++i)
        if (r + i < n) old[i] = to_f32(d[i * ld]);
    }
#pragma unroll
    for (int i = 0; i < 4; ++i)
      if (r + i < n) d[i * ld] = from_f32<__nv_bfloat16>(old[i] + stage.get(r + i, lane));
  }
}

// CHAINS: items may take more than one chain.
template <int MODE, bool CHAINS>
__global__ void __cluster_dims__(2, 1, 1) __launch_bounds__(kThreads, 1)
    ts_vocab_kernel(const __grid_constant__ VocabKernel P) {
  extern __shared__ uint8_t smem_raw[];
  __shared__ __align__(8) uint64_t bar_mem[2 * kMaxSlots + 5];
  __shared__ int abort_flag, issued[2];         // slots that either producer has issued copies for
  __shared__ int peer_gave_up, peer_issued;     // written by the pair's other CTA
  __shared__ uint32_t tmem_slot;
  uint8_t* ring = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  const uint32_t full0 = smem_u32(bar_mem), empty0 = full0 + 8 * kMaxSlots, tfull0 = empty0 + 8 * kMaxSlots,
                 tempty0 = tfull0 + 16, done_bar = tempty0 + 16;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int h = (int)cluster_ctarank();
  const bool leader = h == 0;
  const uint16_t pair_mask = 3u;
  const int npair = gridDim.x / 2, pair = blockIdx.x / 2;
  const int half_n = MODE == kGrad ? kHalf : P.tile_n / 2;   // columns of B that a CTA stages, and of an epilogue set
  if (threadIdx.x == 0) {
    abort_flag = issued[0] = issued[1] = 0;
    for (int s = 0; s < P.slots; ++s) {
      mbar_init(full0 + 8 * s, 1);   // the even CTA's expect_tx
      mbar_init(empty0 + 8 * s, 1);
    }
    for (int b = 0; b < 2; ++b) {
      mbar_init(tfull0 + 8 * b, 1);
      mbar_init(tempty0 + 8 * b, 16);   // the epilogue warps of the pair
    }
    mbar_init(done_bar, 1);
    fence_mbar_init();
  }
  if (warp == 1) tmem_alloc<2>(smem_u32(&tmem_slot), 512);
  tc_fence_before();
  __syncthreads();
  cluster_sync();   // the peer's barriers are initialised before any remote arrival
  tc_fence_after();
  const uint32_t tmem = tmem_slot;
  pdl_launch_dependents();
  pdl_wait();

  if (warp == 0 || warp == 2) {
    // ---- operand producers ----
    if (lane == 0 && !P.inject) {
      const bool isA = warp == 0;
      const uint64_t keep = l2_evict_last();
      const uint32_t cbar0 = cluster_addr(full0, 0), dst0 = smem_u32(ring) + (isA ? 0 : 2 * P.box_rows * kRowBytes);
      int it = 0, s = 0;
      uint32_t ph = 0;
      bool ok = true;
      for (int k = 0; ok; ++k) {
        const Item w = item_of<MODE>(P, pair, npair, k);
        if (w.kind < 0) break;
        // an operand lies K-major (columns are K) or MN-major (rows are K)
        const CUtensorMap* map;
        bool mn;
        if constexpr (MODE == kGrad) {
          map = isA ? &P.d : w.kind == 1 ? &P.w : &P.x;
          mn = !isA || w.kind == 2;
        } else {
          map = isA ? &P.x : &P.w;
          mn = false;
        }
        const int o = isA ? w.m0 + h * kHalf : w.n0 + h * half_n;
        // two boxes of each operand; B's rows are columns of the logits, or of K
        const int b_rows = MODE != kGrad ? half_n : w.kind == 1 ? kHalf : P.box_rows;
        const uint32_t box_bytes = (isA ? P.box_rows : b_rows) * kRowBytes;
        for (int kb = w.kb0; kb < w.kb1; ++kb) {
          if (it >= P.slots && !wait_bar(empty0 + 8 * s, ph ^ 1, P.wait_limit_ns, &abort_flag)) {
            ok = false;
            break;
          }
          if (leader && isA) mbar_expect_tx(full0 + 8 * s, 4 * (P.box_rows + b_rows) * kRowBytes);
          const uint32_t dst = dst0 + s * P.slot_bytes, cbar = cbar0 + 8 * s;
          tma_load_2d_pair(dst, map, mn ? o : kb * kKB, mn ? kb * kKB : o, cbar, keep);
          tma_load_2d_pair(dst + box_bytes, map, (mn ? o : kb * kKB) + 64, mn ? kb * kKB : o, cbar, keep);
          ++it;
          if (++s == P.slots) {
            s = 0;
            ph ^= 1;
          }
        }
      }
      issued[isA ? 0 : 1] = it;
      if (!ok) {
        abort_flag = 1;
        set_error(P.err, DEVERR_TIMEOUT);
      }
    }
  } else if (warp == 1) {
    // ---- MMA issuer ----
    if (lane == 0 && leader) {
      const uint32_t base = smem_u32(ring);
      int s = 0, i = 0;
      uint32_t ph = 0;
      bool ok = true;
      for (int k = 0; ok; ++k) {
        const Item w = item_of<MODE>(P, pair, npair, k);
        if (w.kind < 0) break;
        // MN-major: atoms of 64 columns x 8 of K, the second 64 columns one box
        // on, 16 of K 2 KB on.  K-major: atoms of 8 rows x 64 of K, 16 of K 32
        // bytes on, the second 64 of K one box on.
        const bool a_mn = MODE == kGrad && w.kind == 2, b_mn = MODE == kGrad;
        const uint32_t idesc = idesc_bf16_f32(kTile, 2 * half_n, a_mn, b_mn);
        const uint32_t a_box = P.box_rows * kRowBytes,
                       b_box = (MODE != kGrad ? half_n : w.kind == 1 ? kHalf : P.box_rows) * kRowBytes;
        const uint64_t ad0 = smem_desc_sw128(base, a_mn ? a_box : 16, 1024),
                       bd0 = smem_desc_sw128(base + 2 * a_box, b_mn ? b_box : 16, 1024);
        const uint32_t a_step = (a_mn ? 2048 : 32) >> 4, b_step = (b_mn ? 2048 : 32) >> 4;
        const uint32_t a_half = (a_mn ? 4 * 2048 : a_box) >> 4, b_half = (b_mn ? 4 * 2048 : b_box) >> 4;
        int s0 = w.kb0;
        do {
          const int s1 = chain_end<MODE, CHAINS>(s0, w.kb1), b = i & 1;
          if (i >= 2 && !wait_bar(tempty0 + 8 * b, ((i >> 1) & 1) ^ 1, P.wait_limit_ns, &abort_flag)) {
            ok = false;
            break;
          }
          tc_fence_after();
          for (int kb = s0; kb < s1; ++kb) {
            if (!wait_bar(full0 + 8 * s, ph, P.wait_limit_ns, &abort_flag)) {
              ok = false;
              break;
            }
            tc_fence_after();
            const uint32_t so = (uint32_t)(s * P.slot_bytes) >> 4;
            const int left = w.K - kb * kKB;   // (past K both operands are zeros)
#pragma unroll
            for (int kk = 0; kk < kKB / 16; ++kk) {
              if (kk * 16 >= left) break;
              tc_mma_bf16<2>(tmem + b * kTile, ad0 + so + (kk >> 2) * a_half + (kk & 3) * a_step,
                             bd0 + so + (kk >> 2) * b_half + (kk & 3) * b_step, idesc, kb != s0 || kk != 0);
            }
            tc_commit_mask(empty0 + 8 * s, pair_mask);
            if (++s == P.slots) {
              s = 0;
              ph ^= 1;
            }
          }
          if (ok) tc_commit_mask(tfull0 + 8 * b, pair_mask);
          s0 = s1;
          ++i;
        } while (ok && s0 < w.kb1);
      }
      if (!ok) {
        abort_flag = 1;
        set_error(P.err, DEVERR_TIMEOUT);
      }
      // every MMA issued has completed before either CTA may free TMEM
      tc_commit_mask(done_bar, pair_mask);
      mbar_wait(done_bar, 0, kDrainLimitNs);
    }
  } else if (warp == 3) {
    if constexpr (MODE == kDlogits) {
      // ---- x for dw: rows that take no gradient as zeros ----
      copy_rows<4>(P.copy, blockIdx.x * 32 + lane, gridDim.x * 32);
    }
  } else if (warp >= 4) {
    // ---- epilogue ----
    const int q = warp & 3, set = (warp - 4) >> 2;   // the TMEM lane quarter this warp may access, its column half
    const Stage stage = {ring + kRingBytes + (warp - 4) * kStageBytes};
    const uint32_t stage_u32 = smem_u32(stage.p);
    bool ok = true;
    int i = 0;   // accumulators so far
    for (int k = 0; ok; ++k) {
      const Item w = item_of<MODE>(P, pair, npair, k);
      if (w.kind < 0) break;
      const int r0 = w.m0 + h * kHalf + q * 32, row = r0 + lane;
      const int c0 = w.n0 + set * half_n;   // this warp's first column
      // d is |coef| p - (its sign) g at the target, as bf16 with coef's sign, or
      // masked out; |coef| goes into the exponent
      float lse = 0.f, shift = 0.f, g = 0.f;
      uint32_t sign = 0, keep = 0;
      int target = -1;   // the target's column of the piece
      if constexpr (MODE != kGrad) {
        if (row < P.rows) {
          const int64_t t = P.targets ? P.targets[row] : -1;
          target = t >= P.v0 && t < (int64_t)P.v0 + P.vocab ? (int)(t - P.v0) : -1;
          if constexpr (MODE == kDlogits) {
            // (a row of -inf logits takes no gradient)
            const float l = P.lse[row];
            if (l != -INFINITY) {
              g = t >= 0 && t < P.total ? P.g_loss[row] : 0.f;
              const float coef = g + (P.g_lse ? P.g_lse[row] : 0.f);
              lse = l;   // (taken off before the change of base: in log2 a finite one may overflow)
              shift = log2f(fabsf(coef));
              if (coef < 0.f) {
                sign = 0x80008000u;
                g = -g;
              }
              // rows without a gradient have zeros whatever their logits
              keep = coef == 0.f && g == 0.f ? 0 : 0xffffffffu;
            }
          }
        }
      }
      uint32_t acc = 0;
      auto next_acc = [&]() {
        const int b = i & 1;
        ok = __all_sync(0xffffffffu, wait_bar(tfull0 + 8 * b, (i >> 1) & 1, P.wait_limit_ns, &abort_flag));
        tc_fence_after();
        acc = tmem + ((uint32_t)(q * 32) << 16) + b * kTile + set * half_n;
        return ok;
      };
      auto release = [&]() {
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive_cluster(cluster_addr(tempty0 + 8 * (i & 1), 0));
        ++i;
      };
      // a thread's half row, the chains added up
      auto collect = [&](float (&v)[4][32]) {
        int s0 = w.kb0;
        do {
          if (!next_acc()) return;
          if (s0 == w.kb0) {
#pragma unroll
            for (int j = 0; j < 4; ++j) tmem_ld32(acc + 32 * j, v[j]);
          } else {
#pragma unroll
            for (int j = 0; j < 8; ++j) {
              float o[16];
              tmem_ld16(acc + 16 * j, o);
#pragma unroll
              for (int c = 0; c < 16; ++c) v[j / 2][j % 2 * 16 + c] += o[c];
            }
          }
          release();
          s0 = chain_end<MODE, CHAINS>(s0, w.kb1);
        } while (s0 < w.kb1);
      };
      // before the stage is written again, its last store has read it
      auto stage_free = [&]() {
        if (lane == 0) bulk_wait_read<0>();
        __syncwarp();
      };
      auto stage_full = [&]() {
        fence_proxy_async_smem();
        __syncwarp();
      };
      if constexpr (MODE == kLoss) {
        float v[4][32];
        collect(v);
        if (!ok) break;
        // the sum's reference is the largest logit itself: its term is exactly 1, and
        // no finite logit overflows, as one in log2 would
        const int left = min(half_n, P.vocab - c0), at = target - c0;
        if (left < kHalf) {
#pragma unroll
          for (int j = 0; j < 4; ++j)
#pragma unroll
            for (int c = 0; c < 32; ++c)
              if (32 * j + c >= left) v[j][c] = -INFINITY;
        }
        if (at >= 0 && at < left) {
          float l = 0.f;
#pragma unroll
          for (int j = 0; j < 4; ++j)
#pragma unroll
            for (int c = 0; c < 32; ++c) l = 32 * j + c == at ? v[j][c] : l;
          P.tlogit[row] = l;
        }
        float top[4] = {-INFINITY, -INFINITY, -INFINITY, -INFINITY};
        F2 sum[2] = {};
#pragma unroll
        for (int j = 0; j < 4; ++j)
#pragma unroll
          for (int c = 0; c < 32; ++c) top[c & 3] = fmaxf(top[c & 3], v[j][c]);
        const float m = fmaxf(fmaxf(top[0], top[1]), fmaxf(top[2], top[3]));
        const float ref = m == -INFINITY ? 0.f : m;
#pragma unroll
        for (int j = 0; j < 4; ++j)
#pragma unroll
          for (int c = 0; c < 32; c += 2) {
            const F2 e = mul2(add2(pack2f(v[j][c], v[j][c + 1]), pack2f(-ref, -ref)), pack2f(kLog2e, kLog2e));
            float a, b;
            unpack2f(e, a, b);
            sum[c / 2 & 1] = add2(sum[c / 2 & 1], pack2f(exp2_approx(a), exp2_approx(b)));
          }
        if (row < P.rows)
          P.part[(int64_t)(c0 / half_n) * P.rows + row] = make_float2(m, sum2(sum[0]) + sum2(sum[1]));
      } else if constexpr (MODE == kDlogits) {
        // 32 columns, from j on, into the stage; 64 of it leave
        auto turn = [&](float (&u)[32], int j) {
          const int cc = c0 + j, left = P.vocab - cc, at = target - cc;
#pragma unroll
          for (int c = 0; c < 32; c += 2) {
            const F2 e = fma2(add2(pack2f(u[c], u[c + 1]), pack2f(-lse, -lse)), pack2f(kLog2e, kLog2e),
                              pack2f(shift, shift));
            float a, b;
            unpack2f(e, a, b);
            u[c] = exp2_approx(a);
            u[c + 1] = exp2_approx(b);
          }
          if (at >= 0 && at < 32) {
#pragma unroll
            for (int c = 0; c < 32; ++c) u[c] -= c == at ? g : 0.f;
          }
          if (left < 32) {
#pragma unroll
            for (int c = 0; c < 32; ++c)
              if (c >= left) u[c] = 0.f;
          }
          if (j % 64 == 0) stage_free();
          stage.put_bf16(lane, j / 32 & 1, u, sign, keep);
        };
        auto send = [&](int j) {
          stage_full();
          if (lane == 0) {
            if (r0 < P.rows) tma_store_2d(&P.store_d, c0 + j, r0, stage_u32);
            bulk_commit();
          }
        };
        if constexpr (CHAINS) {
          float v[4][32];
          collect(v);
          if (!ok) break;
          turn(v[0], 0);
          turn(v[1], 32);
          send(0);
          if (half_n > 64) {
            turn(v[2], 64);
            turn(v[3], 96);
            send(64);
          }
        } else {
          if (!next_acc()) break;
#pragma unroll 1
          for (int j = 0; j < half_n; j += 64) {
#pragma unroll
            for (int k = 0; k < 2; ++k) {
              float u[32];
              tmem_ld32(acc + j + 32 * k, u);
              if (j + 64 == half_n && k == 1) release();
              turn(u, j + 32 * k);
            }
            send(j);
          }
        }
      } else {
        const Out& out = P.out[w.kind - 1];
        const int m_end = w.kind == 1 ? P.rows : P.vocab;
        // 32 columns as float32 in the stage, to rows that TMA cannot write or that
        // bf16 values are added to
        auto by_threads = [&](int j) {
          __syncwarp();
          const int col = c0 + j + lane, n = col < P.cols ? min(32, m_end - r0) : 0;
          const int64_t at = (int64_t)r0 * out.ld + col;
          if (out.bf16) to_rows(stage, static_cast<__nv_bfloat16*>(out.p) + at, out.ld, n, out.add);
          else to_rows(stage, static_cast<float*>(out.p) + at, out.ld, n, out.add);
          __syncwarp();
        };
        float v[CHAINS ? 4 : 1][32];
        bool one = true;
        if constexpr (CHAINS) {
          one = chain_end<MODE, CHAINS>(w.kb0, w.kb1) == w.kb1;
          if (!one) collect(v);
        }
        if (one) next_acc();
        if (!ok) break;
#pragma unroll (CHAINS ? 2 : 1)
        for (int j = 0; j < kHalf; j += 64) {
          const bool tma = out.tma && (out.whole || c0 + j + 64 <= P.cols);
          const bool both = tma && out.bf16;   // both 32 columns in one store
#pragma unroll
          for (int k = 0; k < 2; ++k) {
            float (&u)[32] = v[CHAINS ? j / 32 + k : 0];
            if (one) {
              tmem_ld32(acc + j + 32 * k, u);
              if (j + 64 == kHalf && k == 1) release();
            }
            if (!both || k == 0) stage_free();
            if (w.kb0 == w.kb1) {   // (a piece of fewer blocks than dx is cut in)
#pragma unroll
              for (int c = 0; c < 32; ++c) u[c] = 0.f;
            }
            if (both) {
              stage.put_bf16(lane, k, u);
              if (k == 0) continue;
            } else {
              stage.put_f32(lane, u);
              if (!tma) {
                by_threads(j + 32 * k);
                continue;
              }
            }
            stage_full();
            const int col = c0 + j + (both ? 0 : 32 * k);
            if (lane == 0) {
              if (r0 < m_end && col < P.cols) {
                if (out.add) tma_add_3d(&out.map, col, r0, w.split, stage_u32);
                else tma_store_3d(&out.map, col, r0, w.split, stage_u32);
              }
              bulk_commit();
            }
          }
        }
      }
    }
    if (!ok && lane == 0) {
      abort_flag = 1;
      set_error(P.err, DEVERR_TIMEOUT);
    }
    if (lane == 0) bulk_wait<0>();   // the stores issued here have completed
  }
  tc_fence_before();
  __syncthreads();
  const int mine = issued[0] > issued[1] ? issued[0] : issued[1];
  if (threadIdx.x == 0) {
    st_cluster(cluster_addr(smem_u32(&peer_gave_up), h ^ 1), abort_flag);
    st_cluster(cluster_addr(smem_u32(&peer_issued), h ^ 1), mine);
  }
  __syncwarp();
  // no CTA leaves while its peer may still write to its shared memory or
  // issue MMAs into its TMEM
  cluster_sync();
  if (abort_flag || peer_gave_up) {   // (the same in both CTAs)
    // either CTA's copies in flight complete on the even CTA's barriers; the
    // slots they fill may lack copies, so each wait may run to its limit
    if (leader && threadIdx.x == 0) {
      const int last = mine > peer_issued ? mine : peer_issued;
      for (int k = last - P.slots < 0 ? 0 : last - P.slots; k < last; ++k)
        mbar_wait(full0 + 8 * (k % P.slots), (k / P.slots) & 1, kDrainLimitNs);
    }
    __syncwarp();
    cluster_sync();
  }
  tc_fence_after();
  if (warp == 1) tmem_dealloc<2>(tmem, 512);
}

// ---- small kernels ------------------------------------------------------------------

struct JoinKernel {
  const float2* part;
  const float* tlogit;
  const int64_t* targets;
  float* loss;
  float* lse;
  int64_t vocab;
  int rows, parts;
};

// The parts of 32 rows: lane = row, the block's warps share the parts.  (With 8
// warps a block 16 rows of 250 parts took 9 us, a chain of loads.)
constexpr int kJoinWarps = 32;

__global__ void __launch_bounds__(kJoinWarps * 32) ts_loss_join_kernel(const __grid_constant__ JoinKernel P) {
  __shared__ float2 sm[kJoinWarps][33];
  pdl_launch_dependents();
  pdl_wait();
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  int row = blockIdx.x * 32 + lane;
  float m = -INFINITY, s = 0.f;
  auto add = [&](float2 v) { join_sums(m, s, v.x, v.y); };
  if (row < P.rows) {
    const float2* p = P.part + row;
    for (int k0 = warp; k0 < P.parts; k0 += 8 * kJoinWarps) {
      float2 v[8];
#pragma unroll
      for (int k = 0; k < 8; ++k) {
        const int at = k0 + k * kJoinWarps;
        v[k] = at < P.parts ? p[(int64_t)at * P.rows] : make_float2(-INFINITY, 0.f);
      }
#pragma unroll
      for (int k = 0; k < 8; ++k) add(v[k]);
    }
  }
  sm[lane][warp] = make_float2(m, s);
  __syncthreads();
  // warp w now joins row w's sums, one a lane
  row = blockIdx.x * 32 + warp;
  const float2 v = sm[warp][lane];
  m = v.x;
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, o));
  const float ref = m == -INFINITY ? 0.f : m;
  s = warp_sum(v.y * exp2_approx((v.x - ref) * kLog2e));
  if (lane || row >= P.rows) return;
  if (P.lse) P.lse[row] = lse_of(m, s);
  if (P.loss) {
    const int64_t t = P.targets[row];
    P.loss[row] = t < 0 || t >= P.vocab ? 0.f : loss_of(m, s, P.tlogit[row]);
  }
}

__global__ void __launch_bounds__(256) ts_loss_copy_kernel(const __grid_constant__ CopyRows C) {
  pdl_launch_dependents();
  pdl_wait();
  copy_rows<2>(C, (int64_t)blockIdx.x * 256 + threadIdx.x, (int64_t)gridDim.x * 256);
}

struct DxKernel {
  const float* sums;   // [splits][rows][pitch]
  void* dx;
  int64_t pitch, rows, ld, units;
  int cols, groups, splits;
};

template <class T, bool VEC>
__global__ void __launch_bounds__(256) ts_loss_dx_kernel(const __grid_constant__ DxKernel P) {
  pdl_launch_dependents();
  pdl_wait();
  const int lane = threadIdx.x & 31;
  const int64_t u = (int64_t)blockIdx.x * 8 + (threadIdx.x >> 5);
  if (u >= P.units) return;
  const int64_t r = u / P.groups;
  const int c0 = (int)(u - r * P.groups) * kGroupCols;
  float v[8];
  load_group<VEC>(P.sums + r * P.pitch, c0, P.cols, lane, v);
  for (int s = 1; s < P.splits; s += 4) {
    float x[4][8];
#pragma unroll
    for (int k = 0; k < 4; ++k)
      if (s + k < P.splits) load_group<VEC>(P.sums + ((int64_t)(s + k) * P.rows + r) * P.pitch, c0, P.cols, lane, x[k]);
#pragma unroll
    for (int k = 0; k < 4; ++k)
      if (s + k < P.splits) {
#pragma unroll
        for (int j = 0; j < 8; ++j) v[j] += x[k][j];
      }
  }
  store_group<VEC>(static_cast<T*>(P.dx) + r * P.ld, c0, P.cols, lane, v);
}

// dw of no rows
template <class T>
__global__ void __launch_bounds__(256) ts_loss_zero_kernel(T* dw, int64_t lddw, int vocab, int cols) {
  pdl_launch_dependents();
  pdl_wait();
  for (int64_t v = blockIdx.x; v < vocab; v += gridDim.x)
    for (int c = threadIdx.x; c < cols; c += 256) dw[v * lddw + c] = from_f32<T>(0.f);
}

// ---- host ----------------------------------------------------------------------------

using EncodeFn = CUresult (*)(CUtensorMap*, CUtensorMapDataType, cuuint32_t, void*, const cuuint64_t*,
                              const cuuint64_t*, const cuuint32_t*, const cuuint32_t*, CUtensorMapInterleave,
                              CUtensorMapSwizzle, CUtensorMapL2promotion, CUtensorMapFloatOOBfill);
EncodeFn encoder() {
  static EncodeFn fn = nullptr;
  static std::once_flag once;
  std::call_once(once, [] {
    void* p = nullptr;
    cudaDriverEntryPointQueryResult q;
    if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &p, 12000, cudaEnableDefault, &q) == cudaSuccess &&
        q == cudaDriverEntryPointSuccess)
      fn = reinterpret_cast<EncodeFn>(p);
  });
  return fn;
}

// A map of a matrix, or (rank 3) of `depth` dense ones, with boxes of box_cols x
// box_rows.
cudaError_t make_map(CUtensorMap* m, const void* p, int bf16, int64_t cols, int64_t rows, int64_t ld, int box_cols,
                     int box_rows, int rank = 2, int64_t depth = 1) {
  EncodeFn enc = encoder();
  if (!enc) return cudaErrorNotSupported;
  const int size = bf16 ? 2 : 4;
  const cuuint64_t dims[3] = {(cuuint64_t)cols, (cuuint64_t)rows, (cuuint64_t)depth};
  const cuuint64_t strides[2] = {(cuuint64_t)(ld * size), (cuuint64_t)(ld * size * rows)};
  const cuuint32_t box[3] = {(cuuint32_t)box_cols, (cuuint32_t)box_rows, 1}, es[3] = {1, 1, 1};
  return enc(m, bf16 ? CU_TENSOR_MAP_DATA_TYPE_BFLOAT16 : CU_TENSOR_MAP_DATA_TYPE_FLOAT32, rank,
             const_cast<void*>(p), dims, strides, box, es, CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B,
             CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS
             ? cudaSuccess
             : cudaErrorInvalidValue;
}

// The pairs that run at once on the device; also opts in to the shared memory.
cudaError_t resident_pairs(int device, int* out) {
  static std::atomic<int> cached[64];
  int n = device < 64 ? cached[device].load(std::memory_order_acquire) : 0;
  if (!n) {
    const void* kernels[5] = {(const void*)ts_vocab_kernel<kLoss, true>, (const void*)ts_vocab_kernel<kDlogits, false>,
                              (const void*)ts_vocab_kernel<kDlogits, true>, (const void*)ts_vocab_kernel<kGrad, false>,
                              (const void*)ts_vocab_kernel<kGrad, true>};
    for (const void* k : kernels) {
      const cudaError_t e = cudaFuncSetAttribute(k, cudaFuncAttributeMaxDynamicSharedMemorySize, kSmem);
      if (e != cudaSuccess) return e;
    }
    cudaLaunchConfig_t cfg = pdl_config(2, kThreads, kSmem, nullptr);
    cudaLaunchAttribute at[1];
    at[0].id = cudaLaunchAttributeClusterDimension;
    at[0].val.clusterDim.x = 2;
    at[0].val.clusterDim.y = at[0].val.clusterDim.z = 1;
    cfg.attrs = at;
    cfg.numAttrs = 1;
    const cudaError_t e = cudaOccupancyMaxActiveClusters(&n, ts_vocab_kernel<kGrad, true>, &cfg);
    if (e != cudaSuccess) return e;
    if (n < 1) return cudaErrorLaunchOutOfResources;
    if (device < 64) cached[device].store(n, std::memory_order_release);
  }
  *out = n;
  return cudaSuccess;
}

template <class K, class A>
cudaError_t launch(K kernel, int64_t grid, int block, int smem, const A& args, cudaStream_t st) {
  cudaLaunchConfig_t cfg = pdl_config((int)grid, block, smem, st);
  cudaLaunchAttribute at[1];
  pdl_attr(cfg, at);
  return cudaLaunchKernelEx(&cfg, kernel, args);
}

int64_t round_up(int64_t n, int64_t m) { return (n + m - 1) / m * m; }
int64_t tiles(int64_t n) { return (n + kTile - 1) / kTile; }
// Copies' rows begin on whole lines (a box's rows of 128 bytes then are one each),
// narrow ones on 16 bytes.
int64_t pitch_of(int64_t cols) { return round_up(cols, cols < 256 ? 8 : 64); }

CopyRows copy_of(const TsMat& m, int64_t rows, int cols, void* dst) {
  CopyRows C = {};
  C.src = static_cast<const __nv_bfloat16*>(m.p);
  C.dst = static_cast<__nv_bfloat16*>(dst);
  C.ld = m.ld;
  C.pitch = pitch_of(cols);
  C.cols = cols;
  C.units = rows * (C.pitch / 8);
  return C;
}
cudaError_t launch_copy(const CopyRows& C, cudaStream_t st) {
  return launch(ts_loss_copy_kernel, (C.units + 511) / 512, 256, 0, C, st);
}
// Copies the matrix to `at` and describes the copy.
cudaError_t copy_aligned(TsMat& m, int64_t rows, int cols, void* at, cudaStream_t st) {
  const cudaError_t e = launch_copy(copy_of(m, rows, cols, at), st);
  m.p = at;
  m.ld = pitch_of(cols);
  return e;
}

// The logits' tiles are half as wide where that still leaves a pair without one.
// (512 x 1024 x 4000, backward: 28 us, with the wider tiles 33.)
int logits_width(int64_t tiles_t, int64_t vocab, int pairs) {
  return tiles_t * ((vocab + kHalf - 1) / kHalf) <= pairs ? kHalf : kTile;
}
// Rows of the boxes of x and d: past the last row TMA would fill with zeros,
// which takes as long as reading.
int box_rows(int64_t rows) { return (int)std::min<int64_t>(kHalf, round_up(rows, 16)); }

// Whether dw's copy of x (`units` of 16 bytes) fits beside the first piece's logits:
// a warp of each CTA takes 1 to 2 us for every 128 units, the pair 0.5 us for each
// block of K of its items; before them it is a launch, 3 us, and bound by memory.
// (Backward, us, beside and before: 300 x 256 x 1000 15.3 and 16.1, 2048 x 256 x
// 32000 95 and 98, 4096 x 1024 x 8000 137 and 132, 8192 x 4096 x 8000 1000 and 892,
// 16384 x 2048 x 4000 756 and 456, 256 x 4096 x 100 491 and 27.)
bool copy_beside(int64_t units, int64_t items, int64_t cols, int pairs) {
  const int64_t ctas = 2 * std::min<int64_t>(items, pairs);
  const int64_t blocks = (items + pairs - 1) / pairs * ((cols + kKB - 1) / kKB);
  return units / (ctas * 128) <= blocks / 4 + 3;
}

// An item of dw takes at least about three blocks of K for its epilogue.
int64_t dw_blocks(int64_t rows) { return std::max<int64_t>(3, (rows + kKB - 1) / kKB); }

// How nx items of dx of cx blocks of K each and nw of dw of cw share `pairs`
// pairs (see item_of), and how many blocks the last one ends after, an item's
// start and end being about one.
struct Schedule {
  int dw_first, late, extra;
  int64_t blocks;
};
Schedule schedule(int64_t nx, int64_t cx, int64_t nw, int64_t cw, int pairs) {
  Schedule s = {};
  ++cx;
  ++cw;
  s.dw_first = cw > cx;
  if (s.dw_first) {
    std::swap(nx, nw);
    std::swap(cx, cw);
  }
  s.late = (int)(nx % pairs);
  s.extra = s.late ? (int)((cx + cw / 2) / cw) : 0;
  const int64_t rounds = nx / pairs, early = pairs - s.late, ahead = std::min<int64_t>(nw, early * s.extra);
  const int64_t both = (nw - ahead) / pairs, rest = (nw - ahead) % pairs;   // items of all pairs
  // a late pair's, and an early one's: the pairs that come first take the rest
  const int64_t late = s.late ? rounds * cx + cx + (both + (rest > 0)) * cw : 0;
  const int64_t first = rounds * cx + ((ahead + early - 1) / early + both + (rest > s.late)) * cw;
  s.blocks = std::max(late, first);
  return s;
}

// Launches the product kernel on `pairs` pairs, with as many ring slots of the
// operands' rows (256 bytes each) as there is room for.  (Three where there could
// be six cost 33 x 1024 x 4000 1.5 of its 8 us: the way of a copy is longer than
// the MMAs of two slots.)
template <int MODE, bool CHAINS>
cudaError_t launch_product(VocabKernel& P, int64_t pairs, cudaStream_t st) {
  const int b_rows = MODE != kGrad ? P.tile_n / 2 : P.nx ? kHalf : P.box_rows;
  P.slot_bytes = (P.box_rows + b_rows) * 2 * kRowBytes;
  P.slots = std::min(kMaxSlots, kRingBytes / P.slot_bytes);
  return launch(ts_vocab_kernel<MODE, CHAINS>, 2 * pairs, kThreads, kSmem, P, st);
}

// The forward pass's workspace for `rows` rows, its copy of w's rows aside: two
// parts a tile, and tiles of half the width.
int64_t forward_bytes(int64_t rows, int64_t cols, int64_t vocab, bool copy_x) {
  return (copy_x ? round_up(rows * pitch_of(cols) * 2, 256) : 0) + round_up(rows * 4, 256) +
         round_up(rows * 4 * tiles(vocab) * 8, 256);
}
// The backward pass's, d's piece aside, and d's for 256 of the vocabulary.
int64_t backward_bytes(int64_t rows, int64_t cols, int64_t splits) {
  return round_up(rows * pitch_of(cols) * 2, 256) + round_up(splits * rows * pitch_of(cols) * 4, 256);
}
// The parts that dx's K is cut in at most: some items a pair, where there are not
// enough without.
int64_t most_splits(int64_t rows, int64_t cols, int64_t vocab) {
  return std::max<int64_t>(1, std::min<int64_t>(tiles(vocab) / 2, 256 / (tiles(rows) * tiles(cols))));
}
int64_t piece_bytes(int64_t rows, int64_t cols, bool copy_w) {
  return kTile * (rows + (copy_w ? pitch_of(cols) : 0)) * 2;
}

}  // namespace

int64_t vocab_loss_workspace(int64_t rows, int64_t cols, int64_t vocab, bool copy_x, bool copy_w, bool backward,
                             bool whole) {
  if (backward)
    return backward_bytes(rows, cols, whole && rows > 0 ? most_splits(rows, cols, vocab) : 1) +
           (whole ? tiles(vocab) : 1) * piece_bytes(rows, cols, copy_w);
  if (whole)
    return forward_bytes(rows, cols, vocab, copy_x) + (copy_w ? tiles(vocab) * kTile * pitch_of(cols) * 2 : 0);
  return forward_bytes(std::min<int64_t>(rows, kTile), cols, vocab, copy_x) +
         (copy_w ? kTile * pitch_of(cols) * 2 : 0);
}

cudaError_t launch_vocab_loss(const ts_ops& h, const VocabLossArgs& a, cudaStream_t st) {
  if (few_rows(a)) return launch_few_loss(h, a, st);
  int pairs = 0;
  cudaError_t e = resident_pairs(h.device, &pairs);
  if (e != cudaSuccess) return e;
  const bool copy_x = !rows_aligned(a.x), copy_w = !rows_aligned(a.w);
  const int64_t pitch = pitch_of(a.cols);
  // w's rows are copied whole where they fit beside all of x's, or as many at a time
  // as half of the workspace takes
  int64_t piece = a.vocab, wbytes = 0;
  if (copy_w) {
    piece = tiles(a.vocab) * kTile;
    if (forward_bytes(a.rows, a.cols, a.vocab, copy_x) + piece * pitch * 2 > h.ws_bytes)
      piece = std::min<int64_t>(piece, std::max<int64_t>(1, h.ws_bytes / 2 / (kTile * pitch * 2)) * kTile);
    wbytes = piece * pitch * 2;
  }
  // all rows at once, or as many as leave w's room
  int64_t block = a.rows;
  if (forward_bytes(block, a.cols, a.vocab, copy_x) + wbytes > h.ws_bytes) {
    block = std::max<int64_t>(0, h.ws_bytes - wbytes) / forward_bytes(kTile, a.cols, a.vocab, copy_x) * kTile;
    if (block < kTile) {   // (room for one tile of each was checked)
      block = kTile;
      piece = kTile;
      wbytes = copy_w ? piece * pitch * 2 : 0;
    }
  }
  uint8_t* wcopy = h.ws + h.ws_bytes - wbytes;   // (all of these are multiples of 256)
  for (int64_t t0 = 0; t0 < a.rows; t0 += block) {
    const int64_t rows = std::min(block, a.rows - t0);
    uint8_t* at = h.ws;
    TsMat x = a.x;
    x.p = static_cast<const __nv_bfloat16*>(a.x.p) + t0 * a.x.ld;
    if (copy_x) {
      e = copy_aligned(x, rows, a.cols, at, st);
      if (e != cudaSuccess) return e;
      at += round_up(rows * pitch * 2, 256);
    }
    JoinKernel J = {};
    J.tlogit = reinterpret_cast<float*>(at);
    at += round_up(rows * 4, 256);
    J.part = reinterpret_cast<float2*>(at);
    J.targets = a.targets ? a.targets + t0 : nullptr;
    J.loss = a.loss ? a.loss + t0 : nullptr;
    J.lse = a.lse ? a.lse + t0 : nullptr;
    J.vocab = a.vocab;
    J.rows = (int)rows;
    VocabKernel P = {};
    P.rows = (int)rows;
    P.cols = a.cols;
    P.total = a.vocab;
    P.tiles_t = (int)tiles(rows);
    P.box_rows = box_rows(rows);
    P.tlogit = const_cast<float*>(J.tlogit);
    P.targets = a.loss ? J.targets : nullptr;
    P.err = h.err;
    P.wait_limit_ns = h.wait_limit_ns;
    P.inject = h.inject;
    e = make_map(&P.x, x.p, 1, a.cols, rows, x.ld, 64, P.box_rows);
    if (e != cudaSuccess) return e;
    for (int64_t v0 = 0; v0 < a.vocab; v0 += piece) {
      const int64_t nv = std::min(piece, a.vocab - v0);
      TsMat w = a.w;
      w.p = static_cast<const __nv_bfloat16*>(a.w.p) + v0 * a.w.ld;
      if (copy_w) {
        e = copy_aligned(w, nv, a.cols, wcopy, st);
        if (e != cudaSuccess) return e;
      }
      P.vocab = (int)nv;
      P.v0 = (int)v0;
      P.tile_n = logits_width(P.tiles_t, nv, pairs);
      P.tiles_v = (int)((nv + P.tile_n - 1) / P.tile_n);
      e = make_map(&P.w, w.p, 1, a.cols, nv, w.ld, 64, P.tile_n / 2);
      if (e != cudaSuccess) return e;
      P.part = const_cast<float2*>(J.part) + J.parts * rows;
      J.parts += 2 * P.tiles_v;
      const int64_t items = (int64_t)P.tiles_t * P.tiles_v;
      e = launch_product<kLoss, true>(P, std::min<int64_t>(pairs, items), st);
      if (e != cudaSuccess) return e;
    }
    e = launch(ts_loss_join_kernel, (rows + 31) / 32, kJoinWarps * 32, 0, J, st);
    if (e != cudaSuccess) return e;
  }
  return cudaSuccess;
}

cudaError_t launch_vocab_loss_backward(const ts_ops& h, const VocabLossArgs& a, cudaStream_t st) {
  int pairs = 0;
  cudaError_t e = resident_pairs(h.device, &pairs);
  if (e != cudaSuccess) return e;
  if (!a.dx.p && !a.dw.p) return cudaSuccess;
  if (a.rows == 0) {
    if (!a.dw.p || a.accumulate) return cudaSuccess;
    cudaLaunchConfig_t cfg = pdl_config((int)std::min<int64_t>(a.vocab, 8 * h.nsm), 256, 0, st);
    cudaLaunchAttribute at[1];
    pdl_attr(cfg, at);
    return a.dw.bf16 ? cudaLaunchKernelEx(&cfg, ts_loss_zero_kernel<__nv_bfloat16>,
                                          static_cast<__nv_bfloat16*>(a.dw.p), a.dw.ld, (int)a.vocab, a.cols)
                     : cudaLaunchKernelEx(&cfg, ts_loss_zero_kernel<float>, static_cast<float*>(a.dw.p), a.dw.ld,
                                          (int)a.vocab, a.cols);
  }
  bool copy_x = !rows_aligned(a.x);
  const bool copy_w = !rows_aligned(a.w);
  const int64_t pitch = pitch_of(a.cols), tiles_t = tiles(a.rows), tiles_c = tiles(a.cols), tiles_v = tiles(a.vocab);
  // dx's items are cut along the vocabulary where that shortens the gradients'
  // launch by more than the sums' own kernel costs (about six blocks of K)
  const int64_t one_dx = a.rows * pitch * 4, cost = piece_bytes(a.rows, a.cols, copy_w);
  // (as if dw were wanted too: dx does not depend on whether it is)
  const int64_t nkb = (a.vocab + kKB - 1) / kKB, nw = tiles_v * tiles_c;
  int64_t splits = 1, least = INT64_MAX;
  // (not where the whole vocabulary would fit in one piece without; where it does
  // not, cuts may cost pieces: 4096 x 256 x 131072 in 64 MiB takes 942 us with 4 cuts
  // and 23 pieces, 1079 uncut in 18, but 16 x 4096 x 131072 in 4 MiB 701 and 576)
  const int64_t rest = (backward_bytes(a.rows, a.cols, 1) + tiles_v * cost <= h.ws_bytes ? tiles_v : 1) * cost;
  for (int64_t n = 1; n <= most_splits(a.rows, a.cols, a.vocab); ++n) {
    if (n > 1 && backward_bytes(a.rows, a.cols, n) + rest > h.ws_bytes) break;
    const Schedule s = schedule(tiles_t * tiles_c * n, (nkb + n - 1) / n, nw, dw_blocks(a.rows), pairs);
    // (dw of few rows is bound by memory, like dx: neither runs beside the other
    // for free, so each kind's rounds count by themselves)
    const int64_t nx = tiles_t * tiles_c * n;
    const int64_t blocks = a.rows > kHalf ? s.blocks
                                          : (nx + pairs - 1) / pairs * ((nkb + n - 1) / n + 1) +
                                                (nw + pairs - 1) / pairs * (dw_blocks(a.rows) + 1);
    const int64_t t = blocks + (n > 1 ? 6 + one_dx * n / (int64_t(4) << 20) : 0);
    if (t < least) {
      least = t;
      splits = n;
    }
  }
  // equal pieces of the vocabulary, as few as the workspace allows
  const int64_t most = std::max<int64_t>(1, (h.ws_bytes - backward_bytes(a.rows, a.cols, splits)) / cost);
  const int64_t pieces = (tiles_v + most - 1) / most, piece = (tiles_v + pieces - 1) / pieces * kTile;
  uint8_t* xcopy = h.ws;
  float* sums = reinterpret_cast<float*>(h.ws + round_up(a.rows * pitch * 2, 256));
  uint8_t* d = h.ws + backward_bytes(a.rows, a.cols, splits);
  uint8_t* wcopy = d + a.rows * piece * 2;
  VocabKernel P = {};
  P.rows = (int)a.rows;
  P.cols = a.cols;
  P.total = a.vocab;
  P.tiles_t = (int)tiles_t;
  P.tiles_c = (int)tiles_c;
  P.box_rows = box_rows(a.rows);
  P.targets = a.targets;
  P.lse = a.lse;
  P.g_loss = a.g_loss;
  P.g_lse = a.g_lse;
  P.splits = (int)splits;
  P.err = h.err;
  P.wait_limit_ns = h.wait_limit_ns;
  P.inject = h.inject;
  // dw's copy of x: beside the first piece's logits, or before them where they are
  // too short to hide it, or TMA cannot read x itself
  TsMat x = a.x;
  CopyRows C = copy_of(a.x, a.rows, a.cols, xcopy);
  C.targets = a.g_lse ? nullptr : a.targets;
  C.lse = a.lse;
  C.vocab = a.vocab;
  const bool few = few_rows(a) && pieces == 1;   // (their logits take rows as they lie)
  if (few) {
    copy_x = false;
    if (!a.dw.p) C.units = 0;
  } else if (copy_x) {
    e = launch_copy(C, st);
    if (e != cudaSuccess) return e;
    x.p = xcopy;
    x.ld = pitch;
  } else if (a.dw.p) {
    const int64_t first = std::min(piece, a.vocab), width = logits_width(tiles_t, first, pairs);
    if (copy_beside(C.units, tiles_t * ((first + width - 1) / width), a.cols, pairs)) {
      P.copy = C;
    } else {
      e = launch_copy(C, st);
      if (e != cudaSuccess) return e;
    }
  }
  auto describe = [](Out& o, const TsOut& m, int64_t rows, int cols, bool add) {
    o.p = m.p;
    o.ld = m.ld;
    o.bf16 = m.bf16;
    o.add = add;
    o.tma = rows_aligned(m) && !(m.bf16 && add);
    o.whole = cols * m.elem() % 16 == 0;
    return o.tma ? make_map(&o.map, m.p, m.bf16, cols, rows, m.ld, m.bf16 ? 64 : 32, 32, 3) : cudaSuccess;
  };
  // one piece that is not cut is dx itself
  const bool direct = splits == 1 && pieces == 1;
  if (a.dx.p) {
    if (direct) {
      e = describe(P.out[0], a.dx, a.rows, a.cols, false);
    } else {
      P.out[0].tma = P.out[0].whole = 1;
      e = make_map(&P.out[0].map, sums, 0, a.cols, a.rows, pitch, 32, 32, 3, splits);
    }
  }
  for (int64_t v0 = 0; v0 < a.vocab && e == cudaSuccess; v0 += piece) {
    const int64_t nv = std::min(piece, a.vocab - v0), dpitch = tiles(nv) * kTile;
    TsMat w = a.w;
    w.p = static_cast<const __nv_bfloat16*>(a.w.p) + v0 * a.w.ld;
    if (copy_w) {
      e = copy_aligned(w, nv, a.cols, wcopy, st);
      if (e != cudaSuccess) return e;
    }
    P.vocab = (int)nv;
    P.v0 = (int)v0;
    P.out[0].add = v0 > 0;
    if (few) {
      e = launch_few_dlogits(h, a, C, reinterpret_cast<__nv_bfloat16*>(d), dpitch, st);
    } else {
      P.tile_n = logits_width(tiles_t, nv, pairs);
      P.tiles_v = (int)((nv + P.tile_n - 1) / P.tile_n);
      e = make_map(&P.x, x.p, 1, a.cols, a.rows, x.ld, 64, P.box_rows);
      if (e == cudaSuccess) e = make_map(&P.w, w.p, 1, a.cols, nv, w.ld, 64, P.tile_n / 2);
      if (e == cudaSuccess) e = make_map(&P.store_d, d, 1, dpitch, a.rows, dpitch, 64, 32);
      if (e != cudaSuccess) return e;
      const int64_t np = std::min<int64_t>(pairs, tiles_t * P.tiles_v);
      e = a.cols > kLossChain * kKB ? launch_product<kDlogits, true>(P, np, st)
                                    : launch_product<kDlogits, false>(P, np, st);
      P.copy.units = 0;
    }
    if (e == cudaSuccess && a.dw.p) {
      TsOut dw = a.dw;
      dw.p = static_cast<uint8_t*>(a.dw.p) + v0 * a.dw.ld * a.dw.elem();
      e = describe(P.out[1], dw, nv, a.cols, a.accumulate);
      if (e == cudaSuccess) e = make_map(&P.x, xcopy, 1, a.cols, a.rows, pitch, 64, P.box_rows);
    }
    if (e == cudaSuccess) e = make_map(&P.d, d, 1, dpitch, a.rows, dpitch, 64, P.box_rows);
    if (e == cudaSuccess && P.tile_n != kTile && a.dx.p) e = make_map(&P.w, w.p, 1, a.cols, nv, w.ld, 64, kHalf);
    if (e != cudaSuccess) return e;
    P.tiles_v = (int)tiles(nv);
    P.nx = a.dx.p ? (int)(tiles_t * tiles_c * splits) : 0;
    P.nw = a.dw.p ? (int)(P.tiles_v * tiles_c) : 0;
    const int np = std::min(pairs, P.nx + P.nw);
    const Schedule s = schedule(P.nx, (nv + kKB - 1) / kKB / splits, P.nw, dw_blocks(a.rows), np);
    P.dw_first = s.dw_first;
    P.late = s.late;
    P.extra = s.extra;
    const int64_t dx_blocks = P.nx ? ((nv + kKB - 1) / kKB + splits - 1) / splits : 0;
    const int64_t most_blocks = std::max(dx_blocks, P.nw ? (a.rows + kKB - 1) / kKB : 0);
    e = most_blocks > kGradChain ? launch_product<kGrad, true>(P, np, st) : launch_product<kGrad, false>(P, np, st);
  }
  if (direct) return e;
  if (e != cudaSuccess || !a.dx.p) return e;
  DxKernel D = {};
  D.sums = sums;
  D.dx = a.dx.p;
  D.pitch = pitch;
  D.rows = a.rows;
  D.ld = a.dx.ld;
  D.cols = a.cols;
  D.groups = (a.cols + kGroupCols - 1) / kGroupCols;
  D.units = a.rows * D.groups;
  D.splits = (int)splits;
  const bool vec = rows_aligned(a.dx);
  auto* kernel = a.dx.bf16 ? vec ? ts_loss_dx_kernel<__nv_bfloat16, true> : ts_loss_dx_kernel<__nv_bfloat16, false>
                 : vec     ? ts_loss_dx_kernel<float, true>
                           : ts_loss_dx_kernel<float, false>;
  return launch(kernel, (D.units + 7) / 8, 256, 0, D, st);
}

}  // namespace fg
