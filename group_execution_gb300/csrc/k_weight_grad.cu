// A matmul's weight gradient from its 8-bit saved input: dW = X^T dY over the
// rows (tokens).  With an affine input X = gamma h + beta by column, h the
// checkpoint,
//   dW_cj = gamma_c sum_t h_tc dY_tj + beta_c db_j,   db_j = sum_t dY_tj,
// so the product is of h alone and gamma and beta enter in the epilogue.
//
// The product runs on the 5th-generation tensor cores.  A checkpoint's values
// are exact in bf16, so the products are exact and the sums are float32:
// bf16 operands cost no accuracy.  Persistent CTA pairs walk 256 x 256 tiles
// of dW (2-SM tcgen05.mma, cta_group::2), tokens 128 at a time; each CTA
// stages half of the tile's columns of h and half of its columns of dY in a
// ring of shared-memory slots, both MN-major, 128-byte swizzled.  Warps, in
// each CTA:
//   warp 0      TMA producer of its dY half (two lanes, 64 columns each;
//               counted on the even CTA's slot barrier),
//   warp 1      allocates TMEM (two accumulators) and, in the even CTA,
//               issues the MMAs from one thread,
//   warps 4-11  epilogue: a thread owns half of one row of the CTA's 128 x
//               256 accumulator; it overlaps the next tile's MMAs,
//   warps 12-27 the checkpoint: two groups of eight that take turns by slot,
//               64 tokens to each half: 16-byte loads of int8 values, a slot
//               ahead, expanded to bf16, scaled and stored swizzled.
// At 8192 x 4096 x 4096 this takes 210 us, 1309 TFLOP/s (68 % of the burst rate
// of a plain bf16 product, 76 % of its sustained rate; 224 us when it runs for
// 100 ms on end): the expansion's stores, the copies' writes and the MMA's reads
// fill the 1024 cycles of shared memory that a slot's MMAs take.  dY's column
// sums, where asked for, are a pass of their own before it, 15 to 20 us.  What was measured on the way (us a
// call, and cycles of the issuing warp): a slot's wait, commit and first MMA
// cost about 600 cycles beside the MMAs, so slots hold 128 tokens; an arrival
// that releases to the cluster costs about 2000 (626 us), so arrivals release
// to the CTA, after the proxy fence; the bytes through a shared-memory ring of
// their own 226 us; the expanded operand in tensor memory (256 x 192 tiles)
// leaves room for four slots of 64 tokens, fewer than the way from an MMA's end
// over the expanding warps to the next MMA is long, 252 us.
//
// A float32 accumulator that takes all 8192 tokens one MMA after the other is
// 2.8e-6 off (2-norm): the tensor core truncates as it adds.  So a sum runs
// over at most 2048 tokens; what it came to is added to a float32 partial in
// the workspace, which the same thread of the same pair reads back (L2).
//
// Tiles past the last full round of pairs are cut along the tokens when that
// balances the round: each piece writes its float32 partial to the workspace
// and a second kernel adds the pieces in order.
//
// Rows of dY that TMA cannot read (a start or pitch off 16 bytes) are first
// copied to the workspace at an aligned pitch, as many tokens at a time as
// half of it takes.
//
// Every wait is bounded; on expiry the CTA records the error, the pair waits
// for the copies that either CTA has in flight, frees its TMEM and returns.
#include <cuda.h>

#include <algorithm>
#include <atomic>
#include <mutex>

#include "launch.h"
#include "ts_device.cuh"

namespace fg {
namespace {

constexpr int kTile = 256;                       // rows and columns of dW a pair's tile covers
constexpr int kHalf = kTile / 2;                 // ... and one CTA stages of each operand
constexpr int kKB = 128;                         // tokens of a ring slot
constexpr int kGroupBytes = kKB * 128;           // 64 columns of either operand
constexpr int kOperandBytes = 2 * kGroupBytes;   // 32 KB
constexpr int kSlotBytes = 2 * kOperandBytes;
constexpr int kSlots = 3;
constexpr int kGroups = 2;                       // groups of expanding warps, which take turns by slot
constexpr int kSets = 2 * kGroups;               // two sets of four warps a group, half a slot's tokens each
constexpr int kSetTokens = kKB / 2;
constexpr int kExpandWarps = 4 * kSets;
constexpr int kThreads = (12 + kExpandWarps) * 32;
constexpr int kStagePitch = 17;                  // floats of a row of 16 columns on the way to an unaligned dw
constexpr int kStageFloats = 32 * kStagePitch;   // an epilogue warp's
template <bool WIDE>
constexpr int kSmem = kSlots * kSlotBytes + 1024 + (WIDE ? 0 : 8 * kStageFloats * 4);
constexpr int kChain = 16;                       // blocks of kKB tokens one accumulation runs over
constexpr int64_t kPieceFloats = (int64_t)kTile * kTile;

struct WgradKernel {
  CUtensorMap dy;
  TsCkpt x;
  int rows, cols, n;
  int tiles_n;         // tiles along n; tile t covers columns of h from (t / tiles_n) * kTile
  int full, pieces;    // tiles taken whole, and pieces per later tile
  int items;           // full + pieces * (tiles - full)
  const float* gamma;
  const float* beta;
  const float* colsum;
  float* dw;
  int64_t lddw;
  int accumulate;
  float4* part;        // the cut tiles' pieces
  float4* chain;       // each pair's running partial
  int32_t* err;
  int64_t wait_limit_ns;
  int inject;
};

struct Item {
  int tile, piece, kb0, kb1;   // piece = -1: a whole tile
};
__device__ __forceinline__ Item item_of(const WgradKernel& P, int idx, int nkb) {
  if (idx < P.full) return Item{idx, -1, 0, nkb};
  const int q = idx - P.full, p = q % P.pieces;
  if (P.pieces == 1) return Item{P.full + q, -1, 0, nkb};
  return Item{P.full + q / P.pieces, q, (int)((int64_t)nkb * p / P.pieces), (int)((int64_t)nkb * (p + 1) / P.pieces)};
}

// What one accumulator takes of an item: token blocks [kb0, kb1).
__device__ __forceinline__ int segment_end(const Item& w, int kb0) {
  return w.kb1 - kb0 > kChain ? kb0 + kChain : w.kb1;
}

// Waits for the phase with the given parity, at most `limit` ns and only while
// no thread of the CTA has given up.
__device__ __forceinline__ bool wait_bar(uint32_t bar, uint32_t parity, int64_t limit, volatile int* abort_flag) {
  if (mbar_try_wait(bar, parity)) return true;
  const uint64_t t0 = global_ns();
  while (!mbar_try_wait(bar, parity))
    if (*abort_flag || (int64_t)(global_ns() - t0) > limit) return false;
  return true;
}
// Four int8 values -> two bf16 pairs, times a power of two, exactly: with
// byte b under 0x43 (a bf16 of exponent 2^7), 0x4300 | (b & 127) is 128 + (b &
// 127) and 0x4300 | (b & 128) is 128 or 256, and their difference is b as a
// signed number.
__device__ __forceinline__ void expand4(uint32_t w, __nv_bfloat162 step, uint32_t& lo, uint32_t& hi) {
  const uint32_t a = __byte_perm(w, 0x43434343u, 0x4140), b = __byte_perm(w, 0x43434343u, 0x4342);
  const uint32_t am = a & 0xff7fff7fu, as = a & 0xff80ff80u, bm = b & 0xff7fff7fu, bs = b & 0xff80ff80u;
  const __nv_bfloat162 l = __hmul2(__hsub2(*reinterpret_cast<const __nv_bfloat162*>(&am),
                                           *reinterpret_cast<const __nv_bfloat162*>(&as)), step);
  const __nv_bfloat162 h = __hmul2(__hsub2(*reinterpret_cast<const __nv_bfloat162*>(&bm),
                                           *reinterpret_cast<const __nv_bfloat162*>(&bs)), step);
  lo = *reinterpret_cast<const uint32_t*>(&l);
  hi = *reinterpret_cast<const uint32_t*>(&h);
}
__device__ __forceinline__ __nv_bfloat162 bf16_step(uint32_t e) {
  const uint32_t h = e < 255 ? (max(e, 7u) - 6) << 7 : 0x7fc0u, w = h | h << 16;
  return *reinterpret_cast<const __nv_bfloat162*>(&w);
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

// Eight values of one row of dw, scaled and, with beta, shifted by dy's column
// sums s.
__device__ __forceinline__ void affine8(const WgradKernel& P, const float* s, float g, float b, float (&v)[8]) {
#pragma unroll
  for (int i = 0; i < 8; ++i) v[i] *= g;
  if (P.beta) {
    float c[8];
    load8(s, c);
#pragma unroll
    for (int i = 0; i < 8; ++i) v[i] += b * c[i];
  }
}
// Stores them (vec: 8 or 4 floats at a time), accumulated as asked.
__device__ __forceinline__ void finish8(const WgradKernel& P, const float* s, float* row, int j, float g, float b,
                                        int vec, float (&v)[8]) {
  affine8(P, s, g, b, v);
  float* d = row + j;
  if (vec == 8 && j + 8 <= P.n) {
    if (P.accumulate) {
      float o[8];
      load8(d, o);
#pragma unroll
      for (int i = 0; i < 8; ++i) v[i] = o[i] + v[i];
    }
    asm volatile("st.global.v8.f32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};" ::"l"(d), "f"(v[0]), "f"(v[1]), "f"(v[2]),
                 "f"(v[3]), "f"(v[4]), "f"(v[5]), "f"(v[6]), "f"(v[7])
                 : "memory");
  } else if (j + 8 <= P.n) {
    if (P.accumulate) {
      float o[8];
      load8(d, o);
#pragma unroll
      for (int i = 0; i < 8; ++i) v[i] = o[i] + v[i];
    }
    store8(d, v);
  } else {
#pragma unroll
    for (int i = 0; i < 8; ++i)
      if (j + i < P.n) d[i] = P.accumulate ? d[i] + v[i] : v[i];
  }
}
// The floats of dw that a thread stores at a time; 1: a row is spread over
// threads.
__host__ __device__ __forceinline__ int store_width(const WgradKernel& P) {
  const uint64_t p = reinterpret_cast<uint64_t>(P.dw);
  return p % 32 == 0 && P.lddw % 8 == 0 ? 8 : p % 16 == 0 && P.lddw % 4 == 0 ? 4 : 1;
}

// WIDE: rows of dw on 16 bytes, at least.
template <bool WIDE>
__global__ void __cluster_dims__(2, 1, 1) __launch_bounds__(kThreads, 1)
    ts_wgrad_kernel(const __grid_constant__ WgradKernel P) {
  extern __shared__ uint8_t smem_raw[];
  __shared__ __align__(8) uint64_t bar_mem[2 * kSlots + 5];
  __shared__ int abort_flag, issued[2];         // copies that either lane of warp 0 has issued
  __shared__ int peer_gave_up, peer_issued;     // written by the pair's other CTA
  __shared__ uint32_t tmem_slot;
  __shared__ __align__(16) float colsums[8][kTile / 2];
  uint8_t* ring = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  const uint32_t full0 = smem_u32(bar_mem), empty0 = full0 + 8 * kSlots, tfull0 = empty0 + 8 * kSlots,
                 tempty0 = tfull0 + 16, done_bar = tempty0 + 16;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int h = (int)cluster_ctarank();
  const bool leader = h == 0;
  const uint16_t pair_mask = 3u;
  const int npair = gridDim.x / 2, pair = blockIdx.x / 2;
  const int nkb = (P.rows + kKB - 1) / kKB;
  if (threadIdx.x == 0) {
    abort_flag = issued[0] = issued[1] = 0;
    for (int s = 0; s < kSlots; ++s) {
      mbar_init(full0 + 8 * s, 1 + 2 * 8);   // the even CTA's expect_tx, a group of eight warps in each CTA
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

  if (warp == 0) {
    // ---- dY producer: lane 0 the first 64 columns, lane 1 the rest ----
    if (lane < 2 && !P.inject) {
      const int g = lane;
      tma_prefetch(&P.dy);
      const uint64_t keep = l2_evict_last();
      const uint32_t cbar0 = cluster_addr(full0, 0), dst0 = smem_u32(ring) + kOperandBytes + g * kGroupBytes;
      int it = 0, s = 0;
      uint32_t ph = 0;
      bool ok = true;
      for (int x = pair; x < P.items && ok; x += npair) {
        const Item w = item_of(P, x, nkb);
        const int n0 = w.tile % P.tiles_n * kTile + h * kHalf + g * 64;
        for (int kb = w.kb0; kb < w.kb1; ++kb) {
          if (it >= kSlots && !wait_bar(empty0 + 8 * s, ph ^ 1, P.wait_limit_ns, &abort_flag)) {
            ok = false;
            break;
          }
          if (leader && g == 0) mbar_expect_tx(full0 + 8 * s, 2 * kOperandBytes);
          tma_load_2d_pair(dst0 + s * kSlotBytes, &P.dy, n0, kb * kKB, cbar0 + 8 * s, keep);
          ++it;
          if (++s == kSlots) {
            s = 0;
            ph ^= 1;
          }
        }
      }
      issued[g] = it;
      if (!ok) {
        abort_flag = 1;
        set_error(P.err, DEVERR_TIMEOUT);
      }
    }
  } else if (warp == 1) {
    // ---- MMA issuer ----
    if (lane == 0 && leader) {
      const uint32_t idesc = idesc_bf16_f32(kTile, kTile, 1, 1);
      // MN-major: atoms of 64 columns x 8 tokens, groups of 64 columns 16 KB apart
      const uint32_t base = smem_u32(ring);
      const uint64_t ad0 = smem_desc_sw128(base, kGroupBytes, 1024),
                     bd0 = smem_desc_sw128(base + kOperandBytes, kGroupBytes, 1024);
      int s = 0, i = 0;
      uint32_t ph = 0;
      bool ok = true;
      for (int x = pair; x < P.items && ok; x += npair) {
        const Item w = item_of(P, x, nkb);
        for (int s0 = w.kb0; s0 < w.kb1 && ok; ++i) {
          const int s1 = segment_end(w, s0), b = i & 1;
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
            const uint32_t so = (uint32_t)(s * kSlotBytes) >> 4;
#pragma unroll
            for (int kk = 0; kk < kKB / 16; ++kk)
              tc_mma_bf16<2>(tmem + b * kTile, ad0 + so + kk * (2048 >> 4), bd0 + so + kk * (2048 >> 4), idesc,
                             kb != s0 || kk != 0);
            tc_commit_mask(empty0 + 8 * s, pair_mask);
            if (++s == kSlots) {
              s = 0;
              ph ^= 1;
            }
          }
          if (ok) tc_commit_mask(tfull0 + 8 * b, pair_mask);
          s0 = s1;
        }
      }
      if (!ok) {
        abort_flag = 1;
        set_error(P.err, DEVERR_TIMEOUT);
      }
      // every MMA issued has completed before either CTA may free TMEM
      tc_commit_mask(done_bar, pair_mask);
      mbar_wait(done_bar, 0, kDrainLimitNs);
    }
  } else if (warp >= 4 && warp < 12) {
    // ---- epilogue ----
    const int q = warp & 3;   // the TMEM lane quarter this warp may access
    const int r = q * 32 + lane;
    const int vec = WIDE ? store_width(P) : 1;
    // partials: [64 column quads][128 rows][4], so that a warp's 16-byte
    // accesses cover 512 contiguous bytes
    float4* chain = P.chain + (int64_t)(pair * 2 + h) * (kPieceFloats / 8) + r;
    int i = 0;
    bool ok = true;
    for (int x = pair; x < P.items && ok; x += npair) {
      const Item w = item_of(P, x, nkb);
      const int c = w.tile / P.tiles_n * kTile + h * kHalf + r, n0 = w.tile % P.tiles_n * kTile;
      const float g = P.gamma && c < P.cols ? P.gamma[c] : 1.f, be = P.beta && c < P.cols ? P.beta[c] : 0.f;
      float* row = P.dw + (int64_t)c * P.lddw;
      if (P.beta) {
        // dy's column sums of this warp's columns, fetched during the products
        // (chunk by chunk in the epilogue they took 13 x 3720 x 1880 from 14
        // to 19 us and 512 x 4096 x 4096 from 38 to 45; the product of 8192
        // tokens, bound by shared memory, was 207 us that way and is 211 this
        // way, without beta too)
#pragma unroll
        for (int k = 0; k < kTile / 2; k += 32) {
          const int at = n0 + (warp >= 8 ? kTile / 2 : 0) + k + lane;
          colsums[warp - 4][k + lane] = at < P.n ? P.colsum[at] : 0.f;
        }
        __syncwarp();
      }
      float4* piece = w.piece < 0 ? nullptr : P.part + (int64_t)(w.piece * 2 + h) * (kPieceFloats / 8) + r;
      for (int s0 = w.kb0; s0 < w.kb1; ++i) {
        const int s1 = segment_end(w, s0), b = i & 1;
        ok = __all_sync(0xffffffffu, wait_bar(tfull0 + 8 * b, (i >> 1) & 1, P.wait_limit_ns, &abort_flag));
        if (!ok) break;
        tc_fence_after();
        const uint32_t acc0 = tmem + ((uint32_t)(q * 32) << 16) + b * kTile;
        const bool first = s0 == w.kb0, last = s1 == w.kb1;
        float4* dst = last ? piece : chain;
        // the partial's next chunk is fetched (from L2) before one is used
        float4 o[4];
        auto fetch = [&](int j) {
#pragma unroll
          for (int k = 0; k < 4; ++k) o[k] = __ldcg(chain + (j / 4 + k) * kHalf);
        };
        // two warps to a lane quarter, half the columns each
        const int j0 = warp >= 8 ? kTile / 2 : 0, j1 = j0 + kTile / 2;
        if (!first) fetch(j0);
#pragma unroll 1
        for (int j = j0; j < j1; j += 16) {
          if (n0 + j >= P.n) break;
          float v[16];
          tmem_ld16(acc0 + j, v);
          if (!first) {
#pragma unroll
            for (int k = 0; k < 4; ++k) {
              v[4 * k] += o[k].x;
              v[4 * k + 1] += o[k].y;
              v[4 * k + 2] += o[k].z;
              v[4 * k + 3] += o[k].w;
            }
            if (j + 16 < j1) fetch(j + 16);
          }
          if (dst) {
#pragma unroll
            for (int k = 0; k < 4; ++k)
              dst[(j / 4 + k) * kHalf] = make_float4(v[4 * k], v[4 * k + 1], v[4 * k + 2], v[4 * k + 3]);
          } else if constexpr (WIDE) {
            if (c < P.cols) {
#pragma unroll
              for (int k = 0; k < 2; ++k) {
                float e[8];
#pragma unroll
                for (int m = 0; m < 8; ++m) e[m] = v[8 * k + m];
                finish8(P, &colsums[warp - 4][j % (kTile / 2) + 8 * k], row, n0 + j + 8 * k, g, be, vec, e);
              }
            }
          } else {
            // rows of dw off 16 bytes go out through shared memory, half a
            // warp to a row: 786 x 2810 x 1142 takes 16 us, a thread to a row 31
            float* stage = reinterpret_cast<float*>(ring + kSlots * kSlotBytes) + (warp - 4) * kStageFloats;
#pragma unroll
            for (int k = 0; k < 2; ++k) {
              float e[8];
#pragma unroll
              for (int m = 0; m < 8; ++m) e[m] = v[8 * k + m];
              affine8(P, &colsums[warp - 4][j % (kTile / 2) + 8 * k], g, be, e);
#pragma unroll
              for (int m = 0; m < 8; ++m) stage[lane * kStagePitch + 8 * k + m] = e[m];
            }
            __syncwarp();
            // half a warp to a row
            const int col = n0 + j + (lane & 15);
            int left = P.cols - (c - lane + (lane >> 4));   // rows from this one on
            if (col >= P.n) left = 0;
            float* d = P.dw + (int64_t)(c - lane + (lane >> 4)) * P.lddw + col;
            const float* s = stage + (lane >> 4) * kStagePitch + (lane & 15);
#pragma unroll 1
            for (int k0 = 0; k0 < 4; ++k0) {
              float old[4] = {};
              if (P.accumulate) {
#pragma unroll
                for (int k = 0; k < 4; ++k)
                  if (2 * k < left) old[k] = d[2 * k * P.lddw];
              }
#pragma unroll
              for (int k = 0; k < 4; ++k)
                if (2 * k < left) d[2 * k * P.lddw] = old[k] + s[2 * k * kStagePitch];
              d += 8 * P.lddw;
              s += 8 * kStagePitch;
              left -= 8;
            }
            __syncwarp();
          }
        }
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive_cluster(cluster_addr(tempty0 + 8 * b, 0));
        s0 = s1;
      }
    }
    if (!ok && lane == 0) {
      abort_flag = 1;
      set_error(P.err, DEVERR_TIMEOUT);
    }
  } else if (warp >= 12) {
    // ---- expansion ----
    // a set's 64 tokens x 128 columns of every kGroups-th slot: thread t takes
    // tokens t / 8 + 16 u, columns (t % 8) * 16 .. + 15 (a warp's loads cover
    // four whole 128-byte lines)
    const int set = (warp - 12) >> 2, group = set >> 1, t = threadIdx.x & 127, jc = t & 7;
    const int tr = (set & 1) * kSetTokens + (t >> 3);   // this thread's first token of a slot
    const uint32_t written0 = cluster_addr(full0, 0);
    // the slot addresses of a thread's two 16-byte halves; lanes 4-7 of every
    // eight store them in the other order, so that eight lanes cover all banks
    const uint32_t g = (uint32_t)(jc >> 2) * kGroupBytes + (uint32_t)tr * 128;
    const uint32_t first = (uint32_t)(jc >> 2), c0 = (uint32_t)((jc & 3) * 2);
    const uint32_t off_a = g + (((c0 + first) ^ (tr & 7)) << 4), off_b = g + (((c0 + (first ^ 1)) ^ (tr & 7)) << 4);
    constexpr int kU = kSetTokens / 16;
    const int64_t spitch = P.x.pitch / kCkptBlock;
    // the load cursor: item, block, and the blocks left to the group's next
    int lx = pair, lkb = 0, lend = 0, lm0 = 0;
    auto open_item = [&]() {
      const Item w = item_of(P, lx, nkb);
      lkb = w.kb0;
      lend = w.kb1;
      lm0 = w.tile / P.tiles_n * kTile + h * kHalf;
    };
    auto skip = [&](int n) {   // n blocks on
      while (lx < P.items && n >= lend - lkb) {
        n -= lend - lkb;
        lx += npair;
        if (lx < P.items) open_item();
      }
      lkb += n;
    };
    uint4 v[kU];
    uint32_t e[kU];
    auto load = [&]() {
      const int row = lkb * kKB + tr, col = lm0 + jc * 16;
      const int8_t* q = P.x.q + (int64_t)row * P.x.pitch + col;
      const uint8_t* sc = P.x.scale + (int64_t)row * spitch + col / kCkptBlock;
#pragma unroll
      for (int u = 0; u < kU; ++u) {
        v[u] = make_uint4(0, 0, 0, 0);
        e[u] = 7;
        if (row + 16 * u < P.rows && col < P.x.pitch) {
          v[u] = *reinterpret_cast<const uint4*>(q + 16 * u * P.x.pitch);
          e[u] = sc[16 * u * spitch];
        }
      }
    };
    bool ok = true;
    if (lx < P.items) open_item();
    skip(group);
    if (lx < P.items) load();
    for (int blk = group; lx < P.items; blk += kGroups) {
      const int s = blk % kSlots;
      if (blk >= kSlots) {
        ok = __all_sync(0xffffffffu, wait_bar(empty0 + 8 * s, ((blk / kSlots) & 1) ^ 1, P.wait_limit_ns, &abort_flag));
        if (!ok) break;
      }
      uint8_t* dst = ring + s * kSlotBytes;
#pragma unroll
      for (int u = 0; u < kU; ++u) {
        const __nv_bfloat162 step = bf16_step(e[u]);
        uint4 lo, hi;
        expand4(v[u].x, step, lo.x, lo.y);
        expand4(v[u].y, step, lo.z, lo.w);
        expand4(v[u].z, step, hi.x, hi.y);
        expand4(v[u].w, step, hi.z, hi.w);
        *reinterpret_cast<uint4*>(dst + off_a + u * 16 * 128) = first ? hi : lo;
        *reinterpret_cast<uint4*>(dst + off_b + u * 16 * 128) = first ? lo : hi;
      }
      skip(kGroups);
      fence_proxy_async_smem();
      __syncwarp();
      if (lane == 0) mbar_arrive_cluster(written0 + 8 * s);
      if (lx < P.items) load();   // the next slot's bytes arrive while the tensor core is on the ones before it
    }
    if (!ok && lane == 0) {
      abort_flag = 1;
      set_error(P.err, DEVERR_TIMEOUT);
    }
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
    // slots they fill may lack arrivals, so each wait may run to its limit
    if (leader && threadIdx.x == 0) {
      const int last = mine > peer_issued ? mine : peer_issued;
      for (int k = last - kSlots < 0 ? 0 : last - kSlots; k < last; ++k)
        mbar_wait(full0 + 8 * (k % kSlots), (k / kSlots) & 1, kDrainLimitNs);
    }
    __syncwarp();
    cluster_sync();
  }
  tc_fence_after();
  if (warp == 1) tmem_dealloc<2>(tmem, 512);
}

// The cut tiles: a thread adds the pieces of one row's eight columns in order.
__global__ void __launch_bounds__(256) ts_wgrad_finish_kernel(const __grid_constant__ WgradKernel P) {
  pdl_launch_dependents();
  pdl_wait();
  const int tile = P.full + blockIdx.x / 32, b = blockIdx.x % 32;   // 32 blocks a tile: 8 columns of all 256 rows each
  const int h = threadIdx.x / kHalf, r = threadIdx.x % kHalf;
  const int c = tile / P.tiles_n * kTile + threadIdx.x, j = tile % P.tiles_n * kTile + b * 8;
  const bool in = c < P.cols && j < P.n;
  float v[8] = {};
  for (int p = 0; in && p < P.pieces; ++p) {
    const float4* o =
        P.part + (int64_t)((blockIdx.x / 32 * P.pieces + p) * 2 + h) * (kPieceFloats / 8) + b * 2 * kHalf + r;
    const float4 x = __ldcg(o), y = __ldcg(o + kHalf);
    v[0] += x.x; v[1] += x.y; v[2] += x.z; v[3] += x.w;
    v[4] += y.x; v[5] += y.y; v[6] += y.z; v[7] += y.w;
  }
  const float g = in && P.gamma ? P.gamma[c] : 1.f, be = in && P.beta ? P.beta[c] : 0.f;
  __shared__ __align__(16) float colsum[8];
  if (P.beta && threadIdx.x < 8) colsum[threadIdx.x] = j + (int)threadIdx.x < P.n ? P.colsum[j + threadIdx.x] : 0.f;
  __syncthreads();
  const int vec = store_width(P);
  if (vec > 1) {
    if (in) finish8(P, colsum, P.dw + (int64_t)c * P.lddw, j, g, be, vec, v);
    return;
  }
  // rows off 16 bytes: eight threads to a row's columns
  __shared__ float sm[kTile][9];
  if (in) affine8(P, colsum, g, be, v);
#pragma unroll
  for (int k = 0; k < 8; ++k) sm[threadIdx.x][k] = v[k];
  __syncthreads();
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    const int at = i * (kTile / 8) + threadIdx.x / 8, k = threadIdx.x % 8, row = c - threadIdx.x + at;
    if (row < P.cols && j + k < P.n) {
      float* d = P.dw + (int64_t)row * P.lddw + j + k;
      *d = P.accumulate ? *d + sm[at][k] : sm[at][k];
    }
  }
}

// dy's rows at an aligned pitch.  A thread makes eight elements, out of the two
// aligned pieces of 16 bytes that hold them, or by single ones where a piece
// would reach past the row's ends.  (By single elements throughout, 8192 x
// 4096 x 4096 took 348 us, 142 more than without the copy.)
__global__ void __launch_bounds__(256) ts_repack_kernel(const __nv_bfloat16* src, int64_t ld, int64_t rows, int n,
                                                        __nv_bfloat16* dst, int64_t pitch) {
  pdl_launch_dependents();
  pdl_wait();
  const int per_row = (int)(pitch / 8);
  const int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x, r = i / per_row;
  if (r >= rows) return;
  const int j = (int)(i - r * per_row) * 8;
  const __nv_bfloat16* s = src + r * ld + j;
  __nv_bfloat16* d = dst + r * pitch + j;
  const int off = (int)(reinterpret_cast<uintptr_t>(s) % 16 / 2);   // the same for all of a row
  if (j < off || j - off + 16 > n) {
    for (int k = 0; k < 8 && j + k < n; ++k) d[k] = s[k];
    return;
  }
  const uint4* q = reinterpret_cast<const uint4*>(s - off);
  const uint4 a = __ldcs(q), b = __ldcs(q + 1);
  uint32_t w[8] = {a.x, a.y, a.z, a.w, b.x, b.y, b.z, b.w};
  // the elements before the first one drop out: four, two and one of them
  if (off & 4) {
#pragma unroll
    for (int k = 0; k < 6; ++k) w[k] = w[k + 2];
  }
  if (off & 2) {
#pragma unroll
    for (int k = 0; k < 5; ++k) w[k] = w[k + 1];
  }
  if (off & 1) {
#pragma unroll
    for (int k = 0; k < 4; ++k) w[k] = __funnelshift_r(w[k], w[k + 1], 16);
  }
  *reinterpret_cast<uint4*>(d) = make_uint4(w[0], w[1], w[2], w[3]);
}

// dW of no tokens: beta's part is 0 too.
__global__ void __launch_bounds__(256) ts_zero_kernel(float* dw, int64_t lddw, int cols, int n) {
  pdl_launch_dependents();
  pdl_wait();
  for (int c = blockIdx.y; c < cols; c += gridDim.y)
    for (int64_t j = (int64_t)blockIdx.x * 256 + threadIdx.x; j < n; j += (int64_t)gridDim.x * 256)
      dw[c * lddw + j] = 0.f;
}

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

// The pairs that run at once on the device; also opts in to the shared memory.
cudaError_t resident_pairs(int device, int* out) {
  static std::atomic<int> cached[64];
  int n = device < 64 ? cached[device].load(std::memory_order_acquire) : 0;
  if (!n) {
    cudaError_t e = cudaFuncSetAttribute(ts_wgrad_kernel<true>, cudaFuncAttributeMaxDynamicSharedMemorySize, kSmem<true>);
    if (e != cudaSuccess) return e;
    e = cudaFuncSetAttribute(ts_wgrad_kernel<false>, cudaFuncAttributeMaxDynamicSharedMemorySize, kSmem<false>);
    if (e != cudaSuccess) return e;
    cudaLaunchConfig_t cfg = pdl_config(2, kThreads, kSmem<false>, nullptr);
    cudaLaunchAttribute at[1];
    at[0].id = cudaLaunchAttributeClusterDimension;
    at[0].val.clusterDim.x = 2;
    at[0].val.clusterDim.y = at[0].val.clusterDim.z = 1;
    cfg.attrs = at;
    cfg.numAttrs = 1;
    e = cudaOccupancyMaxActiveClusters(&n, ts_wgrad_kernel<false>, &cfg);
    if (e != cudaSuccess) return e;
    if (n < 1) return cudaErrorLaunchOutOfResources;
    if (device < 64) cached[device].store(n, std::memory_order_release);
  }
  *out = n;
  return cudaSuccess;
}

// The product over `rows` tokens of dy rows that TMA can read.
cudaError_t product(const ts_ops& h, WgradKernel& P, const TsCkpt& x, const TsMat& dy, int64_t rows, uint8_t* ws,
                    int64_t ws_bytes, cudaStream_t st) {
  EncodeFn enc = encoder();
  if (!enc) return cudaErrorNotSupported;
  const cuuint64_t dims[2] = {(cuuint64_t)P.n, (cuuint64_t)rows}, strides[1] = {(cuuint64_t)dy.ld * 2};
  const cuuint32_t box[2] = {64, kKB}, es[2] = {1, 1};
  if (enc(&P.dy, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 2, const_cast<void*>(dy.p), dims, strides, box, es,
          CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
          CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) != CUDA_SUCCESS)
    return cudaErrorInvalidValue;
  int pairs = 0;
  cudaError_t e = resident_pairs(h.device, &pairs);
  if (e != cudaSuccess) return e;
  P.x = x;
  P.rows = (int)rows;
  P.tiles_n = (P.n + kTile - 1) / kTile;
  const int tiles = (P.cols + kTile - 1) / kTile * P.tiles_n, nkb = (int)((rows + kKB - 1) / kKB);
  // partials of long sums, one a pair (a small workspace runs fewer pairs)
  const int64_t slots = ws_bytes / (kPieceFloats * 4);
  if (nkb > kChain) pairs = (int)std::min<int64_t>(pairs, std::max<int64_t>(slots, 1));
  P.full = tiles / pairs * pairs;
  const int rem = tiles - P.full;
  P.pieces = 1;
  if (rem) {
    const int64_t room = (slots - (nkb > kChain ? pairs : 0)) / rem;
    P.pieces = (int)std::max<int64_t>(1, std::min<int64_t>({pairs / rem, nkb / 4, room}));
  }
  P.items = P.full + P.pieces * rem;
  P.chain = reinterpret_cast<float4*>(ws);
  P.part = P.chain + (nkb > kChain ? pairs : 0) * (kPieceFloats / 4);
  const bool wide = store_width(P) > 1;
  cudaLaunchConfig_t cfg = pdl_config(2 * std::min(pairs, P.items), kThreads, wide ? kSmem<true> : kSmem<false>, st);
  cudaLaunchAttribute at[1];
  pdl_attr(cfg, at);
  e = cudaLaunchKernelEx(&cfg, wide ? ts_wgrad_kernel<true> : ts_wgrad_kernel<false>, P);
  if (e != cudaSuccess || P.pieces == 1) return e;
  cudaLaunchConfig_t fin = pdl_config(rem * 32, 256, 0, st);
  pdl_attr(fin, at);
  return cudaLaunchKernelEx(&fin, ts_wgrad_finish_kernel, P);
}

}  // namespace

cudaError_t launch_weight_grad(const ts_ops& h, const WgradArgs& a, cudaStream_t st) {
  cudaLaunchAttribute at[1];
  cudaError_t e;
  // dy's column sums: this call's own at the workspace's end, for beta
  const int64_t keep = a.beta ? ((int64_t)a.n * 4 + 255) / 256 * 256 : 0;
  int64_t room = h.ws_bytes - keep;
  float* colsum = keep ? reinterpret_cast<float*>(h.ws + room) : nullptr;
  const bool aligned = rows_aligned(a.dy);
  if ((colsum || a.db) && (aligned || a.rows == 0)) {
    e = launch_column_sums(h, a.dy, a.rows, a.n, colsum, a.db, a.accumulate, st);
    if (e != cudaSuccess) return e;
  }
  if (a.rows == 0) {
    if (a.accumulate) return cudaSuccess;
    cudaLaunchConfig_t cfg = pdl_config(1, 256, 0, st);
    cfg.gridDim = dim3((a.n + 255) / 256, std::min(a.cols, 1024));
    pdl_attr(cfg, at);
    return cudaLaunchKernelEx(&cfg, ts_zero_kernel, a.dw, a.lddw, a.cols, a.n);
  }
  WgradKernel P = {};
  P.cols = a.cols;
  P.n = a.n;
  P.gamma = a.gamma;
  P.beta = a.beta;
  P.colsum = colsum;
  P.dw = a.dw;
  P.lddw = a.lddw;
  P.accumulate = a.accumulate;
  P.err = h.err;
  P.wait_limit_ns = h.wait_limit_ns;
  P.inject = h.inject;
  if (aligned) return product(h, P, a.x, a.dy, a.rows, h.ws, room, st);
  // an aligned copy of as many tokens of dy as leave the column sums' room and
  // about half of the workspace; a call's whole work for each copy
  TsMat dy;
  dy.p = h.ws;
  dy.bf16 = 1;
  dy.ld = (a.n + 7) / 8 * 8;
  const int64_t most = std::max<int64_t>(1, (h.ws_bytes - 16 * (int64_t)a.n) / 16 * 9 / (dy.ld * 2));
  const int64_t times = (a.rows + most - 1) / most, each = (a.rows + times - 1) / times;
  for (int64_t t = 0; t < a.rows; t += each) {
    const int64_t rows = std::min(each, a.rows - t);
    cudaLaunchConfig_t cfg = pdl_config((int)((rows * (dy.ld / 8) + 255) / 256), 256, 0, st);
    pdl_attr(cfg, at);
    e = cudaLaunchKernelEx(&cfg, ts_repack_kernel, static_cast<const __nv_bfloat16*>(a.dy.p) + t * a.dy.ld, a.dy.ld,
                           rows, a.n, reinterpret_cast<__nv_bfloat16*>(h.ws), dy.ld);
    if (e != cudaSuccess) return e;
    const int64_t used = (rows * dy.ld * 2 + 255) / 256 * 256;
    if (colsum || a.db) {
      ts_ops rest = h;
      rest.ws += used;
      rest.ws_bytes -= used;
      e = launch_column_sums(rest, dy, rows, a.n, colsum, a.db, P.accumulate, st);
      if (e != cudaSuccess) return e;
    }
    TsCkpt x = a.x;
    x.q += t * x.pitch;
    x.scale += t * (x.pitch / kCkptBlock);
    e = product(h, P, x, dy, rows, h.ws + used, room - used, st);
    if (e != cudaSuccess) return e;
    P.accumulate = 1;   // the later tokens add to the first ones'
  }
  return cudaSuccess;
}

}  // namespace fg
