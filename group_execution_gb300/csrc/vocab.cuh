// What the kernels of the cross entropy over a vocabulary share: copies of bf16
// rows, exponentials, and the launch of the kernels for few rows.
#pragma once
#include "ts_device.cuh"

namespace fg {

constexpr float kLog2e = 1.4426950408889634f;

// Rows of bf16 that are copied to a pitch that TMA can read.  Rows that take no
// gradient (without a target, or of an lse of -inf) have d = 0 and may hold
// anything: where targets or lse are given, the copy has them as zeros.
struct CopyRows {
  const __nv_bfloat16* src;
  __nv_bfloat16* dst;
  int64_t ld, pitch, vocab, units;   // a unit: eight columns of a row
  int cols;
  const int64_t* targets;
  const float* lse;
};

__device__ __forceinline__ float exp2_approx(float v) {
  float r;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(v));
  return r;
}
// A row's logits so far: the largest, m, and s = sum of exp(l - m).  Adds others'.
__device__ __forceinline__ void join_sums(float& m, float& s, float m2, float s2) {
  const float next = fmaxf(m, m2), ref = next == -INFINITY ? 0.f : next;
  s = s * exp2_approx((m - ref) * kLog2e) + s2 * exp2_approx((m2 - ref) * kLog2e);
  m = next;
}
// lse and the target's loss.  The loss is not lse - logit: lse is rounded at the
// size of the logits, while m - logit is exact where they are close, and log s is
// never negative (the largest logit's term is 1).
__device__ __forceinline__ float lse_of(float m, float s) { return s == 0.f ? -INFINITY : m + logf(s); }
__device__ __forceinline__ float loss_of(float m, float s, float logit) {
  return s == 0.f ? INFINITY : (m - logit) + logf(s);
}
// Eight elements of a row from column j on, zeros past `cols`: out of the two
// aligned pieces of 16 bytes that hold them, or one by one where those would
// reach past the row's ends.
__device__ __forceinline__ uint4 row_piece(const __nv_bfloat16* row, int j, int cols) {
  const __nv_bfloat16* s = row + j;
  const int off = (int)(reinterpret_cast<uintptr_t>(s) % 16 / 2);   // the same for all of a row
  if (off == 0 && j + 8 <= cols) return __ldcs(reinterpret_cast<const uint4*>(s));
  if (j < off || j - off + 16 > cols) {
    __align__(16) __nv_bfloat16 e[8];
#pragma unroll
    for (int k = 0; k < 8; ++k) e[k] = j + k < cols ? s[k] : from_f32<__nv_bfloat16>(0.f);
    return *reinterpret_cast<const uint4*>(e);
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
  return make_uint4(w[0], w[1], w[2], w[3]);
}
// Copies the rows, 16 bytes a thread: thread `t` of `n`, U pieces in flight.
template <int U>
__device__ __forceinline__ void copy_rows(const CopyRows& C, int64_t t, int64_t n) {
  const int per = (int)(C.pitch / 8);
  for (int64_t u0 = t; u0 < C.units; u0 += U * n) {
    uint4 v[U];
#pragma unroll
    for (int k = 0; k < U; ++k) {
      const int64_t u = u0 + k * n, r = u / per;
      if (u >= C.units) break;
      bool keep = true;
      if (C.targets) {
        const int64_t i = C.targets[r];
        keep = i >= 0 && i < C.vocab;
      }
      if (C.lse && C.lse[r] == -INFINITY) keep = false;
      v[k] = row_piece(C.src + r * C.ld, (int)(u - r * per) * 8, keep ? C.cols : 0);
    }
#pragma unroll
    for (int k = 0; k < U; ++k) {
      const int64_t u = u0 + k * n;
      if (u >= C.units) break;
      reinterpret_cast<uint4*>(C.dst)[u] = v[k];   // (the copy's rows lie together)
    }
  }
}

// The logits of few rows of small weights (k_vocab_few.cu).  Forward, us in a
// graph, there and by the tiles of 256 (k_vocab_loss.cu): 16 rows, 4000 x 1024 10
// and 11, 8000 x 1024 12.5 and 11.5; one row 7 and 11, 9.5 and 11.5, and 32000 x
// 1024 21.5 and 19.
constexpr int kFewRows = 16;
inline bool few_rows(const VocabLossArgs& a) {
  return a.rows <= kFewRows && a.vocab * a.cols <= (a.rows == 1 ? 8 : 5) * int64_t(1 << 20);
}
// Forward: loss and lse.  (1 MiB of workspace is enough.)
cudaError_t launch_few_loss(const ts_ops& h, const VocabLossArgs& a, cudaStream_t st);
// Backward: d [rows, dpitch] of the whole vocabulary, and the copy that C describes.
cudaError_t launch_few_dlogits(const ts_ops& h, const VocabLossArgs& a, const CopyRows& C, __nv_bfloat16* d,
                               int64_t dpitch, cudaStream_t st);

}  // namespace fg
