// Device code the training-step operators share: typed loads and stores of
// eight values a thread, reductions in a fixed order, and the 8-bit
// checkpoint's encoding.
#pragma once
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include <cstdint>

#include "fg_device.cuh"
#include "ts.h"

namespace fg {

__device__ __forceinline__ float to_f32(float v) { return v; }
__device__ __forceinline__ float to_f32(__nv_bfloat16 v) { return __bfloat162float(v); }
template <class T>
__device__ __forceinline__ T from_f32(float v);
template <>
__device__ __forceinline__ float from_f32<float>(float v) {
  return v;
}
template <>
__device__ __forceinline__ __nv_bfloat16 from_f32<__nv_bfloat16>(float v) {
  return __float2bfloat16_rn(v);
}

// Eight consecutive values at a 16-byte aligned address.
__device__ __forceinline__ void load8(const float* p, float (&v)[8]) {
  const float4 a = *reinterpret_cast<const float4*>(p), b = *reinterpret_cast<const float4*>(p + 4);
  v[0] = a.x; v[1] = a.y; v[2] = a.z; v[3] = a.w;
  v[4] = b.x; v[5] = b.y; v[6] = b.z; v[7] = b.w;
}
__device__ __forceinline__ void load8(const __nv_bfloat16* p, float (&v)[8]) {
  const uint4 a = *reinterpret_cast<const uint4*>(p);
  const uint32_t w[4] = {a.x, a.y, a.z, a.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    v[2 * i] = __uint_as_float(w[i] << 16);
    v[2 * i + 1] = __uint_as_float(w[i] & 0xffff0000u);
  }
}
__device__ __forceinline__ void store8(float* p, const float (&v)[8]) {
  reinterpret_cast<float4*>(p)[0] = make_float4(v[0], v[1], v[2], v[3]);
  reinterpret_cast<float4*>(p)[1] = make_float4(v[4], v[5], v[6], v[7]);
}
__device__ __forceinline__ uint32_t bf16x2(float lo, float hi) {
  const __nv_bfloat162 h = __floats2bfloat162_rn(lo, hi);
  return *reinterpret_cast<const uint32_t*>(&h);
}
__device__ __forceinline__ void store8(__nv_bfloat16* p, const float (&v)[8]) {
  *reinterpret_cast<uint4*>(p) = make_uint4(bf16x2(v[0], v[1]), bf16x2(v[2], v[3]), bf16x2(v[4], v[5]),
                                            bf16x2(v[6], v[7]));
}

// A warp works on groups of 256 columns of one row, eight values a lane.  VEC
// (every row of every operand starts on 16 bytes): a lane's eight columns are
// consecutive and move in 16-byte accesses.  Otherwise value j of a lane is
// column j * 32 + lane, so that single-element accesses are consecutive
// across the warp.  Either way a block of 32 columns (a checkpoint's scale)
// lies within the warp: four lanes, or one value of all lanes.
constexpr int kGroupCols = 256;

template <bool VEC>
__device__ __forceinline__ int group_col(int lane, int j) {
  return VEC ? lane * 8 + j : j * 32 + lane;
}
// Values of the group of row `p` that starts at column c0; columns at or past
// `cols` read as 0.
template <bool VEC, class T>
__device__ __forceinline__ void load_group(const T* p, int c0, int cols, int lane, float (&v)[8]) {
  if (VEC && c0 + lane * 8 + 8 <= cols) {
    load8(p + c0 + lane * 8, v);
  } else {
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      const int c = c0 + group_col<VEC>(lane, j);
      v[j] = c < cols ? to_f32(p[c]) : 0.f;
    }
  }
}
template <bool VEC, class T>
__device__ __forceinline__ void store_group(T* p, int c0, int cols, int lane, const float (&v)[8]) {
  if (VEC && c0 + lane * 8 + 8 <= cols) {
    store8(p + c0 + lane * 8, v);
  } else {
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      const int c = c0 + group_col<VEC>(lane, j);
      if (c < cols) p[c] = from_f32<T>(v[j]);
    }
  }
}

__device__ __forceinline__ float warp_sum(float v) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
  return v;
}

// ---- 8-bit checkpoints ------------------------------------------------------
// A block's scale byte E is the exponent field of its largest magnitude, at
// least 7 so that the step 2^(E - 133) is a normal float; 255 marks a block
// that holds an infinity or a NaN.
__device__ __forceinline__ float ckpt_step(int e) {
  return e < 255 ? __uint_as_float((uint32_t)(e - 6) << 23) : __uint_as_float(0x7fc00000u);
}
// 1 / step, or 0 where the block is marked (its values are then stored as 0).
__device__ __forceinline__ float ckpt_inv_step(int e) {
  return e < 255 ? __uint_as_float((uint32_t)(260 - e) << 23) : 0.f;
}
// Dividing by the step is exact (a power of two), so the one rounding is to
// the nearest integer, ties to even.
__device__ __forceinline__ int ckpt_quantise(float v, float inv) {
  const int q = __float2int_rn(v * inv);   // NaN gives 0
  return q < -127 ? -127 : q > 127 ? 127 : q;
}

// Writes this warp's group (columns from c0, those at or past cols as zeros,
// up to the pitch) of checkpoint row `r`.
template <bool VEC>
__device__ __forceinline__ void ckpt_store_group(const TsCkpt& c, int64_t r, int c0, int lane, const float (&v)[8]) {
  int8_t* q = c.q + r * c.pitch;
  uint8_t* s = c.scale + r * (c.pitch / kCkptBlock);
  if (VEC) {
    uint32_t m = 0;
#pragma unroll
    for (int j = 0; j < 8; ++j) m = max(m, __float_as_uint(v[j]) & 0x7fffffffu);
    m = max(m, __shfl_xor_sync(0xffffffffu, m, 1));
    m = max(m, __shfl_xor_sync(0xffffffffu, m, 2));
    const int e = max((int)(m >> 23), 7);
    const float inv = ckpt_inv_step(e);
    uint32_t w[2] = {0, 0};
#pragma unroll
    for (int j = 0; j < 8; ++j) w[j >> 2] |= (uint32_t)(ckpt_quantise(v[j], inv) & 0xff) << (8 * (j & 3));
    const int col = c0 + lane * 8;
    if (col < c.pitch) {
      *reinterpret_cast<uint2*>(q + col) = make_uint2(w[0], w[1]);
      if ((lane & 3) == 0) s[col / kCkptBlock] = (uint8_t)e;
    }
  } else {
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      const uint32_t m = __reduce_max_sync(0xffffffffu, __float_as_uint(v[j]) & 0x7fffffffu);
      const int e = max((int)(m >> 23), 7);
      const int col = c0 + j * 32 + lane;
      if (col < c.pitch) {
        q[col] = (int8_t)ckpt_quantise(v[j], ckpt_inv_step(e));
        if (lane == 0) s[col / kCkptBlock] = (uint8_t)e;
      }
    }
  }
}

// The values of this warp's group of checkpoint row `r`; 0 past the pitch.
template <bool VEC>
__device__ __forceinline__ void ckpt_load_group(const TsCkpt& c, int64_t r, int c0, int lane, float (&v)[8]) {
  const int8_t* q = c.q + r * c.pitch;
  const uint8_t* s = c.scale + r * (c.pitch / kCkptBlock);
  if (VEC) {
    const int col = c0 + lane * 8;
    if (col < c.pitch) {
      const uint2 w = *reinterpret_cast<const uint2*>(q + col);
      const float step = ckpt_step(s[col / kCkptBlock]);
#pragma unroll
      for (int j = 0; j < 8; ++j)
        v[j] = (float)(int8_t)((j < 4 ? w.x : w.y) >> (8 * (j & 3))) * step;
    } else {
#pragma unroll
      for (int j = 0; j < 8; ++j) v[j] = 0.f;
    }
  } else {
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      const int col = c0 + j * 32 + lane;
      v[j] = col < c.pitch ? (float)q[col] * ckpt_step(s[col / kCkptBlock]) : 0.f;
    }
  }
}

}  // namespace fg
