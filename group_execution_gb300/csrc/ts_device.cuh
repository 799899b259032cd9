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
// (Two 16-byte stores a lane leave gaps in each that the other fills; one of
// 32, where the address allows, takes layer norm of 8192 x 4096 f32 from 53 to
// 45 us and loading a checkpoint to f32 from 32 to 26.  HALVES keeps two, for
// kernels that have no register left for the choice.)
template <bool HALVES = false>
__device__ __forceinline__ void store8(float* p, const float (&v)[8]) {
  if (!HALVES && reinterpret_cast<uintptr_t>(p) % 32 == 0) {
    asm volatile("st.global.v8.f32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};" ::"l"(p), "f"(v[0]), "f"(v[1]), "f"(v[2]),
                 "f"(v[3]), "f"(v[4]), "f"(v[5]), "f"(v[6]), "f"(v[7])
                 : "memory");
    return;
  }
  reinterpret_cast<float4*>(p)[0] = make_float4(v[0], v[1], v[2], v[3]);
  reinterpret_cast<float4*>(p)[1] = make_float4(v[4], v[5], v[6], v[7]);
}
__device__ __forceinline__ uint32_t bf16x2(float lo, float hi) {
  const __nv_bfloat162 h = __floats2bfloat162_rn(lo, hi);
  return *reinterpret_cast<const uint32_t*>(&h);
}
template <bool HALVES = false>
__device__ __forceinline__ void store8(__nv_bfloat16* p, const float (&v)[8]) {
  *reinterpret_cast<uint4*>(p) = make_uint4(bf16x2(v[0], v[1]), bf16x2(v[2], v[3]), bf16x2(v[4], v[5]),
                                            bf16x2(v[6], v[7]));
}

// Two float32 values in one register pair: one instruction works on both.
using F2 = uint64_t;
__device__ __forceinline__ F2 pack2f(float a, float b) {
  F2 r;
  asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "f"(a), "f"(b));
  return r;
}
__device__ __forceinline__ void unpack2f(F2 v, float& a, float& b) {
  asm("mov.b64 {%0, %1}, %2;" : "=f"(a), "=f"(b) : "l"(v));
}
__device__ __forceinline__ F2 fma2(F2 a, F2 b, F2 c) {
  F2 r;
  asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r) : "l"(a), "l"(b), "l"(c));
  return r;
}
__device__ __forceinline__ F2 mul2(F2 a, F2 b) {
  F2 r;
  asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
  return r;
}
__device__ __forceinline__ F2 add2(F2 a, F2 b) {
  F2 r;
  asm("add.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
  return r;
}
__device__ __forceinline__ float sum2(F2 v) {
  float a, b;
  unpack2f(v, a, b);
  return a + b;
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
template <bool VEC, bool HALVES = false, class T>
__device__ __forceinline__ void store_group(T* p, int c0, int cols, int lane, const float (&v)[8]) {
  if (VEC && c0 + lane * 8 + 8 <= cols) {
    store8<HALVES>(p + c0 + lane * 8, v);
  } else {
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      const int c = c0 + group_col<VEC>(lane, j);
      if (c < cols) p[c] = from_f32<T>(v[j]);
    }
  }
}

// A group of a row as it lies in memory, fetched some time before it is used.
// Columns at or past `cols` are zeros.
template <class T, bool VEC>
struct RawGroup;
template <class T>
struct RawGroup<T, false> {
  T e[8];
  __device__ __forceinline__ void load(const T* p, int c0, int cols, int lane) {
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      const int c = c0 + j * 32 + lane;
      e[j] = c < cols ? p[c] : from_f32<T>(0.f);
    }
  }
  __device__ __forceinline__ void get(float (&v)[8]) const {
#pragma unroll
    for (int j = 0; j < 8; ++j) v[j] = to_f32(e[j]);
  }
};
template <class T>
struct RawGroup<T, true> {
  static constexpr int kQuads = sizeof(T) / 2;   // 16-byte quads of eight values
  uint4 q[kQuads];
  __device__ __forceinline__ void load(const T* p, int c0, int cols, int lane) {
    const int c = c0 + lane * 8;
    if (c + 8 <= cols) {
#pragma unroll
      for (int i = 0; i < kQuads; ++i) q[i] = reinterpret_cast<const uint4*>(p + c)[i];
    } else {
      __align__(16) T e[8];
#pragma unroll
      for (int j = 0; j < 8; ++j) e[j] = c + j < cols ? p[c + j] : from_f32<T>(0.f);
#pragma unroll
      for (int i = 0; i < kQuads; ++i) q[i] = reinterpret_cast<const uint4*>(e)[i];
    }
  }
  __device__ __forceinline__ void get(float (&v)[8]) const {
    if constexpr (sizeof(T) == 4) {
      const uint32_t u[8] = {q[0].x, q[0].y, q[0].z, q[0].w, q[kQuads - 1].x, q[kQuads - 1].y, q[kQuads - 1].z, q[kQuads - 1].w};
#pragma unroll
      for (int j = 0; j < 8; ++j) v[j] = __uint_as_float(u[j]);
    } else {
      const uint32_t u[4] = {q[0].x, q[0].y, q[0].z, q[0].w};
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        v[2 * j] = __uint_as_float(u[j] << 16);
        v[2 * j + 1] = __uint_as_float(u[j] & 0xffff0000u);
      }
    }
  }
};
__device__ __forceinline__ float warp_sum(float v) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
  return v;
}

// ---- 8-bit checkpoints ------------------------------------------------------
// A block's scale byte E is the exponent field of its largest magnitude, at
// least 7 so that the step 2^(E - 133) is a normal float; 255 marks a block
// that holds an infinity or a NaN.
__device__ __forceinline__ float ckpt_step(uint32_t e) {
  return e < 255 ? __uint_as_float((e - 6) << 23) : __uint_as_float(0x7fc00000u);
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
// up to the pitch) of checkpoint row `r`.  Without VEC the warp's values
// change places in `scratch`, 256 floats of its own, first: a lane then has
// eight columns that lie together, as with VEC (a byte at a time, and a block's
// maximum over the whole warp, saving 8192 x 4096 bf16 at odd elements took 43 us
// in place of 31).
template <bool VEC>
__device__ __forceinline__ void ckpt_store_group(const TsCkpt& c, int64_t r, int c0, int lane, const float (&v)[8],
                                                 float* scratch) {
  float x[8];
  if (VEC) {
#pragma unroll
    for (int j = 0; j < 8; ++j) x[j] = v[j];
  } else {
#pragma unroll
    for (int j = 0; j < 8; ++j) scratch[j * 32 + lane] = v[j];
    __syncwarp();
    load8(scratch + lane * 8, x);
    __syncwarp();
  }
  uint32_t m = 0;
#pragma unroll
  for (int j = 0; j < 8; ++j) m = max(m, __float_as_uint(x[j]) & 0x7fffffffu);
  const unsigned quad = 0xfu << (threadIdx.x & 28);   // (half warps may be in different rows)
  m = max(m, __shfl_xor_sync(quad, m, 1));
  m = max(m, __shfl_xor_sync(quad, m, 2));
  const int e = max((int)(m >> 23), 7);
  const float inv = ckpt_inv_step(e);
  uint32_t w[2] = {0, 0};
#pragma unroll
  for (int j = 0; j < 8; ++j) w[j >> 2] |= (uint32_t)(ckpt_quantise(x[j], inv) & 0xff) << (8 * (j & 3));
  const int col = c0 + lane * 8;
  if (col < c.pitch) {
    *reinterpret_cast<uint2*>(c.q + r * c.pitch + col) = make_uint2(w[0], w[1]);
    if ((lane & 3) == 0) c.scale[r * (c.pitch / kCkptBlock) + col / kCkptBlock] = (uint8_t)e;
  }
}

// A group of a checkpoint row, fetched some time before it is used: eight
// columns that lie together to a lane.  Without VEC its bytes change places in
// `scratch`, 256 bytes of the warp's own, when they are used (loaded one by
// one, 8192 x 4096 from a checkpoint to bf16 rows at odd elements took 32 us in
// place of 28).
template <bool VEC>
struct RawCkpt {
  uint2 q;
  uint32_t e[VEC ? 1 : 2];   // the eight columns' scale byte, or all eight of the group (a row's are a multiple of 4)
  __device__ __forceinline__ void load(const TsCkpt& c, int64_t r, int c0, int lane) {
    const int col = c0 + lane * 8;
    const uint8_t* s = c.scale + r * (c.pitch / kCkptBlock);
    q = col < c.pitch ? *reinterpret_cast<const uint2*>(c.q + r * c.pitch + col) : make_uint2(0, 0);
    if constexpr (VEC) {
      e[0] = col < c.pitch ? s[col / kCkptBlock] : 7;
    } else {
#pragma unroll
      for (int i = 0; i < 2; ++i)
        e[i] = c0 + i * 128 < c.pitch ? *reinterpret_cast<const uint32_t*>(s + c0 / kCkptBlock + 4 * i) : 0x07070707u;
    }
  }
  __device__ __forceinline__ void get(float (&v)[8], int lane, int8_t* scratch) const {
    if constexpr (VEC) {
      const float step = ckpt_step(e[0]);
#pragma unroll
      for (int j = 0; j < 8; ++j) v[j] = (float)(int8_t)((j < 4 ? q.x : q.y) >> (8 * (j & 3))) * step;
    } else {
      *reinterpret_cast<uint2*>(scratch + lane * 8) = q;
      __syncwarp();
#pragma unroll
      for (int j = 0; j < 8; ++j)
        v[j] = (float)scratch[j * 32 + lane] * ckpt_step((e[j / 4] >> (8 * (j & 3))) & 0xffu);
      __syncwarp();
    }
  }
};
// The scratch of a block's WARPS for it.
template <bool NEEDED, int WARPS>
struct CkptScratch {
  int8_t bytes[NEEDED ? WARPS : 1][kGroupCols];
  __device__ __forceinline__ int8_t* mine() { return bytes[NEEDED ? threadIdx.x >> 5 : 0]; }
};

}  // namespace fg
