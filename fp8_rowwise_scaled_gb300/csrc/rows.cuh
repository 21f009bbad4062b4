// rows.cuh -- device helpers of the row-wise operators (norm, routing, dispatch, combine,
// SwiGLU): eight elements at a time between memory and fp32 registers, packing to e4m3, and
// reductions over a warp or a CTA.
#pragma once

#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>

#include <cstdint>

#include "ptx.cuh"

namespace mslkb {

constexpr float kE4m3Max = 448.f;
// a row or block whose largest magnitude is below this (2^-80) is stored as zeros, scale 1:
// its 448 / amax would come near the end of fp32's range
constexpr float kQuantTiny = 8.271806125530277e-25f;
constexpr int kScaleBlock = 128;  // columns per scale of the block-scaled layouts

// Plain (coherent) global accesses: an output may be the same buffer as an input.
__device__ __forceinline__ uint4 load16(const void* p) {
  return *reinterpret_cast<const uint4*>(p);
}
__device__ __forceinline__ void store16(void* p, uint4 v) { *reinterpret_cast<uint4*>(p) = v; }

__device__ __forceinline__ float to_float(__nv_bfloat16 v) { return __bfloat162float(v); }
__device__ __forceinline__ float to_float(__half v) { return __half2float(v); }
__device__ __forceinline__ float to_float(float v) { return v; }

template <class T>
__device__ __forceinline__ T from_float(float v);
template <>
__device__ __forceinline__ __nv_bfloat16 from_float<__nv_bfloat16>(float v) {
  return __float2bfloat16_rn(v);
}
template <>
__device__ __forceinline__ __half from_float<__half>(float v) {
  return __float2half_rn(v);
}
template <>
__device__ __forceinline__ float from_float<float>(float v) {
  return v;
}

// Two 16-bit floats of one word, the lower half first.
__device__ __forceinline__ float2 unpack2(uint32_t w, __nv_bfloat16) {
  return make_float2(__uint_as_float(w << 16), __uint_as_float(w & 0xFFFF0000u));
}
__device__ __forceinline__ float2 unpack2(uint32_t w, __half) {
  __half2_raw r;
  r.x = static_cast<unsigned short>(w & 0xFFFFu);
  r.y = static_cast<unsigned short>(w >> 16);
  return __half22float2(__half2(r));
}
__device__ __forceinline__ uint32_t pack2(float a, float b, __nv_bfloat16) {
  const __nv_bfloat162_raw r = __floats2bfloat162_rn(a, b);
  return static_cast<uint32_t>(r.x) | (static_cast<uint32_t>(r.y) << 16);
}
__device__ __forceinline__ uint32_t pack2(float a, float b, __half) {
  const __half2_raw r = __floats2half2_rn(a, b);
  return static_cast<uint32_t>(r.x) | (static_cast<uint32_t>(r.y) << 16);
}

// Eight consecutive elements as loaded (kept packed until they are used).
template <class T>
struct Raw8 {
  uint4 w[sizeof(T) / 2];
};

template <class T>
__device__ __forceinline__ void unpack8(const Raw8<T>& r, float (&v)[8]) {
  if constexpr (sizeof(T) == 4) {
    v[0] = __uint_as_float(r.w[0].x), v[1] = __uint_as_float(r.w[0].y);
    v[2] = __uint_as_float(r.w[0].z), v[3] = __uint_as_float(r.w[0].w);
    v[4] = __uint_as_float(r.w[1].x), v[5] = __uint_as_float(r.w[1].y);
    v[6] = __uint_as_float(r.w[1].z), v[7] = __uint_as_float(r.w[1].w);
  } else {
    const uint32_t w[4] = {r.w[0].x, r.w[0].y, r.w[0].z, r.w[0].w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const float2 f = unpack2(w[i], T());
      v[2 * i] = f.x;
      v[2 * i + 1] = f.y;
    }
  }
}

template <class T>
__device__ __forceinline__ Raw8<T> pack8(const float (&v)[8]) {
  Raw8<T> r;
  if constexpr (sizeof(T) == 4) {
    r.w[0] = make_uint4(__float_as_uint(v[0]), __float_as_uint(v[1]), __float_as_uint(v[2]),
                        __float_as_uint(v[3]));
    r.w[1] = make_uint4(__float_as_uint(v[4]), __float_as_uint(v[5]), __float_as_uint(v[6]),
                        __float_as_uint(v[7]));
  } else {
    r.w[0] = make_uint4(pack2(v[0], v[1], T()), pack2(v[2], v[3], T()), pack2(v[4], v[5], T()),
                        pack2(v[6], v[7], T()));
  }
  return r;
}

// Elements [c, c + 8) of a row of n elements; kWide: the row is 16-byte aligned and n a
// multiple of 8.  Past the row's end: zeros, nothing read.
template <class T, bool kWide>
__device__ __forceinline__ Raw8<T> load8(const T* row, int c, int n) {
  Raw8<T> r;
  if constexpr (kWide) {
#pragma unroll
    for (int i = 0; i < static_cast<int>(sizeof(T) / 2); ++i)
      r.w[i] = c < n ? load16(row + c + i * (16 / sizeof(T))) : make_uint4(0, 0, 0, 0);
  } else {
    float v[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) v[i] = c + i < n ? to_float(row[c + i]) : 0.f;
    r = pack8<T>(v);  // exact: the values came from T
  }
  return r;
}

template <class T, bool kWide>
__device__ __forceinline__ void store8(T* row, int c, int n, const float (&v)[8]) {
  if constexpr (kWide) {
    if (c < n) {
      const Raw8<T> r = pack8<T>(v);
#pragma unroll
      for (int i = 0; i < static_cast<int>(sizeof(T) / 2); ++i)
        store16(row + c + i * (16 / sizeof(T)), r.w[i]);
    }
  } else {
#pragma unroll
    for (int i = 0; i < 8; ++i)
      if (c + i < n) row[c + i] = from_float<T>(v[i]);
  }
}

// Four values to four e4m3 codes, the first in the lowest byte; past +-448 saturates, NaN
// stays NaN.
__device__ __forceinline__ uint32_t pack_e4m3x4(float a, float b, float c, float d) {
  uint16_t lo, hi;
  asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(lo) : "f"(b), "f"(a));
  asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(hi) : "f"(d), "f"(c));
  return static_cast<uint32_t>(lo) | (static_cast<uint32_t>(hi) << 16);
}

// Two e4m3 codes (low byte first) to floats: exact, e4m3 is a subset of fp16.
__device__ __forceinline__ float2 unpack_e4m3x2(uint16_t codes) {
  uint32_t h;
  asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(h) : "h"(codes));
  return unpack2(h, __half());
}

__device__ __forceinline__ void unpack_e4m3x8(uint2 codes, float (&v)[8]) {
  const uint32_t w[2] = {codes.x, codes.y};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const float2 f = unpack_e4m3x2(static_cast<uint16_t>(w[i / 2] >> (16 * (i & 1))));
    v[2 * i] = f.x;
    v[2 * i + 1] = f.y;
  }
}

// Codes [c, c + 8) of a row of n codes (kWide: 8-byte aligned rows, n a multiple of 8).
template <bool kWide>
__device__ __forceinline__ void store_codes8(uint8_t* row, int c, int n, uint2 codes) {
  if constexpr (kWide) {
    if (c < n) *reinterpret_cast<uint2*>(row + c) = codes;
  } else {
#pragma unroll
    for (int i = 0; i < 8; ++i)
      if (c + i < n)
        row[c + i] = static_cast<uint8_t>((i < 4 ? codes.x : codes.y) >> (8 * (i & 3)));
  }
}

// Magnitudes are compared as the bit patterns of |v|: the order of the floats, with NaN
// above infinity, so that a NaN is never lost in a maximum.
__device__ __forceinline__ uint32_t abs_bits(float v) { return __float_as_uint(v) & 0x7FFFFFFFu; }

__device__ __forceinline__ uint32_t abs_max8(const float (&v)[8]) {
  uint32_t m = abs_bits(v[0]);
#pragma unroll
  for (int i = 1; i < 8; ++i) m = max(m, abs_bits(v[i]));
  return m;
}

__device__ __forceinline__ float warp_sum(float v) {
#pragma unroll
  for (int d = 16; d > 0; d >>= 1) v += __shfl_xor_sync(0xFFFFFFFFu, v, d);
  return v;
}

// over the 16 lanes that share a block of 128 columns (eight per lane)
__device__ __forceinline__ uint32_t block16_max(uint32_t m) {
#pragma unroll
  for (int d = 8; d > 0; d >>= 1) m = max(m, __shfl_xor_sync(0xFFFFFFFFu, m, d));
  return m;
}

// The scale of a row or block whose largest magnitude is `amax`, and the factor from values
// to codes; zeros below kQuantTiny (a NaN amax is not below it and stays).
struct QuantScale {
  float scale, inv;
};
__device__ __forceinline__ QuantScale quant_scale(float amax) {
  QuantScale q;
  const bool zero = amax < kQuantTiny;
  q.scale = zero ? 1.f : amax / kE4m3Max;
  q.inv = zero ? 0.f : kE4m3Max / amax;
  return q;
}

__device__ __forceinline__ uint2 quantize8(const float (&v)[8], float inv) {
  return make_uint2(pack_e4m3x4(v[0] * inv, v[1] * inv, v[2] * inv, v[3] * inv),
                    pack_e4m3x4(v[4] * inv, v[5] * inv, v[6] * inv, v[7] * inv));
}

}  // namespace mslkb
