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

// How a thread reaches eight or sixteen columns of a row of n, named by c, a multiple of their
// number; past the row's end nothing is touched and zeros are read.
//   k32       columns [c, c + 16) in 32-byte pieces: aligned rows, n a multiple of 16
//   k16       columns [c, c + 8) in 16-byte pieces: aligned rows, n a multiple of 8
//   kElement  columns [c, c + 8) one by one
//   kStride   one by one, a warp's 256 columns dealt to its lanes in turn, so that each access
//             of the warp is one run of 32 elements (its threads name consecutive c)
enum class Access { kElement, kStride, k16, k32 };

template <Access kAccess>
__device__ __forceinline__ int element(int c, int j) {
  return kAccess == Access::kStride ? (c & ~255) + j * 32 + ((c >> 3) & 31) : c + j;
}

template <class T, Access kAccess>
__device__ __forceinline__ Raw8<T> load8(const T* row, int c, int n) {
  Raw8<T> r;
  if constexpr (kAccess == Access::k16 || kAccess == Access::k32) {
#pragma unroll
    for (int i = 0; i < static_cast<int>(sizeof(T) / 2); ++i)
      r.w[i] = c < n ? load16(row + c + i * (16 / sizeof(T))) : make_uint4(0, 0, 0, 0);
  } else {
    float v[8];
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      const int e = element<kAccess>(c, j);
      v[j] = e < n ? to_float(row[e]) : 0.f;
    }
    r = pack8<T>(v);  // exact: the values came from T
  }
  return r;
}

template <class T, Access kAccess>
__device__ __forceinline__ void store8(T* row, int c, int n, const float (&v)[8]) {
  if constexpr (kAccess == Access::k16 || kAccess == Access::k32) {
    if (c < n) {
      const Raw8<T> r = pack8<T>(v);
#pragma unroll
      for (int i = 0; i < static_cast<int>(sizeof(T) / 2); ++i)
        store16(row + c + i * (16 / sizeof(T)), r.w[i]);
    }
  } else {
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      const int e = element<kAccess>(c, j);
      if (e < n) row[e] = from_float<T>(v[j]);
    }
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

// The larger of two or three, NaN if one of them is.
__device__ __forceinline__ float max_nan(float a, float b) {
  float m;
  asm("max.NaN.f32 %0, %1, %2;" : "=f"(m) : "f"(a), "f"(b));
  return m;
}
__device__ __forceinline__ float max_nan(float a, float b, float c) {
  float m;
  asm("max.NaN.f32 %0, %1, %2, %3;" : "=f"(m) : "f"(a), "f"(b), "f"(c));
  return m;
}
// Largest magnitude, as the bit pattern of |v|: integers in the order of the floats with NaN
// above infinity, so that a NaN is never lost in a maximum.
template <int kN>
__device__ __forceinline__ uint32_t abs_max(const float (&v)[kN]) {
  static_assert(kN % 2 == 0, "pairs");
  float m = max_nan(fabsf(v[0]), fabsf(v[1]));
#pragma unroll
  for (int i = 2; i < kN; i += 2) m = max_nan(m, fabsf(v[i]), fabsf(v[i + 1]));
  return __float_as_uint(m);
}

__device__ __forceinline__ float warp_sum(float v) {
#pragma unroll
  for (int d = 16; d > 0; d >>= 1) v += __shfl_xor_sync(0xFFFFFFFFu, v, d);
  return v;
}

// over the kLanes lanes that share a block of 128 columns
template <int kLanes>
__device__ __forceinline__ uint32_t block_max(uint32_t m) {
#pragma unroll
  for (int d = kLanes / 2; d > 0; d >>= 1) m = max(m, __shfl_xor_sync(0xFFFFFFFFu, m, d));
  return m;
}

// 1 / x to one ulp for 2^-126 <= x <= 2^126 (0 and NaN as IEEE), one instruction
__device__ __forceinline__ float recip(float x) {
  float r;
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(x));
  return r;
}

// The scale of values whose largest magnitude is `amax`, and the factor from `u` to codes,
// where u are the values divided by a common factor and `u_max` their largest magnitude
// (values that are not scaled: u_max = amax).  Zeros below kQuantTiny; a NaN amax is not
// below it and stays.  Two roundings and recip's ulp: 4 u in all; the 1/16 keeps recip's
// argument and result normal up to the largest float.
struct QuantScale {
  float scale, inv;
};
__device__ __forceinline__ QuantScale quant_scale(float amax, float u_max) {
  QuantScale q;
  const bool zero = amax < kQuantTiny;
  q.scale = zero ? 1.f : amax * (1.f / kE4m3Max);
  q.inv = zero ? 0.f : (kE4m3Max / 16) * recip(u_max * 0.0625f);
  return q;
}

__device__ __forceinline__ uint2 quantize8(const float (&v)[8], float inv) {
  return make_uint2(pack_e4m3x4(v[0] * inv, v[1] * inv, v[2] * inv, v[3] * inv),
                    pack_e4m3x4(v[4] * inv, v[5] * inv, v[6] * inv, v[7] * inv));
}

// ---------------------------------------------------------------------------------
// kCols columns per thread: 16 with Access::k32, else 8
// ---------------------------------------------------------------------------------
struct Words8 {
  uint32_t w[8];
};
__device__ __forceinline__ Words8 load32(const void* p) {
  Words8 r;
  asm volatile("ld.global.v8.b32 {%0, %1, %2, %3, %4, %5, %6, %7}, [%8];"
               : "=r"(r.w[0]), "=r"(r.w[1]), "=r"(r.w[2]), "=r"(r.w[3]), "=r"(r.w[4]),
                 "=r"(r.w[5]), "=r"(r.w[6]), "=r"(r.w[7])
               : "l"(p)
               : "memory");
  return r;
}
__device__ __forceinline__ void store32(void* p, const Words8& r) {
  asm volatile("st.global.v8.b32 [%8], {%0, %1, %2, %3, %4, %5, %6, %7};" ::"r"(r.w[0]),
               "r"(r.w[1]), "r"(r.w[2]), "r"(r.w[3]), "r"(r.w[4]), "r"(r.w[5]), "r"(r.w[6]),
               "r"(r.w[7]), "l"(p)
               : "memory");
}

template <class T, int kCols, Access kAccess>
__device__ __forceinline__ void load_cols(const T* row, int c, int n, float (&v)[kCols]) {
  if constexpr (kAccess == Access::k32) {
    static_assert(kCols == 16, "32-byte accesses take 16 columns");
    constexpr int kEach = 32 / sizeof(T);
#pragma unroll
    for (int k = 0; k < kCols / kEach; ++k) {
      Words8 r = {};
      if (c < n) r = load32(row + c + k * kEach);
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        if constexpr (sizeof(T) == 4) {
          v[k * kEach + i] = __uint_as_float(r.w[i]);
        } else {
          const float2 f = unpack2(r.w[i], T());
          v[2 * i] = f.x;
          v[2 * i + 1] = f.y;
        }
      }
    }
  } else {
    static_assert(kCols == 8, "narrower accesses take 8 columns");
    unpack8(load8<T, kAccess>(row, c, n), v);
  }
}

template <class T, int kCols, Access kAccess>
__device__ __forceinline__ void store_cols(T* row, int c, int n, const float (&v)[kCols]) {
  if constexpr (kAccess == Access::k32) {
    constexpr int kEach = 32 / sizeof(T);
    if (c < n) {
#pragma unroll
      for (int k = 0; k < kCols / kEach; ++k) {
        Words8 r;
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          if constexpr (sizeof(T) == 4)
            r.w[i] = __float_as_uint(v[k * kEach + i]);
          else
            r.w[i] = pack2(v[2 * i], v[2 * i + 1], T());
        }
        store32(row + c + k * kEach, r);
      }
    }
  } else {
    store8<T, kAccess>(row, c, n, v);
  }
}

// e4m3 codes of v * inv.
template <int kCols, Access kAccess>
__device__ __forceinline__ void store_codes(uint8_t* row, int c, int n, const float (&v)[kCols],
                                            float inv) {
  if constexpr (kAccess == Access::k32) {
    uint32_t w[4];
#pragma unroll
    for (int i = 0; i < 4; ++i)
      w[i] = pack_e4m3x4(v[4 * i] * inv, v[4 * i + 1] * inv, v[4 * i + 2] * inv,
                         v[4 * i + 3] * inv);
    if (c < n) store16(row + c, make_uint4(w[0], w[1], w[2], w[3]));
  } else {
    const uint2 codes = quantize8(v, inv);
    if constexpr (kAccess == Access::k16) {
      if (c < n) *reinterpret_cast<uint2*>(row + c) = codes;
    } else {
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        const int e = element<kAccess>(c, j);
        if (e < n) row[e] = static_cast<uint8_t>((j < 4 ? codes.x : codes.y) >> (8 * (j & 3)));
      }
    }
  }
}

// e4m3 codes of columns that are all in the row.
template <int kCols, Access kAccess>
__device__ __forceinline__ void load_codes(const uint8_t* row, int c, float (&v)[kCols]) {
  uint32_t w[kCols / 4] = {};
  if constexpr (kAccess == Access::k32) {
    const uint4 r = load16(row + c);
    w[0] = r.x, w[1] = r.y, w[2] = r.z, w[3] = r.w;
  } else if constexpr (kAccess == Access::k16) {
    const uint2 r = *reinterpret_cast<const uint2*>(row + c);
    w[0] = r.x, w[1] = r.y;
  } else {
#pragma unroll
    for (int i = 0; i < kCols; ++i)
      w[i / 4] |= static_cast<uint32_t>(row[c + i]) << (8 * (i & 3));
  }
#pragma unroll
  for (int i = 0; i < kCols / 2; ++i) {
    const float2 f = unpack_e4m3x2(static_cast<uint16_t>(w[i / 2] >> (16 * (i & 1))));
    v[2 * i] = f.x;
    v[2 * i + 1] = f.y;
  }
}

}  // namespace mslkb
