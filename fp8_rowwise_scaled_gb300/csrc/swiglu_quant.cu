// swiglu_quant.cu -- silu(gate) * up between the two expert products: e4m3 output with its
// scales, optionally an e4m3 checkpoint of the input, and the gradient from the input or its
// checkpoint.
#include "host.h"
#include "rows.cuh"

namespace mslkb {
namespace {

struct SwigluParams {
  const void* x;
  uint8_t* q;
  float* scale;
  uint8_t* saved;
  float* saved_scale;
  int64_t R, ldx;
  int32_t W;
};

__device__ __forceinline__ float sigmoid_of(float x) { return 1.f / (1.f + expf(-x)); }

// e4m3 of eight columns whose block of 128 is spread over 16 lanes, and the block's scale.
template <bool kWide>
__device__ __forceinline__ void quantize_block(const float (&v)[8], uint8_t* codes, float* scale,
                                               int c, int n) {
  const QuantScale s = quant_scale(__uint_as_float(block16_max(abs_max8(v))));
  if (c < n && c % kScaleBlock == 0) scale[c / kScaleBlock] = s.scale;
  store_codes8<kWide>(codes, c, n, quantize8(v, s.inv));
}

// One CTA per row (kBlocks: threadIdx.y rows per CTA).
template <class T, int kVecs, bool kWide, bool kBlocks>
__global__ void __launch_bounds__(1024)
    swiglu_kernel(const __grid_constant__ SwigluParams p) {
  __shared__ uint32_t slot[32];
  ptx::griddep_wait();
  ptx::griddep_launch_dependents();
  const int64_t row = static_cast<int64_t>(blockIdx.x) * blockDim.y + threadIdx.y;
  const int n = p.W;
  const bool there = row < p.R;
  const T* gate = static_cast<const T*>(p.x) + row * p.ldx;
  const T* up = gate + n;
  float a[kVecs][8];
  uint32_t largest = 0;
#pragma unroll
  for (int i = 0; i < kVecs; ++i) {
    const int c = (i * blockDim.x + threadIdx.x) * 8;
    float g[8], u[8];
    unpack8(load8<T, kWide>(gate, c, there ? n : 0), g);
    unpack8(load8<T, kWide>(up, c, there ? n : 0), u);
#pragma unroll
    for (int j = 0; j < 8; ++j) a[i][j] = g[j] * sigmoid_of(g[j]) * u[j];
    if (p.saved != nullptr) {
      uint8_t* codes = p.saved + row * 2 * n;
      float* scale = p.saved_scale + row * (2 * n / kScaleBlock);
      quantize_block<kWide>(g, codes, scale, c, there ? n : 0);
      quantize_block<kWide>(u, codes + n, scale + n / kScaleBlock, c, there ? n : 0);
    }
    if constexpr (kBlocks)
      quantize_block<kWide>(a[i], p.q + row * n, p.scale + row * (n / kScaleBlock), c,
                            there ? n : 0);
    else
      largest = max(largest, abs_max8(a[i]));
  }
  if constexpr (!kBlocks) {
    largest = __reduce_max_sync(0xFFFFFFFFu, largest);
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, warps = blockDim.x >> 5;
    if (warps > 1) {
      if (lane == 0) slot[warp] = largest;
      __syncthreads();
      largest = __reduce_max_sync(0xFFFFFFFFu, lane < warps ? slot[lane] : 0u);
    }
    const QuantScale s = quant_scale(__uint_as_float(largest));
    if (threadIdx.x == 0) p.scale[row] = s.scale;
#pragma unroll
    for (int i = 0; i < kVecs; ++i)
      store_codes8<kWide>(p.q + row * n, (i * blockDim.x + threadIdx.x) * 8, n,
                          quantize8(a[i], s.inv));
  }
}

struct SwigluBackwardParams {
  const void* dy;
  const void* saved;
  const float* saved_scale;
  void* dx;
  int64_t R;
  int32_t W;
};

template <class T, bool kSaved8, bool kWide>
__global__ void __launch_bounds__(256)
    swiglu_backward_kernel(const __grid_constant__ SwigluBackwardParams p) {
  ptx::griddep_wait();
  ptx::griddep_launch_dependents();
  const int64_t row = static_cast<int64_t>(blockIdx.x) * blockDim.y + threadIdx.y;
  if (row >= p.R) return;
  const int n = p.W;
  T* dgate = static_cast<T*>(p.dx) + row * 2 * n;
  for (int c = threadIdx.x * 8; c < n; c += blockDim.x * 8) {
    float d[8], g[8], u[8];
    unpack8(load8<T, kWide>(static_cast<const T*>(p.dy) + row * n, c, n), d);
    if constexpr (kSaved8) {
      const uint8_t* codes = static_cast<const uint8_t*>(p.saved) + row * 2 * n;
      const float* scale = p.saved_scale + row * (2 * n / kScaleBlock) + c / kScaleBlock;
      uint2 gc, uc;
      if constexpr (kWide) {
        gc = *reinterpret_cast<const uint2*>(codes + c);
        uc = *reinterpret_cast<const uint2*>(codes + n + c);
      } else {
        uint32_t w[4] = {};
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          w[i / 4] |= static_cast<uint32_t>(codes[c + i]) << (8 * (i & 3));
          w[2 + i / 4] |= static_cast<uint32_t>(codes[n + c + i]) << (8 * (i & 3));
        }
        gc = make_uint2(w[0], w[1]);
        uc = make_uint2(w[2], w[3]);
      }
      unpack_e4m3x8(gc, g);
      unpack_e4m3x8(uc, u);
      const float gs = scale[0], us = scale[n / kScaleBlock];
#pragma unroll
      for (int j = 0; j < 8; ++j) g[j] *= gs, u[j] *= us;
    } else {
      const T* gate = static_cast<const T*>(p.saved) + row * 2 * n;
      unpack8(load8<T, kWide>(gate, c, n), g);
      unpack8(load8<T, kWide>(gate + n, c, n), u);
    }
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      const float s = sigmoid_of(g[j]);
      u[j] = d[j] * u[j] * s * (1.f + g[j] * (1.f - s));
      g[j] = d[j] * g[j] * s;
    }
    store8<T, kWide>(dgate, c, n, u);
    store8<T, kWide>(dgate + n, c, n, g);
  }
}

template <class T, int kVecs, bool kWide>
cudaError_t launch_swiglu(const SwigluParams& p, bool blocks, void* stream) {
  int64_t x = ((p.W + 7) / 8 + kVecs - 1) / kVecs;
  if (blocks) {  // rows of 16-lane blocks: several narrow rows per CTA
    x = (x + 15) / 16 * 16;
    int64_t y = 256 / x;
    if (y == 0) {
      y = 1;
      x = (x + 31) / 32 * 32;
    } else if (x * y % 32 != 0) {
      ++y;  // whole warps
    }
    return launch_dependent(swiglu_kernel<T, kVecs, kWide, true>,
                            dim3(static_cast<unsigned>((p.R + y - 1) / y)),
                            dim3(static_cast<unsigned>(x), static_cast<unsigned>(y)), 0, stream,
                            p);
  }
  x = (x + 31) / 32 * 32;
  return launch_dependent(swiglu_kernel<T, kVecs, kWide, false>,
                          dim3(static_cast<unsigned>(p.R)), dim3(static_cast<unsigned>(x)), 0,
                          stream, p);
}

template <class T>
cudaError_t launch_swiglu(const SwigluParams& p, bool wide, bool blocks, void* stream) {
  if (!wide) return launch_swiglu<T, 4, false>(p, blocks, stream);
  if (p.W <= 8192) return launch_swiglu<T, 1, true>(p, blocks, stream);
  return launch_swiglu<T, 4, true>(p, blocks, stream);
}

template <class T>
cudaError_t launch_swiglu_backward(const SwigluBackwardParams& p, bool wide, void* stream) {
  int64_t x = (p.W + 7) / 8;
  x = x > 256 ? 256 : x;
  const int64_t y = 256 / x;
  const dim3 grid(static_cast<unsigned>((p.R + y - 1) / y));
  const dim3 block(static_cast<unsigned>(x), static_cast<unsigned>(y));
  if (p.saved_scale != nullptr)
    return wide ? launch_dependent(swiglu_backward_kernel<T, true, true>, grid, block, 0, stream, p)
                : launch_dependent(swiglu_backward_kernel<T, true, false>, grid, block, 0, stream,
                                   p);
  return wide ? launch_dependent(swiglu_backward_kernel<T, false, true>, grid, block, 0, stream, p)
              : launch_dependent(swiglu_backward_kernel<T, false, false>, grid, block, 0, stream,
                                 p);
}

mslkb_status check_swiglu(int64_t R, int64_t W, int32_t dtype) {
  if (R < 0 || W < 0 || R > MSLKB_MAX_DIM || W > MSLKB_MAX_HIDDEN) return MSLKB_ERR_SHAPE;
  return dtype_ok(dtype) ? MSLKB_OK : MSLKB_ERR_DTYPE;
}

}  // namespace
}  // namespace mslkb

extern "C" {

mslkb_status mslkb_swiglu_quant(const void* x, void* q, float* scale, void* saved,
                                float* saved_scale, int64_t R, int64_t W, int64_t ldx,
                                int32_t dtype, int32_t groupwise, void* stream) {
  using namespace mslkb;
  mslkb_status s = check_swiglu(R, W, dtype);
  if (s != MSLKB_OK) return s;
  if ((groupwise || saved != nullptr) && W % kScaleBlock != 0) return MSLKB_ERR_SHAPE;
  if (ldx < 2 * W || ldx > MSLKB_MAX_DIM) return MSLKB_ERR_SHAPE;
  if (R == 0 || W == 0) return MSLKB_OK;
  if (x == nullptr || q == nullptr || scale == nullptr ||
      (saved != nullptr && saved_scale == nullptr))
    return MSLKB_ERR_NULL;
  int sms = 0;
  if ((s = device_sms(&sms)) != MSLKB_OK) return s;
  const bool wide = W % 8 == 0 && ldx * dtype_bytes(dtype) % 16 == 0 && aligned_to(x, 16) &&
                    aligned_to(q, 8) && aligned_to(saved, 8);
  const SwigluParams p{x, static_cast<uint8_t*>(q), scale, static_cast<uint8_t*>(saved),
                       saved_scale, R, ldx, static_cast<int32_t>(W)};
  TraceRange range("swiglu_quant", R);
  cudaError_t e;
  if (dtype == MSLKB_BF16)
    e = launch_swiglu<__nv_bfloat16>(p, wide, groupwise != 0, stream);
  else if (dtype == MSLKB_FP16)
    e = launch_swiglu<__half>(p, wide, groupwise != 0, stream);
  else
    e = launch_swiglu<float>(p, wide, groupwise != 0, stream);
  return launch_status(e);
}

mslkb_status mslkb_swiglu_quant_backward(const void* dy, const void* saved,
                                         const float* saved_scale, void* dx, int64_t R,
                                         int64_t W, int32_t dtype, void* stream) {
  using namespace mslkb;
  mslkb_status s = check_swiglu(R, W, dtype);
  if (s != MSLKB_OK) return s;
  if (saved_scale != nullptr && W % kScaleBlock != 0) return MSLKB_ERR_SHAPE;
  if (R == 0 || W == 0) return MSLKB_OK;
  if (dy == nullptr || saved == nullptr || dx == nullptr) return MSLKB_ERR_NULL;
  int sms = 0;
  if ((s = device_sms(&sms)) != MSLKB_OK) return s;
  const bool wide = W % 8 == 0 && aligned_to(dy, 16) && aligned_to(dx, 16) &&
                    aligned_to(saved, saved_scale != nullptr ? 8 : 16);
  const SwigluBackwardParams p{dy, saved, saved_scale, dx, R, static_cast<int32_t>(W)};
  TraceRange range("swiglu_quant_backward", R);
  cudaError_t e;
  if (dtype == MSLKB_BF16)
    e = launch_swiglu_backward<__nv_bfloat16>(p, wide, stream);
  else if (dtype == MSLKB_FP16)
    e = launch_swiglu_backward<__half>(p, wide, stream);
  else
    e = launch_swiglu_backward<float>(p, wide, stream);
  return launch_status(e);
}

}  // extern "C"
