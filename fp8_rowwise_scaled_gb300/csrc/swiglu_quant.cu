// swiglu_quant.cu -- silu(gate) * up between the two expert products: e4m3 output with its
// scales, optionally an e4m3 checkpoint of the input, and the gradient from the input or its
// checkpoint.
//
// Every input is read once and every output written once; the floor is HBM's, but with a
// sigmoid, two or three block maxima and as many roundings per element the instructions come
// close to it.  Hence 16 columns per thread: a block of 128 columns is eight lanes (three
// shuffles), a scale's division is shared by 16 elements, and accesses are 32 bytes wide.
// GB300, 32768 rows of 2 x 2048 bf16: block scales and checkpoint 74 us (6.4 TB/s; with eight
// columns per thread and IEEE divisions 136 us), the gradient from the checkpoint 79 us (6.9).
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

// 1 / (1 + e^-x) with e^-x = 2^(-x log2 e): the exponent's rounding is |x| 2^-24 of it, ex2 and
// recip are good to 2 and 1 ulp.  Far out (below -87.4, where it would be a subnormal, as well)
// it is exactly 0 or 1, NaN stays NaN.  For results of 16 bits, and for e4m3 codes with their
// scale (whose error, at gates of -16 2^-20 of it, is far below a code's 2^-4).
__device__ __forceinline__ float sigmoid_of(float x) {
  float e;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(e) : "f"(x * -1.4426950408889634f));
  return recip(1.f + e);
}

// sigmoid(x) and sigmoid(-x) = 1 - sigmoid(x), for results of type T.  In 32 bits from e^-|x|,
// which neither overflows nor loses bits in its argument; 1 - s past x = 2 as e s, since s's
// rounding times the gate would grow to |x| units there (below, it partly cancels s's own).
// Gradients of gates to +-80 are off by 4e-8 on average (as above: 4.8e-7), and 32768 x 2048
// rows are as fast (GB300, from the input 189 us, from the checkpoint 134; 20000 x 125 that stay
// in L2 8.4, not 6.1).
template <class T>
__device__ __forceinline__ void sigmoids_of(float x, float& s, float& rest) {
  if constexpr (sizeof(T) == 4) {
    const float e = expf(-fabsf(x));
    s = (x < 0.f ? e : 1.f) / (1.f + e);
    rest = x > 2.f ? e * s : 1.f - s;
  } else {
    s = sigmoid_of(x);
    rest = 1.f - s;
  }
}

// e4m3 of a thread's kCols columns, whose block of 128 is spread over 128 / kCols lanes.
template <int kCols, Access kAccess>
__device__ __forceinline__ void quantize_block(const float (&v)[kCols], uint8_t* codes,
                                               float* scale, int c, int n) {
  const float amax = __uint_as_float(block_max<kScaleBlock / kCols>(abs_max(v)));
  const QuantScale s = quant_scale(amax, amax);
  if (c < n && c % kScaleBlock == 0) scale[c / kScaleBlock] = s.scale;
  store_codes<kCols, kAccess>(codes, c, n, v, s.inv);
}

// blockDim.y rows per CTA.  kBlocks: nothing is shared between threads but the lanes of a
// block.  Otherwise a row is a power of two lanes of one warp, or whole warps, with
// kVecs * kCols columns per thread.
template <class T, int kCols, int kVecs, Access kAccess, bool kBlocks>
__global__ void __launch_bounds__(kVecs == 1 ? (kBlocks ? 256 : 512) : 1024,
                                  kVecs == 1 ? (kBlocks ? 4 : 2) : 1)
    swiglu_kernel(const __grid_constant__ SwigluParams p) {
  __shared__ uint32_t slot[32];
  ptx::griddep_wait();
  ptx::griddep_launch_dependents();
  const int64_t row = static_cast<int64_t>(blockIdx.x) * blockDim.y + threadIdx.y;
  const int n = row < p.R ? p.W : 0;  // no columns past the last row
  const T* gate = static_cast<const T*>(p.x) + row * p.ldx;
  const T* up = gate + n;
  float a[kVecs][kCols];
  uint32_t largest = 0;
#pragma unroll
  for (int i = 0; i < kVecs; ++i) {
    const int c = ((blockIdx.y * kVecs + i) * blockDim.x + threadIdx.x) * kCols;
    float g[kCols], u[kCols];
    load_cols<T, kCols, kAccess>(gate, c, n, g);
    load_cols<T, kCols, kAccess>(up, c, n, u);
#pragma unroll
    for (int j = 0; j < kCols; ++j) a[i][j] = g[j] * sigmoid_of(g[j]) * u[j];
    if constexpr (kAccess != Access::kStride) {
      if (p.saved != nullptr) {
        uint8_t* codes = p.saved + row * 2 * n;
        float* scale = p.saved_scale + row * (2 * n / kScaleBlock);
        quantize_block<kCols, kAccess>(g, codes, scale, c, n);
        quantize_block<kCols, kAccess>(u, codes + n, scale + n / kScaleBlock, c, n);
      }
    }
    if constexpr (kBlocks)
      quantize_block<kCols, kAccess>(a[i], p.q + row * n, p.scale + row * (n / kScaleBlock), c, n);
    else
      largest = max(largest, abs_max(a[i]));
  }
  if constexpr (!kBlocks) {
    const int lanes = blockDim.x < 32 ? blockDim.x : 32, warps = blockDim.x >> 5;
    for (int d = lanes >> 1; d > 0; d >>= 1)
      largest = max(largest, __shfl_xor_sync(0xFFFFFFFFu, largest, d));
    if (warps > 1) {
      const int lane = threadIdx.x & 31;
      uint32_t* mine = slot + threadIdx.y * warps;
      if (lane == 0) mine[threadIdx.x >> 5] = largest;
      __syncthreads();
      largest = __reduce_max_sync(0xFFFFFFFFu, lane < warps ? mine[lane] : 0u);
    }
    const float amax = __uint_as_float(largest);
    const QuantScale s = quant_scale(amax, amax);
    if (threadIdx.x == 0 && row < p.R) p.scale[row] = s.scale;
#pragma unroll
    for (int i = 0; i < kVecs; ++i)
      store_codes<kCols, kAccess>(p.q + row * n, (i * blockDim.x + threadIdx.x) * kCols, n, a[i],
                                  s.inv);
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

template <class T, int kCols, Access kAccess, bool kSaved8>
__global__ void __launch_bounds__(256)
    swiglu_backward_kernel(const __grid_constant__ SwigluBackwardParams p) {
  ptx::griddep_wait();
  ptx::griddep_launch_dependents();
  const int64_t row = static_cast<int64_t>(blockIdx.x) * blockDim.y + threadIdx.y;
  const int n = p.W, c = (blockIdx.y * blockDim.x + threadIdx.x) * kCols;
  if (row >= p.R || (c >= n && kAccess != Access::kStride)) return;
  float d[kCols], g[kCols], u[kCols];
  if constexpr (kSaved8) {
    const uint8_t* codes = static_cast<const uint8_t*>(p.saved) + row * 2 * n;
    const float* scale = p.saved_scale + row * (2 * n / kScaleBlock) + c / kScaleBlock;
    load_codes<kCols, kAccess>(codes, c, g);
    load_codes<kCols, kAccess>(codes + n, c, u);
    const float gs = scale[0], us = scale[n / kScaleBlock];
    load_cols<T, kCols, kAccess>(static_cast<const T*>(p.dy) + row * n, c, n, d);
#pragma unroll
    for (int j = 0; j < kCols; ++j) g[j] *= gs, u[j] *= us;
  } else {
    const T* gate = static_cast<const T*>(p.saved) + row * 2 * n;
    load_cols<T, kCols, kAccess>(gate, c, n, g);
    load_cols<T, kCols, kAccess>(gate + n, c, n, u);
    load_cols<T, kCols, kAccess>(static_cast<const T*>(p.dy) + row * n, c, n, d);
  }
#pragma unroll
  for (int j = 0; j < kCols; ++j) {
    float s, rest;
    sigmoids_of<T>(g[j], s, rest);
    u[j] = d[j] * u[j] * s * fmaf(g[j], rest, 1.f);
    g[j] = d[j] * g[j] * s;
  }
  T* dgate = static_cast<T*>(p.dx) + row * 2 * n;
  store_cols<T, kCols, kAccess>(dgate, c, n, u);
  store_cols<T, kCols, kAccess>(dgate + n, c, n, g);
}

// ---------------------------------------------------------------------------------
// launches
// ---------------------------------------------------------------------------------
// Threads of a CTA over rows of `lanes` steps: x along a row, y rows, at most 256 in all.  With
// block_lanes > 1 (a multiple of 8): whole groups of that many along x, whole warps.
dim3 tile_threads(int64_t lanes, int64_t block_lanes) {
  int64_t x = (lanes + block_lanes - 1) / block_lanes * block_lanes;
  if (x > 128) return dim3(256);
  if (x > 64) x = (x + 31) / 32 * 32;
  const int64_t y = x > 64 ? 256 / x : 256 / x / 4 * 4;
  return dim3(static_cast<unsigned>(x), static_cast<unsigned>(y));
}

template <class T, int kCols, Access kAccess>
cudaError_t launch_blocks(const SwigluParams& p, void* stream) {
  const int64_t lanes = (p.W + kCols - 1) / kCols;
  const dim3 block = tile_threads(lanes, kScaleBlock / kCols);
  const dim3 grid(static_cast<unsigned>((p.R + block.y - 1) / block.y),
                  static_cast<unsigned>((lanes + block.x - 1) / block.x));
  return launch_dependent(swiglu_kernel<T, kCols, 1, kAccess, true>, grid, block, 0, stream, p);
}

template <class T, int kCols, Access kAccess>
cudaError_t launch_rows(const SwigluParams& p, void* stream) {
  const int64_t lanes = (p.W + kCols - 1) / kCols;
  if (lanes <= 512) {
    // a narrow row: a power of two lanes (whole blocks of the checkpoint; all 32 where the
    // warp shares its columns out), several rows per CTA
    int64_t x = kAccess == Access::kStride ? 32 : kScaleBlock / kCols;
    while (x < 32 && x < lanes) x *= 2;
    if (lanes > 32) x = (lanes + 31) / 32 * 32;
    const int64_t y = x >= 128 ? 1 : 128 / x;
    return launch_dependent(swiglu_kernel<T, kCols, 1, kAccess, false>,
                            dim3(static_cast<unsigned>((p.R + y - 1) / y)),
                            dim3(static_cast<unsigned>(x), static_cast<unsigned>(y)), 0, stream,
                            p);
  }
  constexpr int kMost = MSLKB_MAX_HIDDEN / kCols / 1024;
  const int64_t x = ((lanes + kMost - 1) / kMost + 31) / 32 * 32;
  return launch_dependent(swiglu_kernel<T, kCols, kMost, kAccess, false>,
                          dim3(static_cast<unsigned>(p.R)), dim3(static_cast<unsigned>(x)), 0,
                          stream, p);
}

template <class T>
cudaError_t launch_swiglu(const SwigluParams& p, Access access, bool blocks, void* stream) {
  if (access == Access::k32)
    return blocks ? launch_blocks<T, 16, Access::k32>(p, stream)
                  : launch_rows<T, 16, Access::k32>(p, stream);
  if (access == Access::k16)
    return blocks ? launch_blocks<T, 8, Access::k16>(p, stream)
                  : launch_rows<T, 8, Access::k16>(p, stream);
  if (blocks) return launch_blocks<T, 8, Access::kElement>(p, stream);
  return p.saved != nullptr ? launch_rows<T, 8, Access::kElement>(p, stream)
                            : launch_rows<T, 8, Access::kStride>(p, stream);
}

template <class T, int kCols, Access kAccess>
cudaError_t launch_backward(const SwigluBackwardParams& p, void* stream) {
  const int64_t lanes = (p.W + kCols - 1) / kCols;
  const dim3 block = tile_threads(lanes, kAccess == Access::kStride ? 32 : 1);
  const dim3 grid(static_cast<unsigned>((p.R + block.y - 1) / block.y),
                  static_cast<unsigned>((lanes + block.x - 1) / block.x));
  if constexpr (kAccess != Access::kStride)
    if (p.saved_scale != nullptr)
      return launch_dependent(swiglu_backward_kernel<T, kCols, kAccess, true>, grid, block, 0,
                              stream, p);
  return launch_dependent(swiglu_backward_kernel<T, kCols, kAccess, false>, grid, block, 0, stream,
                          p);
}

template <class T>
cudaError_t launch_backward(const SwigluBackwardParams& p, Access access, void* stream) {
  if (access == Access::k32) return launch_backward<T, 16, Access::k32>(p, stream);
  if (access == Access::k16) return launch_backward<T, 8, Access::k16>(p, stream);
  return p.saved_scale != nullptr ? launch_backward<T, 8, Access::kElement>(p, stream)
                                  : launch_backward<T, 8, Access::kStride>(p, stream);
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
  const int64_t size = dtype_bytes(dtype);
  Access access = Access::kElement;
  if (W % 16 == 0 && ldx * size % 32 == 0 && aligned_to(x, 32) && aligned_to(q, 16) &&
      aligned_to(saved, 16))
    access = Access::k32;
  else if (W % 8 == 0 && ldx * size % 16 == 0 && aligned_to(x, 16) && aligned_to(q, 8) &&
           aligned_to(saved, 8))
    access = Access::k16;
  const SwigluParams p{x, static_cast<uint8_t*>(q), scale, static_cast<uint8_t*>(saved),
                       saved_scale, R, ldx, static_cast<int32_t>(W)};
  TraceRange range("swiglu_quant", R);
  cudaError_t e;
  if (dtype == MSLKB_BF16)
    e = launch_swiglu<__nv_bfloat16>(p, access, groupwise != 0, stream);
  else if (dtype == MSLKB_FP16)
    e = launch_swiglu<__half>(p, access, groupwise != 0, stream);
  else
    e = launch_swiglu<float>(p, access, groupwise != 0, stream);
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
  Access access = Access::kElement;
  if (W % 16 == 0 && aligned_to(dy, 32) && aligned_to(dx, 32) &&
      aligned_to(saved, saved_scale != nullptr ? 16 : 32))
    access = Access::k32;
  else if (W % 8 == 0 && aligned_to(dy, 16) && aligned_to(dx, 16) &&
           aligned_to(saved, saved_scale != nullptr ? 8 : 16))
    access = Access::k16;
  const SwigluBackwardParams p{dy, saved, saved_scale, dx, R, static_cast<int32_t>(W)};
  TraceRange range("swiglu_quant_backward", R);
  cudaError_t e;
  if (dtype == MSLKB_BF16)
    e = launch_backward<__nv_bfloat16>(p, access, stream);
  else if (dtype == MSLKB_FP16)
    e = launch_backward<__half>(p, access, stream);
  else
    e = launch_backward<float>(p, access, stream);
  return launch_status(e);
}

}  // extern "C"
