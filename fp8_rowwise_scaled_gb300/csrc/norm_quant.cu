// norm_quant.cu -- residual addition + root-mean-square norm + e4m3 output, and the gradient.
//
// Forward, one CTA per row, the row in registers between its one read and its one write:
//   h = x + residual, u = h * weight, and in one pass sum(h^2) and max|u|.
// The codes need no rstd: y / scale = h rstd w * 448 / (rstd max|h w|) = u * (448 / max|u|).
// So one exchange over the CTA gives both rstd and the row's scale (block scales need only
// the 16 lanes that hold a block), where norm-then-quantise would need two.
#include "host.h"
#include "rows.cuh"

namespace mslkb {
namespace {

constexpr int kMaxThreads = 1024;

struct NormParams {
  const void* x;
  const void* residual;
  const void* weight;
  uint8_t* q;
  float* scale;
  void* residual_out;
  void* y;
  float* rstd;
  int64_t ldx, ldr;
  int32_t H;
  int32_t weight_fp32;
  float eps;
};

// weight elements [c, c + 8): fp32 or T
template <class T, bool kWide>
__device__ __forceinline__ void load_weight8(const void* w, int fp32, int c, int n,
                                             float (&v)[8]) {
  if (fp32)
    unpack8(load8<float, kWide>(static_cast<const float*>(w), c, n), v);
  else
    unpack8(load8<T, kWide>(static_cast<const T*>(w), c, n), v);
}

// Sum and maximum over the CTA, to every thread; `slot` holds one pair per warp.
__device__ __forceinline__ void cta_sum_max(float& sum, uint32_t& largest, float2* slot) {
  sum = warp_sum(sum);
  largest = __reduce_max_sync(0xFFFFFFFFu, largest);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, warps = blockDim.x >> 5;
  if (warps == 1) return;
  if (lane == 0) slot[warp] = make_float2(sum, __uint_as_float(largest));
  __syncthreads();
  const float2 mine = lane < warps ? slot[lane] : make_float2(0.f, 0.f);
  sum = warp_sum(mine.x);
  largest = __reduce_max_sync(0xFFFFFFFFu, __float_as_uint(mine.y));
}

template <class T, int kVecs, bool kWide, bool kBlocks>
__global__ void __launch_bounds__(kMaxThreads)
    norm_quant_kernel(const __grid_constant__ NormParams p) {
  __shared__ float2 slot[32];
  ptx::griddep_wait();
  ptx::griddep_launch_dependents();
  const int64_t row = blockIdx.x;
  const int n = p.H;
  const T* x = static_cast<const T*>(p.x) + row * p.ldx;
  const T* residual = static_cast<const T*>(p.residual) + row * p.ldr;
  T* residual_out = static_cast<T*>(p.residual_out) + row * n;

  float u[kVecs][8];  // h
  {
    Raw8<T> rx[kVecs], rr[kVecs];
#pragma unroll
    for (int i = 0; i < kVecs; ++i)
      rx[i] = load8<T, kWide>(x, (i * blockDim.x + threadIdx.x) * 8, n);
    if (p.residual != nullptr) {
#pragma unroll
      for (int i = 0; i < kVecs; ++i)
        rr[i] = load8<T, kWide>(residual, (i * blockDim.x + threadIdx.x) * 8, n);
    }
#pragma unroll
    for (int i = 0; i < kVecs; ++i) {
      unpack8(rx[i], u[i]);
      if (p.residual != nullptr) {
        float r[8];
        unpack8(rr[i], r);
#pragma unroll
        for (int j = 0; j < 8; ++j) u[i][j] += r[j];
      }
    }
  }
  float sum = 0.f;
  uint32_t largest = 0, block_largest[kVecs];
#pragma unroll
  for (int i = 0; i < kVecs; ++i) {
    const int c = (i * blockDim.x + threadIdx.x) * 8;
    if (p.residual_out != nullptr) store8<T, kWide>(residual_out, c, n, u[i]);
    float w[8];
    load_weight8<T, kWide>(p.weight, p.weight_fp32, c, n, w);
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      sum = fmaf(u[i][j], u[i][j], sum);
      w[j] *= u[i][j];
    }
    block_largest[i] = abs_max8(w);
    if constexpr (kBlocks)
      block_largest[i] = block16_max(block_largest[i]);
    else
      largest = max(largest, block_largest[i]);
  }
  cta_sum_max(sum, largest, slot);
  const float rstd = 1.f / sqrtf(sum / static_cast<float>(n) + p.eps);
  if (threadIdx.x == 0 && p.rstd != nullptr) p.rstd[row] = rstd;
  float inv = 0.f;
  if constexpr (!kBlocks) {
    const float m = __uint_as_float(largest), amax = m * rstd;
    const bool zero = amax < kQuantTiny;
    inv = zero ? 0.f : kE4m3Max / m;
    if (threadIdx.x == 0) p.scale[row] = zero ? 1.f : amax / kE4m3Max;
  }
#pragma unroll
  for (int i = 0; i < kVecs; ++i) {
    const int c = (i * blockDim.x + threadIdx.x) * 8;
    if constexpr (kBlocks) {
      const float m = __uint_as_float(block_largest[i]), amax = m * rstd;
      const bool zero = amax < kQuantTiny;
      inv = zero ? 0.f : kE4m3Max / m;
      if (c < n && c % kScaleBlock == 0)
        p.scale[row * (n / kScaleBlock) + c / kScaleBlock] = zero ? 1.f : amax / kE4m3Max;
    }
    float w[8], v[8];
    load_weight8<T, kWide>(p.weight, p.weight_fp32, c, n, w);
#pragma unroll
    for (int j = 0; j < 8; ++j) v[j] = u[i][j] * w[j];
    store_codes8<kWide>(p.q + row * n, c, n, quantize8(v, inv));
    if (p.y != nullptr) {
      // (h * rstd) * weight: h * weight alone may fall among the subnormals
#pragma unroll
      for (int j = 0; j < 8; ++j) v[j] = u[i][j] * rstd * w[j];
      store8<T, kWide>(static_cast<T*>(p.y) + row * n, c, n, v);
    }
  }
}

// ---------------------------------------------------------------------------------
// gradient
// ---------------------------------------------------------------------------------
// Rows of partial weight gradients: the CTAs of the first kernel.
constexpr int64_t kMaxParts = 608;

struct NormBackwardParams {
  const void* dy;
  const void* h;
  const void* weight;
  const float* rstd;
  const void* dresidual;
  void* dx;
  float* parts;  // [gridDim.x, H]
  int64_t T;
  int32_t H;
  int32_t weight_fp32;
};

__device__ __forceinline__ float cta_sum(float sum, float* slot) {
  sum = warp_sum(sum);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, warps = blockDim.x >> 5;
  if (warps == 1) return sum;
  if (lane == 0) slot[warp] = sum;
  __syncthreads();
  return warp_sum(lane < warps ? slot[lane] : 0.f);
}

// A thread keeps its columns over the CTA's rows, so the weight gradient stays in registers
// and is written once per CTA.
template <class T, int kVecs, bool kWide>
__global__ void __launch_bounds__(kMaxThreads)
    norm_backward_kernel(const __grid_constant__ NormBackwardParams p) {
  __shared__ float slot[2][32];
  ptx::griddep_wait();
  ptx::griddep_launch_dependents();
  const int n = p.H;
  float dw[kVecs][8];
#pragma unroll
  for (int i = 0; i < kVecs; ++i)
#pragma unroll
    for (int j = 0; j < 8; ++j) dw[i][j] = 0.f;
  int turn = 0;
  for (int64_t row = blockIdx.x; row < p.T; row += gridDim.x, turn ^= 1) {
    const float rstd = p.rstd[row];
    float g[kVecs][8], xhat[kVecs][8];
    float sum = 0.f;
#pragma unroll
    for (int i = 0; i < kVecs; ++i) {
      const int c = (i * blockDim.x + threadIdx.x) * 8;
      unpack8(load8<T, kWide>(static_cast<const T*>(p.dy) + row * n, c, n), g[i]);
      unpack8(load8<T, kWide>(static_cast<const T*>(p.h) + row * n, c, n), xhat[i]);
    }
#pragma unroll
    for (int i = 0; i < kVecs; ++i) {
      float w[8];
      load_weight8<T, kWide>(p.weight, p.weight_fp32, (i * blockDim.x + threadIdx.x) * 8, n, w);
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        xhat[i][j] *= rstd;
        dw[i][j] = fmaf(g[i][j], xhat[i][j], dw[i][j]);
        g[i][j] *= w[j];
        sum = fmaf(g[i][j], xhat[i][j], sum);
      }
    }
    const float mean = cta_sum(sum, slot[turn]) / static_cast<float>(n);
#pragma unroll
    for (int i = 0; i < kVecs; ++i) {
      const int c = (i * blockDim.x + threadIdx.x) * 8;
      float d[8];
      if (p.dresidual != nullptr) {
        unpack8(load8<T, kWide>(static_cast<const T*>(p.dresidual) + row * n, c, n), d);
      } else {
#pragma unroll
        for (int j = 0; j < 8; ++j) d[j] = 0.f;
      }
#pragma unroll
      for (int j = 0; j < 8; ++j) d[j] = fmaf(rstd, g[i][j] - xhat[i][j] * mean, d[j]);
      store8<T, kWide>(static_cast<T*>(p.dx) + row * n, c, n, d);
    }
  }
#pragma unroll
  for (int i = 0; i < kVecs; ++i)
    store8<float, kWide>(p.parts + static_cast<int64_t>(blockIdx.x) * n,
                         (i * blockDim.x + threadIdx.x) * 8, n, dw[i]);
}

// Column sums of parts [rows, H], in a fixed order: 8 threads per column.
__global__ void __launch_bounds__(256)
    sum_parts_kernel(const float* parts, float* out, int rows, int n) {
  __shared__ float slot[8][33];
  ptx::griddep_wait();
  ptx::griddep_launch_dependents();
  const int c = blockIdx.x * 32 + (threadIdx.x & 31), part = threadIdx.x >> 5;
  float s = 0.f;
  if (c < n) {
#pragma unroll 4
    for (int r = part; r < rows; r += 8) s += parts[static_cast<int64_t>(r) * n + c];
  }
  slot[part][threadIdx.x & 31] = s;
  __syncthreads();
  if (part == 0 && c < n) {
#pragma unroll
    for (int i = 1; i < 8; ++i) s += slot[i][threadIdx.x];
    out[c] = s;
  }
}

// ---------------------------------------------------------------------------------
// launches
// ---------------------------------------------------------------------------------
int threads_for(int64_t n, int vecs) {
  const int64_t t = ((n + 7) / 8 + vecs - 1) / vecs;
  return static_cast<int>((t + 31) / 32 * 32);
}

template <class T, int kVecs, bool kWide>
cudaError_t launch_norm(const NormParams& p, int64_t rows, bool blocks, void* stream) {
  const dim3 grid(static_cast<unsigned>(rows)), block(threads_for(p.H, kVecs));
  return blocks ? launch_dependent(norm_quant_kernel<T, kVecs, kWide, true>, grid, block, 0,
                                   stream, p)
                : launch_dependent(norm_quant_kernel<T, kVecs, kWide, false>, grid, block, 0,
                                   stream, p);
}

template <class T>
cudaError_t launch_norm(const NormParams& p, int64_t rows, bool wide, bool blocks,
                        void* stream) {
  const int64_t n = p.H;
  if (!wide) return launch_norm<T, 4, false>(p, rows, blocks, stream);
  if (n <= 8 * kMaxThreads) return launch_norm<T, 1, true>(p, rows, blocks, stream);
  if (n <= 16 * kMaxThreads) return launch_norm<T, 2, true>(p, rows, blocks, stream);
  return launch_norm<T, 4, true>(p, rows, blocks, stream);
}

template <class T, int kVecs, bool kWide>
cudaError_t launch_backward(const NormBackwardParams& p, int64_t parts, void* stream) {
  return launch_dependent(norm_backward_kernel<T, kVecs, kWide>,
                          dim3(static_cast<unsigned>(parts)), dim3(threads_for(p.H, kVecs)), 0,
                          stream, p);
}

template <class T>
cudaError_t launch_backward(const NormBackwardParams& p, bool wide, int64_t parts,
                            void* stream) {
  const int64_t n = p.H;
  if (!wide) return launch_backward<T, 4, false>(p, parts, stream);
  if (n <= 16 * kMaxThreads) return launch_backward<T, 2, true>(p, parts, stream);
  return launch_backward<T, 4, true>(p, parts, stream);
}

int64_t backward_parts(int64_t T) { return T < kMaxParts ? T : kMaxParts; }

mslkb_status check_rows(int64_t T, int64_t H, int32_t dtype) {
  if (T < 0 || H < 0 || T > MSLKB_MAX_DIM || H > MSLKB_MAX_HIDDEN) return MSLKB_ERR_SHAPE;
  return dtype_ok(dtype) ? MSLKB_OK : MSLKB_ERR_DTYPE;
}

}  // namespace
}  // namespace mslkb

extern "C" {

mslkb_status mslkb_add_rms_norm_quant(const void* x, const void* residual, const void* weight,
                                      void* q, float* scale, void* residual_out, void* y,
                                      float* rstd, int64_t T, int64_t H, int64_t ldx,
                                      int64_t ldr, double eps, int32_t dtype,
                                      int32_t weight_fp32, int32_t groupwise, void* stream) {
  using namespace mslkb;
  mslkb_status s = check_rows(T, H, dtype);
  if (s != MSLKB_OK) return s;
  if (groupwise && H % kScaleBlock != 0) return MSLKB_ERR_SHAPE;
  if (!(eps >= 1e-12 && eps < 1.0)) return MSLKB_ERR_SHAPE;
  if (ldx < H || ldx > MSLKB_MAX_DIM || (residual != nullptr && (ldr < H || ldr > MSLKB_MAX_DIM)))
    return MSLKB_ERR_SHAPE;
  if (T == 0 || H == 0) return MSLKB_OK;
  if (x == nullptr || weight == nullptr || q == nullptr || scale == nullptr)
    return MSLKB_ERR_NULL;
  int sms = 0;
  if ((s = device_sms(&sms)) != MSLKB_OK) return s;
  const int64_t size = dtype_bytes(dtype);
  const bool wide = H % 8 == 0 && ldx * size % 16 == 0 && aligned_to(x, 16) &&
                    (residual == nullptr || (ldr * size % 16 == 0 && aligned_to(residual, 16))) &&
                    aligned_to(weight, 16) && aligned_to(q, 8) && aligned_to(residual_out, 16) &&
                    aligned_to(y, 16);
  NormParams p{x,    residual, weight, static_cast<uint8_t*>(q),
               scale, residual_out, y, rstd, ldx, ldr,
               static_cast<int32_t>(H), weight_fp32, static_cast<float>(eps)};
  TraceRange range("add_rms_norm_quant", T);
  cudaError_t e;
  if (dtype == MSLKB_BF16)
    e = launch_norm<__nv_bfloat16>(p, T, wide, groupwise != 0, stream);
  else if (dtype == MSLKB_FP16)
    e = launch_norm<__half>(p, T, wide, groupwise != 0, stream);
  else
    e = launch_norm<float>(p, T, wide, groupwise != 0, stream);
  return launch_status(e);
}

int64_t mslkb_add_rms_norm_quant_backward_workspace_bytes(int64_t T, int64_t H) {
  if (T <= 0 || H <= 0 || H > MSLKB_MAX_HIDDEN) return 0;
  return mslkb::backward_parts(T) * H * static_cast<int64_t>(sizeof(float));
}

mslkb_status mslkb_add_rms_norm_quant_backward(const void* dy, const void* h, const void* weight,
                                               const float* rstd, const void* dresidual,
                                               void* dx, float* dweight, void* workspace,
                                               int64_t workspace_bytes, int64_t T, int64_t H,
                                               int32_t dtype, int32_t weight_fp32,
                                               void* stream) {
  using namespace mslkb;
  mslkb_status s = check_rows(T, H, dtype);
  if (s != MSLKB_OK) return s;
  if (H == 0) return MSLKB_OK;
  if (dweight == nullptr) return MSLKB_ERR_NULL;
  if (T > 0 && (dy == nullptr || h == nullptr || weight == nullptr || rstd == nullptr ||
                dx == nullptr))
    return MSLKB_ERR_NULL;
  const int64_t need = mslkb_add_rms_norm_quant_backward_workspace_bytes(T, H);
  if (need > 0 && (workspace == nullptr || !aligned_to(workspace, 16) || workspace_bytes < need))
    return MSLKB_ERR_WORKSPACE;
  int sms = 0;
  if ((s = device_sms(&sms)) != MSLKB_OK) return s;
  const bool wide = H % 8 == 0 && aligned_to(dy, 16) && aligned_to(h, 16) &&
                    aligned_to(weight, 16) && aligned_to(dresidual, 16) && aligned_to(dx, 16);
  int64_t parts = backward_parts(T);
  if (parts > 4 * static_cast<int64_t>(sms)) parts = 4 * static_cast<int64_t>(sms);
  float* partial = static_cast<float*>(workspace);
  NormBackwardParams p{dy, h, weight, rstd, dresidual, dx, partial, T,
                       static_cast<int32_t>(H), weight_fp32};
  TraceRange range("add_rms_norm_quant_backward", T);
  cudaError_t e = cudaSuccess;
  if (T > 0) {
    if (dtype == MSLKB_BF16)
      e = launch_backward<__nv_bfloat16>(p, wide, parts, stream);
    else if (dtype == MSLKB_FP16)
      e = launch_backward<__half>(p, wide, parts, stream);
    else
      e = launch_backward<float>(p, wide, parts, stream);
  }
  if (e == cudaSuccess)
    e = launch_dependent(sum_parts_kernel, dim3(static_cast<unsigned>((H + 31) / 32)), dim3(256),
                         0, stream, partial, dweight, static_cast<int>(T > 0 ? parts : 0),
                         static_cast<int>(H));
  return launch_status(e);
}

}  // extern "C"
