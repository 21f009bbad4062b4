// norm_quant.cu -- residual addition + root-mean-square norm + e4m3 output, and the gradient.
//
// Forward, the row in registers between its one read and its one write:
//   h = x + residual, u = h * weight, and in one pass sum(h^2) and max|u|;
// rstd is the row's common factor, so max|y| = rstd max|u| and one exchange over the CTA gives
// both rstd and the row's scale (block scales need only the 16 lanes that hold a block), where
// norm-then-quantise would need two.  Where y is not asked for, the codes do without rstd:
// y / scale = h rstd w * 448 / (rstd max|h w|) = u * (448 / max|u|).
//
// Both directions read every input once and write every output once and are bound by HBM
// (GB300, 8192 rows of 7168 bf16: with residual, block scales, y and rstd 88 us, 6.0 TB/s of
// the 6.8 that a copy reaches; the gradient 72 us, 6.5 TB/s with the weight's sums).
// With a row per CTA, the CTA's loads wait while it reduces and stores; so for many rows the
// kernels are persistent, and each warp copies its own columns of the next rows into a ring of
// stages in shared memory (cp.async, 16 bytes per lane) while it works on this one.  A warp
// reads back only what it copied itself: cp.async.wait_group and warp barriers are all the
// synchronisation that the ring needs (tests/test_norm_ring_lanes.py runs it on the CPU with its
// lanes as far apart as these let them come).
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
  int64_t T, ldx, ldr;
  int32_t H;
  int32_t weight_fp32;
  float eps, inv_h;
};

// weight elements [c, c + kCols): fp32 or T
template <class T, int kCols, Access kAccess>
__device__ __forceinline__ void load_weight(const void* w, int fp32, int c, int n,
                                            float (&v)[kCols]) {
  if (fp32)
    load_cols<float, kCols, kAccess>(static_cast<const float*>(w), c, n, v);
  else
    load_cols<T, kCols, kAccess>(static_cast<const T*>(w), c, n, v);
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

// The first of a thread's kCols columns, step i.
template <int kCols>
__device__ __forceinline__ int column(int i) {
  return (i * blockDim.x + threadIdx.x) * kCols;
}

// One row whose h is in registers, a thread's columns [column(i), column(i) + kCols):
// everything from there to the outputs.
template <class T, int kCols, int kVecs, Access kAccess, bool kBlocks, class Weight>
__device__ __forceinline__ void finish_row(const NormParams& p, int64_t row,
                                           float (&h)[kVecs][kCols], Weight weight,
                                           float2* slot) {
  const int n = p.H;
  T* residual_out = static_cast<T*>(p.residual_out) + row * n;
  float sum = 0.f;
  uint32_t largest = 0, block_largest[kVecs];
#pragma unroll
  for (int i = 0; i < kVecs; ++i) {
    if (p.residual_out != nullptr)
      store_cols<T, kCols, kAccess>(residual_out, column<kCols>(i), n, h[i]);
    float w[kCols];
    weight(i, w);
#pragma unroll
    for (int j = 0; j < kCols; ++j) {
      sum = fmaf(h[i][j], h[i][j], sum);
      w[j] *= h[i][j];
    }
    block_largest[i] = abs_max(w);
    if constexpr (kBlocks)
      block_largest[i] = block_max<kScaleBlock / kCols>(block_largest[i]);
    else
      largest = max(largest, block_largest[i]);
  }
  cta_sum_max(sum, largest, slot);
  const float rstd = rsqrtf(fmaf(sum, p.inv_h, p.eps));  // 2 ulp
  if (threadIdx.x == 0 && p.rstd != nullptr) p.rstd[row] = rstd;
  QuantScale s;
  if constexpr (!kBlocks) {
    const float m = __uint_as_float(largest);
    s = quant_scale(m * rstd, p.y != nullptr ? m * rstd : m);
    if (threadIdx.x == 0) p.scale[row] = s.scale;
  }
#pragma unroll
  for (int i = 0; i < kVecs; ++i) {
    const int c = column<kCols>(i);
    if constexpr (kBlocks) {
      const float m = __uint_as_float(block_largest[i]);
      s = quant_scale(m * rstd, p.y != nullptr ? m * rstd : m);
      if (c < n && c % kScaleBlock == 0)
        p.scale[row * (n / kScaleBlock) + c / kScaleBlock] = s.scale;
    }
    float w[kCols], v[kCols];
    weight(i, w);
    if (p.y != nullptr) {
      // (h * rstd) * weight: h * weight alone may fall among the subnormals
#pragma unroll
      for (int j = 0; j < kCols; ++j) v[j] = h[i][j] * rstd * w[j];
      store_cols<T, kCols, kAccess>(static_cast<T*>(p.y) + row * n, c, n, v);
    } else {
#pragma unroll
      for (int j = 0; j < kCols; ++j) v[j] = h[i][j] * w[j];
    }
    store_codes<kCols, kAccess>(p.q + row * n, c, n, v, s.inv);
  }
}

// One CTA per row, straight from global memory.  (A row's columns are spread over the threads
// as in the ring's kernel, so its sums do not depend on the number of rows.)
template <class T, int kCols, int kVecs, Access kAccess, bool kBlocks>
__global__ void __launch_bounds__(kAccess == Access::k32 ? 512 : kMaxThreads)
    norm_quant_kernel(const __grid_constant__ NormParams p) {
  __shared__ float2 slot[32];
  ptx::griddep_wait();
  ptx::griddep_launch_dependents();
  const int64_t row = blockIdx.x;
  const int n = p.H;
  const T* x = static_cast<const T*>(p.x) + row * p.ldx;
  const T* residual = static_cast<const T*>(p.residual) + row * p.ldr;
  float h[kVecs][kCols], r[kVecs][kCols];
  // x and residual need no more than 16-byte aligned rows, as in the ring
  const auto input = [&](const T* from, int c, float (&v)[kCols]) {
#pragma unroll
    for (int j = 0; j < kCols; j += 8) {
      float u[8];
      unpack8(load8<T, kAccess>(from, c + j, n), u);
#pragma unroll
      for (int k = 0; k < 8; ++k) v[j + k] = u[k];
    }
  };
#pragma unroll
  for (int i = 0; i < kVecs; ++i) input(x, column<kCols>(i), h[i]);
  if (p.residual != nullptr) {
#pragma unroll
    for (int i = 0; i < kVecs; ++i) input(residual, column<kCols>(i), r[i]);
#pragma unroll
    for (int i = 0; i < kVecs; ++i)
#pragma unroll
      for (int j = 0; j < kCols; ++j) h[i][j] += r[i][j];
  }
  finish_row<T, kCols, kVecs, kAccess, kBlocks>(
      p, row, h,
      [&](int i, float (&w)[kCols]) {
        load_weight<T, kCols, kAccess>(p.weight, p.weight_fp32, column<kCols>(i), n, w);
      },
      slot);
}

// ---------------------------------------------------------------------------------
// the ring of rows
// ---------------------------------------------------------------------------------
// A warp's columns of a stage, step i of input `stream`: 32 * kCols of them, in 16-byte pieces
// that the lanes copy side by side (whole sectors of each access) and lane l reads as pieces
// l * kPieces ...  The permutation keeps those reads free of bank conflicts.
template <class T, int kCols, int kVecs>
__device__ __forceinline__ uint32_t ring_piece(int stream, int i, int piece) {
  constexpr int kPieces = kCols * sizeof(T) / 16;
  if constexpr (kPieces == 1) return ((stream * kVecs + i) * blockDim.x + threadIdx.x) * 16;
  const int at = piece ^ ((piece >> 3) & (kPieces - 1));
  return (((stream * kVecs + i) * (blockDim.x >> 5) + (threadIdx.x >> 5)) * 32 * kPieces + at) * 16;
}

template <class T, int kCols, int kVecs>
__device__ __forceinline__ void ring_fetch(uint32_t stage, int stream, const T* row, int n) {
  constexpr int kPieces = kCols * sizeof(T) / 16, kEach = 16 / sizeof(T);
  const int lane = threadIdx.x & 31;
#pragma unroll
  for (int i = 0; i < kVecs; ++i) {
    const int c0 = (i * static_cast<int>(blockDim.x) + (threadIdx.x & ~31)) * kCols;
#pragma unroll
    for (int k = 0; k < kPieces; ++k) {
      const int piece = k * 32 + lane, c = c0 + piece * kEach;
      // past the row's end nothing is read and zeros are written
      ptx::cp_async<16>(stage + ring_piece<T, kCols, kVecs>(stream, i, piece),
                        c < n ? row + c : row, c < n ? 16 : 0);
    }
  }
}

template <class T, int kCols, int kVecs>  // the lane's columns 8 j ... of step i
__device__ __forceinline__ Raw8<T> ring_raw(const uint8_t* stage, int stream, int i, int j) {
  constexpr int kPieces = kCols * sizeof(T) / 16, kRaw = sizeof(T) / 2;
  const int first = (threadIdx.x & 31) * kPieces + j * kRaw;
  Raw8<T> r;
#pragma unroll
  for (int k = 0; k < kRaw; ++k)
    r.w[k] = load16(stage + ring_piece<T, kCols, kVecs>(stream, i, first + k));
  return r;
}

template <class T, int kCols, int kVecs>
__device__ __forceinline__ void ring_read(const uint8_t* stage, int stream, int i,
                                          float (&v)[kCols]) {
#pragma unroll
  for (int j = 0; j < kCols / 8; ++j) {
    float u[8];
    unpack8(ring_raw<T, kCols, kVecs>(stage, stream, i, j), u);
#pragma unroll
    for (int k = 0; k < 8; ++k) v[j * 8 + k] = u[k];
  }
}

// The calling warp's pieces of the oldest stage are in shared memory, the others' copies
// included.
template <int kStages, int kBytes>
__device__ __forceinline__ void ring_wait() {
  ptx::cp_async_wait<kStages - 1>();
  if constexpr (kBytes > 16) __syncwarp();  // 16 bytes of columns: a lane reads its own piece
}

// All lanes of the warp have read the stage that it fills next.  For reads after the row's
// reduction only: of what is read before it, the reduction's sum comes, which no lane has until
// all have brought theirs.
template <int kBytes>
__device__ __forceinline__ void ring_release() {
  if constexpr (kBytes > 16) __syncwarp();
}

template <class T, int kCols, int kVecs>
constexpr int ring_stage_bytes(int streams, int threads) {
  return streams * kVecs * threads * kCols * static_cast<int>(sizeof(T));
}

// 16 columns per thread and step: a block of 128 columns is eight lanes, outputs leave in
// 32-byte stores.
template <class T, int kVecs, int kStages, bool kBlocks>
__global__ void __launch_bounds__(512, kVecs == 1 ? 2 : 1)
    norm_ring_kernel(const __grid_constant__ NormParams p) {
  extern __shared__ __align__(16) uint8_t ring[];
  __shared__ float2 slot[2][32];
  const int n = p.H;
  const bool add = p.residual != nullptr;
  const int stage_bytes =
      (add ? 2 : 1) * kVecs * static_cast<int>(blockDim.x * 16 * sizeof(T));
  const uint32_t base = ptx::smem_addr(ring);
  ptx::griddep_wait();
  ptx::griddep_launch_dependents();
  auto fetch = [&](int64_t row, int stage) {
    if (row < p.T) {
      const uint32_t at = base + stage * stage_bytes;
      ring_fetch<T, 16, kVecs>(at, 0, static_cast<const T*>(p.x) + row * p.ldx, n);
      if (add) ring_fetch<T, 16, kVecs>(at, 1, static_cast<const T*>(p.residual) + row * p.ldr, n);
    }
    ptx::cp_async_commit();
  };
#pragma unroll
  for (int s = 0; s < kStages - 1; ++s)
    fetch(blockIdx.x + static_cast<int64_t>(s) * gridDim.x, s);
  float w[kVecs][16];
#pragma unroll
  for (int i = 0; i < kVecs; ++i)
    load_weight<T, 16, Access::k32>(p.weight, p.weight_fp32, column<16>(i), n, w[i]);
  int stage = 0, turn = 0;
  for (int64_t row = blockIdx.x; row < p.T; row += gridDim.x) {
    fetch(row + static_cast<int64_t>(kStages - 1) * gridDim.x,
          stage == 0 ? kStages - 1 : stage - 1);
    ring_wait<kStages, 16 * sizeof(T)>();
    const uint8_t* at = ring + stage * stage_bytes;
    float h[kVecs][16];
#pragma unroll
    for (int i = 0; i < kVecs; ++i) {
      ring_read<T, 16, kVecs>(at, 0, i, h[i]);
      if (add) {
        float r[16];
        ring_read<T, 16, kVecs>(at, 1, i, r);
#pragma unroll
        for (int j = 0; j < 16; ++j) h[i][j] += r[j];
      }
    }
    finish_row<T, 16, kVecs, Access::k32, kBlocks>(
        p, row, h,
        [&](int i, float (&v)[16]) {
#pragma unroll
          for (int j = 0; j < 16; ++j) v[j] = w[i][j];
        },
        slot[turn]);
    turn ^= 1;
    stage = stage == kStages - 1 ? 0 : stage + 1;
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
  float inv_h;
};

// Sum over the threads of a row, to each of them: the CTA's, or with kRows row y's blockDim.x.
template <bool kRows>
__device__ __forceinline__ float row_sum(float sum, float* slot, int y) {
  sum = warp_sum(sum);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, warps = blockDim.x >> 5;
  if (warps == 1) return sum;
  float* mine = kRows ? slot + y * warps : slot;
  if (lane == 0) mine[warp] = sum;
  if constexpr (kRows)
    ptx::named_bar_sync(1 + y, blockDim.x);
  else
    __syncthreads();
  return warp_sum(lane < warps ? mine[lane] : 0.f);
}

// One row of the gradient; `inputs` gives a thread's eight columns i of dy (g) and h, `weight` and
// `residual` those of the others, `total` the row's sum.  dy and h are taken twice (from the
// ring or L1), before and after the row's mean, rather than kept: with the weight gradient in
// registers over all the CTA's rows, that is what leaves room for enough threads on an SM.
// kEarly: `residual` is read before the reduction (from memory, where registers allow: 16384 x
// 1025 bf16 79 us, not 95).
template <class T, int kVecs, Access kAccess, bool kEarly, class Inputs, class Weight,
          class Residual, class Total>
__device__ __forceinline__ void backward_row(const NormBackwardParams& p, int64_t row, int n,
                                             float rstd, float (&dw)[kVecs][8], Inputs inputs,
                                             Weight weight, Residual residual, Total total) {
  float sum = 0.f;
  Raw8<T> early[kVecs];
  if constexpr (kEarly) {
#pragma unroll
    for (int i = 0; i < kVecs; ++i) early[i] = residual(i);
  }
#pragma unroll
  for (int i = 0; i < kVecs; ++i) {
    float g[8], h[8], w[8];
    inputs(i, g, h);
    weight(i, w);
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      sum = fmaf(g[j] * w[j], h[j], sum);
      dw[i][j] = fmaf(g[j], h[j] * rstd, dw[i][j]);
    }
  }
  // dx = rstd (g w - h rstd mean), mean = rstd sum / H (rstd^3 alone might underflow)
  const float along = -(total(sum) * p.inv_h * rstd * rstd * rstd);
#pragma unroll
  for (int i = 0; i < kVecs; ++i) {
    float g[8], h[8], w[8], d[8];
    inputs(i, g, h);
    weight(i, w);
    unpack8(kEarly ? early[i] : residual(i), d);
#pragma unroll
    for (int j = 0; j < 8; ++j) d[j] = fmaf(along, h[j], fmaf(rstd, g[j] * w[j], d[j]));
    store8<T, kAccess>(static_cast<T*>(p.dx) + row * p.H, column<8>(i), n, d);
  }
}

// Adds up the weight gradients of the CTA's rows, through shared memory [rows][kVecs * 8][x], and
// writes them out: row y's threads those of step y.
template <int kVecs, Access kAccess>
__device__ __forceinline__ void store_row_sums(const NormBackwardParams& p, float* sums,
                                               const float (&dw)[kVecs][8]) {
  const int y = threadIdx.y, rows = blockDim.y;
#pragma unroll
  for (int i = 0; i < kVecs; ++i)
#pragma unroll
    for (int j = 0; j < 8; ++j)
      sums[((y * kVecs + i) * 8 + j) * blockDim.x + threadIdx.x] = dw[i][j];
  __syncthreads();
  if (y >= kVecs) return;
  float total[8] = {};
  for (int r = 0; r < rows; ++r)
#pragma unroll
    for (int j = 0; j < 8; ++j)
      total[j] += sums[((r * kVecs + y) * 8 + j) * blockDim.x + threadIdx.x];
  store8<float, kAccess>(p.parts + static_cast<int64_t>(blockIdx.x) * p.H, column<8>(y), p.H,
                         total);
}

// Straight from global memory.  kRows: blockDim.y narrow rows at a time, as below.
template <class T, int kVecs, Access kAccess, bool kRows>
__global__ void __launch_bounds__(kRows ? 512 : kMaxThreads, kRows ? 2 : 1)
    norm_backward_kernel(const __grid_constant__ NormBackwardParams p) {
  __shared__ float slot[2][32];
  ptx::griddep_wait();
  ptx::griddep_launch_dependents();
  const int n = p.H, y = kRows ? threadIdx.y : 0, rows = kRows ? blockDim.y : 1;
  float dw[kVecs][8] = {};
  int turn = 0;
  for (int64_t row = static_cast<int64_t>(blockIdx.x) * rows + y; row < p.T;
       row += static_cast<int64_t>(gridDim.x) * rows, turn ^= 1) {
    backward_row<T, kVecs, kAccess, kVecs * sizeof(T) <= 4>(
        p, row, n, p.rstd[row], dw,
        [&](int i, float (&g)[8], float (&h)[8]) {
          const int c = column<8>(i);
          unpack8(load8<T, kAccess>(static_cast<const T*>(p.dy) + row * n, c, n), g);
          unpack8(load8<T, kAccess>(static_cast<const T*>(p.h) + row * n, c, n), h);
        },
        [&](int i, float (&w)[8]) {
          load_weight<T, 8, kAccess>(p.weight, p.weight_fp32, column<8>(i), n, w);
        },
        [&](int i) {
          const T* from = static_cast<const T*>(p.dresidual) + row * n;
          return load8<T, kAccess>(from, column<8>(i), p.dresidual != nullptr ? n : 0);
        },
        [&](float sum) { return row_sum<kRows>(sum, slot[turn], y); });
  }
  if constexpr (kRows) {
    __shared__ float sums[512 * 8 * kVecs];
    store_row_sums<kVecs, kAccess>(p, sums, dw);
  } else {
#pragma unroll
    for (int i = 0; i < kVecs; ++i)
      store8<float, kAccess>(p.parts + static_cast<int64_t>(blockIdx.x) * n, column<8>(i), n,
                             dw[i]);
  }
}

// From the ring.  kRows: blockDim.y narrow rows at a time, each with a barrier of its own (one
// warp: none), whose weight gradients are added up at the end.
constexpr int backward_registers(int steps) { return steps == 4 ? 128 : 64; }

template <class T, int kVecs, int kStages, bool kRows>
__global__ void __launch_bounds__(kRows ? 512 : (kVecs == 4 ? 256 : kMaxThreads),
                                  kRows ? (kVecs == 4 ? 1 : 2) : (kVecs == 4 ? 2 : 1))
    norm_backward_ring_kernel(const __grid_constant__ NormBackwardParams p) {
  extern __shared__ __align__(16) uint8_t ring[];
  __shared__ float slot[2][32];
  const int y = kRows ? threadIdx.y : 0, rows = kRows ? blockDim.y : 1;
  const bool add = p.dresidual != nullptr;
  const int row_bytes = (add ? 3 : 2) * kVecs * static_cast<int>(blockDim.x * 8 * sizeof(T));
  const int stage_bytes = rows * row_bytes;
  const uint32_t base = ptx::smem_addr(ring) + y * row_bytes;
  ptx::griddep_wait();
  ptx::griddep_launch_dependents();
  const int64_t first = static_cast<int64_t>(blockIdx.x) * rows + y;
  const int64_t step = static_cast<int64_t>(gridDim.x) * rows;
  auto fetch = [&](int64_t row, int stage) {
    if (row < p.T) {
      const uint32_t at = base + stage * stage_bytes;
      const int n = p.H;
      ring_fetch<T, 8, kVecs>(at, 0, static_cast<const T*>(p.dy) + row * n, n);
      ring_fetch<T, 8, kVecs>(at, 1, static_cast<const T*>(p.h) + row * n, n);
      if (add) ring_fetch<T, 8, kVecs>(at, 2, static_cast<const T*>(p.dresidual) + row * n, n);
    }
    ptx::cp_async_commit();
  };
#pragma unroll
  for (int s = 0; s < kStages - 1; ++s) fetch(first + s * step, s);
  float w[kVecs][8], dw[kVecs][8] = {};
#pragma unroll
  for (int i = 0; i < kVecs; ++i)
    load_weight<T, 8, Access::k16>(p.weight, p.weight_fp32, column<8>(i), p.H, w[i]);
  int stage = 0, turn = 0;
  float rstd = first < p.T ? p.rstd[first] : 0.f;
  for (int64_t row = first; row < p.T; row += step) {
    fetch(row + (kStages - 1) * step, stage == 0 ? kStages - 1 : stage - 1);
    const float next_rstd = row + step < p.T ? p.rstd[row + step] : 0.f;
    ring_wait<kStages, 8 * sizeof(T)>();
    const uint8_t* at = ring + y * row_bytes + stage * stage_bytes;
    backward_row<T, kVecs, Access::k16, false>(
        p, row, p.H, rstd, dw,
        [&](int i, float (&g)[8], float (&h)[8]) {
          ring_read<T, 8, kVecs>(at, 0, i, g);
          ring_read<T, 8, kVecs>(at, 1, i, h);
        },
        [&](int i, float (&v)[8]) {
#pragma unroll
          for (int j = 0; j < 8; ++j) v[j] = w[i][j];
        },
        [&](int i) {
          return add ? ring_raw<T, 8, kVecs>(at, 2, i, 0) : Raw8<T>{};
        },
        [&](float sum) { return row_sum<kRows>(sum, slot[turn], y); });
    ring_release<8 * sizeof(T)>();  // dy, h and the residual's gradient were read after the sum
    rstd = next_rstd;
    turn ^= 1;
    stage = stage == kStages - 1 ? 0 : stage + 1;
  }
  if constexpr (kRows) {  // through the ring, which nobody reads any more
    ptx::cp_async_wait<0>();
    __syncthreads();
    store_row_sums<kVecs, Access::k16>(p, reinterpret_cast<float*>(ring), dw);
  } else {
#pragma unroll
    for (int i = 0; i < kVecs; ++i)
      store8<float, Access::k16>(p.parts + static_cast<int64_t>(blockIdx.x) * p.H, column<8>(i),
                                 p.H, dw[i]);
  }
}

// Column sums of parts [rows, H], in a fixed order: a warp takes 32 columns of every
// (blockDim.x / 32)-th row.
__global__ void __launch_bounds__(1024)
    sum_parts_kernel(const float* parts, float* out, int rows, int n) {
  __shared__ float slot[32][32];
  ptx::griddep_wait();
  ptx::griddep_launch_dependents();
  const int lane = threadIdx.x & 31, part = threadIdx.x >> 5, warps = blockDim.x >> 5;
  const int c = blockIdx.x * 32 + lane;
  float s = 0.f;
  constexpr int kAhead = 10;  // loads under way together
  for (int r0 = part; c < n && r0 < rows; r0 += warps * kAhead) {
    float v[kAhead];
#pragma unroll
    for (int i = 0; i < kAhead; ++i) {
      const int r = r0 + warps * i;
      v[i] = r < rows ? parts[static_cast<int64_t>(r) * n + c] : 0.f;
    }
#pragma unroll
    for (int i = 0; i < kAhead; ++i) s += v[i];
  }
  slot[part][lane] = s;
  __syncthreads();
  if (part > 0 || c >= n) return;
  for (int w = 1; w < warps; ++w) s += slot[w][lane];
  out[c] = s;
}

// Its warps: four up to 40 parts, then one per ten rows or so, 32 at most (19 rows each of 608
// parts).  Few parts take small CTAs, which find room beside those of the first kernel: 64 rows
// of 8192 bf16 6.0 us in all, by 32 warps each 8.0; 8192 rows (304 parts) by 16 warps each 1 us
// more than by 32.
int sum_warps(int64_t parts) {
  return parts <= 40 ? 4 : (parts <= 80 ? 8 : (parts <= 160 ? 16 : 32));
}

// ---------------------------------------------------------------------------------
// launches
// ---------------------------------------------------------------------------------
int threads_for(int64_t n, int cols) {  // cols: columns per thread in all
  return static_cast<int>(((n + cols - 1) / cols + 31) / 32 * 32);
}

template <class T, int kCols, int kVecs, Access kAccess, bool kBlocks>
cudaError_t launch_norm_kernel(const NormParams& p, void* stream) {
  return launch_dependent(norm_quant_kernel<T, kCols, kVecs, kAccess, kBlocks>,
                          dim3(static_cast<unsigned>(p.T)), dim3(threads_for(p.H, kCols * kVecs)),
                          0, stream, p);
}

template <class T, int kCols, int kVecs, Access kAccess>
cudaError_t launch_norm(const NormParams& p, bool blocks, void* stream) {
  return blocks ? launch_norm_kernel<T, kCols, kVecs, kAccess, true>(p, stream)
                : launch_norm_kernel<T, kCols, kVecs, kAccess, false>(p, stream);
}

// CTAs of a ring kernel that an SM holds, by shared memory and registers per thread.
int ring_ctas(int smem, int threads, int registers) {
  int c = kMaxSmSmem / (smem + 1024);
  if (c > 65536 / registers / threads) c = 65536 / registers / threads;
  return c < 1 ? 1 : c;
}

template <class T, int kVecs, int kStages>
cudaError_t launch_norm_ring(const NormParams& p, int sms, bool blocks, void* stream) {
  const int threads = threads_for(p.H, 16 * kVecs);
  const int smem =
      kStages * ring_stage_bytes<T, 16, kVecs>(p.residual != nullptr ? 2 : 1, threads);
  const int64_t most = static_cast<int64_t>(sms) * ring_ctas(smem, threads, kVecs == 1 ? 64 : 128);
  const dim3 grid(static_cast<unsigned>(p.T < most ? p.T : most));
  cudaError_t e = blocks ? allow_smem<norm_ring_kernel<T, kVecs, kStages, true>>()
                         : allow_smem<norm_ring_kernel<T, kVecs, kStages, false>>();
  if (e != cudaSuccess) return e;
  return blocks ? launch_dependent(norm_ring_kernel<T, kVecs, kStages, true>, grid, dim3(threads),
                                   smem, stream, p)
                : launch_dependent(norm_ring_kernel<T, kVecs, kStages, false>, grid,
                                   dim3(threads), smem, stream, p);
}

// Stages of the ring: the rows under way should be about 28 KB per CTA at H = 7168.  More
// slows the memory down (GB300, 8192 x 7168 bf16, block scales, y: with a residual, two rows
// to a stage, 2 / 3 / 4 stages take 88.3 / 94.0 / 95.0 us), less does not cover its latency
// (without: 52.9 / 48.0 / 47.7 us).  From memory directly, a row per CTA: 100.3 and 68.5 us.
template <class T, int kVecs>
cudaError_t launch_norm_ring(const NormParams& p, int sms, bool blocks, void* stream) {
  if constexpr (sizeof(T) == 2)
    if (p.residual == nullptr) return launch_norm_ring<T, kVecs, 3>(p, sms, blocks, stream);
  return launch_norm_ring<T, kVecs, 2>(p, sms, blocks, stream);
}

template <class T>
cudaError_t launch_norm(const NormParams& p, int sms, Access access, bool blocks, void* stream) {
  const int64_t n = p.H;
  if (access == Access::k32) {
    // from memory directly against the ring, H = 7168 bf16 with everything, us: 152 rows 2.89 /
    // 2.99, 304 3.71 / 3.92, 608 6.45 / 6.16, 1216 12.1 / 10.7, 4864 60.5 / 53.6
    const bool many = p.T > 2 * sms;
    if (n <= 8192)
      return many ? launch_norm_ring<T, 1>(p, sms, blocks, stream)
                  : launch_norm<T, 16, 1, Access::k32>(p, blocks, stream);
    if (n <= 16384) {
      if constexpr (sizeof(T) == 2)  // (stages of 32-bit rows would not fit)
        if (many) return launch_norm_ring<T, 2>(p, sms, blocks, stream);
      return launch_norm<T, 16, 2, Access::k32>(p, blocks, stream);
    }
    return launch_norm<T, 16, 4, Access::k32>(p, blocks, stream);
  }
  // Steps per thread, with a residual and y, us at 1 / 2 / 4: bf16 8192 x 7176 105.6 / 96.4 /
  // 91.1, 16384 x 2056 55.6 / 56.8 / 57.6, 16384 x 1000 26.8 / 26.8 / 25.7 (fp32 43.0 / 44.1 /
  // 50.3), 4096 x 12296 - / 119.7 / 88.3; one row of 7176 2.9 / 3.2 / 3.8
  if (access == Access::k16) return launch_norm<T, 8, 4, Access::k16>(p, blocks, stream);
  // whole blocks that are not aligned, or rows of any length with one scale: one step as far as
  // 1024 threads reach (bf16, 1 / 2 / 4 steps, us: 16384 x 1025 38.2 / 48.8 / 83.4, 8192 x 8191
  // 152.6 / 162.2 / 229.9; fp32 43.7 / 48.2 / 54.5 and 180.5 / 186.8 / 181.0), then four (4096 x
  // 12289 fp32 - / 180.2 / 157.9, but bf16 - / 154.3 / 224.7)
  if (blocks) return launch_norm_kernel<T, 8, 4, Access::kElement, true>(p, stream);
  return n <= 8192 ? launch_norm_kernel<T, 8, 1, Access::kStride, false>(p, stream)
                   : launch_norm_kernel<T, 8, 4, Access::kStride, false>(p, stream);
}

// The gradient's first kernel; *parts: the rows of partial weight gradients that it writes.
template <class T, int kVecs, Access kAccess>
cudaError_t launch_backward(const NormBackwardParams& p, int64_t* parts, void* stream) {
  return launch_dependent(norm_backward_kernel<T, kVecs, kAccess, false>,
                          dim3(static_cast<unsigned>(*parts)),
                          dim3(threads_for(p.H, 8 * kVecs)), 0, stream, p);
}

// Rows of a CTA of 512 threads with x threads each, at least `least`: fewer where the rows would
// not reach all SMs.
int rows_of_cta(int64_t T, int x, int sms, int least) {
  const int64_t y = T / sms < 512 / x ? T / sms : 512 / x;
  return y < least ? least : static_cast<int>(y);
}

template <class T>
cudaError_t launch_backward_rows(const NormBackwardParams& p, int sms, int64_t* parts,
                                 void* stream) {
  const int x = threads_for(p.H, 8), y = rows_of_cta(p.T, x, sms, 1);
  const int64_t ctas = (p.T + y - 1) / y;
  if (*parts > ctas) *parts = ctas;
  return launch_dependent(norm_backward_kernel<T, 1, Access::kStride, true>,
                          dim3(static_cast<unsigned>(*parts)),
                          dim3(static_cast<unsigned>(x), static_cast<unsigned>(y)), 0, stream, p);
}

template <class T, int kVecs, int kStages, bool kRows>
cudaError_t launch_backward_ring(const NormBackwardParams& p, int sms, int64_t* parts,
                                 void* stream) {
  const int x = threads_for(p.H, 8 * kVecs);
  const int row = ring_stage_bytes<T, 8, kVecs>(p.dresidual != nullptr ? 3 : 2, x);
  const int y = kRows ? rows_of_cta(p.T, x, sms, kVecs) : 1;
  const int smem = kStages * y * row;
  const int64_t most = static_cast<int64_t>(sms) * ring_ctas(smem, x * y, backward_registers(kVecs));
  const int64_t ctas = (p.T + y - 1) / y;
  if (*parts > ctas) *parts = ctas;
  if (*parts > most) *parts = most;
  cudaError_t e = allow_smem<norm_backward_ring_kernel<T, kVecs, kStages, kRows>>();
  if (e != cudaSuccess) return e;
  return launch_dependent(norm_backward_ring_kernel<T, kVecs, kStages, kRows>,
                          dim3(static_cast<unsigned>(*parts)),
                          dim3(static_cast<unsigned>(x), static_cast<unsigned>(y)), smem, stream,
                          p);
}

template <class T>
cudaError_t launch_backward(const NormBackwardParams& p, int sms, bool wide, int64_t* parts,
                            void* stream) {
  const int64_t n = p.H;
  // rows of any length: several per CTA against one (16384 rows, bf16): 129 16.2 / 40.4 us,
  // 513 51.2 / 87.7, 1025 80.4 / 97.0 (fp32 81.3 / 64.4), 2047 127 / 111
  if (!wide && n <= 768) return launch_backward_rows<T>(p, sms, parts, stream);
  if (!wide)
    return n <= 8192 ? launch_backward<T, 1, Access::kStride>(p, parts, stream)
                     : launch_backward<T, 4, Access::kStride>(p, parts, stream);
  // From memory directly against the ring, bf16, us: 8192 columns 32 rows 5.7 / 5.6, 100 rows
  // 7.5 / 6.8, 133 9.4 / 7.5; 16384 columns 64 rows 8.5 / 8.8, 133 11.1 / 11.5; 1024 columns,
  // several rows per CTA, 76 4.4 / 5.2, 152 5.3 / 5.2, 1216 9.1 / 6.7.
  const bool many = p.T >= (n > 2048 && n <= 8192 ? 32 : sms);
  // Steps of eight columns per thread (few threads with many columns reduce and synchronise less,
  // many steps leave fewer rows under way), rows per CTA and stages.  GB300, 16384 rows with a
  // residual, device us, 1 / 2 / 4 steps:
  //   bf16, several rows:  256 9.9 / 13.3 / 16.8   512 17.8 / 17.2 / 19.5   640 24.5 / 28.1 / 22.1
  //                        1024 30.3 / 32.2 / 27.4   2048 (one row: 56.5 / 48.1 / 50.0) - / - / 46.9
  //   bf16, one row:       4096 108.9 / 81.8 / 83.5   8192 rows of 7168 111.5 / 72.4 / 72.5
  //                        2 steps, 2 / 3 stages: 4096 84.9 / 81.8, 8192 rows of 2560 36.1 /
  //                        31.0, 5120 55.3 / 54.5, 5632 59.1 / 59.3, 7168 72.4 / 79.3
  //   fp32, several rows:  512 25.9 / 32.0   1024 45.9 / 57.0      one row: 2048 84.2 / 86.1 / 83.7
  //                        8192 rows of 5120 128.6 / 132.0 / 126.3, without a residual 125.5 /
  //                        88.0 / 82.9
  // A row per CTA from memory directly, 6103 x 16384 bf16: 201 us (the ring 122).
  if constexpr (sizeof(T) == 2) {
    if (n <= 256)
      return many ? launch_backward_ring<T, 1, 2, true>(p, sms, parts, stream)
                  : launch_backward<T, 1, Access::k16>(p, parts, stream);
    if (n <= 512)
      return many ? launch_backward_ring<T, 2, 3, true>(p, sms, parts, stream)
                  : launch_backward<T, 1, Access::k16>(p, parts, stream);
    if (n <= 2048)
      return many ? launch_backward_ring<T, 4, 2, true>(p, sms, parts, stream)
                  : launch_backward<T, 1, Access::k16>(p, parts, stream);
    if (many && n <= 5120) return launch_backward_ring<T, 2, 3, false>(p, sms, parts, stream);
    if (many && n <= 16384) return launch_backward_ring<T, 2, 2, false>(p, sms, parts, stream);
  } else {
    if (many && n <= 1024) return launch_backward_ring<T, 1, 2, true>(p, sms, parts, stream);
    if (many && n <= 4096) return launch_backward_ring<T, 1, 2, false>(p, sms, parts, stream);
    if (many && n <= 8192) return launch_backward_ring<T, 4, 2, false>(p, sms, parts, stream);
    // (two stages of longer rows would not fit)
  }
  if (n <= 4096) return launch_backward<T, 1, Access::k16>(p, parts, stream);
  if (n <= 16384) return launch_backward<T, 2, Access::k16>(p, parts, stream);
  return launch_backward<T, 4, Access::k16>(p, parts, stream);
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
  if (residual != nullptr && residual_out == residual && ldr != H && T > 1)
    return MSLKB_ERR_SHAPE;  // the rows written would lie across others still to be read
  if (T == 0 || H == 0) return MSLKB_OK;
  if (x == nullptr || weight == nullptr || q == nullptr || scale == nullptr)
    return MSLKB_ERR_NULL;
  int sms = 0;
  if ((s = device_sms(&sms)) != MSLKB_OK) return s;
  const int64_t size = dtype_bytes(dtype);
  const auto aligned = [&](int64_t out, int64_t in) {  // bytes of the outputs' and inputs' rows
    return H * size % out == 0 && ldx * size % in == 0 && aligned_to(x, in) &&
           (residual == nullptr || (ldr * size % in == 0 && aligned_to(residual, in))) &&
           aligned_to(weight, out) && aligned_to(q, out / 2) && aligned_to(residual_out, out) &&
           aligned_to(y, out);
  };
  Access access = Access::kElement;
  if (H % 16 == 0 && aligned(32, 16))
    access = Access::k32;
  else if (H % 8 == 0 && aligned(16, 16))
    access = Access::k16;
  NormParams p{x,    residual, weight, static_cast<uint8_t*>(q),
               scale, residual_out, y, rstd, T, ldx, ldr,
               static_cast<int32_t>(H), weight_fp32, static_cast<float>(eps),
               1.f / static_cast<float>(H)};
  TraceRange range("add_rms_norm_quant", T);
  cudaError_t e;
  if (dtype == MSLKB_BF16)
    e = launch_norm<__nv_bfloat16>(p, sms, access, groupwise != 0, stream);
  else if (dtype == MSLKB_FP16)
    e = launch_norm<__half>(p, sms, access, groupwise != 0, stream);
  else
    e = launch_norm<float>(p, sms, access, groupwise != 0, stream);
  return launch_status(e);
}

int64_t mslkb_add_rms_norm_quant_backward_workspace_bytes(int64_t T, int64_t H) {
  if (T <= 1 || H <= 0 || H > MSLKB_MAX_HIDDEN) return 0;
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
                    aligned_to(weight, 16) && aligned_to(dresidual, 16) && aligned_to(dx, 16) &&
                    (T != 1 || aligned_to(dweight, 16));
  int64_t parts = backward_parts(T);
  // one part is the gradient itself
  float* partial = parts == 1 ? dweight : static_cast<float*>(workspace);
  NormBackwardParams p{dy, h, weight, rstd, dresidual, dx, partial, T,
                       static_cast<int32_t>(H), weight_fp32, 1.f / static_cast<float>(H)};
  TraceRange range("add_rms_norm_quant_backward", T);
  cudaError_t e = cudaSuccess;
  if (T > 0) {
    if (dtype == MSLKB_BF16)
      e = launch_backward<__nv_bfloat16>(p, sms, wide, &parts, stream);
    else if (dtype == MSLKB_FP16)
      e = launch_backward<__half>(p, sms, wide, &parts, stream);
    else
      e = launch_backward<float>(p, sms, wide, &parts, stream);
  }
  if (e == cudaSuccess && partial != dweight)
    e = launch_dependent(sum_parts_kernel, dim3(static_cast<unsigned>((H + 31) / 32)),
                         dim3(32 * sum_warps(parts)), 0, stream, partial, dweight, static_cast<int>(T > 0 ? parts : 0),
                         static_cast<int>(H));
  return launch_status(e);
}

}  // extern "C"
