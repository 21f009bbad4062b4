// dispatch.cu -- the rows of the chosen experts: packed by expert into the stacked layout
// (dispatch), and summed back per token with the routing weights (combine), with the gradient.
#include "host.h"
#include "rows.cuh"

namespace mslkb {
namespace {

// ---------------------------------------------------------------------------------
// dispatch: a stable counting sort of the choices by expert, then the copies.
//   count_kernel   tile histograms                counts[tile][E]
//   place_kernel   row of every choice            dest, m_sizes
//   copy_kernel    each token's row, read once, to its rows
// ---------------------------------------------------------------------------------
constexpr int kTile = 1024;      // choices per tile
constexpr int kTileWarps = 8;    // a warp places kTile / kTileWarps choices, 32 at a time
constexpr int kWarpChoices = kTile / kTileWarps;

__global__ void __launch_bounds__(256)
    count_kernel(const int32_t* ids, uint32_t* counts, int64_t N, int E) {
  extern __shared__ uint32_t histogram[];
  for (int e = threadIdx.x; e < E; e += blockDim.x) histogram[e] = 0;
  ptx::griddep_wait();
  ptx::griddep_launch_dependents();
  __syncthreads();
  const int64_t begin = static_cast<int64_t>(blockIdx.x) * kTile;
  for (int i = threadIdx.x; i < kTile; i += blockDim.x) {
    const int e = begin + i < N ? ids[begin + i] : -1;
    if (e >= 0 && e < E) atomicAdd(&histogram[e], 1u);  // whole numbers: any order is the same
  }
  __syncthreads();
  for (int e = threadIdx.x; e < E; e += blockDim.x)
    counts[static_cast<int64_t>(blockIdx.x) * E + e] = histogram[e];
}

// Shared memory: base[E] (first row of this tile's choices of an expert), warp_count
// [kTileWarps][E].
__global__ void __launch_bounds__(kTileWarps * 32)
    place_kernel(const int32_t* ids, const uint32_t* counts, int32_t* dest, int64_t* m_sizes,
                 int64_t N, int E, int tiles) {
  extern __shared__ uint32_t place_shared[];
  uint32_t* base = place_shared;
  uint32_t* warp_count = place_shared + E;
  __shared__ uint32_t chunk_sum[kTileWarps];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, threads = kTileWarps * 32;
  for (int i = threadIdx.x; i < kTileWarps * E; i += threads) warp_count[i] = 0;
  ptx::griddep_wait();
  ptx::griddep_launch_dependents();
  const int tile = blockIdx.x;
  // choices of each expert in all tiles (total) and in the tiles before this one
  uint32_t carry = 0;  // rows of the experts before this round's
  for (int e0 = 0; e0 < E; e0 += threads) {
    const int e = e0 + threadIdx.x;
    uint32_t before = 0, total = 0;
    if (e < E) {
#pragma unroll 16
      for (int i = 0; i < tiles; ++i) {
        const uint32_t c = counts[static_cast<int64_t>(i) * E + e];
        if (i < tile) before += c;
        total += c;
      }
      if (tile == 0) m_sizes[e] = total;
    }
    uint32_t sum = total;  // inclusive scan over the threads
#pragma unroll
    for (int d = 1; d < 32; d <<= 1) {
      const uint32_t v = __shfl_up_sync(0xFFFFFFFFu, sum, d);
      if (lane >= d) sum += v;
    }
    if (lane == 31) chunk_sum[warp] = sum;
    __syncthreads();
    uint32_t warps_before = 0, all = 0;
#pragma unroll
    for (int w = 0; w < kTileWarps; ++w) {
      if (w < warp) warps_before += chunk_sum[w];
      all += chunk_sum[w];
    }
    if (e < E) base[e] = carry + warps_before + sum - total + before;
    carry += all;
    __syncthreads();
  }
  // rank of each choice among its warp's choices of the same expert, in order
  const int64_t begin = static_cast<int64_t>(tile) * kTile + warp * kWarpChoices;
  uint32_t* mine = warp_count + warp * E;
  int expert[kWarpChoices / 32];
  uint32_t rank[kWarpChoices / 32];
#pragma unroll
  for (int r = 0; r < kWarpChoices / 32; ++r) {
    const int64_t i = begin + r * 32 + lane;
    int e = i < N ? ids[i] : -1;
    if (e >= E) e = -1;
    const uint32_t same = __match_any_sync(0xFFFFFFFFu, e);
    const uint32_t earlier = __popc(same & ((1u << lane) - 1u));
    const uint32_t seen = e >= 0 ? mine[e] : 0;
    __syncwarp();
    if (e >= 0 && earlier == 0) mine[e] = seen + __popc(same);
    __syncwarp();
    expert[r] = e < 0 ? -1 : e;
    rank[r] = seen + earlier;
  }
  __syncthreads();
  // first row of each warp's choices of an expert
  for (int e = threadIdx.x; e < E; e += threads) {
    uint32_t at = base[e];
#pragma unroll
    for (int w = 0; w < kTileWarps; ++w) {
      const uint32_t c = warp_count[w * E + e];
      warp_count[w * E + e] = at;
      at += c;
    }
  }
  __syncthreads();
#pragma unroll
  for (int r = 0; r < kWarpChoices / 32; ++r) {
    const int64_t i = begin + r * 32 + lane;
    if (i < N) dest[i] = expert[r] < 0 ? -1 : static_cast<int32_t>(mine[expert[r]] + rank[r]);
  }
}

struct CopyParams {
  const uint8_t* x;
  const float* x_scale;
  const int32_t* dest;
  uint8_t* x_out;
  float* scale_out;
  int64_t row_bytes;
  int32_t scale_cols;
  int32_t top_k;
};

// One CTA per token: its row is read once, 16 bytes (kWide) or one byte at a time, and
// written to each of its rows.
template <bool kWide>
__device__ __forceinline__ void copy_row(const CopyParams& p, int64_t t, const int32_t* dest) {
  const uint8_t* from = p.x + t * p.row_bytes;
  if constexpr (kWide) {
    const int n = static_cast<int>(p.row_bytes / 16);
    for (int c = threadIdx.x; c < n; c += blockDim.x) {
      const uint4 v = load16(from + static_cast<int64_t>(c) * 16);
      for (int j = 0; j < p.top_k; ++j) {
        const int32_t d = dest[j];
        if (d >= 0) store16(p.x_out + d * p.row_bytes + static_cast<int64_t>(c) * 16, v);
      }
    }
  } else {
    for (int64_t c = threadIdx.x; c < p.row_bytes; c += blockDim.x) {
      const uint8_t v = from[c];
      for (int j = 0; j < p.top_k; ++j) {
        const int32_t d = dest[j];
        if (d >= 0) p.x_out[d * p.row_bytes + c] = v;
      }
    }
  }
  for (int c = threadIdx.x; c < p.scale_cols; c += blockDim.x) {
    const float v = p.x_scale[t * p.scale_cols + c];
    for (int j = 0; j < p.top_k; ++j) {
      const int32_t d = dest[j];
      if (d >= 0) p.scale_out[static_cast<int64_t>(d) * p.scale_cols + c] = v;
    }
  }
}

template <bool kWide>
__global__ void __launch_bounds__(512) copy_kernel(const __grid_constant__ CopyParams p) {
  __shared__ int32_t dest[MSLKB_MAX_TOPK];
  ptx::griddep_wait();
  ptx::griddep_launch_dependents();
  const int64_t t = blockIdx.x;
  if (threadIdx.x < p.top_k) dest[threadIdx.x] = p.dest[t * p.top_k + threadIdx.x];
  __syncthreads();
  copy_row<kWide>(p, t, dest);
}

// Few choices: one launch, no workspace.  The CTA of a token finds each of its rows by itself:
// the row of choice i is the number of choices that come before it, those of a lower expert
// and the earlier ones of its own.  One more CTA counts the experts' rows.
struct DirectParams {
  CopyParams copy;
  const int32_t* ids;
  int32_t* dest;
  int64_t* m_sizes;
  int32_t T, E;
};

template <bool kWide>
__global__ void __launch_bounds__(512) direct_kernel(const __grid_constant__ DirectParams p) {
  __shared__ uint32_t before[MSLKB_MAX_EXPERTS];  // a token's rows; or the experts' counts
  __shared__ int32_t dest[MSLKB_MAX_TOPK];
  const int k = p.copy.top_k, N = p.T * k, lane = threadIdx.x & 31;
  const int counters = blockIdx.x == p.T ? p.E : k;
  for (int i = threadIdx.x; i < counters; i += blockDim.x) before[i] = 0;
  ptx::griddep_wait();
  ptx::griddep_launch_dependents();
  __syncthreads();
  if (blockIdx.x == p.T) {
    for (int i = threadIdx.x; i < N; i += blockDim.x) {
      const int e = p.ids[i];
      if (e >= 0 && e < p.E) atomicAdd(&before[e], 1u);
    }
    __syncthreads();
    for (int e = threadIdx.x; e < p.E; e += blockDim.x) p.m_sizes[e] = before[e];
    return;
  }
  const int first = blockIdx.x * k;
  // a lane of each warp holds one of the token's choices; foreign ids order last and count
  // for nobody
  int own = lane < k ? p.ids[first + lane] : -1;
  if (own < 0 || own >= p.E) own = -1;
  for (int i0 = 0; i0 < N; i0 += blockDim.x) {
    const int i = i0 + threadIdx.x;
    int e = i < N ? p.ids[i] : -1;
    if (e < 0 || e >= p.E) e = 0x7FFFFFFF;
    for (int j = 0; j < k; ++j) {
      const int mine = __shfl_sync(0xFFFFFFFFu, own, j);
      const uint32_t earlier =
          __ballot_sync(0xFFFFFFFFu, e < mine || (e == mine && i < first + j));
      if (lane == 0 && earlier != 0) atomicAdd(&before[j], __popc(earlier));
    }
  }
  __syncthreads();
  if (threadIdx.x < k) {
    const int row = own >= 0 ? static_cast<int>(before[threadIdx.x]) : -1;
    dest[threadIdx.x] = row;
    p.dest[first + threadIdx.x] = row;
  }
  __syncthreads();
  copy_row<kWide>(p.copy, blockIdx.x, dest);
}

// ---------------------------------------------------------------------------------
// combine and its gradient: one CTA per token, 8 columns per thread and step
// ---------------------------------------------------------------------------------
struct CombineParams {
  const void* rows;
  const int32_t* dest;
  const float* weights;
  void* out;
  int64_t H, R;
  int32_t top_k;
};

// The token's valid rows, in slot order, with their weights; returns how many.
__device__ __forceinline__ int gather_choices(const int32_t* dest, const float* weights,
                                              int64_t t, int top_k, int64_t R, int32_t* row,
                                              float* weight, int32_t* slot) {
  __shared__ int count;
  if (threadIdx.x < 32) {
    const int lane = threadIdx.x;
    const int32_t d = lane < top_k ? dest[t * top_k + lane] : -1;
    const bool here = d >= 0 && d < R;
    const uint32_t mask = __ballot_sync(0xFFFFFFFFu, here);
    if (here) {
      const int at = __popc(mask & ((1u << lane) - 1u));
      row[at] = d;
      weight[at] = weights != nullptr ? weights[t * top_k + lane] : 1.f;
      slot[at] = lane;
    }
    if (lane == 0) count = __popc(mask);
  }
  __syncthreads();
  return count;
}

template <class T, bool kWide>
__global__ void __launch_bounds__(512) combine_kernel(const __grid_constant__ CombineParams p) {
  __shared__ int32_t row[MSLKB_MAX_TOPK], slot[MSLKB_MAX_TOPK];
  __shared__ float weight[MSLKB_MAX_TOPK];
  ptx::griddep_wait();
  ptx::griddep_launch_dependents();
  const int64_t t = blockIdx.x;
  const int n = static_cast<int>(p.H);
  const int count = gather_choices(p.dest, p.weights, t, p.top_k, p.R, row, weight, slot);
  const T* rows = static_cast<const T*>(p.rows);
  for (int c = threadIdx.x * 8; c < n; c += blockDim.x * 8) {
    float sum[8] = {};
    for (int j0 = 0; j0 < count; j0 += 4) {
      Raw8<T> r[4];
#pragma unroll
      for (int j = 0; j < 4; ++j)
        if (j0 + j < count) r[j] = load8<T, kWide>(rows + row[j0 + j] * p.H, c, n);
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        if (j0 + j < count) {
          float v[8];
          unpack8(r[j], v);
#pragma unroll
          for (int i = 0; i < 8; ++i) sum[i] = fmaf(weight[j0 + j], v[i], sum[i]);
        }
      }
    }
    store8<T, kWide>(static_cast<T*>(p.out) + t * p.H, c, n, sum);
  }
}

struct CombineBackwardParams {
  const void* dout;
  const void* rows;
  const int32_t* dest;
  const float* weights;
  void* drows;
  float* dweights;
  int64_t H, R;
  int32_t top_k;
};

template <class T, bool kWide>
__global__ void __launch_bounds__(512)
    combine_backward_kernel(const __grid_constant__ CombineBackwardParams p) {
  __shared__ int32_t row[MSLKB_MAX_TOPK], slot[MSLKB_MAX_TOPK];
  __shared__ float weight[MSLKB_MAX_TOPK];
  __shared__ float partial[MSLKB_MAX_TOPK][16];  // per warp
  ptx::griddep_wait();
  ptx::griddep_launch_dependents();
  const int64_t t = blockIdx.x;
  const int n = static_cast<int>(p.H);
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, warps = blockDim.x >> 5;
  const int count = gather_choices(p.dest, p.weights, t, p.top_k, p.R, row, weight, slot);
  const T* dout = static_cast<const T*>(p.dout) + t * p.H;
  constexpr int kRound = 4;
  for (int j0 = 0; j0 < count; j0 += kRound) {
    float dot[kRound] = {};
    for (int c = threadIdx.x * 8; c < n; c += blockDim.x * 8) {
      float d[8];
      unpack8(load8<T, kWide>(dout, c, n), d);
      Raw8<T> r[kRound];
#pragma unroll
      for (int j = 0; j < kRound; ++j)
        if (j0 + j < count)
          r[j] = load8<T, kWide>(static_cast<const T*>(p.rows) + row[j0 + j] * p.H, c, n);
#pragma unroll
      for (int j = 0; j < kRound; ++j) {
        if (j0 + j < count) {
          float v[8];
          unpack8(r[j], v);
          const float w = weight[j0 + j];
#pragma unroll
          for (int i = 0; i < 8; ++i) {
            dot[j] = fmaf(d[i], v[i], dot[j]);
            v[i] = w * d[i];
          }
          store8<T, kWide>(static_cast<T*>(p.drows) + row[j0 + j] * p.H, c, n, v);
        }
      }
    }
#pragma unroll
    for (int j = 0; j < kRound; ++j) {
      const float s = warp_sum(dot[j]);
      if (lane == 0 && j0 + j < count) partial[j0 + j][warp] = s;
    }
  }
  __syncthreads();
  if (threadIdx.x < p.top_k) p.dweights[t * p.top_k + threadIdx.x] = 0.f;
  __syncthreads();
  if (threadIdx.x < count) {
    float s = 0.f;
    for (int w = 0; w < warps; ++w) s += partial[threadIdx.x][w];
    p.dweights[t * p.top_k + slot[threadIdx.x]] = s;
  }
}

// ---------------------------------------------------------------------------------
// launches
// ---------------------------------------------------------------------------------
int row_threads(int64_t vectors) {
  const int64_t t = (vectors + 31) / 32 * 32;
  return static_cast<int>(t < 32 ? 32 : (t > 512 ? 512 : t));
}

int64_t tiles_of(int64_t choices) { return (choices + kTile - 1) / kTile; }

// Choices up to which each token's CTA finds its rows by itself.
constexpr int64_t kDirectChoices = 2048;

template <class T>
cudaError_t launch_combine(const CombineParams& p, int64_t T_, bool wide, void* stream) {
  const dim3 grid(static_cast<unsigned>(T_)), block(row_threads((p.H + 7) / 8));
  return wide ? launch_dependent(combine_kernel<T, true>, grid, block, 0, stream, p)
              : launch_dependent(combine_kernel<T, false>, grid, block, 0, stream, p);
}

template <class T>
cudaError_t launch_combine_backward(const CombineBackwardParams& p, int64_t T_, bool wide,
                                    void* stream) {
  const dim3 grid(static_cast<unsigned>(T_)), block(row_threads((p.H + 7) / 8));
  return wide ? launch_dependent(combine_backward_kernel<T, true>, grid, block, 0, stream, p)
              : launch_dependent(combine_backward_kernel<T, false>, grid, block, 0, stream, p);
}

mslkb_status check_combine(int64_t T, int64_t top_k, int64_t H, int64_t R, int32_t dtype) {
  if (T < 0 || top_k < 0 || H < 0 || R < 0) return MSLKB_ERR_SHAPE;
  if (T > MSLKB_MAX_DIM || top_k > MSLKB_MAX_TOPK || R > MSLKB_MAX_DIM || H > (1 << 30) ||
      T * top_k > MSLKB_MAX_DIM)
    return MSLKB_ERR_SHAPE;
  return dtype_ok(dtype) ? MSLKB_OK : MSLKB_ERR_DTYPE;
}

}  // namespace
}  // namespace mslkb

extern "C" {

int64_t mslkb_moe_dispatch_workspace_bytes(int64_t T, int64_t top_k, int64_t E) {
  if (T <= 0 || top_k <= 0 || E <= 0 || E > MSLKB_MAX_EXPERTS || top_k > MSLKB_MAX_TOPK ||
      T > MSLKB_MAX_DIM / 2 / top_k)
    return 0;
  if (T * top_k <= mslkb::kDirectChoices) return 0;
  return mslkb::tiles_of(T * top_k) * E * static_cast<int64_t>(sizeof(uint32_t));
}

mslkb_status mslkb_moe_dispatch(const void* x, const float* x_scale, const int32_t* ids,
                                void* x_out, float* scale_out, int64_t* m_sizes, int32_t* dest,
                                void* workspace, int64_t workspace_bytes, int64_t T,
                                int64_t top_k, int64_t E, int64_t row_bytes, int64_t scale_cols,
                                void* stream) {
  using namespace mslkb;
  if (T < 0 || top_k < 0 || E < 0 || row_bytes < 0 || scale_cols < 0) return MSLKB_ERR_SHAPE;
  if (E > MSLKB_MAX_EXPERTS || top_k > MSLKB_MAX_TOPK || row_bytes > MSLKB_MAX_DIM ||
      scale_cols > MSLKB_MAX_DIM || (top_k > 0 && T > MSLKB_MAX_DIM / 2 / top_k) ||
      T > MSLKB_MAX_DIM)
    return MSLKB_ERR_SHAPE;
  if (E > 0 && m_sizes == nullptr) return MSLKB_ERR_NULL;
  const int64_t N = T * top_k;
  if (N > 0) {
    if (ids == nullptr || dest == nullptr) return MSLKB_ERR_NULL;
    if (row_bytes > 0 && (x == nullptr || x_out == nullptr)) return MSLKB_ERR_NULL;
    if (scale_cols > 0 && (x_scale == nullptr || scale_out == nullptr)) return MSLKB_ERR_NULL;
    const int64_t need = mslkb_moe_dispatch_workspace_bytes(T, top_k, E);
    if (need > 0 &&
        (workspace == nullptr || !aligned_to(workspace, 16) || workspace_bytes < need))
      return MSLKB_ERR_WORKSPACE;
  }
  int sms = 0;
  mslkb_status s = device_sms(&sms);
  if (s != MSLKB_OK) return s;
  cudaStream_t cs = static_cast<cudaStream_t>(stream);
  if (N == 0 || E == 0) {  // no choice is here
    cudaError_t e = cudaSuccess;
    if (E > 0) e = cudaMemsetAsync(m_sizes, 0, sizeof(int64_t) * E, cs);
    if (e == cudaSuccess && N > 0) e = cudaMemsetAsync(dest, 0xFF, sizeof(int32_t) * N, cs);
    return launch_status(e);
  }
  uint32_t* counts = static_cast<uint32_t*>(workspace);
  const int tiles = static_cast<int>(tiles_of(N)), experts = static_cast<int>(E);
  const bool wide = row_bytes % 16 == 0 && aligned_to(x, 16) && aligned_to(x_out, 16);
  const CopyParams p{static_cast<const uint8_t*>(x), x_scale, dest, static_cast<uint8_t*>(x_out),
                     scale_out, row_bytes, static_cast<int32_t>(scale_cols),
                     static_cast<int32_t>(top_k)};
  TraceRange range("moe_dispatch", T);
  const dim3 copy_block(row_threads(wide ? row_bytes / 16 : row_bytes));
  if (N <= kDirectChoices) {
    const DirectParams d{p, ids, dest, m_sizes, static_cast<int32_t>(T), experts};
    const dim3 grid(static_cast<unsigned>(T) + 1);
    const dim3 block(copy_block.x < 256 ? 256 : copy_block.x);  // they share the counting too
    return launch_status(wide
                             ? launch_dependent(direct_kernel<true>, grid, block, 0, stream, d)
                             : launch_dependent(direct_kernel<false>, grid, block, 0, stream, d));
  }
  cudaError_t e = launch_dependent(count_kernel, dim3(tiles), dim3(256),
                                   sizeof(uint32_t) * experts, stream, ids, counts, N, experts);
  if (e == cudaSuccess)
    e = launch_dependent(place_kernel, dim3(tiles), dim3(kTileWarps * 32),
                         sizeof(uint32_t) * experts * (kTileWarps + 1), stream, ids, counts, dest,
                         m_sizes, N, experts, tiles);
  if (e == cudaSuccess && (row_bytes > 0 || scale_cols > 0)) {
    const dim3 grid(static_cast<unsigned>(T));
    e = wide ? launch_dependent(copy_kernel<true>, grid, copy_block, 0, stream, p)
             : launch_dependent(copy_kernel<false>, grid, copy_block, 0, stream, p);
  }
  return launch_status(e);
}

mslkb_status mslkb_moe_combine(const void* rows, const int32_t* dest, const float* weights,
                               void* out, int64_t T, int64_t top_k, int64_t H, int64_t R,
                               int32_t dtype, void* stream) {
  using namespace mslkb;
  mslkb_status s = check_combine(T, top_k, H, R, dtype);
  if (s != MSLKB_OK) return s;
  if (T == 0 || H == 0) return MSLKB_OK;
  if (out == nullptr || (top_k > 0 && dest == nullptr) || (R > 0 && rows == nullptr))
    return MSLKB_ERR_NULL;
  int sms = 0;
  if ((s = device_sms(&sms)) != MSLKB_OK) return s;
  const bool wide = H % 8 == 0 && aligned_to(rows, 16) && aligned_to(out, 16);
  const CombineParams p{rows, dest, weights, out, H, R, static_cast<int32_t>(top_k)};
  TraceRange range("moe_combine", T);
  cudaError_t e;
  if (dtype == MSLKB_BF16)
    e = launch_combine<__nv_bfloat16>(p, T, wide, stream);
  else if (dtype == MSLKB_FP16)
    e = launch_combine<__half>(p, T, wide, stream);
  else
    e = launch_combine<float>(p, T, wide, stream);
  return launch_status(e);
}

mslkb_status mslkb_moe_combine_backward(const void* dout, const void* rows, const int32_t* dest,
                                        const float* weights, void* drows, float* dweights,
                                        int64_t T, int64_t top_k, int64_t H, int64_t R,
                                        int32_t dtype, void* stream) {
  using namespace mslkb;
  mslkb_status s = check_combine(T, top_k, H, R, dtype);
  if (s != MSLKB_OK) return s;
  if (T == 0 || top_k == 0) return MSLKB_OK;
  if (dest == nullptr || weights == nullptr || dweights == nullptr ||
      (H > 0 && (dout == nullptr || (R > 0 && (rows == nullptr || drows == nullptr)))))
    return MSLKB_ERR_NULL;
  int sms = 0;
  if ((s = device_sms(&sms)) != MSLKB_OK) return s;
  const bool wide = H % 8 == 0 && aligned_to(dout, 16) && aligned_to(rows, 16) &&
                    aligned_to(drows, 16);
  const CombineBackwardParams p{dout, rows, dest, weights, drows, dweights,
                                H,    R,    static_cast<int32_t>(top_k)};
  TraceRange range("moe_combine_backward", T);
  cudaError_t e;
  if (dtype == MSLKB_BF16)
    e = launch_combine_backward<__nv_bfloat16>(p, T, wide, stream);
  else if (dtype == MSLKB_FP16)
    e = launch_combine_backward<__half>(p, T, wide, stream);
  else
    e = launch_combine_backward<float>(p, T, wide, stream);
  return launch_status(e);
}

}  // extern "C"
