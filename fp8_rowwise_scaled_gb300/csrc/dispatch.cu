// dispatch.cu -- the rows of the chosen experts: packed by expert into the stacked layout
// (dispatch), and summed back per token with the routing weights (combine), with the gradient.
#include <type_traits>

#include "host.h"
#include "rows.cuh"

namespace mslkb {
namespace {

// ---------------------------------------------------------------------------------
// dispatch: a stable counting sort of the choices by expert (place_kernel: the row of every
// choice), then each token's row is read once and written to its rows (copy_kernel).  The
// copies are bound by HBM's writes; the sort in front of them by latency, so it is one kernel
// of one cluster: the eight CTAs exchange their counts through distributed shared memory.
// ---------------------------------------------------------------------------------
constexpr int kCluster = 8;
constexpr int kPlaceWarps = 32;

constexpr int kAhead = 8;  // loads of a warp under way together

// The experts of choices [i0, i0 + 32 * kAhead) below `end`, one per lane and step; -1: not here.
__device__ __forceinline__ void load_choices(const int32_t* ids, int64_t i0, int64_t end, int E,
                                             int (&choice)[kAhead]) {
  const int64_t i = i0 + (threadIdx.x & 31);
#pragma unroll
  for (int r = 0; r < kAhead; ++r) choice[r] = i + r * 32 < end ? ids[i + r * 32] : -1;
#pragma unroll
  for (int r = 0; r < kAhead; ++r)
    if (choice[r] < 0 || choice[r] >= E) choice[r] = -1;
}

// The lanes of the warp whose choice is this lane's, from one ballot per bit of the expert
// (match.any walks through the distinct values, some thirty of them here).
template <int kBits>
__device__ __forceinline__ uint32_t same_expert(int choice) {
  uint32_t same = __ballot_sync(0xFFFFFFFFu, choice >= 0);
#pragma unroll
  for (int b = 0; b < kBits; ++b) {
    const bool set = choice & (1 << b);
    const uint32_t lanes = __ballot_sync(0xFFFFFFFFu, set);
    same &= lanes ^ (set ? 0u : 0xFFFFFFFFu);
  }
  return same;
}

// The choices in contiguous chunks, one per warp of the cluster, each a multiple of 32.
// Shared memory: first[kPlaceWarps][E]: a warp's choices per expert, then those before its next
// choice in the CTA; cta_total[E]: this CTA's choices per expert, read by the others; base[E]:
// the row of the CTA's first choice of an expert.  E <= 2^kBits.
template <int kBits>
__global__ void __launch_bounds__(kPlaceWarps * 32)
    place_kernel(const int32_t* ids, int32_t* dest, int64_t* m_sizes, int N, int E, int chunk) {
  extern __shared__ uint32_t place_shared[];
  uint32_t* first = place_shared;
  uint32_t* cta_total = place_shared + kPlaceWarps * E;
  uint32_t* base = cta_total + E;
  __shared__ uint32_t warp_total[kPlaceWarps];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const uint32_t rank = ptx::cluster_ctarank();
  for (int i = threadIdx.x; i < kPlaceWarps * E; i += blockDim.x) first[i] = 0;
  ptx::griddep_wait();
  ptx::griddep_launch_dependents();
  __syncthreads();
  uint32_t* mine = first + warp * E;
  const int64_t begin = (static_cast<int64_t>(rank) * kPlaceWarps + warp) * chunk;
  const int64_t end = begin + chunk < N ? begin + chunk : N;
  for (int64_t i0 = begin; i0 < end; i0 += 32 * kAhead) {
    int choice[kAhead];
    load_choices(ids, i0, end, E, choice);
#pragma unroll
    for (int r = 0; r < kAhead; ++r)
      if (choice[r] >= 0) atomicAdd(&mine[choice[r]], 1u);  // whole numbers, in any order
  }
  __syncthreads();
  // one expert per thread (E <= 1024): the warps' counts become offsets within the CTA
  const int e = threadIdx.x;
  uint32_t sum = 0;
  if (e < E) {
#pragma unroll
    for (int w = 0; w < kPlaceWarps; ++w) {
      const uint32_t c = first[w * E + e];
      first[w * E + e] = sum;
      sum += c;
    }
    cta_total[e] = sum;
  }
  ptx::cluster_sync();
  uint32_t before = 0, total = 0;
  if (e < E) {
    const uint32_t at = ptx::smem_addr(cta_total + e);
#pragma unroll
    for (uint32_t r = 0; r < kCluster; ++r) {
      const uint32_t c = ptx::ld_shared_cluster_u32(ptx::mapa_shared(at, r));
      if (r < rank) before += c;
      total += c;
    }
    if (rank == 0) m_sizes[e] = total;
  }
  uint32_t scan = total;  // inclusive, over the experts
#pragma unroll
  for (int d = 1; d < 32; d <<= 1) {
    const uint32_t v = __shfl_up_sync(0xFFFFFFFFu, scan, d);
    if (lane >= d) scan += v;
  }
  if (lane == 31) warp_total[warp] = scan;
  __syncthreads();
  uint32_t warps_before = warp_total[lane];
  warps_before = __reduce_add_sync(0xFFFFFFFFu, lane < warp ? warps_before : 0u);
  if (e < E) base[e] = warps_before + scan - total + before;
  ptx::cluster_sync();  // rows are set; nobody reads another CTA's shared memory any more
  for (int64_t i0 = begin; i0 < end; i0 += 32 * kAhead) {
    int choice[kAhead];
    load_choices(ids, i0, end, E, choice);
#pragma unroll
    for (int r = 0; r < kAhead; ++r) {
      if (i0 + r * 32 >= end) break;
      const int64_t i = i0 + r * 32 + lane;
      const uint32_t same = same_expert<kBits>(choice[r]);
      const uint32_t earlier = __popc(same & ((1u << lane) - 1u));
      const uint32_t next = choice[r] >= 0 ? mine[choice[r]] : 0;
      __syncwarp();
      if (choice[r] >= 0 && earlier == 0) mine[choice[r]] = next + __popc(same);
      __syncwarp();
      if (i < end)
        dest[i] = choice[r] >= 0 ? static_cast<int32_t>(base[choice[r]] + next + earlier) : -1;
    }
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

// A token's row is read once, 16 bytes (kWide) or one byte at a time, and written to each of
// its rows.  A lane of each warp holds one of them, `own` (-1: none); their load and the
// row's are under way together.
template <bool kWide>
__device__ __forceinline__ void copy_row(const CopyParams& p, int64_t t, int32_t own) {
  using Piece = std::conditional_t<kWide, uint4, uint8_t>;
  const Piece* from = reinterpret_cast<const Piece*>(p.x + t * p.row_bytes);
  const int n = static_cast<int>(p.row_bytes / sizeof(Piece));
  for (int c0 = 0; c0 < n; c0 += blockDim.x) {
    const int c = c0 + threadIdx.x;
    Piece v{};
    if (c < n) v = from[c];
    for (int j = 0; j < p.top_k; ++j) {
      const int32_t d = __shfl_sync(0xFFFFFFFFu, own, j);
      if (d >= 0 && c < n) reinterpret_cast<Piece*>(p.x_out + d * p.row_bytes)[c] = v;
    }
  }
  for (int c0 = 0; c0 < p.scale_cols; c0 += blockDim.x) {
    const int c = c0 + threadIdx.x;
    float v = 0.f;
    if (c < p.scale_cols) v = p.x_scale[t * p.scale_cols + c];
    for (int j = 0; j < p.top_k; ++j) {
      const int32_t d = __shfl_sync(0xFFFFFFFFu, own, j);
      if (d >= 0 && c < p.scale_cols)
        p.scale_out[static_cast<int64_t>(d) * p.scale_cols + c] = v;
    }
  }
}

// One CTA per token.
template <bool kWide>
__global__ void __launch_bounds__(512) copy_kernel(const __grid_constant__ CopyParams p) {
  ptx::griddep_wait();
  ptx::griddep_launch_dependents();
  const int64_t t = blockIdx.x;
  const int lane = threadIdx.x & 31;
  copy_row<kWide>(p, t, lane < p.top_k ? p.dest[t * p.top_k + lane] : -1);
}

// Few choices: one launch.  The CTA of a token finds each of its rows by itself:
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
  uint32_t count = 0;  // lane j: of the token's choice j
  for (int i0 = 0; i0 < N; i0 += blockDim.x) {
    const int i = i0 + threadIdx.x;
    int e = i < N ? p.ids[i] : -1;
    if (e < 0 || e >= p.E) e = 0x7FFFFFFF;
    for (int j = 0; j < k; ++j) {
      const int mine = __shfl_sync(0xFFFFFFFFu, own, j);
      const uint32_t earlier =
          __ballot_sync(0xFFFFFFFFu, e < mine || (e == mine && i < first + j));
      if (lane == j) count += __popc(earlier);
    }
  }
  if (lane < k) atomicAdd(&before[lane], count);  // whole numbers: any order is the same
  __syncthreads();
  own = own >= 0 ? static_cast<int>(before[lane]) : -1;
  if (threadIdx.x < k) p.dest[first + threadIdx.x] = own;
  copy_row<kWide>(p.copy, blockIdx.x, own);
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

mslkb_status mslkb_moe_dispatch(const void* x, const float* x_scale, const int32_t* ids,
                                void* x_out, float* scale_out, int64_t* m_sizes, int32_t* dest,
                                int64_t T, int64_t top_k, int64_t E, int64_t row_bytes,
                                int64_t scale_cols, void* stream) {
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
  const int experts = static_cast<int>(E);
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
  const int64_t per_warp = (N + kCluster * kPlaceWarps - 1) / (kCluster * kPlaceWarps);
  const auto place = experts <= 256 ? place_kernel<8> : place_kernel<10>;
  cudaError_t e = experts <= 256 ? allow_smem<place_kernel<8>>() : allow_smem<place_kernel<10>>();
  if (e == cudaSuccess)
    e = launch_cluster(place, dim3(kCluster), dim3(kPlaceWarps * 32),
                       sizeof(uint32_t) * experts * (kPlaceWarps + 2), kCluster, stream, ids, dest,
                       m_sizes, static_cast<int>(N), experts,
                       static_cast<int>((per_warp + 31) / 32 * 32));
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
