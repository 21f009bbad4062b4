// dispatch.cu -- the rows of the chosen experts: packed by expert into the stacked layout
// (dispatch), and summed back per token with the routing weights (combine), with the gradient.
#include "host.h"
#include "rows.cuh"

namespace mslkb {
namespace {

// ---------------------------------------------------------------------------------
// dispatch: a stable counting sort of the choices by expert (place_kernel: the row of every
// choice), then each token's row is read once and written to its rows (copy_kernel).  The
// copies are bound by HBM's writes (GB300, 8192 tokens x 8 rows of 7168 bytes: 82 us, 6.6 TB/s);
// the sort in front of them (6.5 us for 65536 choices among 256 experts, 25 us for 524288) by the
// ballots that number a warp's choices and by latency, so it is one kernel of one cluster, whose
// 8 or 16 CTAs exchange their counts through distributed shared memory.
// ---------------------------------------------------------------------------------
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

// Numbers a warp's choices: each one's position among the warp's of its expert, of which
// mine[expert] came before (and counts on).  Of the kAhead steps those of `left` choices.
template <int kBits>
__device__ __forceinline__ void number_choices(const int (&choice)[kAhead], int64_t left,
                                               uint32_t* mine, uint32_t (&position)[kAhead]) {
  const uint32_t lower = (1u << (threadIdx.x & 31)) - 1u;
  uint32_t same[kAhead];
#pragma unroll
  for (int r = 0; r < kAhead; ++r)
    if (r * 32 < left) same[r] = same_expert<kBits>(choice[r]);
#pragma unroll
  for (int r = 0; r < kAhead; ++r) {
    if (r * 32 >= left) break;
    const uint32_t earlier = __popc(same[r] & lower);
    const uint32_t next = choice[r] >= 0 ? mine[choice[r]] : 0;
    __syncwarp();
    if (choice[r] >= 0 && earlier == 0) mine[choice[r]] = next + __popc(same[r]);
    __syncwarp();
    position[r] = next + earlier;
  }
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
  const uint32_t rank = ptx::cluster_ctarank(), ranks = gridDim.x;  // one cluster
  for (int i = threadIdx.x; i < kPlaceWarps * E; i += blockDim.x) first[i] = 0;
  ptx::griddep_wait();
  ptx::griddep_launch_dependents();
  __syncthreads();
  uint32_t* mine = first + warp * E;
  const int64_t begin = (static_cast<int64_t>(rank) * kPlaceWarps + warp) * chunk;
  const int64_t end = begin + chunk < N ? begin + chunk : N;
  // a warp with no more than these keeps their numbers
  int choice[kAhead];
  uint32_t position[kAhead];
  const bool once = chunk <= 32 * kAhead;
  for (int64_t i0 = begin; i0 < end; i0 += 32 * kAhead) {
    load_choices(ids, i0, end, E, choice);
    if (once) {
      number_choices<kBits>(choice, end - i0, mine, position);
    } else {
#pragma unroll
      for (int r = 0; r < kAhead; ++r)
        if (choice[r] >= 0) atomicAdd(&mine[choice[r]], 1u);  // whole numbers, in any order
    }
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
#pragma unroll 8
    for (uint32_t r = 0; r < ranks; ++r) {
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
    if (!once) {  // mine now counts from the warps before on
      load_choices(ids, i0, end, E, choice);
      number_choices<kBits>(choice, end - i0, mine, position);
    }
#pragma unroll
    for (int r = 0; r < kAhead; ++r) {
      const int64_t i = i0 + r * 32 + lane;
      const int e = choice[r];
      uint32_t to = 0xFFFFFFFFu;
      if (e >= 0) to = base[e] + position[r] + (once ? mine[e] : 0);
      if (i < end) dest[i] = static_cast<int32_t>(to);
    }
  }
}

struct CopyParams {
  const uint8_t* x;
  const float* x_scale;
  const int32_t* dest;
  uint8_t* x_out;
  float* scale_out;
  int64_t row_bytes, T;
  int32_t scale_cols;
  int32_t top_k;
  int64_t ahead;  // tokens of the CTAs that an SM full of them starts with
};

template <class Piece>
__device__ __forceinline__ Piece load_piece(const Piece* p) {
  if constexpr (sizeof(Piece) == 32)
    return load32(p);
  else
    return *p;
}
template <class Piece>
__device__ __forceinline__ void store_piece(Piece* p, const Piece& v) {
  if constexpr (sizeof(Piece) == 32)
    store32(p, v);
  else
    *p = v;
}

// A token's row is read once, a Piece (32, 16, 8, 4, 2 or 1 bytes) at a time, and written to each
// of its rows.  A lane of each warp holds one of them, `own` (-1: none); their load and the
// row's are under way together.
template <class Piece>
__device__ __forceinline__ void copy_row(const CopyParams& p, int64_t t, int32_t own) {
  const Piece* from = reinterpret_cast<const Piece*>(p.x + t * p.row_bytes);
  const int n = static_cast<int>(p.row_bytes / sizeof(Piece));
  for (int c0 = 0; c0 < n; c0 += blockDim.x) {
    const int c = c0 + threadIdx.x;
    Piece v{};
    if (c < n) v = load_piece(from + c);
    for (int j = 0; j < p.top_k; ++j) {
      const int32_t d = __shfl_sync(0xFFFFFFFFu, own, j);
      if (d >= 0 && c < n) store_piece(reinterpret_cast<Piece*>(p.x_out + d * p.row_bytes) + c, v);
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

// Rows per waiting CTA and token.  GB300, 0 / 1 / 2 / 4, us: 8192 tokens x 8 rows of 7168 bytes
// 89.7 / 88.8 / 88.8 / 89.6, x 2 33.5 / 32.2 / 31.3 / 31.4, 16384 x 1 of 4096 26.9 / 25.6 / 24.8.
constexpr int kRowsAhead = 2;

// blockDim.y tokens per CTA, whole warps per token.
template <class Piece>
__global__ void __launch_bounds__(512) copy_kernel(const __grid_constant__ CopyParams p) {
  const int64_t t = static_cast<int64_t>(blockIdx.x) * blockDim.y + threadIdx.y;
  // While the sort runs, the CTAs that wait for it have the first rows brought to L2 (x itself
  // is there already: the sort's CTAs let this kernel start after their own wait)
  if (t < p.ahead) {
#pragma unroll
    for (int r = 0; r < kRowsAhead; ++r) {
      const int64_t row = t + r * p.ahead;
      if (row < p.T)
        for (int64_t c = threadIdx.x * 128; c < p.row_bytes; c += blockDim.x * 128)
          ptx::prefetch_l2(p.x + row * p.row_bytes + c);
    }
  }
  ptx::griddep_wait();
  ptx::griddep_launch_dependents();
  const int lane = threadIdx.x & 31;
  if (t >= p.T) return;
  const int32_t own = lane < p.top_k ? p.dest[t * p.top_k + lane] : -1;
  if (__any_sync(0xFFFFFFFFu, own >= 0)) copy_row<Piece>(p, t, own);
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

template <class Piece>
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
  copy_row<Piece>(p.copy, blockIdx.x, own);
}

// ---------------------------------------------------------------------------------
// combine and its gradient: 8 columns per thread and step.  Bound by HBM: GB300, bf16 rows of
// 7168, 8111 tokens x 8 combined in 148 us (7.0 TB/s, nearly all of it reads), the gradient of
// 4096 x 8 in 150 us (6.7 TB/s).
// ---------------------------------------------------------------------------------
struct CombineParams {
  const void* rows;
  const int32_t* dest;
  const float* weights;
  void* out;
  int64_t T, H, R;
  int32_t top_k;
};

// Every warp of a token holds its choices, one per lane: the row (-1: none) and the weight.
struct Choice {
  int32_t row;
  float weight;
};
__device__ __forceinline__ Choice load_choice(const int32_t* dest, const float* weights,
                                              int64_t t, int top_k, int64_t R) {
  const int lane = threadIdx.x & 31;
  Choice c{-1, 0.f};
  if (lane < top_k) {
    const int32_t d = dest[t * top_k + lane];
    if (d >= 0 && d < R) {
      c.row = d;
      c.weight = weights != nullptr ? weights[t * top_k + lane] : 1.f;
    }
  }
  return c;
}

// The next kAhead choices that have a row, off the bits of `left`: their lanes (-1: none left).
template <int kAhead>
__device__ __forceinline__ void take_choices(uint32_t& left, int (&lane)[kAhead]) {
#pragma unroll
  for (int j = 0; j < kAhead; ++j) {
    lane[j] = __ffs(left) - 1;
    left &= left - 1;
  }
}

// blockDim.y tokens per CTA, whole warps per token.
template <class T, Access kAccess>
__global__ void __launch_bounds__(512) combine_kernel(const __grid_constant__ CombineParams p) {
  ptx::griddep_wait();
  ptx::griddep_launch_dependents();
  const int64_t t = static_cast<int64_t>(blockIdx.x) * blockDim.y + threadIdx.y;
  if (t >= p.T) return;
  const int n = static_cast<int>(p.H);
  const Choice own = load_choice(p.dest, p.weights, t, p.top_k, p.R);
  const uint32_t there = __ballot_sync(0xFFFFFFFFu, own.row >= 0);
  const T* rows = static_cast<const T*>(p.rows);
  constexpr int kRound = 4;
  for (int c0 = 0; c0 < n; c0 += blockDim.x * 8) {
    const int c = c0 + threadIdx.x * 8;
    float sum[8] = {};
    for (uint32_t left = there; left != 0;) {
      int from[kRound];
      take_choices(left, from);
      Raw8<T> r[kRound];
#pragma unroll
      for (int j = 0; j < kRound; ++j) {
        const int32_t row = __shfl_sync(0xFFFFFFFFu, own.row, from[j] & 31);
        if (from[j] >= 0) r[j] = load8<T, kAccess>(rows + row * p.H, c, n);
      }
#pragma unroll
      for (int j = 0; j < kRound; ++j) {
        const float w = __shfl_sync(0xFFFFFFFFu, own.weight, from[j] & 31);
        if (from[j] >= 0) {
          float v[8];
          unpack8(r[j], v);
#pragma unroll
          for (int i = 0; i < 8; ++i) sum[i] = fmaf(w, v[i], sum[i]);
        }
      }
    }
    store8<T, kAccess>(static_cast<T*>(p.out) + t * p.H, c, n, sum);
  }
}

struct CombineBackwardParams {
  const void* dout;
  const void* rows;
  const int32_t* dest;
  const float* weights;
  void* drows;
  float* dweights;
  int64_t T, H, R;
  int32_t top_k;
};

// kRound rows at a time; dout is read again for each round.
template <class T, Access kAccess, int kRound>
__global__ void __launch_bounds__(512)
    combine_backward_kernel(const __grid_constant__ CombineBackwardParams p) {
  __shared__ float partial[MSLKB_MAX_TOPK][16];  // per warp
  ptx::griddep_wait();
  ptx::griddep_launch_dependents();
  const int64_t t = static_cast<int64_t>(blockIdx.x) * blockDim.y + threadIdx.y;
  const int n = static_cast<int>(p.H);
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, warps = blockDim.x >> 5;
  const bool token = t < p.T;
  const Choice own = token ? load_choice(p.dest, p.weights, t, p.top_k, p.R) : Choice{-1, 0.f};
  const T* dout = static_cast<const T*>(p.dout) + t * p.H;
  float mine = 0.f;  // lane j: this warp's part of the j-th choice's dot product
  for (uint32_t left = __ballot_sync(0xFFFFFFFFu, own.row >= 0); left != 0;) {
    int from[kRound];
    int32_t row[kRound];
    float w[kRound], dot[kRound] = {};
    take_choices(left, from);
#pragma unroll
    for (int j = 0; j < kRound; ++j) {
      row[j] = __shfl_sync(0xFFFFFFFFu, own.row, from[j] & 31);
      w[j] = __shfl_sync(0xFFFFFFFFu, own.weight, from[j] & 31);
    }
    for (int c = threadIdx.x * 8; c - static_cast<int>(threadIdx.x) * 8 < n; c += blockDim.x * 8) {
      float d[8];
      unpack8(load8<T, kAccess>(dout, c, n), d);
      Raw8<T> r[kRound];
#pragma unroll
      for (int j = 0; j < kRound; ++j)
        if (from[j] >= 0)
          r[j] = load8<T, kAccess>(static_cast<const T*>(p.rows) + row[j] * p.H, c, n);
#pragma unroll
      for (int j = 0; j < kRound; ++j) {
        if (from[j] >= 0) {
          float v[8];
          unpack8(r[j], v);
#pragma unroll
          for (int i = 0; i < 8; ++i) {
            dot[j] = fmaf(d[i], v[i], dot[j]);
            v[i] = w[j] * d[i];
          }
          store8<T, kAccess>(static_cast<T*>(p.drows) + row[j] * p.H, c, n, v);
        }
      }
    }
#pragma unroll
    for (int j = 0; j < kRound; ++j) {
      const float s = warp_sum(dot[j]);
      if (lane == from[j]) mine = s;
    }
  }
  if (warps > 1) {  // one token per CTA
    if (lane < p.top_k) partial[lane][warp] = mine;
    __syncthreads();
    if (warp > 0) return;
    mine = 0.f;
    if (lane < p.top_k)
      for (int i = 0; i < warps; ++i) mine += partial[lane][i];
  }
  if (token && lane < p.top_k) p.dweights[t * p.top_k + lane] = mine;
}

// ---------------------------------------------------------------------------------
// launches
// ---------------------------------------------------------------------------------
// Threads over a row of `steps`: x along the row, whole warps, in as few and even rounds as
// `most` allow; with `tokens`, y rows per CTA, 256 threads together, where a warp is enough for
// each.
dim3 row_threads(int64_t steps, bool tokens, int most = 512) {
  const int64_t rounds = (steps + most - 1) / most;
  const int64_t each = rounds > 0 ? (steps + rounds - 1) / rounds : 0;
  const int64_t x = each <= 32 ? 32 : (each + 31) / 32 * 32;
  return dim3(static_cast<unsigned>(x), tokens && x == 32 ? 8 : 1);
}

dim3 token_grid(int64_t T, dim3 block) {
  return dim3(static_cast<unsigned>((T + block.y - 1) / block.y));
}

// Each token's CTA finds its rows by itself for up to so many choices, and up to so many
// comparisons of one choice with another token's.  GB300, rows of 2048 bytes, alone against
// sort and copy, us: 8 choices a token, 512 choices 3.0 / 6.2, 2048 6.3 / 7.0, 3072 9.5 / 7.3;
// one choice a token, 1024 4.1 / 5.8, 1536 6.5 / 6.2, 2048 8.7 / 6.5.
constexpr int64_t kDirectComparisons = 3 << 19;
constexpr int64_t kDirectChoices = 2048;

// Threads per token (GB300, bf16, 512 / 256 / 128): 8192 tokens x 8 of 7168 149 / 153 / 153 us,
// x 2 58.3 / 53.8 / 53.8, x 1 47.0 / 41.3 / 40.7: with few rows a thread takes more columns.
template <class T>
cudaError_t launch_combine(const CombineParams& p, bool wide, void* stream) {
  const dim3 block = row_threads((p.H + 7) / 8, true, p.top_k > 4 ? 512 : 256);
  const dim3 grid = token_grid(p.T, block);
  return wide ? launch_dependent(combine_kernel<T, Access::k16>, grid, block, 0, stream, p)
              : launch_dependent(combine_kernel<T, Access::kStride>, grid, block, 0, stream, p);
}

// Rows at a time by top_k: all of up to eight, as each round reads dout again (GB300, 4096
// tokens x 8 of 7168 bf16: 8 / 4 / 2 at a time 150 / 161 / 192 us; 8192 x 2: 102 / 101 / 94).
// 128 threads per token: 256 take 163 us, 64 173 us on the first.  Few tokens take as many as
// there are columns for (91 x 6 of 7168, one in ten here: 128 threads 6.2 us, 448 3.8 us).
template <class T, Access kAccess>
cudaError_t launch_combine_backward(const CombineBackwardParams& p, int sms, void* stream) {
  dim3 block = row_threads((p.H + 7) / 8, true, p.T > 4 * sms ? 128 : 512);
  if (block.y > 1) block.y = 4;
  const dim3 grid = token_grid(p.T, block);
  if (p.top_k <= 2)
    return launch_dependent(combine_backward_kernel<T, kAccess, 2>, grid, block, 0, stream, p);
  if (p.top_k <= 4)
    return launch_dependent(combine_backward_kernel<T, kAccess, 4>, grid, block, 0, stream, p);
  return launch_dependent(combine_backward_kernel<T, kAccess, 8>, grid, block, 0, stream, p);
}

template <class T>
cudaError_t launch_combine_backward(const CombineBackwardParams& p, int sms, bool wide,
                                    void* stream) {
  return wide ? launch_combine_backward<T, Access::k16>(p, sms, stream)
              : launch_combine_backward<T, Access::kStride>(p, sms, stream);
}

size_t place_smem(int experts) { return sizeof(uint32_t) * experts * (kPlaceWarps + 2); }

// CTAs of the sort, one cluster: 16, or the portable 8 where the device has no 16 SMs together
// to give.  Asked once per device.
template <auto kKernel>
cudaError_t place_ctas(int* ctas) {
  static std::atomic<int8_t> known[64];
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  std::atomic<int8_t>& mine = known[dev & 63];
  if ((*ctas = mine.load()) != 0) return cudaSuccess;
  e = allow_smem<kKernel>();
  if (e == cudaSuccess)
    e = cudaFuncSetAttribute(kKernel, cudaFuncAttributeNonPortableClusterSizeAllowed, 1);
  if (e != cudaSuccess) return e;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(16);
  cfg.blockDim = dim3(kPlaceWarps * 32);
  cfg.dynamicSmemBytes = place_smem(MSLKB_MAX_EXPERTS);
  cudaLaunchAttribute attr;
  attr.id = cudaLaunchAttributeClusterDimension;
  attr.val.clusterDim.x = 16;
  attr.val.clusterDim.y = attr.val.clusterDim.z = 1;
  cfg.attrs = &attr;
  cfg.numAttrs = 1;
  int clusters = 0;
  if ((e = cudaOccupancyMaxActiveClusters(&clusters, kKernel, &cfg)) != cudaSuccess) return e;
  *ctas = clusters > 0 ? 16 : 8;
  mine.store(static_cast<int8_t>(*ctas));
  return cudaSuccess;
}

// Dispatch with rows copied in Pieces.
template <class Piece>
cudaError_t launch_dispatch(CopyParams p, int sms, const int32_t* ids, int32_t* dest,
                            int64_t* m_sizes, int64_t T, int64_t E, void* stream) {
  const int64_t steps = p.row_bytes / static_cast<int64_t>(sizeof(Piece)), N = T * p.top_k;
  const int experts = static_cast<int>(E);
  if (N <= kDirectChoices && N * T <= kDirectComparisons) {
    const DirectParams d{p, ids, dest, m_sizes, static_cast<int32_t>(T), experts};
    dim3 block = row_threads(steps, false);
    if (block.x < 256) block.x = 256;  // they share the counting too
    return launch_dependent(direct_kernel<Piece>, dim3(static_cast<unsigned>(T) + 1), block, 0,
                            stream, d);
  }
  const auto place = experts <= 256 ? place_kernel<8> : place_kernel<10>;
  int ctas = 0;
  cudaError_t e = experts <= 256 ? place_ctas<place_kernel<8>>(&ctas)
                                 : place_ctas<place_kernel<10>>(&ctas);
  if (e != cudaSuccess) return e;
  // us: 4320 choices by 8 CTAs 4.2, by 16 4.5; 16384 4.8 and 4.9; 65536 8.0 and 6.5
  if (N <= 16384) ctas = 8;
  const int64_t per_warp = (N + ctas * kPlaceWarps - 1) / (ctas * kPlaceWarps);
  e = launch_cluster(place, dim3(static_cast<unsigned>(ctas)), dim3(kPlaceWarps * 32),
                     place_smem(experts), ctas, stream, ids, dest, m_sizes, static_cast<int>(N),
                     experts, static_cast<int>((per_warp + 31) / 32 * 32));
  if (e == cudaSuccess && (p.row_bytes > 0 || p.scale_cols > 0)) {
    // 32 bytes a thread against 16 and twice the threads, us: 8192 tokens x 8 of 7168, all here,
    // 91.1 / 90.3, one in four here 36.6 / 43.3; x 2 33.3 / 39.3; 16384 x 1 of 4096 26.9 / 31.9
    dim3 block = row_threads(steps, false);
    if (block.x <= 128) block.y = 256 / block.x;
    p.ahead = static_cast<int64_t>(sms) * (2048 / (block.x * block.y)) * block.y;
    e = launch_dependent(copy_kernel<Piece>, token_grid(T, block), block, 0, stream, p);
  }
  return e;
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
  if (E > MSLKB_MAX_EXPERTS || top_k > MSLKB_MAX_TOPK || row_bytes > (1 << 30) ||
      scale_cols > (1 << 30) || (top_k > 0 && T > MSLKB_MAX_DIM / 2 / top_k) ||
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
  const CopyParams p{static_cast<const uint8_t*>(x), x_scale, dest, static_cast<uint8_t*>(x_out),
                     scale_out, row_bytes, T, static_cast<int32_t>(scale_cols),
                     static_cast<int32_t>(top_k), 0};
  const auto fits = [&](int64_t piece) {
    return row_bytes % piece == 0 && aligned_to(x, piece) && aligned_to(x_out, piece);
  };
  TraceRange range("moe_dispatch", T);
  cudaError_t e;
  if (fits(32))
    e = launch_dispatch<Words8>(p, sms, ids, dest, m_sizes, T, E, stream);
  else if (fits(16))
    e = launch_dispatch<uint4>(p, sms, ids, dest, m_sizes, T, E, stream);
  else if (fits(8))
    e = launch_dispatch<uint2>(p, sms, ids, dest, m_sizes, T, E, stream);
  else if (fits(4))
    e = launch_dispatch<uint32_t>(p, sms, ids, dest, m_sizes, T, E, stream);
  else if (fits(2))
    e = launch_dispatch<uint16_t>(p, sms, ids, dest, m_sizes, T, E, stream);
  else
    e = launch_dispatch<uint8_t>(p, sms, ids, dest, m_sizes, T, E, stream);
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
  const CombineParams p{rows, dest, weights, out, T, H, R, static_cast<int32_t>(top_k)};
  TraceRange range("moe_combine", T);
  cudaError_t e;
  if (dtype == MSLKB_BF16)
    e = launch_combine<__nv_bfloat16>(p, wide, stream);
  else if (dtype == MSLKB_FP16)
    e = launch_combine<__half>(p, wide, stream);
  else
    e = launch_combine<float>(p, wide, stream);
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
  const CombineBackwardParams p{dout, rows, dest, weights, drows, dweights, T, H, R,
                                static_cast<int32_t>(top_k)};
  TraceRange range("moe_combine_backward", T);
  cudaError_t e;
  if (dtype == MSLKB_BF16)
    e = launch_combine_backward<__nv_bfloat16>(p, sms, wide, stream);
  else if (dtype == MSLKB_FP16)
    e = launch_combine_backward<__half>(p, sms, wide, stream);
  else
    e = launch_combine_backward<float>(p, sms, wide, stream);
  return launch_status(e);
}

}  // extern "C"
