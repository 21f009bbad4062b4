// grad_norm.cu -- the norm of a list of gradients taken together, and the gradients scaled so that
// it does not exceed a bound.
//
//   norm = (sum_i sum_j g_ij^2)^(1/2)  or  max |g_ij|
//   out_ij = g_ij * (norm + eps <= max_norm ? 1 : max_norm / (norm + eps))
//
// Bound by memory: everything is read once for the norm, and read again and written once for the
// clipping.  The list is cut into chunks of kChunkBytes, and every CTA takes an equal run of them
// across the tensors' borders (small tensors by its warps in turn), so that many small tensors and
// a few large ones load the SMs alike; where a tensor starts is looked up in the kernel's
// parameters (no copy of the list to the device, so that a call can be captured).  Partial sums go
// to the workspace and are added in a fixed order.  The clipping walks each CTA's run backwards:
// what the norm read last is still in L2.  A short list is one launch of one cluster, which
// exchanges its sums through shared memory.
//
// Sums.  A square overflows fp32 from 2^64 on and is lost below 2^-63, and a gradient that has run
// away or died has such elements; so a vector of 16 bytes whose largest magnitude is outside
// [2^-50, 2^50] has its elements scaled by 2^-70 or 2^100 before they are squared, and sums of its
// own.  (Beside an element of 2^-50 those below 2^-63 do not matter.)  A batch of at most 32
// squares is summed in fp32 and then added to a pair of fp32 numbers without loss (the two-sum
// of Knuth), so that long runs of equal values do not drift; the pairs of the threads and CTAs are
// added in fp64.
#include <algorithm>
#include <atomic>
#include <cmath>
#include <cstring>
#include <type_traits>
#include <vector>

#include "host.h"
#include "rows.cuh"

namespace mslkb {
namespace {

constexpr int kThreads = 512;
constexpr int kChunkBytes = 4096;
constexpr int kMaxParts = 512;            // CTAs of a launch, and partial sums of it
// Tensors of a launch, by the size of its parameters.
constexpr int kFew = 64, kSome = 256, kMany = 1024;
constexpr int kCluster = 16;       // most CTAs of a cluster
constexpr int kSmallChunks = 512;  // of a list that one cluster takes

// A list of tensors and the chunks before each.
template <int kMost>
struct List {
  struct Tensor {
    const void* in;
    void* out;
    int64_t size;             // elements * 4 + type
  } t[kMost];
  uint32_t first[kMost + 1];  // chunks before tensor i
  uint16_t start[kMaxParts + 1];   // the tensor of run r's first chunk (the last chunk's past it)
  int32_t count;
};

__host__ __device__ inline uint32_t share(uint32_t total, uint32_t i, uint32_t of) {
  return static_cast<uint32_t>(static_cast<uint64_t>(total) * i / of);
}

// A sum in two fp32 numbers.
struct Pair {
  float hi = 0.f, lo = 0.f;
  __device__ __forceinline__ void add(float v) {
    const float t = hi + v, b = t - hi;
    lo += (hi - (t - b)) + (v - b);
    hi = t;
  }
  __device__ __forceinline__ void add_lanes() {   // of a warp, all lanes get the sum
#pragma unroll
    for (int m = 16; m > 0; m >>= 1) {
      const float l = __shfl_xor_sync(0xffffffffu, lo, m);
      add(__shfl_xor_sync(0xffffffffu, hi, m));
      lo += l;
    }
  }
  __device__ __forceinline__ double value() const {
    // (beside an infinite hi, lo is infinity less infinity)
    return isinf(hi) ? static_cast<double>(hi) : static_cast<double>(hi) + static_cast<double>(lo);
  }
};

struct Sums {   // of squares, of squares scaled by 2^-140 and 2^200; the largest magnitude's bits
  Pair mid, big, small;
  uint32_t most = 0u;
};

constexpr float kBigFrom = 1125899906842624.f;             // 2^50
constexpr float kSmallTo = 8.8817841970012523e-16f;        // 2^-50
constexpr float kUp = 1.2676506002282294e30f;              // 2^100
constexpr float kDown = 8.4703294725430034e-22f;           // 2^-70

template <bool kInf, int kN>
__device__ __forceinline__ void take(Sums& s, float& batch, const float (&v)[kN]) {
  if constexpr (kInf) {
#pragma unroll
    for (int j = 0; j < kN; ++j) s.most = max(s.most, __float_as_uint(v[j]) & 0x7FFFFFFFu);
  } else {
    float top = 0.f;
#pragma unroll
    for (int j = 0; j < kN; ++j) top = fmaxf(top, fabsf(v[j]));
    if (top >= kSmallTo && top <= kBigFrom) {
#pragma unroll
      for (int j = 0; j < kN; ++j) batch = fmaf(v[j], v[j], batch);
    } else {  // (NaN beside zeros only: in the small ones' sum)
      const bool big = top > kBigFrom;
      const float f = big ? kDown : kUp;
      float sum = 0.f;
#pragma unroll
      for (int j = 0; j < kN; ++j) sum = fmaf(v[j] * f, v[j] * f, sum);
      if (big) s.big.add(sum);
      else s.small.add(sum);
    }
  }
}

template <class T>
__device__ __forceinline__ void unpack16(uint4 w, float (&v)[16 / sizeof(T)]) {
  if constexpr (sizeof(T) == 4) {
    v[0] = __uint_as_float(w.x), v[1] = __uint_as_float(w.y);
    v[2] = __uint_as_float(w.z), v[3] = __uint_as_float(w.w);
  } else {
    const uint32_t u[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const float2 f = unpack2(u[i], T());
      v[2 * i] = f.x, v[2 * i + 1] = f.y;
    }
  }
}
template <class T>
__device__ __forceinline__ uint4 pack16(const float (&v)[16 / sizeof(T)]) {
  if constexpr (sizeof(T) == 4)
    return make_uint4(__float_as_uint(v[0]), __float_as_uint(v[1]), __float_as_uint(v[2]),
                      __float_as_uint(v[3]));
  else
    return make_uint4(pack2(v[0], v[1], T()), pack2(v[2], v[3], T()), pack2(v[4], v[5], T()),
                      pack2(v[6], v[7], T()));
}

// Elements up to the next 16-byte boundary, at most n.
template <class T>
__device__ __forceinline__ int64_t head_of(const T* p, int64_t n) {
  const int64_t h = static_cast<int64_t>((16 - (reinterpret_cast<uintptr_t>(p) & 15)) & 15) /
                    static_cast<int64_t>(sizeof(T));
  return h < n ? h : n;
}

// Vectors of a thread under way.
template <int kStep>
constexpr int kBatchOf = kStep == 32 ? 8 : 4;

// By kStep threads, of which this is `tid`.
template <bool kInf, int kStep, class T>
__device__ void sum_run(const T* p, int64_t n, Sums& s, int tid) {
  constexpr int kN = 16 / sizeof(T);
  const int64_t head = head_of(p, n);
  const T* mid = p + head;
  const int64_t vecs = (n - head) / kN, tail = n - head - vecs * kN;
  constexpr int kBatch = kBatchOf<kStep>;
  // the ends, fewer than kN elements each
  const float edge = tid < head + tail ? to_float(tid < head ? p[tid] : mid[vecs * kN + tid - head])
                                       : 0.f;
  int64_t i = tid;
  for (; i + (kBatch - 1) * kStep < vecs; i += kBatch * kStep) {
    uint4 w[kBatch];
#pragma unroll
    for (int u = 0; u < kBatch; ++u) w[u] = load16(mid + (i + u * kStep) * kN);
    float even = 0.f, odd = 0.f;
#pragma unroll
    for (int u = 0; u < kBatch; ++u) {
      float v[kN];
      unpack16<T>(w[u], v);
      take<kInf>(s, (u & 1) ? odd : even, v);
    }
    if (!kInf) s.mid.add(even + odd);
  }
  if (i < vecs) {   // fewer vectors than a batch
    uint4 w[kBatch - 1];
#pragma unroll
    for (int u = 0; u < kBatch - 1; ++u)
      w[u] = i + u * kStep < vecs ? load16(mid + (i + u * kStep) * kN) : make_uint4(0u, 0u, 0u, 0u);
#pragma unroll
    for (int u = 0; u < kBatch - 1; ++u) {
      float v[kN], batch = 0.f;
      unpack16<T>(w[u], v);
      if (i + u * kStep < vecs) take<kInf>(s, batch, v);
      if (!kInf) s.mid.add(batch);
    }
  }
  if (tid < head + tail) {
    const float v[1] = {edge};
    float batch = 0.f;
    take<kInf>(s, batch, v);
    if (!kInf) s.mid.add(batch);
  }
}

template <int kStep, int kBatch, class T>
__device__ void scale_run(const T* p, T* o, int64_t n, float f, int tid) {
  constexpr int kN = 16 / sizeof(T);
  // whole vectors where both lie alike, else element by element
  const bool alike = ((reinterpret_cast<uintptr_t>(p) ^ reinterpret_cast<uintptr_t>(o)) & 15) == 0;
  const int64_t head = alike ? head_of(p, n) : n;
  const int64_t vecs = (n - head) / kN;
  const T* pm = p + head;
  T* om = o + head;
  auto one = [&](int64_t at, uint4 w) {
    float v[kN];
    unpack16<T>(w, v);
#pragma unroll
    for (int j = 0; j < kN; ++j) v[j] *= f;
    __stcs(reinterpret_cast<uint4*>(om + at * kN), pack16<T>(v));
  };
  const int64_t tail = n - head - vecs * kN;
  const bool at_head = alike && tid < head;
  const float edge = at_head ? to_float(p[tid]) : 0.f;
  const float last = tid < tail ? to_float(pm[vecs * kN + tid]) : 0.f;
  int64_t i = vecs - 1 - tid;   // from the end: what was read last is in L2
  for (; i - (kBatch - 1) * kStep >= 0; i -= kBatch * kStep) {
    uint4 w[kBatch];
#pragma unroll
    for (int u = 0; u < kBatch; ++u) w[u] = load16(pm + (i - u * kStep) * kN);
#pragma unroll
    for (int u = 0; u < kBatch; ++u) one(i - u * kStep, w[u]);
  }
  if (i >= 0) {
    uint4 w[kBatch - 1];
#pragma unroll
    for (int u = 0; u < kBatch - 1; ++u)
      if (i - u * kStep >= 0) w[u] = load16(pm + (i - u * kStep) * kN);
#pragma unroll
    for (int u = 0; u < kBatch - 1; ++u)
      if (i - u * kStep >= 0) one(i - u * kStep, w[u]);
  }
  if (at_head) o[tid] = from_float<T>(edge * f);
  if (tid < tail) om[vecs * kN + tid] = from_float<T>(last * f);
  if (!alike)
    for (int64_t k = tid; k < head; k += kStep) o[k] = from_float<T>(to_float(p[k]) * f);
}

// Run `r` of `of`, tensor by tensor: f(tensor, first element, elements).
template <bool kBack, class L, class F>
__device__ __forceinline__ void each_run(const L& l, uint32_t r, uint32_t of, F f) {
  const uint32_t total = l.first[l.count];
  const uint32_t c0 = share(total, r, of), c1 = share(total, r + 1, of);
  if (c0 >= c1) return;
  for (int i = l.start[kBack ? r + 1 : r]; i >= 0 && i < l.count; i += kBack ? -1 : 1) {
    const uint32_t a = l.first[i], b = l.first[i + 1];
    if (kBack ? b <= c0 : a >= c1) break;
    const auto& t = l.t[i];
    const int64_t size = t.size >> 2;
    const int64_t each = kChunkBytes / ((t.size & 3) == MSLKB_FP32 ? 4 : 2);
    const int64_t e0 = a > c0 ? 0 : static_cast<int64_t>(c0 - a) * each;
    const int64_t e1 = b <= c1 ? size : min(size, static_cast<int64_t>(c1 - a) * each);
    if (a < c1 && e1 > e0) f(t, e0, e1 - e0);
  }
}

template <class F>
__device__ __forceinline__ void by_type(int64_t size, F f) {
  switch (size & 3) {
    case MSLKB_BF16: return f(__nv_bfloat16());
    case MSLKB_FP16: return f(__half());
    default: return f(0.f);
  }
}

// By whom a run's part of a tensor is taken: kStep threads of the run together, or, few bytes of it
// by a CTA's warps in turn, so that the latencies of small tensors side by side pass together (two
// tensors of 0.5 GB and 100 of 2 KB on GB300, us for norm / clipping: 164 / 507 so, 235 / 610 by
// the CTA).
constexpr int64_t kAlone = 4 * kChunkBytes;
template <int kStep, class T, class F>
__device__ __forceinline__ void share_out(int64_t n, uint32_t& turn, F f) {
  if (kStep > 32 && n * static_cast<int64_t>(sizeof(T)) <= kAlone) {
    if (turn++ % (kStep / 32) == threadIdx.x >> 5)
      f(std::integral_constant<int, 32>(), static_cast<int>(threadIdx.x & 31u));
  } else {
    f(std::integral_constant<int, kStep>(), static_cast<int>(threadIdx.x) % kStep);
  }
}

template <bool kInf, int kStep, class L>
__device__ __forceinline__ Sums sum_chunks(const L& l, uint32_t r, uint32_t of) {
  Sums s;
  uint32_t turn = 0;
  each_run<false>(l, r, of, [&](const auto& g, int64_t e0, int64_t n) {
    by_type(g.size, [&](auto t) {
      using T = decltype(t);
      share_out<kStep, T>(n, turn, [&](auto step, int tid) {
        sum_run<kInf, decltype(step)::value>(static_cast<const T*>(g.in) + e0, n, s, tid);
      });
    });
  });
  return s;
}

template <int kStep, class L>
__device__ __forceinline__ void scale_chunks(const L& l, uint32_t r, uint32_t of, float f) {
  uint32_t turn = 0;
  each_run<true>(l, r, of, [&](const auto& g, int64_t e0, int64_t n) {
    if (f == 1.f && g.in == g.out) return;   // nothing changes
    by_type(g.size, [&](auto t) {
      using T = decltype(t);
      share_out<kStep, T>(n, turn, [&](auto step, int tid) {
        constexpr int kBy = decltype(step)::value;
        // (a warp beside others of its CTA: four vectors, not eight; of clip_kernel, which has 64
        // registers a thread, 112 bytes spill even so)
        constexpr int kBatch = kBy < kStep ? 4 : kBatchOf<kBy>;
        scale_run<kBy, kBatch>(static_cast<const T*>(g.in) + e0, static_cast<T*>(g.out) + e0, n, f,
                               tid);
      });
    });
  });
}

// The fp64 unit of an SM takes 16 cycles for an operation of a warp, so one warp does those, and
// the others wait (done by all 16 warps of two CTAs, sums and root took 13 us).
struct Joined {
  Pair mid, big, small;
};

// A CTA's sum of squares, or (kInf) largest magnitude, in the lanes of warp 0, as fp64.
template <bool kInf>
__device__ __forceinline__ double cta_sum(Sums s, Joined* shared) {
  const uint32_t lane = threadIdx.x & 31u, warp = threadIdx.x >> 5;
  constexpr uint32_t kWarps = kThreads / 32;
  if constexpr (kInf) {
    const uint32_t m = __reduce_max_sync(0xffffffffu, s.most);
    if (lane == 0) shared[warp].mid.hi = __uint_as_float(m);
    __syncthreads();
    if (warp != 0) return 0.0;
    const uint32_t mine = lane < kWarps ? __float_as_uint(shared[lane].mid.hi) : 0u;
    return static_cast<double>(__uint_as_float(__reduce_max_sync(0xffffffffu, mine)));
  } else {
    s.mid.add_lanes();
    if (__any_sync(0xffffffffu, s.big.hi != 0.f || s.small.hi != 0.f)) {
      s.big.add_lanes();
      s.small.add_lanes();
    }
    if (lane == 0) shared[warp] = {s.mid, s.big, s.small};
    __syncthreads();
    if (warp != 0) return 0.0;
    const Joined j = lane < kWarps ? shared[lane] : Joined{};
    double d = j.mid.value();
    if (__any_sync(0xffffffffu, j.big.hi != 0.f || j.small.hi != 0.f))
      d += j.big.value() * 1.3937965749081639e+42 +     // 2^140
           j.small.value() * 6.2230152778611417e-61;    // 2^-200
#pragma unroll
    for (int m = kWarps / 2; m > 0; m >>= 1) d += __shfl_xor_sync(0xffffffffu, d, m);
    return d;
  }
}

__device__ __forceinline__ double join(bool inf, double a, double b) {
  if (!inf) return a + b;
  return a != a || b != b ? a + b : (a > b ? a : b);   // (a NaN stays)
}

// Where partial sums come together.
struct Together {
  double part[kThreads];
  float norm;
};

// The norm from `count` partial sums, in every thread of the CTA: fetched by all threads at once,
// added by one warp.
template <bool kInf>
__device__ __forceinline__ float norm_of(const double* parts, int count, Together& t) {
  double d = 0.0;
  for (int i0 = 0; i0 < count; i0 += kThreads) {
    const int i = i0 + static_cast<int>(threadIdx.x);
    if (i0 > 0) __syncthreads();
    if (i < count) t.part[threadIdx.x] = parts[i];
    __syncthreads();
    if (threadIdx.x < 32)
      for (int k = static_cast<int>(threadIdx.x); k < min(kThreads, count - i0); k += 32)
        d = join(kInf, d, t.part[k]);
  }
  if (threadIdx.x < 32) {
#pragma unroll
    for (int m = 16; m > 0; m >>= 1) d = join(kInf, d, __shfl_xor_sync(0xffffffffu, d, m));
    const float norm = static_cast<float>(kInf ? d : sqrt(d));
    if (threadIdx.x == 0) t.norm = norm;
  }
  __syncthreads();
  return t.norm;
}

// The scale: the quotient is only taken where it is below 1, so that neither an infinite bound over an
// infinite norm nor 0 / 0 comes into it.  (A NaN stays.)
__device__ __forceinline__ float scale_of(float norm, float max_norm, float eps) {
  const float n = norm + eps;
  return n <= max_norm ? 1.f : max_norm / n;
}

struct ClipArgs {
  float* norm;
  double* parts;
  int32_t part0;       // of this launch's first partial sum
  int32_t part_count;  // of all launches
  float max_norm, eps;
  int32_t write_norm;
};

template <bool kInf, int kMost>
__global__ void __launch_bounds__(kThreads, 2)
    norm_parts_kernel(const __grid_constant__ List<kMost> l, const __grid_constant__ ClipArgs a) {
  __shared__ Joined shared[kThreads / 32];
  if (threadIdx.x == 0) ptx::griddep_launch_dependents();
  ptx::griddep_wait();
  const Sums s = sum_chunks<kInf, kThreads>(l, blockIdx.x, gridDim.x);
  const double d = cta_sum<kInf>(s, shared);
  if (threadIdx.x == 0) a.parts[a.part0 + blockIdx.x] = d;
}

template <bool kInf>
__global__ void __launch_bounds__(kThreads) norm_total_kernel(const __grid_constant__ ClipArgs a) {
  __shared__ Together together;
  if (threadIdx.x == 0) ptx::griddep_launch_dependents();
  ptx::griddep_wait();
  const float norm = norm_of<kInf>(a.parts, a.part_count, together);
  if (threadIdx.x == 0) *a.norm = norm;
}

template <bool kInf, int kMost>
__global__ void __launch_bounds__(kThreads, 2)
    clip_kernel(const __grid_constant__ List<kMost> l, const __grid_constant__ ClipArgs a) {
  __shared__ Together together;
  if (threadIdx.x == 0) ptx::griddep_launch_dependents();
  ptx::griddep_wait();
  const float norm = norm_of<kInf>(a.parts, a.part_count, together);
  if (a.write_norm && blockIdx.x == 0 && threadIdx.x == 0) *a.norm = norm;
  scale_chunks<kThreads>(l, blockIdx.x, gridDim.x, scale_of(norm, a.max_norm, a.eps));
}

// A short list: one cluster, which sums and, if wanted, scales.  The runs are the warps', so that
// the latencies of many small tensors pass together.
template <bool kInf, bool kClip>
__global__ void __launch_bounds__(kThreads)
    small_list_kernel(const __grid_constant__ List<kFew> list, const __grid_constant__ ClipArgs a) {
  // The list in shared memory, fetched while the kernel before this one ends: read where it is
  // needed, each of its lines would be a miss of the constant cache in its own turn.
  __shared__ List<kFew> l;
  static_assert(sizeof(l) % 4 == 0, "copied by words");
  for (int i = static_cast<int>(threadIdx.x); i < static_cast<int>(sizeof(l) / 4); i += kThreads)
    reinterpret_cast<uint32_t*>(&l)[i] = reinterpret_cast<const uint32_t*>(&list)[i];
  __syncthreads();
  __shared__ Joined shared[kThreads / 32];
  __shared__ double all[kCluster];
  if (threadIdx.x == 0) ptx::griddep_launch_dependents();
  if (gridDim.x > 1) ptx::cluster_arrive();   // (waited for before others' memory is written)
  ptx::griddep_wait();
  const uint32_t rank = blockIdx.x, of = gridDim.x;
  const uint32_t warp = rank * (kThreads / 32) + (threadIdx.x >> 5), warps = of * (kThreads / 32);
  const Sums s = sum_chunks<kInf, 32>(l, warp, warps);
  const double d = cta_sum<kInf>(s, shared);
  if (of > 1) {
    ptx::cluster_wait();
    if (threadIdx.x == 0) {
      const uint32_t mine = ptx::smem_addr(all + rank);
      const uint64_t bits = static_cast<uint64_t>(__double_as_longlong(d));
      for (uint32_t r = 0; r < of; ++r) {
        const uint32_t to = ptx::mapa_shared(mine, r);
        ptx::st_shared_cluster_u32(to, static_cast<uint32_t>(bits));
        ptx::st_shared_cluster_u32(to + 4u, static_cast<uint32_t>(bits >> 32));
      }
    }
    ptx::cluster_sync();
  } else {
    if (threadIdx.x == 0) all[0] = d;
    __syncthreads();
  }
  __shared__ Together together;
  const float norm = norm_of<kInf>(all, static_cast<int>(of), together);
  if (rank == 0 && threadIdx.x == 0) *a.norm = norm;
  if constexpr (kClip) scale_chunks<32>(l, warp, warps, scale_of(norm, a.max_norm, a.eps));
}

// ---------------------------------------------------------------------------------------
// host
// ---------------------------------------------------------------------------------------
struct Args {
  const void* const* in;
  void* const* out;   // null: the norm alone
  const int64_t* sizes;
  const int32_t* types;
  int64_t count;
};

int64_t chunks_of(int64_t size, int32_t type) {
  const int64_t each = kChunkBytes / dtype_bytes(type);
  return (size + each - 1) / each;
}

template <int kMost>
void fill(List<kMost>* l, const Args& a, int64_t from, int64_t to) {
  uint32_t chunks = 0;
  l->count = static_cast<int32_t>(to - from);
  for (int64_t i = from; i < to; ++i) {
    const int64_t k = i - from;
    l->t[k] = {a.in[i], a.out != nullptr ? a.out[i] : nullptr, a.sizes[i] * 4 + a.types[i]};
    l->first[k] = chunks;
    chunks += static_cast<uint32_t>(chunks_of(a.sizes[i], a.types[i]));
  }
  l->first[to - from] = chunks;
}

// Where each of `runs` runs starts, and for those that walk back where it ends: start[r] is the
// tensor of chunk share(r), start[runs] that of the last chunk (a run that walks back starts at
// the tensor of the next run's first chunk, and passes over it where that is not its own).
template <int kMost>
void cut(List<kMost>* l, int runs) {
  const uint32_t total = l->first[l->count];
  int i = 0;
  for (int r = 0; r <= runs; ++r) {
    uint32_t c = share(total, static_cast<uint32_t>(r), static_cast<uint32_t>(runs));
    if (c == total && total > 0) --c;
    while (i + 1 < l->count && l->first[i + 1] <= c) ++i;
    l->start[r] = static_cast<uint16_t>(i);
  }
}

template <bool kInf, int kMost>
cudaError_t run_list(const Args& a, ClipArgs c, int sms, void* stream) {
  const int64_t launches = (a.count + kMost - 1) / kMost;
  const int most = std::min(2 * sms, kMaxParts);
  auto each = [&](auto f) -> cudaError_t {
    c.part0 = 0;
    for (int64_t i = 0; i < launches; ++i) {
      List<kMost> l;
      fill(&l, a, i * kMost, std::min(a.count, (i + 1) * kMost));
      const int grid = static_cast<int>(
          std::min<int64_t>(most, std::max<int64_t>(1, l.first[l.count])));
      cut(&l, grid);
      const cudaError_t e = f(l, grid, i);
      if (e != cudaSuccess) return e;
      c.part0 += grid;
    }
    return cudaSuccess;
  };
  cudaError_t e = each([&](const List<kMost>& l, int grid, int64_t) {
    return launch_dependent(norm_parts_kernel<kInf, kMost>, dim3(grid), dim3(kThreads), 0, stream,
                            l, c);
  });
  if (e != cudaSuccess) return e;
  c.part_count = c.part0;
  if (a.out == nullptr)
    return launch_dependent(norm_total_kernel<kInf>, dim3(1), dim3(kThreads), 0, stream, c);
  return each([&](const List<kMost>& l, int grid, int64_t i) {
    c.write_norm = i == 0;
    return launch_dependent(clip_kernel<kInf, kMost>, dim3(grid), dim3(kThreads), 0, stream, l, c);
  });
}

// CTAs that a cluster of `kKernel` can have on this device: 16, or 8 where 16 do not fit.
template <auto kKernel>
cudaError_t most_ctas(int* ctas) {
  static std::atomic<int8_t> known[64];
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  std::atomic<int8_t>& mine = known[dev & 63];
  if ((*ctas = mine.load()) != 0) return cudaSuccess;
  e = cudaFuncSetAttribute(kKernel, cudaFuncAttributeNonPortableClusterSizeAllowed, 1);
  if (e != cudaSuccess) return e;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(kCluster);
  cfg.blockDim = dim3(kThreads);
  cudaLaunchAttribute attr;
  attr.id = cudaLaunchAttributeClusterDimension;
  attr.val.clusterDim.x = kCluster;
  attr.val.clusterDim.y = attr.val.clusterDim.z = 1;
  cfg.attrs = &attr;
  cfg.numAttrs = 1;
  int fit = 0;
  e = cudaOccupancyMaxActiveClusters(&fit, kKernel, &cfg);
  if (e != cudaSuccess) return e;
  *ctas = fit > 0 ? kCluster : 8;
  mine.store(static_cast<int8_t>(*ctas));
  return cudaSuccess;
}

template <bool kInf, bool kClip>
cudaError_t run_small(List<kFew>& l, const ClipArgs& c, void* stream) {
  // a chunk per warp, as far as they go: 1, 8 or 16 CTAs
  const uint32_t chunks = l.first[l.count];
  int grid = chunks <= kThreads / 32 ? 1 : 8;
  if (chunks > 8 * kThreads / 32) {
    const cudaError_t e = most_ctas<small_list_kernel<kInf, kClip>>(&grid);
    if (e != cudaSuccess) return e;
  }
  cut(&l, grid * (kThreads / 32));
  return launch_cluster(small_list_kernel<kInf, kClip>, dim3(grid), dim3(kThreads), 0, grid,
                        stream, l, c);
}

template <bool kInf>
cudaError_t run(const Args& a, const ClipArgs& c, int sms, void* stream) {
  if (a.count <= kFew) {
    int64_t chunks = 0;
    for (int64_t i = 0; i < a.count; ++i) chunks += chunks_of(a.sizes[i], a.types[i]);
    if (chunks <= kSmallChunks) {
      List<kFew> l;
      fill(&l, a, 0, a.count);
      return a.out != nullptr ? run_small<kInf, true>(l, c, stream)
                              : run_small<kInf, false>(l, c, stream);
    }
  }
  if (a.count <= kFew) return run_list<kInf, kFew>(a, c, sms, stream);
  if (a.count <= kSome) return run_list<kInf, kSome>(a, c, sms, stream);
  return run_list<kInf, kMany>(a, c, sms, stream);
}

// Whether no result (the norm is one) lies over another, or over a gradient other than its own.
bool apart(const Args& a, const float* norm) {
  struct Span {
    uintptr_t from, to;
    bool written;
  };
  std::vector<Span> spans;
  spans.reserve(static_cast<size_t>(2 * a.count));
  for (int64_t i = 0; i < a.count; ++i) {
    const uintptr_t bytes = static_cast<uintptr_t>(a.sizes[i]) * dtype_bytes(a.types[i]);
    if (bytes == 0) continue;
    const uintptr_t o = reinterpret_cast<uintptr_t>(a.out[i]);
    const uintptr_t g = reinterpret_cast<uintptr_t>(a.in[i]);
    spans.push_back({o, o + bytes, true});
    if (g != o) spans.push_back({g, g + bytes, false});
  }
  auto before = [](const Span& x, const Span& y) { return x.from < y.from; };
  if (!std::is_sorted(spans.begin(), spans.end(), before))
    std::sort(spans.begin(), spans.end(), before);
  const uintptr_t at = reinterpret_cast<uintptr_t>(norm);
  uintptr_t any = 0, written = 0;   // ends of the spans so far, of those that are written
  for (const Span& s : spans) {
    if (s.from < (s.written ? any : written)) return false;
    if (at < s.to && s.from < at + sizeof *norm) return false;
    any = std::max(any, s.to);
    if (s.written) written = std::max(written, s.to);
  }
  return true;
}

mslkb_status run_checked(const Args& a, int32_t kind, float* norm, double max_norm, double eps,
                         void* workspace, int64_t workspace_bytes, void* stream,
                         const char* name) try {
  if (a.count < 0 || a.count > MSLKB_MAX_TENSORS ||
      (kind != MSLKB_NORM_2 && kind != MSLKB_NORM_INF))
    return MSLKB_ERR_SHAPE;
  if (norm == nullptr) return MSLKB_ERR_NULL;
  if (a.count > 0 && (a.in == nullptr || a.sizes == nullptr || a.types == nullptr))
    return MSLKB_ERR_NULL;
  int64_t chunks = 0;
  for (int64_t i = 0; i < a.count; ++i) {
    if (!dtype_ok(a.types[i])) return MSLKB_ERR_DTYPE;
    if (a.sizes[i] < 0 || a.sizes[i] > (1ll << 40)) return MSLKB_ERR_SHAPE;
    if (a.sizes[i] > 0 && (a.in[i] == nullptr || (a.out != nullptr && a.out[i] == nullptr)))
      return MSLKB_ERR_NULL;
    const size_t width = static_cast<size_t>(dtype_bytes(a.types[i]));
    if (!aligned_to(a.in[i], width) || (a.out != nullptr && !aligned_to(a.out[i], width)))
      return MSLKB_ERR_ALIGN;
    chunks += chunks_of(a.sizes[i], a.types[i]);
    if (chunks > INT32_MAX) return MSLKB_ERR_SHAPE;
  }
  if (!aligned_to(norm, 4)) return MSLKB_ERR_ALIGN;
  if (workspace == nullptr || !aligned_to(workspace, 16) ||
      workspace_bytes < mslkb_grad_norm_workspace_bytes(a.count))
    return MSLKB_ERR_WORKSPACE;
  if (a.out != nullptr && !apart(a, norm)) return MSLKB_ERR_SHAPE;
  int sms = 0;
  const mslkb_status s = device_sms(&sms);
  if (s != MSLKB_OK) return s;
  ClipArgs c{};
  c.norm = norm;
  c.parts = static_cast<double*>(workspace);
  c.max_norm = static_cast<float>(max_norm);
  c.eps = static_cast<float>(eps);
  const TraceRange range(name, a.count);
  return launch_status(kind == MSLKB_NORM_INF ? run<true>(a, c, sms, stream)
                                              : run<false>(a, c, sms, stream));
} catch (...) {   // (no room for the list of spans)
  return launch_status(cudaErrorMemoryAllocation);
}

}  // namespace
}  // namespace mslkb

extern "C" {

int64_t mslkb_grad_norm_workspace_bytes(int64_t count) {
  using namespace mslkb;
  if (count < 0 || count > MSLKB_MAX_TENSORS) return 0;
  const int64_t launches = (count + kMany - 1) / kMany;
  return (launches > 0 ? launches : 1) * kMaxParts * static_cast<int64_t>(sizeof(double));
}

mslkb_status mslkb_grad_norm(const void* const* grads, const int64_t* sizes, const int32_t* dtypes,
                             int64_t count, int32_t kind, float* norm, void* workspace,
                             int64_t workspace_bytes, void* stream) {
  const mslkb::Args a{grads, nullptr, sizes, dtypes, count};
  return mslkb::run_checked(a, kind, norm, 0.0, 0.0, workspace, workspace_bytes, stream,
                            "grad_norm");
}

mslkb_status mslkb_clip_grad_norm(const void* const* grads, void* const* outs,
                                  const int64_t* sizes, const int32_t* dtypes, int64_t count,
                                  int32_t kind, double max_norm, double eps, float* norm,
                                  void* workspace, int64_t workspace_bytes, void* stream) {
  if (!(max_norm >= 0.0) || !(eps >= 0.0) || std::isinf(eps)) return MSLKB_ERR_SHAPE;
  if (count > 0 && outs == nullptr) return MSLKB_ERR_NULL;
  static void* const none[1] = {nullptr};
  const mslkb::Args a{grads, outs != nullptr ? outs : none, sizes, dtypes, count};
  return mslkb::run_checked(a, kind, norm, max_norm, eps, workspace, workspace_bytes, stream,
                            "clip_grad_norm");
}

}  // extern "C"
