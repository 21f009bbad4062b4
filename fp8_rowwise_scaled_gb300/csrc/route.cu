// route.cu -- the choice of each token's experts from the router's logits, and its gradient.
//
// One warp per token.  A lane holds up to kPer consecutive experts in registers (of one group,
// where the groups are a power of two: their lanes divide each evenly), as integer keys that
// order like their choice values, so that the largest of the warp is one redux instruction.
// Bound by instructions, not by memory: 256 experts are 8 scores per lane, and top_k dependent
// maxima.  The loop over the maxima is kept short by sorting each lane's keys once, with the
// expert's index in place of the key's lowest bits: keys are then unique, the lane that holds the
// maximum drops its first key, and the maximum itself names the expert.  Where the bits that gave
// way to the index decide, the chosen are put in the order of their exact values, or, where
// another expert comes that close, chosen again by exact keys.
// GB300, 16384 tokens x 256 experts, top 8: softmax 8 us, sigmoid + bias 12 us, with 4 of 8
// groups 13.8 us (some 800 instructions per token at 0.8 a cycle; the logits alone are 2.6 us
// of HBM); taking the maxima from unsorted keys took 21.9 us.
#include "host.h"
#include "rows.cuh"

namespace mslkb {
namespace {

constexpr int kWarps = 4;  // tokens per CTA
constexpr float kMasked = -__builtin_huge_valf();

struct RouteParams {
  const void* logits;
  const float* bias;
  int32_t* ids;
  float* weights;
  int64_t T, ld;
  int32_t E, top_k;
  int32_t groups, top_groups, group_top;
  int32_t per_group;    // experts of a group
  int32_t whole;        // each group has 2^group_shift lanes of its own; no groups: all 32
  int32_t dealt;        // those lanes have room for more than their group
  int32_t group_shift;  // if not whole, log2 of the lanes that look through a group
  int32_t renormalize;
  int32_t wide, wide_bias;  // lanes' experts in whole, aligned pieces
  float scale;
};

// What experts are chosen by: the logits (a softmax keeps their order), or the score + bias.
enum class Score { kLogits, kSoftmax, kSigmoid };

// An integer that orders as the float does: NaN above all; -inf, which masks, is kMaskedKey,
// and nothing else comes that low.
constexpr uint32_t kMaskedKey = 0x007FFFFFu;
__device__ __forceinline__ uint32_t order_key(float v) {
  const uint32_t b = __float_as_uint(v + 0.f);  // -0 as +0, every NaN as the one above +inf
  return b ^ (static_cast<uint32_t>(static_cast<int32_t>(b) >> 31) | 0x80000000u);
}
__device__ __forceinline__ float key_value(uint32_t k) {
  return __uint_as_float(k & 0x80000000u ? k & 0x7FFFFFFFu : ~k);
}

// (the IEEE forms: the choice is defined by the rounded scores)
__device__ __forceinline__ float sigmoid_of(float x) { return 1.f / (1.f + expf(-x)); }

// What a group is worth: its best choice, and with group_top = 2 the second as well.
__device__ __forceinline__ uint32_t worth_key(uint32_t best, uint32_t second, int group_top) {
  if (group_top == 1 || second <= kMaskedKey) return best;
  return order_key(key_value(best) + key_value(second));
}

// Descending order of a lane's keys (odd-even merge sort; Batcher 1968).
template <int kN>
__device__ __forceinline__ void sort_keys(uint32_t (&s)[kN]) {
#pragma unroll
  for (int p = 1; p < kN; p *= 2)
#pragma unroll
    for (int k = p; k >= 1; k /= 2)
#pragma unroll
      for (int j = k % p; j + k < kN; j += 2 * k)
#pragma unroll
        for (int i = 0; i < k; ++i)
          if (i + j + k < kN && (i + j) / (2 * p) == (i + j + k) / (2 * p)) {
            const uint32_t a = s[i + j], b = s[i + j + k];
            s[i + j] = max(a, b);
            s[i + j + k] = min(a, b);
          }
}

// Bytes of the pieces in which a lane reads kPer consecutive elements, where they are aligned.
template <class T, int kPer>
__host__ __device__ constexpr int piece_bytes() {
  constexpr int n = kPer * static_cast<int>(sizeof(T));
  return n % 16 == 0 ? 16 : (n % 8 == 0 ? 8 : static_cast<int>(sizeof(T)));
}

// `count` (of kPer) consecutive floats, `fill` past them.
template <class T, int kPer>
__device__ __forceinline__ void load_lane(const T* from, int count, bool wide, float fill,
                                          float (&x)[kPer]) {
  constexpr int kBytes = piece_bytes<T, kPer>();
  if constexpr (kBytes > static_cast<int>(sizeof(T))) {
    if (wide) {
      constexpr int kPiece = kBytes / sizeof(T);
#pragma unroll
      for (int i = 0; i < kPer; i += kPiece) {
        const bool in = i < count;
        uint32_t w[kBytes / 4] = {};
        if constexpr (kBytes == 16) {
          const uint4 r = in ? load16(from + i) : make_uint4(0, 0, 0, 0);
          w[0] = r.x, w[1] = r.y, w[2] = r.z, w[3] = r.w;
        } else {
          const uint2 r = in ? *reinterpret_cast<const uint2*>(from + i) : make_uint2(0, 0);
          w[0] = r.x, w[1] = r.y;
        }
#pragma unroll
        for (int j = 0; j < kBytes / 4; ++j) {
          if constexpr (sizeof(T) == 4) {
            x[i + j] = in ? __uint_as_float(w[j]) : fill;
          } else {
            const float2 f = unpack2(w[j], T());
            x[i + 2 * j] = in ? f.x : fill;
            x[i + 2 * j + 1] = in ? f.y : fill;
          }
        }
      }
      return;
    }
  }
#pragma unroll
  for (int i = 0; i < kPer; ++i) x[i] = i < count ? to_float(from[i]) : fill;
}

__host__ __device__ constexpr uint32_t index_mask(int n) {  // 2^b - 1 for the least 2^b >= n
  uint32_t m = 1;
  while (m < static_cast<uint32_t>(n)) m *= 2;
  return m - 1;
}

// Where expert e's key lies in shared memory: lanes kPer experts apart fall into other banks.
__host__ __device__ __forceinline__ constexpr int padded(int e) { return e + (e >> 5); }

// The two largest keys of each run of 2^shift lanes, from those of its lanes.
__device__ __forceinline__ void merge_best(uint32_t& best, uint32_t& second, int shift) {
  for (int d = 1; d < 1 << shift; d <<= 1) {
    const uint32_t b = __shfl_xor_sync(0xFFFFFFFFu, best, d);
    const uint32_t s = __shfl_xor_sync(0xFFFFFFFFu, second, d);
    second = max(max(second, s), min(best, b));
    best = max(best, b);
  }
}

// How many of the groups are worth more than this lane's, `mine`, ties to the lower group.
// Lane g << shift holds what group g is worth; a group's lanes share the comparisons.
__device__ __forceinline__ int better_groups(uint32_t mine, int group, int groups, int shift) {
  const int lane = threadIdx.x & 31, lanes = 1 << shift;
  int better = 0;
  for (int g0 = 0; g0 < groups; g0 += lanes) {
    const int g = g0 + (lane & (lanes - 1));
    const uint32_t other = __shfl_sync(0xFFFFFFFFu, mine, (g << shift) & 31);
    better += g < groups && (other > mine || (other == mine && g < group));
  }
  for (int d = 1; d < lanes; d <<= 1) better += __shfl_xor_sync(0xFFFFFFFFu, better, d);
  return better;
}

template <class T, int kPer, Score kScore>
__global__ void __launch_bounds__(kWarps * 32)
    route_kernel(const __grid_constant__ RouteParams p) {
  extern __shared__ uint32_t shared_keys[];  // [kWarps][padded(E)], groups that are not whole
  ptx::griddep_wait();
  ptx::griddep_launch_dependents();
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int64_t t = static_cast<int64_t>(blockIdx.x) * kWarps + warp;
  if (t >= p.T) return;
  const T* row = static_cast<const T*>(p.logits) + t * p.ld;
  // the lane's experts, first ... first + count - 1
  int first = lane * kPer, count = p.E - first;
  if (p.dealt) {
    const int within = (lane & ((1 << p.group_shift) - 1)) * kPer;
    first = (lane >> p.group_shift) * p.per_group + within;
    count = p.per_group - within;
  }

  float x[kPer];
  load_lane<T, kPer>(row + first, count, p.wide, kMasked, x);

  // softmax over all experts: its maximum and sum
  float top = 0.f, total = 1.f;
  if (kScore == Score::kSoftmax || (kScore == Score::kLogits && !p.renormalize)) {
    float m = x[0];
#pragma unroll
    for (int i = 1; i < kPer; ++i) m = fmaxf(m, x[i]);
#pragma unroll
    for (int d = 16; d > 0; d >>= 1) m = fmaxf(m, __shfl_xor_sync(0xFFFFFFFFu, m, d));
    float s = 0.f;
#pragma unroll
    for (int i = 0; i < kPer; ++i)
      if (i < count) s += expf(x[i] - m);  // a NaN logit makes the sum NaN
    top = m;
    total = warp_sum(s);
  }
  // the key of an expert with logit v and bias b (0 without): masked by its logit or its bias
  auto choice_key = [&](float v, float b) {
    if constexpr (kScore == Score::kLogits) return order_key(v);
    const float c = (kScore == Score::kSigmoid ? sigmoid_of(v) : expf(v - top) / total) + b;
    return order_key(v == kMasked ? v : c);
  };
  uint32_t key[kPer];
  {
    float b[kPer];
    if (kScore != Score::kLogits && p.bias != nullptr) {
      load_lane<float, kPer>(p.bias + first, count, p.wide_bias, 0.f, b);
    } else {
#pragma unroll
      for (int i = 0; i < kPer; ++i) b[i] = 0.f;
    }
#pragma unroll
    for (int i = 0; i < kPer; ++i) key[i] = choice_key(x[i], b[i]);
  }

  if (p.groups > 1) {
    if (p.whole) {
      uint32_t best = 0, second = 0;
#pragma unroll
      for (int i = 0; i < kPer; ++i) {
        second = max(second, min(best, key[i]));
        best = max(best, key[i]);
      }
      merge_best(best, second, p.group_shift);
      const uint32_t mine = worth_key(best, second, p.group_top);
      if (better_groups(mine, lane >> p.group_shift, p.groups, p.group_shift) >= p.top_groups) {
#pragma unroll
        for (int i = 0; i < kPer; ++i) key[i] = 0;
      }
    } else {
      const int per = p.per_group;
      uint32_t* keys = shared_keys + warp * padded(p.E);
#pragma unroll
      for (int i = 0; i < kPer; ++i)
        if (i < count) keys[padded(first + i)] = key[i];
      __syncwarp();
      const int mine_group = lane >> p.group_shift, lanes = 1 << p.group_shift;
      uint32_t best = 0, second = 0;
      if (mine_group < p.groups) {
        for (int i = lane & (lanes - 1); i < per; i += lanes) {
          const uint32_t k = keys[padded(mine_group * per + i)];
          second = max(second, min(best, k));
          best = max(best, k);
        }
      }
      merge_best(best, second, p.group_shift);
      const uint32_t mine = worth_key(best, second, p.group_top);
      const int better = better_groups(mine, mine_group, p.groups, p.group_shift);
      const uint32_t kept = __ballot_sync(0xFFFFFFFFu, better < p.top_groups);
      // the groups of the lane's experts, from the first one's on
      int group = first / per, left = per - (first - group * per);
#pragma unroll
      for (int i = 0; i < kPer; ++i) {
        if (!((kept >> ((group << p.group_shift) & 31)) & 1u)) key[i] = 0;
        if (--left == 0) ++group, left = per;
      }
    }
  }

  // keys with the expert's index in the lowest bits, the lower index larger; a lane's keys as
  // sorted lists of at most eight (sorting 8 takes 19 comparisons, 32 would take 191)
  constexpr uint32_t kIndex = index_mask(32 * kPer);
  constexpr int kLists = (kPer + 7) / 8, kList = kPer / kLists;
  int id = -1;  // lane j: the j-th choice
  float logit = kMasked;
  {
    uint32_t s[kLists][kList];
#pragma unroll
    for (int l = 0; l < kLists; ++l) {
#pragma unroll
      for (int i = 0; i < kList; ++i)
        s[l][i] = (key[l * kList + i] & ~kIndex) | (kIndex - (first + l * kList + i));
      sort_keys(s[l]);
    }
    auto largest = [&] {
      uint32_t m = s[0][0];
#pragma unroll
      for (int l = 1; l < kLists; ++l) m = max(m, s[l][0]);
      return __reduce_max_sync(0xFFFFFFFFu, m);
    };
    uint32_t mine = 0;
    for (int j = 0; j < p.top_k; ++j) {
      const uint32_t m = largest();
      if (lane == j) mine = m;
#pragma unroll
      for (int l = 0; l < kLists; ++l) {
        if (s[l][0] == m) {  // one list of one lane, unless nothing is left
#pragma unroll
          for (int i = 0; i + 1 < kList; ++i) s[l][i] = s[l][i + 1];
          s[l][kList - 1] = 0;
        }
      }
    }
    if ((mine | kIndex) > kMaskedKey) {
      id = static_cast<int>(kIndex - (mine & kIndex));
      logit = to_float(row[id]);  // an L1 hit
    }
    // A logit of 16 bits has the index's bits to spare.  Otherwise the chosen are the right ones
    // if the next differs from the last in the bits kept, or, as with equal keys, nothing that
    // is above the least of them was left out; then only their order may be wrong.
    if constexpr (!(kScore == Score::kLogits && sizeof(T) == 2)) {
      const uint32_t next = largest();
      const float b = kScore != Score::kLogits && p.bias != nullptr && id >= 0 ? p.bias[id] : 0.f;
      const uint32_t exact = id >= 0 ? choice_key(logit, b) : 0;
      bool again = false;
      if (__any_sync(0xFFFFFFFFu,
                     id >= 0 && lane == p.top_k - 1 && ((mine ^ next) & ~kIndex) == 0)) {
        const uint32_t least = __reduce_min_sync(0xFFFFFFFFu, id >= 0 ? exact : 0xFFFFFFFFu);
        int above = 0;
#pragma unroll
        for (int i = 0; i < kPer; ++i) above += key[i] > least;
        above = __reduce_add_sync(0xFFFFFFFFu, above);
        again = above != __popc(__ballot_sync(0xFFFFFFFFu, id >= 0 && exact > least));
      }
      const uint32_t above_key = __shfl_up_sync(0xFFFFFFFFu, exact, 1);
      const int above_id = __shfl_up_sync(0xFFFFFFFFu, id, 1);
      const bool wrong =
          id >= 0 && lane > 0 && (above_key < exact || (above_key == exact && above_id > id));
      if (!again && __any_sync(0xFFFFFFFFu, wrong)) {
        int rank = 0;  // among the chosen
        for (int j = 0; j < p.top_k; ++j) {
          const uint32_t other = __shfl_sync(0xFFFFFFFFu, exact, j);
          const int other_id = __shfl_sync(0xFFFFFFFFu, id, j);
          rank += other > exact || (other == exact && other_id < id);
        }
        if (id < 0) rank = lane;  // those without an expert are last already
        int from = lane;
        for (int j = 0; j < p.top_k; ++j) {
          const int at = __ffs(__ballot_sync(0xFFFFFFFFu, lane < p.top_k && rank == j)) - 1;
          if (lane == j) from = at;
        }
        id = __shfl_sync(0xFFFFFFFFu, id, from);
        logit = __shfl_sync(0xFFFFFFFFu, logit, from);
      }
      if (again) {
        id = -1;
        for (int j = 0; j < p.top_k; ++j) {
          uint32_t best = key[0];
          int at = 0;
#pragma unroll
          for (int i = 1; i < kPer; ++i)
            if (key[i] > best) best = key[i], at = i;
          const uint32_t m = __reduce_max_sync(0xFFFFFFFFu, best);
          if (m <= kMaskedKey) break;
          const int winner = __ffs(__ballot_sync(0xFFFFFFFFu, best == m)) - 1;
          const int chosen = __shfl_sync(0xFFFFFFFFu, first + at, winner);
          if (lane == j) id = chosen;
#pragma unroll
          for (int i = 0; i < kPer; ++i)
            if (first + i == chosen) key[i] = 0;
        }
        logit = id >= 0 ? to_float(row[id]) : kMasked;
      }
    }
  }

  // weights, one choice per lane
  float w = 0.f;
  if (kScore == Score::kSigmoid) {
    if (id >= 0) w = sigmoid_of(logit);
    if (p.renormalize) w /= warp_sum(w) + 1e-20f;
  } else if (p.renormalize) {
    float m = logit;
#pragma unroll
    for (int d = 16; d > 0; d >>= 1) m = fmaxf(m, __shfl_xor_sync(0xFFFFFFFFu, m, d));
    if (id >= 0) w = expf(logit - m);
    w /= warp_sum(w);
  } else if (id >= 0) {
    w = expf(logit - top) / total;
  }
  if (lane < p.top_k) {
    p.ids[t * p.top_k + lane] = id;
    p.weights[t * p.top_k + lane] = id >= 0 ? w * p.scale : 0.f;
  }
}

// ---------------------------------------------------------------------------------
// gradient
// ---------------------------------------------------------------------------------
struct RouteBackwardParams {
  const float* dweights;
  const void* logits;
  const int32_t* ids;
  void* dlogits;
  int64_t T, ld;
  int32_t E, top_k;
  int32_t sigmoid;
  int32_t renormalize;
  float scale;
};

// One warp per token, its lanes take runs of kV experts in turn: what all experts get is written
// first, then the lanes of the chosen write theirs again, from the same values.
template <class T, int kV>
__device__ __forceinline__ void store_run(T* to, const float* v) {
  if constexpr (kV == 1) {
    *to = from_float<T>(v[0]);
  } else {
    uint32_t w[kV * sizeof(T) / 4];
#pragma unroll
    for (int j = 0; j < static_cast<int>(kV * sizeof(T) / 4); ++j) {
      if constexpr (sizeof(T) == 4)
        w[j] = __float_as_uint(v[j]);
      else
        w[j] = pack2(v[2 * j], v[2 * j + 1], T());
    }
    if constexpr (kV * sizeof(T) == 16)
      store16(to, make_uint4(w[0], w[1], w[2], w[3]));
    else
      *reinterpret_cast<uint2*>(to) = make_uint2(w[0], w[1]);
  }
}

template <class T, int kPer, int kV>
__global__ void __launch_bounds__(kWarps * 32)
    route_backward_kernel(const __grid_constant__ RouteBackwardParams p) {
  __shared__ int32_t sign[kWarps][32 * kPer];
  ptx::griddep_wait();
  ptx::griddep_launch_dependents();
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int64_t t = static_cast<int64_t>(blockIdx.x) * kWarps + warp;
  if (t >= p.T) return;
  const T* row = static_cast<const T*>(p.logits) + t * p.ld;
  T* out = static_cast<T*>(p.dlogits) + t * p.E;

  int id = -1;
  float g = 0.f;
  if (lane < p.top_k) {
    id = p.ids[t * p.top_k + lane];
    if (id < 0 || id >= p.E) id = -1;
    if (id >= 0) g = p.dweights[t * p.top_k + lane] * p.scale;
  }
  const float logit = id >= 0 ? to_float(row[id]) : kMasked;
  float mine;        // what the chosen expert's logit gets
  float all = 0.f;   // and that it shares with every expert
  if (!p.sigmoid && !p.renormalize) {
    float v[kPer];
#pragma unroll
    for (int i = 0; i < kPer; i += kV) {
      const int e = lane * kV + 32 * i;
      float run[kV];
      load_lane<T, kV>(row + e, p.E - e, kV > 1, kMasked, run);
#pragma unroll
      for (int j = 0; j < kV; ++j) v[i + j] = run[j];
    }
    float m = v[0];
#pragma unroll
    for (int i = 1; i < kPer; ++i) m = fmaxf(m, v[i]);
#pragma unroll
    for (int s = 16; s > 0; s >>= 1) m = fmaxf(m, __shfl_xor_sync(0xFFFFFFFFu, m, s));
    float sum = 0.f;
#pragma unroll
    for (int i = 0; i < kPer; ++i) {
      v[i] = v[i] == kMasked ? 0.f : expf(v[i] - m);
      sum += v[i];
    }
    sum = warp_sum(sum);
    const float w = logit != kMasked ? expf(logit - m) : 0.f;
    mine = logit != kMasked ? w / sum * g : 0.f;
    const float along = warp_sum(mine);
    const float factor = sum == 0.f ? 0.f : -along / sum;  // all masked: no gradient
    all = w * factor;
#pragma unroll
    for (int i = 0; i < kPer; ++i) v[i] *= factor;
#pragma unroll
    for (int i = 0; i < kPer; i += kV) {
      const int e = lane * kV + 32 * i;
      if (e < p.E) store_run<T, kV>(out + e, v + i);
    }
  } else {
    if (p.sigmoid) {
      const float s = id >= 0 ? sigmoid_of(logit) : 0.f;
      if (p.renormalize) {
        const float total = warp_sum(s) + 1e-20f;
        g = (g - warp_sum(g * s) / total) / total;
      }
      mine = g * s * (id >= 0 ? sigmoid_of(-logit) : 0.f);  // 1 - s without cancellation
    } else {
      float m = logit;
#pragma unroll
      for (int s = 16; s > 0; s >>= 1) m = fmaxf(m, __shfl_xor_sync(0xFFFFFFFFu, m, s));
      float w = logit != kMasked ? expf(logit - m) : 0.f;
      const float total = warp_sum(w);
      w = logit != kMasked ? w / total : 0.f;
      mine = w * (g - warp_sum(w * g));
    }
    const float zero[kV] = {};
#pragma unroll
    for (int i = 0; i < kPer; i += kV) {
      const int e = lane * kV + 32 * i;
      if (e < p.E) store_run<T, kV>(out + e, zero);
    }
  }
  // an expert named twice (ids of another origin; of the lanes that sign its place, one stays)
  // gets the sum, in the order of the slots, and each of its lanes writes it
  if (id >= 0) sign[warp][id] = lane;
  __syncwarp();
  if (__any_sync(0xFFFFFFFFu, id >= 0 && sign[warp][id] != lane)) {
    float sum = 0.f;
    for (int j = 0; j < p.top_k; ++j) {
      const int other = __shfl_sync(0xFFFFFFFFu, id, j);
      const float part = __shfl_sync(0xFFFFFFFFu, mine, j);
      if (other == id) sum += part;
    }
    mine = sum;
  }
  __syncwarp();  // after the stores above
  if (id >= 0) out[id] = from_float<T>(all + mine);
}

template <class T, int kPer>
cudaError_t launch_route(RouteParams p, Score score, void* stream) {
  const dim3 grid(static_cast<unsigned>((p.T + kWarps - 1) / kWarps)), block(kWarps * 32);
  constexpr int kBytes = piece_bytes<T, kPer>(), kBiasBytes = piece_bytes<float, kPer>();
  p.dealt = p.whole && p.groups > 1 && p.per_group != kPer << p.group_shift;
  const int64_t each = p.dealt ? p.per_group : p.E;
  p.wide = aligned_to(p.logits, kBytes) && p.ld * sizeof(T) % kBytes == 0 &&
           each * sizeof(T) % kBytes == 0;
  p.wide_bias = aligned_to(p.bias, kBiasBytes) && each * sizeof(float) % kBiasBytes == 0;
  const size_t smem = p.whole ? 0 : sizeof(uint32_t) * kWarps * padded(p.E);
  if (score == Score::kLogits)
    return launch_dependent(route_kernel<T, kPer, Score::kLogits>, grid, block, smem, stream, p);
  if (score == Score::kSoftmax)
    return launch_dependent(route_kernel<T, kPer, Score::kSoftmax>, grid, block, smem, stream, p);
  return launch_dependent(route_kernel<T, kPer, Score::kSigmoid>, grid, block, smem, stream, p);
}

// The experts per lane: as few as hold them, 160 and 384 (5 and 12) included.
template <class T>
cudaError_t launch_route(RouteParams p, Score score, void* stream) {
  p.group_shift = 5;
  p.whole = (p.groups & (p.groups - 1)) == 0;
  for (; p.groups > 32 >> p.group_shift; --p.group_shift) {
  }
  const int lanes = p.whole ? 1 << p.group_shift : 32, each = p.whole ? p.per_group : p.E;
  const int per = (each + lanes - 1) / lanes;
  if (per <= 1) return launch_route<T, 1>(p, score, stream);
  if (per <= 2) return launch_route<T, 2>(p, score, stream);
  if (per <= 4) return launch_route<T, 4>(p, score, stream);
  if (per <= 5) return launch_route<T, 5>(p, score, stream);
  if (per <= 8) return launch_route<T, 8>(p, score, stream);
  if (per <= 12) return launch_route<T, 12>(p, score, stream);
  if (per <= 16) return launch_route<T, 16>(p, score, stream);
  return launch_route<T, 32>(p, score, stream);
}

template <class T, int kPer>
cudaError_t launch_backward(const RouteBackwardParams& p, void* stream) {
  const dim3 grid(static_cast<unsigned>((p.T + kWarps - 1) / kWarps)), block(kWarps * 32);
  constexpr int kBytes = piece_bytes<T, kPer>(), kV = kBytes / static_cast<int>(sizeof(T));
  if constexpr (kV > 1)
    if (aligned_to(p.logits, kBytes) && aligned_to(p.dlogits, kBytes) && p.E % kV == 0 &&
        p.ld % kV == 0)
      return launch_dependent(route_backward_kernel<T, kPer, kV>, grid, block, 0, stream, p);
  return launch_dependent(route_backward_kernel<T, kPer, 1>, grid, block, 0, stream, p);
}

template <class T>
cudaError_t launch_backward(const RouteBackwardParams& p, void* stream) {
  if (p.E <= 32) return launch_backward<T, 1>(p, stream);
  if (p.E <= 64) return launch_backward<T, 2>(p, stream);
  if (p.E <= 128) return launch_backward<T, 4>(p, stream);
  if (p.E <= 160) return launch_backward<T, 5>(p, stream);
  if (p.E <= 256) return launch_backward<T, 8>(p, stream);
  if (p.E <= 384) return launch_backward<T, 12>(p, stream);
  if (p.E <= 512) return launch_backward<T, 16>(p, stream);
  return launch_backward<T, 32>(p, stream);
}

mslkb_status check_route(int64_t T, int64_t E, int64_t ld, int64_t top_k, int32_t score,
                         double scale, int32_t dtype) {
  if (T < 0 || E < 0 || T > MSLKB_MAX_DIM || E > MSLKB_MAX_EXPERTS) return MSLKB_ERR_SHAPE;
  if (top_k < 0 || top_k > E || top_k > MSLKB_MAX_TOPK) return MSLKB_ERR_SHAPE;
  if (ld < E || ld > MSLKB_MAX_DIM || T * top_k > MSLKB_MAX_DIM) return MSLKB_ERR_SHAPE;
  if (score != MSLKB_SOFTMAX && score != MSLKB_SIGMOID) return MSLKB_ERR_SHAPE;
  if (!(scale > -1e30 && scale < 1e30)) return MSLKB_ERR_SHAPE;
  return dtype_ok(dtype) ? MSLKB_OK : MSLKB_ERR_DTYPE;
}

}  // namespace
}  // namespace mslkb

extern "C" {

mslkb_status mslkb_route_experts(const void* logits, const float* bias, int32_t* ids,
                                 float* weights, int64_t T, int64_t E, int64_t ld, int64_t top_k,
                                 int32_t score, int64_t num_groups, int64_t topk_groups,
                                 int32_t group_top, int32_t renormalize, double scale,
                                 int32_t dtype, void* stream) {
  using namespace mslkb;
  mslkb_status s = check_route(T, E, ld, top_k, score, scale, dtype);
  if (s != MSLKB_OK) return s;
  if (num_groups < 1 || num_groups > 32 || E % num_groups != 0) return MSLKB_ERR_SHAPE;
  if (topk_groups < 1 || topk_groups > num_groups) return MSLKB_ERR_SHAPE;
  if (top_k > E / num_groups * topk_groups) return MSLKB_ERR_SHAPE;
  if (group_top != 1 && group_top != 2) return MSLKB_ERR_SHAPE;
  if (T == 0 || top_k == 0) return MSLKB_OK;
  if (logits == nullptr || ids == nullptr || weights == nullptr) return MSLKB_ERR_NULL;
  int sms = 0;
  if ((s = device_sms(&sms)) != MSLKB_OK) return s;
  const bool by_logits = score == MSLKB_SOFTMAX && bias == nullptr &&
                         (group_top == 1 || num_groups == 1);
  const Score by = score == MSLKB_SIGMOID ? Score::kSigmoid
                                          : (by_logits ? Score::kLogits : Score::kSoftmax);
  if (topk_groups == num_groups) num_groups = topk_groups = 1;  // all of them stay
  RouteParams p{};
  p.logits = logits, p.bias = bias, p.ids = ids, p.weights = weights;
  p.T = T, p.ld = ld, p.E = static_cast<int32_t>(E), p.top_k = static_cast<int32_t>(top_k);
  p.groups = static_cast<int32_t>(num_groups), p.top_groups = static_cast<int32_t>(topk_groups);
  p.group_top = group_top, p.per_group = static_cast<int32_t>(E / num_groups);
  p.renormalize = renormalize, p.scale = static_cast<float>(scale);
  TraceRange range("route_experts", T);
  cudaError_t e;
  if (dtype == MSLKB_BF16)
    e = launch_route<__nv_bfloat16>(p, by, stream);
  else if (dtype == MSLKB_FP16)
    e = launch_route<__half>(p, by, stream);
  else
    e = launch_route<float>(p, by, stream);
  return launch_status(e);
}

mslkb_status mslkb_route_experts_backward(const float* dweights, const void* logits,
                                          const int32_t* ids, void* dlogits, int64_t T, int64_t E,
                                          int64_t ld, int64_t top_k, int32_t score,
                                          int32_t renormalize, double scale, int32_t dtype,
                                          void* stream) {
  using namespace mslkb;
  mslkb_status s = check_route(T, E, ld, top_k, score, scale, dtype);
  if (s != MSLKB_OK) return s;
  if (T == 0 || E == 0) return MSLKB_OK;
  if (logits == nullptr || dlogits == nullptr ||
      (top_k > 0 && (dweights == nullptr || ids == nullptr)))
    return MSLKB_ERR_NULL;
  int sms = 0;
  if ((s = device_sms(&sms)) != MSLKB_OK) return s;
  const RouteBackwardParams p{dweights, logits, ids, dlogits, T, ld, static_cast<int32_t>(E),
                              static_cast<int32_t>(top_k), score == MSLKB_SIGMOID, renormalize,
                              static_cast<float>(scale)};
  TraceRange range("route_experts_backward", T);
  cudaError_t e;
  if (dtype == MSLKB_BF16)
    e = launch_backward<__nv_bfloat16>(p, stream);
  else if (dtype == MSLKB_FP16)
    e = launch_backward<__half>(p, stream);
  else
    e = launch_backward<float>(p, stream);
  return launch_status(e);
}

}  // extern "C"
