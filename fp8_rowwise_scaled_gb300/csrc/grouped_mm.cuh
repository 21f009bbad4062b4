// grouped_mm.cuh -- 16-bit products by expert on the tensor cores (bf16 or fp16 operands, fp32
// sums in tensor memory):
//
//   kRows   out[r, c]   = sum_k x[r, k] * w[g, c, k]              r in expert g's rows
//   kTurned out[r, c]   = sum_k x[r, k] * w[g, k, c]              the same weights the other way
//   kGrad   out[g, n, c] = (add[g, n, c]) + sum_r dy[r, n] * x[r, c]  over expert g's rows
//
// All three are D[c, r] = sum_k P[c, k] * Q[r, k] with the output's columns c on the MMA's M side
// (TMEM lanes) and its rows r on the N side (TMEM columns).  So the rows of an expert, ragged,
// cost the tensor core what they are, rounded up to 32, and not to a tile's 128 or 256; and a warp
// reads 32 neighbouring columns of one output row from TMEM, which it stores as one piece.  P is w
// or x, Q is x or dy; an operand whose contracted index is its rows (w turned, both operands of
// kGrad) is read as it lies in memory, "MN-major": the tensor core takes either.
//
// A pair of CTAs on two SMs (tiles of 256 x 256, each CTA holding half of either operand) is
// persistent and specialised by warp:
//   warp 0      loads by TMA (operands whose rows do not start on 16 bytes are copied to rows that
//               do, before: aligned_rows_kernel)
//   warp 1      issues the MMAs
//   warp 2      zeroes what a stage holds past the end of an expert's rows (kGrad)
//   warp 3      works out the tiles and hands them to the other warps
//   warp 4      loads what is added to a gradient (with three idle ones, only where there is some)
//   the last 8  the epilogue: four and four in turns, or all of them where they keep sums.
//
// Sums.  The tensor core's fp32 sums lose what lies below their last bit, always towards zero: up
// to 2^-23 of the sum for each step of 16 terms, some 1e-9 of it for every term (4096 terms of normal
// values were 4.4e-6 off).  So it sums kSumLen16 or kSumLen32 terms at the most,
// and these sums are added with rounding:
//   * kLong, contractions that are longer everywhere, or for most experts: in registers, which eight
//     warps have for a tile's 256 rows (and take from the others), while the tensor core goes on;
//   * else, where some experts have more rows than that: in tensor memory, the sum so far in one of
//     its buffers and the next sum in the other, for which the tensor core has to wait.
#pragma once

#include <cuda.h>
#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include <cstdint>
#include <type_traits>

#include "kernel.cuh"
#include "ptx.cuh"

namespace mslkb {

enum class Mm { kRows = 0, kTurned = 1, kGrad = 2 };

struct MmParams {
  const uint16_t* P;       // w, or x (kGrad)
  const uint16_t* Q;       // x, or dy (kGrad)
  const int64_t* m_sizes;  // [G]
  void* out;
  const void* add;         // kGrad: of out's type, or null
  uint32_t* status;        // device status word
  uint64_t timeout_ns;     // give-up time of one pipeline wait
  int64_t ldp, ldq;        // elements from row to row of P and of Q
  int32_t total;           // rows of x (and dy)
  int32_t G;
  int32_t C;               // output columns
  int32_t R;               // kGrad: rows of each expert's output
  int32_t K;               // contraction length (kGrad: each expert's rows instead)
  int32_t bf16;            // 1: bf16 operands, 0: fp16
  int32_t out32;           // 1: fp32 output, 0: the operands' type
  int32_t wide, ct;        // output columns of a tile per CTA: 128, or less for kRows; such tiles
  int32_t p_pieces, q_pieces;  // an MN-major operand's 64-element pieces in one box (see encode)
  int32_t splits;          // parts of each contraction, whose sums go to slices of out (fp32)
  int64_t slice;           // elements from slice to slice
  int32_t sums;            // 0: the contraction is empty everywhere, and P and Q are not read
  int32_t test_stall;      // test hook: the first pair withholds its first stage
};

// Tensor maps.  p, q: the operands, by boxes of a CTA's share of a stage; q64: by halves of
// it, for tiles of few rows; add: what is added (kGrad).
struct MmMaps {
  CUtensorMap p, q, q64, add;
};

// Terms that the tensor core sums at a time, for results in 16 bits and in fp32.  Each sum taken
// out of tensor memory costs the tensor core some 100 cycles of the 8192 that 1024 terms take
// (32 experts of 1024 rows, 4096 x 7168 bf16 on GB300: 1127 us with sums of 1024, 1160 of 512, 1106 in
// one; where normal values add up, results are 1e-6 off, 5e-7 and 7e-6 before they are rounded).
constexpr int kSumLen16 = 1024, kSumLen32 = 512;

template <Mm kMode_, int kAdd_ = 0, bool kLong_ = false>
struct MmCfg {
  static constexpr Mm kMode = kMode_;
  static constexpr bool kGrad = kMode == Mm::kGrad;
  static constexpr bool kPMn = kMode != Mm::kRows;  // the operand's rows are the contraction
  static constexpr bool kQMn = kGrad;
  static constexpr int kCtas = 2;
  static constexpr int kTileN = 256;               // output rows of a tile
  static constexpr int kBK = 64;                   // contraction per stage: 128-byte pieces
  static constexpr int kAdd = kAdd_;               // bytes of an element that is added; 0: none
  static constexpr int kStages = kAdd == 0 ? 6 : (kAdd == 4 ? 3 : 4);
  static constexpr int kQRows = kTileN / kCtas;    // of Q in one CTA
  static constexpr int kPBytes = 128 * kBK * 2;
  static constexpr int kQBytes = kQRows * kBK * 2;
  static constexpr int kStageBytes = kPBytes + kQBytes;
  static constexpr int kMmaWarp = 1;
  static constexpr int kEdgeWarp = 2;
  static constexpr int kTileWarp = 3;  // hands out the tiles
  // kGrad with something to add: that comes by TMA too, in slots of 8 KB, through a ring of its own
  // for each four of the epilogue's warps (32 experts of 75 rows, 4096 x 7168 on GB300: 1120 us
  // fp32, 710 bf16; loaded by the epilogue's threads themselves, a chunk ahead, 1541 and 1031).
  // Bound by what is on its way: fp32 with four stages and four slots each 1330, three and seven
  // 1120, two and nine 1180; bf16, whose tiles take half as long, four and four 706, three and
  // six 750.  (One warp loads for both rings, in the order of the tiles: one each 1122 and 737.)
  static constexpr bool kAddRing = kAdd > 0;
  static constexpr int kAddRows = kAdd == 4 ? 16 : 32;   // of 128, in a slot
  static constexpr int kAddSlot = 8192;
  static constexpr int kAddSlots = kAdd == 0 ? 0 : (kAdd == 4 ? 7 : 4);
  static constexpr bool kLong = kLong_;   // the tensor core's sums are added in registers
  static constexpr int kRegsFew = 56, kRegsMany = 224;   // of warps 0-3, of the epilogue's
  static constexpr int kAddWarp = 4;
  static constexpr int kAddBytes = kAddSlots * kAddSlot;
  static constexpr int kEpiWarp0 = kAddRing ? 8 : 4;
  static constexpr int kEpiWarps = 8;
  static constexpr int kThreads = 32 * (kEpiWarp0 + kEpiWarps);
  static constexpr int kRowStep = 16 * kCtas;      // a tile's rows are rounded up to these
  static constexpr int kTmemCols = 2 * kTileN;
  static constexpr int kChunk = 32;                // TMEM columns read at a time
  // rows of tiles that run next to each other: 8 x 9.5 tiles of 256 x 256 on 76 CTA pairs read
  // the fewest bytes between them
  static constexpr int kBand = 8;
  // bytes between the 64-element pieces of an MN-major operand
  static constexpr uint32_t kMnPiece = kBK * 128;

  static constexpr int kOffP = 0;
  static constexpr int kOffQ = kStages * kPBytes;
  static constexpr int kStagePart = 8192;  // the epilogue's rows: 32 x 128 in 16 bits
  static constexpr int kOffStage = kOffQ + kStages * kQBytes;
  static constexpr int kOffAdd = kOffStage + (kAdd == 4 ? 0 : 2 * kStagePart);
  static constexpr int kOffBar = kOffAdd + 2 * kAddBytes;
  // the scheduler warp hands tiles to the other roles through a ring
  static constexpr int kRing = 4;
  static constexpr int kRingUsers = 2 + (kGrad ? 1 : 0) + (kAddRing ? 1 : 0) + kEpiWarps;
  static constexpr int kNumBars = 4 * kStages + 6 + 2 * kRing + 4 * kAddSlots;
  static constexpr int kOffMisc = kOffBar + 8 * kNumBars;  // tmem address, abort flag
  static constexpr int kOffRing = (kOffMisc + 8 + 15) / 16 * 16;
  static constexpr int kOffSched = kOffRing + kRing * 32;
  static constexpr int kSmemBytes = kOffSched + 2 * 4 * (kMaxGroups + 1) + 1024;

  static_assert(kPBytes % 1024 == 0 && kQBytes % 1024 == 0, "swizzle atoms");
  static_assert(kSmemBytes <= 232448, "shared memory per CTA");
  static_assert(kSumLen16 % kBK == 0 && kSumLen32 % kBK == 0, "whole stages");
  static_assert(!kLong || (!kAddRing && kThreads == 384 &&
                           128 * kRegsFew + 256 * kRegsMany <= 384 * 168), "registers");
  static_assert(!kAddRing || kGrad, "what is added");
};

// A tile: its group (-1: past the last tile), first output column and row, rows (h: rounded up,
// valid: real), and the contraction [k0, k0 + len) (kGrad: rows of x and dy), or the part of it
// that is this tile's.
struct MmTile {
  int32_t g, c0, r0, h, valid, k0, len, part;
};

// Terms of each of the tensor core's sums in a contraction of `len`, at most `most`: whole stages, as
// many in each, so that no sum is over before the one before it has been taken (32 x 1024 rows, 4096 x
// 1088 on GB300: 177 us, 186 with 1024 terms and the rest).
template <class Cfg>
__device__ __forceinline__ int32_t mm_sum_len(int32_t len, int32_t most) {
  if (len <= most) return most;
  const uint32_t sums = static_cast<uint32_t>(len + most - 1) / static_cast<uint32_t>(most);
  const uint32_t stages = static_cast<uint32_t>(len + Cfg::kBK - 1) / Cfg::kBK;
  return static_cast<int32_t>((stages + sums - 1) / sums) * Cfg::kBK;
}

// Output columns of a tile, and of each CTA.
template <class Cfg>
__device__ __forceinline__ int32_t mm_wide(const MmParams& p) {
  return Cfg::kMode == Mm::kRows ? p.wide : 128;
}
template <class Cfg>
__device__ __forceinline__ int32_t mm_tile_c(const MmParams& p) {
  return Cfg::kCtas * mm_wide<Cfg>(p);
}

template <class Cfg>
__device__ __forceinline__ MmTile mm_tile(const MmParams& p, const int32_t* first,
                                          const int32_t* tile_pre, int32_t tiles, int32_t t) {
  const int32_t ct = p.ct;
  MmTile o;
  o.part = 0;
  if (p.splits > 1) {
    o.part = t / tiles;
    t -= o.part * tiles;
  }
  int32_t local, rows;
  if constexpr (Cfg::kGrad) {
    const int32_t per = ct * ((p.R + Cfg::kTileN - 1) / Cfg::kTileN);
    o.g = t / per;
    local = t - o.g * per;
    rows = p.R;
    o.k0 = first[o.g];
    o.len = first[o.g + 1] - o.k0;
  } else {
    int32_t lo = 0, hi = p.G;  // the largest g with tile_pre[g] <= t
    while (hi - lo > 1) {
      const int32_t mid = (lo + hi) >> 1;
      if (tile_pre[mid] <= t) lo = mid;
      else hi = mid;
    }
    o.g = lo;
    local = t - tile_pre[lo];
    rows = first[lo + 1] - first[lo];
    o.k0 = 0;
    o.len = p.K;
  }
  // row tiles in bands of kBand, column by column of tiles
  const int32_t rt = (rows + Cfg::kTileN - 1) / Cfg::kTileN;
  int32_t c = local, r = 0, each = rows;
  if (rt > 1) {
    const int32_t band = rt <= Cfg::kBand ? 0 : local / (Cfg::kBand * ct);
    const int32_t in = local - band * Cfg::kBand * ct;
    const int32_t deep = min(Cfg::kBand, rt - band * Cfg::kBand);
    c = deep == Cfg::kBand ? in / Cfg::kBand : in / deep;
    r = band * Cfg::kBand + (in - c * deep);
    // (row tiles of one height, rounded up; the last may have fewer rows, or none)
    each = (rows + rt - 1) / rt;
  }
  o.c0 = c * mm_tile_c<Cfg>(p);
  const int32_t height = (each + Cfg::kRowStep - 1) / Cfg::kRowStep * Cfg::kRowStep;
  o.valid = max(0, min(height, rows - r * height));
  o.h = (o.valid + Cfg::kRowStep - 1) / Cfg::kRowStep * Cfg::kRowStep;
  o.r0 = r * height + (Cfg::kGrad ? 0 : first[o.g]);
  if (p.splits > 1) {   // by whole stages
    const int64_t stages = (o.len + Cfg::kBK - 1) / Cfg::kBK;
    const int32_t a = static_cast<int32_t>(stages * o.part / p.splits) * Cfg::kBK;
    const int32_t b = static_cast<int32_t>(stages * (o.part + 1) / p.splits) * Cfg::kBK;
    o.k0 += a;
    o.len = min(o.len, b) - a;
  }
  return o;
}

// Rows a and b together, at most `most`: a, b <= most, whose sum 32 bits need not hold.
__device__ __forceinline__ int32_t mm_add_rows(int32_t a, int32_t b, int32_t most) {
  return a + min(b, most - a);
}

// v of the lanes up to this one, added up (at most `most`).
__device__ __forceinline__ int32_t mm_lanes_up_to(int32_t v, int32_t most, uint32_t lane) {
#pragma unroll
  for (int d = 1; d < 32; d <<= 1) {
    const int32_t o = __shfl_up_sync(0xffffffffu, v, d);
    if (lane >= static_cast<uint32_t>(d)) v = mm_add_rows(v, o, most);
  }
  return v;
}

// One warp: first[g] = rows before group g, clamped to [0, total] (G + 1 entries), and the tiles
// before it.  Returns all tiles.  Up to 32 groups, one to a lane, stay in registers: the first
// loads of a call wait for this (16 experts on GB300: 2050 cycles by the general way, 1200 so, of
// which the counts take 600 to come).
template <class Cfg>
__device__ __forceinline__ int32_t mm_schedule(const MmParams& p, int32_t* first,
                                               int32_t* tile_pre, uint32_t lane) {
  const int32_t G = p.G, total = p.total, ct = p.ct;
  bool clamped = false;
  auto count = [&](int32_t g) {
    const int64_t m = p.m_sizes[g];
    clamped |= m < 0 || m > total;
    return static_cast<int32_t>(m < 0 ? 0 : (m > total ? total : m));
  };
  auto tiles_of = [&](int32_t rows) { return (rows + Cfg::kTileN - 1) / Cfg::kTileN; };
  int32_t tiles = 0;   // (row tiles first: there are at most total / kTileN + G of them)
  if (G <= 32) {
    const int32_t g = static_cast<int32_t>(lane);
    const int32_t mc = g < G ? count(g) : 0;
    const int32_t end = mm_lanes_up_to(mc, total, lane);
    int32_t from = __shfl_up_sync(0xffffffffu, end, 1);
    if (lane == 0) from = 0;
    clamped |= mc > total - from;
    if (g < G) first[g + 1] = end;
    if (lane == 0) first[0] = 0;
    if constexpr (!Cfg::kGrad) {
      const int32_t up_to = mm_lanes_up_to(tiles_of(end - from), INT32_MAX, lane);
      if (g < G) tile_pre[g + 1] = up_to * ct;
      if (lane == 0) tile_pre[0] = 0;
      tiles = __shfl_sync(0xffffffffu, up_to, 31) * ct;
    }
  } else {
    const int32_t per = (G + 31) / 32;
    const int32_t g0 = min(G, static_cast<int32_t>(lane) * per), g1 = min(G, g0 + per);
    int32_t sum = 0;
    for (int32_t g = g0; g < g1; ++g) {
      const int32_t mc = count(g);
      first[g] = mc;
      clamped |= mc > total - sum;
      sum = mm_add_rows(sum, mc, total);
    }
    int32_t run = __shfl_up_sync(0xffffffffu, mm_lanes_up_to(sum, total, lane), 1);
    if (lane == 0) run = 0;
    clamped |= sum > total - run;
    for (int32_t g = g0; g < g1; ++g) {
      const int32_t mc = first[g];
      first[g] = run;
      run = mm_add_rows(run, mc, total);
    }
    if (lane == 31) first[G] = run;
    __syncwarp();
    if constexpr (!Cfg::kGrad) {
      int32_t mine = 0;
      for (int32_t g = g0; g < g1; ++g) mine += tiles_of(first[g + 1] - first[g]);
      const int32_t up_to = mm_lanes_up_to(mine, INT32_MAX, lane);
      int32_t at = up_to - mine;
      for (int32_t g = g0; g < g1; ++g) {
        tile_pre[g] = at * ct;
        at += tiles_of(first[g + 1] - first[g]);
      }
      if (lane == 31) tile_pre[G] = at * ct;
      tiles = __shfl_sync(0xffffffffu, up_to, 31) * ct;
    }
  }
  if constexpr (Cfg::kGrad) tiles = G * ct * tiles_of(p.R);
  if (__any_sync(0xffffffffu, clamped) && lane == 0 && blockIdx.x == 0)
    atomicOr(p.status, kStatusClamped);
  __syncwarp();
  return tiles;
}

// kind::f16 MMA, fp32 accumulator: D (+)= P * Q^T.  Instruction descriptor: bits 4-5 D format
// (1: fp32), 7-9 and 10-12 A and B format (0: fp16, 1: bf16), 15 and 16 A and B MN-major,
// 17-22 N >> 3, 24-28 M >> 4.
template <class Cfg>
__device__ __forceinline__ uint32_t mm_idesc(int32_t bf16, int32_t n) {
  const uint32_t f = static_cast<uint32_t>(bf16);
  return (1u << 4) | (f << 7) | (f << 10) | (static_cast<uint32_t>(Cfg::kPMn) << 15) |
         (static_cast<uint32_t>(Cfg::kQMn) << 16) | (static_cast<uint32_t>(n >> 3) << 17) |
         (static_cast<uint32_t>((128 * Cfg::kCtas) >> 4) << 24);
}

// Low word of an operand's descriptor (128-byte swizzle): its address and, for an MN-major
// operand, the bytes from one 64-element piece of M or N to the next (the high word, the 1024
// bytes between groups of eight rows, is that of every 128-byte swizzled operand).
template <bool kMn, uint32_t kPiece>
__device__ __forceinline__ uint32_t mm_desc_lo(uint32_t saddr) {
  return ((saddr & 0x3FFFFu) >> 4) | ((kMn ? (kPiece >> 4) : 1u) << 16);
}

__device__ __forceinline__ void mm_mma(uint32_t d, uint32_t p_lo, uint32_t q_lo, uint32_t idesc,
                                       uint32_t accumulate) {
  asm volatile(
      "{\n\t.reg .pred p;\n\t.reg .b64 ad, bd;\n\t"
      "mov.b64 ad, {%1, %5};\n\tmov.b64 bd, {%2, %5};\n\t"
      "setp.ne.b32 p, %4, 0;\n\t"
      "tcgen05.mma.cta_group::2.kind::f16 [%0], ad, bd, %3, p;\n\t}\n" ::"r"(d),
      "r"(p_lo), "r"(q_lo), "r"(idesc), "r"(accumulate), "n"(ptx::kSw128DescHi)
      : "memory");
}

__device__ __forceinline__ uint16_t mm_round16(float v, bool bf16) {
  return bf16 ? __bfloat16_as_ushort(__float2bfloat16_rn(v)) : __half_as_ushort(__float2half_rn(v));
}
__device__ __forceinline__ float mm_widen(uint16_t v, bool bf16) {
  return bf16 ? __bfloat162float(__ushort_as_bfloat16(v)) : __half2float(__ushort_as_half(v));
}

// f(row, pointer to it) for rows 0 .. kN - 1, C elements apart.  Four running pointers: computed
// ahead, addresses would take two registers each, and a single one makes every row wait for the
// 64-bit addition of the row before.
template <int kN, class T, class F>
__device__ __forceinline__ void mm_rows(T* p, int32_t C, F f) {
  T* r[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) r[i] = p + static_cast<int64_t>(i) * C;
  const int64_t step = 4 * static_cast<int64_t>(C);
#pragma unroll
  for (int j = 0; j < kN; j += 4) {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      f(j + i, r[i]);
      r[i] += step;
    }
  }
}

// The epilogue's chunk of a tile: a warp's 32 output columns (one per lane) of kN output rows, C
// elements apart, of which n are there.  load_add reads what is added to them, ahead of the
// sums; store adds it, rounds and stores.
template <class T, int kN>
struct MmChunk {
  T a[kN];
  __device__ __forceinline__ void load_add(const T* add, int32_t C, int32_t n, bool in) {
    if (!in) n = 0;
    mm_rows<kN>(add, C, [&](int j, const T* p) { a[j] = j < n ? *p : T(0); });
  }
  template <bool kAdd>
  __device__ __forceinline__ void store(T* out, int32_t C, int32_t n, bool in,
                                        const uint32_t (&v)[kN], bool bf16) {
    auto put = [&](int j, T* to) {
      float f = __uint_as_float(v[j]);
      if constexpr (sizeof(T) == 4) {
        if (kAdd) f = a[j] + f;
        *to = f;
      } else {
        if (kAdd) f = mm_widen(a[j], bf16) + f;
        *to = mm_round16(f, bf16);
      }
    };
    if (!in) return;
    if (n >= kN) mm_rows<kN>(out, C, put);
    else mm_rows<kN>(out, C, [&](int j, T* to) { if (j < n) put(j, to); });
  }
};

// 16-bit results in rows of whole, aligned fours: four warps put their 128 columns of some rows
// side by side in shared memory, and each then stores whole rows, 256 bytes at a time.  (A warp by
// itself has 64 bytes of a row, and a store of half a line takes as long as one of a line:
// weights' gradient of 256 rows, 32 x 4096 x 7168 bf16 on GB300 524 us so, 383 by whole rows.)
template <int kN>
struct MmRows {
  static __device__ __forceinline__ uint32_t pack(float lo, float hi, bool bf16) {
    if (bf16) {
      const __nv_bfloat162 h = __floats2bfloat162_rn(lo, hi);
      return *reinterpret_cast<const uint32_t*>(&h);
    }
    const __half2 h = __floats2half2_rn(lo, hi);
    return *reinterpret_cast<const uint32_t*>(&h);
  }
  // out: the chunk's first row and column; stage: shared memory of these four warps, `bar` their
  // barrier, `which` of them this is
  static __device__ __forceinline__ void store(uint16_t* out, int32_t C, int32_t n, int32_t cols,
                                               uint32_t which, const uint32_t (&v)[kN], bool bf16,
                                               uint32_t stage, uint32_t bar, uint32_t lane) {
    ptx::named_bar_sync(bar, 128);  // the rows before these have been read
#pragma unroll
    for (int j = 0; j < kN; j += 2)  // rows j and j + 1 in a word
      ptx::st_shared_u32(stage + (which * 32u + lane) * 4u + j * 256u,
                         pack(__uint_as_float(v[j]), __uint_as_float(v[j + 1]), bf16));
    ptx::named_bar_sync(bar, 128);
    out += static_cast<int64_t>(2 * which) * C + lane * 4u;
    const bool in = static_cast<int32_t>(lane) * 4 < cols;
#pragma unroll
    for (int i = 0; i < kN / 8; ++i, out += 8 * static_cast<int64_t>(C)) {
      const int32_t row = static_cast<int32_t>(2 * which) + 8 * i;
      const uint4 w = ptx::ld_shared_v4(stage + row * 256u + lane * 16u);
      if (in && row < n)
        *reinterpret_cast<uint2*>(out) =
            make_uint2(__byte_perm(w.x, w.y, 0x5410), __byte_perm(w.z, w.w, 0x5410));
      if (in && row + 1 < n)
        *reinterpret_cast<uint2*>(out + C) =
            make_uint2(__byte_perm(w.x, w.y, 0x7632), __byte_perm(w.z, w.w, 0x7632));
    }
  }
};

// Whether `ok` holds in all 128 threads at a barrier.
__device__ __forceinline__ bool named_bar_and(uint32_t id, bool ok) {
  uint32_t all;
  asm volatile(
      "{\n\t.reg .pred p, q;\n\tsetp.ne.u32 q, %1, 0;\n\t"
      "barrier.cta.red.and.pred p, %2, 128, q;\n\tselp.u32 %0, 1, 0, p;\n\t}"
      : "=r"(all)
      : "r"(static_cast<uint32_t>(ok)), "r"(id)
      : "memory");
  return all != 0;
}

template <class Cfg>
__global__ void __launch_bounds__(Cfg::kThreads, 1)
    grouped_mm_kernel(const __grid_constant__ MmParams p, const __grid_constant__ MmMaps maps) {
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>(
      (reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~static_cast<uintptr_t>(1023));
  const uint32_t s_p = ptx::smem_addr(smem + Cfg::kOffP);
  const uint32_t s_q = ptx::smem_addr(smem + Cfg::kOffQ);
  const uint32_t s_bar = ptx::smem_addr(smem + Cfg::kOffBar);
  auto full_bar = [&](int s) { return s_bar + 8u * s; };
  auto empty_bar = [&](int s) { return s_bar + 8u * (Cfg::kStages + s); };
  // sums in TMEM buffer b for the epilogue's four warps `part` (each four see all completions of
  // their own barriers, one after the other, however many sums the others take in between)
  auto tfull_bar = [&](uint32_t part, uint32_t b) {
    return s_bar + 8u * (2 * Cfg::kStages + 2 * part + b);
  };
  auto tempty_bar = [&](uint32_t b) { return s_bar + 8u * (2 * Cfg::kStages + 4 + b); };
  auto edge_bar = [&](int s) { return s_bar + 8u * (2 * Cfg::kStages + 6 + s); };
  auto peer_bar = [&](int s) { return s_bar + 8u * (3 * Cfg::kStages + 6 + s); };
  auto tile_bar = [&](int i) { return s_bar + 8u * (4 * Cfg::kStages + 6 + i); };
  auto taken_bar = [&](int i) { return s_bar + 8u * (4 * Cfg::kStages + 6 + Cfg::kRing + i); };
  // ring of what is added, of the epilogue's warps `part`: slot full, slot free
  auto add_bar = [&](uint32_t part, uint32_t slot) {
    return s_bar + 8u * (4 * Cfg::kStages + 6 + 2 * Cfg::kRing + part * 2 * Cfg::kAddSlots + slot);
  };
  auto addfree_bar = [&](uint32_t part, uint32_t slot) {
    return add_bar(part, slot) + 8u * Cfg::kAddSlots;
  };
  const uint32_t s_add = ptx::smem_addr(smem + Cfg::kOffAdd);
  uint32_t* tmem_holder = reinterpret_cast<uint32_t*>(smem + Cfg::kOffMisc);
  volatile uint32_t* abort_flag = reinterpret_cast<volatile uint32_t*>(smem + Cfg::kOffMisc + 4);
  int32_t* first = reinterpret_cast<int32_t*>(smem + Cfg::kOffSched);
  int32_t* tile_pre = first + (kMaxGroups + 1);

  const uint32_t warp = threadIdx.x >> 5, lane = threadIdx.x & 31u;
  const uint32_t crank = ptx::cluster_ctarank();
  const int32_t worker = static_cast<int32_t>(blockIdx.x) / Cfg::kCtas;
  const int32_t workers = static_cast<int32_t>(gridDim.x) / Cfg::kCtas;

  if (threadIdx.x == 0) {
    for (int s = 0; s < Cfg::kStages; ++s) {
      ptx::mbar_init(full_bar(s), 1u);
      ptx::mbar_init(empty_bar(s), 1u);
      ptx::mbar_init(edge_bar(s), 1u);
      ptx::mbar_init(peer_bar(s), 1u);
    }
    for (int b = 0; b < 2; ++b) {
      ptx::mbar_init(tfull_bar(0u, b), 1u);
      ptx::mbar_init(tfull_bar(1u, b), 1u);
      ptx::mbar_init(tempty_bar(b),
                     static_cast<uint32_t>((Cfg::kLong ? Cfg::kEpiWarps : 4) * Cfg::kCtas));
    }
    for (int i = 0; i < Cfg::kRing; ++i) {
      ptx::mbar_init(tile_bar(i), 1u);
      // (a pair's second CTA issues no MMAs)
      ptx::mbar_init(taken_bar(i), static_cast<uint32_t>(Cfg::kRingUsers) - (crank != 0 ? 1u : 0u));
    }
    if constexpr (Cfg::kAddRing)
      for (uint32_t i = 0; i < 2; ++i)
        for (uint32_t j = 0; j < Cfg::kAddSlots; ++j) {
          ptx::mbar_init(add_bar(i, j), 1u);
          ptx::mbar_init(addfree_bar(i, j), 4u);
        }
    *abort_flag = 0u;
    ptx::fence_mbar_init();
    ptx::fence_proxy_async_smem();
  }
  if (threadIdx.x == 0 && p.sums) {
    ptx::prefetch_tensormap(&maps.p);
    ptx::prefetch_tensormap(&maps.q);
    ptx::prefetch_tensormap(&maps.q64);
  }
  if (warp == Cfg::kMmaWarp) {
    ptx::tmem_alloc_pair(ptx::smem_addr(tmem_holder), Cfg::kTmemCols);
    ptx::tmem_relinquish_pair();
  }
  if (threadIdx.x == 0) ptx::griddep_launch_dependents();
  ptx::tc_fence_before_sync();
  ptx::cluster_sync();  // the peer's barriers are set up too
  ptx::tc_fence_after_sync();
  const uint32_t tmem_base = *tmem_holder;
  const int32_t wide = mm_wide<Cfg>(p);
  // (all that comes before passes while the kernel before this one ends)
  ptx::griddep_wait();

  // Tile i of this CTA (or pair), from the ring: by a whole warp, or by one lane of it.  False past
  // the last one, or if a wait gave up.
  int4* ring = reinterpret_cast<int4*>(smem + Cfg::kOffRing);
  auto take = [&](int32_t i, MmTile& c, bool whole_warp) -> bool {
    const int slot = i % Cfg::kRing;
    bool ok = wait_bar(tile_bar(slot), static_cast<uint32_t>(i / Cfg::kRing) & 1u, abort_flag,
                       p.status, p.timeout_ns);
    if (whole_warp) ok = __all_sync(0xffffffffu, ok) != 0;
    if (!ok) return false;
    const int4 a = ring[2 * slot], b = ring[2 * slot + 1];
    c = MmTile{a.x, a.y, a.z, a.w, b.x, b.y, b.z, b.w};
    if (whole_warp) __syncwarp();
    if (!whole_warp || lane == 0) ptx::mbar_arrive(taken_bar(slot));
    return c.g >= 0;
  };

  const int32_t sum_most = Cfg::kGrad && p.out32 ? kSumLen32 : kSumLen16;
  if (warp < static_cast<uint32_t>(Cfg::kEpiWarp0)) {
    if constexpr (Cfg::kLong) ptx::setmaxnreg_dec<Cfg::kRegsFew>();
    if (warp == 0) {
      // -------------------------------------------------------------- loads
      // (by the whole warp, with one lane issuing, as the MMAs below)
      const bool issuer = ptx::elect_one();
      int stage = 0;
      uint32_t phase = 0;
      bool ok = true;
      // (test hook: neither CTA arrives or loads, so that the wait for this stage runs out)
      bool withhold = p.test_stall != 0 && worker == 0;
      MmTile taken;
      for (int32_t i = 0; ok && take(i, taken, true); ++i) {
        // (the same in every lane, which the compiler is told)
        auto all = [](int32_t v) { return __shfl_sync(0xffffffffu, v, 0); };
        const MmTile c{all(taken.g), all(taken.c0), all(taken.r0), all(taken.h), 0, all(taken.k0),
                       all(taken.len), 0};
        if (c.len == 0) continue;
        const int32_t col = c.c0 + static_cast<int32_t>(crank) * wide;
        const int32_t mine = c.h / Cfg::kCtas;  // rows of Q in this CTA
        const int32_t row = c.r0 + static_cast<int32_t>(crank) * mine;
        // of Q 64 rows or 128 (of kGrad, columns) are loaded
        const bool half = mine <= 64;
        const uint32_t bytes =
            static_cast<uint32_t>((wide + (half ? 64 : 128)) * Cfg::kBK * 2);
        for (int32_t k = 0; k < c.len; k += Cfg::kBK) {
          ok = __all_sync(0xffffffffu, wait_bar(empty_bar(stage), phase ^ 1u, abort_flag,
                                                p.status, p.timeout_ns)) != 0;
          if (!ok) break;
          if (issuer && !withhold) {
            // the bytes of both CTAs (as many in each) complete on the leader's barrier.  A stage
            // that ends between two MMA steps (kGrad) passes through the edge warp of each CTA
            // first.
            uint32_t bar = ptx::mapa_shared(full_bar(stage), 0u);
            const bool edge = Cfg::kGrad && c.len - k < Cfg::kBK && (c.len & 15) != 0;
            if (edge) {
              bar = ptx::mapa_shared(edge_bar(stage), crank);
              ptx::mbar_arrive_expect_tx(edge_bar(stage), bytes);
            } else if (crank == 0) {
              ptx::mbar_arrive_expect_tx(full_bar(stage), bytes * Cfg::kCtas);
            }
            const int32_t x = c.k0 + k;
            const uint32_t dp = s_p + stage * Cfg::kPBytes, dq = s_q + stage * Cfg::kQBytes;
            auto load2 = [&](uint32_t dst, const CUtensorMap* m, int32_t a, int32_t b) {
              ptx::tma_load_2d_pair(dst, m, bar, a, b);
            };
            auto load3 = [&](uint32_t dst, const CUtensorMap* m, int32_t a, int32_t b, int32_t g) {
              ptx::tma_load_3d_pair(dst, m, bar, a, b, g);
            };
            // (few, large operations: an SM's loads are limited by their number as well)
            if constexpr (Cfg::kMode == Mm::kRows) {
              load3(dp, &maps.p, x, col, c.g);
            } else if constexpr (Cfg::kMode == Mm::kTurned) {
              if (p.p_pieces) {
                ptx::tma_load_4d_pair(dp, &maps.p, bar, 0, x, col / 64, c.g);
              } else {
                load3(dp, &maps.p, col, x, c.g);
                load3(dp + Cfg::kMnPiece, &maps.p, col + 64, x, c.g);
              }
            } else {
              if (p.p_pieces) {
                load3(dp, &maps.p, 0, x, col / 64);
              } else {
                load2(dp, &maps.p, col, x);
                load2(dp + Cfg::kMnPiece, &maps.p, col + 64, x);
              }
            }
            if constexpr (Cfg::kQMn) {
              if (p.q_pieces && !half && row % 64 == 0) {
                load3(dq, &maps.q, 0, x, row / 64);
              } else {
                load2(dq, &maps.q64, row, x);
                if (!half) load2(dq + Cfg::kMnPiece, &maps.q64, row + 64, x);
              }
            } else {
              load2(dq, half ? &maps.q64 : &maps.q, x, row);
            }
          }
          withhold = false;
          if (++stage == Cfg::kStages) {
            stage = 0;
            phase ^= 1u;
          }
        }
      }
      // wait until the MMAs have released every stage
      for (int i = 0; ok && i < Cfg::kStages; ++i) {
        ok = __all_sync(0xffffffffu, wait_bar(empty_bar(stage), phase ^ 1u, abort_flag, p.status,
                                              p.timeout_ns)) != 0;
        if (++stage == Cfg::kStages) {
          stage = 0;
          phase ^= 1u;
        }
      }
      __syncwarp();
    } else if (warp == Cfg::kMmaWarp) {
      // -------------------------------------------------------------- MMAs
      // The whole warp walks the loop, so that stages and descriptors stay in uniform registers,
      // and one lane issues (by that lane alone, in a branch of its own, a stage took 580 cycles
      // to issue; the tensor core takes 512 for it).
      if (crank == 0) {
        const bool issuer = ptx::elect_one();
        int stage = 0;
        // cur: the buffer of a tile's first sum; used: the parity of either one's uses, a bit each
        uint32_t phase = 0, cur = 0, used = 0, turn = 0;
        bool ok = true;
        const uint32_t p_lo0 = mm_desc_lo<Cfg::kPMn, Cfg::kMnPiece>(s_p);
        const uint32_t q_lo0 = mm_desc_lo<Cfg::kQMn, Cfg::kMnPiece>(s_q);
        MmTile c;
        for (int32_t i = 0; ok && take(i, c, true); ++i) {
          const int32_t len = __shfl_sync(0xffffffffu, c.len, 0);
          if (len == 0) continue;
          const uint32_t idesc = mm_idesc<Cfg>(p.bf16, __shfl_sync(0xffffffffu, c.h, 0));
          const int32_t sum_len = mm_sum_len<Cfg>(len, sum_most);
          for (int32_t k = 0; k < len;) {
            const uint32_t b = Cfg::kLong || k == 0 ? cur : cur ^ 1u;
            ok = __all_sync(0xffffffffu,
                            wait_bar<true>(tempty_bar(b), ((used >> b) & 1u) ^ 1u, abort_flag,
                                                 p.status, p.timeout_ns)) != 0;
            if (!ok) break;
            used ^= 1u << b;
            ptx::tc_fence_after_sync();
            const uint32_t d = tmem_base + b * Cfg::kTileN;
            const int32_t from = k, end = len - k > sum_len ? k + sum_len : len;
            for (; k < end; k += Cfg::kBK) {
              ok = __all_sync(0xffffffffu, wait_bar(full_bar(stage), phase, abort_flag, p.status,
                                                    p.timeout_ns)) != 0;
              if (!ok) break;
              ptx::tc_fence_after_sync();
              const uint32_t p_lo = p_lo0 + static_cast<uint32_t>(stage * (Cfg::kPBytes >> 4));
              const uint32_t q_lo = q_lo0 + static_cast<uint32_t>(stage * (Cfg::kQBytes >> 4));
              const int32_t steps = min(Cfg::kBK / 16, (len - k + 15) / 16);
              if (issuer) {
#pragma unroll
                for (int s = 0; s < Cfg::kBK / 16; ++s) {
                  constexpr uint32_t kMn16 = 16 * 128 / 16;
                  if (s < steps)
                    mm_mma(d, p_lo + s * (Cfg::kPMn ? kMn16 : 2u),
                           q_lo + s * (Cfg::kQMn ? kMn16 : 2u), idesc,
                           (k > from || s > 0) ? 1u : 0u);
                }
                ptx::mma_commit_pair(empty_bar(stage), 0x3);
              }
              if (++stage == Cfg::kStages) {
                stage = 0;
                phase ^= 1u;
              }
            }
            if (!ok) break;
            if (issuer) ptx::mma_commit_pair(tfull_bar(turn, b), 0x3);
            if (Cfg::kLong) cur ^= 1u;
          }
          if (!Cfg::kLong) turn ^= 1u, cur ^= 1u;
        }
      }
      __syncwarp();
    } else if (Cfg::kGrad && warp == Cfg::kEdgeWarp) {
      // -------------------------------------------------------------- ends of experts' rows
      // The last stage of an expert whose rows do not end with an MMA step of 16: its last step
      // holds rows of the next expert (or past the buffers).  They are zeroed in both operands (0 x
      // NaN is NaN): whole 128-byte lines here, since the rows are the operands' lines.
      int stage = 0;
      uint32_t parity = 0;  // of each stage's edge barrier, one bit
      MmTile c;
      for (int32_t i = 0; take(i, c, true); ++i) {
        if (c.len == 0) continue;
        const int32_t kbs = (c.len + Cfg::kBK - 1) / Cfg::kBK;
        const int last = (stage + kbs - 1) % Cfg::kStages;
        stage = (stage + kbs) % Cfg::kStages;
        if ((c.len & 15) == 0) continue;
        const bool ok = wait_bar(edge_bar(last), (parity >> last) & 1u, abort_flag, p.status,
                                 p.timeout_ns);
        if (!__all_sync(0xffffffffu, ok)) break;
        parity ^= 1u << last;
        const int32_t in = c.len - (kbs - 1) * Cfg::kBK;  // rows of the stage that are the expert's
        const int32_t lines = ((in + 15) & ~15) - in;
        const int32_t boxes = c.h / Cfg::kCtas <= 64 ? 1 : 2;
        for (int32_t i = static_cast<int32_t>(lane); i < (2 + boxes) * lines * 8; i += 32) {
          const int32_t line = in + (i >> 3) % lines, piece = (i >> 3) / lines;
          const uint32_t base = piece < 2 ? s_p + last * Cfg::kPBytes + piece * Cfg::kMnPiece
                                          : s_q + last * Cfg::kQBytes + (piece - 2) * Cfg::kMnPiece;
          ptx::st_shared_v4(base + static_cast<uint32_t>(line) * 128u + (i & 7) * 16u, 0u, 0u, 0u,
                            0u);
        }
        ptx::fence_proxy_async_smem();
        __syncwarp();
        // the leader's edge warp hands the stage on when the peer's has done its part
        if (crank != 0) {
          if (lane == 0) ptx::mbar_arrive_cluster(ptx::mapa_shared(peer_bar(last), 0u));
        } else {
          const bool there = wait_bar<true>(peer_bar(last), ((parity >> last) & 1u) ^ 1u,
                                            abort_flag, p.status, p.timeout_ns);
          if (!__all_sync(0xffffffffu, there)) break;
          if (lane == 0) ptx::mbar_arrive(full_bar(last));
        }
      }
    } else if (Cfg::kAddRing && warp == Cfg::kAddWarp) {
      // -------------------------------------------------------------- what is added
      if (lane == 0) {
        uint32_t turn = 0, next[2] = {0, 0}, phase[2] = {0, 0};   // of either ring
        bool ok = true;
        MmTile c;
        for (int32_t i = 0; ok && take(i, c, false); ++i) {
          // (the same turns as the epilogue's)
          const uint32_t part = (c.len > 0 ? turn++ : static_cast<uint32_t>(i)) & 1u;
          uint32_t slot = part == 0 ? next[0] : next[1], parity = part == 0 ? phase[0] : phase[1];
          for (int32_t j0 = 0; j0 < c.valid; j0 += Cfg::kAddRows) {
            ok = wait_bar(addfree_bar(part, slot), parity ^ 1u, abort_flag, p.status,
                          p.timeout_ns);
            if (!ok) break;
            ptx::mbar_arrive_expect_tx(add_bar(part, slot), Cfg::kAddSlot);
            ptx::tma_load_3d(s_add + part * Cfg::kAddBytes + slot * Cfg::kAddSlot, &maps.add,
                             add_bar(part, slot), c.c0 + static_cast<int32_t>(crank) * wide,
                             c.r0 + j0, c.g);
            if (++slot == Cfg::kAddSlots) slot = 0, parity ^= 1u;
          }
          if (part == 0) next[0] = slot, phase[0] = parity;
          else next[1] = slot, phase[1] = parity;
        }
      }
      __syncwarp();
    } else if (warp == static_cast<uint32_t>(Cfg::kTileWarp)) {
      // -------------------------------------------------------------- tiles
      // Round n goes over the workers from the n-th on, so that a worker does not get the same row
      // tile of every column: those of fewer rows take less time, and workers that get ahead of
      // others read the weights from memory instead of sharing them in L2 (32 experts of 480 rows,
      // 4096 x 7168 on GB300: 630 us without the turn, 558 with it).  32 tiles are worked out at a
      // time, one by each lane (a search and up to four divisions), and handed on one by one.
      const int32_t part = mm_schedule<Cfg>(p, first, tile_pre, lane);   // of a split product
      const int32_t tiles = part * p.splits;
      int32_t i = 0, turn = static_cast<int32_t>(static_cast<uint32_t>(worker + lane) %
                                                 static_cast<uint32_t>(workers));
      bool ok = true;
      for (int64_t n0 = 0; ok; n0 += 32) {
        const int64_t t = (n0 + lane) * workers + (Cfg::kGrad ? worker : turn);
        turn = static_cast<int32_t>(static_cast<uint32_t>(turn + 32) %
                                    static_cast<uint32_t>(workers));
        MmTile c{-1, 0, 0, 0, 0, 0, 0, 0};
        if (t < tiles) c = mm_tile<Cfg>(p, first, tile_pre, part, static_cast<int32_t>(t));
        const uint32_t past = __ballot_sync(0xffffffffu, c.g < 0);   // (the first of these says so)
        const bool more = past == 0u;
        uint32_t left = more ? 0xffffffffu : (2u << (__ffs(past) - 1)) - 1u;
        left &= __ballot_sync(0xffffffffu, c.g < 0 || c.h > 0);
        while (left != 0) {
          const int src = __ffs(left) - 1;
          left &= left - 1;
          const int slot = i % Cfg::kRing;
          const uint32_t par = (static_cast<uint32_t>(i / Cfg::kRing) & 1u) ^ 1u;
          ok = __all_sync(0xffffffffu, wait_bar(taken_bar(slot), par, abort_flag, p.status,
                                                p.timeout_ns)) != 0;
          if (!ok) break;
          if (static_cast<int>(lane) == src) {
            ring[2 * slot] = make_int4(c.g, c.c0, c.r0, c.h);
            ring[2 * slot + 1] = make_int4(c.valid, c.k0, c.len, c.part);
            ptx::mbar_arrive(tile_bar(slot));
          }
          __syncwarp();
          ++i;
        }
        if (!more) break;
      }
    }
  } else if constexpr (Cfg::kLong) {
    // -------------------------------------------------------------- epilogue, long contractions
    // Eight warps for a tile: one for each quarter of the TMEM lanes and half of the output rows,
    // whose sums they keep.
    ptx::setmaxnreg_inc<Cfg::kRegsMany>();
    constexpr int kHalf = Cfg::kTileN / 2;
    const uint32_t q = warp & 3u, part = (warp - Cfg::kEpiWarp0) >> 2;
    const uint32_t stage = ptx::smem_addr(smem + Cfg::kOffStage) + part * Cfg::kStagePart;
    const uint32_t bar = 1u + part;  // of this half's four warps
    // kWhole: 16-bit results by whole rows
    auto work = [&](auto* out0, auto whole) {
      using T = std::remove_pointer_t<decltype(out0)>;
      constexpr bool kWhole = decltype(whole)::value;
      const bool bf16 = p.bf16 != 0;
      uint32_t used = 0;
      MmTile c;
      for (int32_t i = 0;; ++i) {
        bool ok = take(i, c, true);
        const int32_t n = min(kHalf, c.valid - static_cast<int32_t>(part) * kHalf);
        const int32_t col0 = c.c0 + static_cast<int32_t>(crank) * wide;
        const int32_t cols = min(wide, p.C - col0);   // of this CTA
        const int32_t col = col0 + static_cast<int32_t>(q * 32u + lane);
        const bool in = col < col0 + cols;
        const int64_t row0 = Cfg::kGrad ? static_cast<int64_t>(c.g) * p.R + c.r0 : c.r0;
        const int64_t at = (row0 + part * kHalf) * p.C + c.part * p.slice;
        float sum[kHalf];
#pragma unroll
        for (int j = 0; j < kHalf; ++j) sum[j] = 0.f;
        if constexpr (Cfg::kGrad && sizeof(T) == 4) {
          // what is added comes first: its loads pass while the first rows are summed
          const int32_t there = in ? n : 0;
          if (ok && p.add != nullptr)
            mm_rows<kHalf>(static_cast<const T*>(p.add) + at + col, p.C,
                           [&](int j, const T* a) { sum[j] = j < there ? *a : 0.f; });
        }
        const int32_t sum_len = mm_sum_len<Cfg>(c.len, sum_most);
        for (int32_t k = 0; ok && k < c.len; k += sum_len) {
          const uint32_t b = used & 1u;
          ok = wait_bar(tfull_bar(0u, b), (used >> 1) & 1u, abort_flag, p.status, p.timeout_ns);
          ok = __all_sync(0xffffffffu, ok) != 0;
          if (!ok) break;
          ++used;
          ptx::tc_fence_after_sync();
          // 64 rows on their way at a time
          const uint32_t from = tmem_base + b * Cfg::kTileN + part * kHalf + ((q * 32u) << 16);
#pragma unroll
          for (int j0 = 0; j0 < kHalf; j0 += 64) {
            if (j0 < n) {
              uint32_t v[32], w[32];
              ptx::tmem_ld_x32(from + j0, v);
              ptx::tmem_ld_x32(from + j0 + 32, w);
              ptx::tmem_ld_wait();
#pragma unroll
              for (int j = 0; j < 32; ++j) {
                sum[j0 + j] += __uint_as_float(v[j]);
                sum[j0 + 32 + j] += __uint_as_float(w[j]);
              }
            }
          }
          ptx::tc_fence_before_sync();
          __syncwarp();
          if (lane == 0) {
            if (crank != 0)
              ptx::mbar_arrive_cluster(ptx::mapa_shared(tempty_bar(b), 0u));
            else
              ptx::mbar_arrive(tempty_bar(b));
          }
        }
        if constexpr (kWhole) ok = named_bar_and(bar, ok);  // (they meet at it: leave together)
        if (!ok) break;
        if constexpr (kWhole) {
#pragma unroll
          for (int j0 = 0; j0 < kHalf; j0 += 32) {
            if (j0 < n) {
              uint32_t v[32];
#pragma unroll
              for (int j = 0; j < 32; ++j) v[j] = __float_as_uint(sum[j0 + j]);
              MmRows<32>::store(out0 + at + static_cast<int64_t>(j0) * p.C + col0, p.C, n - j0, cols,
                                q, v, bf16, stage, bar, lane);
            }
          }
        } else {
          auto put = [&](int j, T* to) {
            if constexpr (sizeof(T) == 4) *to = sum[j];
            else *to = mm_round16(sum[j], bf16);
          };
          if (in && n >= kHalf)
            mm_rows<kHalf>(out0 + at + col, p.C, put);
          else if (in)
            mm_rows<kHalf>(out0 + at + col, p.C, [&](int j, T* to) { if (j < n) put(j, to); });
        }
      }
    };
    uint16_t* out16 = static_cast<uint16_t*>(p.out);
    if (p.out32) work(static_cast<float*>(p.out), std::false_type());
    else if (p.C % 4 == 0 && (reinterpret_cast<uintptr_t>(p.out) & 7) == 0)
      work(out16, std::true_type());
    else work(out16, std::false_type());
  } else {
    // -------------------------------------------------------------- epilogue
    // Four warps for a tile, one for each quarter of the TMEM lanes.  Eight warps take turns: while
    // four store a tile the others wait for the sums of the next (weights' gradient of 256 rows, 32
    // x 4096 x 7168 bf16 on GB300: 417 us; all eight at one tile 599).
    const uint32_t q = warp & 3u, part = (warp - Cfg::kEpiWarp0) >> 2;
    const uint32_t stage = ptx::smem_addr(smem + Cfg::kOffStage) + part * Cfg::kStagePart;
    const uint32_t bar = 1u + part;  // of this part's four warps
    uint32_t slot = 0, parity = 0;   // of the ring
    // kWhole: 16-bit results by whole rows; kLoad: what is added is loaded here
    auto work = [&](auto* out0, auto whole, auto load) {
      using T = std::remove_pointer_t<decltype(out0)>;
      constexpr bool kWhole = decltype(whole)::value, kLoad = decltype(load)::value;
      constexpr int kN = Cfg::kChunk;
      MmChunk<T, kN> chunk;
      const T* add0 = static_cast<const T*>(p.add);
      const bool bf16 = p.bf16 != 0;
      uint32_t cur = 0, turn = 0;
      uint32_t seen = 0;   // parity of the completions seen, a bit for each buffer
      MmTile c;
      for (int32_t i = 0;; ++i) {
        bool ok = take(i, c, true);
        const int32_t col0 = c.c0 + static_cast<int32_t>(crank) * wide;
        const int32_t cols = min(wide, p.C - col0);   // of this CTA
        const int32_t col = col0 + static_cast<int32_t>(q * 32u + lane);
        const bool in = col < col0 + cols;
        const int64_t row0 = Cfg::kGrad ? static_cast<int64_t>(c.g) * p.R + c.r0 : c.r0;
        const int64_t at0 = row0 * p.C + c.part * p.slice;
        const bool any = ok && c.len > 0;  // else the empty sum
        const bool mine = ((any ? turn : static_cast<uint32_t>(i)) & 1u) == part;
        if constexpr (kLoad) {
          if (ok && mine) chunk.load_add(add0 + at0 + col, p.C, c.valid, in);
        }
        auto rows_of = [&](uint32_t buffer, int32_t j0) {
          return tmem_base + buffer * Cfg::kTileN + static_cast<uint32_t>(j0) + ((q * 32u) << 16);
        };
        auto release = [&](uint32_t buffer) {
          ptx::tc_fence_before_sync();
          __syncwarp();
          if (lane != 0) return;
          if (crank != 0)
            ptx::mbar_arrive_cluster(ptx::mapa_shared(tempty_bar(buffer), 0u));
          else
            ptx::mbar_arrive(tempty_bar(buffer));
        };
        // the tensor core's sums: the first stays where it is, others are added to it
        const int32_t sum_len = mm_sum_len<Cfg>(c.len, sum_most);
        for (int32_t k = 0; ok && any && mine && k < c.len; k += sum_len) {
          const uint32_t b = k == 0 ? cur : cur ^ 1u;
          ok = wait_bar(tfull_bar(part, b), (seen >> b) & 1u, abort_flag, p.status, p.timeout_ns);
          ok = __all_sync(0xffffffffu, ok) != 0;
          seen ^= 1u << b;
          ptx::tc_fence_after_sync();
          if (!ok || k == 0) continue;
#pragma unroll 1
          for (int32_t j0 = 0; j0 < c.valid; j0 += 16) {
            uint32_t sum[16], v[16];
            ptx::tmem_ld_x16(rows_of(cur, j0), sum);
            ptx::tmem_ld_x16(rows_of(b, j0), v);
            ptx::tmem_ld_wait();
#pragma unroll
            for (int j = 0; j < 16; ++j)
              v[j] = __float_as_uint(__uint_as_float(sum[j]) + __uint_as_float(v[j]));
            ptx::tmem_st_x16(rows_of(cur, j0), v);
          }
          ptx::tmem_st_wait();
          release(b);
        }
        if constexpr (kWhole) ok = named_bar_and(bar, ok);  // (they meet at it: leave together)
        if (!ok) break;
        const uint32_t done = cur;
        if (any) ++turn, cur ^= 1u;
        if (!mine) continue;
        int64_t at = at0;
        for (int32_t j0 = 0; j0 < c.valid; j0 += kN, at += static_cast<int64_t>(kN) * p.C) {
          uint32_t v[kN];
          if (any) {
            ptx::tmem_ld_x32(rows_of(done, j0), v);
            ptx::tmem_ld_wait();
          } else {
#pragma unroll
            for (int j = 0; j < kN; ++j) v[j] = 0u;
          }
          const int32_t n = c.valid - j0;
          if constexpr (Cfg::kAddRing) {
#pragma unroll
            for (int h = 0; h < kN; h += Cfg::kAddRows) {
              if (h > 0 && n <= h) break;
              bool got = wait_bar(add_bar(part, slot), parity, abort_flag, p.status, p.timeout_ns);
              got = __all_sync(0xffffffffu, got) != 0;
              if constexpr (kWhole) got = named_bar_and(bar, got);
              if (!got) return;
              const uint32_t from = s_add + part * Cfg::kAddBytes + slot * Cfg::kAddSlot +
                                    (q * 32u + lane) * Cfg::kAdd;
#pragma unroll
              for (int j = 0; j < Cfg::kAddRows; ++j) {
                float a;
                if constexpr (sizeof(T) == 4)
                  a = __uint_as_float(ptx::ld_shared_u32(from + j * 512u));
                else
                  a = mm_widen(ptx::ld_shared_u16(from + j * 256u), bf16);
                v[h + j] = __float_as_uint(a + __uint_as_float(v[h + j]));
              }
              __syncwarp();
              if (lane == 0) ptx::mbar_arrive(addfree_bar(part, slot));
              if (++slot == Cfg::kAddSlots) slot = 0, parity ^= 1u;
            }
          }
          if constexpr (kWhole) {
            MmRows<kN>::store(out0 + at + col0, p.C, n, cols, q, v, bf16, stage, bar, lane);
          } else {
            auto now = chunk;  // what is added to these rows; the next ones' is loaded meanwhile
            if constexpr (kLoad) {
              if (n > kN)
                chunk.load_add(add0 + at + col + static_cast<int64_t>(kN) * p.C, p.C, n - kN, in);
            }
            now.template store<kLoad>(out0 + at + col, p.C, n, in, v, bf16);
          }
        }
        if (any) release(done);
      }
    };
    const std::true_type yes{};
    const std::false_type no{};
    uint16_t* out16 = static_cast<uint16_t*>(p.out);
    const bool rows = p.C % 4 == 0 && (reinterpret_cast<uintptr_t>(p.out) & 7) == 0;
    if constexpr (Cfg::kGrad) {
      float* out32 = static_cast<float*>(p.out);
      // what is added, where it does not come through the ring
      const bool load = !Cfg::kAddRing && p.add != nullptr;
      if constexpr (!Cfg::kAddRing) {
        if (load && p.out32) work(out32, no, yes);
        else if (load) work(out16, no, yes);
      }
      if constexpr (Cfg::kAdd != 2)
        if (!load && p.out32) work(out32, no, no);
      if constexpr (Cfg::kAdd != 4) {
        if (!load && !p.out32 && rows) work(out16, yes, no);
        else if (!load && !p.out32) work(out16, no, no);
      }
    } else {
      if (p.out32) work(static_cast<float*>(p.out), no, no);
      else if (rows) work(out16, yes, no);
      else work(out16, no, no);
    }
  }

  // ---------------------------------------------------------------- teardown
  ptx::tc_fence_before_sync();
  // neither CTA leaves while the other may signal its barriers, and both wait out what is in flight
  // if either gave up
  if (lane == 0 && *abort_flag != 0u)
    ptx::st_shared_cluster_u32(
        ptx::mapa_shared(ptx::smem_addr(smem + Cfg::kOffMisc + 4), crank ^ 1u), 1u);
  ptx::cluster_sync();
  if (*abort_flag != 0u) {
    const uint64_t t0 = ptx::globaltimer_ns();
    while (ptx::globaltimer_ns() - t0 < 2000000ull) ptx::nanosleep(1000);
  }
  if (warp == Cfg::kMmaWarp) {
    ptx::tc_fence_after_sync();
    ptx::tmem_dealloc_pair(tmem_base, Cfg::kTmemCols);
  }
}

// Rows of 16-bit elements at any even address, copied to rows that start on 16 bytes: up to two
// matrices, of which one may be the experts' (those without rows are left out).  A warp takes 512
// elements of a row: words at aligned addresses, lane after lane, put together across lanes where
// the row starts inside a word; nothing outside the row is read.  Bound by memory.  (8 experts x
// 1001 x 1002, 8000 rows on GB300: 31 us for copy and product; loading such rows straight into the
// product's stages, through registers, 95.)
struct AlignedCopy {
  const uint16_t* from;
  uint16_t* to;
  int64_t ld_from, ld_to;   // ld_to: a multiple of 8
  int64_t rows;
  int32_t cols;
  int32_t per_expert;       // rows of an expert's matrix; 0: not the experts'
};

constexpr int kCopyThreads = 256;
constexpr int kCopyCols = 512;

__device__ __forceinline__ uint32_t ldg32_if(const uint16_t* p, bool on) {
  uint32_t v;
  asm volatile(
      "{\n\t.reg .pred p;\n\tsetp.ne.u32 p, %2, 0;\n\tmov.u32 %0, 0;\n\t"
      "@p ld.global.nc.u32 %0, [%1];\n\t}"
      : "=r"(v)
      : "l"(p), "r"(static_cast<uint32_t>(on)));
  return v;
}
__device__ __forceinline__ uint32_t ldg16_if(const uint16_t* p, bool on) {
  uint32_t v;
  asm volatile(
      "{\n\t.reg .pred p;\n\t.reg .b16 h;\n\tsetp.ne.u32 p, %2, 0;\n\tmov.u16 h, 0;\n\t"
      "@p ld.global.nc.u16 h, [%1];\n\tcvt.u32.u16 %0, h;\n\t}"
      : "=r"(v)
      : "l"(p), "r"(static_cast<uint32_t>(on)));
  return v;
}

__global__ void __launch_bounds__(kCopyThreads)
    aligned_rows_kernel(const AlignedCopy a, const AlignedCopy b, const int64_t* m_sizes) {
  constexpr int kWords = kCopyCols / 64;   // of a lane
  if (threadIdx.x == 0) ptx::griddep_launch_dependents();
  ptx::griddep_wait();
  const int32_t lane = static_cast<int32_t>(threadIdx.x & 31u);
  const int64_t warps = static_cast<int64_t>(gridDim.x) * (kCopyThreads / 32);
  const int64_t pieces_a = (a.cols + kCopyCols - 1) / kCopyCols;
  const int64_t pieces_b = (b.cols + kCopyCols - 1) / kCopyCols;
  const int64_t units_a = a.rows * pieces_a, units = units_a + b.rows * pieces_b;
  for (int64_t t = static_cast<int64_t>(blockIdx.x) * (kCopyThreads / 32) + (threadIdx.x >> 5);
       t < units; t += warps) {
    const bool second = t >= units_a;
    const AlignedCopy& c = second ? b : a;
    const int64_t u = second ? t - units_a : t, pieces = second ? pieces_b : pieces_a;
    const int64_t row = u / pieces;
    const int32_t col = static_cast<int32_t>(u - row * pieces) * kCopyCols;
    if (c.per_expert != 0 && m_sizes[row / c.per_expert] <= 0) continue;
    const uint16_t* from = c.from + row * c.ld_from + col;
    const int32_t left = c.cols - col;
    // word w of the piece: elements 2 w - s and 2 w + 1 - s
    const int32_t s = static_cast<int32_t>(reinterpret_cast<uintptr_t>(from) >> 1) & 1;
    uint32_t v[kWords + 1];
#pragma unroll
    for (int i = 0; i < kWords; ++i) {
      const int32_t e = 2 * (lane + 32 * i) - s;
      v[i] = ldg32_if(from + e, e >= 0 && e + 1 < left);
    }
    // elements alone in their words, at the row's ends
    const uint32_t first = ldg16_if(from, s != 0 && lane == 0);
    const uint32_t past = ldg16_if(from + kCopyCols - 1, s != 0 && left >= kCopyCols);
    const int32_t tail = left - 1;
    const uint32_t last = ldg16_if(from + tail, left < kCopyCols && ((tail + s) & 1) == 0);
    if (s != 0 && lane == 0) v[0] = first << 16;
    v[kWords] = past;
    if (left < kCopyCols && ((tail + s) & 1) == 0) {
#pragma unroll
      for (int i = 0; i < kWords; ++i)
        if (2 * (lane + 32 * i) - s == tail) v[i] = last;
    }
    uint32_t* to = reinterpret_cast<uint32_t*>(c.to + row * c.ld_to + col) + lane;
#pragma unroll
    for (int i = 0; i < kWords; ++i) {
      uint32_t w = v[i];
      if (s != 0) {
        const uint32_t next =
            __shfl_sync(0xffffffffu, lane == 0 ? v[i + 1] : v[i], (lane + 1) & 31);
        w = (w >> 16) | (next << 16);
      }
      if (2 * (lane + 32 * i) < left) to[32 * i] = w;
    }
  }
}

// The sum of a split contraction's slices (and of what is added to a gradient), rounded.
struct SliceSum {
  const float* slices;
  void* out;
  const void* add;          // of out's type, or null
  const int64_t* m_sizes;   // not null: only the experts' rows count, of `total`
  int64_t slice, n;         // elements from slice to slice; of out
  int32_t splits, G, total, C, bf16, out32;
};

constexpr int kSumThreads = 256;

template <class T>
__device__ __forceinline__ float sum_get(T v, bool bf16) {
  if constexpr (sizeof(T) == 4) return v;
  else return mm_widen(v, bf16);
}
template <class T>
__device__ __forceinline__ T sum_put(float v, bool bf16) {
  if constexpr (sizeof(T) == 4) return v;
  else return mm_round16(v, bf16);
}

template <class T>
__device__ __forceinline__ void sum_slices(const SliceSum& p, int64_t n) {
  T* out = static_cast<T*>(p.out);
  const T* add = static_cast<const T*>(p.add);
  const bool bf16 = p.bf16 != 0;
  // four elements a thread, their slices' loads under way together
  for (int64_t i = 4 * (static_cast<int64_t>(blockIdx.x) * kSumThreads + threadIdx.x); i < n;
       i += 4ll * kSumThreads * gridDim.x) {
    float s[4] = {0.f, 0.f, 0.f, 0.f};
    const int m = static_cast<int>(min(static_cast<int64_t>(4), n - i));
    if (add != nullptr) {
      for (int j = 0; j < 4; ++j)
        if (j < m) s[j] = sum_get(add[i + j], bf16);
    }
#pragma unroll 4
    for (int k = 0; k < p.splits; ++k) {   // (a slice's length is a multiple of four)
      const float4 v = *reinterpret_cast<const float4*>(p.slices + k * p.slice + i);
      s[0] += v.x, s[1] += v.y, s[2] += v.z, s[3] += v.w;
    }
    for (int j = 0; j < 4; ++j)
      if (j < m) out[i + j] = sum_put<T>(s[j], bf16);
  }
}

__global__ void __launch_bounds__(kSumThreads)
    slice_sum_kernel(const __grid_constant__ SliceSum p) {
  if (threadIdx.x == 0) ptx::griddep_launch_dependents();
  ptx::griddep_wait();
  int64_t n = p.n;
  if (p.m_sizes != nullptr) {
    // rows that are experts': counts clamped as the product's
    __shared__ int32_t warps[kSumThreads / 32];
    int32_t rows = 0;
    for (int g = static_cast<int>(threadIdx.x); g < p.G; g += kSumThreads) {
      const int64_t m = p.m_sizes[g];
      rows = mm_add_rows(rows, static_cast<int32_t>(m < 0 ? 0 : (m > p.total ? p.total : m)), p.total);
    }
#pragma unroll
    for (int d = 16; d > 0; d >>= 1)
      rows = mm_add_rows(rows, __shfl_xor_sync(0xffffffffu, rows, d), p.total);
    if ((threadIdx.x & 31) == 0) warps[threadIdx.x >> 5] = rows;
    __syncthreads();
    rows = 0;
    for (int w = 0; w < kSumThreads / 32; ++w) rows = mm_add_rows(rows, warps[w], p.total);
    n = static_cast<int64_t>(rows) * p.C;
  }
  if (p.out32) sum_slices<float>(p, n);
  else sum_slices<uint16_t>(p, n);
}

}  // namespace mslkb
