// grouped_mm.cu -- 16-bit products by expert: which kernel serves a call, and the entry points.
// (The kernel, its mathematics and layout: grouped_mm.cuh.)
#include <atomic>
#include <cstring>

#include "grouped_mm.cuh"
#include "host.h"

namespace mslkb {
namespace {

constexpr int64_t kMaxSize = 1 << 30;  // of a dimension: indices of a tile stay within 32 bits

int64_t ceil_to(int64_t a, int64_t b) { return (a + b - 1) / b; }

// More tiles than a call can have: every group's last one may be partly filled.
template <class Cfg>
int64_t tiles_bound(const MmParams& p) {
  if (Cfg::kGrad) return p.ct * static_cast<int64_t>(p.G) * ceil_to(p.R, Cfg::kTileN);
  return p.ct * static_cast<int64_t>(p.total / Cfg::kTileN + (p.G < p.total ? p.G : p.total));
}

template <class Cfg>
mslkb_status launch(const MmParams& p, const MmMaps& maps, int sms, void* stream) {
  cudaError_t e = allow_smem<grouped_mm_kernel<Cfg>>();
  if (e != cudaSuccess) return launch_status(e);
  if constexpr (Cfg::kLong) {
    // a kernel that moves registers between its warps waits for ever if it starts with too few
    static std::atomic<int> regs{0};
    if (regs.load() == 0) {
      cudaFuncAttributes a;
      if ((e = cudaFuncGetAttributes(&a, grouped_mm_kernel<Cfg>)) != cudaSuccess)
        return launch_status(e);
      regs.store(a.numRegs);
    }
    if (regs.load() * Cfg::kThreads < 128 * Cfg::kRegsFew + 256 * Cfg::kRegsMany)
      return launch_status(cudaErrorInvalidConfiguration);
  }
  const int64_t tiles = tiles_bound<Cfg>(p) * p.splits;
  if (tiles > INT32_MAX) return MSLKB_ERR_SHAPE;
  const int64_t workers = sms / Cfg::kCtas;
  const int64_t grid = (tiles < workers ? tiles : workers) * Cfg::kCtas;
  return launch_status(launch_cluster(grouped_mm_kernel<Cfg>, dim3(static_cast<unsigned>(grid)),
                                      dim3(Cfg::kThreads), Cfg::kSmemBytes, Cfg::kCtas, stream, p,
                                      maps));
}

// Tensor maps of P, Q and what is added.  Matrices of experts have a dimension of their own, so
// that what lies past one is read as zero and not as the next.  An MN-major operand lies in shared
// memory in pieces of 64 elements: where its rows consist of whole pieces these are a dimension
// too, and one box fetches both pieces of a CTA.
template <class Cfg>
mslkb_status encode(MmParams& p, MmMaps* maps) {
  const uint64_t C = p.C, K = p.K, G = p.G, total = p.total, R = p.R;
  const uint64_t ldp = 2 * p.ldp, ldq = 2 * p.ldq;
  const uint32_t kbk = Cfg::kBK;
  mslkb_status s = MSLKB_OK;
  if (p.sums) {
    p.p_pieces = Cfg::kPMn && C % 64 == 0;
    p.q_pieces = Cfg::kQMn && R % 64 == 0;
    if constexpr (Cfg::kMode == Mm::kRows) {
      const uint64_t extent[3] = {K, C, G}, stride[2] = {ldp, ldp * C};
      const uint32_t box[3] = {64, static_cast<uint32_t>(p.wide), 1};
      s = encode_map16(&maps->p, p.P, 3, extent, stride, box);
    } else if constexpr (Cfg::kMode == Mm::kTurned) {
      const uint64_t extent[4] = {64, K, C / 64, G}, stride[3] = {ldp, 128, ldp * K};
      const uint32_t box[4] = {64, kbk, 2, 1};
      const uint64_t extent3[3] = {C, K, G}, stride3[2] = {ldp, ldp * K};
      const uint32_t box3[3] = {64, kbk, 1};
      s = p.p_pieces ? encode_map16(&maps->p, p.P, 4, extent, stride, box)
                     : encode_map16(&maps->p, p.P, 3, extent3, stride3, box3);
    } else {
      const uint64_t extent[3] = {64, total, C / 64}, stride[2] = {ldp, 128};
      const uint32_t box[3] = {64, kbk, 2};
      const uint64_t extent2[2] = {C, total};
      s = p.p_pieces ? encode_map16(&maps->p, p.P, 3, extent, stride, box)
                     : encode_map16(&maps->p, p.P, 2, extent2, &ldp, box);
    }
    const uint64_t extent[2] = {Cfg::kGrad ? R : K, total};
    const uint32_t box[2] = {64, Cfg::kGrad ? kbk : static_cast<uint32_t>(Cfg::kQRows)};
    const uint32_t box64[2] = {64, Cfg::kGrad ? kbk : 64u};
    if (s == MSLKB_OK) s = encode_map16(&maps->q64, p.Q, 2, extent, &ldq, box64);
    if (s == MSLKB_OK && p.q_pieces) {
      const uint64_t extent3[3] = {64, total, R / 64}, stride3[2] = {ldq, 128};
      const uint32_t box3[3] = {64, kbk, 2};
      s = encode_map16(&maps->q, p.Q, 3, extent3, stride3, box3);
    } else if (s == MSLKB_OK) {
      s = encode_map16(&maps->q, p.Q, 2, extent, &ldq, box);
    }
  }
  if (s == MSLKB_OK && Cfg::kAddRing) {
    const uint64_t bytes = Cfg::kAdd;
    const uint64_t extent[3] = {C, R, G}, stride[2] = {bytes * C, bytes * C * R};
    const uint32_t box[3] = {128, static_cast<uint32_t>(Cfg::kAddRows), 1};
    s = encode_map_plain(&maps->add, p.add, static_cast<int>(bytes), 3, extent, stride, box);
  }
  return s;
}

// Output columns of a CTA's share of a tile.  With few rows per expert the time is that of reading
// the weights, and a worker's that of its tiles' columns: of the widths up to 128, the one with
// which the worker of most columns has fewest, if as many experts have rows as can have.  One token
// on 8 experts of 4096 x 7168 on GB300, 76 pairs: two rounds of 256 columns (128 tiles) 83 us, of
// 216 (152 tiles) 79.
// (Split contractions fill the workers by themselves.)
template <class Cfg>
int32_t tile_columns(const MmParams& p, int sms) {
  const int64_t experts = p.G < p.total ? p.G : p.total, workers = sms / Cfg::kCtas;
  if (Cfg::kMode != Mm::kRows || p.splits > 1 || p.total > 128 * experts) return 128;
  auto columns = [&](int64_t w) {
    return ceil_to(experts * ceil_to(p.C, Cfg::kCtas * w), workers) * w;
  };
  int32_t best = 128;
  int64_t least = columns(128) * 9 / 10;   // (a box of fewer rows costs a little itself)
  for (int32_t w = 120; w >= 64; w -= 8)
    if (columns(w) < least) least = columns(w), best = w;
  return best;
}

template <class Cfg>
mslkb_status run_as(MmParams& p, int sms, void* stream) {
  MmMaps maps;
  std::memset(&maps, 0, sizeof maps);
  p.wide = tile_columns<Cfg>(p, sms);
  p.ct = static_cast<int32_t>(ceil_to(p.C, Cfg::kCtas * p.wide));
  const mslkb_status s = encode<Cfg>(p, &maps);
  return s != MSLKB_OK ? s : launch<Cfg>(p, maps, sms, stream);
}

template <Mm kMode>
mslkb_status run(MmParams& p, int sms, void* stream) {
  if constexpr (kMode == Mm::kGrad) {
    const int64_t row = static_cast<int64_t>(p.C) * (p.out32 ? 4 : 2);
    const bool ring =
        p.add != nullptr && p.splits == 1 && aligned_to(p.add, 16) && row % 16 == 0;
    // Sums in registers (kLong) where experts may well have more rows than the tensor core sums.
    // 32 experts of 4096 x 7168 on GB300, us in registers / in tensor memory: fp32, 256 rows each 803 /
    // 692, but 256 on average and up to 2000, 4096 x 2048, 246 / 280; 384 each onto something 1544 /
    // 1284.  16 bits, 700 rows each 1009 / 988, 1024 1152 / 1105, 1500 1798 / 2057; 1024 on average and up
    // to 9000 1361 / 1466.  (What is added in 16 bits never: loaded by the epilogue's threads it
    // takes 6600 us for 1024 rows each, 1298 through the ring.)
    const int64_t rows_from = p.out32 ? (ring ? 384 : 192) : 768;
    if ((p.out32 || p.add == nullptr) && p.total >= rows_from * p.G * p.splits)
      return run_as<MmCfg<kMode, 0, true>>(p, sms, stream);
    if (ring)
      return p.out32 ? run_as<MmCfg<kMode, 4>>(p, sms, stream)
                     : run_as<MmCfg<kMode, 2>>(p, sms, stream);
  }
  if constexpr (kMode != Mm::kGrad) {
    if (ceil_to(ceil_to(p.K, 64), p.splits) * 64 > kSumLen16)
      return run_as<MmCfg<kMode, 0, true>>(p, sms, stream);
  }
  return run_as<MmCfg<kMode>>(p, sms, stream);
}

// Each size, and the elements of each operand and result: what passes kMaxElements (2 TB in 16 bits)
// fits no device, and numbers of bytes, with all copies and slices, stay within 64 bits.
constexpr double kMaxElements = static_cast<double>(1ll << 40);
bool sizes_ok(int64_t total, int64_t G, int64_t N, int64_t K) {
  if (!(total >= 0 && G >= 0 && N >= 0 && K >= 0 && total <= kMaxSize && N <= kMaxSize &&
        K <= kMaxSize && G <= kMaxGroups))
    return false;
  const double t = static_cast<double>(total), g = static_cast<double>(G);
  const double n = static_cast<double>(N), k = static_cast<double>(K);
  return t * n <= kMaxElements && t * k <= kMaxElements && g * n * k <= kMaxElements;
}

// Parts of each contraction.  Few tiles leave most pairs without one, and a pair takes some 0.2 us
// for a stage of 64, however few the rows (4096 x 7168, one expert and row: 28 us); so the
// contractions of up to two rounds of tiles are split, into the number of parts that takes least by
// this reckoning: rounds of the pairs x (stages of a part, and a tile's ends), or the time that the
// operands take to read; and for the slices' sum a launch and their bytes.
// Warps that work once per tile wait for as long as a contraction takes, so that none may come near
// the time after which a wait gives up (1 s): a part has at most kMostTerms of the `longest` there
// can be, 0.2 s if every stage comes from memory and all pairs read at once (64 KB each, 0.8 us).
constexpr int kPairs = 76, kMostSplits = 16, kLeastStages = 4;
constexpr int64_t kMostTerms = 1 << 24;
int32_t splits_of(int64_t tiles, int64_t contraction, int64_t longest, int64_t elements,
                  int64_t operands) {
  const int64_t stages = ceil_to(contraction, 64);
  const int32_t needed = static_cast<int32_t>(ceil_to(longest, kMostTerms));
  if (tiles > 2 * kPairs) return needed;
  const double read = static_cast<double>(operands) * 2.0 / 6.5e6;
  int32_t best = 1;
  double least = 0.0;
  for (int32_t s = 1; s <= kMostSplits && (s == 1 || s * kLeastStages <= stages); ++s) {
    const double rounds = static_cast<double>(ceil_to(tiles * s, kPairs));
    double us = rounds * (0.2 * static_cast<double>(ceil_to(stages, s)) + 1.0);
    if (us < read) us = read;
    if (s > 1) us += 2.5 + static_cast<double>(elements) * 4.0 * 2.0 * s / 6e6;
    if (s == 1 || us < least) least = us, best = s;
  }
  return best > needed ? best : needed;
}

int64_t slice_of(int64_t elements) { return ceil_to(elements, 4) * 4; }

int32_t mm_splits(int64_t total_M, int64_t G, int64_t N, int64_t K) {
  if (total_M == 0 || G == 0 || N == 0 || K == 0) return 1;
  const int64_t experts = G < total_M ? G : total_M;   // with rows, at most
  return splits_of((total_M / 256 + experts) * ceil_to(N, 256), K, K, total_M * N,
                   experts * N * K + total_M * K);
}

int32_t grad_splits(int64_t total_M, int64_t G, int64_t N, int64_t K) {
  if (total_M == 0 || G == 0 || N == 0 || K == 0) return 1;
  // (experts have different numbers of rows: twice as many as they have on average, and one at
  // most all)
  return splits_of(G * ceil_to(N, 256) * ceil_to(K, 256), ceil_to(2 * total_M, G + 1), total_M,
                   G * N * K, total_M * (N + K));
}

// The slices' place in the workspace, behind the operands' copies.
int64_t slices_bytes(int32_t splits, int64_t elements) {
  return splits > 1 ? splits * slice_of(elements) * 4 : 0;
}

// Runs the product into slices, and sums them.
template <class F>
mslkb_status run_split(MmParams& p, int64_t elements, bool owned_rows, float* slices, int sms,
                       void* stream, F run_product) {
  SliceSum s{};
  s.slices = slices;
  s.out = p.out;
  s.add = p.add;
  s.m_sizes = owned_rows ? p.m_sizes : nullptr;
  s.slice = slice_of(elements);
  s.n = elements;
  s.splits = p.splits;
  s.G = p.G;
  s.total = p.total;
  s.C = p.C;
  s.bf16 = p.bf16;
  s.out32 = p.out32;
  p.out = slices;
  p.add = nullptr;
  p.out32 = 1;
  p.slice = s.slice;
  const mslkb_status status = run_product();
  if (status != MSLKB_OK) return status;
  const int64_t ctas = ceil_to(elements, 4 * kSumThreads), most = 8 * sms;
  return launch_status(launch_dependent(slice_sum_kernel,
                                        dim3(static_cast<unsigned>(ctas < most ? ctas : most)),
                                        dim3(kSumThreads), 0, stream, s));
}

// An operand as the call gives it: rows of a matrix, or of all experts' (per_expert rows each).
struct Operand {
  const void* at;
  int64_t rows, cols, ld, per_expert;

  // TMA fetches rows that start on 16 bytes and are spaced by multiples of 16.
  bool fits() const { return aligned_to(at, 16) && (rows <= 1 || ld % 8 == 0); }
  int64_t copy_ld() const { return ceil_to(cols, 8) * 8; }
  int64_t copy_bytes() const {
    return fits() || rows == 0 || cols == 0 ? 0 : ceil_to(rows * copy_ld() * 2, 256) * 256;
  }
};

// Whether `bytes` at `to` lie over an element of `rows` rows of `cols` 16-bit elements, ld apart.
bool lies_over(const void* to, int64_t bytes, const void* from, int64_t rows, int64_t cols,
               int64_t ld) {
  if (bytes == 0 || rows == 0 || cols == 0) return false;
  const int64_t a = static_cast<int64_t>(reinterpret_cast<uintptr_t>(from));
  const int64_t b = static_cast<int64_t>(reinterpret_cast<uintptr_t>(to));
  if (b + bytes <= a) return false;
  // the last row that starts before the end of `to`
  const int64_t last = (b + bytes - 1 - a) / (2 * ld);
  return a + 2 * ((last < rows ? last : rows - 1) * ld + cols) > b;
}

// The operands as they are, or copied to aligned rows in the workspace.
mslkb_status align_operands(Operand (&o)[2], const int64_t* m_sizes, void* workspace, int sms,
                            void* stream) {
  AlignedCopy c[2] = {};
  int n = 0;
  uint8_t* to = static_cast<uint8_t*>(workspace);
  int64_t units = 0;
  for (Operand& p : o) {
    const int64_t bytes = p.copy_bytes();
    if (bytes == 0) {
      if (p.rows <= 1) p.ld = p.copy_ld();
      continue;
    }
    c[n++] = {static_cast<const uint16_t*>(p.at), reinterpret_cast<uint16_t*>(to), p.ld,
              p.copy_ld(), p.rows, static_cast<int32_t>(p.cols),
              static_cast<int32_t>(p.per_expert)};
    units += p.rows * ceil_to(p.cols, kCopyCols);
    p.at = to;
    p.ld = p.copy_ld();
    to += bytes;
  }
  if (n == 0) return MSLKB_OK;
  const int64_t ctas = ceil_to(units, kCopyThreads / 32), most = 8 * sms;
  return launch_status(launch_dependent(
      aligned_rows_kernel, dim3(static_cast<unsigned>(ctas < most ? ctas : most)),
      dim3(kCopyThreads), 0, stream, c[0], c[1], m_sizes));
}

int64_t copies_bytes(const Operand (&o)[2]) { return o[0].copy_bytes() + o[1].copy_bytes(); }

mslkb_status workspace_status(int64_t need, const void* workspace, int64_t bytes) {
  if (need == 0) return MSLKB_OK;
  return workspace != nullptr && aligned_to(workspace, 16) && bytes >= need ? MSLKB_OK
                                                                            : MSLKB_ERR_WORKSPACE;
}

void mm_operands(Operand (&o)[2], const void* x, const void* w, int64_t total_M, int64_t G,
                 int64_t N, int64_t K, int64_t ldx, int32_t transposed) {
  const int64_t rows = transposed ? K : N, cols = transposed ? N : K;
  o[0] = {w, G * rows, cols, cols, rows};
  o[1] = {x, total_M, K, ldx, 0};
}

}  // namespace
}  // namespace mslkb

extern "C" {

int64_t mslkb_grouped_mm_workspace_bytes(const void* x, const void* w, int64_t total_M, int64_t G,
                                         int64_t N, int64_t K, int64_t ldx, int32_t transposed) {
  using namespace mslkb;
  if (!sizes_ok(total_M, G, N, K) || total_M == 0 || G == 0 || N == 0) return 0;
  Operand o[2];
  mm_operands(o, x, w, total_M, G, N, K, ldx, transposed);
  return copies_bytes(o) + slices_bytes(mm_splits(total_M, G, N, K), total_M * N);
}

mslkb_status mslkb_grouped_mm(const void* x, const void* w, const int64_t* m_sizes, void* out,
                              int64_t total_M, int64_t G, int64_t N, int64_t K, int64_t ldx,
                              int32_t transposed, int32_t dtype, void* workspace,
                              int64_t workspace_bytes, void* stream) {
  using namespace mslkb;
  if (!sizes_ok(total_M, G, N, K) || ldx < K || ldx > MSLKB_MAX_DIM) return MSLKB_ERR_SHAPE;
  if (dtype != MSLKB_BF16 && dtype != MSLKB_FP16) return MSLKB_ERR_DTYPE;
  if (total_M == 0 || G == 0 || N == 0) return MSLKB_OK;
  if (m_sizes == nullptr || out == nullptr || (K > 0 && (x == nullptr || w == nullptr)))
    return MSLKB_ERR_NULL;
  if (!aligned_to(x, 2) || !aligned_to(w, 2) || !aligned_to(out, 2) || !aligned_to(m_sizes, 8))
    return MSLKB_ERR_ALIGN;
  Operand o[2];
  mm_operands(o, x, w, total_M, G, N, K, ldx, transposed);
  const int64_t copies = copies_bytes(o);
  const int32_t splits = mm_splits(total_M, G, N, K);
  mslkb_status s = workspace_status(copies + slices_bytes(splits, total_M * N), workspace,
                                    workspace_bytes);
  if (s != MSLKB_OK) return s;
  for (const Operand& p : o)   // (what is written must not have been an input of other tiles)
    if (lies_over(out, 2 * total_M * N, p.at, p.rows, p.cols, p.ld)) return MSLKB_ERR_SHAPE;
  if (lies_over(out, 2 * total_M * N, m_sizes, 1, 4 * G, 4 * G)) return MSLKB_ERR_SHAPE;
  DeviceHandles h;
  if ((s = device_handles(&h)) != MSLKB_OK) return s;
  const TraceRange range("grouped_mm", total_M);
  if ((s = align_operands(o, m_sizes, workspace, h.sms, stream)) != MSLKB_OK) return s;
  MmParams p{};
  p.P = static_cast<const uint16_t*>(o[0].at);
  p.Q = static_cast<const uint16_t*>(o[1].at);
  p.ldp = o[0].ld;
  p.ldq = o[1].ld;
  p.m_sizes = m_sizes;
  p.out = out;
  p.status = h.status;
  p.timeout_ns = h.timeout_ns;
  p.test_stall = h.test_stall;
  p.total = static_cast<int32_t>(total_M);
  p.G = static_cast<int32_t>(G);
  p.C = static_cast<int32_t>(N);
  p.K = static_cast<int32_t>(K);
  p.bf16 = dtype == MSLKB_BF16;
  p.sums = K > 0;
  p.splits = splits;
  auto product = [&] {
    return transposed ? run<Mm::kTurned>(p, h.sms, stream) : run<Mm::kRows>(p, h.sms, stream);
  };
  if (splits == 1) return product();
  float* slices = reinterpret_cast<float*>(static_cast<uint8_t*>(workspace) + copies);
  return run_split(p, total_M * N, true, slices, h.sms, stream, product);
}

int64_t mslkb_grouped_mm_weight_grad_workspace_bytes(const void* dy, const void* x,
                                                     int64_t total_M, int64_t G, int64_t N,
                                                     int64_t K, int64_t lddy, int64_t ldx) {
  using namespace mslkb;
  if (!sizes_ok(total_M, G, N, K) || G == 0 || N == 0 || K == 0) return 0;
  const Operand o[2] = {{x, total_M, K, ldx, 0}, {dy, total_M, N, lddy, 0}};
  return copies_bytes(o) + slices_bytes(grad_splits(total_M, G, N, K), G * N * K);
}

mslkb_status mslkb_grouped_mm_weight_grad(const void* dy, const void* x, const int64_t* m_sizes,
                                          const void* add, void* dw, int64_t total_M, int64_t G,
                                          int64_t N, int64_t K, int64_t lddy, int64_t ldx,
                                          int32_t dtype, int32_t dw_fp32, void* workspace,
                                          int64_t workspace_bytes, void* stream) {
  using namespace mslkb;
  if (!sizes_ok(total_M, G, N, K) || ldx < K || lddy < N || ldx > MSLKB_MAX_DIM ||
      lddy > MSLKB_MAX_DIM)
    return MSLKB_ERR_SHAPE;
  if (dtype != MSLKB_BF16 && dtype != MSLKB_FP16) return MSLKB_ERR_DTYPE;
  if (G == 0 || N == 0 || K == 0) return MSLKB_OK;
  if (m_sizes == nullptr || dw == nullptr || (total_M > 0 && (x == nullptr || dy == nullptr)))
    return MSLKB_ERR_NULL;
  const size_t wide = dw_fp32 ? 4 : 2;
  if (!aligned_to(x, 2) || !aligned_to(dy, 2) || !aligned_to(m_sizes, 8) ||
      !aligned_to(dw, wide) || !aligned_to(add, wide))
    return MSLKB_ERR_ALIGN;
  if (add != nullptr && add != dw) {   // (added to what has not been written yet)
    const uintptr_t a = reinterpret_cast<uintptr_t>(add), b = reinterpret_cast<uintptr_t>(dw);
    const double bytes = static_cast<double>(G) * N * K * wide;
    if (static_cast<double>(a < b ? b - a : a - b) < bytes) return MSLKB_ERR_SHAPE;
  }
  Operand o[2] = {{x, total_M, K, ldx, 0}, {dy, total_M, N, lddy, 0}};
  const int64_t copies = copies_bytes(o);
  const int32_t splits = grad_splits(total_M, G, N, K);
  mslkb_status s = workspace_status(copies + slices_bytes(splits, G * N * K), workspace,
                                    workspace_bytes);
  if (s != MSLKB_OK) return s;
  const int64_t dw_bytes = G * N * K * static_cast<int64_t>(wide);
  for (const Operand& p : o)
    if (lies_over(dw, dw_bytes, p.at, p.rows, p.cols, p.ld)) return MSLKB_ERR_SHAPE;
  if (lies_over(dw, dw_bytes, m_sizes, 1, 4 * G, 4 * G)) return MSLKB_ERR_SHAPE;
  DeviceHandles h;
  if ((s = device_handles(&h)) != MSLKB_OK) return s;
  const TraceRange range("grouped_mm_weight_grad", total_M);
  if ((s = align_operands(o, m_sizes, workspace, h.sms, stream)) != MSLKB_OK) return s;
  MmParams p{};
  p.P = static_cast<const uint16_t*>(o[0].at);
  p.Q = static_cast<const uint16_t*>(o[1].at);
  p.ldp = o[0].ld;
  p.ldq = o[1].ld;
  p.m_sizes = m_sizes;
  p.out = dw;
  p.add = add;
  p.status = h.status;
  p.timeout_ns = h.timeout_ns;
  p.test_stall = h.test_stall;
  p.total = static_cast<int32_t>(total_M);
  p.G = static_cast<int32_t>(G);
  p.C = static_cast<int32_t>(K);
  p.R = static_cast<int32_t>(N);
  p.bf16 = dtype == MSLKB_BF16;
  p.out32 = dw_fp32 != 0;
  p.sums = total_M > 0;
  p.splits = splits;
  if (splits == 1) return run<Mm::kGrad>(p, h.sms, stream);
  float* slices = reinterpret_cast<float*>(static_cast<uint8_t*>(workspace) + copies);
  return run_split(p, G * N * K, false, slices, h.sms, stream,
                   [&] { return run<Mm::kGrad>(p, h.sms, stream); });
}

}  // extern "C"
