// grouped_mm.cu -- 16-bit products by expert: which kernel serves a call, and the entry points.
// (The kernel, its mathematics and layout: grouped_mm.cuh.)
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
  const int64_t ct = ceil_to(p.C, Cfg::kTileC);
  if (Cfg::kGrad) return p.G * ct * ceil_to(p.R, Cfg::kTileN);
  return ct * (p.total / Cfg::kTileN + (p.G < p.total ? p.G : p.total));
}

template <class Cfg>
mslkb_status launch(const MmParams& p, const CUtensorMap (&maps)[3], int sms, void* stream) {
  cudaError_t e = allow_smem<grouped_mm_kernel<Cfg>>();
  if (e != cudaSuccess) return launch_status(e);
  const int64_t tiles = tiles_bound<Cfg>(p);
  if (tiles > INT32_MAX) return MSLKB_ERR_SHAPE;
  const int64_t workers = sms / Cfg::kCtas;
  const int64_t grid = (tiles < workers ? tiles : workers) * Cfg::kCtas;
  return launch_status(launch_cluster(grouped_mm_kernel<Cfg>, dim3(static_cast<unsigned>(grid)),
                                      dim3(Cfg::kThreads), Cfg::kSmemBytes, Cfg::kCtas, stream, p,
                                      maps[0], maps[1], maps[2]));
}

// Tensor maps of P, Q and what is added.  Matrices of experts have three dimensions, so that what
// lies past one is read as zero and not as the next.
template <class Cfg>
mslkb_status encode(const MmParams& p, CUtensorMap (&maps)[3]) {
  const uint64_t C = p.C, K = p.K, G = p.G, total = p.total, R = p.R;
  const uint64_t ldp = 2 * p.ldp, ldq = 2 * p.ldq;
  const uint32_t kbk = Cfg::kBK;
  mslkb_status s;
  if constexpr (Cfg::kMode == Mm::kRows) {
    const uint64_t extent[3] = {K, C, G}, stride[2] = {2 * K, 2 * K * C};
    const uint32_t box[3] = {64, 128, 1};
    s = encode_map16(&maps[0], p.P, 3, extent, stride, box);
  } else if constexpr (Cfg::kMode == Mm::kTurned) {
    const uint64_t extent[3] = {C, K, G}, stride[2] = {2 * C, 2 * K * C};
    const uint32_t box[3] = {64, kbk, 1};
    s = encode_map16(&maps[0], p.P, 3, extent, stride, box);
  } else {
    const uint64_t extent[2] = {C, total};
    const uint32_t box[2] = {64, kbk};
    s = encode_map16(&maps[0], p.P, 2, extent, &ldp, box);
  }
  if (s == MSLKB_OK) {
    const uint64_t extent[2] = {Cfg::kGrad ? R : K, total};
    const uint32_t box[2] = {64, Cfg::kGrad ? kbk : static_cast<uint32_t>(Cfg::kBoxQ)};
    s = encode_map16(&maps[1], p.Q, 2, extent, &ldq, box);
  }
  if (s == MSLKB_OK && Cfg::kAddRing) {
    const uint64_t bytes = p.out32 ? 4 : 2;
    const uint64_t extent[3] = {C, R, G}, stride[2] = {bytes * C, bytes * C * R};
    const uint32_t box[3] = {128, static_cast<uint32_t>(Cfg::kChunk), 1};
    s = encode_map_plain(&maps[2], p.add, static_cast<int>(bytes), 3, extent, stride, box);
  }
  return s;
}

// Rows that TMA can fetch: 16-byte aligned, and so spaced.
template <Mm kMode>
bool by_tma(const MmParams& p) {
  const int64_t row_p = kMode == Mm::kGrad ? p.ldp : (kMode == Mm::kRows ? p.K : p.C);
  return aligned_to(p.P, 16) && aligned_to(p.Q, 16) && row_p % 8 == 0 && p.ldq % 8 == 0 &&
         (p.add == nullptr ||
          (aligned_to(p.add, 16) && static_cast<int64_t>(p.C) * (p.out32 ? 4 : 2) % 16 == 0));
}

template <class Cfg>
mslkb_status run_as(const MmParams& p, int sms, void* stream) {
  CUtensorMap maps[3];
  std::memset(maps, 0, sizeof maps);
  if (Cfg::kTma) {
    const mslkb_status s = encode<Cfg>(p, maps);
    if (s != MSLKB_OK) return s;
  }
  return launch<Cfg>(p, maps, sms, stream);
}

template <Mm kMode>
mslkb_status run(const MmParams& p, int sms, void* stream) {
  const bool sums = kMode == Mm::kGrad ? p.total > 0 : p.K > 0;
  if (!sums || !by_tma<kMode>(p)) return run_as<MmCfg<kMode, false, 1, 128, 1, 4, 4>>(p, sms, stream);
  if constexpr (kMode == Mm::kGrad) {
    if (p.add != nullptr)
      return run_as<MmCfg<kMode, true, 2, 256, 1, 4, 8, true>>(p, sms, stream);
  }
  return run_as<MmCfg<kMode, true, 2, 256, 1, 6, 8>>(p, sms, stream);
}

bool sizes_ok(int64_t total, int64_t G, int64_t N, int64_t K) {
  return total >= 0 && G >= 0 && N >= 0 && K >= 0 && total <= kMaxSize && N <= kMaxSize &&
         K <= kMaxSize && G <= kMaxGroups;
}

}  // namespace
}  // namespace mslkb

extern "C" {

mslkb_status mslkb_grouped_mm(const void* x, const void* w, const int64_t* m_sizes, void* out,
                              int64_t total_M, int64_t G, int64_t N, int64_t K, int64_t ldx,
                              int32_t transposed, int32_t dtype, void* stream) {
  using namespace mslkb;
  if (!sizes_ok(total_M, G, N, K) || ldx < K || ldx > MSLKB_MAX_DIM) return MSLKB_ERR_SHAPE;
  if (dtype != MSLKB_BF16 && dtype != MSLKB_FP16) return MSLKB_ERR_DTYPE;
  if (total_M == 0 || G == 0 || N == 0) return MSLKB_OK;
  if (m_sizes == nullptr || out == nullptr || (K > 0 && (x == nullptr || w == nullptr)))
    return MSLKB_ERR_NULL;
  if (!aligned_to(x, 2) || !aligned_to(w, 2) || !aligned_to(out, 2) || !aligned_to(m_sizes, 8))
    return MSLKB_ERR_ALIGN;
  DeviceHandles h;
  mslkb_status s = device_handles(&h);
  if (s != MSLKB_OK) return s;
  MmParams p{};
  p.P = static_cast<const uint16_t*>(w);
  p.Q = static_cast<const uint16_t*>(x);
  p.m_sizes = m_sizes;
  p.out = out;
  p.status = h.status;
  p.timeout_ns = h.timeout_ns;
  p.ldq = ldx;
  p.total = static_cast<int32_t>(total_M);
  p.G = static_cast<int32_t>(G);
  p.C = static_cast<int32_t>(N);
  p.K = static_cast<int32_t>(K);
  p.bf16 = dtype == MSLKB_BF16;
  const TraceRange range("grouped_mm", total_M);
  return transposed ? run<Mm::kTurned>(p, h.sms, stream) : run<Mm::kRows>(p, h.sms, stream);
}

mslkb_status mslkb_grouped_mm_weight_grad(const void* dy, const void* x, const int64_t* m_sizes,
                                          const void* add, void* dw, int64_t total_M, int64_t G,
                                          int64_t N, int64_t K, int64_t lddy, int64_t ldx,
                                          int32_t dtype, int32_t dw_fp32, void* stream) {
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
  DeviceHandles h;
  mslkb_status s = device_handles(&h);
  if (s != MSLKB_OK) return s;
  MmParams p{};
  p.P = static_cast<const uint16_t*>(x);
  p.Q = static_cast<const uint16_t*>(dy);
  p.m_sizes = m_sizes;
  p.out = dw;
  p.add = add;
  p.status = h.status;
  p.timeout_ns = h.timeout_ns;
  p.ldp = ldx;
  p.ldq = lddy;
  p.total = static_cast<int32_t>(total_M);
  p.G = static_cast<int32_t>(G);
  p.C = static_cast<int32_t>(K);
  p.R = static_cast<int32_t>(N);
  p.bf16 = dtype == MSLKB_BF16;
  p.out32 = dw_fp32 != 0;
  const TraceRange range("grouped_mm_weight_grad", total_M);
  return run<Mm::kGrad>(p, h.sms, stream);
}

}  // extern "C"
