// host.h -- internal: what the entry points outside mslkb.cu share on the host side (device
// set-up, error record, profiler ranges, launches with programmatic dependence).
#pragma once

#include <cuda_runtime.h>

#include <atomic>
#include <cstdint>

#include "mslkb.h"

namespace mslkb {

// Defined in mslkb.cu.
void record_cuda_error(cudaError_t e);

// Checks the current device (MSLKB_ERR_DEVICE unless sm_103) and returns its SM count.
mslkb_status device_sms(int* sm_count);

// NVTX push/pop range of the domain "mslkb" around a launch: `name` and the call's rows.
struct TraceRange {
  TraceRange(const char* name, int64_t rows);
  ~TraceRange();
};

inline mslkb_status launch_status(cudaError_t e) {
  if (e == cudaSuccess) return MSLKB_OK;
  record_cuda_error(e);
  return MSLKB_ERR_CUDA;
}

// Launches `kernel` with programmatic dependent launch: it may start while the stream's
// previous kernel ends, and waits (griddepcontrol.wait) before its first global access.  (One
// exception: the dispatch's copies bring rows to L2 before they wait, which changes nothing that
// another kernel reads or writes.)
// launch_cluster: in clusters of `cluster` CTAs.
template <class... Params, class... Args>
cudaError_t launch_cluster(void (*kernel)(Params...), dim3 grid, dim3 block, size_t smem,
                           int cluster, void* stream, Args... args) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = grid;
  cfg.blockDim = block;
  cfg.dynamicSmemBytes = smem;
  cfg.stream = static_cast<cudaStream_t>(stream);
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  if (cluster > 1) {
    attr[1].id = cudaLaunchAttributeClusterDimension;
    attr[1].val.clusterDim.x = static_cast<unsigned>(cluster);
    attr[1].val.clusterDim.y = 1;
    attr[1].val.clusterDim.z = 1;
    cfg.numAttrs = 2;
  }
  return cudaLaunchKernelEx(&cfg, kernel, static_cast<Params>(args)...);
}

template <class... Params, class... Args>
cudaError_t launch_dependent(void (*kernel)(Params...), dim3 grid, dim3 block, size_t smem,
                             void* stream, Args... args) {
  return launch_cluster(kernel, grid, block, smem, 1, stream, args...);
}

// Dynamic shared memory that one CTA can have beside a few KB of its own (227 KB in all), and
// what the CTAs of an SM have together.
constexpr int kMaxCtaSmem = 224 * 1024;
constexpr int kMaxSmSmem = 228 * 1024;

// Lets `kKernel` use up to kMaxCtaSmem of dynamic shared memory, once per device.
template <auto kKernel>
cudaError_t allow_smem() {
  static std::atomic<uint64_t> done{0};
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  const uint64_t bit = 1ull << (dev & 63);
  if (done.load() & bit) return cudaSuccess;
  e = cudaFuncSetAttribute(kKernel, cudaFuncAttributeMaxDynamicSharedMemorySize, kMaxCtaSmem);
  if (e == cudaSuccess) done.fetch_or(bit);
  return e;
}

inline bool aligned_to(const void* p, size_t bytes) {
  return reinterpret_cast<uintptr_t>(p) % bytes == 0;
}

inline int dtype_bytes(int32_t dtype) { return dtype == MSLKB_FP32 ? 4 : 2; }
inline bool dtype_ok(int32_t dtype) {
  return dtype == MSLKB_BF16 || dtype == MSLKB_FP16 || dtype == MSLKB_FP32;
}

}  // namespace mslkb
