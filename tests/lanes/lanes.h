// lanes.h -- runs a CUDA kernel of csrc/ on the CPU, thread by thread in a chosen order, to show
// what orders its accesses to shared memory.
//
// Every thread of a CTA is a fibre that runs on until it comes to a barrier or a shuffle that
// others have not reached yet; then the first thread in the order that can run goes on.  So a
// thread gets as far ahead of the others as the program lets it.  Asynchronous copies arrive either
// at once or when they are waited for: both ends of what the hardware may do.
#pragma once

#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_fp8.h>
#include <cuda_runtime.h>
#include <ucontext.h>

#include <algorithm>
#include <cmath>
#include <cstdint>
#include <cstdlib>
#include <cstring>
#include <functional>
#include <memory>
#include <vector>

using std::max;
using std::min;

namespace lanes {

struct Copy {
  uint8_t* to;
  const void* from;
  uint32_t bytes, read;
};

struct Fibre {
  ucontext_t context;
  std::unique_ptr<char[]> stack;
  uint3 thread;
  int index = 0;
  bool done = false;
  // waits until *passed of its barrier exceeds this
  const int64_t* passed = nullptr;
  int64_t until = 0;
  int64_t exchanges = 0;                  // shuffles and reductions so far
  std::vector<std::vector<Copy>> groups;  // committed, not yet arrived
  std::vector<Copy> open;
};

struct Barrier {
  int64_t arrived = 0, passed = 0;
};

constexpr int kStack = 128 << 10;

struct Cta {
  std::vector<Fibre> fibres;
  std::vector<Barrier> warps;
  Barrier named[16];
  std::vector<uint32_t> slots;  // [2][threads]
  ucontext_t scheduler;
  Fibre* current = nullptr;
  std::function<void()> body;
  bool late = false;  // copies arrive when they are waited for
};

inline Cta* g_cta = nullptr;
inline uint3 g_thread, g_block;
inline dim3 g_block_dim, g_grid_dim;
inline uint8_t g_ring[232448];

inline void yield() {
  Fibre* mine = g_cta->current;
  swapcontext(&mine->context, &g_cta->scheduler);
}

inline void arrive(Barrier& b, int64_t threads) {
  Fibre* mine = g_cta->current;
  const int64_t round = b.arrived++ / threads;
  if (b.arrived % threads == 0) b.passed = b.arrived / threads;
  mine->passed = &b.passed;
  mine->until = round;
  yield();
}

inline void warp_arrive() {
  Cta& c = *g_cta;
  const int warp = c.current->index / 32;
  arrive(c.warps[warp], 32);
}

// The warp's values of an exchange, once all its lanes have brought theirs.  A place is taken
// again two exchanges later, when all lanes have passed the one between.
inline const uint32_t* exchange(uint32_t v) {
  Cta& c = *g_cta;
  const size_t turn = c.current->exchanges++ % 2, threads = c.fibres.size();
  c.slots[turn * threads + c.current->index] = v;
  const size_t first = turn * threads + c.current->index / 32 * 32;
  warp_arrive();
  return &c.slots[first];
}

inline void arrive_copy(const Copy& c) {
  if (c.read) std::memcpy(c.to, c.from, c.read);
  std::memset(c.to + c.read, 0, c.bytes - c.read);
}

inline void entry() {
  g_cta->body();
  g_cta->current->done = true;
  yield();
}

// One launch.  The threads' order: 0 ascending, 1 descending, 2 odd threads first.  False: some
// threads wait for ever.
template <class Kernel, class Params>
bool launch(Kernel kernel, dim3 grid, dim3 block, const Params& p, int order, bool late) {
  const int threads = static_cast<int>(block.x * block.y);
  Cta c;
  c.late = late;
  c.body = [&] { kernel(p); };
  g_cta = &c;
  g_block_dim = block;
  g_grid_dim = grid;
  std::vector<int> by(threads);
  for (int i = 0; i < threads; ++i)
    by[i] = order == 0 ? i : (order == 1 ? threads - 1 - i : (2 * i + 1) % (threads | 1));
  std::vector<std::unique_ptr<char[]>> stacks(threads);
  for (auto& s : stacks) s.reset(new char[kStack]);
  for (unsigned b = 0; b < grid.x; ++b) {
    g_block = uint3{b, 0, 0};
    std::memset(g_ring, 0xFF, sizeof(g_ring));  // NaN
    c.fibres = std::vector<Fibre>(threads);
    c.warps.assign(threads / 32, Barrier());
    c.slots.assign(2 * threads, 0);
    for (Barrier& n : c.named) n = Barrier();
    for (int i = 0; i < threads; ++i) {
      Fibre& f = c.fibres[i];
      f.index = i;
      f.thread = uint3{i % block.x, i / block.x, 0};
      getcontext(&f.context);
      f.context.uc_stack.ss_sp = stacks[i].get();
      f.context.uc_stack.ss_size = kStack;
      f.context.uc_link = nullptr;
      makecontext(&f.context, entry, 0);
    }
    for (;;) {
      Fibre* next = nullptr;
      bool left = false;
      for (int i : by) {
        Fibre& f = c.fibres[i];
        if (f.done) continue;
        left = true;
        if (f.passed != nullptr && *f.passed <= f.until) continue;
        next = &f;
        break;
      }
      if (next == nullptr) {
        if (left) return false;
        break;
      }
      next->passed = nullptr;
      c.current = next;
      g_thread = next->thread;
      swapcontext(&c.scheduler, &next->context);
    }
  }
  return true;
}

}  // namespace lanes

// ---------------------------------------------------------------------------------
// what the kernels use of the device
// ---------------------------------------------------------------------------------
#define threadIdx lanes::g_thread
#define blockIdx lanes::g_block
#define blockDim lanes::g_block_dim
#define gridDim lanes::g_grid_dim
#undef __shared__
#define __shared__ static
#undef __launch_bounds__
#define __launch_bounds__(...)
#undef __grid_constant__
#define __grid_constant__

inline float __uint_as_float(uint32_t v) {
  float f;
  std::memcpy(&f, &v, 4);
  return f;
}
inline uint32_t __float_as_uint(float f) {
  uint32_t v;
  std::memcpy(&v, &f, 4);
  return v;
}
inline float rsqrtf(float x) { return static_cast<float>(1.0 / std::sqrt(static_cast<double>(x))); }
inline void __syncwarp() { lanes::warp_arrive(); }
inline void __syncthreads() {
  lanes::arrive(lanes::g_cta->named[0], static_cast<int64_t>(lanes::g_cta->fibres.size()));
}
inline uint32_t __shfl_xor_sync(uint32_t, uint32_t v, int d) {
  const int lane = lanes::g_cta->current->index % 32;
  return lanes::exchange(v)[lane ^ d];
}
inline float __shfl_xor_sync(uint32_t mask, float v, int d) {
  return __uint_as_float(__shfl_xor_sync(mask, __float_as_uint(v), d));
}
inline uint32_t __reduce_max_sync(uint32_t, uint32_t v) {
  const uint32_t* all = lanes::exchange(v);
  return *std::max_element(all, all + 32);
}

namespace mslkb {
namespace ptx {
inline void griddep_wait() {}
inline void griddep_launch_dependents() {}
inline uint32_t smem_addr(const void* p) {
  return static_cast<uint32_t>(static_cast<const uint8_t*>(p) - lanes::g_ring);
}
template <int kBytes>
void cp_async(uint32_t dst, const void* src, uint32_t src_bytes) {
  const lanes::Copy c{lanes::g_ring + dst, src, kBytes, src_bytes};
  if (lanes::g_cta->late)
    lanes::g_cta->current->open.push_back(c);
  else
    lanes::arrive_copy(c);
}
inline void cp_async_commit() {
  lanes::Fibre& f = *lanes::g_cta->current;
  f.groups.push_back(std::move(f.open));
  f.open.clear();
}
template <int kPending>
void cp_async_wait() {
  lanes::Fibre& f = *lanes::g_cta->current;
  while (f.groups.size() > kPending) {
    for (const lanes::Copy& c : f.groups.front()) lanes::arrive_copy(c);
    f.groups.erase(f.groups.begin());
  }
}
inline void named_bar_sync(uint32_t id, uint32_t threads) {
  lanes::arrive(lanes::g_cta->named[id], threads);
}
}  // namespace ptx

// in place of one-instruction forms
inline float max_nan(float a, float b) {
  return std::isnan(a) || std::isnan(b) ? NAN : std::max(a, b);
}
inline float max_nan(float a, float b, float c) { return max_nan(max_nan(a, b), c); }
inline float recip(float x) { return 1.f / x; }
inline uint32_t pack_e4m3x4(float a, float b, float c, float d) {
  const float v[4] = {a, b, c, d};
  uint32_t w = 0;
  for (int i = 0; i < 4; ++i)
    w |= static_cast<uint32_t>(__nv_cvt_float_to_fp8(v[i], __NV_SATFINITE, __NV_E4M3)) << (8 * i);
  return w;
}
}  // namespace mslkb
