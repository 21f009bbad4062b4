// mm_schedule.cpp -- the prefix of the experts' rows of grouped_mm.cuh on the CPU (lanes.h); included
// after its definitions, inside namespace mslkb.
template <bool kGrad_>
struct ScheduleCfg {
  static constexpr bool kGrad = kGrad_;
  static constexpr int kTileN = 256;
};

struct ScheduleRun {
  MmParams p;
  int32_t* first;
  int32_t* tile_pre;
  int32_t* tiles;
};

template <class Cfg>
void schedule_kernel(const ScheduleRun& r) {
  const int32_t tiles = mm_schedule<Cfg>(r.p, r.first, r.tile_pre, threadIdx.x);
  if (threadIdx.x == 0) *r.tiles = tiles;
}

extern "C" int run_schedule(int grad, const int64_t* m_sizes, int32_t G, int32_t total, int32_t ct,
                            int32_t R, int32_t* first, int32_t* tile_pre, int32_t* tiles,
                            uint32_t* status) {
  ScheduleRun r{};
  r.p.m_sizes = m_sizes;
  r.p.status = status;
  r.p.total = total;
  r.p.G = G;
  r.p.R = R;
  r.p.ct = ct;
  r.first = first;
  r.tile_pre = tile_pre;
  r.tiles = tiles;
  return !(grad ? lanes::launch(schedule_kernel<ScheduleCfg<true>>, dim3(1), dim3(32), r, 0, false)
                : lanes::launch(schedule_kernel<ScheduleCfg<false>>, dim3(1), dim3(32), r, 0, false));
}

extern "C" int32_t run_add_rows(int32_t a, int32_t b, int32_t total) {
  return mm_add_rows(a, b, total);
}
