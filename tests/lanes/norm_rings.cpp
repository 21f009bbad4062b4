// norm_rings.cpp -- the ring kernels of norm_quant.cu on the CPU (lanes.h); included after their
// definitions, inside namespace mslkb.
template <class T, int kVecs, int kStages, bool kRows>
int run_backward(const NormBackwardParams& p, dim3 grid, dim3 block, int order, bool late) {
  const int row = ring_stage_bytes<T, 8, kVecs>(p.dresidual != nullptr ? 3 : 2, block.x);
  if (kStages * static_cast<int>(block.y) * row > static_cast<int>(sizeof(lanes::g_ring))) return 2;
  return !lanes::launch(norm_backward_ring_kernel<T, kVecs, kStages, kRows>, grid, block, p, order,
                        late);
}

template <class T, int kVecs, int kStages>
int run_norm(const NormParams& p, dim3 grid, dim3 block, bool blocks, int order, bool late) {
  if (kStages * ring_stage_bytes<T, 16, kVecs>(p.residual != nullptr ? 2 : 1, block.x) >
      static_cast<int>(sizeof(lanes::g_ring)))
    return 2;
  return blocks ? !lanes::launch(norm_ring_kernel<T, kVecs, kStages, true>, grid, block, p, order, late)
                : !lanes::launch(norm_ring_kernel<T, kVecs, kStages, false>, grid, block, p, order, late);
}

extern "C" int run_norm_backward(int dtype, int vecs, int stages, int rows, const void* dy,
                                 const void* h, const void* weight, const float* rstd,
                                 const void* dresidual, void* dx, float* parts, int64_t T, int H,
                                 int grid, int x, int y, int order, int late) {
  const NormBackwardParams p{dy, h, weight, rstd, dresidual, dx, parts, T, H, 0, 1.f / H};
  const dim3 g(grid), b(x, y);
#define FORM(code, type, v, s, r) \
  if (dtype == code && vecs == v && stages == s && rows == r) \
    return run_backward<type, v, s, r>(p, g, b, order, late);
  FORM(0, __nv_bfloat16, 1, 2, true)
  FORM(0, __nv_bfloat16, 2, 3, true)
  FORM(0, __nv_bfloat16, 4, 2, true)
  FORM(0, __nv_bfloat16, 2, 3, false)
  FORM(0, __nv_bfloat16, 2, 2, false)
  FORM(2, float, 1, 2, true)
  FORM(2, float, 1, 2, false)
  FORM(2, float, 4, 2, false)
#undef FORM
  return 3;
}

extern "C" int run_norm_forward(int dtype, int vecs, int stages, const void* x,
                                const void* residual, const void* weight, uint8_t* q,
                                float* scale, void* residual_out, void* y, float* rstd, int64_t T,
                                int H, int blocks, int grid, int threads, int order, int late) {
  const NormParams p{x, residual, weight, q, scale, residual_out, y, rstd, T, H, H, H, 0, 1e-6f,
                     1.f / H};
  const dim3 g(grid), b(threads);
#define FORM(code, type, v, s) \
  if (dtype == code && vecs == v && stages == s) \
    return run_norm<type, v, s>(p, g, b, blocks, order, late);
  FORM(0, __nv_bfloat16, 1, 2)
  FORM(0, __nv_bfloat16, 1, 3)
  FORM(0, __nv_bfloat16, 2, 2)
  FORM(2, float, 1, 2)
#undef FORM
  return 3;
}
