// binding.cpp -- the Python extension _binding: checks the torch tensors of a call of the
// operators around the grouped product, and of those for training, and passes their addresses to
// libmslkb.so.  A call of one token takes 3 us on the device; the checks take about 0.1 us here
// (with Python code and ctypes they took 5).  Nothing is computed here, and nothing allocated but
// a call's scratch: of the norm's gradient, the 16-bit products and the gradients' norm.
//
// Every function takes positional arguments only (moe.py and training.py name them) and returns
// the mslkb_status, or kNoColumns; wrong tensors raise TypeError or ValueError.  `out` is the
// tuple of results, or the result of a function that has one (the clipping's: its list), `stream`
// None (the current stream) or a cudaStream_t as an integer.
#define PY_SSIZE_T_CLEAN
#include <Python.h>

#include <ATen/core/Tensor.h>
#include <c10/cuda/CUDACachingAllocator.h>
#include <c10/cuda/CUDAFunctions.h>
#include <c10/cuda/CUDAStream.h>
#include <c10/util/Exception.h>
#include <torch/csrc/autograd/python_variable.h>

#include <cstdint>
#include <exception>
#include <initializer_list>
#include <string>
#include <vector>

#include "mslkb.h"

namespace {

struct PythonError {};  // thrown once the Python error is set

[[noreturn]] void raise(PyObject* type, const std::string& text) {
  PyErr_SetString(type, text.c_str());
  throw PythonError{};
}

std::string shape_text(c10::IntArrayRef shape) {
  std::string s = "(";
  for (size_t i = 0; i < shape.size(); ++i)
    s += (i ? ", " : "") + std::to_string(shape[i]);
  return s + (shape.size() == 1 ? ",)" : ")");
}

const at::Tensor& tensor(PyObject* o, const char* name) {
  if (!THPVariable_Check(o)) raise(PyExc_TypeError, std::string(name) + " must be a torch.Tensor");
  return THPVariable_Unpack(o);
}

using Shape = std::initializer_list<int64_t>;
constexpr at::ScalarType kE4m3 = at::kFloat8_e4m3fn;

// A call: the device and element type of the tensor that leads it.
struct Call {
  int device = 0;
  at::ScalarType type = at::kFloat;
  int32_t dtype = MSLKB_FP32;

  // The leading tensor is on the current device, a matrix; its type is one of the three
  // floats unless `any_type`.
  const at::Tensor& lead(PyObject* o, const char* name, bool any_type = false) {
    const at::Tensor& t = tensor(o, name);
    type = t.scalar_type();
    if (type == at::kBFloat16)
      dtype = MSLKB_BF16;
    else if (type == at::kHalf)
      dtype = MSLKB_FP16;
    else if (type != at::kFloat && !any_type)
      raise(PyExc_TypeError, std::string(name) + ": dtype " + c10::toString(type) +
                                 " is not bfloat16, float16 or float32");
    if (!t.is_cuda()) raise(PyExc_ValueError, std::string(name) + " must be a CUDA tensor");
    device = t.get_device();
    if (device != c10::cuda::current_device())
      raise(PyExc_ValueError, std::string(name) + " is on another device than the current one");
    matrix(t, name);
    return t;
  }

  static void matrix(const at::Tensor& t, const char* name) {
    if (t.dim() != 2)
      raise(PyExc_ValueError,
            std::string(name) + ": expected 2 dims, got " + std::to_string(t.dim()));
  }

  void check(const at::Tensor& t, const char* name, at::ScalarType want,
             c10::IntArrayRef shape) const {
    const at::ScalarType got = t.scalar_type();
    if (got != want && !(want == kE4m3 && got == at::kByte))
      raise(PyExc_TypeError, std::string(name) + ": dtype " + c10::toString(got) +
                                 ", expected " + c10::toString(want));
    if (t.sizes() != shape)
      raise(PyExc_ValueError, std::string(name) + ": shape " + shape_text(t.sizes()) +
                                  ", expected " + shape_text(shape));
    if (!t.is_cuda() || t.get_device() != device)
      raise(PyExc_ValueError, std::string(name) + " must be a CUDA tensor on the same device");
  }

  // A dense tensor's address.
  void* dense(PyObject* o, const char* name, at::ScalarType want, c10::IntArrayRef shape) const {
    const at::Tensor& t = tensor(o, name);
    check(t, name, want, shape);
    if (!t.is_contiguous())
      raise(PyExc_ValueError, std::string(name) + " must be contiguous");
    return t.data_ptr();
  }
  void* dense(PyObject* o, const char* name, at::ScalarType want, Shape shape) const {
    return dense(o, name, want, c10::IntArrayRef(shape));
  }
  void* dense_or_null(PyObject* o, const char* name, at::ScalarType want, Shape shape) const {
    return o == Py_None ? nullptr : dense(o, name, want, shape);
  }

  // An input whose rows may be slices of wider rows: its address, and elements from row to row.
  void* rows(PyObject* o, const char* name, Shape shape, int64_t* ld) const {
    const at::Tensor& t = tensor(o, name);
    check(t, name, type, c10::IntArrayRef(shape));
    const int64_t cols = t.size(1);
    *ld = cols;
    if (!t.is_contiguous()) {
      if (t.stride(1) != 1 && cols > 1)
        raise(PyExc_ValueError, std::string(name) + ": the elements of a row must be contiguous");
      if (t.size(0) > 1) *ld = t.stride(0);
      if (*ld < cols) raise(PyExc_ValueError, std::string(name) + ": rows must not overlap");
    }
    return t.data_ptr();
  }

  void* stream(PyObject* o) const {
    if (o == Py_None) return c10::cuda::getCurrentCUDAStream(device).stream();
    const unsigned long long v = PyLong_AsUnsignedLongLong(o);
    if (PyErr_Occurred()) throw PythonError{};
    return reinterpret_cast<void*>(static_cast<uintptr_t>(v));
  }
};

bool flag(PyObject* o) {
  const int v = PyObject_IsTrue(o);
  if (v < 0) throw PythonError{};
  return v != 0;
}
int64_t integer(PyObject* o) {
  const long long v = PyLong_AsLongLong(o);
  if (v == -1 && PyErr_Occurred()) throw PythonError{};
  return v;
}
double number(PyObject* o) {
  const double v = PyFloat_AsDouble(o);
  if (v == -1.0 && PyErr_Occurred()) throw PythonError{};
  return v;
}

// The results of a call.
struct Out {
  PyObject* o;
  Out(PyObject* o_, Py_ssize_t count) : o(o_) {
    if (!PyTuple_Check(o)) raise(PyExc_TypeError, "out must be a tuple of tensors");
    if (PyTuple_GET_SIZE(o) != count)
      raise(PyExc_ValueError, "out must hold " + std::to_string(count) +
                                  " tensors (None where there is none)");
  }
  PyObject* operator[](Py_ssize_t i) const { return PyTuple_GET_ITEM(o, i); }
  // a result that is there exactly if it is wanted
  PyObject* if_wanted(Py_ssize_t i, const char* name, bool wanted) const {
    PyObject* t = (*this)[i];
    if ((t != Py_None) != wanted)
      raise(PyExc_ValueError,
            std::string("out: ") + name + " must be " + (wanted ? "a tensor" : "None"));
    return t;
  }
};

// Runs the library's call without the interpreter lock, as a wait for room in the stream's
// queue should not hold other threads up.
template <class F>
PyObject* run(F f) {
  mslkb_status s;
  Py_BEGIN_ALLOW_THREADS;
  s = f();
  Py_END_ALLOW_THREADS;
  return PyLong_FromLong(s);
}

// In place of MSLKB_OK: the rows have no columns, for which the library writes nothing, and the
// caller fills what there is per row.
constexpr long kNoColumns = -1;

template <class F>
PyObject* run(F f, int64_t cols) {
  PyObject* status = run(f);
  if (cols > 0 || status == nullptr || PyLong_AsLong(status) != MSLKB_OK) return status;
  Py_DECREF(status);
  return PyLong_FromLong(kNoColumns);
}

// Shape of e4m3 scales: (rows,), or (rows, cols / 128) block-scaled.
struct ScaleShape {
  int64_t v[2];
  size_t dims;
  ScaleShape(int64_t rows, int64_t cols, bool groupwise) : v{rows, cols / 128}, dims(1 + groupwise) {
    if (groupwise && cols % 128 != 0)
      raise(PyExc_ValueError, "groupwise scales need rows of whole blocks of 128");
  }
  operator c10::IntArrayRef() const { return {v, dims}; }
};

// A norm weight of the call's type, or fp32 beside another type.
void* weight_of(const Call& c, PyObject* o, int64_t H, int32_t* fp32) {
  const at::Tensor& t = tensor(o, "weight");
  *fp32 = t.scalar_type() == at::kFloat && c.type != at::kFloat;
  return c.dense(o, "weight", *fp32 ? at::kFloat : c.type, {H});
}

// x, weight, residual, eps, groupwise, want_y, want_rstd, out, stream
PyObject* add_rms_norm_quant(PyObject* const* a) {
  Call c;
  const at::Tensor& x = c.lead(a[0], "x");
  const int64_t T = x.size(0), H = x.size(1);
  int64_t ldx = H, ldr = H;
  int32_t fp32 = 0;
  const void* xp = c.rows(a[0], "x", {T, H}, &ldx);
  const void* w = weight_of(c, a[1], H, &fp32);
  const bool add = a[2] != Py_None;
  const void* r = add ? c.rows(a[2], "residual", {T, H}, &ldr) : nullptr;
  const double eps = number(a[3]);
  const bool groupwise = flag(a[4]);
  const Out out(a[7], 5);
  void* q = c.dense(out[0], "q", kE4m3, {T, H});
  void* scale = c.dense(out[1], "scale", at::kFloat, ScaleShape(T, H, groupwise));
  void* ro = c.dense_or_null(out.if_wanted(2, "residual", add), "residual (out)", c.type, {T, H});
  void* y = c.dense_or_null(out.if_wanted(3, "y", flag(a[5])), "y", c.type, {T, H});
  void* rstd = c.dense_or_null(out.if_wanted(4, "rstd", flag(a[6])), "rstd", at::kFloat, {T});
  void* s = c.stream(a[8]);
  return run([&] {
    return mslkb_add_rms_norm_quant(xp, r, w, q, static_cast<float*>(scale), ro, y,
                                    static_cast<float*>(rstd), T, H, ldx, ldr, eps, c.dtype, fp32,
                                    groupwise, s);
  }, H);
}

// Scratch of one call from torch's allocator, for the stream of the call; given back once the
// call is enqueued, as a tensor of that stream would be.
struct Scratch {
  void* p;
  Scratch(int64_t bytes, void* stream)
      : p(bytes > 0 ? c10::cuda::CUDACachingAllocator::raw_alloc_with_stream(
                          static_cast<size_t>(bytes), static_cast<cudaStream_t>(stream))
                    : nullptr) {}
  ~Scratch() {
    if (p != nullptr) c10::cuda::CUDACachingAllocator::raw_delete(p);
  }
};

// dy, h, weight, rstd, dresidual, out, stream
PyObject* add_rms_norm_quant_backward(PyObject* const* a) {
  Call c;
  const at::Tensor& lead = c.lead(a[0], "dy");
  const int64_t T = lead.size(0), H = lead.size(1);
  int32_t fp32 = 0;
  const void* dy = c.dense(a[0], "dy", c.type, {T, H});
  const void* h = c.dense(a[1], "h", c.type, {T, H});
  const void* w = weight_of(c, a[2], H, &fp32);
  const void* rstd = c.dense(a[3], "rstd", at::kFloat, {T});
  const void* dres = c.dense_or_null(a[4], "dresidual", c.type, {T, H});
  const Out out(a[5], 2);
  void* dx = c.dense(out[0], "dx", c.type, {T, H});
  void* dw = c.dense(out[1], "dweight", at::kFloat, {H});
  void* s = c.stream(a[6]);
  const int64_t bytes = mslkb_add_rms_norm_quant_backward_workspace_bytes(T, H);
  const Scratch workspace(bytes, s);
  return run([&] {
    return mslkb_add_rms_norm_quant_backward(dy, h, w, static_cast<const float*>(rstd), dres, dx,
                                             static_cast<float*>(dw), workspace.p, bytes, T, H,
                                             c.dtype, fp32, s);
  });
}

// logits, top_k, bias, score, num_groups, topk_groups, group_top, renormalize, scale, out, stream
PyObject* route_experts(PyObject* const* a) {
  Call c;
  const at::Tensor& x = c.lead(a[0], "logits");
  const int64_t T = x.size(0), E = x.size(1), k = integer(a[1]);
  int64_t ld = E;
  const void* logits = c.rows(a[0], "logits", {T, E}, &ld);
  const void* bias = c.dense_or_null(a[2], "bias", at::kFloat, {E});
  const Out out(a[9], 2);
  void* ids = c.dense(out[0], "ids", at::kInt, {T, k});
  void* weights = c.dense(out[1], "weights", at::kFloat, {T, k});
  const int32_t score = static_cast<int32_t>(integer(a[3]));
  const int64_t groups = integer(a[4]), top_groups = integer(a[5]), group_top = integer(a[6]);
  const bool renormalize = flag(a[7]);
  const double scale = number(a[8]);
  void* s = c.stream(a[10]);
  return run([&] {
    return mslkb_route_experts(logits, static_cast<const float*>(bias), static_cast<int32_t*>(ids),
                               static_cast<float*>(weights), T, E, ld, k, score, groups,
                               top_groups, group_top == 1 || group_top == 2
                                               ? static_cast<int32_t>(group_top)
                                               : 0,
                               renormalize, scale, c.dtype, s);
  });
}

// dweights, logits, ids, score, renormalize, scale, out, stream
PyObject* route_experts_backward(PyObject* const* a) {
  Call c;
  const at::Tensor& x = c.lead(a[1], "logits");
  const int64_t T = x.size(0), E = x.size(1);
  int64_t ld = E;
  const void* logits = c.rows(a[1], "logits", {T, E}, &ld);
  const at::Tensor& chosen = tensor(a[2], "ids");
  Call::matrix(chosen, "ids");
  const int64_t k = chosen.size(1);
  const void* ids = c.dense(a[2], "ids", at::kInt, {T, k});
  const void* dw = c.dense(a[0], "dweights", at::kFloat, {T, k});
  const int32_t score = static_cast<int32_t>(integer(a[3]));
  const bool renormalize = flag(a[4]);
  const double scale = number(a[5]);
  void* out = c.dense(a[6], "out", c.type, {T, E});
  void* s = c.stream(a[7]);
  return run([&] {
    return mslkb_route_experts_backward(static_cast<const float*>(dw), logits,
                                        static_cast<const int32_t*>(ids), out, T, E, ld, k, score,
                                        renormalize, scale, c.dtype, s);
  });
}

// x, x_scale, ids, num_experts, out, stream
PyObject* moe_dispatch(PyObject* const* a) {
  Call c;
  const at::Tensor& x = c.lead(a[0], "x", true);
  const int64_t T = x.size(0), H = x.size(1), E = integer(a[3]);
  const at::Tensor& chosen = tensor(a[2], "ids");
  Call::matrix(chosen, "ids");
  const int64_t k = chosen.size(1), N = T * k;
  const void* xp = c.dense(a[0], "x", c.type, {T, H});
  const void* ids = c.dense(a[2], "ids", at::kInt, {T, k});
  const Out out(a[4], 4);
  void* xo = c.dense(out[0], "x (out)", c.type, {N, H});
  const bool scaled = a[1] != Py_None;
  PyObject* scale_out = out.if_wanted(1, "x_scale", scaled);
  const void* sp = nullptr;
  void* so = nullptr;
  int64_t cols = 0;
  if (scaled) {
    const at::Tensor& t = tensor(a[1], "x_scale");
    if (t.dim() != 1 && t.dim() != 2)
      raise(PyExc_ValueError,
            "x_scale: expected 1 or 2 dims, got " + std::to_string(t.dim()));
    cols = t.dim() == 2 ? t.size(1) : 1;
    const int64_t in[2] = {T, cols}, to[2] = {N, cols};
    const size_t dims = static_cast<size_t>(t.dim());
    sp = c.dense(a[1], "x_scale", at::kFloat, c10::IntArrayRef(in, dims));
    so = c.dense(scale_out, "x_scale (out)", at::kFloat, c10::IntArrayRef(to, dims));
  }
  void* m_sizes = c.dense(out[2], "m_sizes", at::kLong, {E});
  void* dest = c.dense(out[3], "dest", at::kInt, {T, k});
  const int64_t row_bytes = H * static_cast<int64_t>(x.element_size());
  void* s = c.stream(a[5]);
  return run([&] {
    return mslkb_moe_dispatch(xp, static_cast<const float*>(sp), static_cast<const int32_t*>(ids),
                              xo, static_cast<float*>(so), static_cast<int64_t*>(m_sizes),
                              static_cast<int32_t*>(dest), T, k, E, row_bytes, cols, s);
  });
}

// rows, dest, weights, out, stream
PyObject* moe_combine(PyObject* const* a) {
  Call c;
  const at::Tensor& lead = c.lead(a[0], "rows");
  const int64_t R = lead.size(0), H = lead.size(1);
  const at::Tensor& chosen = tensor(a[1], "dest");
  Call::matrix(chosen, "dest");
  const int64_t T = chosen.size(0), k = chosen.size(1);
  const void* rows = c.dense(a[0], "rows", c.type, {R, H});
  const void* dest = c.dense(a[1], "dest", at::kInt, {T, k});
  const void* weights = c.dense_or_null(a[2], "weights", at::kFloat, {T, k});
  void* out = c.dense(a[3], "out", c.type, {T, H});
  void* s = c.stream(a[4]);
  return run([&] {
    return mslkb_moe_combine(rows, static_cast<const int32_t*>(dest),
                             static_cast<const float*>(weights), out, T, k, H, R, c.dtype, s);
  });
}

// dout, rows, dest, weights, out, stream
PyObject* moe_combine_backward(PyObject* const* a) {
  Call c;
  const at::Tensor& lead = c.lead(a[0], "dout");
  const int64_t T = lead.size(0), H = lead.size(1);
  const at::Tensor& r = tensor(a[1], "rows");
  Call::matrix(r, "rows");
  const at::Tensor& chosen = tensor(a[2], "dest");
  Call::matrix(chosen, "dest");
  const int64_t R = r.size(0), k = chosen.size(1);
  const void* dout = c.dense(a[0], "dout", c.type, {T, H});
  const void* rows = c.dense(a[1], "rows", c.type, {R, H});
  const void* dest = c.dense(a[2], "dest", at::kInt, {T, k});
  const void* weights = c.dense(a[3], "weights", at::kFloat, {T, k});
  const Out out(a[4], 2);
  void* drows = c.dense(out[0], "drows", c.type, {R, H});
  void* dw = c.dense(out[1], "dweights", at::kFloat, {T, k});
  void* s = c.stream(a[5]);
  return run([&] {
    return mslkb_moe_combine_backward(dout, rows, static_cast<const int32_t*>(dest),
                                      static_cast<const float*>(weights), drows,
                                      static_cast<float*>(dw), T, k, H, R, c.dtype, s);
  });
}

// x, groupwise, checkpoint, out, stream
PyObject* swiglu_quant(PyObject* const* a) {
  Call c;
  const at::Tensor& lead = c.lead(a[0], "x");
  const int64_t R = lead.size(0), W = lead.size(1) / 2;
  if (lead.size(1) % 2 != 0)
    raise(PyExc_ValueError, "x holds gate and up side by side: an even number of columns");
  int64_t ldx = 2 * W;
  const void* x = c.rows(a[0], "x", {R, 2 * W}, &ldx);
  const bool groupwise = flag(a[1]), checkpoint = flag(a[2]);
  const Out out(a[3], 4);
  void* q = c.dense(out[0], "q", kE4m3, {R, W});
  void* scale = c.dense(out[1], "scale", at::kFloat, ScaleShape(R, W, groupwise));
  PyObject* so = out.if_wanted(2, "saved", checkpoint);
  PyObject* sso = out.if_wanted(3, "saved_scale", checkpoint);
  void *saved = nullptr, *saved_scale = nullptr;
  if (checkpoint) {
    const ScaleShape blocks(R, W, true);
    saved = c.dense(so, "saved", kE4m3, {R, 2 * W});
    saved_scale = c.dense(sso, "saved_scale", at::kFloat, {R, 2 * blocks.v[1]});
  }
  void* s = c.stream(a[4]);
  return run([&] {
    return mslkb_swiglu_quant(x, q, static_cast<float*>(scale), saved,
                              static_cast<float*>(saved_scale), R, W, ldx, c.dtype, groupwise, s);
  }, W);
}

// dy, saved, saved_scale, out, stream
PyObject* swiglu_quant_backward(PyObject* const* a) {
  Call c;
  const at::Tensor& lead = c.lead(a[0], "dy");
  const int64_t R = lead.size(0), W = lead.size(1);
  const void* dy = c.dense(a[0], "dy", c.type, {R, W});
  const bool kept8 = a[2] != Py_None;
  const void* saved = c.dense(a[1], "saved", kept8 ? kE4m3 : c.type, {R, 2 * W});
  const void* scale = nullptr;
  if (kept8) {
    const ScaleShape blocks(R, W, true);
    scale = c.dense(a[2], "saved_scale", at::kFloat, {R, 2 * blocks.v[1]});
  }
  void* out = c.dense(a[3], "out", c.type, {R, 2 * W});
  void* s = c.stream(a[4]);
  return run([&] {
    return mslkb_swiglu_quant_backward(dy, saved, static_cast<const float*>(scale), out, R, W,
                                       c.dtype, s);
  });
}

// A call of the 16-bit products, led by `o`: bf16 or fp16.
const at::Tensor& lead16(Call& c, PyObject* o, const char* name) {
  const at::Tensor& t = c.lead(o, name);
  if (c.type == at::kFloat)
    raise(PyExc_TypeError, std::string(name) + ": dtype Float is not bfloat16 or float16");
  return t;
}

const at::Tensor& stack_of(PyObject* o, const char* name) {
  const at::Tensor& t = tensor(o, name);
  if (t.dim() != 3)
    raise(PyExc_ValueError,
          std::string(name) + ": expected 3 dims, got " + std::to_string(t.dim()));
  return t;
}

// x, w, m_sizes, transposed, out, stream
PyObject* grouped_mm(PyObject* const* a) {
  Call c;
  const at::Tensor& x = lead16(c, a[0], "x");
  const at::Tensor& w = stack_of(a[1], "w");
  const bool turned = flag(a[3]);
  const int64_t M = x.size(0), K = x.size(1), G = w.size(0), N = w.size(turned ? 2 : 1);
  int64_t ldx = K;
  const void* xp = c.rows(a[0], "x", {M, K}, &ldx);
  const void* wp = turned ? c.dense(a[1], "w", c.type, {G, K, N})
                          : c.dense(a[1], "w", c.type, {G, N, K});
  const void* m_sizes = c.dense(a[2], "m_sizes", at::kLong, {G});
  void* out = c.dense(a[4], "out", c.type, {M, N});
  void* s = c.stream(a[5]);
  const int64_t bytes = mslkb_grouped_mm_workspace_bytes(xp, wp, M, G, N, K, ldx, turned);
  const Scratch workspace(bytes, s);
  return run([&] {
    return mslkb_grouped_mm(xp, wp, static_cast<const int64_t*>(m_sizes), out, M, G, N, K, ldx,
                            turned, c.dtype, workspace.p, bytes, s);
  });
}

// dy, x, m_sizes, add, out, stream
PyObject* grouped_mm_weight_grad(PyObject* const* a) {
  Call c;
  const at::Tensor& dy = lead16(c, a[0], "dy");
  const at::Tensor& x = tensor(a[1], "x");
  Call::matrix(x, "x");
  const at::Tensor& to = stack_of(a[4], "out");
  const int64_t M = dy.size(0), N = dy.size(1), K = x.size(1), G = to.size(0);
  int64_t lddy = N, ldx = K;
  const void* dyp = c.rows(a[0], "dy", {M, N}, &lddy);
  const void* xp = c.rows(a[1], "x", {M, K}, &ldx);
  const void* m_sizes = c.dense(a[2], "m_sizes", at::kLong, {G});
  const bool fp32 = to.scalar_type() == at::kFloat;
  const at::ScalarType type = fp32 ? at::kFloat : c.type;
  const void* add = c.dense_or_null(a[3], "add", type, {G, N, K});
  void* out = c.dense(a[4], "out", type, {G, N, K});
  void* s = c.stream(a[5]);
  const int64_t bytes =
      mslkb_grouped_mm_weight_grad_workspace_bytes(dyp, xp, M, G, N, K, lddy, ldx);
  const Scratch workspace(bytes, s);
  return run([&] {
    return mslkb_grouped_mm_weight_grad(dyp, xp, static_cast<const int64_t*>(m_sizes), add, out, M,
                                        G, N, K, lddy, ldx, c.dtype, fp32, workspace.p, bytes, s);
  });
}

// A list of gradients: addresses, sizes and types, and the device that all are on.
struct Gradients {
  std::vector<const void*> at;
  std::vector<int64_t> sizes;
  std::vector<int32_t> types;
  std::vector<const at::Tensor*> tensors;
  explicit Gradients(PyObject* o) {
    if (!PyList_Check(o) && !PyTuple_Check(o))
      raise(PyExc_TypeError, "grads must be a list or tuple of tensors");
    const Py_ssize_t n = PySequence_Fast_GET_SIZE(o);
    at.reserve(n), sizes.reserve(n), types.reserve(n), tensors.reserve(n);
    const int device = c10::cuda::current_device();
    for (Py_ssize_t i = 0; i < n; ++i) {
      const at::Tensor& t = tensor(PySequence_Fast_GET_ITEM(o, i), "grads");
      const at::ScalarType type = t.scalar_type();
      if (type != at::kBFloat16 && type != at::kHalf && type != at::kFloat)
        raise(PyExc_TypeError, std::string("grads: dtype ") + c10::toString(type) +
                                   " is not bfloat16, float16 or float32");
      if (!t.is_cuda()) raise(PyExc_ValueError, "grads must be CUDA tensors");
      if (t.get_device() != device)
        raise(PyExc_ValueError, "grads: a tensor is on another device than the current one");
      if (!t.is_non_overlapping_and_dense())
        raise(PyExc_ValueError, "grads must be dense");
      at.push_back(t.data_ptr());
      sizes.push_back(t.numel());
      types.push_back(type == at::kFloat ? MSLKB_FP32
                                         : (type == at::kHalf ? MSLKB_FP16 : MSLKB_BF16));
      tensors.push_back(&t);
    }
  }
  int64_t count() const { return static_cast<int64_t>(at.size()); }
};

// The norm's place: an fp32 tensor of one element on the current device.
float* norm_place(PyObject* o) {
  const at::Tensor& t = tensor(o, "norm");
  if (t.scalar_type() != at::kFloat) raise(PyExc_TypeError, "norm: expected float32");
  if (t.numel() != 1) raise(PyExc_ValueError, "norm: expected one element");
  if (!t.is_cuda() || t.get_device() != c10::cuda::current_device())
    raise(PyExc_ValueError, "norm must be a CUDA tensor on the current device");
  return static_cast<float*>(t.data_ptr());
}

// grads, kind, out, stream
PyObject* grad_norm(PyObject* const* a) {
  const Gradients g(a[0]);
  const int32_t kind = static_cast<int32_t>(integer(a[1]));
  float* norm = norm_place(a[2]);
  Call c;
  c.device = c10::cuda::current_device();
  void* s = c.stream(a[3]);
  const int64_t bytes = mslkb_grad_norm_workspace_bytes(g.count());
  const Scratch workspace(bytes, s);
  return run([&] {
    return mslkb_grad_norm(g.at.data(), g.sizes.data(), g.types.data(), g.count(), kind, norm,
                           workspace.p, bytes, s);
  });
}

// grads, kind, max_norm, eps, norm, outs, stream
PyObject* clip_grad_norm(PyObject* const* a) {
  const Gradients g(a[0]);
  const int32_t kind = static_cast<int32_t>(integer(a[1]));
  const double max_norm = number(a[2]), eps = number(a[3]);
  float* norm = norm_place(a[4]);
  PyObject* o = a[5];
  if (!PyList_Check(o) && !PyTuple_Check(o))
    raise(PyExc_TypeError, "out: expected (norm, list of tensors)");
  if (PySequence_Fast_GET_SIZE(o) != g.count())
    raise(PyExc_ValueError, "out: " + std::to_string(g.count()) + " tensors expected, got " +
                                std::to_string(PySequence_Fast_GET_SIZE(o)));
  std::vector<void*> outs;
  outs.reserve(g.at.size());
  for (int64_t i = 0; i < g.count(); ++i) {
    const at::Tensor& t = tensor(PySequence_Fast_GET_ITEM(o, i), "out");
    const at::Tensor& like = *g.tensors[i];
    if (t.scalar_type() != like.scalar_type())
      raise(PyExc_TypeError, std::string("out: dtype ") + c10::toString(t.scalar_type()) +
                                 ", expected " + c10::toString(like.scalar_type()));
    if (t.sizes() != like.sizes() || t.strides() != like.strides())
      raise(PyExc_ValueError, "out: shape " + shape_text(t.sizes()) + ", expected " +
                                  shape_text(like.sizes()) + " with the gradient's strides");
    if (!t.is_cuda() || t.get_device() != like.get_device())
      raise(PyExc_ValueError, "out must be CUDA tensors on the same device");
    outs.push_back(t.data_ptr());
  }
  Call c;
  c.device = c10::cuda::current_device();
  void* s = c.stream(a[6]);
  const int64_t bytes = mslkb_grad_norm_workspace_bytes(g.count());
  const Scratch workspace(bytes, s);
  return run([&] {
    return mslkb_clip_grad_norm(g.at.data(), outs.data(), g.sizes.data(), g.types.data(),
                                g.count(), kind, max_norm, eps, norm, workspace.p, bytes, s);
  });
}

// The number of arguments, and no C++ exception past this point.
template <PyObject* (*kFn)(PyObject* const*), Py_ssize_t kCount>
PyObject* entry(PyObject*, PyObject* const* args, Py_ssize_t count) {
  if (count != kCount) {
    PyErr_Format(PyExc_TypeError, "expected %zd arguments, got %zd", kCount, count);
    return nullptr;
  }
  try {
    return kFn(args);
  } catch (const PythonError&) {
  } catch (const c10::OutOfMemoryError& e) {  // torch.OutOfMemoryError, as from its own calls
    PyObject* torch = PyImport_ImportModule("torch");
    PyObject* type = torch != nullptr ? PyObject_GetAttrString(torch, "OutOfMemoryError") : nullptr;
    if (type != nullptr) PyErr_SetString(type, e.what_without_backtrace());
    Py_XDECREF(type);
    Py_XDECREF(torch);
  } catch (const std::exception& e) {
    PyErr_SetString(PyExc_RuntimeError, e.what());
  } catch (...) {
    PyErr_SetString(PyExc_RuntimeError, "unknown C++ exception");
  }
  return nullptr;
}

#define MSLKB_ENTRY(name, count) \
  {#name, reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(&entry<name, count>)), \
   METH_FASTCALL, nullptr}
PyMethodDef g_methods[] = {MSLKB_ENTRY(add_rms_norm_quant, 9),
                           MSLKB_ENTRY(add_rms_norm_quant_backward, 7),
                           MSLKB_ENTRY(route_experts, 11),
                           MSLKB_ENTRY(route_experts_backward, 8),
                           MSLKB_ENTRY(moe_dispatch, 6),
                           MSLKB_ENTRY(moe_combine, 5),
                           MSLKB_ENTRY(moe_combine_backward, 6),
                           MSLKB_ENTRY(swiglu_quant, 5),
                           MSLKB_ENTRY(swiglu_quant_backward, 5),
                           MSLKB_ENTRY(grouped_mm, 6),
                           MSLKB_ENTRY(grouped_mm_weight_grad, 6),
                           MSLKB_ENTRY(grad_norm, 4),
                           MSLKB_ENTRY(clip_grad_norm, 7),
                           {nullptr, nullptr, 0, nullptr}};

PyModuleDef g_module = {PyModuleDef_HEAD_INIT, "_binding", nullptr, -1, g_methods,
                        nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__binding() { return PyModule_Create(&g_module); }
