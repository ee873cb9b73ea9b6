// Python marshalling of the operators around the expert products: checks of
// the tensors, allocation of what the caller did not bring, and the call of
// the C ABI on PyTorch's current stream.  These calls are small (a router's or
// a norm's kernel runs for a few microseconds), and the same steps taken in
// Python cost more than the kernels: one token through the norm 15 us against
// 7, through the router 22 us against 9.  No arithmetic here.
//
// Every function takes its arguments by position and returns its result, or
// the status code (an int) with which the call was refused.
#include <Python.h>

#include <ATen/ATen.h>
#include <ATen/cuda/EmptyTensor.h>
#include <c10/cuda/CUDAFunctions.h>
#include <c10/cuda/CUDAStream.h>
#include <cuda_runtime_api.h>
#include <torch/csrc/Exceptions.h>
#include <torch/csrc/autograd/python_variable.h>

#include "../../include/fp8moe.h"

namespace {

using at::Tensor;
using Shape = at::IntArrayRef;

// A refused argument (fp8moe_status) or a Python error already set.
struct Refused {
  int code;
};
struct PyError {};

[[noreturn]] void refuse() { throw Refused{FP8MOE_ERR_INVALID_ARG}; }
void check(fp8moe_status s) {
  if (s != FP8MOE_OK) throw Refused{s};
}

const Tensor& tensor(PyObject* o) {
  if (!THPVariable_Check(o)) {
    PyErr_Format(PyExc_TypeError, "expected a tensor, got %s", Py_TYPE(o)->tp_name);
    throw PyError{};
  }
  return THPVariable_Unpack(o);
}
const Tensor* maybe(PyObject* o) { return o == Py_None ? nullptr : &tensor(o); }
int64_t integer(PyObject* o) {
  const long long v = PyLong_AsLongLong(o);
  if (v == -1 && PyErr_Occurred()) throw PyError{};
  return v;
}
int small(PyObject* o) {   // an enumerator; what no enumerator is stays invalid
  const int64_t v = integer(o);
  return v < -1000 || v > 1000 ? 1000 : (int)v;
}
float real(PyObject* o) {
  const double v = PyFloat_AsDouble(o);
  if (v == -1.0 && PyErr_Occurred()) throw PyError{};
  return (float)v;
}
bool flag(PyObject* o) {
  const int v = PyObject_IsTrue(o);
  if (v < 0) throw PyError{};
  return v != 0;
}

// The call's device: that of its first argument, which has to be current.
struct Call {
  int dev;
  Tensor shared;      // see together()
  int64_t used = 0;
  explicit Call(const Tensor& t) {
    if (!t.is_cuda()) refuse();
    dev = t.get_device();
    if (dev != c10::cuda::current_device()) refuse();
  }
  fp8moe_stream_t stream() const { return (fp8moe_stream_t)c10::cuda::getCurrentCUDAStream(dev).stream(); }
  // Small results that a call makes together share one allocation (0.9 us of
  // host time each, a view of it 0.3): give their bytes first, 0 for one that the
  // caller brings or does not want; empty() then takes them from it in any order.
  // Large ones stay apart, as each holds the memory of all.
  static constexpr int64_t TOGETHER = 256 << 10;
  static int64_t padded(int64_t bytes) { return (bytes + 255) / 256 * 256; }
  void together(std::initializer_list<int64_t> bytes) {
    int64_t sum = 0, n = 0;
    for (int64_t b : bytes) {
      if (b < 0 || b > TOGETHER) return;
      sum += padded(b);
      n += b > 0;
    }
    if (n < 2 || sum > TOGETHER) return;
    shared = at::detail::empty_cuda({sum}, at::kByte, at::Device(at::kCUDA, (c10::DeviceIndex)dev), std::nullopt);
  }
  Tensor empty(Shape s, at::ScalarType t) {
    int64_t n = 1;
    for (int64_t d : s) {
      if (d < 0) refuse();
      n *= d;
    }
    const caffe2::TypeMeta meta = c10::scalarTypeToTypeMeta(t);
    const int64_t bytes = n * (int64_t)meta.itemsize();
    if (shared.defined() && bytes > 0 && used + bytes <= shared.numel()) {
      Tensor p = at::detail::make_tensor<c10::TensorImpl>(c10::Storage(shared.storage()), shared.key_set(), meta);
      p.unsafeGetTensorImpl()->set_storage_offset(used / (int64_t)meta.itemsize());
      p.unsafeGetTensorImpl()->set_sizes_contiguous(s);
      used += padded(bytes);
      return p;
    }
    // (at::empty without its dispatch)
    return at::detail::empty_cuda(s, t, at::Device(at::kCUDA, (c10::DeviceIndex)dev), std::nullopt);
  }
  // bytes, zeroed on the call's stream (at::zeros: 10.5 us of host time against
  // 3.3; where padding is written by nobody and has to be valid)
  Tensor zeros(int64_t n) {
    Tensor t = empty({n}, at::kByte);
    if (n > 0 && cudaMemsetAsync(t.data_ptr(), 0, (size_t)n, (cudaStream_t)stream()) != cudaSuccess) throw Refused{FP8MOE_ERR_CUDA};
    return t;
  }
  bool here(const Tensor& t, at::ScalarType ty, Shape s) const {
    return t.is_cuda() && t.get_device() == dev && t.scalar_type() == ty && t.sizes() == s;
  }
  // address of a contiguous tensor of this type and shape
  void* dense(const Tensor& t, at::ScalarType ty, Shape s) const {
    if (!here(t, ty, s) || !t.is_contiguous()) refuse();
    return t.data_ptr();
  }
  void* dense(const Tensor* t, at::ScalarType ty, Shape s) const { return t ? dense(*t, ty, s) : nullptr; }
  // address and row stride of a [R, C] tensor whose rows are dense
  void* rows(const Tensor& t, at::ScalarType ty, Shape s, int64_t& ld) const {
    if (!here(t, ty, s) || (s[1] > 1 && t.stride(1) != 1)) refuse();
    ld = s[0] > 1 ? t.stride(0) : s[1];
    return t.data_ptr();
  }
  // the given tensor or a new one, checked; its address
  void* out(Tensor& o, PyObject* given, at::ScalarType ty, Shape s) {
    if (given == Py_None) {
      o = empty(s, ty);
      return o.data_ptr();
    }
    o = tensor(given);
    return dense(o, ty, s);
  }
  // a workspace of nbytes: the given one (any type) or a new one
  void* workspace(Tensor& o, PyObject* given, int64_t& nbytes) {
    if (given == Py_None) {
      o = empty({nbytes < 0 ? 0 : nbytes}, at::kByte);
    } else {
      o = tensor(given);
      if (!o.is_cuda() || o.get_device() != dev || !o.is_contiguous()) refuse();
      nbytes = o.nbytes();
    }
    return o.data_ptr();
  }
};

// float32 or bfloat16
at::ScalarType real_type(const Tensor& t) {
  const at::ScalarType ty = t.scalar_type();
  if (ty != at::kFloat && ty != at::kBFloat16) refuse();
  return ty;
}
int type_code(at::ScalarType t) { return t == at::kFloat ? FP8MOE_FP32 : FP8MOE_BF16; }

PyObject* none() { Py_RETURN_NONE; }
PyObject* give(Tensor& t) { return t.defined() ? THPVariable_Wrap(std::move(t)) : none(); }
template <typename... T>
PyObject* give_all(T&... t) {
  PyObject* r = PyTuple_New(sizeof...(t));
  if (!r) throw PyError{};
  Py_ssize_t i = 0;
  ((PyTuple_SET_ITEM(r, i++, give(t))), ...);
  return r;
}

// x, weight, residual, eps, recipe, kind, scale_layout, need_y, need_rstd, h, y, rstd, q, scale
PyObject* add_rmsnorm_fwd(PyObject* const* a) {
  const Tensor &x = tensor(a[0]), &w = tensor(a[1]);
  const Tensor* r = maybe(a[2]);
  if (x.dim() != 2) refuse();
  const int64_t T = x.size(0), H = x.size(1);
  Call c(x);
  int64_t ldx = 0, ldr = 0;
  const void* px = c.rows(x, at::kBFloat16, {T, H}, ldx);
  const at::ScalarType wt = real_type(w);
  const void* pw = c.dense(w, wt, {H});
  const void* pr = r ? c.rows(*r, at::kBFloat16, {T, H}, ldr) : nullptr;
  Tensor h, y, rstd, q, scale;
  const bool mx = a[4] != Py_None;
  c.together({r && a[9] == Py_None ? T * H * 2 : 0, flag(a[7]) && a[10] == Py_None ? T * H * 2 : 0,
              flag(a[8]) && a[11] == Py_None ? T * 4 : 0, mx && a[12] == Py_None ? T * H : 0});
  void *ph = nullptr, *py = nullptr, *ps = nullptr, *pq = nullptr, *pscale = nullptr;
  if (r) {
    ph = c.out(h, a[9], at::kBFloat16, {T, H});
  } else if (a[9] != Py_None) {
    refuse();
  }
  if (flag(a[7])) py = c.out(y, a[10], at::kBFloat16, {T, H});
  if (flag(a[8])) ps = c.out(rstd, a[11], at::kFloat, {T});
  int recipe = FP8MOE_ROWWISE;
  const int layout = small(a[6]);
  if (a[4] != Py_None) {
    recipe = small(a[4]);
    pq = c.out(q, a[12], at::kByte, {T, H});
    if (recipe != FP8MOE_MXFP8) {
      pscale = c.out(scale, a[13], at::kFloat, {T});
    } else if (layout == FP8MOE_SCALES_ROWMAJOR) {
      pscale = c.out(scale, a[13], at::kByte, {T, H / 32});
    } else {
      const int64_t need = fp8moe_swizzled_scales_bytes(1, T, H / 32, 0, FP8MOE_NO_GROUPS);
      if (a[13] == Py_None) {
        // room for the tiles of one group, whose layout is the same: the A
        // operand of a one-group grouped GEMM
        scale = c.zeros(fp8moe_swizzled_scales_bytes(1, T, H / 32, 1, FP8MOE_GROUP_ROWS));
      } else {
        scale = tensor(a[13]);
      }
      if (scale.numel() < need) refuse();
      pscale = c.dense(scale, at::kByte, {scale.numel()});
    }
  }
  check(fp8moe_add_rmsnorm_fwd(px, ldx, pr, ldr, pw, type_code(wt), T, H, real(a[3]), ph, py, (float*)ps, recipe,
                               small(a[5]), pq, pscale, layout, c.stream()));
  return give_all(h, y, rstd, q, scale);
}

// dy, h, rstd, weight, dh, dx, dweight, workspace
PyObject* add_rmsnorm_bwd(PyObject* const* a) {
  const Tensor& dy = tensor(a[0]);
  if (dy.dim() != 2) refuse();
  const int64_t T = dy.size(0), H = dy.size(1);
  Call c(dy);
  const void* pdy = c.dense(dy, at::kBFloat16, {T, H});
  const void* ph = c.dense(tensor(a[1]), at::kBFloat16, {T, H});
  const void* prstd = c.dense(tensor(a[2]), at::kFloat, {T});
  const Tensor& w = tensor(a[3]);
  const at::ScalarType wt = real_type(w);
  const void* pw = c.dense(w, wt, {H});
  const void* pdh = c.dense(maybe(a[4]), at::kBFloat16, {T, H});
  Tensor dx, dw, ws;
  c.together({a[5] == Py_None ? T * H * 2 : 0, a[6] == Py_None ? H * 4 : 0});
  void* pdx = c.out(dx, a[5], at::kBFloat16, {T, H});
  void* pdw = c.out(dw, a[6], at::kFloat, {H});
  int64_t nbytes = fp8moe_add_rmsnorm_bwd_workspace_bytes(T, H);
  void* pws = c.workspace(ws, a[7], nbytes);
  check(fp8moe_add_rmsnorm_bwd(pdy, ph, (const float*)prstd, pw, type_code(wt), pdh, T, H, pdx, (float*)pdw, pws, nbytes,
                               c.stream()));
  return give_all(dx, dw);
}

const uint8_t* token_mask(const Call& c, const Tensor* m, int64_t T) {
  if (!m) return nullptr;
  const at::ScalarType t = m->scalar_type();
  if (t != at::kByte && t != at::kBool) refuse();
  return (const uint8_t*)c.dense(*m, t, {T});
}

// logits, k, score, renormalize, route_scale, bias, token_mask, need_balance, topk_idx, topk_w, counts, prob_sum,
// balance_loss, workspace
PyObject* router_fwd(PyObject* const* a) {
  const Tensor& x = tensor(a[0]);
  if (x.dim() != 2) refuse();
  const int64_t T = x.size(0), E = x.size(1), k = integer(a[1]);
  if (k < 1 || k > E) refuse();
  const at::ScalarType xt = real_type(x);
  Call c(x);
  int64_t ld = 0, nbytes = 0;
  const void* px = c.rows(x, xt, {T, E}, ld);
  const void* pb = c.dense(maybe(a[5]), at::kFloat, {E});
  const uint8_t* pm = token_mask(c, maybe(a[6]), T);
  Tensor idx, w, counts, psum, loss, ws;
  const bool sums = flag(a[7]);
  c.together({a[8] == Py_None ? T * k * 4 : 0, a[9] == Py_None ? T * k * 4 : 0, sums && a[10] == Py_None ? (E + 1) * 4 : 0,
              sums && a[11] == Py_None ? E * 4 : 0, sums && a[12] == Py_None ? 4 : 0});
  void* pi = c.out(idx, a[8], at::kInt, {T, k});
  void* pw = c.out(w, a[9], at::kFloat, {T, k});
  void *pc = nullptr, *pp = nullptr, *pl = nullptr, *pws = nullptr;
  if (sums) {
    pc = c.out(counts, a[10], at::kInt, {E + 1});
    pp = c.out(psum, a[11], at::kFloat, {E});
    pl = c.out(loss, a[12], at::kFloat, {1});
    nbytes = fp8moe_router_workspace_bytes(T, E);
    if (nbytes > 0) pws = c.workspace(ws, a[13], nbytes);
  }
  check(fp8moe_router_fwd(px, type_code(xt), T, E, ld, k, small(a[2]), flag(a[3]), real(a[4]), (const float*)pb, pm,
                          (int32_t*)pi, (float*)pw, (int32_t*)pc, (float*)pp, (float*)pl, pws, nbytes, c.stream()));
  return give_all(idx, w, counts, psum, loss);
}

// logits, topk_idx, counts, dtopk_w, dloss, score, renormalize, route_scale, token_mask, dlogits
PyObject* router_bwd(PyObject* const* a) {
  const Tensor &x = tensor(a[0]), &idx = tensor(a[1]);
  if (x.dim() != 2 || idx.dim() != 2) refuse();
  const int64_t T = x.size(0), E = x.size(1), k = idx.size(1);
  const at::ScalarType xt = real_type(x);
  Call c(x);
  int64_t ld = 0;
  const void* px = c.rows(x, xt, {T, E}, ld);
  const void* pi = c.dense(idx, at::kInt, {T, k});
  const void* pc = c.dense(maybe(a[2]), at::kInt, {E + 1});
  const void* pw = c.dense(maybe(a[3]), at::kFloat, {T, k});
  const void* pl = c.dense(maybe(a[4]), at::kFloat, {1});
  const uint8_t* pm = token_mask(c, maybe(a[8]), T);
  Tensor d;
  void* pd = c.out(d, a[9], xt, {T, E});
  check(fp8moe_router_bwd(px, type_code(xt), T, E, ld, k, small(a[5]), flag(a[6]), real(a[7]), pm, (const int32_t*)pi,
                          (const int32_t*)pc, (const float*)pw, (const float*)pl, pd, c.stream()));
  return give(d);
}

// dout, y, row_of, dw
PyObject* route_weight_grad(PyObject* const* a) {
  const Tensor &dout = tensor(a[0]), &y = tensor(a[1]), &row_of = tensor(a[2]);
  if (dout.dim() != 2 || y.dim() != 2 || row_of.dim() != 2) refuse();
  const int64_t T = dout.size(0), N = dout.size(1), k = row_of.size(1);
  Call c(dout);
  const void* pd = c.dense(dout, at::kBFloat16, {T, N});
  const void* py = c.dense(y, at::kBFloat16, {y.size(0), N});
  const void* pr = c.dense(row_of, at::kInt, {T, k});
  Tensor dw;
  void* pw = c.out(dw, a[3], at::kFloat, {T, k});
  check(fp8moe_route_weight_grad_bounded(pd, py, y.size(0), (const int32_t*)pr, T, N, k, (float*)pw, c.stream()));
  return give(dw);
}

// MXFP8 codes [R, C] and their scales; E: groups of a grouped layout
void mx_out(Call& c, Tensor& q, PyObject* gq, Tensor& s, PyObject* gs, int layout, int64_t R, int64_t C, int64_t E,
            void*& pq, uint8_t*& ps) {
  const bool plain = layout == FP8MOE_SCALES_ROWMAJOR;
  const int64_t need = plain ? R * (C / 32) : fp8moe_swizzled_scales_bytes(1, R, C / 32, E, layout);
  if (need < 0) refuse();
  pq = c.out(q, gq, at::kByte, {R, C});
  if (gs == Py_None) {
    s = plain ? c.empty({R, C / 32}, at::kByte) : c.zeros(need);
  } else {
    s = tensor(gs);
    if (s.numel() < need) refuse();
  }
  ps = (uint8_t*)c.dense(s, at::kByte, s.sizes());
}

// dout (None: forward), h, offs, s0_layout, s1_layout, need_out, dim0, dim1, out, q0, s0, q1, s1
PyObject* swiglu(PyObject* const* a) {
  const Tensor* dout = maybe(a[0]);
  const Tensor& h = tensor(a[1]);
  const Tensor* offs = maybe(a[2]);
  if (h.dim() != 2 || h.size(1) % 2) refuse();
  const int64_t M = h.size(0), F = h.size(1) / 2, W = dout ? 2 * F : F;
  Call c(h);
  int64_t ldh = 0;
  const void* ph = c.rows(h, at::kBFloat16, {M, 2 * F}, ldh);
  const void* pd = c.dense(dout, at::kBFloat16, {M, F});
  const int64_t E = offs ? offs->numel() : 0;
  const void* po = c.dense(offs, at::kInt, {E});
  const int l0 = small(a[3]), l1 = small(a[4]);
  Tensor out, q0, s0, q1, s1;
  void *pout = nullptr, *p0 = nullptr, *p1 = nullptr;
  uint8_t *ps0 = nullptr, *ps1 = nullptr;
  const bool o = flag(a[5]), d0 = flag(a[6]), d1 = flag(a[7]);
  c.together({o && a[8] == Py_None ? M * W * 2 : 0, d0 && a[9] == Py_None ? M * W : 0, d1 && a[11] == Py_None ? M * W : 0});
  if (o) pout = c.out(out, a[8], at::kBFloat16, {M, W});
  if (d0) mx_out(c, q0, a[9], s0, a[10], l0, M, W, E, p0, ps0);
  if (d1) mx_out(c, q1, a[11], s1, a[12], l1, W, M, E, p1, ps1);
  if (dout) {
    check(fp8moe_swiglu_bwd(pd, ph, ldh, M, F, (const int32_t*)po, E, pout, p0, ps0, l0, p1, ps1, l1, c.stream()));
  } else {
    check(fp8moe_swiglu_fwd(ph, ldh, M, F, (const int32_t*)po, E, pout, p0, ps0, l0, p1, ps1, l1, c.stream()));
  }
  return give_all(out, q0, s0, q1, s1);
}

// The Python entry of F with N positional arguments; no C++ exception leaves it.
template <PyObject* (*F)(PyObject* const*), Py_ssize_t N>
PyObject* entry(PyObject*, PyObject* const* args, Py_ssize_t n) {
  HANDLE_TH_ERRORS
  if (n != N) {
    PyErr_Format(PyExc_TypeError, "expected %zd arguments, got %zd", N, n);
    return nullptr;
  }
  try {
    return F(args);
  } catch (const Refused& r) {
    return PyLong_FromLong(r.code);
  } catch (const PyError&) {
    return nullptr;
  }
  END_HANDLE_TH_ERRORS
}

#define FP8MOE_ENTRY(NAME, N) \
  {#NAME, (PyCFunction)(void (*)(void))entry<NAME, N>, METH_FASTCALL, nullptr}
PyMethodDef methods[] = {FP8MOE_ENTRY(add_rmsnorm_fwd, 14),   FP8MOE_ENTRY(add_rmsnorm_bwd, 8),
                         FP8MOE_ENTRY(router_fwd, 14),        FP8MOE_ENTRY(router_bwd, 10),
                         FP8MOE_ENTRY(route_weight_grad, 4),  FP8MOE_ENTRY(swiglu, 13),
                         {nullptr, nullptr, 0, nullptr}};
PyModuleDef module = {PyModuleDef_HEAD_INIT, "_binding", nullptr, -1, methods, nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__binding(void) { return PyModule_Create(&module); }
