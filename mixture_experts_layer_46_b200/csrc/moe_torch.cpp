// The operators around the expert forward as Python functions on torch tensors (module
// _moe_torch): unpacks the tensors, allocates what the caller has not given on the current
// stream of the inputs' device, and calls the C ABI (include/moe.h).  At decoding sizes a call's
// time is its time on the host: one token's two norms took 39 us through ctypes descriptors.
#define PY_SSIZE_T_CLEAN
#include <Python.h>

#include <ATen/core/Tensor.h>
#include <ATen/cuda/EmptyTensor.h>
#include <c10/cuda/CUDAGuard.h>
#include <c10/cuda/CUDAStream.h>
#include <torch/csrc/Dtype.h>
#include <torch/csrc/autograd/python_variable.h>

#include <stdexcept>

#include "moe.h"

namespace {

PyObject* g_check = nullptr;  // (status, name): raises for a status other than MOE_OK

struct Raised {};  // a Python exception is set

[[noreturn]] void value_error(const std::string& what) {
  PyErr_SetString(PyExc_ValueError, what.c_str());
  throw Raised{};
}

const at::Tensor* tensor(PyObject* o, const char* name, bool required = false) {
  if (o == Py_None && !required) return nullptr;
  if (!THPVariable_Check(o)) value_error(std::string(name) + " is not a tensor");
  return &THPVariable_Unpack(o);
}

// a caller's workspace: one block of memory, so that its element count is that of the bytes behind its address
const at::Tensor* scratch(PyObject* o) {
  const at::Tensor* t = tensor(o, "workspace");
  if (t && !t->is_contiguous()) value_error("workspace is not contiguous");
  return t;
}

at::ScalarType dtype_or(PyObject* o, at::ScalarType other) {
  if (o == Py_None) return other;
  if (!THPDtype_Check(o)) value_error("a dtype is not a torch.dtype");
  return reinterpret_cast<THPDtype*>(o)->scalar_type;
}

int32_t code_of(at::ScalarType t) {
  switch (t) {
    case at::kBFloat16: return MOE_BF16;
    case at::kFloat: return MOE_F32;
    case at::kInt: return MOE_I32;
    case at::kLong: return MOE_I64;
    default: return 99;  // rejected by the library
  }
}

struct Desc {
  moe_tensor_t d = {};
  moe_tensor_t* p = nullptr;
  Desc() = default;
  explicit Desc(const at::Tensor* t) {
    if (!t) return;
    fill(*t);
    d.dtype = code_of(t->scalar_type());
  }
  // packed e2m1 codes, two a byte, and their scales of one byte
  Desc(const at::Tensor& codes, const at::Tensor& scale) {
    fill(codes);
    d.dtype = MOE_E2M1X2;
    d.sizes[d.ndim - 1] *= 2;
    d.scale = scale.data_ptr();
    for (int64_t i = 0; i < scale.dim() && i < 4; ++i) d.scale_strides[i] = scale.stride(i);
  }
  void fill(const at::Tensor& t) {
    if (t.dim() > 4) value_error("a tensor of " + std::to_string(t.dim()) + " dimensions");
    d.data = t.data_ptr();
    d.ndim = static_cast<int32_t>(t.dim());
    for (int64_t i = 0; i < t.dim(); ++i) {
      d.sizes[i] = t.size(i);
      d.strides[i] = t.stride(i);
    }
    p = &d;
  }
};

void rows(const at::Tensor& t, const char* name) {
  if (t.dim() != 2) value_error(std::string(name) + " has " + std::to_string(t.dim()) + " dimensions, not 2");
}

// The device and stream of a call: every tensor on the first one's CUDA device, made current.
struct Call {
  c10::Device device;
  c10::cuda::OptionalCUDAGuard guard;
  moe_stream_t stream = nullptr;

  Call(const at::Tensor& first, std::initializer_list<const at::Tensor*> others) : device(first.device()) {
    for (const at::Tensor* t : others)
      if (t && t->device() != device) value_error("tensors on " + device.str() + " and on " + t->device().str());
    if (!device.is_cuda()) value_error("a tensor on " + device.str() + ": the operators run on a CUDA device only");
    guard.set_device(device);
    stream = reinterpret_cast<moe_stream_t>(c10::cuda::getCurrentCUDAStream(device.index()).stream());
  }
  at::Tensor empty(at::IntArrayRef sizes, at::ScalarType t) const {
    return at::detail::empty_cuda(sizes, t, device, std::nullopt);  // (without the dispatcher: half the time)
  }
  at::Tensor given(const at::Tensor* t, at::IntArrayRef sizes, at::ScalarType type) const {
    return t ? *t : empty(sizes, type);
  }
  // the caller's workspace or one of this call's own; keep holds it until the call is enqueued
  void workspace(const at::Tensor* t, size_t need, at::Tensor* keep, void** p, size_t* n) const {
    *keep = t ? *t : empty({static_cast<int64_t>(need > 0 ? need : 1)}, at::kByte);
    *p = keep->data_ptr();
    *n = static_cast<size_t>(keep->numel()) * keep->element_size();
  }
};

void check(moe_status_t s, const char* name) {
  if (s == MOE_OK) return;
  PyObject* r = PyObject_CallFunction(g_check, "is", static_cast<int>(s), name);
  Py_XDECREF(r);
  if (!PyErr_Occurred()) PyErr_SetString(PyExc_RuntimeError, name);
  throw Raised{};
}

float number(PyObject* o) {
  const double v = PyFloat_AsDouble(o);
  if (v == -1.0 && PyErr_Occurred()) throw Raised{};
  return static_cast<float>(v);
}
int32_t integer(PyObject* o) {
  const long v = PyLong_AsLong(o);
  if (v == -1 && PyErr_Occurred()) throw Raised{};
  if (v < INT32_MIN || v > INT32_MAX) value_error("an integer out of range");
  return static_cast<int32_t>(v);
}

bool truth(PyObject* o) {
  const int v = PyObject_IsTrue(o);
  if (v < 0) throw Raised{};
  return v != 0;
}

PyObject* pack(std::initializer_list<const at::Tensor*> ts) {
  PyObject* r = PyTuple_New(static_cast<Py_ssize_t>(ts.size()));
  if (!r) throw Raised{};
  Py_ssize_t i = 0;
  for (const at::Tensor* t : ts) {
    PyObject* o;
    if (t) {
      o = THPVariable_Wrap(*t);
    } else {
      o = Py_None;
      Py_INCREF(o);
    }
    if (!o) {
      Py_DECREF(r);
      throw Raised{};
    }
    PyTuple_SET_ITEM(r, i++, o);
  }
  return r;
}

// No exception leaves a function: each becomes a Python one.
template <PyObject* (*F)(PyObject* const*), int kArgs>
PyObject* entry(PyObject*, PyObject* const* a, Py_ssize_t n) {
  try {
    if (n != kArgs) value_error("wrong number of arguments");
    return F(a);
  } catch (const Raised&) {
  } catch (const std::exception& e) {
    PyErr_SetString(PyExc_RuntimeError, e.what());
  } catch (...) {
    PyErr_SetString(PyExc_RuntimeError, "unknown C++ exception");
  }
  return nullptr;
}

void packed_codes(const at::Tensor& codes) {
  if (codes.scalar_type() != at::kByte && codes.scalar_type() != at::ScalarType::Float4_e2m1fn_x2)
    value_error(std::string("codes of type ") + at::toString(codes.scalar_type()) + ", not uint8 or float4_e2m1fn_x2");
}
bool e8m0_type(at::ScalarType t) { return t == at::kByte || t == at::ScalarType::Float8_e8m0fnu; }
std::string shape_of(const at::Tensor& t) {
  std::string s = "[";
  for (int64_t i = 0; i < t.dim(); ++i) s += (i ? ", " : "") + std::to_string(t.size(i));
  return s + "]";
}

// the scale format of a code matrix, from its scales' type; checks both tensors' sizes
int32_t code_form(const at::Tensor& codes, const at::Tensor& scale) {
  packed_codes(codes);
  if (codes.dim() != 2 || scale.dim() != 2)
    value_error("codes of " + std::to_string(codes.dim()) + " and scales of " + std::to_string(scale.dim()) +
                " dimensions, not 2");
  const bool nv = scale.scalar_type() == at::ScalarType::Float8_e4m3fn;
  if (!nv && !e8m0_type(scale.scalar_type()))
    value_error(std::string("scales of type ") + at::toString(scale.scalar_type()) +
                ": float8_e4m3fn per 16, or uint8 / float8_e8m0fnu per 32");
  const int64_t N = codes.size(0), K = 2 * codes.size(1);
  if (K % 32 != 0 || scale.size(0) != N || scale.size(1) != K / (nv ? 16 : 32))
    value_error("scales of shape " + shape_of(scale) + " for codes of " + std::to_string(N) + " rows of " +
                std::to_string(K) + " elements");
  return nv ? MOE_SCALE_E4M3_16 : MOE_SCALE_E8M0_32;
}

// the experts' codes and their e8m0 scales, one per 32 elements
void expert_scales(const at::Tensor& codes, const at::Tensor& scale) {
  packed_codes(codes);
  if (!e8m0_type(scale.scalar_type()))
    value_error(std::string("expert scales of type ") + at::toString(scale.scalar_type()) + ": uint8 / float8_e8m0fnu per 32");
  if (codes.dim() != 3 || scale.dim() != 3 || scale.size(0) != codes.size(0) || scale.size(1) != codes.size(1) ||
      scale.size(2) * 16 != codes.size(2))
    value_error("expert scales of shape " + shape_of(scale) + " for codes of shape " + shape_of(codes));
}

// x, weight, eps, out, out_dtype, rstd
PyObject* norm_before(PyObject* const* a) {
  const at::Tensor &x = *tensor(a[0], "x", true), *w = tensor(a[1], "weight");
  const float eps = number(a[2]);
  const at::Tensor *o = tensor(a[3], "out"), *rs = tensor(a[5], "rstd");
  rows(x, "x");
  const Call c(x, {w, o, rs});
  const at::Tensor out = c.given(o, x.sizes(), dtype_or(a[4], x.scalar_type()));
  const at::Tensor rstd = c.given(rs, {x.size(0)}, at::kFloat);
  Desc dx(&x), dw(w), dout(&out), dr(&rstd);
  check(moe_norm_before(dx.p, dw.p, eps, dout.p, dr.p, c.stream), "moe_norm_before");
  return pack({&out, &rstd});
}

// y, residual, weight, gate, act, normalize, alpha, eps, out, out_dtype, rstd, next, next_weight, next_out, next_dtype, next_rstd
PyObject* norm_after(PyObject* const* a) {
  const at::Tensor &y = *tensor(a[0], "y", true), *x = tensor(a[1], "residual"), *w = tensor(a[2], "weight"),
                   *g = tensor(a[3], "gate");
  const int32_t act = integer(a[4]), normalize = integer(a[5]);
  const float alpha = number(a[6]), eps = number(a[7]);
  const at::Tensor *o = tensor(a[8], "out"), *rs = tensor(a[10], "rstd"), *wn = tensor(a[12], "next_weight"),
                   *no = tensor(a[13], "next_out"), *nr = tensor(a[15], "next_rstd");
  const bool next = a[11] == Py_None ? (wn || no || nr) : truth(a[11]);
  rows(y, "y");
  const Call c(y, {x, w, g, o, rs, wn, no, nr});
  const at::Tensor out = c.given(o, y.sizes(), dtype_or(a[9], (x ? x : &y)->scalar_type()));
  const at::Tensor rstd = c.given(rs, {y.size(0)}, at::kFloat);
  at::Tensor nout, nrstd;
  if (next || no) nout = c.given(no, y.sizes(), dtype_or(a[14], out.scalar_type()));
  if (next || nr) nrstd = c.given(nr, {y.size(0)}, at::kFloat);
  Desc dy(&y), dx(x), dw(w), dg(g), dout(&out), dr(&rstd), dwn(wn), dno(nout.defined() ? &nout : nullptr),
      dnr(nrstd.defined() ? &nrstd : nullptr);
  check(moe_norm_after(dy.p, dx.p, dw.p, dg.p, act, normalize, alpha, eps, dout.p, dr.p, dwn.p, dno.p, dnr.p, c.stream),
        "moe_norm_after");
  return next ? pack({&out, &rstd, &nout, &nrstd}) : pack({&out, &rstd});
}

// dout, x, rstd, weight, residual_grad, alpha, dx, dweight, weight_grad, grad_dtype, workspace
PyObject* norm_before_backward(PyObject* const* a) {
  const at::Tensor &d = *tensor(a[0], "dout", true), &x = *tensor(a[1], "x", true), &r = *tensor(a[2], "rstd", true);
  const at::Tensor *w = tensor(a[3], "weight"), *res = tensor(a[4], "residual_grad");
  const float alpha = number(a[5]);
  const at::Tensor *dxt = tensor(a[6], "dx"), *dwt = tensor(a[7], "dweight"), *wst = scratch(a[10]);
  const bool want = dwt || (w && truth(a[8]));
  rows(d, "dout");
  const Call c(d, {&x, &r, w, res, dxt, dwt, wst});
  const at::Tensor dx = c.given(dxt, d.sizes(), x.scalar_type());
  at::Tensor dw, keep;
  void* ws = nullptr;
  size_t n = 0;
  if (want) {
    dw = c.given(dwt, {d.size(1)}, dtype_or(a[9], at::kFloat));
    c.workspace(wst, moe_norm_backward_workspace_bytes(d.size(0), d.size(1)), &keep, &ws, &n);
  }
  Desc dd(&d), dxi(&x), dr(&r), dwt_(w), dres(res), ddx(&dx), ddw(want ? &dw : nullptr);
  check(moe_norm_before_backward(dd.p, dxi.p, dr.p, dwt_.p, dres.p, alpha, ddx.p, ddw.p, ws, n, c.stream),
        "moe_norm_before_backward");
  return pack({&dx, want ? &dw : nullptr});
}

// dout, y, rstd, weight, gate, act, normalize, dy, dweight, dgate, weight_grad, gate_grad, grad_dtype, workspace
PyObject* norm_after_backward(PyObject* const* a) {
  const at::Tensor &d = *tensor(a[0], "dout", true), &y = *tensor(a[1], "y", true);
  const at::Tensor *r = tensor(a[2], "rstd"), *w = tensor(a[3], "weight"), *g = tensor(a[4], "gate");
  const int32_t act = integer(a[5]), normalize = integer(a[6]);
  const at::Tensor *dyt = tensor(a[7], "dy"), *dwt = tensor(a[8], "dweight"), *dgt = tensor(a[9], "dgate"),
                   *wst = scratch(a[13]);
  const bool want_w = dwt || (w && truth(a[10])), want_g = dgt || (g && truth(a[11]));
  rows(d, "dout");
  const Call c(d, {&y, r, w, g, dyt, dwt, dgt, wst});
  const at::ScalarType type = dtype_or(a[12], at::kFloat);
  const at::Tensor dy = c.given(dyt, d.sizes(), y.scalar_type());
  at::Tensor dw, dg, keep;
  void* ws = nullptr;
  size_t n = 0;
  if (want_w) dw = c.given(dwt, {d.size(1)}, type);
  if (want_g) dg = dgt ? *dgt : c.empty(g->sizes(), type);
  if (want_w || want_g) c.workspace(wst, moe_norm_backward_workspace_bytes(d.size(0), d.size(1)), &keep, &ws, &n);
  Desc dd(&d), dyi(&y), dr(r), dwi(w), dgi(g), ddy(&dy), ddw(want_w ? &dw : nullptr), ddg(want_g ? &dg : nullptr);
  check(moe_norm_after_backward(dd.p, dyi.p, dr.p, dwi.p, dgi.p, act, normalize, ddy.p, ddw.p, ddg.p, ws, n, c.stream),
        "moe_norm_after_backward");
  return pack({&dy, want_w ? &dw : nullptr, want_g ? &dg : nullptr});
}

// x, router, w13 (address of a moe_w13_t), w2, w2_scale, k, pre_weight, eps, renormalize, shared, post_norm, post_weight,
// gate, act, alpha, out, topk_ids, topk_weights, workspace
PyObject* layer_decode(PyObject* const* a) {
  const at::Tensor &x = *tensor(a[0], "x", true), &router = *tensor(a[1], "router", true), &w2 = *tensor(a[3], "w2", true);
  const moe_w13_t* w13 = static_cast<const moe_w13_t*>(PyLong_AsVoidPtr(a[2]));
  if (!w13 && PyErr_Occurred()) throw Raised{};
  const at::Tensor *s2 = tensor(a[4], "w2_scale"), *pre = tensor(a[6], "pre_weight"), *post = tensor(a[11], "post_weight"),
                   *gate = tensor(a[12], "gate"), *ot = tensor(a[15], "out"), *it = tensor(a[16], "topk_ids"),
                   *wt = tensor(a[17], "topk_weights"), *wst = scratch(a[18]);
  const int32_t k = integer(a[5]), renorm = integer(a[8]), shared = integer(a[9]), post_norm = integer(a[10]),
                act = integer(a[13]);
  const float eps = number(a[7]), alpha = number(a[14]);
  rows(x, "x");
  rows(router, "router");
  if (s2) expert_scales(w2, *s2);
  if (k < 1 || k > 32) value_error("k " + std::to_string(k) + ": 1 to 32");
  const Call c(x, {&router, &w2, s2, pre, post, gate, ot, it, wt, wst});
  const int64_t T = x.size(0), H = x.size(1), kk = k + shared;
  const at::Tensor out = c.given(ot, x.sizes(), at::kBFloat16);
  const at::Tensor ids = c.given(it, {T, kk}, at::kInt), wts = c.given(wt, {T, kk}, at::kFloat);
  at::Tensor keep;
  void* ws = nullptr;
  size_t n = 0;
  c.workspace(wst, moe_layer_decode_workspace_bytes(T, H, w13->gate.sizes[1], router.size(0) + shared, kk,
                                                    s2 ? MOE_E2M1X2 : MOE_BF16), &keep, &ws, &n);
  Desc dx(&x), dpre(pre), drouter(&router), d2 = s2 ? Desc(w2, *s2) : Desc(&w2), dpost(post), dgate(gate), dids(&ids),
      dwts(&wts), dout(&out);
  d2.p = &d2.d;
  check(moe_layer_decode(dx.p, dpre.p, eps, drouter.p, k, renorm, shared, w13, d2.p, post_norm, dpost.p, dgate.p, act,
                         alpha, dids.p, dwts.p, dout.p, ws, n, c.stream), "moe_layer_decode");
  return pack({&out, &ids, &wts});
}

// x, weight, weight_scale, x_global, w_global, out, workspace
PyObject* linear_fp4(PyObject* const* a) {
  const at::Tensor &x = *tensor(a[0], "x", true), &w = *tensor(a[1], "weight", true), &s = *tensor(a[2], "weight_scale", true);
  const at::Tensor *xg = tensor(a[3], "x_global"), *wg = tensor(a[4], "w_global"), *ot = tensor(a[5], "out"),
                   *wst = scratch(a[6]);
  rows(x, "x");
  const int32_t form = code_form(w, s);
  const Call c(x, {&w, &s, xg, wg, ot, wst});
  const int64_t N = w.size(0);
  const at::Tensor out = c.given(ot, {x.size(0), N}, at::kBFloat16);
  at::Tensor keep;
  void* ws = nullptr;
  size_t n = 0;
  c.workspace(wst, moe_linear_fp4_workspace_bytes(x.size(0), N, x.size(1), form), &keep, &ws, &n);
  Desc dx(&x), dw(w, s), dxg(xg), dwg(wg), dout(&out);
  check(moe_linear_fp4(dx.p, dw.p, form, dxg.p, dwg.p, dout.p, ws, n, c.stream), "moe_linear_fp4");
  return THPVariable_Wrap(out);
}

// src, global_scale
PyObject* quantize_nvfp4(PyObject* const* a) {
  const at::Tensor &x = *tensor(a[0], "src", true), &g = *tensor(a[1], "global_scale", true);
  rows(x, "src");
  const Call c(x, {&g});
  const at::Tensor codes = c.empty({x.size(0), x.size(1) / 2}, at::kByte);
  const at::Tensor scale = c.empty({x.size(0), x.size(1) / 16}, at::ScalarType::Float8_e4m3fn);
  Desc dx(&x), dg(&g), dc(codes, scale);
  check(moe_quantize_nvfp4(dx.p, dg.p, dc.p, c.stream), "moe_quantize_nvfp4");
  return pack({&codes, &scale});
}

PyObject* set_check(PyObject*, PyObject* f) {
  Py_INCREF(f);
  Py_XDECREF(g_check);
  g_check = f;
  Py_RETURN_NONE;
}

#define MOE_METHOD(name, args) \
  {#name, reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(&entry<name, args>)), METH_FASTCALL, nullptr}
PyMethodDef methods[] = {MOE_METHOD(norm_before, 6),
                         MOE_METHOD(norm_after, 16),
                         MOE_METHOD(norm_before_backward, 11),
                         MOE_METHOD(norm_after_backward, 14),
                         MOE_METHOD(layer_decode, 19),
                         MOE_METHOD(linear_fp4, 7),
                         MOE_METHOD(quantize_nvfp4, 2),
                         {"set_check", set_check, METH_O, nullptr},
                         {nullptr, nullptr, 0, nullptr}};
PyModuleDef module = {PyModuleDef_HEAD_INIT, "_moe_torch", nullptr, -1, methods, nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__moe_torch() { return PyModule_Create(&module); }
