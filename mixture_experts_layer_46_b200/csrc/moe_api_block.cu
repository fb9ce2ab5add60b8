// Entry points of the operators around the expert forward (include/moe.h): argument
// checks, views and launches.  Every error is found before anything is launched.
#include <cmath>

#include "../../include/moe.h"
#include "moe_block.h"
#include "moe_internal.h"

namespace moe {
namespace {

int64_t float_size(int32_t dt) { return dt == MOE_BF16 ? 2 : dt == MOE_F32 ? 4 : 0; }

// A float row tensor [T, H]: MOE_OK and its view, or what is wrong with it.
moe_status_t rows_of(const moe_tensor_t* t, int64_t T, int64_t H, bool output, RowView* v) {
  if (t->ndim != 2) return MOE_ERR_INVALID_ARG;
  if (float_size(t->dtype) == 0) return MOE_ERR_UNSUPPORTED_DTYPE;
  if (t->sizes[0] != T || t->sizes[1] != H) return MOE_ERR_SHAPE_MISMATCH;
  if (T > 0 && H > 0 && !t->data) return MOE_ERR_INVALID_ARG;
  // rows or columns on top of one another cannot be written
  if (output && ((T > 1 && t->strides[0] == 0) || (H > 1 && t->strides[1] == 0)))
    return MOE_ERR_UNSUPPORTED_LAYOUT;
  v->data = t->data;
  v->s0 = t->strides[0];
  v->s1 = t->strides[1];
  v->dtype = t->dtype;
  return MOE_OK;
}

// A weight vector [H] (null: ones).
moe_status_t vector_of(const moe_tensor_t* t, int64_t n, bool output, RowView* v) {
  *v = RowView();
  if (!t) return MOE_OK;
  if (t->ndim != 1 || !t->data) return MOE_ERR_INVALID_ARG;
  if (float_size(t->dtype) == 0) return MOE_ERR_UNSUPPORTED_DTYPE;
  if (t->sizes[0] != n) return MOE_ERR_SHAPE_MISMATCH;
  if (output && n > 1 && t->strides[0] == 0) return MOE_ERR_UNSUPPORTED_LAYOUT;
  v->data = t->data;
  v->s1 = t->strides[0];
  v->dtype = t->dtype;
  return MOE_OK;
}

// A [T] f32 vector (null allowed unless required).
moe_status_t rstd_of(const moe_tensor_t* t, int64_t T, bool output, float** p, int64_t* s) {
  *p = nullptr;
  *s = 0;
  if (!t) return MOE_OK;
  if (t->ndim != 1) return MOE_ERR_INVALID_ARG;
  if (t->dtype != MOE_F32) return MOE_ERR_UNSUPPORTED_DTYPE;
  if (t->sizes[0] != T) return MOE_ERR_SHAPE_MISMATCH;
  if (T > 0 && !t->data) return MOE_ERR_INVALID_ARG;
  if (output && T > 1 && t->strides[0] == 0) return MOE_ERR_UNSUPPORTED_LAYOUT;
  *p = static_cast<float*>(t->data);
  *s = t->strides[0];
  return MOE_OK;
}

// A gate broadcast over its axes of size 1 (null: none).
moe_status_t gate_of(const moe_tensor_t* t, int64_t T, int64_t H, int32_t act, RowView* v, int* mode) {
  *v = RowView();
  *mode = kGateNone;
  if (act != MOE_GATE_NONE && act != MOE_GATE_SIGMOID && act != MOE_GATE_TANH) return MOE_ERR_INVALID_ARG;
  if (!t) return MOE_OK;
  if (t->ndim != 2) return MOE_ERR_INVALID_ARG;
  if (float_size(t->dtype) == 0) return MOE_ERR_UNSUPPORTED_DTYPE;
  if ((t->sizes[0] != T && t->sizes[0] != 1) || (t->sizes[1] != H && t->sizes[1] != 1))
    return MOE_ERR_SHAPE_MISMATCH;
  if (t->sizes[0] > 0 && !t->data) return MOE_ERR_INVALID_ARG;
  v->data = t->data;
  v->s0 = t->sizes[0] == 1 ? 0 : t->strides[0];
  v->s1 = t->sizes[1] == 1 ? 0 : t->strides[1];
  v->dtype = t->dtype;
  *mode = t->sizes[0] == 1 ? (t->sizes[1] == 1 ? kGateOne : kGateChannel)
                           : (t->sizes[1] == 1 ? kGateToken : kGateFull);
  return MOE_OK;
}

// 16-byte accesses possible: unit inner stride, aligned rows (or no tensor at all).
bool wide_ok(const RowView& v) {
  if (!v.data) return true;
  return v.s1 == 1 && reinterpret_cast<uintptr_t>(v.data) % 16 == 0 && (v.s0 * float_size(v.dtype)) % 16 == 0;
}

bool norm_shape_ok(const moe_tensor_t* t, float eps) {
  return t && t->ndim == 2 && t->sizes[0] >= 0 && t->sizes[1] >= 1 && t->sizes[1] <= kNormMaxH &&
         t->sizes[0] < (int64_t(1) << 40) && std::isfinite(eps) && eps >= 0.0f;
}

#define MOE_TRY(call)                   \
  do {                                  \
    const moe_status_t _s = (call);     \
    if (_s != MOE_OK) return _s;        \
  } while (0)

// a call with nothing to do: no launches, and the count of them says so
moe_status_t api_empty() {
  api_set_launches(0);
  return MOE_OK;
}

size_t round256(size_t v) { return (v + 255) & ~size_t(255); }

// rows of partial column sums of a norm's gradient, either way its rows are read
size_t norm_partial_rows(int64_t T, int64_t H) {
  const int64_t a = norm_backward_rows(T, H, true, kNormMaxSms), b = norm_backward_rows(T, H, false, kNormMaxSms);
  return static_cast<size_t>(a > b ? a : b);
}
size_t norm_partial_bytes(int64_t T, int64_t H) {
  const size_t rows = norm_partial_rows(T, H);
  return round256((rows > 0 ? rows : 1) * static_cast<size_t>(H) * sizeof(float));
}

// A float32 scalar on the device ([1] or 0-d).
moe_status_t scalar_of(const moe_tensor_t* t, const float** p) {
  if (t->ndim > 1 || !t->data) return MOE_ERR_INVALID_ARG;
  if (t->dtype != MOE_F32) return MOE_ERR_UNSUPPORTED_DTYPE;
  if (t->ndim == 1 && t->sizes[0] != 1) return MOE_ERR_SHAPE_MISMATCH;
  *p = static_cast<const float*>(t->data);
  return MOE_OK;
}

constexpr int64_t kFp4MaxRows = int64_t(1) << 24, kFp4MaxK = int64_t(1) << 20;
bool fp4_shape_ok(int64_t T, int64_t N, int64_t K, int32_t fmt) {
  return T >= 0 && T <= kFp4MaxRows && N >= 1 && N <= kFp4MaxRows && K >= 32 && K <= kFp4MaxK && K % 32 == 0 &&
         T * K < (int64_t(1) << 40) && N * K < (int64_t(1) << 40) &&
         (fmt == MOE_SCALE_E8M0_32 || fmt == MOE_SCALE_E4M3_16);
}

}  // namespace
}  // namespace moe

using namespace moe;

extern "C" {

moe_status_t moe_norm_before(const moe_tensor_t* x, const moe_tensor_t* weight, float eps,
                             moe_tensor_t* out, moe_tensor_t* rstd, moe_stream_t stream) {
  if (!out || !norm_shape_ok(x, eps)) return MOE_ERR_INVALID_ARG;
  NormBefore g = {};
  g.T = x->sizes[0];
  g.H = static_cast<int>(x->sizes[1]);
  g.eps = eps;
  MOE_TRY(rows_of(x, g.T, g.H, false, &g.ring.in[0]));
  MOE_TRY(rows_of(out, g.T, g.H, true, &g.out));
  MOE_TRY(vector_of(weight, g.H, false, &g.w));
  MOE_TRY(rstd_of(rstd, g.T, true, &g.rstd, &g.rstd_s));
  if (g.T == 0) return api_empty();
  int sms = 0;
  MOE_TRY(api_device(&sms, &g.ring.err));
  const bool wide = g.H % 8 == 0 && wide_ok(g.ring.in[0]) && wide_ok(g.out) && wide_ok(g.w);
  const cudaError_t rc = launch_norm_before(g, wide, sms, reinterpret_cast<cudaStream_t>(stream));
  if (rc != cudaSuccess) return api_cuda_fail(rc, "norm_before");
  api_set_launches(1);
  return MOE_OK;
}

moe_status_t moe_norm_after(const moe_tensor_t* y, const moe_tensor_t* residual,
                            const moe_tensor_t* weight, const moe_tensor_t* gate, int32_t gate_act,
                            int32_t normalize, float residual_scale, float eps, moe_tensor_t* out,
                            moe_tensor_t* rstd, const moe_tensor_t* next_weight,
                            moe_tensor_t* next_out, moe_tensor_t* next_rstd, moe_stream_t stream) {
  if (!out || !norm_shape_ok(y, eps) || (normalize != 0 && normalize != 1)) return MOE_ERR_INVALID_ARG;
  NormAfter g = {};
  g.T = y->sizes[0];
  g.H = static_cast<int>(y->sizes[1]);
  g.eps = eps;
  g.alpha = residual_scale;
  g.normalize = normalize;
  g.act = gate_act;
  MOE_TRY(rows_of(y, g.T, g.H, false, &g.ring.in[0]));
  if (residual) MOE_TRY(rows_of(residual, g.T, g.H, false, &g.ring.in[1]));
  if (residual_scale == 0.0f) g.ring.in[1] = RowView();
  MOE_TRY(rows_of(out, g.T, g.H, true, &g.out));
  MOE_TRY(vector_of(weight, g.H, false, &g.w));
  MOE_TRY(gate_of(gate, g.T, g.H, gate_act, &g.gate, &g.gate_mode));
  if (g.gate_mode == kGateFull) g.ring.in[2] = g.gate;
  MOE_TRY(rstd_of(rstd, g.T, true, &g.rstd, &g.rstd_s));
  MOE_TRY(vector_of(next_weight, g.H, false, &g.wn));
  if (next_out) MOE_TRY(rows_of(next_out, g.T, g.H, true, &g.nxt));
  MOE_TRY(rstd_of(next_rstd, g.T, true, &g.next_rstd, &g.next_rstd_s));
  if (g.T == 0) return api_empty();
  int sms = 0;
  MOE_TRY(api_device(&sms, &g.ring.err));
  const bool gate_rows = g.gate_mode == kGateFull || g.gate_mode == kGateChannel;
  const bool wide = g.H % 8 == 0 && wide_ok(g.ring.in[0]) && wide_ok(g.ring.in[1]) && wide_ok(g.out) &&
                    wide_ok(g.w) && (!gate_rows || wide_ok(g.gate)) && (!next_out || (wide_ok(g.wn) && wide_ok(g.nxt)));
  const cudaError_t rc = launch_norm_after(g, wide, sms, reinterpret_cast<cudaStream_t>(stream));
  if (rc != cudaSuccess) return api_cuda_fail(rc, "norm_after");
  api_set_launches(1);
  return MOE_OK;
}

size_t moe_norm_backward_workspace_bytes(int64_t T, int64_t H) {
  if (T < 0 || H < 1 || H > kNormMaxH) return 0;
  const size_t rows = norm_partial_rows(T, H);
  return norm_partial_bytes(T, H) + round256((rows > 0 ? rows : 1) * sizeof(float));
}

moe_status_t moe_norm_before_backward(const moe_tensor_t* dout, const moe_tensor_t* x,
                                      const moe_tensor_t* rstd, const moe_tensor_t* weight,
                                      const moe_tensor_t* residual_grad, float residual_scale,
                                      moe_tensor_t* dx, moe_tensor_t* dweight, void* workspace,
                                      size_t workspace_bytes, moe_stream_t stream) {
  if (!x || !rstd || !dx || !norm_shape_ok(dout, 0.0f)) return MOE_ERR_INVALID_ARG;
  NormBeforeBackward g = {};
  g.T = dout->sizes[0];
  g.H = static_cast<int>(dout->sizes[1]);
  g.alpha = residual_scale;
  MOE_TRY(rows_of(dout, g.T, g.H, false, &g.ring.in[0]));
  MOE_TRY(rows_of(x, g.T, g.H, false, &g.ring.in[1]));
  if (residual_grad) MOE_TRY(rows_of(residual_grad, g.T, g.H, false, &g.ring.in[2]));
  if (residual_scale == 0.0f) g.ring.in[2] = RowView();
  MOE_TRY(rows_of(dx, g.T, g.H, true, &g.dx));
  MOE_TRY(vector_of(weight, g.H, false, &g.w));
  ColumnSum c = {};
  MOE_TRY(vector_of(dweight, g.H, true, &c.dw));
  float* r = nullptr;
  MOE_TRY(rstd_of(rstd, g.T, false, &r, &g.rstd_s));
  g.rstd = r;
  if (dweight) {
    if (!workspace || reinterpret_cast<uintptr_t>(workspace) % 256 != 0) return MOE_ERR_INVALID_ARG;
    if (workspace_bytes < moe_norm_backward_workspace_bytes(g.T, g.H)) return MOE_ERR_WORKSPACE_TOO_SMALL;
  }
  if (g.T == 0 && !dweight) return api_empty();
  int sms = 0;
  MOE_TRY(api_device(&sms, &g.ring.err));
  const cudaStream_t st = reinterpret_cast<cudaStream_t>(stream);
  g.part = dweight ? static_cast<float*>(workspace) : nullptr;
  int launches = 0;
  const bool wide = g.H % 8 == 0 && wide_ok(g.ring.in[0]) && wide_ok(g.ring.in[1]) &&
                    wide_ok(g.ring.in[2]) && wide_ok(g.dx) && wide_ok(g.w);
  if (g.T > 0) {
    const cudaError_t rc = launch_norm_before_backward(g, wide, sms, st);
    if (rc != cudaSuccess) return api_cuda_fail(rc, "norm_before_backward");
    ++launches;
  }
  if (dweight) {
    c.rows = static_cast<int>(norm_backward_rows(g.T, g.H, wide, sms));
    c.H = g.H;
    c.part = g.part;
    const cudaError_t rc = launch_column_sum(c, st);
    if (rc != cudaSuccess) return api_cuda_fail(rc, "norm_before_backward column sums");
    ++launches;
  }
  api_set_launches(launches);
  return MOE_OK;
}

moe_status_t moe_norm_after_backward(const moe_tensor_t* dout, const moe_tensor_t* y,
                                     const moe_tensor_t* rstd, const moe_tensor_t* weight,
                                     const moe_tensor_t* gate, int32_t gate_act, int32_t normalize,
                                     moe_tensor_t* dy, moe_tensor_t* dweight, moe_tensor_t* dgate,
                                     void* workspace, size_t workspace_bytes, moe_stream_t stream) {
  if (!y || !dy || !norm_shape_ok(dout, 0.0f) || (normalize != 0 && normalize != 1) ||
      (normalize == 1 && !rstd) || (dgate && !gate))
    return MOE_ERR_INVALID_ARG;
  NormAfterBackward g = {};
  g.T = dout->sizes[0];
  g.H = static_cast<int>(dout->sizes[1]);
  g.normalize = normalize;
  g.act = gate_act;
  MOE_TRY(rows_of(dout, g.T, g.H, false, &g.ring.in[0]));
  MOE_TRY(rows_of(y, g.T, g.H, false, &g.ring.in[1]));
  MOE_TRY(rows_of(dy, g.T, g.H, true, &g.dy));
  MOE_TRY(vector_of(weight, g.H, false, &g.w));
  MOE_TRY(gate_of(gate, g.T, g.H, gate_act, &g.gate, &g.gate_mode));
  if (g.gate_mode == kGateFull) g.ring.in[2] = g.gate;
  ColumnSum c = {};
  MOE_TRY(vector_of(dweight, g.H, true, &c.dw));
  if (dgate) {
    if (dgate->ndim != 2) return MOE_ERR_INVALID_ARG;
    MOE_TRY(rows_of(dgate, gate->sizes[0], gate->sizes[1], true, &g.dgate));
  }
  float* r = nullptr;
  MOE_TRY(rstd_of(rstd, g.T, false, &r, &g.rstd_s));
  g.rstd = r;
  const bool gate_sum = dgate && (g.gate_mode == kGateChannel || g.gate_mode == kGateOne);
  if (dweight || gate_sum) {
    if (!workspace || reinterpret_cast<uintptr_t>(workspace) % 256 != 0) return MOE_ERR_INVALID_ARG;
    if (workspace_bytes < moe_norm_backward_workspace_bytes(g.T, g.H)) return MOE_ERR_WORKSPACE_TOO_SMALL;
  }
  if (g.T == 0 && !dweight && !gate_sum) return api_empty();
  int sms = 0;
  MOE_TRY(api_device(&sms, &g.ring.err));
  const cudaStream_t st = reinterpret_cast<cudaStream_t>(stream);
  // [partial rows][one gate's partials]; a per-channel gate's gradient comes from dweight's sums
  const size_t rows_bytes = norm_partial_bytes(g.T, g.H);
  g.part = dweight || (gate_sum && g.gate_mode == kGateChannel) ? static_cast<float*>(workspace) : nullptr;
  g.part_gate = gate_sum && g.gate_mode == kGateOne
                    ? reinterpret_cast<float*>(static_cast<char*>(workspace) + rows_bytes)
                    : nullptr;
  int launches = 0;
  const bool gate_rows = g.gate_mode == kGateFull || g.gate_mode == kGateChannel;
  const bool wide = g.H % 8 == 0 && wide_ok(g.ring.in[0]) && wide_ok(g.ring.in[1]) && wide_ok(g.dy) && wide_ok(g.w) &&
                    (!gate_rows || wide_ok(g.gate)) && (g.gate_mode != kGateFull || wide_ok(g.dgate));
  if (g.T > 0) {
    const cudaError_t rc = launch_norm_after_backward(g, wide, sms, st);
    if (rc != cudaSuccess) return api_cuda_fail(rc, "norm_after_backward");
    ++launches;
  }
  if (dweight || gate_sum) {
    c.rows = static_cast<int>(norm_backward_rows(g.T, g.H, wide, sms));
    c.H = g.H;
    c.act = gate_act;
    c.gate_mode = g.gate_mode;
    c.part = g.part;
    c.part_gate = g.part_gate;
    c.dgate = g.dgate;
    c.gate = g.gate;
    c.w = g.w;
    const cudaError_t rc = launch_column_sum(c, st);
    if (rc != cudaSuccess) return api_cuda_fail(rc, "norm_after_backward column sums");
    ++launches;
  }
  api_set_launches(launches);
  return MOE_OK;
}

moe_status_t moe_quantize_nvfp4(const moe_tensor_t* src, const moe_tensor_t* global_scale, moe_tensor_t* dst,
                                moe_stream_t stream) {
  if (!src || !global_scale || !dst || src->ndim != 2 || dst->ndim != 2) return MOE_ERR_INVALID_ARG;
  const int64_t R = src->sizes[0], K = src->sizes[1];
  if (R < 0 || K < 0) return MOE_ERR_INVALID_ARG;
  if (dst->dtype != MOE_E2M1X2) return MOE_ERR_UNSUPPORTED_DTYPE;
  RowView x;
  MOE_TRY(rows_of(src, R, K, false, &x));
  if (dst->sizes[0] != R || dst->sizes[1] != K || K % 32 != 0) return MOE_ERR_SHAPE_MISMATCH;
  const float* G = nullptr;
  MOE_TRY(scalar_of(global_scale, &G));
  if (R == 0 || K == 0) return api_empty();
  if (!dst->data || !dst->scale) return MOE_ERR_INVALID_ARG;
  if (dst->strides[1] != 1 || dst->scale_strides[1] != 1) return MOE_ERR_UNSUPPORTED_LAYOUT;
  int sms = 0;
  MOE_TRY(api_device(&sms, nullptr));
  const cudaError_t rc = launch_quantize_nv(x, wide_ok(x), R, K, G, static_cast<uint8_t*>(dst->data), dst->strides[0],
                                            static_cast<uint8_t*>(dst->scale), dst->scale_strides[0],
                                            reinterpret_cast<cudaStream_t>(stream));
  if (rc != cudaSuccess) return api_cuda_fail(rc, "quantize_nvfp4");
  api_set_launches(1);
  return MOE_OK;
}

size_t moe_linear_fp4_workspace_bytes(int64_t T, int64_t N, int64_t K, int32_t scale_format) {
  if (!fp4_shape_ok(T, N, K, scale_format)) return 0;
  const LinearFp4Plan p = linear_fp4_plan(T, N, K, scale_format == MOE_SCALE_E4M3_16);
  return p.total > 256 ? p.total : 256;
}

moe_status_t moe_linear_fp4(const moe_tensor_t* x, const moe_tensor_t* weight, int32_t scale_format,
                            const moe_tensor_t* x_global, const moe_tensor_t* weight_global, moe_tensor_t* out,
                            void* workspace, size_t workspace_bytes, moe_stream_t stream) {
  if (!x || !weight || !out || x->ndim != 2 || weight->ndim != 2 || out->ndim != 2) return MOE_ERR_INVALID_ARG;
  const bool nv = scale_format == MOE_SCALE_E4M3_16;
  if (!nv && scale_format != MOE_SCALE_E8M0_32) return MOE_ERR_INVALID_ARG;
  if (nv ? !x_global : (x_global || weight_global)) return MOE_ERR_INVALID_ARG;
  if (weight->dtype != MOE_E2M1X2 || out->dtype != MOE_BF16) return MOE_ERR_UNSUPPORTED_DTYPE;
  LinearFp4 a = {};
  a.T = x->sizes[0];
  a.K = x->sizes[1];
  a.N = weight->sizes[0];
  a.nv = nv;
  if (a.T < 0 || a.K < 0 || a.N < 0) return MOE_ERR_INVALID_ARG;
  MOE_TRY(rows_of(x, a.T, a.K, false, &a.x));
  RowView o;
  MOE_TRY(rows_of(out, a.T, a.N, true, &o));
  if (weight->sizes[1] != a.K || !fp4_shape_ok(a.T, a.N, a.K, scale_format)) return MOE_ERR_SHAPE_MISMATCH;
  if (x_global) MOE_TRY(scalar_of(x_global, &a.x_global));
  if (weight_global) MOE_TRY(scalar_of(weight_global, &a.w_global));
  if (!weight->data || !weight->scale) return MOE_ERR_INVALID_ARG;
  if (weight->strides[1] != 1 || weight->strides[0] % 16 != 0 || weight->strides[0] < 0 ||
      reinterpret_cast<uintptr_t>(weight->data) % 16 != 0)
    return MOE_ERR_UNSUPPORTED_LAYOUT;
  // (one row: its stride is never walked, but the copy engine wants one of at least a row)
  a.w_ld = a.N == 1 && weight->strides[0] < a.K / 2 ? a.K / 2 : weight->strides[0];
  if (a.w_ld < a.K / 2) return MOE_ERR_UNSUPPORTED_LAYOUT;
  a.wide = wide_ok(a.x);
  a.w = static_cast<const uint8_t*>(weight->data);
  a.w_sf = static_cast<const uint8_t*>(weight->scale);
  a.ws0 = weight->scale_strides[0];
  a.ws1 = weight->scale_strides[1];
  a.out = static_cast<__nv_bfloat16*>(out->data);
  a.os0 = out->strides[0];
  a.os1 = out->strides[1];
  const bool rows = linear_fp4_by_rows(a.T, a.N, a.K);
  const LinearFp4Plan p = linear_fp4_plan(a.T, a.N, a.K, nv);
  if (!workspace || reinterpret_cast<uintptr_t>(workspace) % 256 != 0) return MOE_ERR_INVALID_ARG;
  if (workspace_bytes < (p.total > 256 ? p.total : 256)) return MOE_ERR_WORKSPACE_TOO_SMALL;
  if (a.T == 0) return api_empty();
  int sms = 0;
  MOE_TRY(api_device(&sms, &a.err));
  const cudaStream_t st = reinterpret_cast<cudaStream_t>(stream);
  cudaError_t rc;
  if (rows) {
    rc = launch_linear_fp4_rows(a, sms, st);
  } else {
    uint8_t* w = static_cast<uint8_t*>(workspace);
    CUtensorMap maps[4];
    const uint64_t code_ld = static_cast<uint64_t>(p.num_k) * 128;
    {
      const uint64_t d[2] = {static_cast<uint64_t>(a.K / 2), static_cast<uint64_t>(a.T)}, sb[1] = {code_ld};
      const uint32_t box[2] = {128, 128};
      MOE_TRY(api_make_map(&maps[0], CU_TENSOR_MAP_DATA_TYPE_UINT8, 2, w + p.codes_off, d, sb, box,
                           CU_TENSOR_MAP_SWIZZLE_128B));
    }
    {
      const uint64_t d[2] = {static_cast<uint64_t>(a.K / 2), static_cast<uint64_t>(a.N)},
                     sb[1] = {static_cast<uint64_t>(a.w_ld)};
      const uint32_t box[2] = {128, static_cast<uint32_t>(p.ntile / 2)};
      MOE_TRY(api_make_map(&maps[1], CU_TENSOR_MAP_DATA_TYPE_UINT8, 2, a.w, d, sb, box, CU_TENSOR_MAP_SWIZZLE_128B));
    }
    const uint32_t atoms = nv ? 4 : 2;
    for (int i = 0; i < 2; ++i) {
      const uint64_t d[2] = {128, static_cast<uint64_t>(i == 0 ? p.x_atoms : p.w_atoms)}, sb[1] = {512};
      const uint32_t box[2] = {128, i == 0 ? atoms : atoms * static_cast<uint32_t>(p.nh)};
      MOE_TRY(api_make_map(&maps[2 + i], CU_TENSOR_MAP_DATA_TYPE_INT32, 2, w + (i == 0 ? p.x_off : p.w_off), d, sb,
                           box, CU_TENSOR_MAP_SWIZZLE_NONE));
    }
    rc = launch_linear_fp4_pairs(a, p, maps, w, sms, st);
  }
  if (rc != cudaSuccess) return api_cuda_fail(rc, "linear_fp4");
  api_set_launches(rows ? 1 : 2);
  return MOE_OK;
}

// [expert forward, or h of the kernels over rows][normed rows][the experts' rows: f32, or bf16 with MXFP4 weights]
struct LayerWs {
  size_t xn, y, total;
};
static bool layer_ws(int64_t T, int64_t H, int64_t I, int64_t E, int64_t k, int32_t wdtype, LayerWs* w) {
  if (T < 0 || T > MOE_LAYER_MAX_TOKENS || H > kRouteMaxH) return false;
  const size_t fwd = moe_workspace_bytes(T > 0 ? T : 1, H, I, E, k, wdtype);
  if (fwd == 0) return false;
  const size_t h = layer_by_rows(T, H, I, E, k) ? static_cast<size_t>(T) * k * I * 4 : 0;
  w->xn = round256(fwd > h ? fwd : h);
  w->y = w->xn + round256(static_cast<size_t>(T) * H * 4);
  w->total = w->y + round256(static_cast<size_t>(T) * H * 4);
  return true;
}

size_t moe_layer_decode_workspace_bytes(int64_t T, int64_t H, int64_t I, int64_t E, int64_t k, int32_t wdtype) {
  LayerWs w;
  return layer_ws(T, H, I, E, k, wdtype, &w) ? w.total : 0;
}

moe_status_t moe_layer_decode(const moe_tensor_t* x, const moe_tensor_t* pre_weight, float eps,
                              const moe_tensor_t* router, int32_t k, int32_t renormalize, int32_t shared_expert,
                              const moe_w13_t* w13, const moe_tensor_t* w2, int32_t post_norm,
                              const moe_tensor_t* post_weight, const moe_tensor_t* gate, int32_t gate_act,
                              float residual_scale, moe_tensor_t* topk_ids, moe_tensor_t* topk_weights,
                              moe_tensor_t* out, void* workspace, size_t workspace_bytes, moe_stream_t stream) {
  if (!x || !router || !w13 || !w2 || !topk_ids || !topk_weights || !out || x->ndim != 2 || router->ndim != 2 ||
      topk_ids->ndim != 2 || topk_weights->ndim != 2 || !std::isfinite(eps) || eps < 0.0f ||
      (renormalize != 0 && renormalize != 1) || (shared_expert != 0 && shared_expert != 1) ||
      (post_norm != 0 && post_norm != 1) || (!post_norm && post_weight))
    return MOE_ERR_INVALID_ARG;
  const int64_t T = x->sizes[0], H = x->sizes[1], E = router->sizes[0];
  if (T < 0 || T > MOE_LAYER_MAX_TOKENS || H < 1 || H > kRouteMaxH || E < 1 || E > kRouteMaxE || k < 1 || k > E ||
      k + shared_expert > 32)
    return MOE_ERR_INVALID_ARG;
  if (x->dtype != MOE_BF16 || out->dtype != MOE_BF16) return MOE_ERR_UNSUPPORTED_DTYPE;
  Route r = {};
  MOE_TRY(rows_of(x, T, H, false, &r.x));
  MOE_TRY(rows_of(router, E, H, false, &r.router));
  MOE_TRY(vector_of(pre_weight, H, false, &r.w));
  RowView o, pw;
  MOE_TRY(rows_of(out, T, H, true, &o));
  MOE_TRY(vector_of(post_weight, H, false, &pw));
  if (topk_ids->sizes[1] != k + shared_expert || w13->gate.sizes[0] != E + shared_expert) return MOE_ERR_SHAPE_MISMATCH;
  for (const moe_tensor_t* t : {topk_ids, topk_weights})
    if ((T > 1 && t->strides[0] == 0) || (k + shared_expert > 1 && t->strides[1] == 0)) return MOE_ERR_UNSUPPORTED_LAYOUT;
  MOE_TRY(api_forward_check(x, w13, w2, topk_ids, topk_weights, out));
  RowView gv;
  int gate_mode = 0;
  MOE_TRY(gate_of(gate, T, H, gate_act, &gv, &gate_mode));
  const int32_t wd = w13->gate.dtype;
  const int64_t I = w13->gate.sizes[1];
  LayerWs L;
  if (!layer_ws(T, H, I, E + shared_expert, k + shared_expert, wd, &L)) return MOE_ERR_INVALID_ARG;
  if (!workspace || reinterpret_cast<uintptr_t>(workspace) % 256 != 0) return MOE_ERR_INVALID_ARG;
  if (workspace_bytes < L.total) return MOE_ERR_WORKSPACE_TOO_SMALL;
  if (T == 0) return api_empty();
  int sms = 0;
  MOE_TRY(api_device(&sms, nullptr));
  uint8_t* ws = static_cast<uint8_t*>(workspace);
  const cudaStream_t st = reinterpret_cast<cudaStream_t>(stream);
  r.wide = r.router.dtype == MOE_BF16 && H % 8 == 0 && wide_ok(r.router);
  r.x_wide = r.w.dtype == MOE_BF16 && H % 8 == 0 && wide_ok(r.x) && wide_ok(r.w);
  r.T = T;
  r.H = static_cast<int>(H);
  r.E = static_cast<int>(E);
  r.k = k;
  r.renorm = renormalize;
  r.shared = shared_expert;
  r.eps = eps;
  const bool by_rows = wd == MOE_BF16 && layer_by_rows(T, H, I, E + shared_expert, k + shared_expert);
  r.xn = reinterpret_cast<__nv_bfloat16*>(ws + L.xn);
  r.xn32 = by_rows ? reinterpret_cast<float*>(ws + L.xn) : nullptr;
  r.ids = View2{topk_ids->data, topk_ids->strides[0], topk_ids->strides[1], topk_ids->dtype};
  r.wts = View2{topk_weights->data, topk_weights->strides[0], topk_weights->strides[1], topk_weights->dtype};
  const cudaError_t rc = launch_route(r, st);
  if (rc != cudaSuccess) return api_cuda_fail(rc, "layer_decode route");
  int launches = 1;
  moe_tensor_t xn = {};
  xn.data = ws + L.xn;
  xn.dtype = MOE_BF16;
  xn.ndim = 2;
  xn.sizes[0] = T;
  xn.sizes[1] = H;
  xn.strides[0] = H;
  xn.strides[1] = 1;
  moe_tensor_t y = xn;
  y.data = ws + L.y;
  // The experts' sum: finished where the slots are combined, or kept for the norm after it.  Off the
  // kernels over rows, xn and h are bf16 because the tensor core takes them so, and a slot's row because
  // moe_forward's second product writes it so.  Their errors in root mean square, of an out whose residual is
  // twice its normed y: 0.0011, 0.0007 and 0.0007, with out's own 0.0017 together 0.0022 (H = 4096,
  // I = 1536, k = 8); rows in fp32 would leave 0.0021 for twice their traffic.  With MXFP4 weights the
  // 4-bit operands are far coarser than y's bf16.
  Finish f;
  const bool after = post_norm || wd != MOE_BF16;
  if (!after) {
    f.mode = kFinishGate;
    f.residual = View2{x->data, x->strides[0], x->strides[1], x->dtype};
    f.alpha = residual_scale;
    f.gate = View2{gv.data, gv.s0, gv.s1, gv.dtype};
    f.act = gate_act;
  } else if (wd == MOE_BF16) {
    f.mode = kFinishRows;
    f.y32 = reinterpret_cast<float*>(ws + L.y);
  }
  if (by_rows) {
    LayerRows a = {};
    a.xn = r.xn32;
    a.h = reinterpret_cast<float*>(ws);
    a.ids = r.ids;
    a.wts = r.wts;
    a.T = static_cast<int>(T);
    a.k = k + shared_expert;
    a.H = static_cast<int>(H);
    a.I = static_cast<int>(I);
    a.E = E + shared_expert;
    a.gate = static_cast<const __nv_bfloat16*>(w13->gate.data);
    a.up = static_cast<const __nv_bfloat16*>(w13->up.data);
    a.w2 = static_cast<const __nv_bfloat16*>(w2->data);
    a.gs0 = w13->gate.strides[0];
    a.gs1 = w13->gate.strides[1];
    a.us0 = w13->up.strides[0];
    a.us1 = w13->up.strides[1];
    a.ws0 = w2->strides[0];
    a.ws1 = w2->strides[1];
    a.out = static_cast<__nv_bfloat16*>(out->data);
    a.os0 = out->strides[0];
    a.os1 = out->strides[1];
    a.finish = f;
    const cudaError_t rr = launch_layer_rows(a, sms, st);
    if (rr != cudaSuccess) return api_cuda_fail(rr, "layer_decode rows");
    launches += 2;
  } else {
    MOE_TRY(api_forward(&xn, w13, w2, topk_ids, topk_weights, after ? &y : out, workspace, L.xn, st, f));
    launches += api_launches();
  }
  if (after) {
    if (f.mode == kFinishRows) y.dtype = MOE_F32;
    MOE_TRY(moe_norm_after(&y, x, post_weight, gate, gate_act, post_norm, residual_scale, eps, out, nullptr, nullptr,
                           nullptr, nullptr, stream));
    ++launches;
  }
  api_set_launches(launches);
  return MOE_OK;
}

}  // extern "C"
