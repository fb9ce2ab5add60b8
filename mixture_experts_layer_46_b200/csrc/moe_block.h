// Declarations of the operators around the expert forward (norms, the whole layer for a few
// tokens, the 4-bit linear layer), shared by their entry points and kernels.
#pragma once

#include <cuda.h>
#include <cuda_runtime.h>
#include <stdint.h>

#include "../../include/moe.h"
#include "moe_common.cuh"
#include "moe_internal.h"

namespace moe {

// ---- from the host runtime (moe_api.cu) --------------------------------------

// The current device: SM count and error counters; an error where it is not an sm_100 GPU.
moe_status_t api_device(int* num_sms, DeviceErrors** err);
// Records the CUDA error text of the calling thread and returns MOE_ERR_CUDA.
moe_status_t api_cuda_fail(cudaError_t rc, const char* where);
// A cached rank-2/3 K-major tensor map (dims[0] contiguous, strides in bytes).
moe_status_t api_make_map(CUtensorMap* map, CUtensorMapDataType dt, int rank, const void* base,
                          const uint64_t* dims, const uint64_t* strides_bytes, const uint32_t* box,
                          CUtensorMapSwizzle swz);
void api_set_launches(int32_t n);
int32_t api_launches();
// The expert forward with a finish (bf16 weights; MXFP4 weights: none), and its checks alone.
moe_status_t api_forward_check(const moe_tensor_t* x, const moe_w13_t* w13, const moe_tensor_t* w2,
                               const moe_tensor_t* ids, const moe_tensor_t* wts, const moe_tensor_t* out);
moe_status_t api_forward(const moe_tensor_t* x, const moe_w13_t* w13, const moe_tensor_t* w2,
                         const moe_tensor_t* ids, const moe_tensor_t* wts, moe_tensor_t* out, void* ws,
                         size_t ws_bytes, cudaStream_t st, const Finish& finish);

// ---- norms (moe_norm.cu) -----------------------------------------------------

constexpr int kNormMaxSms = 160;      // the gradient's workspace size is for at most this many SMs
constexpr int64_t kNormMaxH = 16384;  // 1024 threads x 2 slots (or 512 x 4) x 8 elements

// Rows of bf16 or fp32 elements; strides in elements (s0 = 0: the same row for every token).
struct RowView {
  const void* data = nullptr;
  int64_t s0 = 0, s1 = 0;
  int32_t dtype = 0;
};

enum { kGateNone = 0, kGateFull = 1, kGateChannel = 2, kGateToken = 3, kGateOne = 4 };

// A kernel's row inputs, and their ring in shared memory (stages of one row of each).
struct RowRing {
  RowView in[3];
  uint32_t off[3], bytes[3];
  uint32_t stage_bytes;
  int stages;
  DeviceErrors* err;
};

struct NormBefore {
  RowRing ring;  // x
  int64_t T;
  int H;
  float eps;
  RowView w, out;
  float* rstd;
  int64_t rstd_s;
};
struct NormAfter {
  RowRing ring;  // y, the residual (or none), a gate [T, H] (or none)
  int64_t T;
  int H;
  float eps, alpha;
  int normalize, act, gate_mode;
  RowView w, gate, out, wn, nxt;
  float* rstd;
  int64_t rstd_s;
  float* next_rstd;
  int64_t next_rstd_s;
};
struct NormBeforeBackward {
  RowRing ring;  // dout, x, the residual's gradient (or none)
  int64_t T;
  int H;
  float alpha;
  RowView w, dx;
  const float* rstd;
  int64_t rstd_s;
  float* part;  // [blocks, H] column sums, or null
};
struct NormAfterBackward {
  RowRing ring;  // dout, y, a gate [T, H] (or none)
  int64_t T;
  int H;
  int normalize, act, gate_mode;
  RowView w, gate, dy, dgate;
  const float* rstd;
  int64_t rstd_s;
  float* part;       // [blocks, H] column sums, or null
  float* part_gate;  // one gate in all: [blocks], or null
};
struct ColumnSum {
  int rows, H;
  int act, gate_mode;
  const float* part;       // [rows, H]
  const float* part_gate;  // [rows], or null
  RowView dw, dgate, gate, w;
};

// Blocks (= rows of partial column sums) of the gradient kernels.
int64_t norm_backward_rows(int64_t T, int64_t H, bool wide, int num_sms);
// wide: every row tensor allows 16-byte accesses (see moe_norm.cu)
cudaError_t launch_norm_before(NormBefore g, bool wide, int num_sms, cudaStream_t st);
cudaError_t launch_norm_after(NormAfter g, bool wide, int num_sms, cudaStream_t st);
cudaError_t launch_norm_before_backward(NormBeforeBackward g, bool wide, int num_sms, cudaStream_t st);
cudaError_t launch_norm_after_backward(NormAfterBackward g, bool wide, int num_sms, cudaStream_t st);
cudaError_t launch_column_sum(const ColumnSum& g, cudaStream_t st);

// ---- a layer's way in: norm, router, choice (moe_route.cu) --------------------

constexpr int64_t kRouteMaxH = 16384, kRouteMaxE = 1024;
struct Route {
  RowView x, w, router;  // w: no data = ones; router [E, H]
  int wide;              // router: bf16, 16-byte rows
  int x_wide;            // x and w likewise
  int64_t T;
  int H, E, k, renorm, shared;
  float eps;
  __nv_bfloat16* xn;     // [T, H], or
  float* xn32;           // the same unrounded
  View2 ids, wts;
};
cudaError_t launch_route(const Route& g, cudaStream_t st);

// ---- a layer's experts for a few tokens (moe_layer_rows.cu) --------------

struct LayerRows {
  const float* xn;  // [T, H]
  float* h;         // [T k, I]
  View2 ids, wts;
  int T, k, H, I;
  int64_t E;        // the shared expert counted in
  const __nv_bfloat16 *gate, *up, *w2;  // strides in elements, inner stride 1, 16-byte rows
  int64_t gs0, gs1, us0, us1, ws0, ws1;
  __nv_bfloat16* out;
  int64_t os0, os1;
  Finish finish;    // kFinishRows or kFinishGate
};
bool layer_by_rows(int64_t T, int64_t H, int64_t I, int64_t E, int64_t k);
cudaError_t launch_layer_rows(const LayerRows& a, int num_sms, cudaStream_t st);

// ---- 4-bit linear layer (moe_linear_fp4.cu) -----------------------------------

struct LinearFp4 {
  RowView x;       // [T, K]
  int wide;        // x allows 16-byte loads
  int64_t T, N, K;
  bool nv;         // e4m3 scales per 16 (else e8m0 per 32)
  const float* x_global;  // nv: not null
  const float* w_global;  // null: 1
  const uint8_t* w;       // [N, K/2] codes, rows w_ld bytes apart
  int64_t w_ld;
  const uint8_t* w_sf;    // scales, byte strides
  int64_t ws0, ws1;
  __nv_bfloat16* out;
  int64_t os0, os1;
  DeviceErrors* err;
};
// Tiles and workspace of the tensor-core path (all zero where the few-rows kernel runs).
struct LinearFp4Plan {
  int64_t num_k, n_mt, n_nt;
  int ntile, nh;
  int64_t x_atoms, w_atoms;
  size_t codes_off, x_off, w_off, total;
};
bool linear_fp4_by_rows(int64_t T, int64_t N, int64_t K);
LinearFp4Plan linear_fp4_plan(int64_t T, int64_t N, int64_t K, bool nv);
cudaError_t launch_linear_fp4_rows(const LinearFp4& a, int num_sms, cudaStream_t st);
// maps: x codes, weight codes, x scale atoms, weight scale atoms
cudaError_t launch_linear_fp4_pairs(const LinearFp4& a, const LinearFp4Plan& p, const CUtensorMap (&maps)[4],
                                    uint8_t* ws, int num_sms, cudaStream_t st);
cudaError_t launch_quantize_nv(const RowView& x, bool wide, int64_t rows, int64_t K, const float* global,
                               uint8_t* codes, int64_t ld, uint8_t* sf, int64_t sf_ld, cudaStream_t st);

}  // namespace moe
