// A block's gate: the activation of its value, and what the combine of the experts' rows does
// with a sum on its way out (the gate and the scaled residual, or the fp32 row itself).
#pragma once

#include <cuda_runtime.h>
#include <stdint.h>

#include "../../include/moe.h"
#include "moe_internal.h"

namespace moe {

// the gate's activation from the gate's value
__device__ __forceinline__ float gate_value(float g, int act) {
  if (act == MOE_GATE_SIGMOID) return 1.0f / (1.0f + expf(-g));
  if (act == MOE_GATE_TANH) return tanhf(g);
  return g;
}

__device__ __forceinline__ float view_float(const View2& v, int64_t r, int64_t c) {
  const int64_t off = r * v.s0 + c * v.s1;
  return v.dtype == MOE_F32
             ? static_cast<const float*>(v.data)[off]
             : __uint_as_float(static_cast<uint32_t>(static_cast<const uint16_t*>(v.data)[off]) << 16);
}

// Eight neighbouring sums of row t from column c: true when they have gone to y32 unrounded,
// else a holds alpha * residual + gate * sum.
__device__ __forceinline__ bool finish8(const Finish& f, int64_t t, int64_t H, int64_t c, float (&a)[8]) {
  if (f.mode == kFinishNone) return false;
  if (f.mode == kFinishRows) {
    float4* p = reinterpret_cast<float4*>(f.y32 + t * H + c);
    p[0] = make_float4(a[0], a[1], a[2], a[3]);
    p[1] = make_float4(a[4], a[5], a[6], a[7]);
    return true;
  }
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    float v = a[i];
    if (f.gate.data) v *= gate_value(view_float(f.gate, t, c + i), f.act);
    if (f.alpha != 0.0f) v += f.alpha * view_float(f.residual, t, c + i);
    a[i] = v;
  }
  return false;
}

}  // namespace moe
