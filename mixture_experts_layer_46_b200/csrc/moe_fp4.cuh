// Microscaled 4-bit quantisation with e4m3 scales per 16 elements and one float scale
// (moe_quantize_nvfp4, the activations of moe_linear_fp4).
//
//   s = e4m3(amax / (6 G)),  code = e2m1(v / (s G)),   value = code * s * G
// Both roundings go to the nearest number, ties to the even one, of the exact quotient.  In
// fp32 a quotient is off by up to 2^-22, so each is rounded twice, moved down and up by 2^-20:
// equal results are the exact one's too, and where they differ (one in some thousand times) the
// quotient is compared with the border between the two neighbours exactly.
#pragma once

#include <cuda_fp16.h>
#include <cuda_fp8.h>

#include "moe_mx.cuh"

namespace moe {

__device__ __forceinline__ uint32_t cvt_e4m3x2(float lo, float hi) {
  uint16_t r;
  asm volatile("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(r) : "f"(hi), "f"(lo));
  return r;
}
// two e4m3 codes (low byte first) as floats
__device__ __forceinline__ float2 e4m3x2_floats(uint32_t two) {
  uint32_t h;
  asm volatile("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(h) : "h"(static_cast<uint16_t>(two)));
  return __half22float2(*reinterpret_cast<const __half2*>(&h));
}
// the two e2m1 codes of a byte (low nibble first) as halves
__device__ __forceinline__ uint32_t e2m1x2_halves(uint32_t byte) {
  uint32_t h;
  asm volatile(
      "{\n\t.reg .b8 b0, b1, b2, b3;\n\t"
      "mov.b32 {b0, b1, b2, b3}, %1;\n\t"
      "cvt.rn.f16x2.e2m1x2 %0, b0;\n\t}"
      : "=r"(h)
      : "r"(byte));
  return h;
}

constexpr float kDown = 1.0f - 1.0f / (1 << 20), kUp = 1.0f + 1.0f / (1 << 20);

// e4m3 code of amax / (6 G); G a positive finite float, amax >= 0
__device__ __forceinline__ uint32_t nv_scale(float amax, float G) {
  const float r = amax / (6.0f * G);
  const uint32_t two = cvt_e4m3x2(r * kDown, r * kUp);
  const uint32_t lo = two & 0xffu, hi = two >> 8;
  const float g6 = 6.0f * G;
  if (lo == hi && g6 < 1e30f && g6 > 1e-30f) return lo;
  // exactly: the neighbours around the quotient in 64 bits
  const double t = static_cast<double>(amax) / (6.0 * static_cast<double>(G));
  if (!(t < 448.0)) return 0x7eu;
  uint32_t c = 0;
  for (uint32_t bit = 64; bit > 0; bit >>= 1)  // the largest code (0 .. 126) whose value is <= t
    if (c + bit <= 0x7eu && static_cast<double>(e4m3x2_floats(c + bit).x) <= t) c += bit;
  if (c == 0x7eu) return c;
  const float2 v = e4m3x2_floats(c | ((c + 1) << 8));
  const double mid = 0.5 * (static_cast<double>(v.x) + static_cast<double>(v.y));
  return t > mid || (t == mid && (c & 1u)) ? c + 1 : c;
}

// e2m1 magnitude code of |v| / (s G), exactly: |v| is compared with border * s * G by a fused
// multiply-add, whose sign is that of the exact difference (border * s has at most 7 bits).
__device__ __forceinline__ uint32_t e2m1_exact(float v, float s, float G) {
  const float border[7] = {0.25f, 0.75f, 1.25f, 1.75f, 2.5f, 3.5f, 5.0f};
  uint32_t c = 0;
#pragma unroll
  for (int i = 0; i < 7; ++i) {
    const float d = fmaf(-(border[i] * s), G, fabsf(v));
    if (d > 0.0f || (d == 0.0f && (i & 1))) c = i + 1;  // a tie goes to the even code
  }
  return c | (v < 0.0f ? 8u : 0u);
}

// Quantises 16 floats: two words of codes (even element in the low nibble), returns the scale.
__device__ __forceinline__ uint32_t nv_quant16(const float* v, float G, uint32_t (&w)[2]) {
  float amax = 0.0f;
#pragma unroll
  for (int i = 0; i < 16; ++i) amax = fmaxf(amax, fabsf(v[i]));
  w[0] = w[1] = 0u;
  if (!(G > 0.0f) || !(amax > 0.0f)) return 0u;
  const uint32_t sc = nv_scale(amax, G);
  if (sc == 0u) return 0u;
  const float s = e4m3x2_floats(sc).x, unit = s * G;
  const float inv = 1.0f / unit, a = inv * kDown, b = inv * kUp;
  uint32_t up[2] = {0u, 0u};
#pragma unroll
  for (int q = 0; q < 2; ++q)
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const float e = v[8 * q + 2 * i], o = v[8 * q + 2 * i + 1];
      w[q] |= cvt_e2m1x2(e * a, o * a) << (8 * i);
      up[q] |= cvt_e2m1x2(e * b, o * b) << (8 * i);
    }
  if (w[0] != up[0] || w[1] != up[1] || !(unit > 1e-30f && unit < 1e30f)) {
#pragma unroll
    for (int q = 0; q < 2; ++q) {
      w[q] = 0u;
#pragma unroll
      for (int i = 0; i < 8; ++i) w[q] |= e2m1_exact(v[8 * q + i], s, G) << (4 * i);
    }
  }
  return sc;
}

}  // namespace moe
