// Microscaled 4-bit quantisation with e4m3 scales per 16 elements and one float scale
// (moe_quantize_nvfp4, the activations of moe_linear_fp4).
//
//   s = e4m3(amax / (6 G)),  code = e2m1(v / (s G)),   value = code * s * G
// Both roundings go to the nearest number, ties to the even one, of the exact quotient.  In
// fp32 a quotient is off by up to 2^-22, so each is rounded twice, moved down and up by 2^-20:
// equal results are the exact one's too, and where they differ the quotient is compared with the
// border between the two neighbours exactly.
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

__device__ __forceinline__ uint64_t pair_of(float a, float b) {
  return static_cast<uint64_t>(__float_as_uint(a)) | (static_cast<uint64_t>(__float_as_uint(b)) << 32);
}
// the e2m1 codes of eight floats times f, the first in the low nibble (+ 0: a zero has no sign)
__device__ __forceinline__ uint32_t cvt_e2m1x8(const float* v, float f) {
  uint32_t r;
  asm("{\n\t.reg .b8 b0, b1, b2, b3;\n\t.reg .b64 t, z;\n\t.reg .f32 x, y;\n\t"
      "mov.b64 z, 0;\n\t"
      "fma.rn.f32x2 t, %1, %5, z;\n\tmov.b64 {x, y}, t;\n\tcvt.rn.satfinite.e2m1x2.f32 b0, y, x;\n\t"
      "fma.rn.f32x2 t, %2, %5, z;\n\tmov.b64 {x, y}, t;\n\tcvt.rn.satfinite.e2m1x2.f32 b1, y, x;\n\t"
      "fma.rn.f32x2 t, %3, %5, z;\n\tmov.b64 {x, y}, t;\n\tcvt.rn.satfinite.e2m1x2.f32 b2, y, x;\n\t"
      "fma.rn.f32x2 t, %4, %5, z;\n\tmov.b64 {x, y}, t;\n\tcvt.rn.satfinite.e2m1x2.f32 b3, y, x;\n\t"
      "mov.b32 %0, {b0, b1, b2, b3};\n\t}"
      : "=r"(r)
      : "l"(pair_of(v[0], v[1])), "l"(pair_of(v[2], v[3])), "l"(pair_of(v[4], v[5])), "l"(pair_of(v[6], v[7])),
        "l"(pair_of(f, f)));
  return r;
}

// A block with a NaN gets a NaN for its scale, so that whatever it meets in a product is NaN.
constexpr uint32_t kNanE4m3 = 0x7fu, kNanE8m0 = 0xffu;

constexpr float kDown = 1.0f - 1.0f / (1 << 20), kUp = 1.0f + 1.0f / (1 << 20);

// e4m3 code of amax / (6 G); G a positive finite float, inv6 = 1 / (6 G), amax >= 0.
// Six times the border between neighbours has at most 7 bits: exact as below.
__device__ __forceinline__ uint32_t nv_scale(float amax, float G, float inv6) {
  const float r = amax * inv6;
  const uint32_t two = cvt_e4m3x2(r * kDown, r * kUp), lo = two & 0xffu, hi = two >> 8;
  const float2 v = e4m3x2_floats(two);
  const float d = fmaf(-3.0f * (v.x + v.y), G, amax);
  return d > 0.0f || (d == 0.0f && (lo & 1u)) ? hi : lo;
}
// The same where 6 G or its inverse leaves the range that keeps fp32 products exact.
__device__ __noinline__ uint32_t nv_scale_far(float amax, float G) {
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
__device__ __noinline__ uint32_t e2m1_far(float v, float s, float G) {
  const double t = fabs(static_cast<double>(v)) / (static_cast<double>(s) * static_cast<double>(G));
  const double border[7] = {0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0};
  uint32_t c = 0;
  for (int i = 0; i < 7; ++i)
    if (t > border[i] || (t == border[i] && (i & 1))) c = i + 1;  // a tie goes to the even code
  return c | (v < 0.0f ? 8u : 0u);
}

// Sixteen codes of v / (s G).  Where the two roundings differ, |v| is compared with border * s * G
// by a fused multiply-add, whose sign is that of the exact difference (border * s has 7 bits).
// Ties are not rare: with G = amax / 2688 and bf16 values they meet one block in a hundred.
__device__ __forceinline__ void nv_codes16(const float* v, float s, float G, float down, float up, uint32_t (&w)[2]) {
  w[0] = cvt_e2m1x8(v, down);
  w[1] = cvt_e2m1x8(v + 8, down);
  const uint32_t d0 = w[0] ^ cvt_e2m1x8(v, up), d1 = w[1] ^ cvt_e2m1x8(v + 8, up);
  if ((d0 | d1) == 0u) return;
#pragma unroll
  for (int q = 0; q < 2; ++q) {
    const uint32_t diff = q ? d1 : d0;
    if (diff == 0u) continue;
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      if (((diff >> (4 * i)) & 15u) == 0u) continue;
      const uint32_t l = (w[q] >> (4 * i)) & 7u, h = ((w[q] ^ diff) >> (4 * i)) & 7u;
      const uint32_t two = e2m1x2_halves(l | (h << 4));
      const float2 f = __half22float2(*reinterpret_cast<const __half2*>(&two));
      const float d = fmaf(-(0.5f * (f.x + f.y) * s), G, fabsf(v[8 * q + i]));
      if (d > 0.0f || (d == 0.0f && (l & 1u))) w[q] ^= diff & (15u << (4 * i));
    }
  }
}

// Quantises 16 floats whose largest magnitude is amax: two words of codes (even element in the
// low nibble), returns the scale.  inv6 = 1 / (6 G).
__device__ __forceinline__ uint32_t nv_quant16(const float* v, float amax, float G, float inv6, uint32_t (&w)[2]) {
  w[0] = w[1] = 0u;
  if (amax != amax) return kNanE4m3;
  if (!(G > 0.0f) || !(amax > 0.0f)) return 0u;
  const bool far = !(G > 1e-24f && G < 1e24f);
  const uint32_t sc = far ? nv_scale_far(amax, G) : nv_scale(amax, G, inv6);
  if (sc == 0u) return 0u;
  const float s = e4m3x2_floats(sc).x;
  if (!far) {
    float inv;  // (within one ulp: far inside the 2^-20 that the two roundings are apart)
    asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(inv) : "f"(s * G));
    const float down = inv * kDown, up = inv * kUp;
    nv_codes16(v, s, G, down, up, w);
  } else {
#pragma unroll
    for (int i = 0; i < 16; ++i) w[i >> 3] |= e2m1_far(v[i], s, G) << (4 * (i & 7));
  }
  return sc;
}

// the smaller and the larger of two, NaN where either is
__device__ __forceinline__ float min_nan(float a, float b) {
  float r;
  asm("min.NaN.f32 %0, %1, %2;" : "=f"(r) : "f"(a), "f"(b));
  return r;
}
__device__ __forceinline__ float max_nan(float a, float b) {
  float r;
  asm("max.NaN.f32 %0, %1, %2;" : "=f"(r) : "f"(a), "f"(b));
  return r;
}
// the largest magnitude of 16 (NaN with one among them)
__device__ __forceinline__ float amax16(const float* v) {
  float m = 0.0f;
#pragma unroll
  for (int i = 0; i < 16; ++i) m = max_nan(m, fabsf(v[i]));
  return m;
}

}  // namespace moe
