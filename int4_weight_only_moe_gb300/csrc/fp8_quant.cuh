// Arithmetic of the block quantisers, shared with the products that quantise what they
// compute.
#pragma once
#include <cuda_fp8.h>

#include <cstdint>

namespace moe {

constexpr float kE4m3Max = 448.0f;
constexpr float kScaleFloor = 1.17549435e-38f;  // 2^-126

// SiLU(g) * u with the hardware's exponential and reciprocal, of which e4m3 keeps 2^-4. The
// error is at most 2^-21 + |g| 2^-23 of the result: a few roundings, and the exponent g
// log2(e), rounded to 32 bits before the exponential (the product and its constant, 1.3e-8
// off, together below 2^-23 of it). Below -87.3, where the reciprocal of 1 + exp(-g) is
// below 2^-126 and flushed, the result is 0 (it is at most 1.1e-36 of u there).
__device__ __forceinline__ float swiglu(float g, float u) {
  float e, r;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(e) : "f"(g * -1.44269504f));
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(1.0f + e));
  return g * r * u;
}

// max(m, |v|) that keeps a NaN.
__device__ __forceinline__ float max_nan(float m, float v) {
  float d;
  asm("max.NaN.f32 %0, %1, %2;" : "=f"(d) : "f"(m), "f"(fabsf(v)));
  return d;
}

// Scale of a block from its largest magnitude.
__device__ __forceinline__ float block_scale(float amax) {
  const float s = __fdiv_rn(amax, kE4m3Max);
  return s != s ? s : fmaxf(s, kScaleFloor);
}

// x / s, correctly rounded, from r = 1 / s correctly rounded: q = x r, then one step with
// the exact remainder (Markstein, "Computation of elementary functions on the IBM RISC
// System/6000 processor", 1990). Only for scales in [2^-90, 2^90], where the remainder
// stays in fp32's range. (The remainder is taken as q s - x: x - q s would be +0 for x = -0
// and make the quotient +0.)
__device__ __forceinline__ float quotient(float x, float s, float r) {
  const float q = x * r;
  return fmaf(-fmaf(q, s, -x), r, q);
}

__device__ __forceinline__ uint32_t e4m3_pair(float lo, float hi) {
  return __nv_cvt_float2_to_fp8x2(make_float2(lo, hi), __NV_SATFINITE, __NV_E4M3);
}

// Four values over a scale, as e4m3 bytes (`exact`: quotient() holds for it).
__device__ __forceinline__ uint32_t e4m3_quad(float a, float b, float c, float d, float s, float r, bool exact) {
  if (exact)
    a = quotient(a, s, r), b = quotient(b, s, r), c = quotient(c, s, r), d = quotient(d, s, r);
  else
    a = __fdiv_rn(a, s), b = __fdiv_rn(b, s), c = __fdiv_rn(c, s), d = __fdiv_rn(d, s);
  return e4m3_pair(a, b) | (e4m3_pair(c, d) << 16);
}
// Whether quotient() holds for a scale.
__device__ __forceinline__ bool quotient_ok(float s) { return s >= 0x1p-90f && s <= 0x1p90f; }

}  // namespace moe
