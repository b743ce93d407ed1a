// Addends and outputs of the low-rank adapters, and the parts of a sum.
#pragma once
#include <cuda_bf16.h>

#include "ops.cuh"

namespace moe {

__device__ __forceinline__ float bf16_value(uint16_t v) { return __uint_as_float(static_cast<uint32_t>(v) << 16); }
// The leading bf16 part of a sum: the nearest, and of a number that this would make
// infinite the largest one below.
__device__ __forceinline__ uint16_t bf16_part(float s) {
  const uint16_t h = __bfloat16_as_ushort(__float2bfloat16_rn(s));
  return (h & 0x7FFFu) == 0x7F80u && isfinite(s) ? static_cast<uint16_t>(h - 1) : h;
}
// The first product's fp32 sums enter the second one as so many bf16 parts, whatever the
// output's type: each takes 8 of the 24 bits, and what is left behind the third is 0 (the parts
// below 2^-133 apart). With two parts, 16 bits, a sum is off by up to 2^-17 of itself, which is
// far below a bf16 output's rounding unless an addend, or another of the r terms, cancels
// it: addends that leave 2^-12 of the adapter's term gave errors of 1e-2 of the result.
constexpr int kParts = 3;
__device__ __forceinline__ float addend(const LoraArgs& a, long long at) {
  if (!a.add) return 0.f;
  return a.add_type == kTypeF32 ? static_cast<const float*>(a.add)[at] : bf16_value(static_cast<const uint16_t*>(a.add)[at]);
}
__device__ __forceinline__ void put(const LoraArgs& a, long long at, float v) {
  if (a.out_type == kTypeF32)
    static_cast<float*>(a.out)[at] = v;
  else
    static_cast<__nv_bfloat16*>(a.out)[at] = __float2bfloat16_rn(v);
}
// Eight consecutive ones, 16-byte aligned.
__device__ __forceinline__ void load8(const LoraArgs& a, long long at, float (&d)[8]) {
  if (!a.add) {
#pragma unroll
    for (int i = 0; i < 8; ++i) d[i] = 0.f;
  } else if (a.add_type == kTypeF32) {
    const float4* p = reinterpret_cast<const float4*>(static_cast<const float*>(a.add) + at);
    const float4 u = p[0], v = p[1];
    d[0] = u.x, d[1] = u.y, d[2] = u.z, d[3] = u.w, d[4] = v.x, d[5] = v.y, d[6] = v.z, d[7] = v.w;
  } else {
    const uint4 u = *reinterpret_cast<const uint4*>(static_cast<const uint16_t*>(a.add) + at);
    const uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) d[2 * i] = __uint_as_float(w[i] << 16), d[2 * i + 1] = __uint_as_float(w[i] & 0xFFFF0000u);
  }
}
__device__ __forceinline__ void store8(const LoraArgs& a, long long at, const float (&d)[8]) {
  if (a.out_type == kTypeF32) {
    float4* p = reinterpret_cast<float4*>(static_cast<float*>(a.out) + at);
    p[0] = make_float4(d[0], d[1], d[2], d[3]);
    p[1] = make_float4(d[4], d[5], d[6], d[7]);
  } else {
    uint32_t w[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const __nv_bfloat162 h = __floats2bfloat162_rn(d[2 * i], d[2 * i + 1]);
      w[i] = *reinterpret_cast<const uint32_t*>(&h);
    }
    *reinterpret_cast<uint4*>(static_cast<uint16_t*>(a.out) + at) = make_uint4(w[0], w[1], w[2], w[3]);
  }
}

}  // namespace moe
