// Gradient of the scored router's weights with regard to its logits.
//
// With the chosen experts i_j, their scores s_j, the gradient g_j of the weights:
//   w_j = scale s_j / T, T = sum s  (renormalised)   u_j = dL/ds_j = scale (g_j - sum_i g_i s_i / T) / T
//   w_j = scale s_j                                  u_j = scale g_j
//   sigmoid:  dL/dl_e = sum over j with i_j = e of u_j s_j (1 - s_j)
//   softmax:  dL/dl_e = s_e (sum over those of u_j - sum_j u_j s_j), for every e
// Renormalised, u_j s_j is scale q_j (g_j - sum g q) with q = s / T, which adds up to 0
// over j: only the chosen experts get a gradient, and it needs their logits alone (a
// softmax's q are the softmax of the chosen logits). Only the plain softmax reads the row.
//
// One warp per token, the row of gradients put together in shared memory and written once.
// What bounds it is that write (and the plain softmax's read).
#include <cuda_bf16.h>

#include <cfloat>

#include "ops.cuh"

namespace moe {
namespace {

constexpr int kThreads = 128, kWarps = kThreads / 32;

__device__ __forceinline__ float to_f32(float v) { return v; }
__device__ __forceinline__ float to_f32(uint16_t v) { return __uint_as_float(static_cast<uint32_t>(v) << 16); }
__device__ __forceinline__ void put(float* p, float v) { *p = v; }
__device__ __forceinline__ void put(uint16_t* p, float v) { *reinterpret_cast<__nv_bfloat16*>(p) = __float2bfloat16_rn(v); }
// (as the router reads it: a NaN logit is -infinity, +infinity the largest number)
__device__ __forceinline__ float clean_logit(float x) { return fminf(fmaxf(x, -INFINITY), FLT_MAX); }

__device__ __forceinline__ float warp_sum(float v) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
  return v;
}
__device__ __forceinline__ float warp_max(float v) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) v = fmaxf(v, __shfl_xor_sync(0xffffffffu, v, o));
  return v;
}

template <typename T>
__global__ void __launch_bounds__(kThreads) route_backward_kernel(const RouteBackwardArgs a) {
  extern __shared__ float rows[];
  const int lane = threadIdx.x & 31, w = threadIdx.x >> 5;
  float* d = rows + static_cast<size_t>(w) * a.E;
  for (int e = lane; e < a.E; e += 32) d[e] = 0.f;
  pdl_wait();
  const long long t = static_cast<long long>(blockIdx.x) * kWarps + w;
  if (t >= a.M) return;
  const T* l = static_cast<const T*>(a.logits) + t * a.row_stride;
  int id = -1 - lane;
  float g = 0.f, x = -INFINITY;
  if (lane < a.topk) {
    const int i = a.ids[t * a.topk + lane];
    if (static_cast<uint32_t>(i) < static_cast<uint32_t>(a.E)) {
      id = i;
      x = clean_logit(to_f32(l[i]));
    }
    g = a.dweights[t * a.topk + lane];
  }
  // (an expert that is not to be chosen fills a place with weight 0, whatever its logit's
  // neighbourhood: no gradient)
  const bool live = x != -INFINITY;
  if (!live) g = 0.f;
  float own = 0.f;    // u_j s_j (1 - s_j), or u_j s_j
  float every = 0.f;  // sum_j u_j s_j, which a softmax takes from every expert
  float top = -INFINITY, z = 1.f;  // of the whole row, for the plain softmax
  if (a.softmax && !a.renormalize) {
    for (int e = lane; e < a.E; e += 32) top = fmaxf(top, clean_logit(to_f32(l[e])));
    top = warp_max(top);
    z = 0.f;
    if (top != -INFINITY)
      for (int e = lane; e < a.E; e += 32) z += expf(clean_logit(to_f32(l[e])) - top);
    z = warp_sum(z);
    if (live) own = a.scale * g * (expf(x - top) / z);
    every = warp_sum(own);
  } else {
    // the score, or where only quotients of scores count a multiple that 32 bits do not
    // round to 0; and 1 - s
    float s, rest = 1.f;
    const float most = warp_max(x);
    if (a.softmax) {
      s = live ? expf(x - most) : 0.f;
    } else {
      rest = 1.0f / (1.0f + expf(x));
      s = !live ? 0.f : a.renormalize && most < 0.f ? expf(x - most) * rest : 1.0f / (1.0f + expf(-x));
    }
    if (a.renormalize) {
      const float sum = warp_sum(s);
      const float q = sum > 0.f ? s / sum : 0.f;
      own = a.scale * q * (g - warp_sum(g * q)) * rest;
    } else {
      own = a.scale * g * s * rest;
    }
    if (!live) own = 0.f;
  }
  // The same expert twice: the lowest lane adds the others', in their order.
  const unsigned peers = __match_any_sync(0xffffffffu, id);
  if (__any_sync(0xffffffffu, peers != (1u << lane))) {
    float sum = 0.f;
    for (int j = 0; j < 32; ++j) {
      const float v = __shfl_sync(0xffffffffu, own, j);
      if (peers >> j & 1) sum += v;
    }
    own = sum;
  }
  __syncwarp();
  if (id >= 0 && lane == __ffs(peers) - 1) d[id] = own;
  __syncwarp();
  T* out = static_cast<T*>(a.dlogits) + t * a.E;
  const bool plain = a.softmax && !a.renormalize;
  for (int e = lane; e < a.E; e += 32) {
    float v = d[e];
    if (plain && top != -INFINITY) v -= expf(clean_logit(to_f32(l[e])) - top) / z * every;
    put(out + e, v);
  }
}

}  // namespace

cudaError_t launch_route_backward(const RouteBackwardArgs& a, cudaStream_t stream) {
  const dim3 grid((static_cast<unsigned>(a.M) + kWarps - 1) / kWarps);
  const size_t smem = static_cast<size_t>(kWarps) * a.E * sizeof(float);
  if (a.logits_type == kTypeF32) return launch_k(route_backward_kernel<float>, grid, dim3(kThreads), smem, stream, true, a);
  return launch_k(route_backward_kernel<uint16_t>, grid, dim3(kThreads), smem, stream, true, a);
}

}  // namespace moe
