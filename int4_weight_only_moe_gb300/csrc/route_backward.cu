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
// Where only the chosen experts get a gradient a token takes 8, 16 or 32 lanes, as topk
// asks; rows are filled with zeros first, which waits for nothing, and the few others are
// written over them (in L2). The plain softmax takes a warp to a token and puts its row
// together in shared memory. What bounds it is the writing (and the plain softmax's read),
// and the latency of one chain of loads. 16,384 tokens of 384 experts, top-8: 8.6 us, 9.5
// with a warp to a token.
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

// Over the kLanes lanes of a token.
template <int kLanes>
__device__ __forceinline__ float sum_of(float v) {
#pragma unroll
  for (int o = kLanes / 2; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
  return v;
}
template <int kLanes>
__device__ __forceinline__ float max_of(float v) {
#pragma unroll
  for (int o = kLanes / 2; o > 0; o >>= 1) v = fmaxf(v, __shfl_xor_sync(0xffffffffu, v, o));
  return v;
}
// What lane j of a token has found for its expert `id` (negative ones are nobody's), with
// those of later lanes with the same expert added to it in their order; whether it is the
// first of them. `token`: the token's number in the warp.
template <int kLanes>
__device__ __forceinline__ bool add_same(float* own, int id, int token) {
  const int lane = threadIdx.x & 31;
  const unsigned peers = __match_any_sync(0xffffffffu, id < 0 ? -1 - lane : id * (32 / kLanes) + token);
  if (__any_sync(0xffffffffu, peers != (1u << lane))) {
    float sum = 0.f;
    for (int j = 0; j < 32; ++j) {
      const float v = __shfl_sync(0xffffffffu, *own, j);
      if (peers >> j & 1) sum += v;
    }
    *own = sum;
  }
  return id >= 0 && lane == __ffs(peers) - 1;
}

// Four consecutive values of a row (aligned to them), and one.
__device__ __forceinline__ void put4(float* p, const float (&v)[4]) { *reinterpret_cast<float4*>(p) = make_float4(v[0], v[1], v[2], v[3]); }
__device__ __forceinline__ void put4(uint16_t* p, const float (&v)[4]) {
  const __nv_bfloat162 a = __floats2bfloat162_rn(v[0], v[1]), b = __floats2bfloat162_rn(v[2], v[3]);
  *reinterpret_cast<uint2*>(p) = make_uint2(*reinterpret_cast<const uint32_t*>(&a), *reinterpret_cast<const uint32_t*>(&b));
}

// All but the plain softmax. `four`: rows of whole, aligned fours.
template <typename T, int kLanes>
__global__ void __launch_bounds__(kThreads) route_backward_kernel(const RouteBackwardArgs a, bool four) {
  constexpr int kTokens = 32 / kLanes;
  const int lane = threadIdx.x & 31, j = lane % kLanes, token = lane / kLanes;
  pdl_wait();
  const long long t0 = (static_cast<long long>(blockIdx.x) * kWarps + (threadIdx.x >> 5)) * kTokens, t = t0 + token;
  if (t0 >= a.M) return;
  int id = -1;
  float g = 0.f, x = -INFINITY;
  if (j < a.topk && t < a.M) {
    id = a.ids[t * a.topk + j];
    g = a.dweights[t * a.topk + j];
  }
  {
    T* out = static_cast<T*>(a.dlogits) + t0 * a.E;
    const int n = static_cast<int>(min(static_cast<long long>(kTokens), a.M - t0)) * a.E;
    const float zero[4] = {};
    if (four)
      for (int e = 4 * lane; e < n; e += 128) put4(out + e, zero);
    else
      for (int e = lane; e < n; e += 32) put(out + e, 0.f);
  }
  if (static_cast<uint32_t>(id) < static_cast<uint32_t>(a.E))
    x = clean_logit(to_f32(static_cast<const T*>(a.logits)[t * a.row_stride + id]));
  else
    id = -1;
  // (an expert that is not to be chosen fills a place with weight 0: no gradient)
  const bool live = x != -INFINITY;
  if (!live) g = 0.f;
  // the score, or where only quotients of scores count a multiple that 32 bits do not
  // round to 0; and 1 - s
  float s, rest = 1.f;
  const float most = max_of<kLanes>(x);
  if (a.softmax) {
    s = live ? expf(x - most) : 0.f;
  } else {
    rest = 1.0f / (1.0f + expf(x));
    s = !live ? 0.f : a.renormalize && most < 0.f ? expf(x - most) * rest : 1.0f / (1.0f + expf(-x));
  }
  float own;  // u_j s_j (1 - s_j), or u_j s_j
  if (a.renormalize) {
    const float sum = sum_of<kLanes>(s);
    const float q = sum > 0.f ? s / sum : 0.f;
    own = a.scale * q * (g - sum_of<kLanes>(g * q)) * rest;
  } else {
    own = a.scale * g * s * rest;
  }
  if (!live) own = 0.f;
  const bool first = add_same<kLanes>(&own, id, token);
  __syncwarp();  // (behind the zeros)
  if (first) put(static_cast<T*>(a.dlogits) + t * a.E + id, own);
}

// Softmax scores that are not renormalised.
template <typename T>
__global__ void __launch_bounds__(kThreads) route_backward_plain_kernel(const RouteBackwardArgs a, bool four) {
  extern __shared__ float rows[];
  const int lane = threadIdx.x & 31, w = threadIdx.x >> 5;
  pdl_wait();
  const long long t = static_cast<long long>(blockIdx.x) * kWarps + w;
  if (t >= a.M) return;
  const T* l = static_cast<const T*>(a.logits) + t * a.row_stride;
  T* out = static_cast<T*>(a.dlogits) + t * a.E;
  float* d = rows + static_cast<size_t>(w) * a.E;  // (a lane's own values until the row is written)
  int id = -1;
  float g = 0.f, x = -INFINITY;
  if (lane < a.topk) {
    id = a.ids[t * a.topk + lane];
    g = a.dweights[t * a.topk + lane];
  }
  float top = -INFINITY, z = 0.f;
  for (int e = lane; e < a.E; e += 32) {
    d[e] = clean_logit(to_f32(l[e]));
    top = fmaxf(top, d[e]);
  }
  if (static_cast<uint32_t>(id) < static_cast<uint32_t>(a.E))
    x = clean_logit(to_f32(l[id]));
  else
    id = -1;
  const bool live = x != -INFINITY;
  top = max_of<32>(top);
  if (top == -INFINITY) top = 0.f;  // (a row of nothing: all 0)
  for (int e = lane; e < a.E; e += 32) {
    d[e] = expf(d[e] - top);
    z += d[e];
  }
  z = sum_of<32>(z);
  float own = live ? a.scale * g * (expf(x - top) / z) : 0.f;  // u_j s_j
  const float by = z > 0.f ? sum_of<32>(own) / z : 0.f;        // what a softmax takes from every expert
  const bool first = add_same<32>(&own, id, 0);
  for (int e = lane; e < a.E; e += 32) d[e] *= -by;
  __syncwarp();
  if (first) d[id] += own;
  __syncwarp();
  if (four)
    for (int e = 4 * lane; e < a.E; e += 128) {
      const float v[4] = {d[e], d[e + 1], d[e + 2], d[e + 3]};
      put4(out + e, v);
    }
  else
    for (int e = lane; e < a.E; e += 32) put(out + e, d[e]);
}

}  // namespace

cudaError_t launch_route_backward(const RouteBackwardArgs& a, cudaStream_t stream) {
  auto go = [&](auto value) {
    using T = decltype(value);
    const bool four = a.E % 4 == 0 && reinterpret_cast<uintptr_t>(a.dlogits) % (4 * sizeof(T)) == 0;
    auto with = [&](auto kernel, int tokens, size_t smem) {  // `tokens` to a CTA
      const dim3 grid(static_cast<unsigned>((a.M + static_cast<long long>(tokens) - 1) / tokens));
      return launch_k(kernel, grid, dim3(kThreads), smem, stream, true, a, four);
    };
    if (a.softmax && !a.renormalize)
      return with(route_backward_plain_kernel<T>, kWarps, static_cast<size_t>(kWarps) * a.E * sizeof(float));
    if (a.topk <= 8) return with(route_backward_kernel<T, 8>, 4 * kWarps, 0);
    if (a.topk <= 16) return with(route_backward_kernel<T, 16>, 2 * kWarps, 0);
    return with(route_backward_kernel<T, 32>, kWarps, 0);
  };
  return a.logits_type == kTypeF32 ? go(float{}) : go(uint16_t{});
}

}  // namespace moe
