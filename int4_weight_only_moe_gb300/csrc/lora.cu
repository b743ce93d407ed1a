// Low-rank adapters of many requests beside a projection:
//
//   out[m] = add[m] + scale[l] b[l] (a[l] x[m]),  l = index[m]
//
// and out[m] = add[m] for a row without an adapter.
#include <cuda_bf16.h>

#include "ops.cuh"

namespace moe {
namespace {

constexpr int kThreads = 256;

__device__ __forceinline__ float bf16_value(uint16_t v) { return __uint_as_float(static_cast<uint32_t>(v) << 16); }
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

// Any shape and alignment: one CTA to a row, everything in fp32 on the CUDA cores.
__global__ void __launch_bounds__(kThreads) lora_plain_kernel(const LoraArgs a) {
  __shared__ float v[kMaxRank];
  pdl_wait();
  const long long m = blockIdx.x;
  const int l = a.index[m], lane = threadIdx.x & 31;
  const bool has = static_cast<uint32_t>(l) < static_cast<uint32_t>(a.L);
  if (!has && a.add == a.out) return;
  if (has) {
    const uint16_t* x = a.x + m * a.ldx;
    const float scale = a.scale ? a.scale[l] : 1.f;
    for (int i = threadIdx.x / 32; i < a.r; i += kThreads / 32) {
      const uint16_t* w = a.a + (static_cast<long long>(l) * a.r + i) * a.K;
      float sum = 0.f;
      for (int k = lane; k < a.K; k += 32) sum = fmaf(bf16_value(x[k]), bf16_value(w[k]), sum);
#pragma unroll
      for (int o = 16; o > 0; o >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
      if (lane == 0) v[i] = sum * scale;
    }
    __syncthreads();
  }
  for (int n = threadIdx.x; n < a.N; n += kThreads) {
    float sum = 0.f;
    if (has) {
      const uint16_t* w = a.b + (static_cast<long long>(l) * a.N + n) * a.r;
      for (int i = 0; i < a.r; ++i) sum = fmaf(v[i], bf16_value(w[i]), sum);
    }
    put(a, m * a.N + n, sum + addend(a, m * a.N + n));
  }
}

}  // namespace

size_t lora_workspace_bytes(int M, int r, int L) {
  (void)M, (void)r, (void)L;
  return 0;
}

cudaError_t launch_lora(const LoraArgs& a, int num_sms, cudaStream_t stream) {
  (void)num_sms;
  return launch_k(lora_plain_kernel, dim3(static_cast<unsigned>(a.M)), dim3(kThreads), 0, stream, true, a);
}

}  // namespace moe
