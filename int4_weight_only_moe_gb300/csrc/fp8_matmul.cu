// 8-bit block-scaled matrix product
//
//   out[m, n] = sum_kb a_s[m, kb] b_s[n / 128, kb] sum_{k in block kb} a[m, k] b[n, k]
//               (+ add[m, n])
//
// with e4m3 operands, a scale for each 128 values of a row of `a` and for each 128 x 128
// block of `b`. A block's products are summed in fp32 unscaled; the scaled block sums
// are added in fp32 and rounded once to the output type.
#include <cuda_bf16.h>
#include <cuda_fp8.h>

#include "ops.cuh"

namespace moe {
namespace {

__device__ __forceinline__ float e4m3_f32(uint8_t v) {
  return __half2float(__half(__nv_cvt_fp8_to_halfraw(v, __NV_E4M3)));
}

__device__ __forceinline__ void store_out(const Fp8MatmulArgs& a, long long at, float y) {
  if (a.add) y += __uint_as_float(static_cast<uint32_t>(a.add[at]) << 16);
  if (a.out_type == kTypeF32)
    static_cast<float*>(a.out)[at] = y;
  else
    static_cast<__nv_bfloat16*>(a.out)[at] = __float2bfloat16_rn(y);
}

// Plain tiles on the CUDA cores: 64 x 64 outputs, 4 x 4 per thread, 32 reduction
// elements at a time.
constexpr int kT = 64, kStep = 32;
__global__ void __launch_bounds__(256) fp8_matmul_plain_kernel(Fp8MatmulArgs a) {
  pdl_wait();
  pdl_launch_dependents();
  __shared__ float sa[kStep][kT + 1], sb[kStep][kT + 1];
  const long long m0 = static_cast<long long>(blockIdx.x) * kT;
  const int n0 = blockIdx.y * kT;
  const int tx = threadIdx.x & 15, ty = threadIdx.x >> 4;
  const int Kb = (a.K + kScaleBlock - 1) / kScaleBlock;
  float acc[4][4] = {};
  for (int kb = 0; kb < Kb; ++kb) {
    float part[4][4] = {};
    const int end = min(a.K, (kb + 1) * kScaleBlock);
    for (int k0 = kb * kScaleBlock; k0 < end; k0 += kStep) {
      for (int i = threadIdx.x; i < kT * kStep; i += 256) {
        const int r = i / kStep, k = i % kStep;
        const bool in = k0 + k < end;
        sa[k][r] = in && m0 + r < a.M ? e4m3_f32(a.a[(m0 + r) * a.lda + k0 + k]) : 0.f;
        sb[k][r] = in && n0 + r < a.N ? e4m3_f32(a.b[(n0 + r) * a.ldb + k0 + k]) : 0.f;
      }
      __syncthreads();
#pragma unroll 8
      for (int k = 0; k < kStep; ++k) {
        float x[4], y[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) x[i] = sa[k][ty + 16 * i], y[i] = sb[k][tx + 16 * i];
#pragma unroll
        for (int i = 0; i < 4; ++i)
#pragma unroll
          for (int j = 0; j < 4; ++j) part[i][j] = fmaf(x[i], y[j], part[i][j]);
      }
      __syncthreads();
    }
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const long long m = m0 + ty + 16 * i;
      const float s = m < a.M ? a.a_s[m * Kb + kb] : 0.f;
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const int n = n0 + tx + 16 * j;
        if (n < a.N) acc[i][j] = fmaf(part[i][j], s * a.b_s[static_cast<long long>(n / kScaleBlock) * Kb + kb], acc[i][j]);
      }
    }
  }
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const long long m = m0 + ty + 16 * i;
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const int n = n0 + tx + 16 * j;
      if (m < a.M && n < a.N) store_out(a, m * a.N + n, acc[i][j]);
    }
  }
}

}  // namespace

cudaError_t launch_fp8_matmul(const Fp8MatmulArgs& a, int num_sms, cudaStream_t stream) {
  (void)num_sms;
  const dim3 grid((a.M + kT - 1) / kT, (a.N + kT - 1) / kT);
  return launch_k(fp8_matmul_plain_kernel, grid, dim3(256), 0, stream, true, a);
}

}  // namespace moe
