// Block quantisers: 8-bit (e4m3) values with one fp32 scale for each 128 columns of a
// row (activations) or each 128 x 128 block (weights).
//
//   s = max(amax / 448, 2^-126),  q = e4m3(x / s)   (nearest, ties to even)
//
// 448 is e4m3's largest value; the floor keeps 1 / s a finite number for blocks that
// are zero or nearly so. The SwiGLU form quantises h = g / (1 + exp(-g)) * u of rows
// [g | u] without storing h. A NaN in a block makes its scale and all its values NaN,
// an infinity its scale infinite and itself NaN, so neither passes unseen.
#include <cuda_fp8.h>

#include "ops.cuh"

namespace moe {
namespace {

constexpr float kE4m3Max = 448.0f;
constexpr float kScaleFloor = 1.17549435e-38f;  // 2^-126

__device__ __forceinline__ float bf16_lo(uint32_t w) { return __uint_as_float(w << 16); }
__device__ __forceinline__ float bf16_hi(uint32_t w) { return __uint_as_float(w & 0xFFFF0000u); }
__device__ __forceinline__ float to_f32(float v) { return v; }
__device__ __forceinline__ float to_f32(uint16_t v) { return __uint_as_float(static_cast<uint32_t>(v) << 16); }

// Eight consecutive values: 16 (bf16) or 32 (fp32) bytes.
__device__ __forceinline__ void load8(const uint16_t* p, float (&v)[8]) {
  const uint4 t = *reinterpret_cast<const uint4*>(p);
  v[0] = bf16_lo(t.x), v[1] = bf16_hi(t.x), v[2] = bf16_lo(t.y), v[3] = bf16_hi(t.y);
  v[4] = bf16_lo(t.z), v[5] = bf16_hi(t.z), v[6] = bf16_lo(t.w), v[7] = bf16_hi(t.w);
}
__device__ __forceinline__ void load8(const float* p, float (&v)[8]) {
  const float4 a = *reinterpret_cast<const float4*>(p), b = *reinterpret_cast<const float4*>(p + 4);
  v[0] = a.x, v[1] = a.y, v[2] = a.z, v[3] = a.w, v[4] = b.x, v[5] = b.y, v[6] = b.z, v[7] = b.w;
}

__device__ __forceinline__ float swiglu(float g, float u) { return g / (1.0f + expf(-g)) * u; }

__device__ __forceinline__ uint32_t magnitude(float v) { return __float_as_uint(v) & 0x7FFFFFFFu; }

// Scale of a block from the largest magnitude's bits (as integers NaN is above
// infinity is above every number, so neither is lost in the maximum).
__device__ __forceinline__ float block_scale(uint32_t amax) {
  const float m = __uint_as_float(amax);
  const float s = __fdiv_rn(m, kE4m3Max);
  return s != s ? s : fmaxf(s, kScaleFloor);
}

__device__ __forceinline__ uint32_t e4m3_pair(float lo, float hi) {
  return __nv_cvt_float2_to_fp8x2(make_float2(lo, hi), __NV_SATFINITE, __NV_E4M3);
}

template <bool kSwiglu, bool kVec, typename T>
__device__ __forceinline__ void load_chunk(const T* row, int col, int N, float (&v)[8]) {
  if (kVec) {
    if (col < N) {
      load8(row + col, v);
      if (kSwiglu) {
        float u[8];
        load8(row + N + col, u);
#pragma unroll
        for (int i = 0; i < 8; ++i) v[i] = swiglu(v[i], u[i]);
      }
    } else {
#pragma unroll
      for (int i = 0; i < 8; ++i) v[i] = 0.f;
    }
  } else {
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      v[i] = col + i < N ? to_f32(row[col + i]) : 0.f;
      if (kSwiglu) v[i] = swiglu(v[i], col + i < N ? to_f32(row[N + col + i]) : 0.f);
    }
  }
}

template <bool kVec>
__device__ __forceinline__ void store_chunk(uint8_t* q, long long row_at, int col, int N, const float (&v)[8],
                                            float s) {
  uint32_t w[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) w[i] = e4m3_pair(__fdiv_rn(v[2 * i], s), __fdiv_rn(v[2 * i + 1], s));
  if (kVec) {
    if (col < N) *reinterpret_cast<uint2*>(q + row_at + col) = make_uint2(w[0] | (w[1] << 16), w[2] | (w[3] << 16));
  } else {
#pragma unroll
    for (int i = 0; i < 8; ++i)
      if (col + i < N) q[row_at + col + i] = static_cast<uint8_t>(w[i >> 1] >> (8 * (i & 1)));
  }
}

// 16 lanes to a block of 128 columns, 8 values each.
template <bool kSwiglu, bool kVec, typename T>
__global__ void __launch_bounds__(256) quantize_kernel(QuantArgs a) {
  pdl_wait();
  pdl_launch_dependents();
  const int nb = (a.N + kScaleBlock - 1) / kScaleBlock;
  const long long blk = static_cast<long long>(blockIdx.x) * 16 + (threadIdx.x >> 4);
  // (lanes of a warp's idle half stay for the shuffles)
  const bool live = blk < static_cast<long long>(a.M) * nb;
  const long long m = live ? blk / nb : 0;
  const int kb = live ? static_cast<int>(blk % nb) : 0;
  const int col = kb * kScaleBlock + (threadIdx.x & 15) * 8;
  const T* row = static_cast<const T*>(a.x) + m * a.row_stride;
  float v[8];
  load_chunk<kSwiglu, kVec>(row, live ? col : a.N, a.N, v);
  uint32_t amax = 0;
#pragma unroll
  for (int i = 0; i < 8; ++i) amax = max(amax, magnitude(v[i]));
#pragma unroll
  for (int off = 8; off > 0; off >>= 1) amax = max(amax, __shfl_xor_sync(0xffffffffu, amax, off));
  if (!live) return;
  const float s = block_scale(amax);
  store_chunk<kVec>(a.q, m * a.N, col, a.N, v, s);
  if ((threadIdx.x & 15) == 0) a.s[blk] = s;
}

// One CTA per 128 x 128 block: 16 lanes to a row, 16 rows at a time.
template <bool kVec, typename T>
__global__ void __launch_bounds__(256) quantize_weight_kernel(QuantArgs a) {
  // (waits for the producer of x, and lets nothing start early: a later kernel may
  // read these weights ahead of its own wait)
  pdl_wait();
  __shared__ uint32_t warp_max[8];
  const int kb = blockIdx.x, m0 = blockIdx.y * kScaleBlock;
  const int col = kb * kScaleBlock + (threadIdx.x & 15) * 8;
  const int r0 = threadIdx.x >> 4;
  uint32_t amax = 0;
  float v[8];
  for (int r = r0; r < kScaleBlock && m0 + r < a.M; r += 16) {
    load_chunk<false, kVec>(static_cast<const T*>(a.x) + (m0 + r) * a.row_stride, col, a.N, v);
#pragma unroll
    for (int i = 0; i < 8; ++i) amax = max(amax, magnitude(v[i]));
  }
  amax = __reduce_max_sync(0xffffffffu, amax);
  if ((threadIdx.x & 31) == 0) warp_max[threadIdx.x >> 5] = amax;
  __syncthreads();
#pragma unroll
  for (int i = 0; i < 8; ++i) amax = max(amax, warp_max[i]);
  const float s = block_scale(amax);
  for (int r = r0; r < kScaleBlock && m0 + r < a.M; r += 16) {
    load_chunk<false, kVec>(static_cast<const T*>(a.x) + (m0 + r) * a.row_stride, col, a.N, v);
    store_chunk<kVec>(a.q, static_cast<long long>(m0 + r) * a.N, col, a.N, v, s);
  }
  if (threadIdx.x == 0) a.s[static_cast<long long>(blockIdx.y) * gridDim.x + kb] = s;
}

// Whether every chunk of eight values is whole and its loads and stores aligned.
bool vector_ok(const QuantArgs& a) {
  return a.N % 8 == 0 && a.row_stride % 8 == 0 && reinterpret_cast<uintptr_t>(a.x) % 16 == 0 &&
         reinterpret_cast<uintptr_t>(a.q) % 8 == 0;
}

template <bool kSwiglu, typename T>
cudaError_t launch_rows(const QuantArgs& a, cudaStream_t stream) {
  const long long blocks = static_cast<long long>(a.M) * ((a.N + kScaleBlock - 1) / kScaleBlock);
  const dim3 grid(static_cast<unsigned>((blocks + 15) / 16));
  return vector_ok(a) ? launch_k(quantize_kernel<kSwiglu, true, T>, grid, dim3(256), 0, stream, true, a)
                      : launch_k(quantize_kernel<kSwiglu, false, T>, grid, dim3(256), 0, stream, true, a);
}

}  // namespace

cudaError_t launch_quantize(const QuantArgs& a, bool swiglu, cudaStream_t stream) {
  if (a.x_type == kTypeF32) return swiglu ? launch_rows<true, float>(a, stream) : launch_rows<false, float>(a, stream);
  return swiglu ? launch_rows<true, uint16_t>(a, stream) : launch_rows<false, uint16_t>(a, stream);
}

cudaError_t launch_quantize_weight(const QuantArgs& a, cudaStream_t stream) {
  const dim3 grid((a.N + kScaleBlock - 1) / kScaleBlock, (a.M + kScaleBlock - 1) / kScaleBlock);
  const bool vec = vector_ok(a);
  auto go = [&](auto kernel) { return launch_k(kernel, grid, dim3(256), 0, stream, true, a); };
  if (a.x_type == kTypeF32)
    return vec ? go(quantize_weight_kernel<true, float>) : go(quantize_weight_kernel<false, float>);
  return vec ? go(quantize_weight_kernel<true, uint16_t>) : go(quantize_weight_kernel<false, uint16_t>);
}

}  // namespace moe
