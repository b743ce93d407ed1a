// Block quantisers: 8-bit (e4m3) values with one fp32 scale for each 128 columns of a
// row (activations) or each 128 x 128 block (weights).
//
//   s = max(amax / 448, 2^-126),  q = e4m3(x / s)   (nearest, ties to even)
//
// 448 is e4m3's largest value; the floor keeps 1 / s a finite number for blocks that
// are zero or nearly so. The SwiGLU form quantises h = g / (1 + exp(-g)) * u of rows
// [g | u] without storing h. A NaN in a block makes its scale and all its values NaN,
// an infinity its scale infinite and itself NaN, so neither passes unseen.
#include "fp8_quant.cuh"
#include "ops.cuh"

namespace moe {
namespace {

__device__ __forceinline__ float bf16_lo(uint32_t w) { return __uint_as_float(w << 16); }
__device__ __forceinline__ float bf16_hi(uint32_t w) { return __uint_as_float(w & 0xFFFF0000u); }
__device__ __forceinline__ float to_f32(float v) { return v; }
__device__ __forceinline__ float to_f32(uint16_t v) { return __uint_as_float(static_cast<uint32_t>(v) << 16); }

constexpr int kLane = 16;                       // values of a thread
constexpr int kLanes = kScaleBlock / kLane;     // threads to a block of 128 columns

// kLane consecutive values: 32 (bf16) or 64 (fp32) bytes.
__device__ __forceinline__ void load_lane(const uint16_t* p, float (&v)[kLane]) {
  const uint4* q = reinterpret_cast<const uint4*>(p);
  const uint4 t[2] = {q[0], q[1]};
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    v[8 * i + 0] = bf16_lo(t[i].x), v[8 * i + 1] = bf16_hi(t[i].x), v[8 * i + 2] = bf16_lo(t[i].y);
    v[8 * i + 3] = bf16_hi(t[i].y), v[8 * i + 4] = bf16_lo(t[i].z), v[8 * i + 5] = bf16_hi(t[i].z);
    v[8 * i + 6] = bf16_lo(t[i].w), v[8 * i + 7] = bf16_hi(t[i].w);
  }
}
__device__ __forceinline__ void load_lane(const float* p, float (&v)[kLane]) {
#pragma unroll
  for (int i = 0; i < kLane / 4; ++i) {
    const float4 t = reinterpret_cast<const float4*>(p)[i];
    v[4 * i] = t.x, v[4 * i + 1] = t.y, v[4 * i + 2] = t.z, v[4 * i + 3] = t.w;
  }
}

template <bool kSwiglu, bool kVec, typename T>
__device__ __forceinline__ void load_chunk(const T* row, int col, int N, float (&v)[kLane]) {
  if (kVec) {
    if (col < N) {
      load_lane(row + col, v);
      if (kSwiglu) {
        float u[kLane];
        load_lane(row + N + col, u);
#pragma unroll
        for (int i = 0; i < kLane; ++i) v[i] = swiglu(v[i], u[i]);
      }
    } else {
#pragma unroll
      for (int i = 0; i < kLane; ++i) v[i] = 0.f;
    }
  } else {
#pragma unroll
    for (int i = 0; i < kLane; ++i) {
      v[i] = col + i < N ? to_f32(row[col + i]) : 0.f;
      if (kSwiglu) v[i] = swiglu(v[i], col + i < N ? to_f32(row[N + col + i]) : 0.f);
    }
  }
}

template <bool kVec>
__device__ __forceinline__ void store_chunk(uint8_t* q, long long row_at, int col, int N, const float (&v)[kLane],
                                            float s) {
  const bool exact = quotient_ok(s);
  const float r = __frcp_rn(s);
  uint32_t w[kLane / 4];
#pragma unroll
  for (int i = 0; i < kLane / 4; ++i) w[i] = e4m3_quad(v[4 * i], v[4 * i + 1], v[4 * i + 2], v[4 * i + 3], s, r, exact);
  if (kVec) {
    if (col < N) *reinterpret_cast<uint4*>(q + row_at + col) = make_uint4(w[0], w[1], w[2], w[3]);
  } else {
#pragma unroll
    for (int i = 0; i < kLane; ++i)
      if (col + i < N) q[row_at + col + i] = static_cast<uint8_t>(w[i >> 2] >> (8 * (i & 3)));
  }
}

constexpr int kThreads = 256;
constexpr int kPerCta = kThreads / kLanes;  // blocks, or rows of a weight block

// kLanes threads to a block of 128 columns, kLane values each. Bound by memory: 8,191 x
// 2,048 SwiGLU pairs (84 MB) in 14.4 us, 5.9 TB/s (15.2 with 6 CTAs to an SM instead of
// 8). With full-precision exponentials and divisions and eight values a thread its
// instructions bound it: 28 us.
template <bool kSwiglu, bool kVec, typename T>
__global__ void __launch_bounds__(kThreads, 8) quantize_kernel(QuantArgs a, uint32_t blocks) {
  pdl_wait();
  pdl_launch_dependents();
  const uint32_t nb = (a.N + kScaleBlock - 1) / kScaleBlock;
  const uint32_t blk = blockIdx.x * kPerCta + threadIdx.x / kLanes;
  // (lanes without a block stay for the shuffles)
  const bool live = blk < blocks;
  const uint32_t m = live ? blk / nb : 0;
  const int col = static_cast<int>(live ? blk - m * nb : 0) * kScaleBlock + (threadIdx.x % kLanes) * kLane;
  const T* row = static_cast<const T*>(a.x) + m * a.row_stride;
  float v[kLane];
  load_chunk<kSwiglu, kVec>(row, live ? col : a.N, a.N, v);
  float amax = 0.f;
#pragma unroll
  for (int i = 0; i < kLane; ++i) amax = max_nan(amax, v[i]);
#pragma unroll
  for (int off = kLanes / 2; off > 0; off >>= 1) amax = max_nan(amax, __shfl_xor_sync(0xffffffffu, amax, off));
  if (!live) return;
  const float s = block_scale(amax);
  store_chunk<kVec>(a.q, static_cast<long long>(m) * a.N, col, a.N, v, s);
  if (threadIdx.x % kLanes == 0) a.s[blk] = s;
}

// One CTA per 128 x 128 block: kLanes threads to a row.
template <bool kVec, typename T>
__global__ void __launch_bounds__(kThreads) quantize_weight_kernel(QuantArgs a) {
  // (waits for the producer of x, and lets nothing start early: a later kernel may
  // read these weights ahead of its own wait)
  pdl_wait();
  __shared__ float warp_max[kThreads / 32];
  const int kb = blockIdx.x, m0 = blockIdx.y * kScaleBlock;
  const int col = kb * kScaleBlock + (threadIdx.x % kLanes) * kLane;
  const int r0 = threadIdx.x / kLanes;
  float amax = 0.f;
  float v[kLane];
  for (int r = r0; r < kScaleBlock && m0 + r < a.M; r += kPerCta) {
    load_chunk<false, kVec>(static_cast<const T*>(a.x) + (m0 + r) * a.row_stride, col, a.N, v);
#pragma unroll
    for (int i = 0; i < kLane; ++i) amax = max_nan(amax, v[i]);
  }
#pragma unroll
  for (int off = 16; off > 0; off >>= 1) amax = max_nan(amax, __shfl_xor_sync(0xffffffffu, amax, off));
  if ((threadIdx.x & 31) == 0) warp_max[threadIdx.x >> 5] = amax;
  __syncthreads();
#pragma unroll
  for (int i = 0; i < kThreads / 32; ++i) amax = max_nan(amax, warp_max[i]);
  const float s = block_scale(amax);
  for (int r = r0; r < kScaleBlock && m0 + r < a.M; r += kPerCta) {
    load_chunk<false, kVec>(static_cast<const T*>(a.x) + (m0 + r) * a.row_stride, col, a.N, v);
    store_chunk<kVec>(a.q, static_cast<long long>(m0 + r) * a.N, col, a.N, v, s);
  }
  if (threadIdx.x == 0) a.s[static_cast<long long>(blockIdx.y) * gridDim.x + kb] = s;
}

// Whether every thread's values are whole and its loads and stores aligned.
bool vector_ok(const QuantArgs& a) {
  return a.N % kLane == 0 && a.row_stride % (a.x_type == kTypeF32 ? 4 : 8) == 0 &&
         (reinterpret_cast<uintptr_t>(a.x) | reinterpret_cast<uintptr_t>(a.q)) % 16 == 0;
}

// (blocks are counted in 32 bits: rows beyond that go in launches of their own)
template <bool kSwiglu, typename T>
cudaError_t launch_rows(QuantArgs a, cudaStream_t stream) {
  const long long nb = (a.N + kScaleBlock - 1) / kScaleBlock;
  const bool vec = vector_ok(a);
  const int rows = a.M;
  const long long most = (1LL << 30) / nb;
  for (long long m = 0; m < rows; m += most) {
    QuantArgs b = a;
    b.M = static_cast<int>(rows - m < most ? rows - m : most);
    b.x = static_cast<const T*>(a.x) + m * a.row_stride;
    b.q += m * a.N;
    b.s += m * nb;
    const uint32_t blocks = static_cast<uint32_t>(b.M * nb);
    const dim3 grid((blocks + kPerCta - 1) / kPerCta);
    const cudaError_t e =
        vec ? launch_k(quantize_kernel<kSwiglu, true, T>, grid, dim3(kThreads), 0, stream, true, b, blocks)
            : launch_k(quantize_kernel<kSwiglu, false, T>, grid, dim3(kThreads), 0, stream, true, b, blocks);
    if (e != cudaSuccess) return e;
  }
  return cudaSuccess;
}

}  // namespace

cudaError_t launch_quantize(const QuantArgs& a, bool swiglu, cudaStream_t stream) {
  if (a.x_type == kTypeF32) return swiglu ? launch_rows<true, float>(a, stream) : launch_rows<false, float>(a, stream);
  return swiglu ? launch_rows<true, uint16_t>(a, stream) : launch_rows<false, uint16_t>(a, stream);
}

cudaError_t launch_quantize_weight(const QuantArgs& a, cudaStream_t stream) {
  const dim3 grid((a.N + kScaleBlock - 1) / kScaleBlock, (a.M + kScaleBlock - 1) / kScaleBlock);
  const bool vec = vector_ok(a);
  auto go = [&](auto kernel) { return launch_k(kernel, grid, dim3(kThreads), 0, stream, true, a); };
  if (a.x_type == kTypeF32)
    return vec ? go(quantize_weight_kernel<true, float>) : go(quantize_weight_kernel<false, float>);
  return vec ? go(quantize_weight_kernel<true, uint16_t>) : go(quantize_weight_kernel<false, uint16_t>);
}

}  // namespace moe
