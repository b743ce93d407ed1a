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

#include "fp8_tma.cuh"

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

// ---------------------------------------------------------------- few rows
//
// A batch of few rows reads every weight once and does little with it: the weights are
// the MMA's 128 rows (M) and the batch its columns (N = 16 .. 128), so one token costs
// 16 columns, not 128 rows. A tile's reduction is split over the CTAs of a cluster, so
// that every SM streams weights; the fp32 partial sums meet in distributed shared memory
// and are added in the order of the ranks (the same result every time).
//
// Warps of a CTA: 0 copies (one lane; a stage is 128 x 128 weight bytes and the batch's
// 128 bytes per row), 1 issues the MMAs (four of 32 reduction elements for a block) into
// one of kAccs accumulators, 2..5 take the block sum out of tensor memory, scale it and
// add it to the running sum in registers (thread = weight row).
constexpr int kFewThreads = 6 * 32;
constexpr int kFewEpi = 128;
constexpr int kWTile = 128 * 128;  // bytes of a weight box
constexpr int kScaleRun = 32;      // blocks whose scales are staged at a time

__device__ int32_t g_fp8_status;

struct FewLayout {  // shared memory
  int stages, stage_bytes, scales, bars, total;
};
constexpr int kMaxStages = 10;
template <int kChunks>
__host__ __device__ constexpr FewLayout few_layout() {
  FewLayout L{};
  const int bt = 16 * kChunks;
  L.stage_bytes = kWTile + bt * 128;
  // two CTAs to an SM while the registers allow it
  const int room = (kChunks <= 2 ? 113 : 226) * 1024 - 1024;
  const int fixed = kScaleRun * bt * 4 + 512;
  L.stages = (room - fixed) / L.stage_bytes;
  if (L.stages > kMaxStages) L.stages = kMaxStages;
  L.scales = L.stages * L.stage_bytes;
  L.bars = L.scales + kScaleRun * bt * 4;
  L.total = L.bars + 512 + 1024;  // (1,024: the base is rounded up to the swizzle atom)
  return L;
}
template <int kChunks>
__host__ __device__ constexpr int few_accs() { return kChunks <= 4 ? 4 : 2; }

template <int kChunks>
__global__ void __launch_bounds__(kFewThreads)
    fp8_matmul_few_kernel(const __grid_constant__ CUtensorMap wmap, const __grid_constant__ CUtensorMap xmap,
                          const __grid_constant__ Fp8MatmulArgs a, int bt, int split, int32_t* status) {
  constexpr FewLayout L = few_layout<kChunks>();
  constexpr int kAccs = few_accs<kChunks>();
  constexpr int kCols = kAccs * 16 * kChunks < 32 ? 32 : kAccs * 16 * kChunks;
  static_assert(L.stages >= 2 && 8 * (2 * L.stages + 2 * kAccs + 1) + 8 <= 512, "shared memory layout");
  // the reduction reuses the stages
  static_assert(L.stages * L.stage_bytes >= 16 * kChunks * 128 * 4, "partial sums fit the stages");
  extern __shared__ uint8_t smem_raw[];
  const uint32_t base = (smem_u32(smem_raw) + 1023u) & ~1023u;
  uint8_t* gbase = smem_raw + (base - smem_u32(smem_raw));
  float* scales = reinterpret_cast<float*>(gbase + L.scales);  // [kScaleRun][bt max]
  auto full = [&](int i) { return base + L.bars + 8 * i; };
  auto empty = [&](int i) { return base + L.bars + 8 * (L.stages + i); };
  auto tfull = [&](int i) { return base + L.bars + 8 * (2 * L.stages + i); };
  auto tempty = [&](int i) { return base + L.bars + 8 * (2 * L.stages + kAccs + i); };
  const uint32_t drain = base + L.bars + 8 * (2 * L.stages + 2 * kAccs);
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(gbase + L.bars + 8 * (2 * L.stages + 2 * kAccs + 1));
  volatile int* abort_flag = reinterpret_cast<volatile int*>(tmem_slot + 1);

  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int rank = split > 1 ? static_cast<int>(cluster_rank()) : 0;
  const int n0 = static_cast<int>(blockIdx.x / split) * 128;
  const long long m0 = static_cast<long long>(blockIdx.y) * bt;
  const int Kb = (a.K + kScaleBlock - 1) / kScaleBlock;
  const int kb0 = static_cast<int>(static_cast<long long>(Kb) * rank / split);
  const int kb1 = static_cast<int>(static_cast<long long>(Kb) * (rank + 1) / split);
  const uint32_t bytes = kWTile + bt * 128;
  const uint32_t limit = kWaitLimitKCyclesDefault;

  if (threadIdx.x == 0) {
    tma_prefetch_map(&wmap);
    tma_prefetch_map(&xmap);
    for (int i = 0; i < L.stages; ++i) mbar_init(full(i), 1), mbar_init(empty(i), 1);
    for (int i = 0; i < kAccs; ++i) mbar_init(tfull(i), 1), mbar_init(tempty(i), 4);
    mbar_init(drain, 1);
    *abort_flag = 0;
    fence_mbar_init();
  }
  if (warp == 1) {
    __syncwarp();
    tmem_alloc(smem_u32(tmem_slot), kCols);
    tmem_relinquish();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = *tmem_slot;

  if (warp == 0) {
    if (lane == 0) {
      const uint64_t once = l2_policy_evict_first(), keep = l2_policy_evict_last();
      // weights that no preceding kernel of this call writes may stream ahead of the wait
      int ahead = 0;
      if (a.weights_ready)
        for (; ahead < L.stages && kb0 + ahead < kb1; ++ahead) {
          mbar_arrive_expect_tx(full(ahead), bytes);
          tma_load_2d(base + ahead * L.stage_bytes, &wmap, (kb0 + ahead) * 128, n0, full(ahead), once);
        }
      pdl_wait();
      int st = 0, it = 0;
      uint32_t ph = 0;
      for (int kb = kb0; kb < kb1; ++kb, ++it) {
        if (it >= ahead) {
          if (!mbar_wait(empty(st), ph ^ 1u, abort_flag, status, kStatusTimeout, limit)) break;
          mbar_arrive_expect_tx(full(st), bytes);
          tma_load_2d(base + st * L.stage_bytes, &wmap, kb * 128, n0, full(st), once);
        }
        tma_load_2d(base + st * L.stage_bytes + kWTile, &xmap, kb * 128, static_cast<int>(m0), full(st), keep);
        if (++st == L.stages) st = 0, ph ^= 1u;
      }
      // shared memory is released only after the last copies have landed, whoever gave up
      for (int i = it > L.stages ? it - L.stages : 0; i < it; ++i) mbar_drain(full(i % L.stages), (i / L.stages) & 1);
    }
  } else if (warp == 1) {
    const uint32_t idesc = idesc_e4m3_f32(128, bt);
    const bool leader = elect_one();
    int st = 0, ac = 0;
    uint32_t ph = 0, aph = 0;
    for (int kb = kb0; kb < kb1; ++kb) {
      // (the lanes decide together, so that none leaves the loop alone)
      if (!__all_sync(0xffffffffu, mbar_wait(tempty(ac), aph ^ 1u, abort_flag, status, kStatusTimeout, limit) &&
                                       mbar_wait(full(st), ph, abort_flag, status, kStatusTimeout, limit)))
        break;
      tc_fence_after();
      if (leader) {
        const uint64_t wd = sw128_kmajor_desc(base + st * L.stage_bytes);
        const uint64_t xd = sw128_kmajor_desc(base + st * L.stage_bytes + kWTile);
        const uint32_t d = tmem + ac * 16 * kChunks;
#pragma unroll
        for (int i = 0; i < 4; ++i)  // (32 bytes on: 2 descriptor units)
          tc_mma_e4m3(d, wd + 2 * i, xd + 2 * i, idesc, i > 0);
        tc_commit(empty(st));
        tc_commit(tfull(ac));
      }
      __syncwarp();
      if (++st == L.stages) st = 0, ph ^= 1u;
      if (++ac == kAccs) ac = 0, aph ^= 1u;
    }
    if (leader) {  // tensor memory is freed only after the last MMAs, whoever gave up
      tc_commit(drain);
      mbar_drain(drain, 0);
    }
    __syncwarp();
  } else {
    pdl_wait();
    if (warp == 2 && lane == 0) pdl_launch_dependents();
    const int tid = threadIdx.x - 64;
    const int row = (warp & 3) * 32 + lane;
    const int n = n0 + row;
    const uint32_t t_lane = static_cast<uint32_t>((warp & 3) * 32) << 16;
    const int rows = static_cast<int>(a.M - m0 < bt ? a.M - m0 : bt);
    const int chunks = bt / 16;
    float acc[16 * kChunks];
#pragma unroll
    for (int j = 0; j < 16 * kChunks; ++j) acc[j] = 0.f;
    int ac = 0;
    uint32_t aph = 0;
    bool ok = true;  // (a warp that gave up goes on without sums: the others meet it at the barrier)
    for (int kb = kb0; kb < kb1; ++kb) {
      const int at = (kb - kb0) % kScaleRun;
      if (at == 0) {  // both scales of the next blocks, multiplied
        const int run = min(kScaleRun, kb1 - kb);
        named_bar_sync(1, kFewEpi);
        for (int i = tid; i < run * bt; i += kFewEpi) {
          const int j = i / run, k = i % run;
          scales[k * bt + j] = j < rows ? a.a_s[(m0 + j) * Kb + kb + k] *
                                              a.b_s[static_cast<long long>(n0 / kScaleBlock) * Kb + kb + k]
                                        : 0.f;
        }
        named_bar_sync(1, kFewEpi);
      }
      ok = ok && __all_sync(0xffffffffu, mbar_wait(tfull(ac), aph, abort_flag, status, kStatusTimeout, limit));
      if (!ok) continue;
      tc_fence_after();
#pragma unroll
      for (int c = 0; c < kChunks; ++c) {
        if (c >= chunks) break;
        uint32_t v[16];
        tmem_ld16(tmem + t_lane + ac * 16 * kChunks + 16 * c, v);
        tmem_ld_wait();
        const float4* sc = reinterpret_cast<const float4*>(scales + at * bt + 16 * c);
#pragma unroll
        for (int q = 0; q < 4; ++q) {
          const float4 s4 = sc[q];
          acc[16 * c + 4 * q + 0] = fmaf(__uint_as_float(v[4 * q + 0]), s4.x, acc[16 * c + 4 * q + 0]);
          acc[16 * c + 4 * q + 1] = fmaf(__uint_as_float(v[4 * q + 1]), s4.y, acc[16 * c + 4 * q + 1]);
          acc[16 * c + 4 * q + 2] = fmaf(__uint_as_float(v[4 * q + 2]), s4.z, acc[16 * c + 4 * q + 2]);
          acc[16 * c + 4 * q + 3] = fmaf(__uint_as_float(v[4 * q + 3]), s4.w, acc[16 * c + 4 * q + 3]);
        }
      }
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive(tempty(ac));
      if (++ac == kAccs) ac = 0, aph ^= 1u;
    }
    if (split == 1) {
      if (n < a.N)
#pragma unroll
        for (int j = 0; j < 16 * kChunks; ++j)
          if (j < rows) store_out(a, (m0 + j) * a.N + n, acc[j]);
    } else {
      // (every MMA is done -- the last accumulator was waited for -- so the stages are free)
      float* part = reinterpret_cast<float*>(gbase);
#pragma unroll
      for (int j = 0; j < 16 * kChunks; ++j)
        if (j < rows) part[j * 128 + row] = acc[j];
    }
  }
  __syncwarp();
  tc_fence_before();
  if (split > 1) {
    cluster_sync();
    if (warp >= 2) {
      const int row = (warp & 3) * 32 + lane;
      const int rows = static_cast<int>(a.M - m0 < bt ? a.M - m0 : bt);
      for (int j = rank; j < rows; j += split) {
        float y = 0.f;
        for (int r = 0; r < split; ++r) y += ld_cluster_f32(map_rank(base + (j * 128 + row) * 4, r));
        if (n0 + row < a.N) store_out(a, (m0 + j) * a.N + n0 + row, y);
      }
    }
    __syncwarp();
    cluster_sync();  // no CTA leaves while another reads its sums
  } else {
    __syncthreads();
  }
  if (warp == 1) {
    __syncwarp();
    tc_fence_after();
    tmem_dealloc(tmem, kCols);
  }
}

// ---------------------------------------------------------------- host

template <int kChunks>
cudaError_t launch_few(const Fp8MatmulArgs& a, int bt, int split, int32_t* status, cudaStream_t stream) {
  constexpr FewLayout L = few_layout<kChunks>();
  static cudaError_t set = cudaFuncSetAttribute(fp8_matmul_few_kernel<kChunks>,
                                                cudaFuncAttributeMaxDynamicSharedMemorySize, L.total);
  if (set != cudaSuccess) return set;
  CUtensorMap wmap, xmap;
  if (!make_byte_map(&wmap, a.b, a.N, a.K, a.ldb, 128) || !make_byte_map(&xmap, a.a, a.M, a.K, a.lda, bt))
    return cudaErrorInvalidValue;
  const dim3 grid(static_cast<unsigned>((a.N + 127) / 128 * split), static_cast<unsigned>((a.M + bt - 1) / bt));
  return launch_cluster(fp8_matmul_few_kernel<kChunks>, grid, dim3(kFewThreads), L.total, stream, split, wmap, xmap, a,
                        bt, split, status);
}

}  // namespace

bool make_byte_map(CUtensorMap* map, const void* base, long long rows, long long cols, long long stride, int box_rows) {
  using Encode = CUresult (*)(CUtensorMap*, CUtensorMapDataType, cuuint32_t, void*, const cuuint64_t*,
                              const cuuint64_t*, const cuuint32_t*, const cuuint32_t*, CUtensorMapInterleave,
                              CUtensorMapSwizzle, CUtensorMapL2promotion, CUtensorMapFloatOOBfill);
  static const Encode encode = [] {
    void* fn = nullptr;
    cudaDriverEntryPointQueryResult found{};
    const cudaError_t e = cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &fn, 12000, cudaEnableDefault, &found);
    return e == cudaSuccess && found == cudaDriverEntryPointSuccess ? reinterpret_cast<Encode>(fn) : nullptr;
  }();
  if (!encode) return false;
  const cuuint64_t dims[2] = {static_cast<cuuint64_t>(cols), static_cast<cuuint64_t>(rows)};
  const cuuint64_t strides[1] = {static_cast<cuuint64_t>(rows > 1 ? stride : (cols + 15) / 16 * 16)};
  const cuuint32_t box[2] = {128, static_cast<cuuint32_t>(box_rows)}, step[2] = {1, 1};
  return encode(map, CU_TENSOR_MAP_DATA_TYPE_UINT8, 2, const_cast<void*>(base), dims, strides, box, step,
                CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

namespace {
// Whether the tensor copies can read the operands: 16-byte rows and addresses.
bool tma_ok(const Fp8MatmulArgs& a) {
  return a.K % 16 == 0 && (a.M == 1 || a.lda % 16 == 0) && (a.N == 1 || a.ldb % 16 == 0) &&
         (reinterpret_cast<uintptr_t>(a.a) | reinterpret_cast<uintptr_t>(a.b)) % 16 == 0;
}
}  // namespace

cudaError_t launch_fp8_matmul(const Fp8MatmulArgs& a, int num_sms, cudaStream_t stream) {
  if (!tma_ok(a)) {
    const dim3 grid((a.M + kT - 1) / kT, (a.N + kT - 1) / kT);
    return launch_k(fp8_matmul_plain_kernel, grid, dim3(256), 0, stream, true, a);
  }
  int32_t* status = fp8_status_word();
  if (!status) return cudaErrorInvalidSymbol;
  if (a.M > 128) return launch_fp8_many(a, status, num_sms, stream);
  const int Kb = (a.K + kScaleBlock - 1) / kScaleBlock;
  // tokens a tile: the batch in equal parts of at most 128, in steps of 16
  const long long parts = (static_cast<long long>(a.M) + 127) / 128;
  const int bt = static_cast<int>(((a.M + parts - 1) / parts + 15) / 16 * 16);
  const long long tiles = (a.N + 127) / 128 * ((static_cast<long long>(a.M) + bt - 1) / bt);
  const long long slots = static_cast<long long>(num_sms) * (bt <= 32 ? 2 : 1);
  int split = 1;
  while (split < 8 && tiles * split * 2 <= slots && Kb >= 2 * split * 2) split *= 2;
  if (bt <= 16) return launch_few<1>(a, bt, split, status, stream);
  if (bt <= 32) return launch_few<2>(a, bt, split, status, stream);
  if (bt <= 64) return launch_few<4>(a, bt, split, status, stream);
  return launch_few<8>(a, bt, split, status, stream);
}

int32_t* fp8_status_word() {
  // (one context per device in a process; asked once per device)
  static int32_t* cached[64];
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess) return nullptr;
  if (dev >= 0 && dev < 64 && cached[dev]) return cached[dev];
  void* p = nullptr;
  if (cudaGetSymbolAddress(&p, g_fp8_status) != cudaSuccess) return nullptr;
  if (dev >= 0 && dev < 64) cached[dev] = static_cast<int32_t*>(p);
  return static_cast<int32_t*>(p);
}

cudaError_t fp8_status(int32_t* out, cudaStream_t stream) {
  int32_t* p = fp8_status_word();
  if (!p) return cudaErrorInvalidSymbol;
  cudaError_t e = cudaMemcpyAsync(out, p, sizeof(*p), cudaMemcpyDeviceToHost, stream);
  if (e == cudaSuccess) e = cudaMemsetAsync(p, 0, sizeof(*p), stream);
  if (e == cudaSuccess) e = cudaStreamSynchronize(stream);
  return e;
}

}  // namespace moe
