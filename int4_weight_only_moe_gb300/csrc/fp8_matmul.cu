// 8-bit block-scaled matrix product
//
//   out[m, n] = sum_kb a_s[m, kb] b_s[n / 128, kb] sum_{k in block kb} a[m, k] b[n, k]
//               (+ add[m, n])
//
// with e4m3 operands, a scale for each 128 values of a row of `a` and for each 128 x 128
// block of `b`. A block's products are summed in fp32 unscaled; the scaled block sums
// are added in fp32 and rounded once to the output type.
#include <cuda_bf16.h>

#include "fp8_quant.cuh"
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
  const uint32_t tiles_m = (static_cast<uint32_t>(a.M) + kT - 1) / kT;
  const long long m0 = static_cast<long long>(blockIdx.x % tiles_m) * kT;
  const long long n0 = static_cast<long long>(blockIdx.x / tiles_m) * kT;
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
        const long long n = n0 + tx + 16 * j;
        if (n < a.N) acc[i][j] = fmaf(part[i][j], s * a.b_s[n / kScaleBlock * Kb + kb], acc[i][j]);
      }
    }
  }
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const long long m = m0 + ty + 16 * i;
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const long long n = n0 + tx + 16 * j;
      if (m < a.M && n < a.N) store_out(a, m * a.N + n, acc[i][j]);
    }
  }
}

// ---------------------------------------------------------------- few rows
//
// A batch of few rows reads every weight once and does little with it. Up to 64 rows the
// weights are the MMA's 128 rows (M) and the batch its columns (N = 16, 32 or 64), so one
// token costs 16 columns, not 128 rows, and a thread sums one weight row over the batch.
// From 65 rows on the batch is the MMA's 128 rows and 128 weights its columns: a thread
// sums one batch row, whose scale is one number a block (with the weights as rows it has
// one for each column, and 128 columns took 850 cycles a block; 64 columns pay: 33 x 7,168
// x 2,048 takes 6.5 us, 7.6 with the batch as rows). A tile's reduction is split over the
// CTAs of a cluster, so that every SM streams weights; the fp32 partial sums meet in
// distributed shared memory and are added in the order of the ranks (the same result every
// time). Sent by bulk copies instead of read where they are added they took 0.3 us longer.
//
// Warps of a CTA: the first four (eight from 64 rows on, half of the columns each) take
// the block sums out of tensor memory, scale them and add them to the running sums in
// registers; then one that copies (one lane; a stage is 128 x 128 weight bytes and the
// batch's 128 bytes per row) and one that issues the MMAs (four of 32 reduction elements
// for a block) into four accumulators in turn.
//
// The SwiGLU form carries two weight boxes, 128 gate rows and the 128 up rows of the same
// features: where the partial sums meet, a warp holds both for a whole scale block of 128
// features of a batch row, and writes SiLU(gate) * up as e4m3 with its scale.
constexpr int kWTile = 128 * 128;  // bytes of a weight box
constexpr int kMaxStages = 10;

__device__ int32_t g_fp8_status;

template <int kRows, bool kSwiglu>  // batch rows of a tile: 16, 32, 64 or 128
struct Few {
  static constexpr bool kBatchIsM = kRows == 128;
  static constexpr int kW = kSwiglu ? 2 : 1;               // weight boxes
  static constexpr int kBoxCols = kBatchIsM ? 128 : kRows;  // accumulator columns of a box
  static constexpr int kAccCols = kW * kBoxCols;
  // CTAs to an SM, by registers and shared memory
  static constexpr int kPerSm = kBatchIsM || (kRows == 64 && kSwiglu) ? 1 : 2;
  static constexpr int kCols = 512 / kPerSm;  // of tensor memory
  static constexpr int kAccs = 4 * kAccCols <= kCols ? 4 : kCols / kAccCols;
  static constexpr int kTmem = kAccs * kAccCols;
  static constexpr int kEpiWarps = kRows >= 64 ? 8 : 4;
  static constexpr int kEpiThreads = kEpiWarps * 32;
  static constexpr int kThreads = kEpiThreads + 64;
  static constexpr int kMine = kBoxCols / (kEpiWarps / 4);  // columns of a box for a thread
  static constexpr int kPiece = kMine < 32 ? kMine : 32;
  static constexpr int kStageBytes = kW * kWTile + kRows * 128;
  static constexpr int kRoom = 226 * 1024 / kPerSm;
  static constexpr int kScaleRun = kBatchIsM && kSwiglu ? 16 : 32;  // blocks whose scales are staged at a time
  static constexpr int kScaleRow = kRows + 4;  // (padded: the staging's stores spread over the banks)
  static constexpr int kScaleBox = kScaleRun * kScaleRow;
  static constexpr int kFixed = kW * kScaleBox * 4 + 512 + 1024;  // (1,024: up to the swizzle atom)
  static constexpr int kFit = (kRoom - kFixed) / kStageBytes;
  static constexpr int kStages = kFit < kMaxStages ? kFit : kMaxStages;
  static constexpr int kScales = kStages * kStageBytes;
  static constexpr int kBars = kScales + kW * kScaleBox * 4;
  static constexpr int kSmem = kBars + 512 + 1024;
  static constexpr int kPart = kRows * 512;  // partial sums of a box
  static_assert(kStages >= 2 && 8 * (2 * kStages + 2 * kAccs + 2) + 8 <= 512, "barriers");
  static_assert(kStages * kStageBytes >= kW * kPart, "the partial sums fit the stages");
};

__device__ __forceinline__ void tmem_piece(uint32_t src, uint32_t (&v)[16]) { tmem_ld16(src, v); }
__device__ __forceinline__ void tmem_piece(uint32_t src, uint32_t (&v)[32]) { tmem_ld32(src, v); }

// Byte offset of weights 4 c .. 4 c + 3 in row j of the partial sums.
__device__ __forceinline__ uint32_t part_at(int j, int c) { return j * 512 + ((c ^ (j & 7)) << 4); }
__device__ __forceinline__ float4 ld_cluster_v4(uint32_t addr) {
  float4 v;
  asm volatile("ld.shared::cluster.v4.f32 {%0, %1, %2, %3}, [%4];"
               : "=f"(v.x), "=f"(v.y), "=f"(v.z), "=f"(v.w)
               : "r"(addr)
               : "memory");
  return v;
}

// Sum of four weights' partial sums over the cluster's CTAs, in the order of the ranks.
// All loads are under way before the first addition (one after the other they cost 0.25
// us each).
template <int kSplit>
__device__ __forceinline__ float4 join_sums(uint32_t at) {
  float4 v[kSplit];
#pragma unroll
  for (int r = 0; r < kSplit; ++r) v[r] = ld_cluster_v4(kSplit > 1 ? map_rank(at, r) : at);
  float4 y = v[0];
#pragma unroll
  for (int r = 1; r < kSplit; ++r) y.x += v[r].x, y.y += v[r].y, y.z += v[r].z, y.w += v[r].w;
  return y;
}
__device__ __forceinline__ void join_pair(uint32_t at0, uint32_t at1, int split, float4* y0, float4* y1) {
  switch (split) {
    case 8: *y0 = join_sums<8>(at0), *y1 = join_sums<8>(at1); break;
    case 7: *y0 = join_sums<7>(at0), *y1 = join_sums<7>(at1); break;
    case 6: *y0 = join_sums<6>(at0), *y1 = join_sums<6>(at1); break;
    case 5: *y0 = join_sums<5>(at0), *y1 = join_sums<5>(at1); break;
    case 4: *y0 = join_sums<4>(at0), *y1 = join_sums<4>(at1); break;
    case 3: *y0 = join_sums<3>(at0), *y1 = join_sums<3>(at1); break;
    case 2: *y0 = join_sums<2>(at0), *y1 = join_sums<2>(at1); break;
    default: *y0 = join_sums<1>(at0), *y1 = join_sums<1>(at1);
  }
}

// Four consecutive outputs; `vec`: whole and aligned for one access.
__device__ __forceinline__ void store_out4(const Fp8MatmulArgs& a, long long m, int n, float4 y, bool vec) {
  const long long at = m * a.N + n;
  if (!vec) {
    float v[4] = {y.x, y.y, y.z, y.w};
    if (n >= a.N) return;
    if (a.add) {  // (all loads before the first store, which may be to the same array, and none conditional)
      uint16_t d[4];
#pragma unroll
      for (int i = 0; i < 4; ++i) d[i] = a.add[at + min(i, a.N - 1 - n)];
#pragma unroll
      for (int i = 0; i < 4; ++i) v[i] += __uint_as_float(static_cast<uint32_t>(d[i]) << 16);
    }
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      if (n + i >= a.N) break;
      if (a.out_type == kTypeF32)
        static_cast<float*>(a.out)[at + i] = v[i];
      else
        static_cast<__nv_bfloat16*>(a.out)[at + i] = __float2bfloat16_rn(v[i]);
    }
    return;
  }
  if (n >= a.N) return;
  if (a.add) {
    const uint2 d = *reinterpret_cast<const uint2*>(a.add + at);
    y.x += __uint_as_float(d.x << 16), y.y += __uint_as_float(d.x & 0xFFFF0000u);
    y.z += __uint_as_float(d.y << 16), y.w += __uint_as_float(d.y & 0xFFFF0000u);
  }
  if (a.out_type == kTypeF32) {
    *reinterpret_cast<float4*>(static_cast<float*>(a.out) + at) = y;
  } else {
    const __nv_bfloat162 lo = __floats2bfloat162_rn(y.x, y.y), hi = __floats2bfloat162_rn(y.z, y.w);
    *reinterpret_cast<uint2*>(static_cast<uint16_t*>(a.out) + at) =
        make_uint2(*reinterpret_cast<const uint32_t*>(&lo), *reinterpret_cast<const uint32_t*>(&hi));
  }
}

template <int kRows, bool kSwiglu>
__global__ void __launch_bounds__(Few<kRows, kSwiglu>::kThreads)
    fp8_matmul_few_kernel(const __grid_constant__ CUtensorMap wmap, const __grid_constant__ CUtensorMap xmap,
                          const __grid_constant__ Fp8MatmulArgs a, int split, bool vec, int32_t* status) {
  using L = Few<kRows, kSwiglu>;
  extern __shared__ uint8_t smem_raw[];
  const uint32_t base = (smem_u32(smem_raw) + 1023u) & ~1023u;
  uint8_t* gbase = smem_raw + (base - smem_u32(smem_raw));
  float* scales = reinterpret_cast<float*>(gbase + L::kScales);  // [kW][kScaleRun][kScaleRow]
  auto full = [&](int i) { return base + L::kBars + 8 * i; };
  auto empty = [&](int i) { return base + L::kBars + 8 * (L::kStages + i); };
  auto tfull = [&](int i) { return base + L::kBars + 8 * (2 * L::kStages + i); };
  auto tempty = [&](int i) { return base + L::kBars + 8 * (2 * L::kStages + L::kAccs + i); };
  const uint32_t drain = base + L::kBars + 8 * (2 * L::kStages + 2 * L::kAccs);
  const uint32_t never = drain + 8;  // (the test hook's)
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(gbase + L::kBars + 8 * (2 * L::kStages + 2 * L::kAccs + 2));
  volatile int* abort_flag = reinterpret_cast<volatile int*>(tmem_slot + 1);
  constexpr int kWarpTma = L::kEpiWarps, kWarpMma = L::kEpiWarps + 1;

  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int rank = split > 1 ? static_cast<int>(cluster_rank()) : 0;
  const int n0 = static_cast<int>(blockIdx.x / split) * 128;
  const long long m0 = static_cast<long long>(blockIdx.y) * kRows;
  const int rows = static_cast<int>(a.M - m0 < kRows ? a.M - m0 : kRows);
  const int Kb = (a.K + kScaleBlock - 1) / kScaleBlock;
  const int kb0 = static_cast<int>(static_cast<long long>(Kb) * rank / split);
  const int kb1 = static_cast<int>(static_cast<long long>(Kb) * (rank + 1) / split);
  constexpr uint32_t bytes = L::kStageBytes;
  const uint32_t limit = a.wait_kcycles;

  if (threadIdx.x == 0) {
    tma_prefetch_map(&wmap);
    tma_prefetch_map(&xmap);
    for (int i = 0; i < L::kStages; ++i) mbar_init(full(i), 1), mbar_init(empty(i), 1);
    for (int i = 0; i < L::kAccs; ++i) mbar_init(tfull(i), 1), mbar_init(tempty(i), L::kEpiWarps);
    mbar_init(drain, 1);
    mbar_init(never, 1);
    *abort_flag = 0;
    fence_mbar_init();
  }
  if (warp == kWarpMma) {
    __syncwarp();
    tmem_alloc(smem_u32(tmem_slot), L::kTmem);
    tmem_relinquish();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = *tmem_slot;

  if (warp == kWarpTma) {
    if (lane == 0) {
      const uint64_t once = l2_policy_evict_first(), keep = l2_policy_evict_last();
      // weights that no preceding kernel of this call writes may stream ahead of the wait
      int ahead = 0;
      if (a.weights_ready)
        for (; ahead < L::kStages && kb0 + ahead < kb1; ++ahead) {
          mbar_arrive_expect_tx(full(ahead), bytes);
#pragma unroll
          for (int w = 0; w < L::kW; ++w)
            tma_load_2d(base + ahead * L::kStageBytes + w * kWTile, &wmap, (kb0 + ahead) * 128, n0 + w * a.N, full(ahead),
                        once);
        }
      pdl_wait();
      int st = 0, it = 0;
      uint32_t ph = 0;
      for (int kb = kb0; kb < kb1; ++kb, ++it) {
        if (it >= ahead) {
          if (!mbar_wait(empty(st), ph ^ 1u, abort_flag, status, kStatusTimeout, limit)) break;
          mbar_arrive_expect_tx(full(st), bytes);
#pragma unroll
          for (int w = 0; w < L::kW; ++w)
            tma_load_2d(base + st * L::kStageBytes + w * kWTile, &wmap, kb * 128, n0 + w * a.N, full(st), once);
        }
        tma_load_2d(base + st * L::kStageBytes + L::kW * kWTile, &xmap, kb * 128, static_cast<int>(m0), full(st), keep);
        if (++st == L::kStages) st = 0, ph ^= 1u;
      }
      // shared memory is released only after the last copies have landed, whoever gave up
      for (int i = it > L::kStages ? it - L::kStages : 0; i < it; ++i)
        mbar_drain(full(i % L::kStages), (i / L::kStages) & 1);
    }
  } else if (warp == kWarpMma) {
    constexpr uint32_t idesc = idesc_e4m3_f32(128, L::kBatchIsM ? L::kAccCols : L::kBoxCols);
    const bool leader = elect_one();
    pdl_wait();  // (the waits' clocks start behind the preceding kernel: the rows come no earlier)
    int st = 0, ac = 0;
    uint32_t ph = 0, aph = 0;
    for (int kb = kb0; kb < kb1; ++kb) {
      // (the lanes decide together, so that none leaves the loop alone)
      if (!__all_sync(0xffffffffu, mbar_wait(tempty(ac), aph ^ 1u, abort_flag, status, kStatusTimeout, limit) &&
                                       mbar_wait(full(st), ph, abort_flag, status, kStatusTimeout, limit)))
        break;
      tc_fence_after();
      if (leader) {
        const uint64_t wd = sw128_kmajor_desc(base + st * L::kStageBytes);
        const uint64_t xd = sw128_kmajor_desc(base + st * L::kStageBytes + L::kW * kWTile);
        const uint32_t d = tmem + ac * L::kAccCols;
        // (32 bytes on: 2 descriptor units; with the batch as rows both boxes are one operand)
#pragma unroll
        for (int w = 0; w < (L::kBatchIsM ? 1 : L::kW); ++w)
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            const uint64_t wi = wd + w * (kWTile / 16) + 2 * i, xi = xd + 2 * i;
            tc_mma_e4m3(d + w * L::kBoxCols, L::kBatchIsM ? xi : wi, L::kBatchIsM ? wi : xi, idesc, i > 0);
          }
        tc_commit(empty(st));
        tc_commit(tfull(ac));
      }
      __syncwarp();
      if (++st == L::kStages) st = 0, ph ^= 1u;
      if (++ac == L::kAccs) ac = 0, aph ^= 1u;
    }
    if (leader) {  // tensor memory is freed only after the last MMAs, whoever gave up
      tc_commit(drain);
      mbar_drain(drain, 0);
    }
    __syncwarp();
  } else {
    pdl_wait();
    if (threadIdx.x == 0) pdl_launch_dependents();
    if (!kSwiglu && a.add)  // (the addends of the rows that this CTA will write, to L2)
      for (int i = threadIdx.x; rank + split * (i >> 1) < rows; i += L::kEpiThreads) {
        const int n = n0 + (i & 1) * 64;
        if (n < a.N) prefetch_l2(a.add + (m0 + rank + split * (i >> 1)) * a.N + n);
      }
    const int row = (warp & 3) * 32 + lane;
    const int c0 = (warp >> 2) * L::kMine;  // first column
    const uint32_t src0 = tmem + (static_cast<uint32_t>((warp & 3) * 32) << 16) + c0;
    float acc[L::kW][L::kMine];
#pragma unroll
    for (int j = 0; j < L::kMine; ++j)
#pragma unroll
      for (int w = 0; w < L::kW; ++w) acc[w][j] = 0.f;
    int ac = 0;
    uint32_t aph = 0;
    bool ok = true;  // (a warp that gave up goes on without sums: the others meet it at the barrier)
    if (a.test_never_wait) ok = __all_sync(0xffffffffu, mbar_wait(never, 0, abort_flag, status, kStatusTimeout, limit));
    for (int kb = kb0; kb < kb1; ++kb) {
      const int at = (kb - kb0) % L::kScaleRun;
      if (at == 0) {  // both scales of the next blocks, multiplied
        const int run = min(L::kScaleRun, kb1 - kb);
        named_bar_sync(1, L::kEpiThreads);
        if (lane < run) {  // (lanes along the blocks: whole lines of a_s)
          float sb[L::kW];
#pragma unroll
          for (int w = 0; w < L::kW; ++w) sb[w] = a.b_s[static_cast<long long>((n0 + w * a.N) / kScaleBlock) * Kb + kb + lane];
          constexpr int kEach = kRows / L::kEpiWarps;
          float sa[kEach];  // (all loads before the first store: one latency)
#pragma unroll
          for (int i = 0; i < kEach; ++i) {
            const int j = warp + i * L::kEpiWarps;
            sa[i] = j < rows ? a.a_s[(m0 + j) * Kb + kb + lane] : 0.f;
          }
#pragma unroll
          for (int i = 0; i < kEach; ++i)
#pragma unroll
            for (int w = 0; w < L::kW; ++w)
              scales[w * L::kScaleBox + lane * L::kScaleRow + warp + i * L::kEpiWarps] = sa[i] * sb[w];
        }
        named_bar_sync(1, L::kEpiThreads);
      }
      ok = ok && __all_sync(0xffffffffu, mbar_wait(tfull(ac), aph, abort_flag, status, kStatusTimeout, limit));
      if (!ok) continue;
      tc_fence_after();
#pragma unroll
      for (int w = 0; w < L::kW; ++w) {
        const float* table = scales + w * L::kScaleBox + at * L::kScaleRow;
        const float mine = table[L::kBatchIsM ? row : 0];
#pragma unroll
        for (int c = 0; c < L::kMine / L::kPiece; ++c) {
          uint32_t v[L::kPiece];
          tmem_piece(src0 + ac * L::kAccCols + w * L::kBoxCols + c * L::kPiece, v);
          const float4* sc = reinterpret_cast<const float4*>(table + c0 + c * L::kPiece);
          tmem_ld_wait();
#pragma unroll
          for (int q = 0; q < L::kPiece / 4; ++q) {
            const float4 s4 = L::kBatchIsM ? make_float4(mine, mine, mine, mine) : sc[q];
            float* x = acc[w] + c * L::kPiece + 4 * q;
            x[0] = fmaf(__uint_as_float(v[4 * q + 0]), s4.x, x[0]);
            x[1] = fmaf(__uint_as_float(v[4 * q + 1]), s4.y, x[1]);
            x[2] = fmaf(__uint_as_float(v[4 * q + 2]), s4.z, x[2]);
            x[3] = fmaf(__uint_as_float(v[4 * q + 3]), s4.w, x[3]);
          }
        }
      }
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive(tempty(ac));
      if (++ac == L::kAccs) ac = 0, aph ^= 1u;
    }
    // sums [batch row][128 weights], 16-byte pieces swizzled by the row (every MMA is done --
    // the last accumulator was waited for -- so the stages are free)
#pragma unroll
    for (int w = 0; w < L::kW; ++w) {
      uint8_t* part = gbase + w * L::kPart;
      if (L::kBatchIsM) {
#pragma unroll
        for (int i = 0; i < L::kMine; i += 4)
          *reinterpret_cast<float4*>(part + part_at(row, (c0 + i) / 4)) =
              make_float4(acc[w][i], acc[w][i + 1], acc[w][i + 2], acc[w][i + 3]);
      } else {
#pragma unroll
        for (int j = 0; j < L::kMine; ++j)
          if (c0 + j < rows) *reinterpret_cast<float*>(part + part_at(c0 + j, row / 4) + (row & 3) * 4) = acc[w][j];
      }
    }
  }
  __syncwarp();
  tc_fence_before();
  if (split > 1)
    cluster_sync();
  else
    __syncthreads();
  if (warp < L::kEpiWarps) {
    // a warp takes whole batch rows, four weights a lane: two rows at a time, or a row's
    // gate and up
    const int step = split * L::kEpiWarps;
    const int n = n0 + 4 * lane;
    for (int j = warp * split + rank; j < rows; j += (kSwiglu ? 1 : 2) * step) {
      const bool two = !kSwiglu && j + step < rows;
      const uint32_t at0 = base + part_at(j, lane);
      const uint32_t at1 = kSwiglu ? at0 + L::kPart : base + part_at(two ? j + step : j, lane);
      float4 y0, y1;
      join_pair(at0, at1, split, &y0, &y1);
      if (kSwiglu) {
        const float4 h = make_float4(swiglu(y0.x, y1.x), swiglu(y0.y, y1.y), swiglu(y0.z, y1.z), swiglu(y0.w, y1.w));
        float amax = max_nan(max_nan(max_nan(max_nan(0.f, h.x), h.y), h.z), h.w);
#pragma unroll
        for (int off = 16; off > 0; off >>= 1) amax = max_nan(amax, __shfl_xor_sync(0xffffffffu, amax, off));
        const float s = block_scale(amax);
        const uint32_t q = e4m3_quad(h.x, h.y, h.z, h.w, s, __frcp_rn(s), quotient_ok(s));
        *reinterpret_cast<uint32_t*>(static_cast<uint8_t*>(a.out) + (m0 + j) * a.N + n) = q;
        if (lane == 0) a.out_s[(m0 + j) * (a.N / kScaleBlock) + n0 / kScaleBlock] = s;
      } else {
        store_out4(a, m0 + j, n, y0, vec);
        if (two) store_out4(a, m0 + j + step, n, y1, vec);
      }
    }
  } else if (warp == kWarpTma && lane == 0 && !*abort_flag) {
    // ... and after the MMAs' last signals, which are writes to it too (here, beside the
    // joining, they cost nothing; ahead of the barrier 0.3 us)
    const int it = kb1 - kb0;
    for (int i = it > L::kStages ? it - L::kStages : 0; i < it; ++i)
      if (!mbar_wait(empty(i % L::kStages), (i / L::kStages) & 1, abort_flag, status, kStatusTimeout, limit)) break;
  }
  __syncwarp();
  if (split > 1) cluster_sync();  // no CTA leaves while another reads its sums
  if (warp == kWarpMma) {
    __syncwarp();
    tc_fence_after();
    tmem_dealloc(tmem, L::kTmem);
  }
}

// ---------------------------------------------------------------- host

constexpr int kMaxSplit = 8;

// Clusters of `split` CTAs that run at once on device `dev`, the current one (SMs share a
// cluster only within their part of the chip, so of eight at one CTA to an SM fewer fit than
// the SMs would hold); sets the kernel up for the device when it is first asked.
template <int kRows, bool kSwiglu>
cudaError_t clusters_at_once(int dev, int split, int num_sms, int* clusters) {
  using L = Few<kRows, kSwiglu>;
  static PerDevice<int> known[kMaxSplit + 1];
  std::atomic<int>* entry = known[split].of(dev);
  *clusters = entry ? entry->load() : 0;
  if (*clusters) return cudaSuccess;
  cudaError_t e =
      cudaFuncSetAttribute(fp8_matmul_few_kernel<kRows, kSwiglu>, cudaFuncAttributeMaxDynamicSharedMemorySize, L::kSmem);
  if (e != cudaSuccess) return e;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(split * num_sms);
  cfg.blockDim = dim3(L::kThreads);
  cfg.dynamicSmemBytes = L::kSmem;
  cudaLaunchAttribute attr;
  attr.id = cudaLaunchAttributeClusterDimension;
  attr.val.clusterDim.x = split, attr.val.clusterDim.y = 1, attr.val.clusterDim.z = 1;
  cfg.attrs = &attr;
  cfg.numAttrs = 1;
  int n = 0;
  e = cudaOccupancyMaxActiveClusters(&n, fp8_matmul_few_kernel<kRows, kSwiglu>, &cfg);
  if (e != cudaSuccess) return e;
  // (the query counts one CTA to an SM)
  *clusters = (n < 1 ? 1 : n) * L::kPerSm;
  if (entry) entry->store(*clusters);
  return cudaSuccess;
}

// CTAs to a tile: the number that leaves the busiest SM the fewest blocks, if all run at
// once and have at least four each; the fewest CTAs of equal ones, or where the weights
// stream in ahead of the rows the most (more of them fit: the shared expert of 4 tokens
// 16.8 us with the down product over 2 CTAs, 15.2 over 4). Its share of the blocks, and
// the waves of CTAs. (4,096 x 7,168, one row, 32 tiles of 56 blocks: 18.2,
// 10.9, 6.1, 7.2, 6.7 us with 1, 2, 4, 6, 8 CTAs; 7,168 x 2,048, 56 tiles of 16: 6.4, 4.7,
// 4.9 with 1, 2, 4.)
template <int kRows, bool kSwiglu>
cudaError_t choose_split(const Fp8MatmulArgs& a, int num_sms, int* split, int* share, long long* waves) {
  const int Kb = (a.K + kScaleBlock - 1) / kScaleBlock;
  const long long tiles = (a.N + 127) / 128 * ((static_cast<long long>(a.M) + kRows - 1) / kRows);
  int at_once = 0, dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e == cudaSuccess) e = clusters_at_once<kRows, kSwiglu>(dev, 1, num_sms, &at_once);
  if (e != cudaSuccess) return e;
  *waves = (tiles + at_once - 1) / at_once;
  *split = 1;
  long long best = (tiles + num_sms - 1) / num_sms * Kb;
  for (int c = 2; c <= kMaxSplit && Kb >= 4 * c && tiles * c <= 2LL * num_sms; ++c) {
    e = clusters_at_once<kRows, kSwiglu>(dev, c, num_sms, &at_once);
    if (e != cudaSuccess) return e;
    const long long blocks = (tiles * c + num_sms - 1) / num_sms * ((Kb + c - 1) / c);
    if (tiles <= at_once && (blocks < best || (blocks == best && a.weights_ready))) best = blocks, *split = c;
  }
  *share = (Kb + *split - 1) / *split;
  return cudaSuccess;
}

template <int kRows, bool kSwiglu>
cudaError_t launch_few(const Fp8MatmulArgs& a, int split, int32_t* status, cudaStream_t stream) {
  using L = Few<kRows, kSwiglu>;
  CUtensorMap wmap, xmap;
  if (!make_byte_map(&wmap, a.b, L::kW * static_cast<long long>(a.N), a.K, a.ldb, 128) ||
      !make_byte_map(&xmap, a.a, a.M, a.K, a.lda, kRows))
    return cudaErrorInvalidValue;
  const bool vec = a.N % 4 == 0 && reinterpret_cast<uintptr_t>(a.out) % (a.out_type == kTypeF32 ? 16 : 8) == 0 &&
                   reinterpret_cast<uintptr_t>(a.add) % 8 == 0;
  const dim3 grid(static_cast<unsigned>((a.N + 127) / 128 * split), static_cast<unsigned>((a.M + kRows - 1) / kRows));
  return launch_cluster(fp8_matmul_few_kernel<kRows, kSwiglu>, grid, dim3(L::kThreads), L::kSmem, stream, split, wmap, xmap,
                        a, split, vec, status);
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

namespace {
// Settings of the whole process (moe_w4a16_fp8_set_option).
std::atomic<int> g_wait_us{0}, g_test_never_wait{0};

// Kernel and split by size.
template <bool kSwiglu>
cudaError_t plan_tiles(const Fp8MatmulArgs& a, int num_sms, Fp8Plan* plan) {
  int split = 1, share = 0;
  long long waves = 0;
  plan->rows = a.M <= 16 ? 16 : a.M <= 32 ? 32 : a.M <= 64 ? 64 : 128;
  const cudaError_t e = a.M <= 16   ? choose_split<16, kSwiglu>(a, num_sms, &split, &share, &waves)
                        : a.M <= 32 ? choose_split<32, kSwiglu>(a, num_sms, &split, &share, &waves)
                        : a.M <= 64 ? choose_split<64, kSwiglu>(a, num_sms, &split, &share, &waves)
                                    : choose_split<128, kSwiglu>(a, num_sms, &split, &share, &waves);
  plan->split = split;
  if (e != cudaSuccess || a.M <= 64) return e;
  // Both kernels' times by what they were measured to take, in hundredths of a us: here
  // 30 a block and 500 a wave of CTAs, 300 more with an addend from the second on; there 40 a block and 120 a
  // wave of pairs, 300 in all, and 300 a wave where its output cannot go in whole pieces;
  // with an addend 180 and 700. (256 x 4,096 x 7,168: 14.2 us here, 24.4 there; 512 rows 22.4 and
  // 24.6; 640 x 7,168 x 2,048: 19.2 and 18.5; 2,048 x 1,000 x 1,936 in fp32: 10.8 and
  // 11.1; 2,048 x 2,047 x 1,024: 15.0 and 11.7, with an addend 21.5 and 15.1; 8,192 x
  // 4,095 x 7,168: 316 and 193. The SwiGLU form's two weight boxes count 45 a block here.)
  const int Kb = (a.K + kScaleBlock - 1) / kScaleBlock;
  const long long pairs = num_sms / 2;
  const long long big = (static_cast<long long>(a.M) + 255) / 256 * (kSwiglu ? a.N / 128 : (a.N + 255) / 256);
  const long long odd = kSwiglu ? 0 : fp8_whole_pieces(a) ? (a.add ? 180 : 0) : a.add ? 700 : 300;
  const long long here = waves * ((kSwiglu ? 45LL : 30LL) * share + 500) + 100 + (a.add ? 300 * (waves - 1) : 0);
  const long long there = (big + pairs - 1) / pairs * (40LL * Kb + 120 + odd) + 300;
  // (a grid's second dimension ends at 65,535 tiles of 128 rows)
  if (there < here || a.M > 65535LL * 128) *plan = Fp8Plan{256, 2};
  return cudaSuccess;
}

template <bool kSwiglu>
cudaError_t launch_tiles(Fp8MatmulArgs a, int32_t* status, int num_sms, cudaStream_t stream) {
  a.wait_kcycles = wait_limit_kcycles(static_cast<unsigned long long>(g_wait_us.load(std::memory_order_relaxed)));
  a.test_never_wait = g_test_never_wait.load(std::memory_order_relaxed);
  Fp8Plan plan;
  const cudaError_t e = plan_tiles<kSwiglu>(a, num_sms, &plan);
  if (e != cudaSuccess) return e;
  switch (plan.rows) {
    case 16: return launch_few<16, kSwiglu>(a, plan.split, status, stream);
    case 32: return launch_few<32, kSwiglu>(a, plan.split, status, stream);
    case 64: return launch_few<64, kSwiglu>(a, plan.split, status, stream);
    case 128: return launch_few<128, kSwiglu>(a, plan.split, status, stream);
    default: return launch_fp8_many(a, kSwiglu, status, num_sms, stream);
  }
}
}  // namespace

cudaError_t fp8_plan(const Fp8MatmulArgs& a, bool swiglu, int num_sms, Fp8Plan* plan) {
  *plan = Fp8Plan{0, 1};
  if (!tma_ok(a)) return cudaSuccess;
  return swiglu ? plan_tiles<true>(a, num_sms, plan) : plan_tiles<false>(a, num_sms, plan);
}

cudaError_t launch_fp8_matmul(const Fp8MatmulArgs& a, int num_sms, cudaStream_t stream) {
  if (!tma_ok(a)) {
    const dim3 grid(static_cast<unsigned>((a.M + kT - 1LL) / kT * ((a.N + kT - 1LL) / kT)));
    return launch_k(fp8_matmul_plain_kernel, grid, dim3(256), 0, stream, true, a);
  }
  int32_t* status = fp8_status_word();
  if (!status) return cudaErrorInvalidSymbol;
  return launch_tiles<false>(a, status, num_sms, stream);
}

// (the operands are the library's own: rows of whole 128-byte blocks, 256-byte aligned, and
// weights checked by the caller)
cudaError_t launch_fp8_swiglu(const Fp8MatmulArgs& a, int num_sms, cudaStream_t stream) {
  int32_t* status = fp8_status_word();
  if (!status) return cudaErrorInvalidSymbol;
  return launch_tiles<true>(a, status, num_sms, stream);
}

bool fp8_set_option(int option, int value) {
  if (option == 1 && value >= 0)
    g_wait_us.store(value);
  else if (option == 2 && (value == 0 || value == 1))
    g_test_never_wait.store(value);
  else
    return false;
  return true;
}

int32_t* fp8_status_word() {
  // (one context per device in a process)
  static PerDevice<int32_t*> known;
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess) return nullptr;
  std::atomic<int32_t*>* entry = known.of(dev);
  if (entry)
    if (int32_t* word = entry->load()) return word;
  void* p = nullptr;
  if (cudaGetSymbolAddress(&p, g_fp8_status) != cudaSuccess) return nullptr;
  if (entry) entry->store(static_cast<int32_t*>(p));
  return static_cast<int32_t*>(p);
}

cudaError_t fp8_status(int32_t* out, cudaStream_t stream) {
  int32_t* p = fp8_status_word();
  if (!p) return cudaErrorInvalidSymbol;
  // (cleared only when it is reported: a product of another stream may give up meanwhile, which
  // a clean answer must not hide. It sets the one bit that there is.)
  cudaError_t e = cudaMemcpyAsync(out, p, sizeof(*p), cudaMemcpyDeviceToHost, stream);
  if (e == cudaSuccess) e = cudaStreamSynchronize(stream);
  if (e != cudaSuccess || *out == 0) return e;
  e = cudaMemsetAsync(p, 0, sizeof(*p), stream);
  if (e == cudaSuccess) e = cudaStreamSynchronize(stream);
  return e;
}

}  // namespace moe
