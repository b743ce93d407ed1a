// 8-bit block-scaled product of many rows: the batch as the MMA's rows.
//
// A pair of CTAs computes a tile of 256 rows x 256 features with cta_group::2 MMAs: each
// CTA holds its 128 rows of `a` and half of `b`'s 256 in shared memory, and its rows'
// fp32 sums in tensor memory. Scales differ from block to block of the reduction, so a
// block of 128 elements (four MMAs) goes into a fresh accumulator; eight warps take it
// out of tensor memory, scale it by a_s[row] b_s[feature block] and add it to the running
// sums in registers (thread = one row, 128 features) while the MMAs of the next block
// fill the other accumulator. Tensor memory holds exactly the two.
//
// What bounds it: the way out of tensor memory. A block's MMAs take 512 cycles, its sums
// 450 of loads and additions plus about 550 from the last MMA to the first load and from
// the release to the next MMA, with two accumulators in turn: 750 cycles a block. The
// loads of 16 columns run one piece ahead of the sums.
// Measured and not kept: halves of an accumulator handed back one by one (up to +15%),
// 16 summing warps (+12%), scales staged in shared memory by other warps (+10%), output
// through shared memory and the copy engine (+5%), copies into L2 six blocks ahead (+2%).
//
// The SwiGLU form takes 128 gate features and the same 128 up features as its 256, and a
// thread sums 64 of each: it holds both for its features, agrees with the warp that has
// the row's other 64 on the scale, and writes e4m3.
//
// Warps: 0..7 sums and output, 8 copies (one lane of each CTA, both counting on the
// leader's barriers), 9 the MMAs (the leader's), 10 and 11 idle. Persistent: a pair
// takes every (number of pairs)-th tile. 8,192 x 4,096 x 7,168: 160 to 164 us, 3,000
// TFLOP/s (185 us in a loop of seconds, at the power limit).
#include <cuda_bf16.h>

#include "fp8_quant.cuh"
#include "fp8_tma.cuh"

namespace moe {
namespace {

// 32 bytes at a time (32-byte aligned).
struct Words8 {
  uint32_t w[8];
};
__device__ __forceinline__ void st_global_32b(void* p, const Words8& v) {
  asm volatile("st.global.v8.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};" ::"l"(p), "r"(v.w[0]), "r"(v.w[1]),
               "r"(v.w[2]), "r"(v.w[3]), "r"(v.w[4]), "r"(v.w[5]), "r"(v.w[6]), "r"(v.w[7])
               : "memory");
}
__device__ __forceinline__ Words8 ld_global_32b(const void* p) {
  Words8 v;
  asm volatile("ld.global.v8.b32 {%0, %1, %2, %3, %4, %5, %6, %7}, [%8];"
               : "=r"(v.w[0]), "=r"(v.w[1]), "=r"(v.w[2]), "=r"(v.w[3]), "=r"(v.w[4]), "=r"(v.w[5]), "=r"(v.w[6]),
                 "=r"(v.w[7])
               : "l"(p)
               : "memory");
  return v;
}

constexpr int kEpiWarps = 8, kWarpTma = 8, kWarpMma = 9;
constexpr int kThreads = 12 * 32;  // (two warps idle: registers move between groups of four warps)
constexpr int kEpiRegs = 232, kOtherRegs = 40;
static_assert(256 * kEpiRegs + 128 * kOtherRegs <= kThreads * 168, "more registers than the launch's");
constexpr int kTileM = 256, kTileN = 256;  // of a pair
constexpr int kHalf = 128;                 // rows, and features, of a CTA
constexpr int kSums = kTileN / 2;          // of a thread: one row, 128 features
constexpr int kOperand = 128 * 128;        // bytes of a box
constexpr int kStageBytes = 2 * kOperand;
// Where the sums go: whole 32-byte pieces of a row, any alignment (both without and with
// addends, for whose registers the sums would pay), or SwiGLU and e4m3.
enum Out { kOutPieces, kOutPiecesAdd, kOutAcross, kOutAcrossAdd, kOutSwiglu };
__host__ __device__ constexpr bool across(Out out) { return out == kOutAcross || out == kOutAcrossAdd; }
// Shared memory: maxima, barriers, stages, and for any alignment a tile of 32 rows x 65
// sums for each summing warp, which costs a stage.
__host__ __device__ constexpr int stages(Out out) { return across(out) ? 4 : 5; }
constexpr int kMax = 0;  // SwiGLU: the rows' maxima [tile parity][quarter][half][32]
constexpr int kBars = kMax + 2 * 1024;
constexpr int kStage0 = 3 * 1024;
constexpr int kWide = 64, kAcrossWarp = 32 * (kWide + 1) * 4;
__host__ __device__ constexpr int across_at(Out out) { return kStage0 + stages(out) * kStageBytes; }
__host__ __device__ constexpr int smem_bytes(Out out) { return across_at(out) + (across(out) ? kEpiWarps * kAcrossWarp : 0) + 1024; }
static_assert(kBars + 8 * (2 * 5 + 4 + 1 + 4 + 1) + 8 <= kStage0, "barriers");
static_assert(smem_bytes(kOutAcross) <= 227 * 1024, "shared memory of a CTA");

// acc (two sums) += v (two block sums) * s
__device__ __forceinline__ void fma2(uint64_t& acc, uint32_t lo, uint32_t hi, uint64_t s2) {
  asm("{\n\t.reg .b64 t;\n\tmov.b64 t, {%1, %2};\n\tfma.rn.f32x2 %0, t, %3, %0;\n\t}"
      : "+l"(acc)
      : "r"(lo), "r"(hi), "l"(s2));
}
__device__ __forceinline__ float2 unpack2(uint64_t v) {
  float2 f;
  asm("mov.b64 {%0, %1}, %2;" : "=f"(f.x), "=f"(f.y) : "l"(v));
  return f;
}
__device__ __forceinline__ uint64_t pack2(float a, float b) {
  uint64_t v;
  asm("mov.b64 %0, {%1, %2};" : "=l"(v) : "f"(a), "f"(b));
  return v;
}

// Tile `t` of a grid of mt x nt: bands of 8 row tiles, features outer inside a band, so
// that the pairs at work together share rows and features in L2.
constexpr int kBand = 8;
__device__ __forceinline__ void tile_at(int t, int mt, int nt, int* im, int* in) {
  const int band = t / (kBand * nt);
  const int rows = min(kBand, mt - band * kBand);
  const int r = t - band * kBand * nt;
  *im = band * kBand + r % rows;
  *in = r / rows;
}

__device__ __forceinline__ uint32_t bf16x2(float lo, float hi) {
  const __nv_bfloat162 h = __floats2bfloat162_rn(lo, hi);
  return *reinterpret_cast<const uint32_t*>(&h);
}


// A thread's sums to the output, 32 bytes at a time: rows of whole, aligned such pieces.
__device__ __forceinline__ void store_row(const Fp8MatmulArgs& a, long long m, int n, const uint64_t (&acc)[kSums / 2]) {
  const long long at = m * a.N + n;
  if (a.out_type == kTypeBf16) {
    __nv_bfloat16* out = static_cast<__nv_bfloat16*>(a.out) + at;
#pragma unroll
    for (int c = 0; c < kSums / 16; ++c) {
      if (n + 16 * c >= a.N) break;
      Words8 w;
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        const float2 y = unpack2(acc[8 * c + i]);
        w.w[i] = bf16x2(y.x, y.y);
      }
      st_global_32b(out + 16 * c, w);
    }
  } else {
    float* out = static_cast<float*>(a.out) + at;
#pragma unroll
    for (int c = 0; c < kSums / 8; ++c) {
      if (n + 8 * c >= a.N) break;
      Words8 w;
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const float2 y = unpack2(acc[4 * c + i]);
        w.w[2 * i] = __float_as_uint(y.x), w.w[2 * i + 1] = __float_as_uint(y.y);
      }
      st_global_32b(out + 8 * c, w);
    }
  }
}

__device__ __forceinline__ void st_shared_f32(uint32_t addr, float v) {
  asm volatile("st.shared.f32 [%0], %1;" ::"r"(addr), "f"(v) : "memory");
}
__device__ __forceinline__ float ld_shared_f32(uint32_t addr) { return __uint_as_float(ld_shared_u32(addr)); }

// The same with addends, bf16, four pieces' loads at a time (8,192 x 7,168 x 2,048: 124 us,
// 134 one by one, 98 without addends).
__device__ __forceinline__ void store_row_add(const Fp8MatmulArgs& a, long long m, int n,
                                              const uint64_t (&acc)[kSums / 2]) {
  if (n >= a.N) return;
  const long long at = m * a.N + n;
  __nv_bfloat16* out = static_cast<__nv_bfloat16*>(a.out) + at;
  constexpr int kOnce = 4;  // pieces
#pragma unroll
  for (int c0 = 0; c0 < kSums / 16; c0 += kOnce) {
    Words8 d[kOnce];  // (all loads before the first store, which may be to the same array)
#pragma unroll
    for (int c = 0; c < kOnce; ++c) d[c] = ld_global_32b(a.add + (n + 16 * (c0 + c) < a.N ? at + 16 * (c0 + c) : at));
#pragma unroll
    for (int c = 0; c < kOnce; ++c) {
      if (n + 16 * (c0 + c) >= a.N) break;
      Words8 w;
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        const float2 y = unpack2(acc[8 * (c0 + c) + i]);
        w.w[i] = bf16x2(y.x + __uint_as_float(d[c].w[i] << 16), y.y + __uint_as_float(d[c].w[i] & 0xFFFF0000u));
      }
      st_global_32b(out + 16 * (c0 + c), w);
    }
  }
}

// A warp's sums (32 rows from m0 on, 128 features) to an output of any alignment: 64
// features at a time go through shared memory (`tile`: 32 rows of 65), and a lane writes
// two features of a row at once, from the row's first even address on: 128 bytes or more
// of a row to a store, so that few sectors are written in parts. (8,192 x 4,095 x 1,024
// takes 66 us; 84 with 32 features and one to a store, whether transposed by exchanges or
// through shared memory; 40 is what 4,096 features take.)
template <bool kAdd, typename T, typename T2>
__device__ __forceinline__ void store_across(const Fp8MatmulArgs& a, long long m0, int n, int lane,
                                             const uint64_t (&acc)[kSums / 2], uint32_t tile) {
  const int rows = static_cast<int>(a.M - m0 < 32 ? a.M - m0 : 32);
  constexpr int kOnce = 8;  // rows
  const int N = a.N;
#pragma unroll
  for (int c = 0; c < kSums / kWide; ++c) {
    if (n + kWide * c >= N) break;
    __syncwarp();
#pragma unroll
    for (int i = 0; i < kWide / 2; ++i) {
      const float2 y = unpack2(acc[kWide / 2 * c + i]);
      st_shared_f32(tile + (lane * (kWide + 1) + 2 * i) * 4, y.x);
      st_shared_f32(tile + (lane * (kWide + 1) + 2 * i + 1) * 4, y.y);
    }
    __syncwarp();
    const int left = min(kWide, N - n - kWide * c);
    const long long first = m0 * N + n + kWide * c;
    T* out = static_cast<T*>(a.out) + first;
    const uint32_t odd = static_cast<uint32_t>(reinterpret_cast<uintptr_t>(out) / sizeof(T));
    // features e0 and e1 = e0 + 1 of a row; at odd addresses the last lane's are 63 and 0
    auto place = [&](int r, int* e0, int* e1) {
      *e0 = 2 * lane + ((odd + static_cast<uint32_t>(r) * static_cast<uint32_t>(N)) & 1);
      *e1 = (*e0 + 1) % kWide;
    };
#pragma unroll 1
    for (int r0 = 0; r0 < rows; r0 += kOnce) {
      uint16_t d0[kOnce], d1[kOnce];
      if (kAdd) {  // (all loads before the first store, which may be to the same array, and none conditional)
#pragma unroll
        for (int i = 0; i < kOnce; ++i) {
          int e0, e1;
          place(r0 + i, &e0, &e1);
          const uint16_t* p = a.add + first + static_cast<long long>(min(r0 + i, rows - 1)) * N;
          d0[i] = p[min(e0, left - 1)], d1[i] = p[min(e1, left - 1)];
        }
      }
#pragma unroll
      for (int i = 0; i < kOnce; ++i) {
        const int r = r0 + i;
        int e0, e1;
        place(r, &e0, &e1);
        const uint32_t row = tile + r * (kWide + 1) * 4;
        float y0 = ld_shared_f32(row + e0 * 4), y1 = ld_shared_f32(row + e1 * 4);
        if (kAdd) {
          y0 += __uint_as_float(static_cast<uint32_t>(d0[i]) << 16);
          y1 += __uint_as_float(static_cast<uint32_t>(d1[i]) << 16);
        }
        if (r >= rows) break;
        T* to = out + static_cast<long long>(r) * N;
        T2 w;
        if constexpr (sizeof(T) == 2)
          w = __floats2bfloat162_rn(y0, y1);
        else
          w = make_float2(y0, y1);
        if (e1 > e0 && e1 < left) {
          *reinterpret_cast<T2*>(to + e0) = w;
        } else {
          if (e0 < left) to[e0] = w.x;
          if (e1 < e0) to[e1] = w.y;
        }
      }
    }
  }
}

// SiLU(gate) * up of a thread's 64 features (the first half of its sums are the gate's, the
// other the up projection's), into the first half; the largest magnitude.
__device__ __forceinline__ float join_row(uint64_t (&acc)[kSums / 2]) {
  float amax = 0.f;
#pragma unroll
  for (int i = 0; i < kSums / 4; ++i) {
    const float2 g = unpack2(acc[i]), u = unpack2(acc[kSums / 4 + i]);
    const float h0 = swiglu(g.x, u.x), h1 = swiglu(g.y, u.y);
    amax = max_nan(max_nan(amax, h0), h1);
    acc[i] = pack2(h0, h1);
  }
  return amax;
}
__device__ __forceinline__ void store_quantized(const uint64_t (&acc)[kSums / 2], float s, uint8_t* to) {
  const float r = __frcp_rn(s);
  const bool exact = quotient_ok(s);
#pragma unroll
  for (int c = 0; c < 2; ++c) {
    Words8 w;
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const float2 y = unpack2(acc[16 * c + 2 * i]), z = unpack2(acc[16 * c + 2 * i + 1]);
      w.w[i] = e4m3_quad(y.x, y.y, z.x, z.y, s, r, exact);
    }
    st_global_32b(to + 32 * c, w);
  }
}

template <Out kOut>
__global__ void __launch_bounds__(kThreads, 1)
    fp8_matmul_many_kernel(const __grid_constant__ CUtensorMap amap, const __grid_constant__ CUtensorMap bmap,
                           const __grid_constant__ Fp8MatmulArgs a, int mt, int nt, int32_t* status) {
  constexpr bool kSwiglu = kOut == kOutSwiglu;
  constexpr int kStages = stages(kOut);
  extern __shared__ uint8_t smem_raw[];
  const uint32_t base = (smem_u32(smem_raw) + 1023u) & ~1023u;
  uint8_t* gbase = smem_raw + (base - smem_u32(smem_raw));
  auto full = [&](int i) { return base + kBars + 8 * i; };                    // leader's: both CTAs' copies
  auto empty = [&](int i) { return base + kBars + 8 * (kStages + i); };       // each CTA's
  auto tfull = [&](int i) { return base + kBars + 8 * (2 * kStages + i); };   // each CTA's
  auto tempty = [&](int i) { return base + kBars + 8 * (2 * kStages + 2 + i); };  // leader's: both CTAs' warps
  const uint32_t drain = base + kBars + 8 * (2 * kStages + 4);
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(gbase + kBars + 8 * (2 * kStages + 10));
  const uint32_t never = drain + 8;                         // (the test hook's)
  auto met = [&](int i) { return drain + 16 + 8 * i; };  // a row quarter's two warps have their maxima
  volatile int* abort_flag = reinterpret_cast<volatile int*>(tmem_slot + 1);

  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int rank = static_cast<int>(cluster_rank());
  const int Kb = (a.K + kScaleBlock - 1) / kScaleBlock;
  const int tiles = mt * nt;
  const int pairs = gridDim.x / 2, pair = blockIdx.x / 2;
  const uint32_t limit = a.wait_kcycles;

  if (threadIdx.x == 0) {
    tma_prefetch_map(&amap);
    tma_prefetch_map(&bmap);
    for (int i = 0; i < kStages; ++i) mbar_init(full(i), 1), mbar_init(empty(i), 1);
    for (int i = 0; i < 2; ++i) mbar_init(tfull(i), 1), mbar_init(tempty(i), 2 * kEpiWarps);
    mbar_init(drain, 1);
    mbar_init(never, 1);
    for (int i = 0; i < 4; ++i) mbar_init(met(i), 2);
    *abort_flag = 0;
    fence_mbar_init();
  }
  if (warp == kWarpMma) {
    __syncwarp();
    tmem_alloc_pair(smem_u32(tmem_slot), 512);
  }
  tc_fence_before();
  __syncthreads();
  cluster_sync();
  tc_fence_after();
  const uint32_t tmem = *tmem_slot;

  if (warp >= kEpiWarps) {
    asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(kOtherRegs));
    if (warp == kWarpTma && lane == 0) {
      const uint64_t keep = l2_policy_evict_last();
      pdl_wait();
      int st = 0;
      uint32_t ph = 0;
      int issued = 0;  // (only its last kStages and their phases matter: kept small)
      bool ok = true;
      for (int t = pair; t < tiles && ok; t += pairs) {
        int im, in;
        tile_at(t, mt, nt, &im, &in);
        const int m0 = im * kTileM + rank * kHalf;
        const int n0 = kSwiglu ? in * kHalf + rank * a.N : in * kTileN + rank * kHalf;
        for (int kb = 0; kb < Kb; ++kb) {
          if (!mbar_wait(empty(st), ph ^ 1u, abort_flag, status, kStatusTimeout, limit)) {
            ok = false;
            break;
          }
          if (rank == 0) mbar_arrive_expect_tx(full(st), 2 * kStageBytes);
          const uint32_t bar = map_rank(full(st), 0);
          tma_load_2d_pair(base + kStage0 + st * kStageBytes, &amap, kb * 128, m0, bar, keep);
          tma_load_2d_pair(base + kStage0 + st * kStageBytes + kOperand, &bmap, kb * 128, n0, bar, keep);
          if (++issued == 4 * kStages) issued = 2 * kStages;
          if (++st == kStages) st = 0, ph ^= 1u;
        }
      }
      // shared memory is released only after the last copies have landed, whoever gave up
      if (rank == 0)
        for (int i = issued > kStages ? issued - kStages : 0; i < issued; ++i)
          mbar_drain(full(i % kStages), (i / kStages) & 1);
      // ... and, in either CTA, after the MMAs' last signals have: each of them is a write to
      // this CTA's shared memory that travels on its own, and one that was seen says nothing
      // about the others
      for (int i = issued > kStages ? issued - kStages : 0; i < issued; ++i)
        if (!mbar_wait(empty(i % kStages), (i / kStages) & 1, abort_flag, status, kStatusTimeout, limit)) break;
      if (rank != 0) mbar_drain(drain, 0);  // (the leader's own is waited for where it is sent)
      if (*abort_flag) {  // (the other CTA's copies count on the leader's barriers: give them 2 ms)
        const long long c0 = clock64();
        while (clock64() - c0 < 4000000) {
        }
      }
    }
    if (warp == kWarpMma && rank == 0) {
      const uint32_t idesc = idesc_e4m3_f32(kTileM, kTileN);
      const bool leader = elect_one();
      pdl_wait();  // (the waits' clocks start behind the preceding kernel: the copies come no earlier)
      int st = 0, ac = 0;
      uint32_t ph = 0, aph = 0;
      bool ok = true;
      for (int t = pair; t < tiles && ok; t += pairs) {
        for (int kb = 0; kb < Kb; ++kb) {
          ok = __all_sync(0xffffffffu, mbar_wait(full(st), ph, abort_flag, status, kStatusTimeout, limit) &&
                                           mbar_wait(tempty(ac), aph ^ 1u, abort_flag, status, kStatusTimeout, limit));
          if (!ok) break;
          tc_fence_after();
          if (leader) {
            const uint64_t ad = sw128_kmajor_desc(base + kStage0 + st * kStageBytes);
            const uint64_t bd = sw128_kmajor_desc(base + kStage0 + st * kStageBytes + kOperand);
#pragma unroll
            for (int i = 0; i < 4; ++i)  // (32 bytes on: 2 descriptor units)
              tc_mma_e4m3_pair(tmem + ac * kTileN, ad + 2 * i, bd + 2 * i, idesc, i > 0);
            tc_commit_pair(empty(st));
            tc_commit_pair(tfull(ac));
          }
          __syncwarp();
          if (++st == kStages) st = 0, ph ^= 1u;
          if (++ac == 2) ac = 0, aph ^= 1u;
        }
      }
      if (leader) {  // tensor memory is freed only after the last MMAs, whoever gave up
        tc_commit_pair(drain);
        mbar_drain(drain, 0);
      }
      __syncwarp();
    }
  } else {
    asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(kEpiRegs));
    pdl_wait();
    if (threadIdx.x == 0) pdl_launch_dependents();
    const int half = warp >> 2;
    const int row = (warp & 3) * 32 + lane;
    // (columns: 128 of the tile's 256; of the SwiGLU form 64 gate and, 128 on, 64 up)
    const uint32_t src0 = tmem + (static_cast<uint32_t>((warp & 3) * 32) << 16) + half * (kSwiglu ? kSums / 2 : kSums);
    const uint32_t give0 = map_rank(tempty(0), 0);
    const int nb = (a.N + kScaleBlock - 1) / kScaleBlock;
    int ac = 0;
    uint32_t aph = 0, met_ph = 0;
    bool ok = true;
    if (a.test_never_wait) ok = __all_sync(0xffffffffu, mbar_wait(never, 0, abort_flag, status, kStatusTimeout, limit));
    for (int t = pair; t < tiles && ok; t += pairs) {
      int im, in;
      tile_at(t, mt, nt, &im, &in);
      const int m = im * kTileM + rank * kHalf + row;  // (below 2^31: M is at most 2^30)
      const int n = in * kTileN + half * kSums;
      const bool live = m < a.M;
      // (rows and features behind the end read the scales of the first row, the last block)
      const float* as = a.a_s + static_cast<long long>(live ? m : 0) * Kb;
      const float* bs = a.b_s + static_cast<long long>(kSwiglu ? in : min(n / kScaleBlock, nb - 1)) * Kb;
      const long long up = kSwiglu ? static_cast<long long>(nb) * Kb : 0;  // from a gate block's scales to its up block's
      float sa = *as, sb = *bs, sb2 = bs[up];
      if ((kOut == kOutPiecesAdd || kOut == kOutAcrossAdd) && live)  // (the addends are in L2 when the sums are done)
        for (int f = n; f < a.N && f < n + kSums; f += 64) prefetch_l2(a.add + static_cast<long long>(m) * a.N + f);
      uint64_t acc[kSums / 2];
#pragma unroll
      for (int i = 0; i < kSums / 2; ++i) acc[i] = 0;
      for (int kb = 0; kb < Kb; ++kb) {
        const uint64_t s2 = pack2(sa * sb, sa * sb), s2up = pack2(sa * sb2, sa * sb2);
        if (kb + 1 < Kb) {
          sa = *++as, sb = *++bs;
          if (kSwiglu) sb2 = bs[up];
        }
        ok = __all_sync(0xffffffffu, mbar_wait(tfull(ac), aph, abort_flag, status, kStatusTimeout, limit));
        if (!ok) break;
        tc_fence_after();
        const uint32_t src = src0 + ac * kTileN;
        // the loads of a piece overlap the sums of the one before it
        constexpr int kPiece = 16;  // (pieces of 32 leave the outputs' forms short of registers)
        constexpr int kPieces = kSums / kPiece;
        auto column = [](int c) { return c * kPiece + (kSwiglu && c >= kPieces / 2 ? kSums / 2 : 0); };
        uint32_t v[2][kPiece];
        tmem_ld16(src, v[0]);
#pragma unroll
        for (int c = 0; c < kPieces; ++c) {
          tmem_ld_wait();
          if (c + 1 < kPieces) {
            tmem_ld16(src + column(c + 1), v[(c + 1) & 1]);
          } else {
            tc_fence_before();
            __syncwarp();
            if (lane == 0) mbar_arrive_cluster(give0 + 8 * ac);
          }
          const uint64_t by = kSwiglu && c >= kPieces / 2 ? s2up : s2;
#pragma unroll
          for (int i = 0; i < kPiece / 2; ++i)
            fma2(acc[c * (kPiece / 2) + i], v[c & 1][2 * i], v[c & 1][2 * i + 1], by);
        }
        if (++ac == 2) ac = 0, aph ^= 1u;
      }
      if (!kSwiglu) {
        if (kOut == kOutPieces && ok && live) store_row(a, m, n, acc);
        if (kOut == kOutPiecesAdd && ok && live) store_row_add(a, m, n, acc);
        if (across(kOut) && ok) {
          constexpr bool kAdd = kOut == kOutAcrossAdd;
          const uint32_t tile = base + across_at(kOut) + warp * kAcrossWarp;
          if (a.out_type == kTypeBf16)
            store_across<kAdd, __nv_bfloat16, __nv_bfloat162>(a, m - lane, n, lane, acc, tile);
          else
            store_across<kAdd, float, float2>(a, m - lane, n, lane, acc, tile);
        }
        continue;
      }
      // (bounded waits: a warp that gave up sends nothing, and its partner gives up too)
      if (!ok) break;
      const int quad = warp & 3;
      const float amax = join_row(acc);
      const uint32_t maxima = base + kMax + met_ph * 1024 + (quad * 64 + lane) * 4;
      st_shared_f32(maxima + half * 128, amax);
      __syncwarp();
      if (lane == 0) mbar_arrive(met(quad));
      ok = __all_sync(0xffffffffu, mbar_wait(met(quad), met_ph, abort_flag, status, kStatusTimeout, limit));
      if (!ok) break;
      met_ph ^= 1u;
      const float s = block_scale(max_nan(amax, ld_shared_f32(maxima + (half ^ 1) * 128)));
      // (the other warp writes here again two tiles on, after this one's next arrival)
      if (live) {
        store_quantized(acc, s, static_cast<uint8_t*>(a.out) + static_cast<long long>(m) * a.N + in * kHalf + half * 64);
        if (half == 0) a.out_s[static_cast<long long>(m) * nb + in] = s;
      }
    }
  }
  __syncwarp();
  tc_fence_before();
  cluster_sync();
  if (warp == kWarpMma) {
    __syncwarp();
    tc_fence_after();
    tmem_dealloc_pair(tmem, 512);
  }
}

}  // namespace

namespace {
template <Out kOut>
cudaError_t launch_many(const Fp8MatmulArgs& a, int32_t* status, int num_sms, cudaStream_t stream) {
  constexpr bool kSwiglu = kOut == kOutSwiglu;
  // pairs that can run at once (SMs that have a partner); sets the kernel up for the device
  static PerDevice<int> known;
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  std::atomic<int>* entry = known.of(dev);
  int pairs = entry ? entry->load() : 0;
  if (pairs == 0) {
    e = cudaFuncSetAttribute(fp8_matmul_many_kernel<kOut>, cudaFuncAttributeMaxDynamicSharedMemorySize, smem_bytes(kOut));
    if (e != cudaSuccess) return e;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(2 * (num_sms / 2));
    cfg.blockDim = dim3(kThreads);
    cfg.dynamicSmemBytes = smem_bytes(kOut);
    cudaLaunchAttribute attr;
    attr.id = cudaLaunchAttributeClusterDimension;
    attr.val.clusterDim.x = 2, attr.val.clusterDim.y = 1, attr.val.clusterDim.z = 1;
    cfg.attrs = &attr;
    cfg.numAttrs = 1;
    int n = 0;
    e = cudaOccupancyMaxActiveClusters(&n, fp8_matmul_many_kernel<kOut>, &cfg);
    if (e != cudaSuccess) return e;
    pairs = n < 1 ? 1 : (n > num_sms / 2 ? num_sms / 2 : n);
    if (entry) entry->store(pairs);
  }
  CUtensorMap amap, bmap;
  if (!make_byte_map(&amap, a.a, a.M, a.K, a.lda, kHalf) || !make_byte_map(&bmap, a.b, (kSwiglu ? 2LL : 1LL) * a.N, a.K, a.ldb, kHalf))
    return cudaErrorInvalidValue;
  const int mt = (a.M + kTileM - 1) / kTileM, nt = kSwiglu ? a.N / kHalf : (a.N + kTileN - 1) / kTileN;
  const long long tiles = static_cast<long long>(mt) * nt;
  if (tiles > (1 << 30)) return cudaErrorInvalidValue;  // (7e13 outputs)
  const unsigned grid = 2u * static_cast<unsigned>(tiles < pairs ? tiles : pairs);
  return launch_cluster(fp8_matmul_many_kernel<kOut>, dim3(grid), dim3(kThreads), smem_bytes(kOut), stream, 2, amap, bmap, a, mt, nt,
                        status);
}

}  // namespace

bool fp8_whole_pieces(const Fp8MatmulArgs& a) {
  const uintptr_t where = reinterpret_cast<uintptr_t>(a.out) | reinterpret_cast<uintptr_t>(a.add);
  return a.N % (a.out_type == kTypeBf16 ? 16 : 8) == 0 && where % 32 == 0 && !(a.out_type == kTypeF32 && a.add);
}

cudaError_t launch_fp8_many(const Fp8MatmulArgs& a, bool swiglu, int32_t* status, int num_sms, cudaStream_t stream) {
  if (swiglu) return launch_many<kOutSwiglu>(a, status, num_sms, stream);
  if (fp8_whole_pieces(a))
    return a.add ? launch_many<kOutPiecesAdd>(a, status, num_sms, stream) : launch_many<kOutPieces>(a, status, num_sms, stream);
  return a.add ? launch_many<kOutAcrossAdd>(a, status, num_sms, stream) : launch_many<kOutAcross>(a, status, num_sms, stream);
}

}  // namespace moe
