// Low-rank adapters, many rows: out[m] = add[m] + scale[l] b[l] (a[l] x[m]), l = index[m].
//
// The rows are sorted by adapter (the order of dispatch.cu, filled up to tiles of 128 rows;
// rows without an adapter are the last bucket's). A cluster of CTAs takes a tile. Each CTA
//   1. sums its share of a[l] x's columns: tcgen05 MMAs of 128 rows x r, whose x rows 16
//      warps copy from wherever they lie, a stage's copies under way beside the next ones'
//      (the copy engine's gathers of four rows take 18 cycles a row of 128 bytes here, five
//      times as long);
//   2. joins the sums with the cluster's other CTAs: each sends its sums of a row to the
//      row's CTA, which adds them in the order of the ranks, scales them, splits them into
//      bf16 parts (two, three for an fp32 output: 16 and 24 bits of the sum) and hands them
//      to all CTAs, straight into the second product's operand;
//   3. computes its share of the N columns: MMAs of 128 rows x 128 columns over the parts,
//      one after another against the same tile of b[l], two accumulators in turn, taken out
//      of tensor memory by 16 warps that add the addends, which they have loaded one tile
//      ahead, and write the output, eight columns to a lane.
// Nothing but x, a, b, the addends and the output goes through memory, and each once (a and
// b once for each tile, from L2). The operations are few, r of them for a byte at most: what
// bounds it is memory.
//
// Warps: 0..15 rows of x, joining and output, 16 the copies of a and b, 17 the MMAs. All
// sums have a fixed order.
#include <algorithm>

#include "fp8_tma.cuh"
#include "lora.cuh"

namespace moe {
namespace {

constexpr int kTile = 128;         // rows of a tile, columns of an accumulator
constexpr int kChunk = 64;         // columns of x to a stage: 128 bytes
constexpr int kBox = kTile * 128;  // bytes of 128 rows of 128 bytes
constexpr int kEpiWarps = 16, kEpiThreads = kEpiWarps * 32, kWarpCopy = 16, kWarpMma = 17, kThreads = 18 * 32;
constexpr int kCols = kTile * 4 / kEpiWarps;  // of an accumulator, to a warp
constexpr int kAhead = 4;          // column tiles whose addends are asked into L2 ahead
constexpr int kMaxStages = 6;
constexpr int kHead = 2048;        // barriers, the tile's rows
constexpr int kSmemMost = 227 * 1024;

struct ManyPlan {
  int ctas;         // to a tile
  int parts;        // bf16 parts of a sum
  int rank16;       // r, up to a multiple of 16
  int stages, stage_bytes, smem;
  int tiles;        // at most
};
struct Order {
  const int32_t* offsets;  // [L + 2]
  const int32_t* slots;
};

__device__ __forceinline__ void tc_mma_bf16(uint32_t d_tmem, uint64_t a_desc, uint64_t b_desc, uint32_t idesc, uint32_t accumulate) {
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "setp.ne.b32 p, %4, 0;\n\t"
      "tcgen05.mma.cta_group::1.kind::f16 [%0], %1, %2, %3, p;\n\t}" ::"r"(d_tmem),
      "l"(a_desc), "l"(b_desc), "r"(idesc), "r"(accumulate)
      : "memory");
}
// Instruction descriptor, kind::f16: bf16 A and B (format 1, both K-major), fp32 D, shape M x N.
__host__ __device__ constexpr uint32_t idesc_bf16_f32(int M, int N) {
  return (1u << 4) | (1u << 7) | (1u << 10) | (static_cast<uint32_t>(N >> 3) << 17) | (static_cast<uint32_t>(M >> 4) << 24);
}
// 16 bytes of global memory to shared memory, zeros where `bytes` is 0.
__device__ __forceinline__ void copy16(uint32_t dst, const void* src, uint32_t bytes) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(bytes) : "memory");
}
// Arrive on the barrier when this thread's copies so far have landed.
__device__ __forceinline__ void copies_arrive(uint32_t bar) {
  asm volatile("cp.async.mbarrier.arrive.noinc.shared::cta.b64 [%0];" ::"r"(bar) : "memory");
}
// 16 rows x 32 columns of fp32 sums: lane 4 g + t gets of row g (v[4 i], v[4 i + 1]) and of row
// g + 8 (v[4 i + 2], v[4 i + 3]) the columns 8 i + 2 t, 8 i + 2 t + 1.
__device__ __forceinline__ void tmem_ld_16x32(uint32_t taddr, uint32_t (&v)[16]) {
  asm volatile(
      "tcgen05.ld.sync.aligned.16x256b.x4.b32 "
      "{%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15}, [%16];"
      : "=r"(v[0]), "=r"(v[1]), "=r"(v[2]), "=r"(v[3]), "=r"(v[4]), "=r"(v[5]), "=r"(v[6]), "=r"(v[7]), "=r"(v[8]), "=r"(v[9]),
        "=r"(v[10]), "=r"(v[11]), "=r"(v[12]), "=r"(v[13]), "=r"(v[14]), "=r"(v[15])
      : "r"(taddr)
      : "memory");
}
// Of the four lanes of a row, each with pairs of every eighth column, lane t gets the eight
// columns from 8 t on: a transpose of 4 x 4 pairs in two rounds. v: pairs 0..3 of this lane.
__device__ __forceinline__ void row_pieces(float (&v)[8], int t) {
#pragma unroll
  for (int bit = 1; bit <= 2; bit *= 2)
#pragma unroll
    for (int i = 0; i < 4; ++i)
      if (!(i & bit))
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          float& a = v[2 * i + e];
          float& b = v[2 * (i + bit) + e];
          const bool up = t & bit;
          const float got = __shfl_xor_sync(0xffffffffu, up ? a : b, bit);
          (up ? a : b) = got;
        }
}
__device__ __forceinline__ void st_cluster_v4(uint32_t addr, float4 v) {
  asm volatile("st.shared::cluster.v4.f32 [%0], {%1, %2, %3, %4};" ::"r"(addr), "f"(v.x), "f"(v.y), "f"(v.z), "f"(v.w) : "memory");
}
__device__ __forceinline__ void st_cluster_v2(uint32_t addr, uint32_t a, uint32_t b) {
  asm volatile("st.shared::cluster.v2.b32 [%0], {%1, %2};" ::"r"(addr), "r"(a), "r"(b) : "memory");
}
__device__ __forceinline__ float4 ld_shared_f4(uint32_t addr) {
  const uint4 v = ld_shared_v4(addr);
  return make_float4(__uint_as_float(v.x), __uint_as_float(v.y), __uint_as_float(v.z), __uint_as_float(v.w));
}

// Eight consecutive addends of a row as they are in memory; the output's of eight sums.
template <int kAdd>
struct Addends {
  uint4 w[kAdd == kTypeF32 ? 2 : 1];
  __device__ __forceinline__ void load(const LoraArgs& a, long long at) {
    const uint4* p = reinterpret_cast<const uint4*>(static_cast<const char*>(a.add) + at * (kAdd == kTypeF32 ? 4 : 2));
    w[0] = p[0];
    if constexpr (kAdd == kTypeF32) w[1] = p[1];
  }
  __device__ __forceinline__ float operator[](int i) const {
    if constexpr (kAdd == kTypeF32) {
      const uint4 v = w[i >> 2];
      return __uint_as_float((i & 3) == 0 ? v.x : (i & 3) == 1 ? v.y : (i & 3) == 2 ? v.z : v.w);
    } else {
      const uint32_t v = (i >> 1) == 0 ? w[0].x : (i >> 1) == 1 ? w[0].y : (i >> 1) == 2 ? w[0].z : w[0].w;
      return __uint_as_float(i & 1 ? v & 0xFFFF0000u : v << 16);
    }
  }
};
template <>
struct Addends<-1> {
  __device__ __forceinline__ void load(const LoraArgs&, long long) {}
  __device__ __forceinline__ float operator[](int) const { return 0.f; }
};

template <int kOut>
__device__ __forceinline__ void store_cols(const LoraArgs& a, long long at, const float (&y)[8]) {
  if constexpr (kOut == kTypeF32) {
    float4* p = reinterpret_cast<float4*>(static_cast<float*>(a.out) + at);
    p[0] = make_float4(y[0], y[1], y[2], y[3]);
    p[1] = make_float4(y[4], y[5], y[6], y[7]);
  } else {
    uint32_t w[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const __nv_bfloat162 h = __floats2bfloat162_rn(y[2 * i], y[2 * i + 1]);
      w[i] = *reinterpret_cast<const uint32_t*>(&h);
    }
    *reinterpret_cast<uint4*>(static_cast<uint16_t*>(a.out) + at) = make_uint4(w[0], w[1], w[2], w[3]);
  }
}

// kAdd: the addends' type, -1 without; kOut: the output's.
template <int kAdd, int kOut>
__global__ void __launch_bounds__(kThreads, 1)
    lora_many_kernel(const __grid_constant__ CUtensorMap amap, const __grid_constant__ CUtensorMap bmap, const __grid_constant__ LoraArgs a, const Order order,
                     const ManyPlan plan, uint32_t limit, int test_never_wait, int32_t* status) {
  extern __shared__ uint8_t smem_raw[];
  const uint32_t base = (smem_u32(smem_raw) + 1023u) & ~1023u;
  uint8_t* gbase = smem_raw + (base - smem_u32(smem_raw));
  const int S = plan.stages;
  auto full = [&](int i) { return base + 8 * i; };
  auto empty = [&](int i) { return base + 8 * (kMaxStages + i); };
  auto tfull = [&](int i) { return base + 8 * (2 * kMaxStages + i); };
  auto tempty = [&](int i) { return base + 8 * (2 * kMaxStages + 2 + i); };
  const uint32_t summed = base + 8 * (2 * kMaxStages + 4), drain = summed + 8, never = summed + 16;
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(gbase + 256);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(gbase + 260);
  int* row_of = reinterpret_cast<int*>(gbase + 1024);  // [128] the tile's rows, -1 behind the last
  const uint32_t parts_at = base + kHead;              // second product's operand: blocks of 128 rows x 64 columns
  const int part_blocks = (plan.parts * plan.rank16 + kChunk - 1) / kChunk;
  const uint32_t sums_at = parts_at + part_blocks * kBox;  // arriving sums: [CTA][r / 4][row] of four
  const uint32_t ring = sums_at + kTile * plan.rank16 * 4;

  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int C = plan.ctas, rank = C > 1 ? static_cast<int>(cluster_rank()) : 0;
  const int tile = blockIdx.x / C;
  int* bucket = reinterpret_cast<int*>(gbase + 264);
  if (threadIdx.x == 0) *bucket = -1;
  __syncthreads();
  pdl_wait();
  const int32_t* slots = order.slots + static_cast<long long>(tile) * kTile;
  const int my_row = threadIdx.x < kTile ? slots[threadIdx.x] : -1;
  for (int e = threadIdx.x; e <= a.L; e += kThreads)  // the tile's bucket, if it has one
    if (order.offsets[e] <= tile * kTile && tile * kTile < order.offsets[e + 1]) *bucket = e;
  if (threadIdx.x < kTile) row_of[threadIdx.x] = my_row;
  __syncthreads();
  const int l = *bucket;
  if (l < 0) return;  // (the whole cluster)
  const int nt = (a.N + kTile - 1) / kTile, nper = (nt + C - 1) / C;
  const int nt0 = min(nt, rank * nper), nt1 = min(nt, nt0 + nper);
  if (l == a.L) {  // rows without an adapter
    if (a.add == a.out) return;
    const int n0 = nt0 * kTile, pieces = (min(a.N, nt1 * kTile) - n0) / 8;
    for (int i = warp; i < kTile; i += kThreads / 32) {
      const int m = row_of[i];
      if (m < 0) break;
      for (int v = lane; v < pieces; v += 32) {
        const long long at = static_cast<long long>(m) * a.N + n0 + 8 * v;
        float d[8];
        load8(a, at, d);
        store8(a, at, d);
      }
    }
    return;
  }
  if (threadIdx.x == 0) {
    tma_prefetch_map(&amap);
    tma_prefetch_map(&bmap);
    for (int i = 0; i < S; ++i) mbar_init(full(i), 1 + kEpiThreads), mbar_init(empty(i), 1);
    for (int i = 0; i < 2; ++i) mbar_init(tfull(i), 1), mbar_init(tempty(i), kEpiWarps);
    mbar_init(summed, 1);
    mbar_init(drain, 1);
    mbar_init(never, 1);
    *abort_flag = 0;
    fence_mbar_init();
  }
  if (warp == kWarpMma) {
    __syncwarp();
    tmem_alloc(smem_u32(tmem_slot), 2 * kTile);
    tmem_relinquish();
  }
  tc_fence_before();
  __syncthreads();
  cluster_sync();  // (every CTA runs before another writes to it)
  tc_fence_after();
  const uint32_t tmem = *tmem_slot;

  const int chunks = (a.K + kChunk - 1) / kChunk, cper = (chunks + C - 1) / C;
  const int c0 = min(chunks, rank * cper), c1 = min(chunks, c0 + cper);
  const int kn = c1 - c0, nn = nt1 - nt0;  // this CTA's stages of x, its column tiles
  const int ahead = min(nn, S);            // column tiles copied before the join
  const int wide = plan.rank16 > kChunk ? 2 : 1;  // boxes of a row of b
  auto slot_of = [&](int i) { return ring + (i % S) * plan.stage_bytes; };
  // what the copying lane issues as item i: a stage of a, or a tile of b (and then the arrivals
  // of the threads too, which copy no x into it)
  bool copying = true;
  int issued = 0;
  const uint64_t keep = l2_policy_evict_last();
  auto copy = [&](int i) {
    if (!mbar_wait(empty(i % S), ((i / S) & 1) ^ 1, abort_flag, status, kStatusTimeout, limit)) return false;
    if (i < kn) {
      mbar_arrive_expect_tx(full(i % S), plan.rank16 * 128);
      tma_load_2d(slot_of(i) + kBox, &amap, (c0 + i) * 128, l * a.r, full(i % S), keep);
    } else {
      const int n0 = (nt0 + i - kn) * kTile;
      mbar_arrive_cnt(full(i % S), kEpiThreads);
      mbar_arrive_expect_tx(full(i % S), wide * kBox);
      for (int b = 0; b < wide; ++b) tma_load_2d(slot_of(i) + b * kBox, &bmap, b * 128, l * a.N + n0, full(i % S), keep);
    }
    return true;
  };

  // the output of a joining lane: of each tile eight columns of four rows
  const int col = (warp >> 2) * kCols + 8 * (lane & 3);
  int m[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) m[i] = row_of[(warp & 3) * 32 + 8 * i + (lane >> 2)];
  auto at_of = [&](int i, int j) { return static_cast<long long>(m[i]) * a.N + (nt0 + j) * kTile + col; };
  auto has = [&](int i, int j) { return m[i] >= 0 && j < nn && (nt0 + j) * kTile + col < a.N; };
  auto ask_addends = [&](int j) {
    if (kAdd >= 0)
#pragma unroll
      for (int i = 0; i < 4; ++i)
        if (has(i, j)) prefetch_l2(static_cast<const char*>(a.add) + at_of(i, j) * (kAdd == kTypeF32 ? 4 : 2));
  };

  // ---- 1. this CTA's columns of a[l] x
  bool ok = true;
  if (warp == kWarpCopy) {
    if (lane == 0)
      for (; issued < kn + ahead; ++issued)
        if (!(copying = copy(issued))) break;
    __syncwarp();
  } else if (warp == kWarpMma) {
    const uint32_t idesc = idesc_bf16_f32(kTile, plan.rank16);
    const bool leader = elect_one();
    for (int i = 0; i < kn; ++i) {
      ok = __all_sync(0xffffffffu, mbar_wait(full(i % S), (i / S) & 1, abort_flag, status, kStatusTimeout, limit));
      if (!ok) break;
      fence_proxy_async_smem();  // (x came by ordinary copies, which the threads do not wait for themselves)
      tc_fence_after();
      if (leader) {
        const uint64_t ad = sw128_kmajor_desc(slot_of(i)), bd = sw128_kmajor_desc(slot_of(i) + kBox);
#pragma unroll
        for (int k = 0; k < kChunk / 16; ++k) tc_mma_bf16(tmem, ad + 2 * k, bd + 2 * k, idesc, i + k > 0);
        tc_commit(empty(i % S));
      }
      __syncwarp();
    }
    if (leader) tc_commit(summed);
    __syncwarp();
  } else {
    // the first column tiles' addends are asked into L2 meanwhile
    for (int j = 0; j < min(kAhead, nn); ++j) ask_addends(j);
    // a thread copies the same 16 bytes of each stage's 128 of two rows; the rows' 16-byte
    // pieces are swizzled as the MMA reads them
    {
      const int piece = threadIdx.x & 7, row = threadIdx.x >> 3;
      const int m0 = row_of[row], m1 = row_of[row + kTile / 2];
      const uint16_t* x0 = a.x + max(m0, 0) * a.ldx + 8 * piece;
      const uint16_t* x1 = a.x + max(m1, 0) * a.ldx + 8 * piece;
      const uint32_t at = row * 128 + ((piece ^ (row & 7)) << 4);
      for (int i = 0; i < kn; ++i) {
        ok = ok && __all_sync(0xffffffffu, mbar_wait(empty(i % S), ((i / S) & 1) ^ 1, abort_flag, status, kStatusTimeout, limit));
        if (!ok) break;
        const int k = (c0 + i) * kChunk;
        const bool in = k + 8 * piece < a.K;
        copy16(slot_of(i) + at, in ? x0 + k : x0, in && m0 >= 0 ? 16 : 0);
        copy16(slot_of(i) + at + kBox / 2, in ? x1 + k : x1, in && m1 >= 0 ? 16 : 0);
        copies_arrive(full(i % S));
      }
      asm volatile("cp.async.wait_all;" ::: "memory");
    }
    if (test_never_wait) ok = __all_sync(0xffffffffu, mbar_wait(never, 0, abort_flag, status, kStatusTimeout, limit));
    ok = ok && __all_sync(0xffffffffu, mbar_wait(summed, 0, abort_flag, status, kStatusTimeout, limit));
    tc_fence_after();
    // ---- 2. to the row's CTA
    const int row = (warp & 3) * 32 + lane, share = kTile / C;
    const uint32_t to = map_rank(sums_at + (rank * (plan.rank16 / 4) * share + row % share) * 16, row / share);
    for (int c = warp >> 2; c < plan.rank16 / 16; c += kEpiWarps / 4) {
      uint32_t v[16] = {};
      if (ok && kn > 0) {
        tmem_ld16(tmem + (static_cast<uint32_t>((warp & 3) * 32) << 16) + 16 * c, v);
        tmem_ld_wait();
      }
#pragma unroll
      for (int i = 0; i < 4; ++i)
        st_cluster_v4(to + (4 * c + i) * share * 16, make_float4(__uint_as_float(v[4 * i]), __uint_as_float(v[4 * i + 1]),
                                                                __uint_as_float(v[4 * i + 2]), __uint_as_float(v[4 * i + 3])));
    }
    tc_fence_before();
  }
  __syncwarp();
  cluster_sync();
  {
    const int share = kTile / C, quads = plan.rank16 / 4;
    const float scale = a.scale ? a.scale[l] : 1.f;
    for (int i = threadIdx.x; i < share * quads; i += kThreads) {
      const int q = i / share, row = rank * share + i % share;
      float s[4] = {};
      for (int c = 0; c < C; ++c) {
        const float4 v = ld_shared_f4(sums_at + ((c * quads + q) * share + i % share) * 16);
        s[0] += v.x, s[1] += v.y, s[2] += v.z, s[3] += v.w;
      }
#pragma unroll
      for (int j = 0; j < 4; ++j) s[j] = 4 * q + j < a.r ? s[j] * scale : 0.f;  // (behind r stand the next adapter's)
      for (int p = 0; p < plan.parts; ++p) {
        uint16_t h[4];
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          h[j] = bf16_part(s[j]);
          s[j] = isfinite(s[j]) ? s[j] - bf16_value(h[j]) : 0.f;
        }
        const int k = p * plan.rank16 + 4 * q;  // column of the operand, 8 bytes within its 16
        const uint32_t at = parts_at + k / kChunk * kBox + row * 128 + ((((k % kChunk) >> 3) ^ (row & 7)) << 4) + (k & 4) * 2;
        for (int c = 0; c < C; ++c)
          st_cluster_v2(map_rank(at, c), h[0] | static_cast<uint32_t>(h[1]) << 16, h[2] | static_cast<uint32_t>(h[3]) << 16);
      }
    }
  }
  asm volatile("fence.proxy.async;" ::: "memory");  // (the MMAs read what was written here)
  __syncwarp();
  cluster_sync();
  asm volatile("fence.proxy.async;" ::: "memory");
  tc_fence_after();

  // ---- 3. this CTA's columns of the output
  if (warp == kWarpCopy) {
    if (lane == 0) {
      for (; issued < kn + nn && copying; ++issued)
        if (!(copying = copy(issued))) break;
      // the last copies have landed, and the MMAs' last signals, before shared memory is given up
      for (int i = max(0, issued - S); i < issued; ++i)
        if (!mbar_wait(empty(i % S), (i / S) & 1, abort_flag, status, kStatusTimeout, limit)) break;
    }
    __syncwarp();
    if (*abort_flag) {  // (copies and signals that nobody waited for get 2 ms)
      const long long t0 = clock64();
      while (clock64() - t0 < 4000000) {
      }
    }
  } else if (warp == kWarpMma) {
    const uint32_t idesc = idesc_bf16_f32(kTile, kTile);
    const bool leader = elect_one();
    for (int j = 0; j < nn && ok; ++j) {
      const int i = kn + j, buf = j & 1;
      ok = __all_sync(0xffffffffu, mbar_wait(full(i % S), (i / S) & 1, abort_flag, status, kStatusTimeout, limit) &&
                                       mbar_wait(tempty(buf), ((j >> 1) & 1) ^ 1, abort_flag, status, kStatusTimeout, limit));
      if (!ok) break;
      tc_fence_after();
      if (leader) {
        // (the small parts first)
        uint32_t more = 0;
        for (int p = plan.parts - 1; p >= 0; --p)
          for (int k = 0; k < plan.rank16; k += 16) {
            const int at = p * plan.rank16 + k;
            const uint64_t ad = sw128_kmajor_desc(parts_at + at / kChunk * kBox) + (at % kChunk) / 8;
            const uint64_t bd = sw128_kmajor_desc(slot_of(i) + k / kChunk * kBox) + (k % kChunk) / 8;
            tc_mma_bf16(tmem + buf * kTile, ad, bd, idesc, more);
            more = 1;
          }
        tc_commit(empty(i % S));
        tc_commit(tfull(buf));
      }
      __syncwarp();
    }
    if (leader) {  // tensor memory is freed only after the last MMAs, whoever gave up
      tc_commit(drain);
      mbar_drain(drain, 0);
    }
    __syncwarp();
  } else {
    const uint32_t src = tmem + (static_cast<uint32_t>((warp & 3) * 32) << 16) + (warp >> 2) * kCols;
    Addends<kAdd> next[4];
    auto load = [&](int j) {
#pragma unroll
      for (int i = 0; i < 4; ++i)
        if (has(i, j)) next[i].load(a, at_of(i, j));
    };
    load(0);
    for (int j = 0; j < nn; ++j) {
      const int buf = j & 1;
      ok = ok && __all_sync(0xffffffffu, mbar_wait(tfull(buf), (j >> 1) & 1, abort_flag, status, kStatusTimeout, limit));
      if (!ok) break;
      tc_fence_after();
      uint32_t v[2][16];
      tmem_ld_16x32(src + buf * kTile, v[0]);
      tmem_ld_16x32(src + buf * kTile + (16u << 16), v[1]);
      if (j + kAhead < nn) ask_addends(j + kAhead);
      Addends<kAdd> now[4];
#pragma unroll
      for (int i = 0; i < 4; ++i) now[i] = next[i];
      load(j + 1);
      tmem_ld_wait();
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive(tempty(buf));
#pragma unroll
      for (int i = 0; i < 4; ++i) {  // rows 8 i + lane / 4
        float y[8];
#pragma unroll
        for (int k = 0; k < 4; ++k)
#pragma unroll
          for (int e = 0; e < 2; ++e) y[2 * k + e] = __uint_as_float(v[i >> 1][4 * k + 2 * (i & 1) + e]);
        row_pieces(y, lane & 3);
#pragma unroll
        for (int k = 0; k < 8; ++k) y[k] += now[i][k];
        if (has(i, j)) store_cols<kOut>(a, at_of(i, j), y);
      }
    }
  }
  __syncwarp();
  tc_fence_before();
  __syncthreads();
  if (warp == kWarpMma) {
    __syncwarp();
    tc_fence_after();
    tmem_dealloc(tmem, 2 * kTile);
  }
}

size_t align_up(size_t x) { return (x + 255) / 256 * 256; }
int order_rows(int M, int L) {  // rows of the sorted order, whole tiles
  const int buckets = std::min(L + 1, M);
  return M + buckets * (kTile - 1);
}

ManyPlan plan_many(const LoraArgs& a, int num_sms) {
  ManyPlan p{};
  p.parts = a.out_type == kTypeF32 ? 3 : 2;
  p.rank16 = (a.r + 15) / 16 * 16;
  p.stage_bytes = kBox + (p.rank16 > kChunk ? kBox : p.rank16 * 128);
  const int fixed = kHead + 1024 + (p.parts * p.rank16 + kChunk - 1) / kChunk * kBox + kTile * p.rank16 * 4;
  p.stages = std::min(kMaxStages, (kSmemMost - fixed) / p.stage_bytes);
  p.smem = fixed + p.stages * p.stage_bytes;
  p.tiles = order_rows(a.M, a.L) / kTile;
  // CTAs to a tile: as many as leave the tiles that there will be about (half an extra one
  // for each adapter) in one wave
  const int about = (a.M + kTile - 1) / kTile + std::min(a.L, a.M / kTile) / 2;
  p.ctas = 8;
  while (p.ctas > 1 && about * p.ctas > num_sms) p.ctas /= 2;
  return p;
}

bool make_bf16_map(CUtensorMap* map, const void* base, long long rows, long long cols, long long stride, int box_rows) {
  return make_byte_map(map, base, rows, 2 * cols, 2 * stride, box_rows);
}

}  // namespace

size_t lora_many_workspace(int M, int L) {
  return align_up(sizeof(int32_t) * (L + 2)) + align_up(sizeof(int32_t) * static_cast<size_t>(order_rows(M, L)));
}

namespace {
template <int kAdd, int kOut>
cudaError_t launch(const LoraArgs& a, const CUtensorMap& amap, const CUtensorMap& bmap, const Order& order, const ManyPlan& p,
                   cudaStream_t stream) {
  static PerDevice<int> ready;
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  std::atomic<int>* entry = ready.of(dev);
  if (!entry || !entry->load()) {
    e = cudaFuncSetAttribute(lora_many_kernel<kAdd, kOut>, cudaFuncAttributeMaxDynamicSharedMemorySize, kSmemMost);
    if (e != cudaSuccess) return e;
    if (entry) entry->store(1);
  }
  int32_t* status = fp8_status_word();
  if (!status) return cudaErrorInvalidSymbol;
  uint32_t limit;
  int never;
  fp8_wait_settings(&limit, &never);
  return launch_cluster(lora_many_kernel<kAdd, kOut>, dim3(static_cast<unsigned>(p.tiles) * p.ctas), dim3(kThreads), p.smem, stream,
                        p.ctas, amap, bmap, a, order, p, limit, never, status);
}
}  // namespace

cudaError_t launch_lora_many(const LoraArgs& a, int num_sms, cudaStream_t stream) {
  auto* offsets = static_cast<int32_t*>(a.workspace);
  auto* slots = reinterpret_cast<int32_t*>(static_cast<uint8_t*>(a.workspace) + align_up(sizeof(int32_t) * (a.L + 2)));
  CUtensorMap amap, bmap;
  if (!make_bf16_map(&amap, a.a, static_cast<long long>(a.L) * a.r, a.K, a.K, (a.r + 15) / 16 * 16) ||
      !make_bf16_map(&bmap, a.b, static_cast<long long>(a.L) * a.N, a.r, a.r, kTile))
    return cudaErrorInvalidValue;
  const cudaError_t e = launch_sort(SortArgs{a.index, a.M, 0, a.L, 1, kTile, offsets, slots, order_rows(a.M, a.L), nullptr}, stream);
  if (e != cudaSuccess) return e;
  const ManyPlan p = plan_many(a, num_sms);
  const Order order{offsets, slots};
  auto go = [&](auto out) {
    constexpr int kOut = decltype(out)::value;
    if (!a.add) return launch<-1, kOut>(a, amap, bmap, order, p, stream);
    return a.add_type == kTypeF32 ? launch<kTypeF32, kOut>(a, amap, bmap, order, p, stream)
                                  : launch<kTypeBf16, kOut>(a, amap, bmap, order, p, stream);
  };
  return a.out_type == kTypeF32 ? go(std::integral_constant<int, kTypeF32>{}) : go(std::integral_constant<int, kTypeBf16>{});
}

}  // namespace moe
