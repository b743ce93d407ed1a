// Low-rank adapters, many rows: out[m] = add[m] + scale[l] b[l] (a[l] x[m]), l = index[m].
//
// The rows of an adapter make tiles of 128 (rows without one are the last adapter's). Up to
// 1,536 rows each CTA finds its tile's rows itself: it counts the rows of every adapter and
// looks its own tile's up. Above, they are sorted first (the order of dispatch.cu). (8 adapters
// of rank 64, 900 rows: 24.7 us, 28.2 sorted first; 1,200: 32.2 and 33.1; 1,500: 35.6 and 35.0;
// 2,048: 38.5 and 38.2; 4,096: 58.6 and 55.0.) A cluster of CTAs takes a tile. Each CTA
//   1. sums its share of a[l] x's columns: tcgen05 MMAs of 128 rows x r, whose x rows are
//      copied from wherever they lie;
//   2. joins the sums with the cluster's other CTAs: each sends its sums of a row to the
//      row's CTA, which adds them in the order of the ranks, scales them, splits them into
//      three bf16 parts (all 24 bits of the sum) and hands them to all CTAs, straight into
//      the second product's operand;
//   3. computes its share of the N columns: MMAs of 128 rows x 128 columns over the parts,
//      one after another against the same tile of b[l], two accumulators in turn, taken out
//      of tensor memory by eight warps that add the addends, which each thread has copied
//      for itself to shared memory some pieces ahead, and write the output.
// Two CTAs share an SM where the rank allows, so that one reads x while the other joins or
// writes. Nothing but x, a, b, the addends and the output goes through memory, and each once
// (a and b once for each tile, from L2). The operations are few, r of them for a byte at
// most: what bounds it is memory, if the copies and the output take few instructions:
//   - Operands come by 16-byte copies of single threads, zeros where there is no row or
//     column. (The copy engine's gathers of four rows of 128 bytes take 18 cycles a row
//     here: 2,370 cycles for a stage of x, which these bring in 500.) 64 threads copy a
//     stage of x: each arrives at the stage's barrier by itself, and 256 arrivals took as
//     long as the copies.
//   - b's rows are copied in such an order that the four lanes that get a row's sums out of
//     tensor memory get eight consecutive columns each, not pairs of columns: the addends
//     and the output move in 16- and 32-byte pieces, 64 or 128 bytes of a row to four
//     lanes, without an exchange. (A row to a lane, 32 lines to an access: 4,000 cycles a
//     tile; exchanges: 3,300.)
//   - Addends that wait in registers wait for one another: a warp tells its loads under way
//     apart by few marks, and three halves of a tile ahead took twice as long as one.
//
// Warps: 0..7 x, joining and output, 8 the copies of a and b, 9 the MMAs. All sums have a
// fixed order.
#include <algorithm>

#include "fp8_tma.cuh"
#include "lora.cuh"

namespace moe {
namespace {

constexpr int kTile = 128;         // rows of a tile, columns of an accumulator
constexpr int kChunk = 64;         // columns of x to a stage: 128 bytes
constexpr int kBox = kTile * 128;  // bytes of 128 rows of 128 bytes
constexpr int kEpiWarps = 8, kEpiThreads = kEpiWarps * 32, kWarpCopy = 8, kWarpMma = 9, kThreads = 10 * 32;
constexpr int kCols = kTile * 4 / kEpiWarps;  // of an accumulator, to a warp, 32 at a time
constexpr int kTeam = 64, kTeams = 2;  // threads that copy a stage of x, by turns
// A team asks a stage's barrier for a phase by its parity, which two phases share, and only
// every kTeams-th stage. Its last answer says that the MMAs of kTeams + S stages ago are done;
// that those of 2 S ago are, whose phase has the same parity, follows if kTeams <= S. (Four
// teams and three stages overwrote stages in use, until waits ran out.)
constexpr int kLeastStages = 3;
static_assert(kTeams <= kLeastStages, "a parity is answered by the phase before the last");
constexpr int kMaxStages = 6;
constexpr int kHead = 2048;        // barriers, the tile's rows
constexpr int kSmemMost = 227 * 1024, kSmemHalf = 113 * 1024;
// (Two CTAs to an SM at most, and beside them none of another kernel that takes tensor memory:
// CTAs of a cluster wait for one another with their part of it in hand.)
constexpr int kSmemLeast = 96 * 1024;

struct ManyPlan {
  int ctas;         // to a tile
  int rank16;       // r, up to a multiple of 16
  int stages, stage_bytes, smem;
  int b_stages;     // tiles of b under way,
  int b_early;      // and those of them whose place is free while the sums are joined
  int deep;         // pieces of addends under way
  int tiles;        // at most
};
constexpr int kSelfRows = 1536;  // rows up to which each CTA looks for its own
struct Order {
  const int32_t* offsets;  // [L + 2], null: there is none
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
// Column of a block of 32 whose b row stands in the operand's row c: columns 8 i + 2 t + e
// of the sums, those of lane 4 g + t above, are its columns 8 t + 2 i + e.
__device__ __forceinline__ int column_at(int c) { return 8 * ((c >> 1) & 3) + 2 * (c >> 3) + (c & 1); }
__device__ __forceinline__ void st_cluster_v4(uint32_t addr, float4 v) {
  asm volatile("st.shared::cluster.v4.f32 [%0], {%1, %2, %3, %4};" ::"r"(addr), "f"(v.x), "f"(v.y), "f"(v.z), "f"(v.w) : "memory");
}
__device__ __forceinline__ void st_cluster_b4(uint32_t addr, const uint32_t (&w)[4]) {
  asm volatile("st.shared::cluster.v4.b32 [%0], {%1, %2, %3, %4};" ::"r"(addr), "r"(w[0]), "r"(w[1]), "r"(w[2]), "r"(w[3]) : "memory");
}
__device__ __forceinline__ float4 ld_shared_f4(uint32_t addr) {
  const uint4 v = ld_shared_v4(addr);
  return make_float4(__uint_as_float(v.x), __uint_as_float(v.y), __uint_as_float(v.z), __uint_as_float(v.w));
}

// All but the last `left` groups of this thread's copies have landed.
constexpr int kMaxDeep = 6;
__device__ __forceinline__ void copies_left(int left) {
  switch (left) {
    case 0: asm volatile("cp.async.wait_group 0;" ::: "memory"); break;
    case 1: asm volatile("cp.async.wait_group 1;" ::: "memory"); break;
    case 2: asm volatile("cp.async.wait_group 2;" ::: "memory"); break;
    case 3: asm volatile("cp.async.wait_group 3;" ::: "memory"); break;
    case 4: asm volatile("cp.async.wait_group 4;" ::: "memory"); break;
    default: asm volatile("cp.async.wait_group 5;" ::: "memory"); break;
  }
}
static_assert(kMaxDeep - 1 <= 5, "cases above");
// The two halves of cluster_sync().
__device__ __forceinline__ void cluster_arrive() { asm volatile("barrier.cluster.arrive.release.aligned;" ::: "memory"); }
__device__ __forceinline__ void cluster_wait() { asm volatile("barrier.cluster.wait.acquire.aligned;" ::: "memory"); }

// Eight consecutive addends of a row, as a thread copied them (a row's bytes of all threads:
// kAddBytes), and eight values of the output.
template <int kAdd>
constexpr int kAddBytes = kEpiThreads * 16 * (kAdd == kTypeF32 ? 2 : 1);
template <int kAdd>
__device__ __forceinline__ void load_addends(uint32_t at, float (&y)[8]) {
  if constexpr (kAdd == kTypeF32) {
    const float4 u = ld_shared_f4(at), v = ld_shared_f4(at + kEpiThreads * 16);
    y[0] = u.x, y[1] = u.y, y[2] = u.z, y[3] = u.w, y[4] = v.x, y[5] = v.y, y[6] = v.z, y[7] = v.w;
  } else {
    const uint4 u = ld_shared_v4(at);
    const uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) y[2 * i] = __uint_as_float(w[i] << 16), y[2 * i + 1] = __uint_as_float(w[i] & 0xFFFF0000u);
  }
}
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
__global__ void __launch_bounds__(kThreads, 2)
    lora_many_kernel(const __grid_constant__ LoraArgs a, const Order order, const ManyPlan plan, uint32_t limit, int test_never_wait, int32_t* status) {
  extern __shared__ uint8_t smem_raw[];
  const uint32_t base = (smem_u32(smem_raw) + 1023u) & ~1023u;
  uint8_t* gbase = smem_raw + (base - smem_u32(smem_raw));
  const int S = plan.stages;
  auto full = [&](int i) { return base + 8 * i; };
  auto empty = [&](int i) { return base + 8 * (kMaxStages + i); };
  auto tfull = [&](int i) { return base + 8 * (2 * kMaxStages + i); };
  auto tempty = [&](int i) { return base + 8 * (2 * kMaxStages + 2 + i); };
  auto bfull = [&](int i) { return base + 8 * (2 * kMaxStages + 8 + i); };
  auto bempty = [&](int i) { return base + 8 * (2 * kMaxStages + 10 + i); };
  const uint32_t summed = base + 8 * (2 * kMaxStages + 4), drain = summed + 8, never = summed + 16;
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(gbase + 256);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(gbase + 260);
  int* row_of = reinterpret_cast<int*>(gbase + 1024);  // [128] the tile's rows, -1 behind the last
  // Arriving sums: [CTA][r / 4][row] of four; then the stages of x and a. When those are done,
  // at the end of their place the second product's operand (blocks of 128 rows x 64 columns),
  // in front of it tiles of b (the last ones partly in the sums' place, and copied when those
  // are joined); and when the sums are joined, up to there addends.
  const uint32_t sums_at = base + kHead, ring = sums_at + kTile * plan.rank16 * 4, adds_at = sums_at;
  const int wide = plan.rank16 > kChunk ? 2 : 1;  // boxes of a row of b
  const uint32_t parts_at = base + plan.smem - 1024 - (kParts * plan.rank16 + kChunk - 1) / kChunk * kBox;
  const uint32_t b_ring = parts_at - plan.b_stages * wide * kBox;

  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int C = plan.ctas, rank = C > 1 ? static_cast<int>(cluster_rank()) : 0;
  const int tile = blockIdx.x / C;
  int* bucket = reinterpret_cast<int*>(gbase + 264);
  if (threadIdx.x == 0) {
    for (int i = 0; i < S; ++i) mbar_init(full(i), kTeam + 32), mbar_init(empty(i), 1);
    for (int i = 0; i < 2; ++i) mbar_init(bfull(i), 32), mbar_init(bempty(i), 1);
    for (int i = 0; i < 2; ++i) mbar_init(tfull(i), 1), mbar_init(tempty(i), kEpiWarps);
    mbar_init(summed, 1);
    mbar_init(drain, 1);
    mbar_init(never, 1);
    *abort_flag = 0;
    *bucket = -1;
    fence_mbar_init();
  }
  if (order.offsets) {
    __syncthreads();
    pdl_wait();
    const int32_t* slots = order.slots + static_cast<long long>(tile) * kTile;
    const int my_row = threadIdx.x < kTile ? slots[threadIdx.x] : -1;
    for (int e = threadIdx.x; e <= a.L; e += kThreads)  // the tile's bucket, if it has one
      if (order.offsets[e] <= tile * kTile && tile * kTile < order.offsets[e + 1]) *bucket = e;
    if (threadIdx.x < kTile) row_of[threadIdx.x] = my_row;
    __syncthreads();
  } else {
    // (in the place of what arrives later)
    uint16_t* bucket_of = reinterpret_cast<uint16_t*>(gbase + kHead);  // [kSelfRows]
    int* count = reinterpret_cast<int*>(bucket_of + kSelfRows);        // [L + 1]
    int* seen = reinterpret_cast<int*>(gbase + 512);                   // [warps] rows of the bucket in a warp's part
    int* skip = bucket + 1;  // rows of the bucket in front of the tile
    constexpr int kWarps = kThreads / 32;
    for (int e = threadIdx.x; e <= a.L; e += kThreads) count[e] = 0;
    if (threadIdx.x < kTile) row_of[threadIdx.x] = -1;
    __syncthreads();
    pdl_wait();
    const int part = (a.M + 32 * kWarps - 1) / (32 * kWarps) * 32, lo = min(a.M, warp * part), hi = min(a.M, lo + part);
    const int bits = 32 - __clz(a.L);  // of a bucket
    constexpr int kOnce = 4;
    for (int i0 = lo; i0 < hi; i0 += 32 * kOnce) {
      int b[kOnce];
#pragma unroll
      for (int k = 0; k < kOnce; ++k) b[k] = i0 + 32 * k + lane < hi ? a.index[i0 + 32 * k + lane] : 0;
#pragma unroll
      for (int k = 0; k < kOnce; ++k) {
        const int i = i0 + 32 * k + lane;
        if (i0 + 32 * k >= hi) break;
        const int mine = i >= hi ? -1 : static_cast<uint32_t>(b[k]) < static_cast<uint32_t>(a.L) ? b[k] : a.L;
        if (i < hi) bucket_of[i] = static_cast<uint16_t>(mine);
        const unsigned peers = lanes_of(mine, bits);
        if (mine >= 0 && lane == __ffs(peers) - 1) atomicAdd(&count[mine], __popc(peers));
      }
    }
    __syncthreads();
    if (warp == 0) {
      int before = 0;  // tiles of the buckets so far
      for (int b0 = 0; b0 <= a.L && before <= tile; b0 += 32) {
        const int tiles = b0 + lane <= a.L ? (count[b0 + lane] + kTile - 1) / kTile : 0;
        int upto = tiles;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
          const int v = __shfl_up_sync(0xffffffffu, upto, o);
          if (lane >= o) upto += v;
        }
        const int first = before + upto - tiles;
        if (first <= tile && tile < first + tiles) *bucket = b0 + lane, *skip = (tile - first) * kTile;
        before += __shfl_sync(0xffffffffu, upto, 31);
      }
    }
    __syncthreads();
    const int mine = *bucket;
    if (mine >= 0) {
      int n = 0;
      for (int i0 = lo; i0 < hi; i0 += 32) n += __popc(__ballot_sync(0xffffffffu, i0 + lane < hi && bucket_of[i0 + lane] == mine));
      if (lane == 0) seen[warp] = n;
      __syncthreads();  // (all of the CTA's threads come here, or none)
      int at = -*skip;
      for (int w = 0; w < warp; ++w) at += seen[w];
      for (int i0 = lo; i0 < hi && at < kTile; i0 += 32) {
        const unsigned same = __ballot_sync(0xffffffffu, i0 + lane < hi && bucket_of[i0 + lane] == mine);
        const int place = at + __popc(same & ((1u << lane) - 1u));
        if ((same >> lane & 1) && place >= 0 && place < kTile) row_of[place] = i0 + lane;
        at += __popc(same);
      }
      __syncthreads();
    }
  }
  const int l = *bucket;
  if (l < 0) return;  // (the whole cluster)
  // A CTA's share of the columns, of x in stages and of the output in tiles: every C-th, so
  // that a row's neighbouring pieces are read and written at about the same time.
  const int nt = (a.N + kTile - 1) / kTile, chunks = (a.K + kChunk - 1) / kChunk;
  const int nn = nt > rank ? (nt - rank - 1) / C + 1 : 0, kn = chunks > rank ? (chunks - rank - 1) / C + 1 : 0;
  auto tile_col = [&](int j) { return (rank + j * C) * kTile; };
  auto chunk_col = [&](int i) { return (rank + i * C) * kChunk; };
  if (l == a.L) {  // rows without an adapter
    if (a.add == a.out) return;
    for (int i = warp; i < kTile; i += kThreads / 32) {
      const int m = row_of[i];
      if (m < 0) break;
      for (int v = 32 * rank + lane; v < a.N / 8; v += 32 * C) {
        const long long at = static_cast<long long>(m) * a.N + 8 * v;
        float d[8];
        load8(a, at, d);
        store8(a, at, d);
      }
    }
    return;
  }
  if (warp == kWarpMma) {
    __syncwarp();
    tmem_alloc(smem_u32(tmem_slot), 2 * kTile);
    tmem_relinquish();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  cluster_arrive();  // (every CTA runs before another writes to it: waited for in front of that)
  const uint32_t tmem = *tmem_slot;

  auto slot_of = [&](int i) { return ring + (i % S) * plan.stage_bytes; };
  const int SB = plan.b_stages;
  auto b_slot_of = [&](int j) { return parts_at - (j % SB + 1) * wide * kBox; };
  const int piece = lane & 7;  // the 16 bytes of a 128-byte row that this lane copies
  // the copying warp's part of tile j of b: 32 columns at a time, rows in their order
  const uint16_t* b_from = a.b + static_cast<long long>(l) * a.N * a.r;
  auto copy_b = [&](int j) {
    if (!__all_sync(0xffffffffu, mbar_wait(bempty(j % SB), ((j / SB) & 1) ^ 1, abort_flag, status, kStatusTimeout, limit))) return false;
    // lanes of 8 copy a row; row c = lane / 8 + 4 i of the operand, whose column is the sum of
    // those of lane / 8 and 4 i
    const int n0 = tile_col(j) + column_at(lane >> 3);
    const uint32_t to = b_slot_of(j) + (lane >> 3) * 128;
    for (int h = 0; h < wide; ++h) {
      const int k = h * kChunk + 8 * piece;
      const bool whole = tile_col(j) + kTile <= a.N;
      const uint16_t* from = b_from + static_cast<long long>(n0) * a.r + k;
      const uint32_t bytes = k < a.r ? 16 : 0;
      if (bytes == 0) from = a.b;
      const long long one = bytes ? a.r : 0;
#pragma unroll 8
      for (int i = 0; i < kTile / 4; ++i) {
        const int on = (i >> 3) * 32 + column_at((i & 7) * 4);
        const bool in = whole || n0 + on < a.N;
        copy16(to + h * kBox + i * 512 + ((piece ^ ((lane >> 3) + 4 * (i & 1))) << 4), in ? from : a.b, in ? bytes : 0);
        from += one * ((i & 7) == 7 ? 32 - column_at(28) : column_at((i & 7) * 4 + 4) - column_at((i & 7) * 4));
      }
    }
    copies_arrive(bfull(j % SB));
    return true;
  };
  int issued = 0;  // tiles of b

  // The output of a joining lane: eight columns of four rows of each half of its warp's
  // columns of a tile. Piece s: rows 2 (s & 1) and 2 (s & 1) + 1 of half s / 2.
  long long row_at[4];  // -1: no row
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const int m = row_of[(warp & 3) * 32 + 8 * i + (lane >> 2)];
    row_at[i] = m < 0 ? -1 : static_cast<long long>(m) * a.N;
  }
  const int col0 = (warp >> 2) * kCols + 8 * (lane & 3), pieces = 4 * nn;
  auto col_of = [&](int s) { return col0 + tile_col(s >> 2) + (s >> 1 & 1) * 32; };

  // ---- 1. this CTA's columns of a[l] x
  bool ok = true;
  if (warp == kWarpCopy) {
    const uint16_t* from = a.a + (static_cast<long long>(l) * a.r + (lane >> 3)) * a.K + 8 * piece;
    for (int i = 0; i < kn && ok; ++i) {
      ok = __all_sync(0xffffffffu, mbar_wait(empty(i % S), ((i / S) & 1) ^ 1, abort_flag, status, kStatusTimeout, limit));
      if (!ok) break;
      const int k = chunk_col(i);
      const bool in_row = k + 8 * piece < a.K;
      const uint32_t to = slot_of(i) + kBox + (lane >> 3) * 128;
      const uint16_t* p = from + k;
#pragma unroll 4
      for (int j = 0; j < plan.rank16 / 4; ++j, p += 4 * static_cast<long long>(a.K)) {
        const bool in = (lane >> 3) + 4 * j < a.r && in_row;
        copy16(to + j * 512 + ((piece ^ ((lane >> 3) + 4 * (j & 1))) << 4), in ? p : a.a, in ? 16 : 0);
      }
      copies_arrive(full(i % S));
    }
    // (the stages' place is free when all of their MMAs are done)
    ok = ok && __all_sync(0xffffffffu, mbar_wait(summed, 0, abort_flag, status, kStatusTimeout, limit));
    cluster_wait();
    cluster_arrive();  // (the join goes on without this warp, which has tiles of b to copy)
    for (; ok && issued < min(nn, plan.b_early); ++issued) ok = copy_b(issued);
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
    cluster_wait();
    cluster_arrive();
  } else {
    // the first addends are asked into L2 meanwhile
    if (kAdd >= 0)
      for (int s = 0; s < min(pieces, plan.deep); ++s)
#pragma unroll
        for (int i = 0; i < 2; ++i) {
          const long long at = s & 1 ? row_at[2 + i] : row_at[i];
          if (at >= 0 && col_of(s) < a.N) prefetch_l2(static_cast<const char*>(a.add) + (at + col_of(s)) * (kAdd == kTypeF32 ? 4 : 2));
        }
    // the rows' 16-byte pieces are swizzled as the MMA reads them
    const int team = threadIdx.x / kTeam;
    if (team < kTeams) {
      constexpr int kEach = kTile * 8 / kTeam, kStep = kTeam / 8;  // rows of a thread, and from one to the next
      const int first = threadIdx.x % kTeam >> 3;
      const uint16_t* from[kEach];  // (in registers: a look-up between two copies holds up the second)
      uint32_t rows = 0;
#pragma unroll
      for (int j = 0; j < kEach; ++j) {
        const int m = row_of[first + j * kStep];
        rows |= (m >= 0 ? 1u : 0u) << j;
        from[j] = a.x + max(m, 0) * a.ldx + 8 * piece;
      }
      for (int i = team; i < kn; i += kTeams) {
        ok = ok && __all_sync(0xffffffffu, mbar_wait(empty(i % S), ((i / S) & 1) ^ 1, abort_flag, status, kStatusTimeout, limit));
        if (!ok) break;
        const int k = chunk_col(i);
        const bool in_row = k + 8 * piece < a.K;
        const uint32_t to = slot_of(i) + first * 128 + ((piece ^ (first & 7)) << 4);
#pragma unroll
        for (int j = 0; j < kEach; ++j)
          copy16(to + j * kStep * 128, in_row ? from[j] + k : a.x, in_row && (rows >> j & 1) ? 16 : 0);
        copies_arrive(full(i % S));
      }
    }
    asm volatile("cp.async.wait_all;" ::: "memory");
    if (test_never_wait) ok = __all_sync(0xffffffffu, mbar_wait(never, 0, abort_flag, status, kStatusTimeout, limit));
    ok = ok && __all_sync(0xffffffffu, mbar_wait(summed, 0, abort_flag, status, kStatusTimeout, limit));
    tc_fence_after();
    cluster_wait();
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
    __syncwarp();
    cluster_arrive();
  }
  __syncwarp();
  cluster_wait();
  if (warp < kEpiWarps) {
    // a thread: eight columns of a row of this CTA's share
    const int share = kTile / C, quads = plan.rank16 / 4;
    const float scale = a.scale ? a.scale[l] : 1.f;
    for (int i = threadIdx.x; i < share * quads / 2; i += kEpiThreads) {
      const int q = i / share, mine = i % share, row = rank * share + mine;
      float s[8] = {};
      for (int c = 0; c < C; ++c) {
        const uint32_t from = sums_at + ((c * quads + 2 * q) * share + mine) * 16;
        const float4 u = ld_shared_f4(from), v = ld_shared_f4(from + share * 16);
        s[0] += u.x, s[1] += u.y, s[2] += u.z, s[3] += u.w, s[4] += v.x, s[5] += v.y, s[6] += v.z, s[7] += v.w;
      }
#pragma unroll
      for (int j = 0; j < 8; ++j) s[j] = 8 * q < a.r ? s[j] * scale : 0.f;  // (infinite x times the zeros behind r)
#pragma unroll
      for (int p = 0; p < kParts; ++p) {
        uint32_t w[4];
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          const uint16_t lo = bf16_part(s[2 * j]), hi = bf16_part(s[2 * j + 1]);
          s[2 * j] = isfinite(s[2 * j]) ? s[2 * j] - bf16_value(lo) : 0.f;
          s[2 * j + 1] = isfinite(s[2 * j + 1]) ? s[2 * j + 1] - bf16_value(hi) : 0.f;
          w[j] = lo | static_cast<uint32_t>(hi) << 16;
        }
        const int k = p * plan.rank16 + 8 * q;  // column of the operand
        const uint32_t at = parts_at + k / kChunk * kBox + row * 128 + ((((k % kChunk) >> 3) ^ (row & 7)) << 4);
        for (int c = 0; c < C; ++c) st_cluster_b4(map_rank(at, c), w);
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
    for (; ok && issued < nn; ++issued) ok = copy_b(issued);
    asm volatile("cp.async.wait_all;" ::: "memory");
    // the MMAs' last signals have arrived before shared memory is given up
    for (int i = max(0, kn - S); i < kn && ok; ++i)
      ok = __all_sync(0xffffffffu, mbar_wait(empty(i % S), (i / S) & 1, abort_flag, status, kStatusTimeout, limit));
    for (int j = max(0, nn - SB); j < nn && ok; ++j)
      ok = __all_sync(0xffffffffu, mbar_wait(bempty(j % SB), (j / SB) & 1, abort_flag, status, kStatusTimeout, limit));
    if (*abort_flag) {  // (copies and signals that nobody waited for get 2 ms)
      const long long t0 = clock64();
      while (clock64() - t0 < 4000000) {
      }
    }
  } else if (warp == kWarpMma) {
    const uint32_t idesc = idesc_bf16_f32(kTile, kTile);
    const bool leader = elect_one();
    for (int j = 0; j < nn && ok; ++j) {
      const int buf = j & 1;
      ok = __all_sync(0xffffffffu, mbar_wait(bfull(j % SB), (j / SB) & 1, abort_flag, status, kStatusTimeout, limit) &&
                                       mbar_wait(tempty(buf), ((j >> 1) & 1) ^ 1, abort_flag, status, kStatusTimeout, limit));
      if (!ok) break;
      fence_proxy_async_smem();
      tc_fence_after();
      if (leader) {
        // (the small parts first)
        uint32_t more = 0;
        for (int p = kParts - 1; p >= 0; --p)
          for (int k = 0; k < plan.rank16; k += 16) {
            const int at = p * plan.rank16 + k;
            const uint64_t ad = sw128_kmajor_desc(parts_at + at / kChunk * kBox) + (at % kChunk) / 8;
            const uint64_t bd = sw128_kmajor_desc(b_slot_of(j) + k / kChunk * kBox) + (k % kChunk) / 8;
            tc_mma_bf16(tmem + buf * kTile, ad, bd, idesc, more);
            more = 1;
          }
        tc_commit(bempty(j % SB));
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
    const uint32_t mine = adds_at + threadIdx.x * 16;  // [piece][row][16 bytes][thread] of 16
    auto copy_addends = [&](int s, int slot) {
      if constexpr (kAdd >= 0) {
        constexpr int kItem = kAdd == kTypeF32 ? 4 : 2;
        const int n = col_of(s);
#pragma unroll
        for (int i = 0; i < 2; ++i) {
          const long long at = s & 1 ? row_at[2 + i] : row_at[i];
          const bool in = s < pieces && at >= 0 && n < a.N;
          const char* from = static_cast<const char*>(a.add) + (in ? (at + n) * kItem : 0);
#pragma unroll
          for (int h = 0; h < kItem / 2; ++h)
            copy16(mine + ((slot * 2 + i) * (kItem / 2) + h) * kEpiThreads * 16, from + 16 * h, in ? 16 : 0);
        }
        asm volatile("cp.async.commit_group;" ::: "memory");
      }
    };
    const int deep = plan.deep;
    for (int s = 0; s < deep; ++s) copy_addends(s, s);
    int slot = 0;
    for (int s0 = 0; s0 < pieces; s0 += 4) {
      const int j = s0 >> 2, buf = j & 1;
      ok = ok && __all_sync(0xffffffffu, mbar_wait(tfull(buf), (j >> 1) & 1, abort_flag, status, kStatusTimeout, limit));
      if (!ok) break;
      tc_fence_after();
#pragma unroll
      for (int u = 0; u < 4; ++u) {
        const int s = s0 + u, n = col_of(s);
        uint32_t v[16];
        tmem_ld_16x32(src + buf * kTile + (u >> 1) * 32 + (static_cast<uint32_t>(16 * (u & 1)) << 16), v);
        float y[2][8];
        if constexpr (kAdd >= 0) {
          copies_left(deep - 1);
#pragma unroll
          for (int i = 0; i < 2; ++i) load_addends<kAdd>(mine + slot * 2 * kAddBytes<kAdd> + i * kAddBytes<kAdd>, y[i]);
        } else {
#pragma unroll
          for (int i = 0; i < 16; ++i) y[i >> 3][i & 7] = 0.f;
        }
        tmem_ld_wait();
        if (u == 3) {
          tc_fence_before();
          __syncwarp();
          if (lane == 0) mbar_arrive(tempty(buf));
        }
#pragma unroll
        for (int i = 0; i < 2; ++i) {  // rows 8 (2 (u & 1) + i) + lane / 4
#pragma unroll
          for (int k = 0; k < 8; ++k) y[i][k] += __uint_as_float(v[4 * (k >> 1) + 2 * i + (k & 1)]);
          const long long at = row_at[2 * (u & 1) + i];
          if (at >= 0 && n < a.N) store_cols<kOut>(a, at + n, y[i]);
        }
        copy_addends(s + deep, slot);
        if (++slot == deep) slot = 0;
      }
    }
    asm volatile("cp.async.wait_all;" ::: "memory");
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
  p.rank16 = (a.r + 15) / 16 * 16;
  p.stage_bytes = kBox + (p.rank16 > kChunk ? kBox : p.rank16 * 128);
  const int fixed = kHead + 1024 + kTile * p.rank16 * 4;
  const int operand = (kParts * p.rank16 + kChunk - 1) / kChunk * kBox, b_tile = p.rank16 > kChunk ? 2 * kBox : kBox;
  // two CTAs to an SM if at least three stages, and the second product's operands in their
  // place, fit a half
  int room = kSmemHalf - fixed;
  if (room < kLeastStages * p.stage_bytes || room < operand + b_tile) room = kSmemMost - fixed;
  p.stages = std::min(kMaxStages, room / p.stage_bytes);  // (five at the least where one CTA has the SM)
  const bool half = room <= kSmemHalf - fixed;
  const int piece = kEpiThreads * 32 * (a.add_type == kTypeF32 ? 2 : 1);
  const int sums = kTile * p.rank16 * 4;
  p.b_stages = room + sums >= operand + 2 * b_tile + 2 * piece ? 2 : 1;
  const int ring = std::max(p.stages * p.stage_bytes, std::min(room, operand + p.b_stages * b_tile));
  p.smem = std::max(kSmemLeast, fixed + ring);
  p.b_early = std::min(p.b_stages, (p.smem - fixed - operand) / b_tile);
  // (the sums' place and what the ring has left are at least a piece of addends: 8 KB, fp32 16)
  p.deep = std::max(1, std::min(kMaxDeep, (p.smem - kHead - 1024 - operand - p.b_stages * b_tile) / piece));
  const int per_sm = half ? 2 : 1;
  p.tiles = order_rows(a.M, a.L) / kTile;
  // CTAs to a tile: as many as leave the tiles that there will be about (half an extra one
  // for each adapter) in one wave
  const int about = (a.M + kTile - 1) / kTile + std::min(a.L, a.M / kTile) / 2;
  p.ctas = 8;
  while (p.ctas > 1 && about * p.ctas > per_sm * num_sms) p.ctas /= 2;
  return p;
}

}  // namespace

size_t lora_many_workspace(int M, int L) {
  if (M <= kSelfRows) return 0;
  return align_up(sizeof(int32_t) * (L + 2)) + align_up(sizeof(int32_t) * static_cast<size_t>(order_rows(M, L)));
}

namespace {
template <int kAdd, int kOut>
cudaError_t launch(const LoraArgs& a, const Order& order, const ManyPlan& p, cudaStream_t stream) {
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
                        p.ctas, a, order, p, limit, never, status);
}
}  // namespace

cudaError_t launch_lora_many(const LoraArgs& a, int num_sms, cudaStream_t stream) {
  Order order{};
  if (a.M > kSelfRows) {
    auto* offsets = static_cast<int32_t*>(a.workspace);
    auto* slots = reinterpret_cast<int32_t*>(static_cast<uint8_t*>(a.workspace) + align_up(sizeof(int32_t) * (a.L + 2)));
    const cudaError_t e = launch_sort(SortArgs{a.index, a.M, 0, a.L, 1, kTile, offsets, slots, order_rows(a.M, a.L), nullptr}, stream);
    if (e != cudaSuccess) return e;
    order = Order{offsets, slots};
  }
  const ManyPlan p = plan_many(a, num_sms);
  auto go = [&](auto out) {
    constexpr int kOut = decltype(out)::value;
    if (!a.add) return launch<-1, kOut>(a, order, p, stream);
    return a.add_type == kTypeF32 ? launch<kTypeF32, kOut>(a, order, p, stream)
                                  : launch<kTypeBf16, kOut>(a, order, p, stream);
  };
  return a.out_type == kTypeF32 ? go(std::integral_constant<int, kTypeF32>{}) : go(std::integral_constant<int, kTypeBf16>{});
}

}  // namespace moe
