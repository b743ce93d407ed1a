// Low-rank adapters of many requests beside a projection:
//
//   out[m] = add[m] + scale[l] b[l] (a[l] x[m]),  l = index[m]
//
// and out[m] = add[m] for a row without an adapter.
//
// Few rows (a decode step), and any shape and alignment: one launch, in which a cluster of eight CTAs takes up to 16 rows
// of one adapter. Each CTA sums an eighth of a[l] x's products, hands its part to all
// eight, and computes an eighth of the outputs; nothing goes through memory in between.
// Each cluster finds its rows itself: it counts the rows of every adapter (up to 32 rows by
// comparing lanes), 16 of which are a group, and takes the group of its own number (rows without an adapter are the last
// adapter's). There are no more groups than L + 1 + M / 16, or than rows.
// What bounds it is latency (index, then x and a, then the exchange, then b and the
// addends, which are asked into L2 ahead) and from about 32 adapters on the reading of a and
// b. The sums run on mma.sync: 16 rows fill its tile, and 2 r (K + N) operations a row are
// far below what it can do.
//
// Rows that are not whole, aligned pieces of 16 bytes (8 of b) are read and written value by
// value, many of them 768 rows to a launch: 2,000 rows of 7,168 x 4,090 take 0.2 ms, where
// 4,096 columns take 38 us.
//
// The first product's sums stay 32 bits: they enter the second product as three bf16 parts,
// 24 bits together. All sums have a fixed order: the same bits in every run.
#include <cuda_bf16.h>

#include <algorithm>

#include "fp8_tma.cuh"
#include "lora.cuh"

namespace moe {
namespace {

constexpr int kThreads = 256;

constexpr int kCluster = 8, kWarps = kThreads / 32;
constexpr int kGroup = 16;      // rows of a cluster
// Rows of a call up to which this kernel takes less time than the one for many rows. At 7,168 to
// 4,096 wide (no other width was measured): 512 rows of 4 adapters of rank 32 and 64 14.5 and 18.5
// us (there 20.0 and 23.6); 900 rows of 8 of rank 64 37.5 (24.8); 1,024 rows of 4, 32 and 48 of rank
// 64 37.8 (25.6), 52.5 (38.9) and 55.7 (56.7); 512 rows of 4 of rank 128 58.6 (29.6).
constexpr int kFewRows = 768, kFewRowsWide = 384;
int few_rows(int r) { return r <= 64 ? kFewRows : kFewRowsWide; }
constexpr int kMaxAdapters = 1023;

__device__ __forceinline__ void mma_bf16(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0,
                                         uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, {%0, %1, %2, %3};"
      : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}
__device__ __forceinline__ void st_cluster_v4(uint32_t addr, float4 v) {
  asm volatile("st.shared::cluster.v4.f32 [%0], {%1, %2, %3, %4};" ::"r"(addr), "f"(v.x), "f"(v.y), "f"(v.z), "f"(v.w) : "memory");
}

// Eight (four) consecutive bf16 values of which `left` are in the row (a whole piece of them, or
// none, where rows are whole pieces), zeros behind them.
template <bool kWhole>
__device__ __forceinline__ uint4 bf16x8(const uint16_t* p, int left) {
  if constexpr (kWhole) {
    return left > 0 ? *reinterpret_cast<const uint4*>(p) : make_uint4(0, 0, 0, 0);
  } else {
    uint32_t w[4];
#pragma unroll
    for (int i = 0; i < 4; ++i)
      w[i] = (2 * i < left ? p[2 * i] : 0u) | (2 * i + 1 < left ? static_cast<uint32_t>(p[2 * i + 1]) << 16 : 0u);
    return make_uint4(w[0], w[1], w[2], w[3]);
  }
}
template <bool kWhole>
__device__ __forceinline__ uint2 bf16x4(const uint16_t* p, int left) {
  if constexpr (kWhole) {
    return left > 0 ? *reinterpret_cast<const uint2*>(p) : make_uint2(0, 0);
  } else {
    uint32_t w[2];
#pragma unroll
    for (int i = 0; i < 2; ++i)
      w[i] = (2 * i < left ? p[2 * i] : 0u) | (2 * i + 1 < left ? static_cast<uint32_t>(p[2 * i + 1]) << 16 : 0u);
    return make_uint2(w[0], w[1]);
  }
}
// Eight addends, and outputs, of which `left` are in the row.
template <bool kWhole>
__device__ __forceinline__ void load_eight(const LoraArgs& a, long long at, int left, float (&d)[8]) {
  if constexpr (kWhole) {
    load8(a, at, d);
  } else {
#pragma unroll
    for (int i = 0; i < 8; ++i) d[i] = i < left ? addend(a, at + i) : 0.f;
  }
}
template <bool kWhole>
__device__ __forceinline__ void store_eight(const LoraArgs& a, long long at, int left, const float (&d)[8]) {
  if constexpr (kWhole) {
    store8(a, at, d);
  } else {
#pragma unroll
    for (int i = 0; i < 8; ++i)
      if (i < left) put(a, at + i, d[i]);
  }
}

// Shared memory of the few-row kernel for ranks up to 8 * kTiles: the warps' sums, the
// CTAs' sums as they arrive from the cluster, and the parts of the sum, rows padded by 8
// values against bank conflicts.
template <int kTiles>
struct Few {
  static constexpr int kRank = 8 * kTiles;               // a multiple of 16
  static constexpr int kSums = kGroup * kRank;           // fp32
  static constexpr int kRow = kRank + 8;                 // bf16 of a row of parts
  static constexpr int kSmem = (kWarps + kCluster) * kSums * 4 + kParts * kGroup * kRow * 2;
};

// Sums of 16 rows and up to 8 kTiles ranks. The order of the reduction's elements is free
// as long as both operands share it: a lane takes 16 consecutive bytes of a row, of which
// the words 0, 1 make one MMA's elements (2t, 2t + 1, 2t + 8, 2t + 9) and 2, 3 the next's.
// kWhole: rows of whole, aligned pieces.
template <int kTiles, bool kWhole>
__global__ void __launch_bounds__(kThreads, kTiles <= 4 ? 3 : kTiles <= 8 ? 2 : 1) lora_few_kernel(const LoraArgs a) {
  using F = Few<kTiles>;
  extern __shared__ __align__(16) uint8_t smem[];
  float* warp_sums = reinterpret_cast<float*>(smem);                                       // [warps][16][kRank]
  float* arrived = warp_sums + kWarps * F::kSums;                                          // [CTAs][16][kRank]
  uint16_t* part_of = reinterpret_cast<uint16_t*>(arrived + kCluster * F::kSums);          // [kParts][16][kRow]
  __shared__ int index_of[kFewRows];
  __shared__ int count_of[kMaxAdapters + 1];
  __shared__ int row_of[kGroup];
  __shared__ int group[3];  // adapter, rows of it in front of the group, rows
  const int tid = threadIdx.x, lane = tid & 31, w = tid >> 5;
  const int rank = static_cast<int>(cluster_rank());
  const int want = blockIdx.x / kCluster;
  if (a.M <= 32) {
    // one row to a lane: the first of an adapter's rows, and every 16th on, begins a group
    pdl_wait();
    if (w == 0) {
      const int i = lane < a.M ? a.index[lane] : 0;
      const int mine = lane >= a.M ? -1 : static_cast<uint32_t>(i) < static_cast<uint32_t>(a.L) ? i : a.L;
      const unsigned peers = __match_any_sync(0xffffffffu, mine), below = (1u << lane) - 1u;
      const int before = __popc(peers & below);
      const unsigned first = __ballot_sync(0xffffffffu, mine >= 0 && before % kGroup == 0);
      const int from = __ffs(__ballot_sync(0xffffffffu, (first >> lane & 1) && __popc(first & below) == want)) - 1;
      if (from < 0) {
        if (lane == 0) group[2] = 0;
      } else {
        const int skip = __shfl_sync(0xffffffffu, before, from);
        const bool in = peers >> from & 1 && before >= skip && before < skip + kGroup;
        if (in) row_of[before - skip] = lane;
        const unsigned all = __ballot_sync(0xffffffffu, in);
        if (lane == from) group[0] = mine, group[2] = __popc(all);
      }
    }
    __syncthreads();
  } else {
    for (int i = tid; i <= a.L; i += kThreads) count_of[i] = 0;
    if (tid < 3) group[tid] = 0;
    __syncthreads();
    pdl_wait();
    for (int i = tid; i < a.M; i += kThreads) {
      const int l = a.index[i];
      const int b = static_cast<uint32_t>(l) < static_cast<uint32_t>(a.L) ? l : a.L;
      index_of[i] = b;
      atomicAdd(&count_of[b], 1);
    }
    __syncthreads();
    if (w == 0) {
      int before = 0;  // groups of the adapters so far
      for (int b0 = 0; b0 <= a.L && before <= want; b0 += 32) {
        const int n = b0 + lane <= a.L ? count_of[b0 + lane] : 0, groups = (n + kGroup - 1) / kGroup;
        int upto = groups;
  #pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
          const int v = __shfl_up_sync(0xffffffffu, upto, o);
          if (lane >= o) upto += v;
        }
        const int first = before + upto - groups;
        if (first <= want && want < first + groups) {
          group[0] = b0 + lane;
          group[1] = (want - first) * kGroup;
          group[2] = min(kGroup, n - group[1]);
        }
        before += __shfl_sync(0xffffffffu, upto, 31);
      }
      __syncwarp();
      const int l = group[0], skip = group[1], rows = group[2];
      int found = 0;
      for (int i0 = 0; i0 < a.M && found < skip + rows; i0 += 32) {
        const unsigned same = __ballot_sync(0xffffffffu, i0 + lane < a.M && index_of[i0 + lane] == l);
        const int at = found + __popc(same & ((1u << lane) - 1u)) - skip;
        if ((same >> lane & 1) && at >= 0 && at < rows) row_of[at] = i0 + lane;
        found += __popc(same);
      }
    }
    __syncthreads();
  }
  const int l = group[0], rows = group[2];
  if (rows == 0) return;  // (the same in the whole cluster, as all that returns here)
  // columns of the output that are this CTA's, in blocks of 32
  const int blocks = (a.N + 31) / 32, per = (blocks + kCluster - 1) / kCluster;
  const int block0 = rank * per, block1 = min(blocks, block0 + per);
  if (l == a.L) {  // rows without an adapter
    if (a.add == a.out) return;
    const int n0 = block0 * 32, pieces = (min(a.N, block1 * 32) - n0 + 7) / 8;
    for (int i = tid; i < rows * pieces; i += kThreads) {
      const int n = n0 + 8 * (i % pieces);
      const long long at = static_cast<long long>(row_of[i / pieces]) * a.N + n;
      float d[8];
      load_eight<kWhole>(a, at, a.N - n, d);
      store_eight<kWhole>(a, at, a.N - n, d);
    }
    return;
  }
  asm volatile("barrier.cluster.arrive.relaxed.aligned;" ::: "memory");  // (every CTA runs before another writes to it)

  const int g = lane >> 2, t = lane & 3;
  const uint16_t* A = a.a + static_cast<long long>(l) * a.r * a.K;
  const uint16_t* B = a.b + static_cast<long long>(l) * a.N * a.r;
  // ---- a[l] x: this CTA's part of the K columns in units of 32, dealt out to its warps
  float sum[kTiles][4] = {};
  {
    const int units = (a.K + 31) / 32, each = (units + kCluster - 1) / kCluster;
    const int u0 = rank * each, u1 = min(units, u0 + each);
    // what comes after the exchange is asked into L2: lines of b, lines of the addends
    {
      const int n0 = block0 * 32, n1 = min(a.N, block1 * 32);
      const char* from = reinterpret_cast<const char*>(B + static_cast<long long>(n0) * a.r);
      for (int i = tid * 128; i < (n1 - n0) * a.r * 2; i += kThreads * 128) prefetch_l2(from + i);
      if (a.add && n1 > n0) {
        const int item = a.add_type == kTypeF32 ? 4 : 2, lines = ((n1 - n0) * item + 127) / 128;
        for (int m = w; m < rows; m += kWarps)
          for (int i = lane; i < lines; i += 32)
            prefetch_l2(static_cast<const char*>(a.add) + (static_cast<long long>(row_of[m]) * a.N + n0) * item + i * 128);
      }
    }
    const uint16_t* x0 = a.x + static_cast<long long>(row_of[min(g, rows - 1)]) * a.ldx + 8 * t;
    const uint16_t* x1 = a.x + static_cast<long long>(row_of[min(g + 8, rows - 1)]) * a.ldx + 8 * t;
    constexpr int kOnce = !kWhole ? 1 : kTiles <= 2 ? 4 : kTiles <= 4 ? 2 : 1;  // units under way (more of them would cost a CTA)
    for (int u = u0 + w; u < u1; u += kOnce * kWarps) {
      uint4 xa[kOnce], xb[kOnce], y[kOnce][kTiles];
#pragma unroll
      for (int i = 0; i < kOnce; ++i) {
        const int k = (u + i * kWarps) * 32;
        const int left = u + i * kWarps < u1 ? a.K - k - 8 * t : 0;
        xa[i] = bf16x8<kWhole>(x0 + k, g < rows ? left : 0);
        xb[i] = bf16x8<kWhole>(x1 + k, g + 8 < rows ? left : 0);
#pragma unroll
        for (int j = 0; j < kTiles; ++j)
          y[i][j] = bf16x8<kWhole>(A + static_cast<long long>(8 * j + g) * a.K + k + 8 * t, 8 * j + g < a.r ? left : 0);
      }
#pragma unroll
      for (int i = 0; i < kOnce; ++i)
#pragma unroll
        for (int j = 0; j < kTiles; ++j) {
          mma_bf16(sum[j], xa[i].x, xb[i].x, xa[i].y, xb[i].y, y[i][j].x, y[i][j].y);
          mma_bf16(sum[j], xa[i].z, xb[i].z, xa[i].w, xb[i].w, y[i][j].z, y[i][j].w);
        }
    }
  }
  {
    float* mine = warp_sums + w * F::kSums;
#pragma unroll
    for (int j = 0; j < kTiles; ++j) {
      *reinterpret_cast<float2*>(mine + g * F::kRank + 8 * j + 2 * t) = make_float2(sum[j][0], sum[j][1]);
      *reinterpret_cast<float2*>(mine + (g + 8) * F::kRank + 8 * j + 2 * t) = make_float2(sum[j][2], sum[j][3]);
    }
  }
  __syncthreads();
  asm volatile("barrier.cluster.wait.aligned;" ::: "memory");
  for (int i = tid; i < rows * F::kRank / 4; i += kThreads) {
    float4 s = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
    for (int v = 0; v < kWarps; ++v) {
      const float4 p = reinterpret_cast<const float4*>(warp_sums + v * F::kSums)[i];
      s.x += p.x, s.y += p.y, s.z += p.z, s.w += p.w;
    }
    const uint32_t at = smem_u32(arrived + rank * F::kSums) + 16 * i;
#pragma unroll
    for (int c = 0; c < kCluster; ++c) st_cluster_v4(map_rank(at, c), s);
  }
  cluster_sync();  // (the only one: afterwards a CTA reads its own shared memory alone)
  const float scale = a.scale ? a.scale[l] : 1.f;
  for (int i = tid; i < rows * F::kRank; i += kThreads) {
    float s = 0.f;
#pragma unroll
    for (int c = 0; c < kCluster; ++c) s += arrived[c * F::kSums + i];
    s = i % F::kRank < a.r ? s * scale : 0.f;  // (an infinite x times the zeros behind r)
    const int at = i / F::kRank * F::kRow + i % F::kRank;
#pragma unroll
    for (int p = 0; p < kParts; ++p) {
      const uint16_t h = bf16_part(s);
      part_of[p * kGroup * F::kRow + at] = h;
      s = isfinite(s) ? s - bf16_value(h) : 0.f;
    }
  }
  __syncthreads();
  // ---- b[l] of that: 16 rows x 32 columns at a time, a lane's outputs 8 consecutive columns
  for (int bl = block0 + w; bl < block1; bl += kWarps) {
    const int n0 = bl * 32, n = n0 + 8 * t;
    const bool live = n < a.N;
    float d0[8], d1[8];  // addends of rows g and g + 8
    const long long at0 = static_cast<long long>(row_of[min(g, rows - 1)]) * a.N + n;
    const long long at1 = static_cast<long long>(row_of[min(g + 8, rows - 1)]) * a.N + n;
    load_eight<kWhole>(a, live ? at0 : 0, live ? a.N - n : 0, d0);
    load_eight<kWhole>(a, live ? at1 : 0, live ? a.N - n : 0, d1);
    float acc[4][4] = {};
    uint2 y[4][kTiles / 2];
#pragma unroll
    for (int s = 0; s < kTiles / 2; ++s)
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const int row = n0 + 8 * (g >> 1) + 2 * j + (g & 1), i = 16 * s + 4 * t;
        y[j][s] = bf16x4<kWhole>(B + static_cast<long long>(row) * a.r + i, row < a.N ? a.r - i : 0);
      }
#pragma unroll
    for (int p = kParts - 1; p >= 0; --p) {  // (the small parts first)
      const uint16_t* v = part_of + p * kGroup * F::kRow;
#pragma unroll
      for (int s = 0; s < kTiles / 2; ++s) {
        const uint2 v0 = *reinterpret_cast<const uint2*>(v + g * F::kRow + 16 * s + 4 * t);
        const uint2 v1 = *reinterpret_cast<const uint2*>(v + (g + 8) * F::kRow + 16 * s + 4 * t);
#pragma unroll
        for (int j = 0; j < 4; ++j) mma_bf16(acc[j], v0.x, v1.x, v0.y, v1.y, y[j][s].x, y[j][s].y);
      }
    }
    if (!live) continue;
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      d0[2 * j] += acc[j][0], d0[2 * j + 1] += acc[j][1];
      d1[2 * j] += acc[j][2], d1[2 * j + 1] += acc[j][3];
    }
    if (g < rows) store_eight<kWhole>(a, at0, a.N - n, d0);
    if (g + 8 < rows) store_eight<kWhole>(a, at1, a.N - n, d1);
  }
}

template <int kTiles, bool kWhole>
cudaError_t launch_few(const LoraArgs& a, cudaStream_t stream) {
  static PerDevice<int> ready;
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  std::atomic<int>* entry = ready.of(dev);
  if (!entry || !entry->load()) {
    e = cudaFuncSetAttribute(lora_few_kernel<kTiles, kWhole>, cudaFuncAttributeMaxDynamicSharedMemorySize, Few<kTiles>::kSmem);
    if (e != cudaSuccess) return e;
    if (entry) entry->store(1);
  }
  const int groups = std::min(a.M, a.L + 1 + (a.M + kGroup - 1) / kGroup);
  return launch_cluster(lora_few_kernel<kTiles, kWhole>, dim3(static_cast<unsigned>(groups) * kCluster), dim3(kThreads),
                        Few<kTiles>::kSmem, stream, kCluster, a);
}

template <bool kWhole>
cudaError_t launch_rank(const LoraArgs& a, cudaStream_t stream) {
  if (a.r <= 16) return launch_few<2, kWhole>(a, stream);
  if (a.r <= 32) return launch_few<4, kWhole>(a, stream);
  if (a.r <= 64) return launch_few<8, kWhole>(a, stream);
  return launch_few<16, kWhole>(a, stream);
}

bool aligned(const void* p, uintptr_t to) { return reinterpret_cast<uintptr_t>(p) % to == 0; }

}  // namespace

namespace {
// 16-byte pieces of every row.
bool in_pieces(const LoraArgs& a) {
  return a.K % 8 == 0 && a.N % 8 == 0 && (a.M == 1 || a.ldx % 8 == 0) && aligned(a.x, 16) && aligned(a.a, 16) && aligned(a.b, 16) &&
         aligned(a.add, 16) && aligned(a.out, 16);
}
// Whether the kernel for many rows takes the call.
bool takes_many(const LoraArgs& a) { return a.M > few_rows(a.r) && in_pieces(a) && a.r % 8 == 0; }
}  // namespace

size_t lora_workspace_bytes(const LoraArgs& a) { return takes_many(a) ? lora_many_workspace(a.M, a.L) : 0; }

cudaError_t launch_lora(const LoraArgs& args, int num_sms, cudaStream_t stream) {
  LoraArgs a = args;
  if (takes_many(a)) return launch_lora_many(a, num_sms, stream);
  const int most = few_rows(a.r);
  const bool whole = in_pieces(a) && a.r % 4 == 0;  // (8 bytes of b's rows will do)
  const long long add_row = a.add_type == kTypeF32 ? 4LL * a.N : 2LL * a.N, out_row = a.out_type == kTypeF32 ? 4LL * a.N : 2LL * a.N;
  for (int m0 = 0; m0 < args.M; m0 += most) {
    a.M = std::min(most, args.M - m0);
    a.x = args.x + m0 * args.ldx;
    a.index = args.index + m0;
    if (args.add) a.add = static_cast<const char*>(args.add) + m0 * add_row;
    a.out = static_cast<char*>(args.out) + m0 * out_row;
    const cudaError_t e = whole ? launch_rank<true>(a, stream) : launch_rank<false>(a, stream);
    if (e != cudaSuccess) return e;
  }
  return cudaSuccess;
}

}  // namespace moe
