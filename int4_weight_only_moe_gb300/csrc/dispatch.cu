// Tokens sorted by expert and back: the order of the experts' rows, the gather of the
// tokens into it, the weighted sum of the experts' rows for each token, and its gradient.
//
//   slot i = t * topk + j: token t's j-th choice. Rows: by expert, then by slot, an
//   expert's rows filled up to a multiple of `block`.
//   gather             out[position[t, j]] = x[t]
//   combine            out[t] = sum_j w[t, j] y[position[t, j]] (+ add[t])
//   combine backward   dy[position[t, j]] = w[t, j] g[t],  dw[t, j] = <g[t], y[position[t, j]]>
//   (the gather's gradient is the combine with weights of 1)
//
// All of it moves memory and computes next to nothing, so each kernel goes by token: it
// reads a token's row once and its topk rows in the sorted order once. Sums are fp32 in the
// order of j: the same bits in every run (no atomics on values).
#include <cuda_bf16.h>

#include <algorithm>

#include "fp8_tma.cuh"
#include "ops.cuh"

namespace moe {
namespace {

// ------------------------------------------------------------------------------ the order

constexpr int kSortThreads = 1024, kSortWarps = kSortThreads / 32;
constexpr int kMaxBuckets = 1024;  // one to a thread

// Bucket of an expert id: the expert's, one more for all other ids (`rest`), or none.
__device__ __forceinline__ int bucket_of(const SortArgs& a, int id) {
  const uint32_t l = static_cast<uint32_t>(id) - static_cast<uint32_t>(a.begin);
  return l < static_cast<uint32_t>(a.E) ? static_cast<int>(l) : (a.rest ? a.E : -1);
}

// Exclusive prefix sum over the block; *total gets the sum.
__device__ int block_scan(int v, int* warp_sum, int* total) {
  const int lane = threadIdx.x & 31, w = threadIdx.x >> 5, warps = blockDim.x >> 5;
  int x = v;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int y = __shfl_up_sync(0xffffffffu, x, o);
    if (lane >= o) x += y;
  }
  if (lane == 31) warp_sum[w] = x;
  __syncthreads();
  if (w == 0) {
    int s = lane < warps ? warp_sum[lane] : 0;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int y = __shfl_up_sync(0xffffffffu, s, o);
      if (lane >= o) s += y;
    }
    warp_sum[lane] = s;
  }
  __syncthreads();
  const int before = (w > 0 ? warp_sum[w - 1] : 0) + x - v;
  *total = warp_sum[warps - 1];
  __syncthreads();
  return before;
}

__device__ __forceinline__ int ld_shared_rank(const int* p, int rank) {
  uint32_t v;
  asm volatile("ld.shared::cluster.u32 %0, [%1];" : "=r"(v) : "r"(map_rank(smem_u32(p), rank)) : "memory");
  return static_cast<int>(v);
}

// Stable counting sort by one cluster. Each warp owns a run of consecutive slots and
// counts it by itself; prefix sums over the warps, the CTAs of the cluster and the buckets
// give every warp the first row of its own slots of each bucket, and a second pass over the
// run hands the rows out in order. What bounds it is latency: the ids of kSteps steps are
// read at once, and kept for the second pass where that is all of the run (up to 65,536
// slots with eight CTAs, 131,072 with 16). 65,536 slots of 384 experts: 7.7 us.
constexpr int kSteps = 8;
__global__ void __launch_bounds__(kSortThreads, 1) sort_kernel(const SortArgs a, int ctas) {
  extern __shared__ int sm[];
  const int B = a.E + (a.rest ? 1 : 0);
  int* hist = sm;                     // [warps][B]: counts, then slots of the bucket already placed by this CTA
  int* mine = hist + kSortWarps * B;  // [B]: this CTA's counts, read by the whole cluster
  int* base = mine + B;               // [B]: row of this CTA's first slot
  int* ends = base + B;               // [B]: row behind the last slot
  __shared__ int warp_sum[32];
  const int tid = threadIdx.x, lane = tid & 31, w = tid >> 5;
  const int rank = ctas > 1 ? static_cast<int>(cluster_rank()) : 0;
  for (int i = tid; i < kSortWarps * B; i += kSortThreads) hist[i] = 0;
  __syncthreads();
  pdl_launch_dependents();  // (they wait for this kernel's end, and set up meanwhile)
  pdl_wait();
  const int run = (a.n + kSortWarps * ctas - 1) / (kSortWarps * ctas);
  const long long first = static_cast<long long>(rank * kSortWarps + w) * run;
  const int lo = static_cast<int>(min(first, static_cast<long long>(a.n)));
  const int hi = static_cast<int>(min(first + run, static_cast<long long>(a.n)));
  const int bits = 32 - __clz(B - 1);  // of a bucket
  int bucket[kSteps];
  auto read = [&](int i0) {
    int id[kSteps];
#pragma unroll
    for (int k = 0; k < kSteps; ++k) id[k] = i0 + 32 * k + lane < hi ? a.ids[i0 + 32 * k + lane] : 0;
#pragma unroll
    for (int k = 0; k < kSteps; ++k) bucket[k] = i0 + 32 * k + lane < hi ? bucket_of(a, id[k]) : -1;
  };
  for (int i0 = lo; i0 < hi; i0 += 32 * kSteps) {
    read(i0);
#pragma unroll
    for (int k = 0; k < kSteps; ++k)
      if (bucket[k] >= 0) atomicAdd(&hist[w * B + bucket[k]], 1);
  }
  __syncthreads();
  int own = 0;
  if (tid < B) {
    int c[kSortWarps];
#pragma unroll
    for (int v = 0; v < kSortWarps; ++v) c[v] = hist[v * B + tid];
#pragma unroll
    for (int v = 0; v < kSortWarps; ++v) {
      hist[v * B + tid] = own;
      own += c[v];
    }
    mine[tid] = own;
  }
  int count = own, before = 0;
  if (ctas > 1) {
    cluster_sync();
    count = 0;
    if (tid < B)
#pragma unroll 8
      for (int r = 0; r < ctas; ++r) {
        const int c = ld_shared_rank(mine + tid, r);
        if (r < rank) before += c;
        count += c;
      }
    asm volatile("barrier.cluster.arrive.release.aligned;" ::: "memory");
  }
  int total;
  const int start = block_scan((count + a.block - 1) / a.block * a.block, warp_sum, &total);
  if (tid < B) {
    base[tid] = start + before;
    ends[tid] = start + count;
    if (rank == 0) a.offsets[tid] = start;
  }
  if (rank == 0 && tid == 0) a.offsets[B] = total;
  __syncthreads();
  // rows that fill up, and rows behind the last
  if (a.block > 1)
    for (int b = rank * kSortWarps + w; b < B; b += ctas * kSortWarps) {
      const int e = ends[b], next = (e + a.block - 1) / a.block * a.block;  // (all starts are multiples of `block`)
      for (int r = e + lane; r < next; r += 32) a.slots[r] = -1;
    }
  for (long long r = total + static_cast<long long>(rank) * kSortThreads + tid; r < a.capacity; r += ctas * kSortThreads)
    a.slots[r] = -1;
  for (int i0 = lo; i0 < hi; i0 += 32 * kSteps) {
    if (hi - lo > 32 * kSteps) read(i0);
#pragma unroll
    for (int k = 0; k < kSteps; ++k) {
      const int i = i0 + 32 * k + lane, b = bucket[k];
      if (i0 + 32 * k >= hi) break;
      const unsigned peers = lanes_of(b, bits);
      int row = -1;
      if (b >= 0) row = base[b] + hist[w * B + b] + __popc(peers & ((1u << lane) - 1u));
      __syncwarp();
      if (b >= 0 && lane == __ffs(peers) - 1) hist[w * B + b] += __popc(peers);
      __syncwarp();
      if (i < hi && a.position) a.position[i] = row;
      if (b >= 0) a.slots[row] = i;
    }
  }
  // (no CTA leaves while another may still read its counts)
  if (ctas > 1) asm volatile("barrier.cluster.wait.acquire.aligned;" ::: "memory");
}

// ------------------------------------------------------------------------------- the rows

constexpr int kRowThreads = 256, kRowWarps = kRowThreads / 32;

// 16-, 4-, 2- or 1-byte pieces, whichever the rows' lengths and addresses allow.
template <int kBytes>
struct Piece;
template <>
struct Piece<16> {
  using T = uint4;
};
template <>
struct Piece<4> {
  using T = uint32_t;
};
template <>
struct Piece<2> {
  using T = uint16_t;
};
template <>
struct Piece<1> {
  using T = uint8_t;
};

// Zeros for the rows that fill up the experts', by CTAs behind those of the tokens: each
// takes kFillRows rows at a multiple of that from the end of an expert's. (Consecutive rows by
// one CTA: 352 MB take 55 us; 94 with the rows dealt out to the warps of two CTAs an SM.)
constexpr int kFillRows = 16;
int fill_parts(int block) { return std::min(64, (block - 1 + kFillRows - 1) / kFillRows); }  // CTAs to an expert
template <int kBytes>
__device__ __forceinline__ void zero_filling(const int32_t* offsets, const int32_t* slots, int capacity, uint8_t* out,
                                             long long row_bytes, int cta, int parts) {
  using T = typename Piece<kBytes>::T;
  const int e = cta / parts, begin = max(offsets[e], 0), end = min(offsets[e + 1], capacity);
  const int n = static_cast<int>(row_bytes / kBytes);
  for (int last = end - (cta % parts) * kFillRows; last > begin; last -= parts * kFillRows) {
    const int first = max(begin, last - kFillRows);
    if (slots[last - 1] >= 0) return;  // (the tokens' rows stand in front)
    for (int r = first; r < last; ++r) {
      if (slots[r] >= 0) continue;
      T* to = reinterpret_cast<T*>(out + r * row_bytes);
      for (int v = threadIdx.x; v < n; v += blockDim.x) to[v] = T{};
    }
  }
}

// Token t's row to its places; `parts` CTAs share a row, `fill` those that fill up an expert's.
template <int kBytes>
__global__ void __launch_bounds__(kRowThreads) gather_kernel(const GatherRowsArgs a, int parts, int fill) {
  using T = typename Piece<kBytes>::T;
  const int threads = blockDim.x;
  __shared__ int row_of[kMaxTopk];
  pdl_wait();
  const long long cta = blockIdx.x;
  if (cta >= static_cast<long long>(a.M) * parts) {
    zero_filling<kBytes>(a.offsets, a.slots, a.capacity, static_cast<uint8_t*>(a.out), a.row_bytes,
                         static_cast<int>(cta - static_cast<long long>(a.M) * parts), fill);
    return;
  }
  const int t = static_cast<int>(cta / parts), part = static_cast<int>(cta % parts);
  if (threadIdx.x < a.topk) row_of[threadIdx.x] = a.position[static_cast<long long>(t) * a.topk + threadIdx.x];
  const int n = static_cast<int>(a.row_bytes / kBytes), per = (n + parts - 1) / parts;
  const int lo = part * per, hi = min(n, lo + per);
  const T* from = reinterpret_cast<const T*>(static_cast<const uint8_t*>(a.x) + t * a.stride_bytes);
  uint8_t* out = static_cast<uint8_t*>(a.out);
  constexpr int kOnce = 4;
  __syncthreads();
  for (int v0 = lo + threadIdx.x; v0 < hi; v0 += kOnce * threads) {
    T x[kOnce];
#pragma unroll
    for (int i = 0; i < kOnce; ++i)
      if (v0 + i * threads < hi) x[i] = from[v0 + i * threads];
    for (int j = 0; j < a.topk; ++j) {
      const int r = row_of[j];
      if (static_cast<uint32_t>(r) >= static_cast<uint32_t>(a.capacity)) continue;
      T* to = reinterpret_cast<T*>(out + r * a.row_bytes);
#pragma unroll
      for (int i = 0; i < kOnce; ++i)
        if (v0 + i * threads < hi) to[v0 + i * threads] = x[i];
    }
  }
}

// Order and gather in one launch, for few slots: every CTA counts the slots of all experts
// for itself (up to kFewSlots ids, from L2) and places its own token's. Top-8 of 384 experts,
// 7,168 wide: 4 tokens 2.8 us, two launches 5.6; 128 tokens 6.2 and 8.6; in blocks of 128, where
// most experts' CTAs have nothing to fill up, 4 tokens 20.7 and 25.9, 128 tokens 96 and 109.
constexpr int kFewSlots = 1024;
template <int kBytes>
__global__ void __launch_bounds__(kRowThreads) sort_gather_few_kernel(const SortArgs o, const GatherRowsArgs a, int parts, int fill) {
  using T = typename Piece<kBytes>::T;
  constexpr int kEach = kMaxBuckets / kRowThreads;  // buckets of a thread in the prefix sum
  __shared__ int count[kMaxBuckets], start[kMaxBuckets + 1];
  __shared__ int bucket[kFewSlots];
  __shared__ int row_of[kMaxTopk];
  __shared__ int warp_sum[32];
  const int tid = threadIdx.x, lane = tid & 31, w = tid >> 5;
  for (int b = tid; b < o.E; b += kRowThreads) count[b] = 0;
  __syncthreads();
  pdl_wait();
  const int cta = blockIdx.x, tokens = a.M * parts;
  const int t = cta / parts, part = cta % parts;
  const int n = static_cast<int>(a.row_bytes / kBytes), per = (n + parts - 1) / parts;
  const int lo = part * per, hi = min(n, lo + per);
  const T* from = reinterpret_cast<const T*>(static_cast<const uint8_t*>(a.x) + t * a.stride_bytes);
  constexpr int kOnce = 4;
  T x[kOnce];
  if (cta < tokens)  // (the row is on its way while its places are found)
#pragma unroll
    for (int i = 0; i < kOnce; ++i)
      if (lo + tid + i * kRowThreads < hi) x[i] = from[lo + tid + i * kRowThreads];
  for (int i = tid; i < o.n; i += kRowThreads) {
    const int b = bucket_of(o, o.ids[i]);
    bucket[i] = b;
    if (b >= 0) atomicAdd(&count[b], 1);
  }
  __syncthreads();
  int padded[kEach], sum = 0, total;
#pragma unroll
  for (int k = 0; k < kEach; ++k) {
    const int b = tid * kEach + k;
    padded[k] = b < o.E ? (count[b] + o.block - 1) / o.block * o.block : 0;
    sum += padded[k];
  }
  int at = block_scan(sum, warp_sum, &total);
#pragma unroll
  for (int k = 0; k < kEach; ++k) {
    const int b = tid * kEach + k;
    if (b < o.E) start[b] = at;
    at += padded[k];
  }
  if (tid == 0) start[o.E] = total;
  __syncthreads();
  uint8_t* out = static_cast<uint8_t*>(a.out);
  if (cta >= tokens) {  // rows that fill up an expert's
    const int e = (cta - tokens) / fill, begin = start[e] + count[e], end = start[e + 1];
    for (int r = begin + (cta - tokens) % fill; r < end; r += fill) {
      if (tid == 0) o.slots[r] = -1;
      T* to = reinterpret_cast<T*>(out + r * a.row_bytes);
      for (int v = tid; v < n; v += kRowThreads) to[v] = T{};
    }
    return;
  }
  if (cta == 0) {
    for (int b = tid; b <= o.E; b += kRowThreads) o.offsets[b] = start[b];
    for (int r = total + tid; r < o.capacity; r += kRowThreads) o.slots[r] = -1;
  }
  for (int j = w; j < a.topk; j += kRowWarps) {
    const int i = t * a.topk + j, b = bucket[i];
    int ahead = 0;
    for (int i0 = 0; i0 < i; i0 += 32) ahead += __popc(__ballot_sync(0xffffffffu, i0 + lane < i && bucket[i0 + lane] == b));
    if (lane == 0) {
      const int row = b >= 0 ? start[b] + ahead : -1;
      row_of[j] = row;
      if (part == 0) {
        o.position[i] = row;
        if (row >= 0) o.slots[row] = i;
      }
    }
  }
  __syncthreads();
  for (int v0 = lo + tid; v0 < hi; v0 += kOnce * kRowThreads) {
    if (v0 >= lo + kOnce * kRowThreads)
#pragma unroll
      for (int i = 0; i < kOnce; ++i)
        if (v0 + i * kRowThreads < hi) x[i] = from[v0 + i * kRowThreads];
    for (int j = 0; j < a.topk; ++j) {
      if (row_of[j] < 0) continue;
      T* to = reinterpret_cast<T*>(out + row_of[j] * a.row_bytes);
#pragma unroll
      for (int i = 0; i < kOnce; ++i)
        if (v0 + i * kRowThreads < hi) to[v0 + i * kRowThreads] = x[i];
    }
  }
}

// n consecutive values of a row as they are in memory, as fp32, and back.
template <typename T, int n>
struct Values;
template <>
struct Values<float, 1> {
  float raw;
  __device__ __forceinline__ void load(const void* p) { raw = *static_cast<const float*>(p); }
  __device__ __forceinline__ float operator[](int) const { return raw; }
  static __device__ __forceinline__ void store(void* p, const float (&f)[1]) { *static_cast<float*>(p) = f[0]; }
};
template <>
struct Values<uint16_t, 1> {
  uint16_t raw;
  __device__ __forceinline__ void load(const void* p) { raw = *static_cast<const uint16_t*>(p); }
  __device__ __forceinline__ float operator[](int) const { return __uint_as_float(static_cast<uint32_t>(raw) << 16); }
  static __device__ __forceinline__ void store(void* p, const float (&f)[1]) {
    *static_cast<__nv_bfloat16*>(p) = __float2bfloat16_rn(f[0]);
  }
};
template <>
struct Values<float, 8> {
  float4 raw[2];
  __device__ __forceinline__ void load(const void* p) {
    raw[0] = static_cast<const float4*>(p)[0], raw[1] = static_cast<const float4*>(p)[1];
  }
  __device__ __forceinline__ float operator[](int i) const {
    const float4 v = raw[i >> 2];
    return (i & 3) == 0 ? v.x : (i & 3) == 1 ? v.y : (i & 3) == 2 ? v.z : v.w;
  }
  static __device__ __forceinline__ void store(void* p, const float (&f)[8]) {
    static_cast<float4*>(p)[0] = make_float4(f[0], f[1], f[2], f[3]);
    static_cast<float4*>(p)[1] = make_float4(f[4], f[5], f[6], f[7]);
  }
};
template <>
struct Values<uint16_t, 8> {
  uint4 raw;
  __device__ __forceinline__ void load(const void* p) { raw = *static_cast<const uint4*>(p); }
  __device__ __forceinline__ float operator[](int i) const {
    const uint32_t w = (i >> 1) == 0 ? raw.x : (i >> 1) == 1 ? raw.y : (i >> 1) == 2 ? raw.z : raw.w;
    return __uint_as_float(i & 1 ? w & 0xFFFF0000u : w << 16);
  }
  static __device__ __forceinline__ void store(void* p, const float (&f)[8]) {
    uint32_t w[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const __nv_bfloat162 h = __floats2bfloat162_rn(f[2 * i], f[2 * i + 1]);
      w[i] = *reinterpret_cast<const uint32_t*>(&h);
    }
    *static_cast<uint4*>(p) = make_uint4(w[0], w[1], w[2], w[3]);
  }
};

template <typename T>
__device__ __forceinline__ T* at(void* p, long long row, long long K, int k) {
  return static_cast<T*>(p) + row * K + k;
}
template <typename T>
__device__ __forceinline__ const T* at(const void* p, long long row, long long K, int k) {
  return static_cast<const T*>(p) + row * K + k;
}

// `f` with the choices j0 .. j0 + C - 1 of a token, eight at a time and then what is left: a
// group's loads are all under way at once, none behind a condition. (8,192 tokens of 8
// choices, 7,168 wide: 152 us; 501 with a condition to each load, behind which the
// conversion of its values waited before the next load began.)
template <typename F>
__device__ __forceinline__ void by_groups(int topk, F&& f) {
  int j = 0;
  for (; j + 8 <= topk; j += 8) f(std::integral_constant<int, 8>{}, j);
  switch (topk - j) {
    case 7: f(std::integral_constant<int, 7>{}, j); break;
    case 6: f(std::integral_constant<int, 6>{}, j); break;
    case 5: f(std::integral_constant<int, 5>{}, j); break;
    case 4: f(std::integral_constant<int, 4>{}, j); break;
    case 3: f(std::integral_constant<int, 3>{}, j); break;
    case 2: f(std::integral_constant<int, 2>{}, j); break;
    case 1: f(std::integral_constant<int, 1>{}, j); break;
  }
}

// out[t] = sum_j w y[row of j] (+ add[t]); `parts` CTAs share a row. A choice without a row
// reads row 0 in its place, which counts nothing.
// (128 threads: 8,192 tokens of 1,024 columns take 24.5 us, 30 with 256; few tokens make six
// CTAs to an SM.)
constexpr int kSumThreads = 128;
template <typename Ty, typename To, int n>
__global__ void __launch_bounds__(kSumThreads) combine_kernel(const CombineArgs a, int parts) {
  __shared__ int row_of[kMaxTopk];
  __shared__ float weight_of[kMaxTopk];
  pdl_wait();
  const int t = static_cast<int>(blockIdx.x / parts), part = static_cast<int>(blockIdx.x % parts);
  if (threadIdx.x < a.topk) {
    const long long i = static_cast<long long>(t) * a.topk + threadIdx.x;
    const int r = a.position[i];
    row_of[threadIdx.x] = static_cast<uint32_t>(r) < static_cast<uint32_t>(a.rows) ? r : -1;
    weight_of[threadIdx.x] = a.weights ? a.weights[i] : 1.0f;
  }
  const int pieces = a.K / n, per = (pieces + parts - 1) / parts;
  const int lo = part * per, hi = min(pieces, lo + per);
  __syncthreads();
  for (int v = lo + threadIdx.x; v < hi; v += kSumThreads) {
    float acc[n];
#pragma unroll
    for (int i = 0; i < n; ++i) acc[i] = 0.f;
    by_groups(a.topk, [&](auto count, int j0) {
      constexpr int C = decltype(count)::value;
      Values<Ty, n> y[C];
#pragma unroll
      for (int j = 0; j < C; ++j) y[j].load(at<Ty>(a.y, max(row_of[j0 + j], 0), a.K, v * n));
#pragma unroll
      for (int j = 0; j < C; ++j) {
        const bool has = row_of[j0 + j] >= 0;
        const float w = weight_of[j0 + j];
#pragma unroll
        for (int i = 0; i < n; ++i) acc[i] = has ? fmaf(w, y[j][i], acc[i]) : acc[i];
      }
    });
    if (a.add) {
      Values<To, n> d;
      d.load(at<To>(a.add, t, a.K, v * n));
#pragma unroll
      for (int i = 0; i < n; ++i) acc[i] += d[i];
    }
    Values<To, n>::store(at<To>(a.out, t, a.K, v * n), acc);
  }
}

// One CTA to a token: each thread keeps its own part of the topk sums of products, which
// the CTA joins at the end. Behind the tokens' CTAs those of the rows that fill up.
constexpr int kBackThreads = 128, kBackWarps = kBackThreads / 32;  // (256: 4,000 tokens of 1,024 columns 44 us, 34 now)
template <typename Tg, typename Ty, int n>
__global__ void __launch_bounds__(kBackThreads, 4) combine_backward_kernel(const CombineBackwardArgs a, int fill) {
  __shared__ int row_of[kMaxTopk];
  __shared__ float weight_of[kMaxTopk];
  __shared__ float part_of[kBackWarps][kMaxTopk];
  pdl_wait();
  if (blockIdx.x >= static_cast<unsigned>(a.M)) {
    zero_filling<n * sizeof(Ty) >= 16 ? 16 : n * static_cast<int>(sizeof(Ty))>(
        a.offsets, a.slots, a.capacity, static_cast<uint8_t*>(a.dy), a.K * static_cast<long long>(sizeof(Ty)),
        blockIdx.x - a.M, fill);
    return;
  }
  const int t = blockIdx.x, lane = threadIdx.x & 31, w = threadIdx.x >> 5;
  if (threadIdx.x < a.topk) {
    const long long i = static_cast<long long>(t) * a.topk + threadIdx.x;
    const int r = a.position[i];
    row_of[threadIdx.x] = static_cast<uint32_t>(r) < static_cast<uint32_t>(a.capacity) ? r : -1;
    weight_of[threadIdx.x] = a.weights[i];
  }
  __syncthreads();
  by_groups(a.topk, [&](auto count, int j0) {
    constexpr int C = decltype(count)::value;
    float dot[C] = {};
    for (int v = threadIdx.x; v < a.K / n; v += kBackThreads) {
      Values<Tg, n> g;
      Values<Ty, n> y[C];
      g.load(at<Tg>(a.g, t, a.K, v * n));
#pragma unroll
      for (int j = 0; j < C; ++j) y[j].load(at<Ty>(a.y, max(row_of[j0 + j], 0), a.K, v * n));
#pragma unroll
      for (int j = 0; j < C; ++j) {
        if (row_of[j0 + j] < 0) continue;
        float d[n];
#pragma unroll
        for (int i = 0; i < n; ++i) {
          dot[j] = fmaf(g[i], y[j][i], dot[j]);
          d[i] = weight_of[j0 + j] * g[i];
        }
        Values<Ty, n>::store(at<Ty>(a.dy, row_of[j0 + j], a.K, v * n), d);
      }
    }
#pragma unroll
    for (int j = 0; j < C; ++j) {
#pragma unroll
      for (int o = 16; o > 0; o >>= 1) dot[j] += __shfl_xor_sync(0xffffffffu, dot[j], o);
      if (lane == 0) part_of[w][j0 + j] = dot[j];
    }
  });
  __syncthreads();
  if (threadIdx.x < a.topk) {
    float sum = 0.f;
    for (int i = 0; i < kBackWarps; ++i) sum += part_of[i][threadIdx.x];
    a.dweights[static_cast<long long>(t) * a.topk + threadIdx.x] = sum;
  }
}

bool aligned(const void* p, uintptr_t to) { return reinterpret_cast<uintptr_t>(p) % to == 0; }

// CTAs of `threads` threads to a row of `pieces` pieces: one, unless the tokens alone make fewer
// than `ctas`.
int row_parts(long long M, int pieces, int threads, int ctas) {
  const int most = (pieces + threads - 1) / threads;
  const long long want = (ctas + M - 1) / std::max(1LL, M);
  return static_cast<int>(std::max(1LL, std::min<long long>(most, want)));
}

}  // namespace

cudaError_t launch_sort(const SortArgs& a, cudaStream_t stream) {
  static PerDevice<int> ready;
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  std::atomic<int>* entry = ready.of(dev);
  if (!entry || !entry->load()) {
    e = cudaFuncSetAttribute(sort_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, (kSortWarps + 3) * kMaxBuckets * 4);
    if (e == cudaSuccess) e = cudaFuncSetAttribute(sort_kernel, cudaFuncAttributeNonPortableClusterSizeAllowed, 1);
    if (e != cudaSuccess) return e;
    if (entry) entry->store(1);
  }
  const int B = a.E + (a.rest ? 1 : 0);
  // (2,048 slots 4.5 us with one CTA and with eight; 16,384 14.9 and 5.9; 65,536 9.7 with eight, 7.7 with 16)
  const int ctas = a.n <= 2048 ? 1 : a.n <= 16384 ? 8 : 16;
  return launch_cluster(sort_kernel, dim3(ctas), dim3(kSortThreads), (kSortWarps + 3) * B * sizeof(int), stream, ctas, a, ctas);
}

cudaError_t launch_gather(const GatherRowsArgs& a, int num_sms, cudaStream_t stream) {
  const int fill = fill_parts(a.block);
  auto go = [&](auto bytes) {
    constexpr int n = decltype(bytes)::value;
    // (short rows: 6,000 of 784 bytes, top-4, 11.4 us with 64 threads, 15.2 with 256; long ones the
    // other way: 14,336 bytes, top-8, 170 and 178)
    const int pieces = static_cast<int>(a.row_bytes / n), threads = pieces <= 128 ? 64 : kRowThreads;
    const int parts = row_parts(a.M, pieces, threads, 2 * num_sms);
    return launch_k(gather_kernel<n>, dim3(static_cast<unsigned>(static_cast<long long>(a.M) * parts + a.E * fill)), dim3(threads), 0,
                    stream, true, a, parts, fill);
  };
  const uintptr_t all = static_cast<uintptr_t>(a.row_bytes) | static_cast<uintptr_t>(a.stride_bytes) |
                        reinterpret_cast<uintptr_t>(a.x) | reinterpret_cast<uintptr_t>(a.out);
  if (all % 16 == 0) return go(std::integral_constant<int, 16>{});
  if (all % 4 == 0) return go(std::integral_constant<int, 4>{});
  if (all % 2 == 0) return go(std::integral_constant<int, 2>{});
  return go(std::integral_constant<int, 1>{});
}

cudaError_t launch_sort_gather(const SortArgs& o, const GatherRowsArgs& a, int num_sms, cudaStream_t stream) {
  if (o.n > kFewSlots || o.rest) {
    const cudaError_t e = launch_sort(o, stream);
    return e == cudaSuccess ? launch_gather(a, num_sms, stream) : e;
  }
  const int fill = fill_parts(a.block);
  auto go = [&](auto bytes) {
    constexpr int n = decltype(bytes)::value;
    const int parts = row_parts(a.M, static_cast<int>(a.row_bytes / n), kRowThreads, 2 * num_sms);
    return launch_k(sort_gather_few_kernel<n>, dim3(static_cast<unsigned>(a.M * parts + a.E * fill)), dim3(kRowThreads), 0, stream, true,
                    o, a, parts, fill);
  };
  const uintptr_t all = static_cast<uintptr_t>(a.row_bytes) | static_cast<uintptr_t>(a.stride_bytes) |
                        reinterpret_cast<uintptr_t>(a.x) | reinterpret_cast<uintptr_t>(a.out);
  if (all % 16 == 0) return go(std::integral_constant<int, 16>{});
  if (all % 4 == 0) return go(std::integral_constant<int, 4>{});
  if (all % 2 == 0) return go(std::integral_constant<int, 2>{});
  return go(std::integral_constant<int, 1>{});
}

cudaError_t launch_combine(const CombineArgs& args, int num_sms, cudaStream_t stream) {
  CombineArgs a = args;
  if (a.rows == 0) a.y = a.out, a.y_type = a.out_type;  // (no row counts; what is read in its place is out's)
  const bool wide = a.K % 8 == 0 && aligned(a.y, 16) && aligned(a.add, 16) && aligned(a.out, 16);
  auto go = [&](auto ty, auto to) {
    using Ty = decltype(ty);
    using To = decltype(to);
    auto with = [&](auto kernel, int n) {
      const int parts = row_parts(a.M, a.K / n, kSumThreads, 6 * num_sms);
      return launch_k(kernel, dim3(static_cast<unsigned>(a.M) * parts), dim3(kSumThreads), 0, stream, true, a, parts);
    };
    return wide ? with(combine_kernel<Ty, To, 8>, 8) : with(combine_kernel<Ty, To, 1>, 1);
  };
  if (a.y_type == kTypeF32) return a.out_type == kTypeF32 ? go(float{}, float{}) : go(float{}, uint16_t{});
  return a.out_type == kTypeF32 ? go(uint16_t{}, float{}) : go(uint16_t{}, uint16_t{});
}

cudaError_t launch_combine_backward(const CombineBackwardArgs& a, int num_sms, cudaStream_t stream) {
  const bool wide = a.K % 8 == 0 && aligned(a.y, 16) && aligned(a.g, 16) && aligned(a.dy, 16);
  const int fill = fill_parts(a.block);
  auto go = [&](auto tg, auto ty) {
    using Tg = decltype(tg);
    using Ty = decltype(ty);
    auto with = [&](auto kernel) {
      return launch_k(kernel, dim3(static_cast<unsigned>(a.M) + a.E * fill), dim3(kBackThreads), 0, stream, true, a, fill);
    };
    return wide ? with(combine_backward_kernel<Tg, Ty, 8>) : with(combine_backward_kernel<Tg, Ty, 1>);
  };
  if (a.g_type == kTypeF32) return a.y_type == kTypeF32 ? go(float{}, float{}) : go(float{}, uint16_t{});
  return a.y_type == kTypeF32 ? go(uint16_t{}, float{}) : go(uint16_t{}, uint16_t{});
}

}  // namespace moe
