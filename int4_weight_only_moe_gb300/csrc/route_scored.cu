// Scored router: the gate's logits to expert ids and weights for the routed experts.
//
//   s_e = sigmoid(l_e)  or  exp(l_e - max) / sum exp(l - max)
//   c_e = s_e + bias_e                         (selection only)
//   groups of E / n_group consecutive experts: a group counts its largest c, or the
//   sum of its two largest; the topk_group best groups stay
//   ids = the topk largest c that stay, weights = s of those
//         (/ their sum) * scale
//
// Equal values go to the lower group and the lower expert id, so the ids are unique.
// A logit of -infinity or NaN marks an expert that is not to be chosen: its c is
// -infinity, it counts nothing in its group, and where a row has too few others it
// fills the remaining places with weight 0.
//
// One warp per token. Lane l holds a run of consecutive experts of one group (32 /
// n_group lanes to a group), so that lower lane, then lower slot, is the lower id: the
// tie rule costs nothing. The lanes' best, sorted, give a bound that leaves little more
// than topk candidates; those move one to a lane and count the better ones.
// 16,384 tokens of 384 experts, top-8, take 12.3 us with sigmoid and bias (26 MB of logits
// could be read in 3.9), 11.0 without a bias; with topk rounds of a warp-wide maximum
// instead, 16.5. Neither the issue slots (59%) nor memory (20%) are full: what bounds it is
// the latency of a token's loads and of its chain of exchanges, beside which a warp has
// nothing else to do.
//
// Without a bias the logits themselves are ranked, whose order the scores keep (a softmax's
// from 104 below the row's largest on, where fp32 has only 0, count as equal). With one, and
// for the sum of a group's two, the scores come from the hardware's exponential and
// reciprocal, results below 2^-126 kept: a few 2^-22 of the score, and |x| 2^-23 more for an
// exponent x (rounded before the exponential), so that values closer than that may rank
// either way; equal logits stay equal. The weights of the chosen take the full-precision
// exponential and divisions; a softmax divides by the sum of the short ones, whose errors
// count by their terms' share (x exp(-x) 2^-23: below 2^-22 in all). All arithmetic is fp32.
#include <cfloat>

#include "ops.cuh"

namespace moe {
namespace {

constexpr int kRouteThreads = 128;

// Order-preserving map of a float to an unsigned integer, and back; NaN ranks as
// -infinity. 0 is below every value: no candidate. (A choice is never -0: what is ranked
// had a bias or +0 added.)
__device__ __forceinline__ uint32_t order_key(float c) {
  const uint32_t u = __float_as_uint(fmaxf(c, -INFINITY));
  return u ^ (static_cast<uint32_t>(static_cast<int32_t>(u) >> 31) | 0x80000000u);
}
__device__ __forceinline__ float key_value(uint32_t k) {
  return k == 0 ? -INFINITY : __uint_as_float(k & 0x80000000u ? k ^ 0x80000000u : ~k);
}

__device__ __forceinline__ float to_f32(float v) { return v; }
__device__ __forceinline__ float to_f32(uint16_t v) { return __uint_as_float(static_cast<uint32_t>(v) << 16); }

// (a NaN logit counts as -infinity; +infinity as the largest number, so that two of
// them share a softmax)
__device__ __forceinline__ float clean_logit(float x) { return fminf(fmaxf(x, -INFINITY), FLT_MAX); }

__device__ __forceinline__ float exp2_fast(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}
__device__ __forceinline__ float rcp_fast(float x) {
  float y;
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}
constexpr float kLog2e = 1.44269504f;

// The selection's score of a logit v plus b (`top`: the row's largest, `rz` 1 / the softmax's
// sum), results below 2^-126 kept: the softmax's exponential as a square, the sigmoid as
// 16 / (1 + exp(-v)) / 16, which is a normal number wherever exp(-v) is finite.
template <bool kSoftmax>
__device__ __forceinline__ float score_plus(float v, float top, float rz, float b) {
  if (kSoftmax) {
    const float root = exp2_fast((v - top) * (0.5f * kLog2e));
    return fmaf(root * root, rz, b);
  }
  return fmaf(rcp_fast(fmaf(exp2_fast(-v * kLog2e), 0.0625f, 0.0625f)), 0.0625f, b);
}
constexpr float kSoftmaxReach = 104.f;  // exp(-104) is 0 in fp32

__device__ __forceinline__ void load4(const float* p, float (&v)[4]) {
  const float4 t = *reinterpret_cast<const float4*>(p);
  v[0] = t.x, v[1] = t.y, v[2] = t.z, v[3] = t.w;
}
__device__ __forceinline__ void load4(const uint16_t* p, float (&v)[4]) {
  const uint2 t = *reinterpret_cast<const uint2*>(p);
  v[0] = __uint_as_float(t.x << 16), v[1] = __uint_as_float(t.x & 0xFFFF0000u);
  v[2] = __uint_as_float(t.y << 16), v[3] = __uint_as_float(t.y & 0xFFFF0000u);
}

// The two best of a run of slots, and which they are: the first of equal ones counts as
// better. (Below: the later slots' pair joined to the earlier ones'.)
struct Best2 {
  uint32_t k1, k2;
  int i1, i2;
};
__device__ __forceinline__ Best2 best2(uint32_t a, uint32_t b, int i) {
  return b > a ? Best2{b, a, i + 1, i} : Best2{a, b, i, i + 1};
}
__device__ __forceinline__ Best2 join(const Best2& a, const Best2& b) {
  const bool later = b.k1 > a.k1;
  // the second: the loser of the firsts, or the winner's own second
  const uint32_t lk = later ? a.k1 : b.k1, sk = later ? b.k2 : a.k2;
  const int li = later ? a.i1 : b.i1, si = later ? b.i2 : a.i2;
  const bool loser = later ? lk >= sk : lk > sk;  // (equal ones: the earlier slot)
  return Best2{later ? b.k1 : a.k1, loser ? lk : sk, later ? b.i1 : a.i1, loser ? li : si};
}
template <int C, typename F>
__device__ __forceinline__ Best2 run_best2(F key) {
  Best2 b = best2(key(0), key(1), 0);
#pragma unroll
  for (int i = 2; i < C; i += 2) b = join(b, best2(key(i), key(i + 1), i));
  return b;
}

// C: slots of a lane, a multiple of 4 (the run length c <= C). `vec`: rows, runs and the
// bias allow loads of four values.
// (The warps an SM holds hide the selection's chain of exchanges: 64 of them for runs of up
// to 8 -- 4,097 x 160 takes 4.9 us, 6.8 with the registers left free -- 48 and 40 up to 16.)
template <int C, bool kSoftmax, bool kBias, typename T>
__global__ void __launch_bounds__(kRouteThreads, C <= 8 ? 16 : C <= 12 ? 12 : C <= 16 ? 10 : 1) route_scored_kernel(RouteScoredArgs a, int P, int c, bool vec) {
  pdl_wait();
  pdl_launch_dependents();
  const int lane = threadIdx.x & 31;
  const long long t = static_cast<long long>(blockIdx.x) * (kRouteThreads / 32) + (threadIdx.x >> 5);
  if (t >= a.M) return;
  const int gs = a.E / a.n_group;
  const int g = lane / P, base = lane % P * c;          // the run's group and first place in it
  const int n = g < a.n_group ? min(c, gs - base) : 0;  // (may be negative: no experts)
  const int e0 = g * gs + base;
  const T* row = static_cast<const T*>(a.logits) + t * a.row_stride;
  float v[C], bias[kBias ? C : 1];
  if (vec) {
#pragma unroll
    for (int i = 0; i < C; i += 4) {
      float q[4] = {-INFINITY, -INFINITY, -INFINITY, -INFINITY}, b[4] = {0.f, 0.f, 0.f, 0.f};
      if (i < n) {
        if (kBias) load4(a.bias + e0 + i, b);
        load4(row + e0 + i, q);
      }
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        v[i + k] = clean_logit(q[k]);
        if (kBias) bias[i + k] = b[k];
      }
    }
  } else {
#pragma unroll
    for (int i = 0; i < C; ++i) {
      v[i] = i < n ? clean_logit(to_f32(row[e0 + i])) : -INFINITY;
      if (kBias) bias[i] = i < n ? a.bias[e0 + i] : 0.f;
    }
  }
  float top = 0.f, z = 1.f, rz = 1.f;
  if (kSoftmax) {
    top = -INFINITY;
#pragma unroll
    for (int i = 0; i < C; ++i) top = fmaxf(top, v[i]);
#pragma unroll
    for (int off = 16; off > 0; off >>= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, off));
    if (top == -INFINITY) top = 0.f;  // (nothing to choose: every score is 0)
    z = 0.f;
#pragma unroll
    for (int i = 0; i < C; ++i) z += exp2_fast((v[i] - top) * kLog2e);
#pragma unroll
    for (int off = 16; off > 0; off >>= 1) z += __shfl_xor_sync(0xffffffffu, z, off);
    if (z == 0.f) z = 1.f;
    rz = rcp_fast(z);
  }
  // selection keys; the run's two best
  uint32_t key[C];
#pragma unroll
  for (int i = 0; i < C; ++i) {
    float choice;
    if constexpr (kBias) {
      choice = v[i] == -INFINITY ? -INFINITY : score_plus<kSoftmax>(v[i], top, rz, bias[i]);
    } else {
      const bool none = kSoftmax && v[i] < top - kSoftmaxReach && v[i] != -INFINITY;
      choice = (none ? -FLT_MAX : v[i]) + 0.f;
    }
    key[i] = order_key(choice);
  }
  if (n < C) {
#pragma unroll
    for (int i = 0; i < C; ++i)
      if (i >= n) key[i] = 0u;
  }
  if (a.topk_group < a.n_group) {
    const Best2 best = run_best2<C>([&](int i) { return key[i]; });
    float t1 = key_value(best.k1), t2 = key_value(best.k2);
    for (int off = 1; off < P; off <<= 1) {
      const float o1 = __shfl_xor_sync(0xffffffffu, t1, off), o2 = __shfl_xor_sync(0xffffffffu, t2, off);
      t2 = fmaxf(fminf(t1, o1), fmaxf(t2, o2));
      t1 = fmaxf(t1, o1);
    }
    if (kBias)
      t1 = a.group_top == 2 && t2 != -INFINITY ? t1 + t2 : t1;
    else if (a.group_top == 2 && t1 != -INFINITY)
      t1 = score_plus<kSoftmax>(t1, top, rz, t2 == -INFINITY ? 0.f : score_plus<kSoftmax>(t2, top, rz, 0.f));
    const uint32_t mine = order_key(t1);
    int ahead = 0;
    for (int j = 0; j < a.n_group; ++j) {
      const uint32_t other = __shfl_sync(0xffffffffu, mine, j * P);
      ahead += other > mine || (other == mine && j < g);
    }
    if (ahead >= a.topk_group) {
#pragma unroll
      for (int i = 0; i < C; ++i) key[i] = 0u;
    }
  }
  // The topk-th largest of the lanes' best bounds the topk-th largest of all from below:
  // what reaches it are the candidates, as a rule little more than topk.
  uint32_t bound = key[0];
#pragma unroll
  for (int i = 1; i < C; ++i) bound = max(bound, key[i]);
#pragma unroll
  for (int size = 2; size <= 32; size *= 2) {  // the lanes' best in descending order
#pragma unroll
    for (int off = size / 2; off > 0; off /= 2) {
      const uint32_t o = __shfl_xor_sync(0xffffffffu, bound, off);
      const bool larger = ((lane & size) == 0) == ((lane & off) == 0);
      bound = larger ? max(bound, o) : min(bound, o);
    }
  }
  bound = max(__shfl_sync(0xffffffffu, bound, a.topk - 1), 1u);
  int mine = 0;
#pragma unroll
  for (int i = 0; i < C; ++i) mine += key[i] >= bound;
  int after = mine;  // candidates up to this lane
#pragma unroll
  for (int off = 1; off < 32; off *= 2) {
    const int o = __shfl_up_sync(0xffffffffu, after, off);
    if (lane >= off) after += o;
  }
  const int total = __shfl_sync(0xffffffffu, after, 31);
  int my_id = 0, rank = a.topk;
  if (total <= 32) {
    // one to a lane, in the order of their ids; its rank is the number of better ones
    __shared__ uint32_t found[kRouteThreads / 32][2][32];
    auto& f = found[threadIdx.x >> 5];
    int at = after - mine;
#pragma unroll
    for (int i = 0; i < C; ++i)
      if (key[i] >= bound) {
        f[0][at] = key[i];
        f[1][at] = e0 + i;
        ++at;
      }
    __syncwarp();
    if (lane < total) {
      const uint32_t k = f[0][lane];
      my_id = f[1][lane];
      rank = 0;
      for (int q = 0; q < total; ++q) {
        const uint32_t o = f[0][q];
        rank += o > k || (o == k && q < lane);
      }
    }
  } else {
    // many equal values, or few lanes with experts: topk rounds in which every lane offers
    // its best and the warp's best wins
    Best2 best = run_best2<C>([&](int i) { return key[i]; });
    for (int j = 0; j < a.topk; ++j) {
      const uint32_t win = __reduce_max_sync(0xffffffffu, best.k1);
      const int src = __ffs(__ballot_sync(0xffffffffu, best.k1 == win)) - 1;
      const int id = __shfl_sync(0xffffffffu, e0 + best.i1, src);
      if (lane == j) my_id = id, rank = j;
      if (lane == src) {
        const uint32_t last = best.k1;
        const int at = best.i1;
        best.k1 = best.k2, best.i1 = best.i2;
        best.k2 = 0u;
        // both are gone: the two best of what ranks behind the one just taken
        if (best.k1 == 0u)
          best = run_best2<C>([&](int i) { return key[i] < last || (key[i] == last && i > at) ? key[i] : 0u; });
      }
    }
  }
  float w = 0.f;
  if (rank < a.topk) {
    const float l = clean_logit(to_f32(row[my_id]));
    if (l != -INFINITY) w = kSoftmax ? expf(l - top) / z : 1.0f / (1.0f + expf(-l));
  }
  if (a.renormalize) {
    float sum = w;
#pragma unroll
    for (int off = 16; off > 0; off >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, off);
    if (sum > 0.f) w /= sum;
  }
  if (rank < a.topk) {
    a.ids[t * a.topk + rank] = my_id;
    a.weights[t * a.topk + rank] = w * a.scale;
  }
}

template <bool kSoftmax, bool kBias, typename T>
cudaError_t launch_typed(const RouteScoredArgs& a, cudaStream_t stream) {
  int groups = 1;
  while (groups < a.n_group) groups *= 2;
  const int P = 32 / groups, gs = a.E / a.n_group;
  const int c = ((gs + P - 1) / P + 3) / 4 * 4;
  const bool vec = gs % 4 == 0 && a.row_stride % 4 == 0 &&
                   reinterpret_cast<uintptr_t>(a.logits) % (4 * sizeof(T)) == 0 &&
                   reinterpret_cast<uintptr_t>(a.bias) % 16 == 0;
  constexpr int per = kRouteThreads / 32;
  const dim3 grid((static_cast<unsigned>(a.M) + per - 1) / per);
  auto go = [&](auto kernel) { return launch_k(kernel, grid, dim3(kRouteThreads), 0, stream, true, a, P, c, vec); };
  if (c <= 4) return go(route_scored_kernel<4, kSoftmax, kBias, T>);
  if (c <= 8) return go(route_scored_kernel<8, kSoftmax, kBias, T>);
  if (c <= 12) return go(route_scored_kernel<12, kSoftmax, kBias, T>);
  if (c <= 16) return go(route_scored_kernel<16, kSoftmax, kBias, T>);
  if (c <= 32) return go(route_scored_kernel<32, kSoftmax, kBias, T>);
  return go(route_scored_kernel<64, kSoftmax, kBias, T>);  // (c <= 60: at most 1,024 experts, over half of the lanes in use)
}

}  // namespace

cudaError_t launch_route_scored(const RouteScoredArgs& a, cudaStream_t stream) {
  auto go = [&](auto value) {
    using T = decltype(value);
    if (a.softmax) return a.bias ? launch_typed<true, true, T>(a, stream) : launch_typed<true, false, T>(a, stream);
    return a.bias ? launch_typed<false, true, T>(a, stream) : launch_typed<false, false, T>(a, stream);
  };
  return a.logits_type == kTypeF32 ? go(float{}) : go(uint16_t{});
}

}  // namespace moe
