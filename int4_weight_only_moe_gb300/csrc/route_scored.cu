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
// n_group lanes to a group), so that lower lane, then lower slot, is the lower id:
// the tie rule costs nothing. All arithmetic is fp32.
#include <cfloat>

#include "ops.cuh"

namespace moe {
namespace {

constexpr int kRouteThreads = 256;

// Order-preserving map of a float to an unsigned integer; NaN ranks as -infinity.
// 0 is below every value: no candidate.
__device__ __forceinline__ uint32_t order_key(float c) {
  if (c != c) c = -INFINITY;
  const uint32_t u = __float_as_uint(c + 0.0f);  // (-0 counts as 0)
  return (u & 0x80000000u) ? ~u : (u | 0x80000000u);
}

__device__ __forceinline__ float to_f32(float v) { return v; }
__device__ __forceinline__ float to_f32(uint16_t v) { return __uint_as_float(static_cast<uint32_t>(v) << 16); }

// (a NaN logit counts as -infinity; +infinity as the largest number, so that two of
// them share a softmax)
__device__ __forceinline__ float clean_logit(float x) { return x != x ? -INFINITY : fminf(x, FLT_MAX); }

__device__ __forceinline__ float sigmoid(float l) { return 1.0f / (1.0f + expf(-l)); }

__device__ __forceinline__ void load4(const float* p, float (&v)[4]) {
  const float4 t = *reinterpret_cast<const float4*>(p);
  v[0] = t.x, v[1] = t.y, v[2] = t.z, v[3] = t.w;
}
__device__ __forceinline__ void load4(const uint16_t* p, float (&v)[4]) {
  const uint2 t = *reinterpret_cast<const uint2*>(p);
  v[0] = __uint_as_float(t.x << 16), v[1] = __uint_as_float(t.x & 0xFFFF0000u);
  v[2] = __uint_as_float(t.y << 16), v[3] = __uint_as_float(t.y & 0xFFFF0000u);
}

// C: slots of a lane, a multiple of 4 (the run length c <= C). `vec`: rows and runs
// allow loads of four values.
template <int C, typename T>
__global__ void __launch_bounds__(kRouteThreads) route_scored_kernel(RouteScoredArgs a, int P, int c, bool vec) {
  pdl_wait();
  pdl_launch_dependents();
  const int lane = threadIdx.x & 31;
  const int gs = a.E / a.n_group;
  const int g = lane / P, sub = lane % P;
  const int base = sub * c;  // first place in the group
  const int n = g < a.n_group ? min(c, gs - base) : 0;  // (may be negative: no experts)
  const int e0 = g * gs + base;
  const long long nwarps = static_cast<long long>(gridDim.x) * (kRouteThreads / 32);
  for (long long t = static_cast<long long>(blockIdx.x) * (kRouteThreads / 32) + (threadIdx.x >> 5); t < a.M;
       t += nwarps) {
    const T* row = static_cast<const T*>(a.logits) + t * a.row_stride;
    float v[C];
    if (vec) {
#pragma unroll
      for (int i = 0; i < C; i += 4) {
        float q[4] = {-INFINITY, -INFINITY, -INFINITY, -INFINITY};
        if (i < n) load4(row + e0 + i, q);
#pragma unroll
        for (int k = 0; k < 4; ++k) v[i + k] = clean_logit(q[k]);
      }
    } else {
#pragma unroll
      for (int i = 0; i < C; ++i) v[i] = i < n ? clean_logit(to_f32(row[e0 + i])) : -INFINITY;
    }
    // scores
    float top = 0.f, z = 1.f;
    if (a.softmax) {
      top = -INFINITY;
#pragma unroll
      for (int i = 0; i < C; ++i) top = fmaxf(top, v[i]);
#pragma unroll
      for (int off = 16; off > 0; off >>= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, off));
      if (top == -INFINITY) top = 0.f;  // (nothing to choose: every score is 0)
      z = 0.f;
#pragma unroll
      for (int i = 0; i < C; ++i) z += expf(v[i] - top);
#pragma unroll
      for (int off = 16; off > 0; off >>= 1) z += __shfl_xor_sync(0xffffffffu, z, off);
      if (z == 0.f) z = 1.f;
    }
    auto score = [&](float l) { return a.softmax ? expf(l - top) / z : sigmoid(l); };
    // selection keys; the two largest of the lane's run
    uint32_t key[C];
    float t1 = -INFINITY, t2 = -INFINITY;
#pragma unroll
    for (int i = 0; i < C; ++i) {
      float ch = -INFINITY;
      if (i < n && v[i] != -INFINITY) {
        ch = score(v[i]);
        if (a.bias) ch += __ldg(a.bias + e0 + i);
      }
      key[i] = i < n ? order_key(ch) : 0u;
      t2 = fmaxf(t2, fminf(t1, ch));
      t1 = fmaxf(t1, ch);
    }
    if (a.topk_group < a.n_group) {
      for (int off = 1; off < P; off <<= 1) {
        const float o1 = __shfl_xor_sync(0xffffffffu, t1, off), o2 = __shfl_xor_sync(0xffffffffu, t2, off);
        t2 = fmaxf(fminf(t1, o1), fmaxf(t2, o2));
        t1 = fmaxf(t1, o1);
      }
      const uint32_t mine = order_key(a.group_top == 2 && t2 != -INFINITY ? t1 + t2 : t1);
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
    // topk rounds: every lane offers its best, the warp's best wins
    uint32_t best = 0;
    int bi = 0;
#pragma unroll
    for (int i = 0; i < C; ++i)
      if (key[i] > best) best = key[i], bi = i;
    int my_id = 0;
    for (int j = 0; j < a.topk; ++j) {
      const uint32_t win = __reduce_max_sync(0xffffffffu, best);
      const int src = __ffs(__ballot_sync(0xffffffffu, best == win)) - 1;
      const int id = __shfl_sync(0xffffffffu, e0 + bi, src);
      if (lane == j) my_id = id;
      if (lane == src) {
        best = 0;
        const int gone = bi;
#pragma unroll
        for (int i = 0; i < C; ++i) {
          if (i == gone) key[i] = 0u;
          if (key[i] > best) best = key[i], bi = i;
        }
      }
    }
    float w = 0.f;
    if (lane < a.topk) {
      const float l = clean_logit(to_f32(row[my_id]));
      w = l == -INFINITY ? 0.f : score(l);
    }
    if (a.renormalize) {
      float sum = w;
#pragma unroll
      for (int off = 16; off > 0; off >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, off);
      if (sum > 0.f) w /= sum;
    }
    if (lane < a.topk) {
      a.ids[t * a.topk + lane] = my_id;
      a.weights[t * a.topk + lane] = w * a.scale;
    }
  }
}

template <typename T>
cudaError_t launch_typed(const RouteScoredArgs& a, int num_sms, cudaStream_t stream) {
  int groups = 1;
  while (groups < a.n_group) groups *= 2;
  const int P = 32 / groups, gs = a.E / a.n_group;
  const int c = ((gs + P - 1) / P + 3) / 4 * 4;
  const bool vec = gs % 4 == 0 && a.row_stride % 4 == 0 &&
                   reinterpret_cast<uintptr_t>(a.logits) % (4 * sizeof(T)) == 0;
  constexpr int per = kRouteThreads / 32;
  long long grid = (static_cast<long long>(a.M) + per - 1) / per;
  if (grid > 8LL * num_sms) grid = 8LL * num_sms;
  auto go = [&](auto kernel) {
    return launch_k(kernel, dim3(static_cast<unsigned>(grid)), dim3(kRouteThreads), 0, stream, true, a, P, c, vec);
  };
  if (c <= 4) return go(route_scored_kernel<4, T>);
  if (c <= 8) return go(route_scored_kernel<8, T>);
  if (c <= 12) return go(route_scored_kernel<12, T>);
  if (c <= 16) return go(route_scored_kernel<16, T>);
  if (c <= 32) return go(route_scored_kernel<32, T>);
  return go(route_scored_kernel<64, T>);  // (c <= 60: at most 1,024 experts, over half of the lanes in use)
}

}  // namespace

cudaError_t launch_route_scored(const RouteScoredArgs& a, int num_sms, cudaStream_t stream) {
  return a.logits_type == kTypeF32 ? launch_typed<float>(a, num_sms, stream)
                                   : launch_typed<uint16_t>(a, num_sms, stream);
}

}  // namespace moe
