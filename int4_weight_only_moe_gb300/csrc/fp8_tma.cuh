// Device and host pieces of the 8-bit tensor-core products: tensor-map copies, the
// e4m3 MMA with both operands in shared memory, cluster helpers.
#pragma once
#include <cuda.h>

#include <cstdint>

#include "ops.cuh"

namespace moe {

// Two-dimensional tensor-map copy of one box into this CTA's shared memory; `x` is the
// byte column (a multiple of 16), `y` the row. Elements outside the tensor arrive as 0.
__device__ __forceinline__ void tma_load_2d(uint32_t dst, const CUtensorMap* map, int x, int y, uint32_t bar,
                                            uint64_t policy) {
  asm volatile(
      "cp.async.bulk.tensor.2d.shared::cluster.global.mbarrier::complete_tx::bytes.L2::cache_hint "
      "[%0], [%1, {%2, %3}], [%4], %5;" ::"r"(dst),
      "l"(map), "r"(x), "r"(y), "r"(bar), "l"(policy)
      : "memory");
}
__device__ __forceinline__ void tma_prefetch_map(const CUtensorMap* map) {
  asm volatile("prefetch.tensormap [%0];" ::"l"(map) : "memory");
}
__device__ __forceinline__ uint64_t l2_policy_evict_normal() {
  uint64_t p;
  asm volatile("createpolicy.fractional.L2::evict_normal.b64 %0, 1.0;" : "=l"(p));
  return p;
}

// D[tmem] (+)= A[smem] * B[smem]^T, e4m3 operands (K-major), fp32 accumulate; 32
// reduction elements.
__device__ __forceinline__ void tc_mma_e4m3(uint32_t d_tmem, uint64_t a_desc, uint64_t b_desc, uint32_t idesc,
                                            uint32_t accumulate) {
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "setp.ne.b32 p, %4, 0;\n\t"
      "tcgen05.mma.cta_group::1.kind::f8f6f4 [%0], %1, %2, %3, p;\n\t}" ::"r"(d_tmem),
      "l"(a_desc), "l"(b_desc), "r"(idesc), "r"(accumulate)
      : "memory");
}
// Instruction descriptor, kind::f8f6f4: e4m3 A and B (format 0), fp32 D, shape M x N.
__host__ __device__ constexpr uint32_t idesc_e4m3_f32(int M, int N) {
  return (1u << 4) | (static_cast<uint32_t>(N >> 3) << 17) | (static_cast<uint32_t>(M >> 4) << 24);
}

__device__ __forceinline__ uint32_t cluster_rank() {
  uint32_t r;
  asm volatile("mov.u32 %0, %%cluster_ctarank;" : "=r"(r));
  return r;
}
__device__ __forceinline__ void cluster_sync() {
  asm volatile("barrier.cluster.arrive.release.aligned;\n\tbarrier.cluster.wait.acquire.aligned;" ::: "memory");
}
// The address of `saddr` (this CTA's shared memory) in CTA `rank` of the cluster.
__device__ __forceinline__ uint32_t map_rank(uint32_t saddr, uint32_t rank) {
  uint32_t d;
  asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(d) : "r"(saddr), "r"(rank));
  return d;
}
__device__ __forceinline__ float ld_cluster_f32(uint32_t addr) {
  float v;
  asm volatile("ld.shared::cluster.f32 %0, [%1];" : "=f"(v) : "r"(addr) : "memory");
  return v;
}

// Wait, for at most kDrainKCycles * 1024 cycles, for a phase of this CTA's own copies
// or MMAs before it leaves; whatever the outcome, go on.
constexpr uint32_t kDrainKCycles = 781250u;  // 8e8 cycles
__device__ __forceinline__ void mbar_drain(uint32_t bar, uint32_t parity) {
  const long long c0 = clock64();
  while (!mbar_try_wait(bar, parity) && ((clock64() - c0) >> 10) <= static_cast<long long>(kDrainKCycles)) {
  }
}

// Tensor map of row-major bytes [rows, cols], rows `stride` bytes apart, read in boxes
// of 128 columns x box_rows rows laid out as 128-byte swizzled rows. False when the
// driver refuses it.
bool make_byte_map(CUtensorMap* map, const void* base, long long rows, long long cols, long long stride, int box_rows);

}  // namespace moe
