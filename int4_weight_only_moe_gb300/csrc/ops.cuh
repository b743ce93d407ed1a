// Launchers of the operators around the routed experts: the scored router, the 8-bit
// block quantisers and the 8-bit block-scaled product (each in its own translation
// unit; argument checks are in ops_api.cu).
#pragma once
#include <atomic>
#include <cstdint>
#include <cuda_runtime.h>

#include "kernels.cuh"

namespace moe {

// Element types of the operators' floating inputs and outputs (as in the header).
constexpr int kTypeF32 = 0;
constexpr int kTypeBf16 = 1;

constexpr int kScaleBlock = 128;  // values that share a scale along the reduction axis
constexpr int kMaxGroups = 32;

// Records `msg` as this thread's last error and returns `code` (api.cu).
int report_error(int code, const char* msg);

// What is asked once for each device, by any thread (kernel attributes, occupancy and
// symbols' addresses hold for one device): the entry of device `dev`, null for a device
// beyond the table, which is asked every time. A zero is not known yet.
constexpr int kMaxDevices = 64;
template <typename T>
struct PerDevice {
  std::atomic<T> entry[kMaxDevices];
  std::atomic<T>* of(int dev) { return dev >= 0 && dev < kMaxDevices ? &entry[dev] : nullptr; }
};

struct RouteScoredArgs {
  const void* logits;  // [M, E], rows row_stride elements apart
  int logits_type;
  long long row_stride;
  int M, E, topk;
  int softmax;         // 1: softmax over E, 0: sigmoid
  const float* bias;   // [E] added for the selection only, or null
  int n_group, topk_group, group_top;
  int renormalize;
  float scale;
  int32_t* ids;        // [M, topk]
  float* weights;      // [M, topk]
};
cudaError_t launch_route_scored(const RouteScoredArgs& a, cudaStream_t stream);

// Block quantiser: x [M, N] (or, for the SwiGLU form, rows [g | u] of 2N) -> q e4m3
// [M, N], s fp32 [M, ceil(N / 128)].
struct QuantArgs {
  const void* x;
  int x_type;
  long long row_stride;
  int M, N;
  uint8_t* q;
  float* s;
};
cudaError_t launch_quantize(const QuantArgs& a, bool swiglu, cudaStream_t stream);
// The same over blocks of 128 rows x 128 columns: s [ceil(M / 128), ceil(N / 128)].
cudaError_t launch_quantize_weight(const QuantArgs& a, cudaStream_t stream);

// out[m, n] = sum_k a[m, k] a_s[m, k/128] b[n, k] b_s[n/128, k/128] (+ add[m, n])
struct Fp8MatmulArgs {
  const uint8_t* a;
  long long lda;
  const float* a_s;
  const uint8_t* b;
  long long ldb;
  const float* b_s;
  const uint16_t* add;  // bf16 [M, N] or null
  void* out;            // [M, N]
  int out_type;
  int M, N, K;
  bool weights_ready;   // `b` and `b_s` were written before the kernel in front of this one began
  float* out_s;         // SwiGLU form: scales [M, N / 128] of `out`, which is e4m3 [M, N]
  uint32_t wait_kcycles;  // longest pipeline wait in units of 1,024 cycles, and the test hook: the
  int test_never_wait;    // sums first wait for what never comes (both set at launch)
};
// The SwiGLU form: `b` has 2 N rows, gate then up (N a multiple of 128), and the output is
// SiLU(gate) * up, quantised.
cudaError_t launch_fp8_swiglu(const Fp8MatmulArgs& a, int num_sms, cudaStream_t stream);
cudaError_t launch_fp8_matmul(const Fp8MatmulArgs& a, int num_sms, cudaStream_t stream);
// What a product takes: batch rows of a tile (16, 32, 64 or 128: the few-row kernel; 256: the
// many-row one; 0: the CUDA cores) and CTAs to a tile.
struct Fp8Plan {
  int rows, split;
};
cudaError_t fp8_plan(const Fp8MatmulArgs& a, bool swiglu, int num_sms, Fp8Plan* plan);

// Settings of the products' pipeline waits (MOE_W4A16_FP8_OPT_*); false: no such option
// or value.
bool fp8_set_option(int option, int value);
// Status word of the products (MOE_W4A16_STATUS_TIMEOUT when a wait gave up); clears it.
cudaError_t fp8_status(int32_t* out, cudaStream_t stream);

}  // namespace moe
