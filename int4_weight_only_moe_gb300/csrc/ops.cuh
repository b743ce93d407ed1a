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

// The order of experts' rows (dispatch.cu). Buckets: E experts from id `begin` on, and with
// `rest` one more that takes every other id (at most 1,024 in all).
struct SortArgs {
  const int32_t* ids;  // [n]
  int n, begin, E;
  int rest;
  int block;           // rows of a bucket are filled up to a multiple
  int32_t* offsets;    // [buckets + 1]
  int32_t* slots;      // [capacity]
  int capacity;
  int32_t* position;   // [n] or null
};
cudaError_t launch_sort(const SortArgs& a, cudaStream_t stream);

constexpr int kMaxTopk = 32;
// out[position[t, j]] = x[t], zeros in the rows that fill up.
struct GatherRowsArgs {
  const void* x;  // [M] rows stride_bytes apart
  long long stride_bytes, row_bytes;
  const int32_t* offsets;
  const int32_t* slots;
  const int32_t* position;
  void* out;      // [capacity] rows
  int M, topk, E, block, capacity;
};
cudaError_t launch_gather(const GatherRowsArgs& a, int num_sms, cudaStream_t stream);
// Both, in one launch for few slots.
cudaError_t launch_sort_gather(const SortArgs& o, const GatherRowsArgs& a, int num_sms, cudaStream_t stream);

// out[t] = sum_j weights[t, j] y[position[t, j]] (+ add[t])
struct CombineArgs {
  const void* y;  // [rows, K]
  int y_type;
  const float* weights;  // [M, topk], or null: 1
  const int32_t* position;
  const void* add;       // [M, K] of the output's type, or null
  void* out;             // [M, K]
  int out_type;
  int M, K, topk, rows;
};
cudaError_t launch_combine(const CombineArgs& a, int num_sms, cudaStream_t stream);

struct CombineBackwardArgs {
  const void* g;  // [M, K]
  int g_type;
  const void* y;  // [capacity, K], and dy
  int y_type;
  const float* weights;
  const int32_t* offsets;
  const int32_t* slots;
  const int32_t* position;
  void* dy;
  float* dweights;  // [M, topk]
  int M, K, topk, E, block, capacity;
};
cudaError_t launch_combine_backward(const CombineBackwardArgs& a, int num_sms, cudaStream_t stream);

struct RouteBackwardArgs {
  const float* dweights;  // [M, topk]
  const void* logits;     // [M, E], rows row_stride elements apart
  int logits_type;
  long long row_stride;
  const int32_t* ids;     // [M, topk]
  int M, E, topk, softmax, renormalize;
  float scale;
  void* dlogits;          // [M, E], of the logits' type
};
cudaError_t launch_route_backward(const RouteBackwardArgs& a, cudaStream_t stream);

// out[m] = add[m] + scale[l] b[l] (a[l] x[m]), l = index[m]; add[m] where that is no adapter.
struct LoraArgs {
  const uint16_t* x;  // [M, K], rows ldx apart
  long long ldx;
  const uint16_t* a;  // [L, r, K]
  const uint16_t* b;  // [L, N, r]
  const float* scale;  // [L] or null: 1
  const int32_t* index;
  const void* add;  // [M, N] or null
  int add_type;
  void* out;
  int out_type;
  int M, K, N, r, L;
  void* workspace;  // lora_workspace_bytes()
};
constexpr int kMaxRank = 128;
// What the call needs: an order of the rows, where the kernel that reads one runs (null
// pointers count as aligned).
size_t lora_workspace_bytes(const LoraArgs& a);
cudaError_t launch_lora(const LoraArgs& a, int num_sms, cudaStream_t stream);

// Its kernel for many rows (lora_many.cu): rows of whole, aligned 16-byte pieces.
size_t lora_many_workspace(int M, int L);
cudaError_t launch_lora_many(const LoraArgs& a, int num_sms, cudaStream_t stream);

// SM count of the current device, and a stream-ordered memory pool of the library's own on
// it (ops_api.cu).
int num_sms(cudaError_t* err);
cudaMemPool_t scratch_pool(cudaError_t* err);

// Settings of the products' pipeline waits (MOE_W4A16_FP8_OPT_*); false: no such option
// or value.
bool fp8_set_option(int option, int value);
// Status word of the products (MOE_W4A16_STATUS_TIMEOUT when a wait gave up); clears it.
cudaError_t fp8_status(int32_t* out, cudaStream_t stream);

}  // namespace moe
