// C entry points of the operators around the routed experts: argument checks and launches.
#include "../../include/moe_w4a16.h"
#include "ops.cuh"

using namespace moe;

namespace {

// (rows are counted in int, tiles of 64 or 128 rows of `b` in a grid's second dimension)
constexpr int kMaxRows = 1 << 30;
constexpr int kMaxCols = 1 << 22;

int bad(const char* msg) { return report_error(MOE_W4A16_INVALID_ARG, msg); }
int shape(const char* msg) { return report_error(MOE_W4A16_UNSUPPORTED_SHAPE, msg); }
int done(cudaError_t e) {
  return e == cudaSuccess ? MOE_W4A16_OK : report_error(MOE_W4A16_CUDA_ERROR, cudaGetErrorString(e));
}

bool misaligned(const void* p, uintptr_t to) { return reinterpret_cast<uintptr_t>(p) % to != 0; }

size_t align_up(size_t x) { return (x + 255) / 256 * 256; }
int blocks(int n) { return (n + kScaleBlock - 1) / kScaleBlock; }

}  // namespace

namespace moe {

// SM count of the current device.
int num_sms(cudaError_t* err) {
  static PerDevice<int> known;
  int dev = 0;
  *err = cudaGetDevice(&dev);
  if (*err != cudaSuccess) return 0;
  std::atomic<int>* entry = known.of(dev);
  int n = entry ? entry->load() : 0;
  if (n) return n;
  *err = cudaDeviceGetAttribute(&n, cudaDevAttrMultiProcessorCount, dev);
  if (*err == cudaSuccess && entry) entry->store(n);
  return n;
}

// Stream-ordered memory pool of the current device, for calls without a workspace; keeps
// up to 64 MiB between calls.
cudaMemPool_t scratch_pool(cudaError_t* err) {
  static PerDevice<cudaMemPool_t> pools;
  int dev = 0;
  *err = cudaGetDevice(&dev);
  if (*err != cudaSuccess) return nullptr;
  std::atomic<cudaMemPool_t>* entry = pools.of(dev);
  if (!entry) {
    *err = cudaErrorInvalidDevice;
    return nullptr;
  }
  cudaMemPool_t pool = entry->load();
  if (pool) return pool;
  // (also during a stream capture, which this touches nothing of)
  cudaStreamCaptureMode mode = cudaStreamCaptureModeRelaxed;
  *err = cudaThreadExchangeStreamCaptureMode(&mode);
  if (*err != cudaSuccess) return nullptr;
  cudaMemPoolProps props = {};
  props.allocType = cudaMemAllocationTypePinned;
  props.location.type = cudaMemLocationTypeDevice;
  props.location.id = dev;
  *err = cudaMemPoolCreate(&pool, &props);
  if (*err == cudaSuccess) {
    unsigned long long keep = 64ull << 20;
    *err = cudaMemPoolSetAttribute(pool, cudaMemPoolAttrReleaseThreshold, &keep);
    cudaMemPool_t none = nullptr;
    if (*err != cudaSuccess || !entry->compare_exchange_strong(none, pool)) {
      cudaMemPoolDestroy(pool);
      pool = *err == cudaSuccess ? none : nullptr;  // (another thread's)
    }
  }
  const cudaError_t back = cudaThreadExchangeStreamCaptureMode(&mode);
  if (*err == cudaSuccess) *err = back;
  return *err == cudaSuccess ? pool : nullptr;
}

}  // namespace moe

namespace {

int check_quant(const void* x, int x_type, long long row_stride, int M, int cols, int width, const void* q,
                const void* s) {
  if (x_type != MOE_W4A16_F32 && x_type != MOE_W4A16_BF16) return bad("x_type must be MOE_W4A16_F32 or MOE_W4A16_BF16");
  if (M < 0 || cols < 1) return bad("need rows >= 0 and at least one column");
  if (M > kMaxRows || cols > kMaxCols) return shape("too many rows or columns (at most 2^30 and 2^22)");
  if (M > 0 && (!x || !q || !s)) return bad("null pointer argument");
  if (M > 1 && row_stride < width) return bad("row_stride is smaller than a row");
  if (misaligned(x, x_type == MOE_W4A16_F32 ? 4 : 2) || misaligned(s, 4)) return bad("x or s is not aligned to its type");
  return MOE_W4A16_OK;
}

}  // namespace

extern "C" {

int moe_w4a16_route_scored(const void* logits, int logits_type, long long row_stride, int M, int E, int topk,
                           int scoring, const float* bias, int n_group, int topk_group, int group_top,
                           int renormalize, float scale, int32_t* topk_ids, float* topk_weights, void* stream) {
  if (logits_type != MOE_W4A16_F32 && logits_type != MOE_W4A16_BF16)
    return bad("logits_type must be MOE_W4A16_F32 or MOE_W4A16_BF16");
  if (scoring != MOE_W4A16_SCORE_SOFTMAX && scoring != MOE_W4A16_SCORE_SIGMOID) return bad("unknown scoring");
  if (M < 0 || E < 1 || topk < 1) return bad("need M >= 0, E >= 1 and topk >= 1");
  if (E > 1024) return shape("the router supports at most 1024 experts");
  if (topk > 32) return shape("the router supports topk <= 32");
  if (n_group < 1 || E % n_group != 0) return bad("n_group must divide E");
  if (n_group > kMaxGroups) return shape("the router supports at most 32 groups");
  if (topk_group < 1 || topk_group > n_group) return bad("need 1 <= topk_group <= n_group");
  if (group_top != 1 && group_top != 2) return bad("group_top must be 1 or 2");
  if (topk > topk_group * (E / n_group)) return bad("topk exceeds the experts of topk_group groups");
  if (M == 0) return MOE_W4A16_OK;
  if (!logits || !topk_ids || !topk_weights) return bad("null pointer argument");
  if (M > 1 && row_stride < E) return bad("row_stride is smaller than a row");
  if (misaligned(logits, logits_type == MOE_W4A16_F32 ? 4 : 2) || misaligned(bias, 4) || misaligned(topk_ids, 4) ||
      misaligned(topk_weights, 4))
    return bad("a pointer is not aligned to its type");
  RouteScoredArgs a{};
  a.logits = logits;
  a.logits_type = logits_type;
  a.row_stride = row_stride;
  a.M = M;
  a.E = E;
  a.topk = topk;
  a.softmax = scoring == MOE_W4A16_SCORE_SOFTMAX;
  a.bias = bias;
  a.n_group = n_group;
  a.topk_group = topk_group;
  a.group_top = group_top;
  a.renormalize = renormalize != 0;
  a.scale = scale;
  a.ids = topk_ids;
  a.weights = topk_weights;
  return done(launch_route_scored(a, static_cast<cudaStream_t>(stream)));
}

int moe_w4a16_fp8_quantize(const void* x, int x_type, long long row_stride, int M, int K, uint8_t* q, float* s,
                           void* stream) {
  if (int rc = check_quant(x, x_type, row_stride, M, K, K, q, s)) return rc;
  if (M == 0) return MOE_W4A16_OK;
  return done(launch_quantize(QuantArgs{x, x_type, row_stride, M, K, q, s}, false, static_cast<cudaStream_t>(stream)));
}

int moe_w4a16_fp8_swiglu_quantize(const void* gate_up, int x_type, long long row_stride, int M, int N, uint8_t* q,
                                  float* s, void* stream) {
  if (int rc = check_quant(gate_up, x_type, row_stride, M, N, 2 * N, q, s)) return rc;
  if (M == 0) return MOE_W4A16_OK;
  return done(launch_quantize(QuantArgs{gate_up, x_type, row_stride, M, N, q, s}, true, static_cast<cudaStream_t>(stream)));
}

int moe_w4a16_fp8_quantize_weight(const void* w, int w_type, long long row_stride, int N, int K, uint8_t* q, float* s,
                                  void* stream) {
  if (int rc = check_quant(w, w_type, row_stride, N, K, K, q, s)) return rc;
  if (N > kMaxCols) return shape("a weight has at most 2^22 rows");
  if (N == 0) return MOE_W4A16_OK;
  return done(launch_quantize_weight(QuantArgs{w, w_type, row_stride, N, K, q, s}, static_cast<cudaStream_t>(stream)));
}

int moe_w4a16_fp8_matmul(const uint8_t* a, long long lda, const float* a_s, const uint8_t* b, long long ldb,
                         const float* b_s, const uint16_t* add, void* out, int out_type, int M, int N, int K,
                         void* stream) {
  if (out_type != MOE_W4A16_F32 && out_type != MOE_W4A16_BF16)
    return bad("out_type must be MOE_W4A16_F32 or MOE_W4A16_BF16");
  if (M < 0 || N < 0 || K < 1) return bad("need M >= 0, N >= 0 and K >= 1");
  if (M > kMaxRows || N > kMaxCols || K > kMaxCols) return shape("too large (at most M = 2^30, N = K = 2^22)");
  if (M == 0 || N == 0) return MOE_W4A16_OK;
  if (!a || !a_s || !b || !b_s || !out) return bad("null pointer argument");
  if ((M > 1 && lda < K) || (N > 1 && ldb < K)) return bad("a row stride is smaller than a row");
  if (misaligned(a_s, 4) || misaligned(b_s, 4) || misaligned(add, 2) || misaligned(out, out_type == MOE_W4A16_F32 ? 4 : 2))
    return bad("a pointer is not aligned to its type");
  cudaError_t e;
  const int sms = num_sms(&e);
  if (e != cudaSuccess) return done(e);
  Fp8MatmulArgs g{a, lda, a_s, b, ldb, b_s, add, out, out_type, M, N, K, false, nullptr, 0, 0};
  return done(launch_fp8_matmul(g, sms, static_cast<cudaStream_t>(stream)));
}

int moe_w4a16_fp8_plan_debug(int stage, const uint16_t* add, const void* out, int out_type, int M, int N, int K,
                             int32_t* plan) {
  if (stage < 0 || stage > 2) return bad("stage must be 0, 1 or 2");
  if (out_type != MOE_W4A16_F32 && out_type != MOE_W4A16_BF16)
    return bad("out_type must be MOE_W4A16_F32 or MOE_W4A16_BF16");
  if (M < 1 || N < 1 || K < 1) return bad("need M, N and K >= 1");
  if (M > kMaxRows || N > kMaxCols || K > kMaxCols) return shape("too large (at most M = 2^30, N = K = 2^22)");
  if (stage > 0 && (N % kScaleBlock != 0 || K % kScaleBlock != 0)) return shape("N and K must be multiples of 128");
  if (!plan) return bad("null pointer argument");
  cudaError_t e;
  const int sms = num_sms(&e);
  if (e != cudaSuccess) return done(e);
  const Fp8MatmulArgs g{nullptr, K, nullptr, nullptr, K, nullptr, add, const_cast<void*>(out), out_type, M, N, K, stage > 0,
                        nullptr, 0, 0};
  Fp8Plan p{};
  e = fp8_plan(g, stage == 1, sms, &p);
  plan[0] = p.rows, plan[1] = p.split;
  return done(e);
}

int moe_w4a16_fp8_set_option(int option, int value) {
  return fp8_set_option(option, value) ? MOE_W4A16_OK : bad("unknown option, or a value out of its range");
}

int moe_w4a16_fp8_status(int32_t* status, void* stream) {
  if (!status) return bad("null pointer argument");
  return done(fp8_status(status, static_cast<cudaStream_t>(stream)));
}

namespace {
struct SharedLayout {
  size_t q1, s1, q2, s2, total;
};
SharedLayout shared_layout(int M, int K, int N) {
  SharedLayout L{};
  const size_t m = static_cast<size_t>(M);
  size_t off = 0;
  L.q1 = off, off = align_up(off + m * K);
  L.s1 = off, off = align_up(off + m * blocks(K) * sizeof(float));
  L.q2 = off, off = align_up(off + m * N);
  L.s2 = off, off = align_up(off + m * blocks(N) * sizeof(float));
  L.total = off;
  return L;
}
bool shared_shape_ok(int M, int K, int N) {
  return M >= 0 && M <= kMaxRows && K >= 1 && K <= kMaxCols && N >= 1 && N <= kMaxCols / 2 && K % kScaleBlock == 0 &&
         N % kScaleBlock == 0;
}
}  // namespace

size_t moe_w4a16_shared_expert_workspace_size(int M, int K, int N) {
  return shared_shape_ok(M, K, N) ? shared_layout(M, K, N).total : 0;
}

int moe_w4a16_shared_expert(const uint16_t* hidden, const uint8_t* w1, const float* w1_s, const uint8_t* w2,
                            const float* w2_s, const uint16_t* add, uint16_t* out, int M, int K, int N,
                            void* workspace, size_t workspace_bytes, void* stream) {
  if (!shared_shape_ok(M, K, N))
    return shape("need 0 <= M <= 2^30 and K, N positive multiples of 128 (at most 2^22 and 2^21)");
  if (M == 0) return MOE_W4A16_OK;
  if (!hidden || !w1 || !w1_s || !w2 || !w2_s || !out) return bad("null pointer argument");
  if (misaligned(workspace, 256)) return bad("workspace must be 256-byte aligned");
  if (misaligned(w1, 16) || misaligned(w2, 16)) return bad("w1 and w2 must be 16-byte aligned");
  if (misaligned(hidden, 2) || misaligned(w1_s, 4) || misaligned(w2_s, 4) || misaligned(add, 2) || misaligned(out, 2))
    return bad("a pointer is not aligned to its type");
  const SharedLayout L = shared_layout(M, K, N);
  if (workspace && workspace_bytes < L.total)
    return report_error(MOE_W4A16_WORKSPACE_TOO_SMALL, "workspace too small (moe_w4a16_shared_expert_workspace_size)");
  cudaError_t e;
  const int sms = num_sms(&e);
  if (e != cudaSuccess) return done(e);
  auto s = static_cast<cudaStream_t>(stream);
  void* scratch = nullptr;
  if (!workspace) {
    cudaMemPool_t pool = scratch_pool(&e);
    if (e == cudaSuccess) e = cudaMallocFromPoolAsync(&scratch, L.total, pool, s);
    if (e != cudaSuccess) return done(e);
  }
  uint8_t* ws = static_cast<uint8_t*>(workspace ? workspace : scratch);
  uint8_t* q1 = ws + L.q1;
  uint8_t* q2 = ws + L.q2;
  float* s1 = reinterpret_cast<float*>(ws + L.s1);
  float* s2 = reinterpret_cast<float*>(ws + L.s2);
  e = launch_quantize(QuantArgs{hidden, kTypeBf16, K, M, K, q1, s1}, false, s);
  if (e == cudaSuccess)
    e = launch_fp8_swiglu(Fp8MatmulArgs{q1, K, s1, w1, K, w1_s, nullptr, q2, kTypeF32, M, N, K, true, s2, 0, 0}, sms, s);
  if (e == cudaSuccess)
    e = launch_fp8_matmul(Fp8MatmulArgs{q2, N, s2, w2, N, w2_s, add, out, kTypeBf16, M, K, N, true, nullptr, 0, 0}, sms, s);
  if (scratch) {
    const cudaError_t freed = cudaFreeAsync(scratch, s);
    if (e == cudaSuccess) e = freed;
  }
  return done(e);
}

}  // extern "C"
