// C entry points of the operators between the router and the experts (order, gather,
// combine, their gradients, the router's) and of the low-rank adapters: argument checks and
// launches.
#include <initializer_list>

#include "../../include/moe_w4a16.h"
#include "ops.cuh"

using namespace moe;

namespace {

constexpr int kMaxRows = 1 << 30;
constexpr int kMaxCols = 1 << 22;
constexpr long long kMaxOrder = 1LL << 30;  // rows of an order

int bad(const char* msg) { return report_error(MOE_W4A16_INVALID_ARG, msg); }
int shape(const char* msg) { return report_error(MOE_W4A16_UNSUPPORTED_SHAPE, msg); }
int done(cudaError_t e) {
  return e == cudaSuccess ? MOE_W4A16_OK : report_error(MOE_W4A16_CUDA_ERROR, cudaGetErrorString(e));
}
bool misaligned(const void* p, uintptr_t to) { return reinterpret_cast<uintptr_t>(p) % to != 0; }
bool float_type(int t) { return t == MOE_W4A16_F32 || t == MOE_W4A16_BF16; }
int item(int type) { return type == MOE_W4A16_F32 ? 4 : type == MOE_W4A16_BF16 ? 2 : 1; }

// An array, of rows `stride` bytes apart where it has more than one.
struct Array {
  const void* p;
  long long bytes;  // of a row
  long long rows = 1, stride = 0;
};
Array matrix(const void* p, int rows, long long stride, int cols, int bytes) {
  return {p, static_cast<long long>(cols) * bytes, rows, stride * bytes};
}
// Whether it shares a byte with the array `q`, of one row (a null or an empty one shares none).
bool share(const Array& x, const Array& q) {
  if (!x.p || !q.p || x.bytes <= 0 || x.rows <= 0 || q.bytes <= 0) return false;
  const auto a = static_cast<__int128>(reinterpret_cast<uintptr_t>(x.p)), b = static_cast<__int128>(reinterpret_cast<uintptr_t>(q.p));
  // the first row that ends behind q's begin
  const __int128 row = b < a + x.bytes ? 0 : x.rows == 1 ? 1 : (b - a - x.bytes) / x.stride + 1;
  return row < x.rows && a + row * x.stride < b + q.bytes;
}
// Every output against every input that the same launches read.
bool share(std::initializer_list<Array> inputs, std::initializer_list<Array> outputs) {
  for (const Array& in : inputs)
    for (const Array& out : outputs)
      if (share(in, out)) return true;
  return false;
}
constexpr const char* kShared = "an output may not share memory with an input";

// Rows of an order, or -1 for sizes that are not supported.
long long rows_of(int M, int topk, int E, int block) {
  if (M < 0 || topk < 1 || topk > kMaxTopk || E < 1 || E > 1024 || block < 1 || block > kMaxCols) return -1;
  const long long n = static_cast<long long>(M) * topk;
  const long long rows = n + (n < E ? n : E) * (block - 1LL);
  return n <= kMaxOrder && rows <= kMaxOrder ? rows : -1;
}

int check_order(int M, int topk, int E, int block) {
  if (M < 0 || topk < 1 || E < 1 || block < 1) return bad("need M >= 0 and topk, E, block >= 1");
  if (topk > kMaxTopk || E > 1024) return shape("at most 32 choices a token and 1,024 experts");
  if (rows_of(M, topk, E, block) < 0) return shape("too many rows (at most 2^30, block at most 2^22)");
  return MOE_W4A16_OK;
}

int check_order_out(const int32_t* offsets, const int32_t* slots, const int32_t* position) {
  if (!offsets || !slots || !position) return bad("null pointer argument");
  if (misaligned(offsets, 4) || misaligned(slots, 4) || misaligned(position, 4))
    return bad("a pointer is not aligned to its type");
  return MOE_W4A16_OK;
}

int check_rows(const void* x, int type, long long row_stride, int M, int K, const void* out) {
  if (!float_type(type) && type != MOE_W4A16_E4M3) return bad("type must be MOE_W4A16_F32, _BF16 or _E4M3");
  if (K < 1) return bad("need K >= 1");
  if (K > kMaxCols) return shape("too many columns (at most 2^22)");
  if (M > 0 && (!x || !out)) return bad("null pointer argument");
  if (M > 1 && row_stride < K) return bad("row_stride is smaller than a row");
  if (misaligned(x, item(type)) || misaligned(out, item(type))) return bad("a pointer is not aligned to its type");
  return MOE_W4A16_OK;
}

}  // namespace

extern "C" {

long long moe_w4a16_dispatch_rows(int M, int topk, int E, int block) { return rows_of(M, topk, E, block); }

int moe_w4a16_dispatch_sort(const int32_t* topk_ids, int M, int topk, int expert_begin, int E, int block,
                            int32_t* offsets, int32_t* slots, int32_t* position, void* stream) {
  if (int rc = check_order(M, topk, E, block)) return rc;
  if (expert_begin < 0) return bad("need expert_begin >= 0");
  if (!offsets || (M > 0 && (!topk_ids || !slots || !position))) return bad("null pointer argument");
  if (misaligned(topk_ids, 4) || misaligned(offsets, 4) || misaligned(slots, 4) || misaligned(position, 4))
    return bad("a pointer is not aligned to its type");
  const long long n = 4LL * M * topk;
  if (share({{topk_ids, n}}, {{offsets, 4LL * (E + 1)}, {slots, 4 * rows_of(M, topk, E, block)}, {position, n}})) return bad(kShared);
  const SortArgs a{topk_ids, M * topk, expert_begin, E, 0, block, offsets, slots,
                   static_cast<int>(rows_of(M, topk, E, block)), position};
  return done(launch_sort(a, static_cast<cudaStream_t>(stream)));
}

int moe_w4a16_dispatch_gather(const void* x, int type, long long row_stride, const int32_t* offsets,
                              const int32_t* slots, const int32_t* position, void* out, int M, int K, int topk, int E,
                              int block, void* stream) {
  if (int rc = check_order(M, topk, E, block)) return rc;
  if (int rc = check_rows(x, type, row_stride, M, K, out)) return rc;
  if (M == 0) return MOE_W4A16_OK;
  if (int rc = check_order_out(offsets, slots, position)) return rc;
  const long long rows = rows_of(M, topk, E, block);
  if (share({matrix(x, M, row_stride, K, item(type)), {offsets, 4LL * (E + 1)}, {slots, 4 * rows}, {position, 4LL * M * topk}},
            {{out, rows * K * item(type)}}))
    return bad(kShared);
  cudaError_t e;
  const int sms = num_sms(&e);
  if (e != cudaSuccess) return done(e);
  const GatherRowsArgs g{x, M > 1 ? row_stride * item(type) : 0, static_cast<long long>(K) * item(type), offsets, slots,
                         position, out, M, topk, E, block, static_cast<int>(rows)};
  return done(launch_gather(g, sms, static_cast<cudaStream_t>(stream)));
}

int moe_w4a16_dispatch_sort_gather(const void* x, int type, long long row_stride, const int32_t* topk_ids, int M, int K,
                                   int topk, int expert_begin, int E, int block, int32_t* offsets, int32_t* slots,
                                   int32_t* position, void* out, void* stream) {
  if (int rc = check_order(M, topk, E, block)) return rc;
  if (int rc = check_rows(x, type, row_stride, M, K, out)) return rc;
  if (expert_begin < 0) return bad("need expert_begin >= 0");
  if (M == 0) return moe_w4a16_dispatch_sort(topk_ids, M, topk, expert_begin, E, block, offsets, slots, position, stream);
  if (int rc = check_order_out(offsets, slots, position)) return rc;
  if (!topk_ids || misaligned(topk_ids, 4)) return bad("topk_ids is null or not aligned to its type");
  const int rows = static_cast<int>(rows_of(M, topk, E, block));
  const long long n = 4LL * M * topk;
  if (share({matrix(x, M, row_stride, K, item(type)), {topk_ids, n}},
            {{offsets, 4LL * (E + 1)}, {slots, 4LL * rows}, {position, n}, {out, static_cast<long long>(rows) * K * item(type)}}))
    return bad(kShared);
  cudaError_t e;
  const int sms = num_sms(&e);
  if (e != cudaSuccess) return done(e);
  const SortArgs o{topk_ids, M * topk, expert_begin, E, 0, block, offsets, slots, rows, position};
  const GatherRowsArgs g{x, M > 1 ? row_stride * item(type) : 0, static_cast<long long>(K) * item(type), offsets, slots,
                         position, out, M, topk, E, block, rows};
  return done(launch_sort_gather(o, g, sms, static_cast<cudaStream_t>(stream)));
}

int moe_w4a16_combine(const void* y, int y_type, const float* weights, const int32_t* position, const void* add,
                      void* out, int out_type, int M, int K, int topk, int rows, void* stream) {
  if (!float_type(y_type) || !float_type(out_type)) return bad("y_type and out_type must be MOE_W4A16_F32 or _BF16");
  if (M < 0 || K < 1 || topk < 1 || rows < 0) return bad("need M >= 0, K >= 1, topk >= 1 and rows >= 0");
  if (M > kMaxRows || K > kMaxCols || topk > kMaxTopk || static_cast<long long>(M) * topk > kMaxOrder || rows > kMaxOrder)
    return shape("too large (at most 2^30 choices and rows, 2^22 columns, 32 choices a token)");
  if (M == 0) return MOE_W4A16_OK;
  if ((rows > 0 && !y) || !position || !out) return bad("null pointer argument");
  if (misaligned(y, item(y_type)) || misaligned(weights, 4) || misaligned(position, 4) ||
      misaligned(add, item(out_type)) || misaligned(out, item(out_type)))
    return bad("a pointer is not aligned to its type");
  const Array to{out, static_cast<long long>(M) * K * item(out_type)};
  const long long n = 4LL * M * topk;
  if (share({{y, static_cast<long long>(rows) * K * item(y_type)}, {weights, n}, {position, n}}, {to})) return bad(kShared);
  if (add != out && share({add, to.bytes}, to)) return bad("add and out may be one array or two, and not overlap");
  cudaError_t e;
  const int sms = num_sms(&e);
  if (e != cudaSuccess) return done(e);
  const CombineArgs c{y, y_type, weights, position, add, out, out_type, M, K, topk, rows};
  return done(launch_combine(c, sms, static_cast<cudaStream_t>(stream)));
}

int moe_w4a16_combine_backward(const void* grad, int grad_type, const void* y, int y_type, const float* weights,
                               const int32_t* offsets, const int32_t* slots, const int32_t* position, void* dy,
                               float* dweights, int M, int K, int topk, int E, int block, void* stream) {
  if (int rc = check_order(M, topk, E, block)) return rc;
  if (!float_type(y_type) || !float_type(grad_type)) return bad("y_type and grad_type must be MOE_W4A16_F32 or _BF16");
  if (K < 1) return bad("need K >= 1");
  if (K > kMaxCols) return shape("too many columns (at most 2^22)");
  if (M == 0) return MOE_W4A16_OK;
  if (!grad || !y || !weights || !dy || !dweights) return bad("null pointer argument");
  if (int rc = check_order_out(offsets, slots, position)) return rc;
  if (misaligned(grad, item(grad_type)) || misaligned(y, item(y_type)) || misaligned(dy, item(y_type)) ||
      misaligned(weights, 4) || misaligned(dweights, 4))
    return bad("a pointer is not aligned to its type");
  const long long rows = rows_of(M, topk, E, block), bytes = rows * K * item(y_type), n = 4LL * M * topk;
  if (share({{grad, static_cast<long long>(M) * K * item(grad_type)}, {y, bytes}, {weights, n}, {offsets, 4LL * (E + 1)}, {slots, 4 * rows},
             {position, n}},
            {{dy, bytes}, {dweights, n}}))
    return bad(kShared);
  cudaError_t e;
  const int sms = num_sms(&e);
  if (e != cudaSuccess) return done(e);
  const CombineBackwardArgs c{grad, grad_type, y, y_type, weights, offsets, slots, position, dy, dweights,
                              M, K, topk, E, block, static_cast<int>(rows)};
  return done(launch_combine_backward(c, sms, static_cast<cudaStream_t>(stream)));
}

int moe_w4a16_route_scored_backward(const float* dweights, const void* logits, int logits_type, long long row_stride,
                                    const int32_t* topk_ids, int M, int E, int topk, int scoring, int renormalize,
                                    float scale, void* dlogits, void* stream) {
  if (!float_type(logits_type)) return bad("logits_type must be MOE_W4A16_F32 or MOE_W4A16_BF16");
  if (scoring != MOE_W4A16_SCORE_SOFTMAX && scoring != MOE_W4A16_SCORE_SIGMOID) return bad("unknown scoring");
  if (M < 0 || E < 1 || topk < 1) return bad("need M >= 0, E >= 1 and topk >= 1");
  if (E > 1024) return shape("the router supports at most 1024 experts");
  if (topk > kMaxTopk) return shape("the router supports topk <= 32");
  if (M > kMaxRows) return shape("too many rows (at most 2^30)");
  if (M == 0) return MOE_W4A16_OK;
  if (!dweights || !logits || !topk_ids || !dlogits) return bad("null pointer argument");
  if (M > 1 && row_stride < E) return bad("row_stride is smaller than a row");
  if (misaligned(logits, item(logits_type)) || misaligned(dlogits, item(logits_type)) || misaligned(dweights, 4) ||
      misaligned(topk_ids, 4))
    return bad("a pointer is not aligned to its type");
  const long long n = 4LL * M * topk;
  if (share({matrix(logits, M, row_stride, E, item(logits_type)), {dweights, n}, {topk_ids, n}},
            {{dlogits, static_cast<long long>(M) * E * item(logits_type)}}))
    return bad(kShared);
  const RouteBackwardArgs a{dweights, logits, logits_type, row_stride, topk_ids, M, E, topk,
                            scoring == MOE_W4A16_SCORE_SOFTMAX, renormalize != 0, scale, dlogits};
  return done(launch_route_backward(a, static_cast<cudaStream_t>(stream)));
}

namespace {
bool lora_shape_ok(int M, int K, int N, int r, int L) {
  return M >= 0 && M <= kMaxRows / 2 && K >= 1 && K <= kMaxCols && N >= 1 && N <= kMaxCols && r >= 1 && r <= kMaxRank &&
         L >= 1 && L < 1024;
}
}  // namespace

size_t moe_w4a16_lora_workspace_size(int M, int K, int N, int r, int L) {
  if (!lora_shape_ok(M, K, N, r, L)) return 0;
  return lora_workspace_bytes(LoraArgs{nullptr, K, nullptr, nullptr, nullptr, nullptr, nullptr, MOE_W4A16_F32, nullptr, MOE_W4A16_F32, M, K, N,
                                       r, L, nullptr});
}

int moe_w4a16_lora(const uint16_t* x, long long ldx, const uint16_t* a, const uint16_t* b, const float* scale,
                   const int32_t* index, const void* add, int add_type, void* out, int out_type, int M, int K, int N,
                   int r, int L, void* workspace, size_t workspace_bytes, void* stream) {
  if (!float_type(out_type) || (add && !float_type(add_type))) return bad("types must be MOE_W4A16_F32 or MOE_W4A16_BF16");
  if (M < 0 || K < 1 || N < 1 || r < 1 || L < 1) return bad("need M >= 0 and K, N, r, L >= 1");
  if (!lora_shape_ok(M, K, N, r, L)) return shape("at most 2^29 rows, 2^22 columns, rank 128 and 1,023 adapters");
  if (M == 0) return MOE_W4A16_OK;
  if (!x || !a || !b || !index || !out) return bad("null pointer argument");
  if (M > 1 && ldx < K) return bad("ldx is smaller than a row");
  if (misaligned(x, 2) || misaligned(a, 2) || misaligned(b, 2) || misaligned(scale, 4) || misaligned(index, 4) ||
      misaligned(out, item(out_type)) || (add && misaligned(add, item(add_type))))
    return bad("a pointer is not aligned to its type");
  if (add == out && add_type != out_type) return bad("add may be out only where they are of one type");
  const Array to{out, static_cast<long long>(M) * N * item(out_type)};
  if (share({matrix(x, M, ldx, K, 2), {a, 2LL * L * r * K}, {b, 2LL * L * N * r}, {scale, 4LL * L}, {index, 4LL * M}}, {to}))
    return bad(kShared);
  if (add != out && share({add, static_cast<long long>(M) * N * item(add_type)}, to))
    return bad("add and out may be one array or two, and not overlap");
  if (misaligned(workspace, 256)) return bad("workspace must be 256-byte aligned");
  LoraArgs args{x, ldx, a, b, scale, index, add, add_type, out, out_type, M, K, N, r, L, workspace};
  const size_t need = lora_workspace_bytes(args);
  if (workspace && workspace_bytes < need)
    return report_error(MOE_W4A16_WORKSPACE_TOO_SMALL, "workspace too small (moe_w4a16_lora_workspace_size)");
  cudaError_t e;
  const int sms = num_sms(&e);
  if (e != cudaSuccess) return done(e);
  auto s = static_cast<cudaStream_t>(stream);
  void* scratch = nullptr;
  if (!workspace && need) {
    cudaMemPool_t pool = scratch_pool(&e);
    if (e == cudaSuccess) e = cudaMallocFromPoolAsync(&scratch, need, pool, s);
    if (e != cudaSuccess) return done(e);
  }
  if (scratch) args.workspace = scratch;
  e = launch_lora(args, sms, s);
  if (scratch) {
    const cudaError_t freed = cudaFreeAsync(scratch, s);
    if (e == cudaSuccess) e = freed;
  }
  return done(e);
}

}  // extern "C"
