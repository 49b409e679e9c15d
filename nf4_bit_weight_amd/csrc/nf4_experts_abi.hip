// extern "C" entry points of nf4_experts.h and nf4_int8.h: argument checks and
// launches.  No entry point allocates, frees or synchronises.
#include <climits>
#include <cmath>

#include "../../include/nf4_experts.h"
#include "../../include/nf4_int8.h"
#include "nf4_experts.hpp"
#include "nf4_int8.hpp"
#include "nf4_internal.hpp"

namespace nf4 {
namespace {

bool aligned(const void* p, uintptr_t n) { return (reinterpret_cast<uintptr_t>(p) & (n - 1)) == 0; }
int to_status(hipError_t e) { return e == hipSuccess ? NF4_OK : NF4_ERR_HIP; }
bool launchable(int64_t workgroups, int64_t threads) { return workgroups <= UINT32_MAX / threads; }
uintptr_t size_of(int dtype) { return dtype == NF4_DTYPE_BF16 ? 2 : 4; }
bool is_float(int dtype) { return dtype == NF4_DTYPE_F32 || dtype == NF4_DTYPE_BF16; }

int check_choices(int64_t T, int32_t E, int32_t k) {
  if (T < 0 || E < 1 || k < 1 || k > E) return NF4_ERR_SHAPE;
  if (E > 1024 || k > 64 || T > (1 << 30) / k) return NF4_ERR_UNSUPPORTED;
  // above 256 experts a wave a token, up to 16 waves a workgroup (which the last one fills up)
  return launchable(E > 256 ? (T + 15) / 16 * 16 : T, 64) ? NF4_OK : NF4_ERR_UNSUPPORTED;
}

// Rows of the tokens and of their choices.
int check_rows(int dtype, int64_t T, int64_t H, int32_t k) {
  if (!is_float(dtype)) return NF4_ERR_DTYPE;
  if (T < 0 || H < 0 || k < 1) return NF4_ERR_SHAPE;
  if (k > 64 || T > (1 << 30) / k || H > 1 << 23) return NF4_ERR_UNSUPPORTED;   // (a grid has 65535 workgroups across)
  return launchable(T * (H > 256 ? (H + 255) / 256 : 1), 256) ? NF4_OK : NF4_ERR_UNSUPPORTED;
}

int check_plan(const int32_t* experts, int64_t T, const int32_t* offsets, const int32_t* tokens, const int32_t* slots, const void* ws,
               size_t ws_bytes, size_t need) {
  if (!offsets || (T > 0 && (!experts || !tokens || !slots))) return NF4_ERR_NULL;
  if (!aligned(experts, 4) || !aligned(offsets, 4) || !aligned(tokens, 4) || !aligned(slots, 4)) return NF4_ERR_ALIGN;
  if (need > 0 && (!ws || ws_bytes < need)) return NF4_ERR_WORKSPACE;
  if (need > 0 && !aligned(ws, 16)) return NF4_ERR_ALIGN;
  return NF4_OK;
}

// What of the product's workspace holds the quantised rows, and all of it.
struct Int8Plan {
  size_t q = 0, scale = 0, bytes = 0;
};
int check_int8(int x_dtype, int64_t x_rows, int64_t M, int64_t N, int64_t K, int32_t E, Int8Plan& pl) {
  if (!is_float(x_dtype) && x_dtype != NF4_DTYPE_I8) return NF4_ERR_DTYPE;
  if (x_rows < 0 || M < 0 || N < 0 || K < 0 || E < 0) return NF4_ERR_SHAPE;
  if (K > 130944 || x_rows > 1 << 28 || M > 1 << 28 || N > 1 << 28 || E > 1024) return NF4_ERR_UNSUPPORTED;
  if (!launchable(x_rows, 256)) return NF4_ERR_UNSUPPORTED;
  if (!int8_launchable(M, N, E)) return NF4_ERR_UNSUPPORTED;
  if (M == 0 || N == 0) return NF4_OK;
  if (x_dtype != NF4_DTYPE_I8) {
    pl.q = static_cast<size_t>(x_rows) * int8_row_bytes(K);
    pl.scale = (static_cast<size_t>(x_rows) * 4 + 15) / 16 * 16;
  }
  pl.bytes = pl.q + pl.scale;
  return NF4_OK;
}

int int8_product(const void* x, int x_dtype, int64_t stride, const float* x_scale, int64_t x_rows, const int32_t* tokens,
                 const int32_t* offsets, int32_t E, int64_t M, const int8_t* q, const float* scale, int64_t N, int64_t K,
                 const float* bias, void* y, int y_dtype, int fill, void* ws, size_t ws_bytes, void* stream) {
  Int8Plan pl;
  const int st = check_int8(x_dtype, x_rows, M, N, K, E, pl);
  if (st) return st;
  if (!is_float(y_dtype)) return NF4_ERR_DTYPE;
  const bool ready = x_dtype == NF4_DTYPE_I8;
  if (!ready && stride < 0) return NF4_ERR_SHAPE;
  if (!aligned(x, ready ? 16 : size_of(x_dtype)) || !aligned(x_scale, 4) || !aligned(tokens, 4) || !aligned(offsets, 4) ||
      !aligned(q, 16) || !aligned(scale, 4) || !aligned(bias, 4) || !aligned(y, 16))
    return NF4_ERR_ALIGN;
  if (M == 0 || N == 0) return NF4_OK;
  if (!y || !scale || (K > 0 && !q)) return NF4_ERR_NULL;
  if (x_rows > 0 && ((K > 0 && !x) || (ready && !x_scale))) return NF4_ERR_NULL;
  if (pl.bytes > 0 && (!ws || ws_bytes < pl.bytes)) return NF4_ERR_WORKSPACE;
  if (pl.bytes > 0 && !aligned(ws, 16)) return NF4_ERR_ALIGN;
  const hipStream_t s = static_cast<hipStream_t>(stream);
  Int8Args a{static_cast<const int8_t*>(x), x_scale, x_rows, tokens, offsets, E, M, N, int8_row_bytes(K), q, scale, bias, y,
             y_dtype == NF4_DTYPE_BF16, fill != 0};
  const Int8Source source{x, x_dtype == NF4_DTYPE_BF16, stride, static_cast<int32_t>(K)};
  if (!ready && int8_fused(a)) return to_status(launch_int8_matmul(a, &source, s));
  if (!ready) {
    int8_t* xq = static_cast<int8_t*>(ws);
    float* xs = reinterpret_cast<float*>(xq + pl.q);
    if (x_rows > 0) {
      const hipError_t e = launch_int8_quantize(x, x_dtype == NF4_DTYPE_BF16, stride, x_rows, K, xq, xs, s);
      if (e != hipSuccess) return NF4_ERR_HIP;
    }
    a.x = xq;
    a.x_scale = xs;
  }
  return to_status(launch_int8_matmul(a, nullptr, s));
}

}  // namespace
}  // namespace nf4

using namespace nf4;

extern "C" {

int nf4_route_fwd(const void* logits, int dtype, int64_t stride, int64_t T, int32_t E, int32_t k, const float* bias, int score,
                  int32_t groups, int32_t top_groups, int group_score, int renormalize, float scale, float* weights,
                  int32_t* experts, int32_t* offsets, int32_t* tokens, int32_t* slots, void* ws, size_t ws_bytes, void* stream) {
  int st = check_choices(T, E, k);
  if (st) return st;
  if (!is_float(dtype)) return NF4_ERR_DTYPE;
  if (stride < 0 || groups < 1 || E % groups || top_groups < 1 || top_groups > groups) return NF4_ERR_SHAPE;
  if (score != NF4_SCORE_SOFTMAX && score != NF4_SCORE_SIGMOID) return NF4_ERR_UNSUPPORTED;
  if (group_score != NF4_GROUP_MAX && group_score != NF4_GROUP_TOP2) return NF4_ERR_UNSUPPORTED;
  if (!(scale > 0.0f) || !std::isfinite(scale)) return NF4_ERR_SHAPE;
  if (T > 0 && (!logits || !weights || !experts)) return NF4_ERR_NULL;
  if (!aligned(logits, size_of(dtype)) || !aligned(bias, 4) || !aligned(weights, 4) || !aligned(experts, 4)) return NF4_ERR_ALIGN;
  const bool plan = offsets || tokens || slots;
  if (plan) {
    st = check_plan(experts, T, offsets, tokens, slots, ws, ws_bytes, plan_ws_bytes(T, k, E));
    if (st) return st;
  }
  const hipStream_t s = static_cast<hipStream_t>(stream);
  const PlanArgs pl{experts, static_cast<int32_t>(T), k, E, offsets, tokens, slots};
  if (T == 0) return plan ? to_status(launch_plan(pl, ws, s)) : NF4_OK;
  const RouteArgs a{logits, dtype == NF4_DTYPE_BF16, stride, static_cast<int32_t>(T), E, k, bias, score == NF4_SCORE_SIGMOID,
                    group_score == NF4_GROUP_TOP2, renormalize != 0, groups, top_groups, scale, weights, experts};
  const hipError_t e = launch_route(a, pl, ws, s);
  if (e == hipSuccess) count_path(NF4_PATH_ROUTE_FWD);
  if (e == hipSuccess && plan) count_path(NF4_PATH_EXPERT_PLAN);
  return to_status(e);
}

int nf4_route_bwd(const float* grad_weights, const void* logits, int dtype, int64_t stride, int64_t T, int32_t E, int32_t k,
                  const float* weights, const int32_t* experts, int score, int renormalize, float scale, void* grad_logits,
                  void* stream) {
  const int st = check_choices(T, E, k);
  if (st) return st;
  if (!is_float(dtype)) return NF4_ERR_DTYPE;
  if (stride < 0) return NF4_ERR_SHAPE;
  if (score != NF4_SCORE_SOFTMAX && score != NF4_SCORE_SIGMOID) return NF4_ERR_UNSUPPORTED;
  if (!(scale > 0.0f) || !std::isfinite(scale)) return NF4_ERR_SHAPE;
  if (T > 0 && (!grad_weights || !logits || !weights || !experts || !grad_logits)) return NF4_ERR_NULL;
  if (!aligned(logits, size_of(dtype)) || !aligned(grad_weights, 4) || !aligned(weights, 4) || !aligned(experts, 4) ||
      !aligned(grad_logits, size_of(dtype)))
    return NF4_ERR_ALIGN;
  if (T == 0) return NF4_OK;
  const RouteArgs a{logits, dtype == NF4_DTYPE_BF16, stride, static_cast<int32_t>(T), E, k, nullptr, score == NF4_SCORE_SIGMOID,
                    false, renormalize != 0, 1, 1, scale, const_cast<float*>(weights), const_cast<int32_t*>(experts)};
  const hipError_t e = launch_route_bwd(a, grad_weights, grad_logits, static_cast<hipStream_t>(stream));
  if (e == hipSuccess) count_path(NF4_PATH_ROUTE_BWD);
  return to_status(e);
}

size_t nf4_expert_plan_workspace(int64_t T, int32_t k, int32_t E) {
  return check_choices(T, E, 1) || k < 1 || k > 64 || T > (1 << 30) / k ? SIZE_MAX : plan_ws_bytes(T, k, E);
}

int nf4_expert_plan(const int32_t* experts, int64_t T, int32_t k, int32_t E, int32_t* offsets, int32_t* tokens, int32_t* slots,
                    void* ws, size_t ws_bytes, void* stream) {
  int st = check_choices(T, E, 1);                             // a choice from elsewhere may name an expert twice: k > E
  if (!st && k < 1) st = NF4_ERR_SHAPE;
  if (!st && (k > 64 || T > (1 << 30) / k)) st = NF4_ERR_UNSUPPORTED;
  if (!st) st = check_plan(experts, T, offsets, tokens, slots, ws, ws_bytes, plan_ws_bytes(T, k, E));
  if (st) return st;
  const hipError_t e = launch_plan({experts, static_cast<int32_t>(T), k, E, offsets, tokens, slots}, ws,
                                   static_cast<hipStream_t>(stream));
  if (e == hipSuccess) count_path(NF4_PATH_EXPERT_PLAN);
  return to_status(e);
}

int nf4_expert_gather(const void* x, int dtype, int64_t stride, int64_t T, int64_t H, int32_t k, const int32_t* slots,
                      const int32_t* end, void* rows, int fill_outside, void* stream) {
  const int st = check_rows(dtype, T, H, k);
  if (st) return st;
  if (stride < 0) return NF4_ERR_SHAPE;
  if (!aligned(x, size_of(dtype)) || !aligned(slots, 4) || !aligned(end, 4) || !aligned(rows, size_of(dtype))) return NF4_ERR_ALIGN;
  if (T == 0 || H == 0) return NF4_OK;
  if (!x || !slots || !rows || (fill_outside && !end)) return NF4_ERR_NULL;
  const RowsArgs a{dtype == NF4_DTYPE_BF16, H, static_cast<int32_t>(T), k, slots, end, fill_outside != 0};
  const hipError_t e = launch_gather(a, x, stride, rows, static_cast<hipStream_t>(stream));
  if (e == hipSuccess) count_path(NF4_PATH_EXPERT_GATHER);
  return to_status(e);
}

int nf4_expert_gather_bwd(const void* grad_rows, int dtype, int64_t T, int64_t H, int32_t k, const int32_t* slots, void* grad_x,
                          void* stream) {
  const int st = check_rows(dtype, T, H, k);
  if (st) return st;
  if (!aligned(grad_rows, size_of(dtype)) || !aligned(slots, 4) || !aligned(grad_x, size_of(dtype))) return NF4_ERR_ALIGN;
  if (T == 0 || H == 0) return NF4_OK;
  if (!grad_rows || !slots || !grad_x) return NF4_ERR_NULL;
  const RowsArgs a{dtype == NF4_DTYPE_BF16, H, static_cast<int32_t>(T), k, slots, nullptr, false};
  const hipError_t e = launch_gather_bwd(a, grad_rows, grad_x, static_cast<hipStream_t>(stream));
  if (e == hipSuccess) count_path(NF4_PATH_EXPERT_GATHER_BWD);
  return to_status(e);
}

int nf4_expert_combine_fwd(const void* rows, int dtype, int64_t T, int64_t H, int32_t k, const float* weights,
                           const int32_t* slots, void* out, void* stream) {
  const int st = check_rows(dtype, T, H, k);
  if (st) return st;
  if (!aligned(rows, size_of(dtype)) || !aligned(weights, 4) || !aligned(slots, 4) || !aligned(out, size_of(dtype)))
    return NF4_ERR_ALIGN;
  if (T == 0 || H == 0) return NF4_OK;
  if (!rows || !weights || !slots || !out) return NF4_ERR_NULL;
  const RowsArgs a{dtype == NF4_DTYPE_BF16, H, static_cast<int32_t>(T), k, slots, nullptr, false};
  const hipError_t e = launch_combine(a, rows, weights, out, static_cast<hipStream_t>(stream));
  if (e == hipSuccess) count_path(NF4_PATH_EXPERT_COMBINE);
  return to_status(e);
}

int nf4_expert_combine_bwd(const void* grad_out, int64_t grad_stride, const void* rows, int dtype, int64_t T, int64_t H, int32_t k,
                           const float* weights, const int32_t* slots, const int32_t* end, void* grad_rows, float* grad_weights,
                           int fill_outside, void* stream) {
  const int st = check_rows(dtype, T, H, k);
  if (st) return st;
  if (grad_stride < 0) return NF4_ERR_SHAPE;
  if (!aligned(grad_out, size_of(dtype)) || !aligned(rows, size_of(dtype)) || !aligned(weights, 4) || !aligned(slots, 4) ||
      !aligned(end, 4) || !aligned(grad_rows, size_of(dtype)) || !aligned(grad_weights, 4))
    return NF4_ERR_ALIGN;
  if (T == 0 || (!grad_rows && !grad_weights)) return NF4_OK;
  if (!slots || (grad_rows && !weights) || (fill_outside && grad_rows && !end)) return NF4_ERR_NULL;
  if (H > 0 && (!grad_out || (grad_weights && !rows))) return NF4_ERR_NULL;
  const RowsArgs a{dtype == NF4_DTYPE_BF16, H, static_cast<int32_t>(T), k, slots, end, fill_outside != 0};
  const hipError_t e = launch_combine_bwd(a, grad_out, grad_stride, rows, weights, grad_rows, grad_weights,
                                          static_cast<hipStream_t>(stream));
  if (e == hipSuccess) count_path(NF4_PATH_EXPERT_COMBINE_BWD);
  return to_status(e);
}

int64_t nf4_int8_row_bytes(int64_t K) { return K < 0 ? -1 : int8_row_bytes(K); }

int nf4_int8_quantize(const void* x, int dtype, int64_t stride, int64_t M, int64_t K, int8_t* q, float* scale, void* stream) {
  if (!is_float(dtype)) return NF4_ERR_DTYPE;
  if (M < 0 || K < 0 || stride < 0) return NF4_ERR_SHAPE;
  if (K > 130944 || M > 1 << 28 || !launchable(M, 256)) return NF4_ERR_UNSUPPORTED;
  if (!aligned(x, size_of(dtype)) || !aligned(q, 16) || !aligned(scale, 4)) return NF4_ERR_ALIGN;
  if (M == 0) return NF4_OK;
  if (!scale || (K > 0 && (!x || !q))) return NF4_ERR_NULL;
  const hipError_t e = launch_int8_quantize(x, dtype == NF4_DTYPE_BF16, stride, M, K, q, scale, static_cast<hipStream_t>(stream));
  if (e == hipSuccess) count_path(NF4_PATH_INT8_QUANTIZE);
  return to_status(e);
}

size_t nf4_int8_workspace(int x_dtype, int64_t x_rows, int64_t M, int64_t N, int64_t K, int32_t E) {
  Int8Plan pl;
  return check_int8(x_dtype, x_rows, M, N, K, E, pl) ? SIZE_MAX : pl.bytes;
}

int nf4_int8_matmul(const void* x, int x_dtype, int64_t stride, const float* x_scale, int64_t M, const int8_t* q,
                    const float* scale, int64_t N, int64_t K, const float* bias, void* y, int y_dtype, void* ws, size_t ws_bytes,
                    void* stream) {
  const int st = int8_product(x, x_dtype, stride, x_scale, M, nullptr, nullptr, 0, M, q, scale, N, K, bias, y, y_dtype, 0, ws,
                              ws_bytes, stream);
  if (st == NF4_OK && M > 0 && N > 0) count_path(NF4_PATH_INT8_MATMUL);
  return st;
}

int nf4_int8_grouped_matmul(const void* x, int x_dtype, int64_t stride, const float* x_scale, int64_t x_rows,
                            const int32_t* tokens, const int32_t* offsets, int32_t E, int64_t total_M, const int8_t* q,
                            const float* scale, int64_t N, int64_t K, void* y, int y_dtype, int fill_outside, void* ws,
                            size_t ws_bytes, void* stream) {
  if (E < 1) return NF4_ERR_SHAPE;
  if (!offsets) return NF4_ERR_NULL;
  if (!tokens && x_rows != total_M) return NF4_ERR_SHAPE;
  if (tokens && x_rows == 0 && total_M > 0) return NF4_ERR_SHAPE;
  const int st = int8_product(x, x_dtype, stride, x_scale, x_rows, tokens, offsets, E, total_M, q, scale, N, K, nullptr, y, y_dtype,
                              fill_outside, ws, ws_bytes, stream);
  if (st == NF4_OK && total_M > 0 && N > 0) count_path(NF4_PATH_INT8_GROUPED);
  return st;
}

}  // extern "C"
