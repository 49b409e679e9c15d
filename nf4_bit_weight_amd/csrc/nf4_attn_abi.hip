// extern "C" entry points of nf4_attn.h: argument checks and launches.  No
// entry point allocates, frees or synchronises.
#include <climits>
#include <cmath>

#include "../../include/nf4_attn.h"
#include "nf4_attn.hpp"
#include "nf4_internal.hpp"

namespace nf4 {
namespace {

// Workgroups of the prompt's kernels: one per (128 rows or sequence, head).
int64_t prompt_groups(int64_t T, int32_t B, int32_t heads) { return (T / 128 + B + 1) * heads; }

bool aligned(const void* p, uintptr_t n) { return (reinterpret_cast<uintptr_t>(p) & (n - 1)) == 0; }
int to_status(hipError_t e) { return e == hipSuccess ? NF4_OK : NF4_ERR_HIP; }

// A launch takes fewer than 2^32 threads.
bool launchable(int64_t workgroups, int64_t threads) { return workgroups <= UINT32_MAX / threads; }

// Sizes of T rows in B sequences with Hq query heads on Hkv key heads of D.
int check_heads(int64_t T, int32_t B, int32_t Hq, int32_t Hkv, int32_t D) {
  if (T < 0 || B < 0 || Hq < 1 || Hkv < 1) return NF4_ERR_SHAPE;
  if (Hq % Hkv) return NF4_ERR_SHAPE;
  if (D != 64 && D != 128) return NF4_ERR_UNSUPPORTED;
  if (T > INT32_MAX / 4 || B > INT32_MAX / 4 || Hq > 1024) return NF4_ERR_UNSUPPORTED;
  if (T * Hq > INT32_MAX) return NF4_ERR_UNSUPPORTED;        // (row, head) pairs are counted in 32 bits
  return NF4_OK;
}

// One tensor of T rows with a row stride.
int check_rows(const void* p, int64_t stride, int64_t T) {
  if (T == 0) return NF4_OK;
  if (!p) return NF4_ERR_NULL;
  if (stride < 0) return NF4_ERR_SHAPE;
  if (stride % 8 || !aligned(p, 16)) return NF4_ERR_ALIGN;
  if (stride > 1 << 24) return NF4_ERR_UNSUPPORTED;          // 64 rows lie within 32 bits of bytes
  return NF4_OK;
}

// Positions in a page table are counted in 32 bits.
int check_table(int32_t width, int32_t page) {
  if (width < 0 || page < 1) return NF4_ERR_SHAPE;
  if (page % 16 || static_cast<int64_t>(width) * page > INT32_MAX - 256) return NF4_ERR_UNSUPPORTED;
  return NF4_OK;
}

// Sizes of a cache attention call, and how it is cut.
int check_plan(int64_t T, int32_t B, int32_t Hq, int32_t Hkv, int32_t D, int32_t width, int32_t page, KVAttnPlan& pl) {
  int st = check_heads(T, B, Hq, Hkv, D);
  if (!st) st = check_table(width, page);
  if (st || T == 0) return st;
  pl = plan_kv_attention(T, B, Hq, Hkv, D, static_cast<int64_t>(width) * page, device_cu_count());
  // units and their steps of 128 tokens are counted in 32 bits
  if (pl.steps > INT32_MAX / 2 || !launchable(pl.workers, 256)) return NF4_ERR_UNSUPPORTED;
  if (!pl.solo && !launchable(kv_join_groups(T, Hq), 256)) return NF4_ERR_UNSUPPORTED;
  return NF4_OK;
}

// Sizes of the prompt's calls: grad_k's workgroups are of 512 threads and split
// the heads of a group at most to one each.
int check_prompt(int64_t T, int32_t B, int32_t Hq, int32_t Hkv, int32_t D, int64_t threads) {
  const int st = check_heads(T, B, Hq, Hkv, D);
  return st || T == 0 ? st : launchable(prompt_groups(T, B, Hq), threads) ? NF4_OK : NF4_ERR_UNSUPPORTED;
}

int check_seqs(int64_t T, const int32_t* offsets, const int32_t* lengths, int32_t B, const int32_t* table,
               int32_t width, int32_t page) {
  if (!offsets && T != B) return NF4_ERR_SHAPE;
  if (B > 0 && (!lengths || (width > 0 && !table))) return NF4_ERR_NULL;
  if (!aligned(offsets, 4) || !aligned(lengths, 4) || !aligned(table, 4)) return NF4_ERR_ALIGN;
  return check_table(width, page);
}

int check_cache(const void* kc, const void* ks, const void* vc, const void* vs, int64_t P, int32_t page) {
  if (P < 0 || page < 1) return NF4_ERR_SHAPE;
  if (page % 16) return NF4_ERR_UNSUPPORTED;
  if (P > INT32_MAX) return NF4_ERR_UNSUPPORTED;
  if (P > 0 && (!kc || !ks || !vc || !vs)) return NF4_ERR_NULL;
  if (!aligned(kc, 16) || !aligned(ks, 16) || !aligned(vc, 16) || !aligned(vs, 16)) return NF4_ERR_ALIGN;
  return NF4_OK;
}

}  // namespace
}  // namespace nf4

using namespace nf4;

extern "C" {

int nf4_kv_append(const void* q, int64_t q_stride, const void* k, int64_t k_stride, const void* v, int64_t v_stride,
                  int64_t T, int32_t Hq, const int32_t* offsets, const int32_t* lengths, int32_t B,
                  const int32_t* page_table, int32_t width, const float* inv_freq, int32_t rotary, int interleaved,
                  uint8_t* k_codes, float* k_scale, uint8_t* v_codes, float* v_scale, int64_t P, int32_t page,
                  int32_t Hkv, int32_t D, void* q_out, void* k_out, int fill_outside, void* stream) {
  int st = check_heads(T, B, Hq, Hkv, D);
  if (!st) st = check_cache(k_codes, k_scale, v_codes, v_scale, P, page);
  if (!st) st = check_seqs(T, offsets, lengths, B, page_table, width, page);
  if (!st) st = check_rows(k, k_stride, T);
  if (!st) st = check_rows(v, v_stride, T);
  if (!st && (q || q_out)) st = check_rows(q, q_stride, T);
  if (st) return st;
  if (rotary < 0 || rotary > D) return NF4_ERR_SHAPE;
  if (rotary % 16) return NF4_ERR_UNSUPPORTED;
  if (rotary > 0 && !inv_freq) return NF4_ERR_NULL;
  if (T > 0 && q && !q_out) return NF4_ERR_NULL;
  if (!aligned(q_out, 16) || !aligned(k_out, 16) || !aligned(inv_freq, 4)) return NF4_ERR_ALIGN;
  if (T == 0) return NF4_OK;
  if (!launchable((T + 3) / 4, 256)) return NF4_ERR_UNSUPPORTED;
  const KVCache c{k_codes, k_scale, v_codes, v_scale, P, page, Hkv, D};
  const KVSeqs s{offsets, lengths, page_table, B, width, static_cast<int32_t>(T)};
  const AppendArgs a{static_cast<const uint16_t*>(q), static_cast<const uint16_t*>(k), static_cast<const uint16_t*>(v),
                     q_stride, k_stride, v_stride, static_cast<uint16_t*>(q_out), static_cast<uint16_t*>(k_out),
                     inv_freq, Hq, rotary / 2, interleaved != 0, fill_outside != 0};
  const hipError_t e = launch_kv_append(c, s, a, static_cast<hipStream_t>(stream));
  if (e == hipSuccess) count_path(NF4_PATH_KV_APPEND);
  return to_status(e);
}

int nf4_kv_dequantize(int64_t T, const int32_t* offsets, const int32_t* lengths, int32_t B, const int32_t* page_table,
                      int32_t width, const uint8_t* k_codes, const float* k_scale, const uint8_t* v_codes,
                      const float* v_scale, int64_t P, int32_t page, int32_t Hkv, int32_t D, void* k_out, void* v_out,
                      int fill_outside, void* stream) {
  int st = check_heads(T, B, Hkv, Hkv, D);
  if (!st) st = check_cache(k_codes, k_scale, v_codes, v_scale, P, page);
  if (!st) st = check_seqs(T, offsets, lengths, B, page_table, width, page);
  if (st) return st;
  if (T > 0 && (!k_out || !v_out)) return NF4_ERR_NULL;
  if (!aligned(k_out, 16) || !aligned(v_out, 16)) return NF4_ERR_ALIGN;
  if (T == 0) return NF4_OK;
  if (!launchable((T + 3) / 4, 256)) return NF4_ERR_UNSUPPORTED;
  const KVCache c{const_cast<uint8_t*>(k_codes), const_cast<float*>(k_scale), const_cast<uint8_t*>(v_codes),
                  const_cast<float*>(v_scale), P, page, Hkv, D};
  const KVSeqs s{offsets, lengths, page_table, B, width, static_cast<int32_t>(T)};
  const hipError_t e = launch_kv_dequantize(c, s, k_out, v_out, fill_outside != 0, static_cast<hipStream_t>(stream));
  if (e == hipSuccess) count_path(NF4_PATH_KV_DEQUANTIZE);
  return to_status(e);
}

size_t nf4_kv_attention_workspace(int64_t T, int32_t B, int32_t Hq, int32_t Hkv, int32_t D, int32_t width,
                                  int32_t page) {
  KVAttnPlan pl{};
  return check_plan(T, B, Hq, Hkv, D, width, page, pl) ? SIZE_MAX : pl.ws_bytes;
}

int nf4_kv_attention(const void* q, int64_t q_stride, int64_t T, int32_t Hq, const int32_t* offsets,
                     const int32_t* lengths, int32_t B, const int32_t* page_table, int32_t width,
                     const uint8_t* k_codes, const float* k_scale, const uint8_t* v_codes, const float* v_scale,
                     int64_t P, int32_t page, int32_t Hkv, int32_t D, float scale, void* out, int fill_outside,
                     void* ws, size_t ws_bytes, void* stream) {
  int st = check_heads(T, B, Hq, Hkv, D);
  if (!st) st = check_cache(k_codes, k_scale, v_codes, v_scale, P, page);
  if (!st) st = check_seqs(T, offsets, lengths, B, page_table, width, page);
  if (!st) st = check_rows(q, q_stride, T);
  if (st) return st;
  if (!(scale > 0.0f) || !std::isfinite(scale)) return NF4_ERR_SHAPE;
  if (T > 0 && !out) return NF4_ERR_NULL;
  if (!aligned(out, 16)) return NF4_ERR_ALIGN;
  if (T == 0) return NF4_OK;
  if (P == 0) width = 0;                                     // no pages: no key is seen (and no workspace is needed)
  KVAttnPlan pl{};
  st = check_plan(T, B, Hq, Hkv, D, width, page, pl);
  if (st) return st;
  if (pl.ws_bytes > 0 && (!ws || ws_bytes < pl.ws_bytes)) return NF4_ERR_WORKSPACE;
  if (pl.ws_bytes > 0 && !aligned(ws, 16)) return NF4_ERR_ALIGN;
  const KVCache c{const_cast<uint8_t*>(k_codes), const_cast<float*>(k_scale), const_cast<uint8_t*>(v_codes),
                  const_cast<float*>(v_scale), P, page, Hkv, D};
  const KVSeqs s{offsets, lengths, page_table, B, width, static_cast<int32_t>(T)};
  const hipError_t e = launch_kv_attention(pl, c, s, q, q_stride, Hq, scale, out, fill_outside != 0, ws,
                                           static_cast<hipStream_t>(stream));
  if (e == hipSuccess) count_path(NF4_PATH_KV_ATTENTION);
  return to_status(e);
}

int nf4_prompt_attention_fwd(const void* q, int64_t q_stride, const void* k, int64_t k_stride, const void* v,
                             int64_t v_stride, int64_t T, const int32_t* offsets, int32_t B, int32_t Hq, int32_t Hkv,
                             int32_t D, float scale, void* out, void* out_rest, float* lse, int fill_outside,
                             void* stream) {
  int st = check_prompt(T, B, Hq, Hkv, D, 256);
  if (!st) st = check_rows(q, q_stride, T);
  if (!st) st = check_rows(k, k_stride, T);
  if (!st) st = check_rows(v, v_stride, T);
  if (st) return st;
  if (!(scale > 0.0f) || !std::isfinite(scale)) return NF4_ERR_SHAPE;
  if (!offsets || (T > 0 && !out)) return NF4_ERR_NULL;
  if (!aligned(out, 16) || !aligned(out_rest, 16) || !aligned(lse, 4) || !aligned(offsets, 4)) return NF4_ERR_ALIGN;
  if (T == 0) return NF4_OK;
  const PromptArgs a{static_cast<const uint16_t*>(q), static_cast<const uint16_t*>(k), static_cast<const uint16_t*>(v),
                     q_stride, k_stride, v_stride, offsets, static_cast<int32_t>(T), B, Hq, Hkv, D, scale,
                     fill_outside != 0};
  const hipError_t e = launch_prompt_fwd(a, out, out_rest, lse, static_cast<hipStream_t>(stream));
  if (e == hipSuccess) count_path(NF4_PATH_PROMPT_FWD);
  return to_status(e);
}

size_t nf4_prompt_attention_bwd_workspace(int64_t T, int32_t B, int32_t Hq, int32_t Hkv, int32_t D) {
  if (check_prompt(T, B, Hq, Hkv, D, 512)) return SIZE_MAX;
  return T == 0 ? 0 : prompt_bwd_ws_bytes(T, Hq, Hkv, D);
}

int nf4_prompt_attention_bwd(const void* grad_out, int64_t grad_stride, const void* q, int64_t q_stride, const void* k,
                             int64_t k_stride, const void* v, int64_t v_stride, const void* out, const void* out_rest,
                             const float* lse, int64_t T, const int32_t* offsets, int32_t B, int32_t Hq, int32_t Hkv,
                             int32_t D, float scale, void* grad_q, void* grad_k, void* grad_v, int fill_outside, void* ws,
                             size_t ws_bytes, void* stream) {
  int st = check_prompt(T, B, Hq, Hkv, D, 512);
  if (!st) st = check_rows(grad_out, grad_stride, T);
  if (!st) st = check_rows(q, q_stride, T);
  if (!st) st = check_rows(k, k_stride, T);
  if (!st) st = check_rows(v, v_stride, T);
  if (st) return st;
  if (!(scale > 0.0f) || !std::isfinite(scale)) return NF4_ERR_SHAPE;
  if (!offsets || (T > 0 && (!out || !lse || !grad_q || !grad_k || !grad_v))) return NF4_ERR_NULL;
  if (!aligned(out, 16) || !aligned(out_rest, 16) || !aligned(lse, 4) || !aligned(grad_q, 16) || !aligned(grad_k, 16) || !aligned(grad_v, 16) ||
      !aligned(offsets, 4))
    return NF4_ERR_ALIGN;
  if (T == 0) return NF4_OK;
  if (!ws || ws_bytes < prompt_bwd_ws_bytes(T, Hq, Hkv, D)) return NF4_ERR_WORKSPACE;
  if (!aligned(ws, 16)) return NF4_ERR_ALIGN;
  const PromptArgs a{static_cast<const uint16_t*>(q), static_cast<const uint16_t*>(k), static_cast<const uint16_t*>(v),
                     q_stride, k_stride, v_stride, offsets, static_cast<int32_t>(T), B, Hq, Hkv, D, scale,
                     fill_outside != 0};
  const hipError_t e = launch_prompt_bwd(a, grad_out, grad_stride, out, out_rest, lse, grad_q, grad_k, grad_v, ws,
                                         static_cast<hipStream_t>(stream));
  if (e == hipSuccess) count_path(NF4_PATH_PROMPT_BWD);
  return to_status(e);
}

}  // extern "C"
