// Launch interface and device helpers of the attention kernels (nf4_kv.hip,
// nf4_prompt.hip), between the C ABI of nf4_attn.h and the kernels.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

#include "nf4_deal.hpp"
#include "nf4_device.hpp"

namespace nf4 {

// Paged 4-bit cache (layout in nf4_attn.h).
struct KVCache {
  uint8_t* k_codes;
  float* k_scale;
  uint8_t* v_codes;
  float* v_scale;
  int64_t P;
  int32_t page, Hkv, D;
};

// Which rows belong to which sequence, and where the sequence's tokens lie.
struct KVSeqs {
  const int32_t* offsets;   // NULL: one row per sequence
  const int32_t* lengths;
  const int32_t* table;
  int32_t B, width;
  int32_t T;
};

struct AppendArgs {
  const uint16_t *q, *k, *v;
  int64_t q_stride, k_stride, v_stride;
  uint16_t *q_out, *k_out;
  const float* inv_freq;
  int32_t Hq, half;         // rotary / 2
  int interleaved, fill;
};

struct PromptArgs {
  const uint16_t *q, *k, *v;
  int64_t q_stride, k_stride, v_stride;
  const int32_t* offsets;
  int32_t T, B, Hq, Hkv, D;
  float scale;
  int fill;
};

hipError_t launch_kv_append(const KVCache& c, const KVSeqs& s, const AppendArgs& a, hipStream_t stream);
hipError_t launch_kv_dequantize(const KVCache& c, const KVSeqs& s, void* k_out, void* v_out, int fill,
                                hipStream_t stream);

// How a cache attention call is cut: `workers` workgroups share the steps of
// all (sequence, row tile, key head) units evenly, and a unit that several of
// them share is joined from their partial results by a second kernel; or, in
// a solo call, each of them takes one unit whole.
struct KVAttnPlan {
  int mt;          // row tiles of 16 (query row, head) rows per unit
  bool solo;
  int64_t workers;
  int64_t steps;   // bound on the units times the most steps of one
  size_t ws_bytes;
};
KVAttnPlan plan_kv_attention(int64_t T, int32_t B, int32_t Hq, int32_t Hkv, int32_t D, int64_t tokens, int cus);
int64_t kv_join_groups(int64_t T, int32_t Hq);                 // workgroups of the join
hipError_t launch_kv_attention(const KVAttnPlan& pl, const KVCache& c, const KVSeqs& s, const void* q,
                               int64_t q_stride, int32_t Hq, float scale, void* out, int fill, void* ws,
                               hipStream_t stream);

hipError_t launch_prompt_fwd(const PromptArgs& a, void* out, void* rest, float* lse, hipStream_t stream);
size_t prompt_bwd_ws_bytes(int64_t T, int32_t Hq, int32_t Hkv, int32_t D);
hipError_t launch_prompt_bwd(const PromptArgs& a, const void* grad_out, int64_t grad_stride, const void* out,
                             const void* rest, const float* lse, void* grad_q, void* grad_k, void* grad_v, void* ws,
                             hipStream_t stream);

// ---- device helpers ----------------------------------------------------------

// The softmax of the forward kernels, in units of log2.  The maximum in use
// moves only when a score passes it by kSlack, so that the sums are rarely
// rescaled; weights are then up to 2^kSlack times those of the true maximum.
// It is carried with headroom(n) on top, n the number of tokens that a row may
// see: no weight passes 1 / 2n, and sums over values of any finite size stay
// finite.  A power of two, so no bit of a weight is lost; products of a weight and
// a value that fall below 2^-126 are, together at most n^2 2^-113 in a result.
constexpr float kSlack = 8.0f;
__device__ __forceinline__ float headroom(int n) {
  return kSlack + static_cast<float>(33 - __builtin_clz(static_cast<unsigned>(larger(n, 1))));
}

// Copies straight into LDS, invisible to the compiler's own waits; the kernels
// wait for them themselves.  The LDS address is uniform, lane i lands 16 i
// (4 i) bytes behind it.
typedef __attribute__((address_space(3))) void lds_ptr_t;
// ONCE: non-temporal, for data that no other workgroup reads.
template <bool ONCE = false>
__device__ __forceinline__ void copy16(uint32_t off, const char* base, uint32_t lds) {
  if constexpr (ONCE)
    asm volatile("s_nop 0\n\tglobal_load_lds_dwordx4 %0, %1 nt" :: "v"(off), "s"(base), "{m0}"(lds) : "memory");
  else
    asm volatile("s_nop 0\n\tglobal_load_lds_dwordx4 %0, %1" :: "v"(off), "s"(base), "{m0}"(lds) : "memory");
}
template <bool ONCE = false>
__device__ __forceinline__ void copy16(const void* src, uint32_t lds) {
  if constexpr (ONCE)
    asm volatile("s_nop 0\n\tglobal_load_lds_dwordx4 %0, off nt" :: "v"(src), "{m0}"(lds) : "memory");
  else
    asm volatile("s_nop 0\n\tglobal_load_lds_dwordx4 %0, off" :: "v"(src), "{m0}"(lds) : "memory");
}
template <bool ONCE = false>
__device__ __forceinline__ void copy4(const void* src, uint32_t lds) {
  if constexpr (ONCE)
    asm volatile("s_nop 0\n\tglobal_load_lds_dword %0, off nt" :: "v"(src), "{m0}"(lds) : "memory");
  else
    asm volatile("s_nop 0\n\tglobal_load_lds_dword %0, off" :: "v"(src), "{m0}"(lds) : "memory");
}
__device__ __forceinline__ uint32_t lds_addr(const void* p) {
  return static_cast<uint32_t>(reinterpret_cast<uintptr_t>((const lds_ptr_t*)p));
}

// Sum over the wave (the same in all lanes) and inclusive prefix sum, in the
// vector unit's lane moves: rows of 16 lanes first, then across the rows.
template <int CTRL, int ROWS>
__device__ __forceinline__ int lane_move(int x) {
  return __builtin_amdgcn_update_dpp(0, x, CTRL, ROWS, 0xF, false);
}
__device__ __forceinline__ int wave_scan(int x) {
  x = wrap_add(x, lane_move<0x111, 0xF>(x));   // row_shr:1
  x = wrap_add(x, lane_move<0x112, 0xF>(x));
  x = wrap_add(x, lane_move<0x114, 0xF>(x));
  x = wrap_add(x, lane_move<0x118, 0xF>(x));
  x = wrap_add(x, lane_move<0x142, 0xA>(x));   // row_bcast:15 into rows 1 and 3
  x = wrap_add(x, lane_move<0x143, 0xC>(x));   // row_bcast:31 into rows 2 and 3
  return x;
}
__device__ __forceinline__ int wave_sum(int x) { return __builtin_amdgcn_readlane(wave_scan(x), 63); }

__device__ __forceinline__ int uniform(int x) { return __builtin_amdgcn_readfirstlane(x); }

// x of this lane and of the lane whose number differs in bit 5 (bit 4).  In
// assembly: compiled from the builtin, both results came out as the first.
// The swap needs two wait states behind the write of its operands.
__device__ __forceinline__ f32x2_t swap32(float x) {
  float y = x;
  asm volatile("s_nop 1\n\tv_permlane32_swap_b32 %0, %1" : "+v"(x), "+v"(y));
  return f32x2_t{x, y};
}
// Two dwords of row chunk b and two of chunk b + 1 (8 elements each, their
// first half in the lower 32 lanes, the other in the upper) become four dwords
// of chunk b in the lower lanes and of chunk b + 1 in the upper.
__device__ __forceinline__ void halves(uint32_t (&x)[4]) {
  asm volatile("s_nop 1\n\tv_permlane32_swap_b32 %0, %2\n\tv_permlane32_swap_b32 %1, %3"
               : "+v"(x[0]), "+v"(x[1]), "+v"(x[2]), "+v"(x[3]));
}
__device__ __forceinline__ f32x2_t swap16(float x) {
  float y = x;
  asm volatile("s_nop 1\n\tv_permlane16_swap_b32 %0, %1" : "+v"(x), "+v"(y));
  return f32x2_t{x, y};
}

// max / sum over the two lanes that hold one row of a 32-wide tile
__device__ __forceinline__ float half_max(float x) {
  const f32x2_t a = swap32(x);
  return fmaxf(a[0], a[1]);
}
__device__ __forceinline__ float half_sum(float x) {
  const f32x2_t a = swap32(x);
  return a[0] + a[1];
}
// and over the four lanes that hold one row of a 16-wide tile
__device__ __forceinline__ float quad_max(float x) {
  const f32x2_t a = swap16(half_max(x));
  return fmaxf(a[0], a[1]);
}
__device__ __forceinline__ float quad_sum(float x) {
  const f32x2_t a = swap16(half_sum(x));
  return a[0] + a[1];
}

// The sequence that row t belongs to, or -1 (all lanes of the wave take part
// and t is the same in all of them).
__device__ __forceinline__ int seq_of(const int32_t* offsets, int B, int T, int t) {
  if (!offsets) return t < B ? t : -1;
  int count = 0;
  for (int i = threadIdx.x & 63; i - (int)(threadIdx.x & 63) <= B; i += 64)
    count += __popcll(__ballot(i <= B && offsets[min(i, B)] <= t));
  return owner_of(offsets, B, t, count);
}

}  // namespace nf4
