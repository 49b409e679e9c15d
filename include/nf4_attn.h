/*
 * nf4_attn.h -- C ABI of the attention operators of libnf4.so: a paged
 * key/value cache held in 4 bits, attention over it, and causal attention over
 * packed prompts with its backward pass.  They stand between the quantised
 * projections of nf4.h: bf16 rows come out of nf4_matmul_fwd and go back in.
 *
 * Conventions (memory, streams, errors, status codes) are those of nf4.h: all
 * pointers are device memory of the caller, work is enqueued asynchronously
 * on `stream`, nothing is allocated, freed or retained, an error enqueues
 * nothing.  Reductions run in a fixed order without atomics, so repeated
 * calls on the same inputs give bitwise identical outputs.  Every call can be
 * captured into a HIP graph: lengths, offsets and page tables are read on the
 * device, and the launch depends on the sizes alone.
 *
 * Heads.  q rows are bf16 [T, Hq, D], k and v rows bf16 [T, Hkv, D], D = 64 or
 * 128, Hq a multiple of Hkv; query head i reads key head i / (Hq / Hkv).
 * *_stride is the distance between rows in elements (a multiple of 8, at most
 * 2^24; the heads of one row are contiguous), so slices of a joint projection are taken
 * as they are.  All row pointers are 16-byte aligned.  Written tensors are
 * contiguous and overlap nothing that the call reads.  Calls are refused
 * (NF4_ERR_UNSUPPORTED) above 1024 query heads, 2^31 - 1 (row, query head) pairs
 * or 2^32 - 1 threads in a launch: 2^26 rows appended, 2^24 groups of 4 (row,
 * query head) pairs joined, and for prompts 2^24 (2^23 backward) tiles of 128
 * rows times query heads, each sequence counting one tile more.
 *
 * Sequences.  offsets int32 [B + 1] as in the grouped calls of nf4.h: rows
 * offsets[b] .. offsets[b+1]-1 belong to sequence b, non-decreasing, empty
 * sequences allowed (offsets that decrease, overlap or leave 0 .. T give
 * wrong rows, but no access out of range).  For the cache calls NULL means one
 * row per sequence (T == B).  Rows outside every sequence (padding behind the
 * last one) are left as they were where fill_outside is 0 and written as zeros
 * where it is 1; they are never read.
 *
 * Cache.  P pages of `page` tokens (a multiple of 16):
 *   codes  u8  [P, Hkv, page, D / 2]    two 4-bit patterns a byte, element 2i in
 *                                       the HIGH half (as nf4.h packs its
 *                                       indices)
 *   scale  f32 [P, Hkv, page, D / 64]   one per block of 64 elements
 * The pattern is a float of 1 sign, 2 exponent and 1 mantissa bit: 0, 0.5, 1,
 * 1.5, 2, 3, 4, 6 and their negatives, the levels of nf4.h's fp4 table times
 * 6, in the bit order that this GPU converts in hardware.  Encoding of a
 * block x: top = max |x|, scale = fp32(top / 6), pattern = the level nearest to
 * 6 x / top, half-way outwards (away from zero); a value is level * scale.  A
 * block with top < 2^-120 is kept as zeros (scale 0); one that holds a NaN or
 * an infinity is kept as NaN (scale NaN, patterns 0).
 *
 * Range.  The forward calls keep every softmax weight at or below 1 / 2n, n the
 * tokens that a row may see, so that sums over finite values of any size are
 * finite; what falls below 2^-126 in them is at most n^2 2^-113 in a result.
 *
 * A workspace belongs to one call at a time: calls that may overlap (other
 * streams, graphs replayed side by side) take different ones.
 *
 * Page table int32 [B, width], row b's entry i holding tokens i * page ..
 * of sequence b.  lengths int32 [B] counts the tokens of each sequence WITH the
 * rows of the call: row j of sequence b's n rows sits at position
 * lengths[b] - n + j.  A position below zero or at or beyond width * page, and a
 * page outside 0 .. P-1, is a hole: nothing is written there and no key is
 * seen there.  A query that sees no key gets zeros.  Pages written by one call
 * must belong to one sequence each.
 */
#ifndef NF4_ATTN_H_
#define NF4_ATTN_H_

#include "nf4.h"

#ifdef __cplusplus
extern "C" {
#endif

/*
 * nf4_kv_append -- rotate new queries and keys by their positions and put the
 * keys and values into the cache.
 *   inv_freq   f32 [rotary / 2]; pair i of the first `rotary` elements of a head
 *              turns by position * inv_freq[i].  Pairs are (i, i + rotary / 2),
 *              or (2i, 2i + 1) where interleaved != 0.  rotary is a multiple of
 *              16, at most D; 0 rotates nothing (inv_freq may then be NULL).
 *              The angle, its sine and cosine and the turn are computed in 64
 *              bits, rounded to fp32 and from there to bf16; the cache keeps the
 *              rounded keys.
 *   q, q_out   NULL together: no queries.  q_out bf16 [T, Hq, D].
 *   k_out      NULL, or bf16 [T, Hkv, D]: the rotated keys.
 */
int nf4_kv_append(const void* q, int64_t q_stride, const void* k, int64_t k_stride,
                  const void* v, int64_t v_stride, int64_t T, int32_t Hq,
                  const int32_t* offsets, const int32_t* lengths, int32_t B,
                  const int32_t* page_table, int32_t width,
                  const float* inv_freq, int32_t rotary, int interleaved,
                  uint8_t* k_codes, float* k_scale, uint8_t* v_codes, float* v_scale,
                  int64_t P, int32_t page, int32_t Hkv, int32_t D,
                  void* q_out, void* k_out, int fill_outside, void* stream);

/*
 * nf4_kv_dequantize -- the values the cache stands for, of the last n rows of
 * each sequence, rounded to bf16: k_out, v_out bf16 [T, Hkv, D].  Holes are
 * zeros.
 */
int nf4_kv_dequantize(int64_t T, const int32_t* offsets, const int32_t* lengths, int32_t B,
                      const int32_t* page_table, int32_t width,
                      const uint8_t* k_codes, const float* k_scale,
                      const uint8_t* v_codes, const float* v_scale,
                      int64_t P, int32_t page, int32_t Hkv, int32_t D,
                      void* k_out, void* v_out, int fill_outside, void* stream);

/*
 * nf4_kv_attention -- out[t, i] = sum_s softmax_s(scale q[t, i] . K[s, h]) V[s, h]
 * over the cached tokens s of t's sequence at or before t's own position.  Made
 * for few rows per sequence (decode, checking guessed tokens).  bf16 products
 * with fp32 sums; scores, softmax statistics and sums are fp32; the weights
 * times the value's scale are rounded once to bf16.
 *   ws  nf4_kv_attention_workspace(...) bytes, 16-byte aligned
 */
int nf4_kv_attention(const void* q, int64_t q_stride, int64_t T, int32_t Hq,
                     const int32_t* offsets, const int32_t* lengths, int32_t B,
                     const int32_t* page_table, int32_t width,
                     const uint8_t* k_codes, const float* k_scale,
                     const uint8_t* v_codes, const float* v_scale,
                     int64_t P, int32_t page, int32_t Hkv, int32_t D, float scale,
                     void* out, int fill_outside, void* ws, size_t ws_bytes, void* stream);

/* Workspace bytes of nf4_kv_attention for these sizes on the current device
 * (0 for page tables of at most 512 tokens); SIZE_MAX for sizes it refuses. */
size_t nf4_kv_attention_workspace(int64_t T, int32_t B, int32_t Hq, int32_t Hkv, int32_t D,
                                  int32_t width, int32_t page);

/*
 * nf4_prompt_attention_fwd -- causal attention inside each packed sequence:
 * out[t, i] = sum over s <= t of t's sequence of softmax_s(scale q[t, i] .
 * k[s, h]) v[s, h].  out bf16 [T, Hq, D].  For the backward pass, NULL if not
 * wanted: lse f32 [Hq, T], the natural logarithm of each row's sum of
 * exponentials, and out_rest bf16 [T, Hq, D], what the rounding of out took
 * away.  bf16 products with fp32 sums; the softmax is fp32, its
 * weights are rounded once to bf16.
 */
int nf4_prompt_attention_fwd(const void* q, int64_t q_stride, const void* k, int64_t k_stride,
                             const void* v, int64_t v_stride, int64_t T,
                             const int32_t* offsets, int32_t B, int32_t Hq, int32_t Hkv,
                             int32_t D, float scale, void* out, void* out_rest,
                             float* lse, int fill_outside, void* stream);

/*
 * nf4_prompt_attention_bwd -- grad_q bf16 [T, Hq, D], grad_k and grad_v bf16
 * [T, Hkv, D] (summed over the query heads that share a key head) from
 * grad_out bf16 (row stride grad_stride), the inputs, and out, out_rest and lse of
 * the forward call.  Without out_rest (NULL) grad_out . out is taken from the
 * rounded output, which adds its rounding to grad_q and grad_k.  A NaN or an
 * infinity in a row may reach every gradient of its sequence, and of no other.
 *   ws  nf4_prompt_attention_bwd_workspace(...) bytes, 16-byte aligned
 */
int nf4_prompt_attention_bwd(const void* grad_out, int64_t grad_stride,
                             const void* q, int64_t q_stride, const void* k, int64_t k_stride,
                             const void* v, int64_t v_stride, const void* out,
                             const void* out_rest, const float* lse,
                             int64_t T, const int32_t* offsets, int32_t B, int32_t Hq,
                             int32_t Hkv, int32_t D, float scale,
                             void* grad_q, void* grad_k, void* grad_v,
                             int fill_outside, void* ws, size_t ws_bytes, void* stream);

/* Workspace bytes of nf4_prompt_attention_bwd for these sizes on the current
 * device; SIZE_MAX for sizes it refuses. */
size_t nf4_prompt_attention_bwd_workspace(int64_t T, int32_t B, int32_t Hq, int32_t Hkv, int32_t D);

#ifdef __cplusplus
}  /* extern "C" */
#endif

#endif  /* NF4_ATTN_H_ */
