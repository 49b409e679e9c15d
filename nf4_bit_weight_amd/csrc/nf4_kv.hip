// Paged key/value cache in 4 bits: append with position rotation, read back,
// and attention over it (nf4_attn.h).
#include "nf4_attn.hpp"

namespace nf4 {

namespace {

constexpr float kDeadBlock = 7.52316384526264e-37f;   // 2^-120

struct Place {
  int seq, pos;         // seq < 0: the row is outside every sequence
  int64_t slot;         // page * page size + place, < 0: a hole
};

// Where row t lies in the cache (t is the same in the whole wave).
__device__ __forceinline__ Place place_of(const KVSeqs& s, const KVCache& c, int t) {
  Place p{seq_of(s.offsets, s.B, s.T, t), 0, -1};
  if (p.seq < 0) return p;
  const int end = s.offsets ? s.offsets[p.seq + 1] : t + 1;
  p.pos = s.lengths[p.seq] - end + t;
  const int i = p.pos / c.page;
  if (p.pos >= 0 && i < s.width) {
    const int64_t pg = s.table[static_cast<int64_t>(p.seq) * s.width + i];
    if (pg >= 0 && pg < c.P) p.slot = pg * c.page + p.pos % c.page;
  }
  return p;
}

// Index of (slot, head) among the cache's vectors of D elements.
__device__ __forceinline__ int64_t vec_of(const KVCache& c, int64_t slot, int h) {
  const int64_t pg = slot / c.page;
  return (pg * c.Hkv + h) * c.page + (slot - pg * c.page);
}

// ---- append ----------------------------------------------------------------
// One workgroup takes `tt` consecutive rows and every `gridDim.y`-th head.  The
// sines and cosines of its rows are computed once in 64 bits into LDS and
// shared by all heads; a thread then turns 8 neighbouring elements, reading
// their partners a second time (from cache), and the 8 threads of a block of
// 64 agree on its largest magnitude.  Bound by memory: 2 bytes in per element
// and 0.5 to 2.5 out.
constexpr int kAppendRows = 16;

__global__ __launch_bounds__(256) void k_kv_append(KVCache c, KVSeqs s, AppendArgs a, int tt) {
  __shared__ double2 turn[kAppendRows * 64];
  __shared__ int64_t slots[kAppendRows];
  __shared__ int seqs[kAppendRows];
  const int D = c.D, D8 = D / 8, half = a.half;
  const int t0 = blockIdx.x * tt, rows = min(tt, s.T - t0);
  for (int r = threadIdx.x >> 6; r < rows; r += 4) {
    const Place p = place_of(s, c, t0 + r);
    const int lane = threadIdx.x & 63;
    if (lane == 0) {
      slots[r] = p.slot;
      seqs[r] = p.seq;
    }
    if (p.seq >= 0 && lane < half) {
      double sn, cs;
      sincos(static_cast<double>(p.pos) * static_cast<double>(a.inv_freq[lane]), &sn, &cs);
      turn[r * 64 + lane] = make_double2(cs, sn);
    }
  }
  __syncthreads();
  const int heads = (a.q ? a.Hq : 0) + 2 * c.Hkv, first_k = a.q ? a.Hq : 0;
  const int per_head = rows * D8;
  const int step = 256 * gridDim.y;
  const int total = heads * per_head;                       // a multiple of 8
  for (int i = blockIdx.y * 256 + threadIdx.x; i < total; i += step) {
    const int hd = i / per_head, j = i - hd * per_head;
    const int r = j / D8, e = 8 * (j - r * D8);
    const int64_t t = t0 + r;
    const bool is_q = hd < first_k, is_v = hd >= first_k + c.Hkv;
    const int h = is_q ? hd : is_v ? hd - first_k - c.Hkv : hd - first_k;
    uint16_t* dst = is_q ? a.q_out + (t * a.Hq + h) * D + e
                         : (!is_v && a.k_out) ? a.k_out + (t * c.Hkv + h) * D + e : nullptr;
    if (seqs[r] < 0) {
      if (dst && a.fill) *reinterpret_cast<uint4*>(dst) = make_uint4(0u, 0u, 0u, 0u);
      continue;
    }
    const uint16_t* src = is_q ? a.q + t * a.q_stride + h * D
                               : is_v ? a.v + t * a.v_stride + h * D : a.k + t * a.k_stride + h * D;
    uint4 w = *reinterpret_cast<const uint4*>(src + e);
    uint32_t x[4] = {w.x, w.y, w.z, w.w};
    if (!is_v && e < 2 * half) {
      if (a.interleaved) {
#pragma unroll
        for (int p = 0; p < 4; ++p) {
          const double2 cs = turn[r * 64 + e / 2 + p];
          const double u = static_cast<double>(__builtin_bit_cast(float, x[p] << 16));
          const double y = static_cast<double>(__builtin_bit_cast(float, x[p] & 0xFFFF0000u));
          x[p] = pack_bf16x2(static_cast<float>(u * cs.x - y * cs.y), static_cast<float>(y * cs.x + u * cs.y));
        }
      } else {
        const bool low = e < half;
        const uint4 wo = *reinterpret_cast<const uint4*>(src + (low ? e + half : e - half));
        const uint32_t o[4] = {wo.x, wo.y, wo.z, wo.w};
        const int f = low ? e : e - half;
        float z[8];
#pragma unroll
        for (int p = 0; p < 8; ++p) {
          const double2 cs = turn[r * 64 + f + p];
          const uint32_t mi = p & 1 ? x[p / 2] & 0xFFFF0000u : x[p / 2] << 16;
          const uint32_t ot = p & 1 ? o[p / 2] & 0xFFFF0000u : o[p / 2] << 16;
          const double m = static_cast<double>(__builtin_bit_cast(float, mi)) * cs.x;
          const double n = static_cast<double>(__builtin_bit_cast(float, ot)) * cs.y;
          z[p] = static_cast<float>(low ? m - n : m + n);
        }
#pragma unroll
        for (int p = 0; p < 4; ++p) x[p] = pack_bf16x2(z[2 * p], z[2 * p + 1]);
      }
    }
    if (dst) *reinterpret_cast<uint4*>(dst) = make_uint4(x[0], x[1], x[2], x[3]);
    if (is_q) continue;
    // the largest magnitude of the block, as bit patterns: they order like the
    // values, and a NaN or infinity (0x7F80 and up) comes out on top
    uint32_t top = 0;
#pragma unroll
    for (int p = 0; p < 4; ++p) {
      top = max(top, x[p] & 0x7FFFu);
      top = max(top, (x[p] >> 16) & 0x7FFFu);
    }
#pragma unroll
    for (int d = 1; d < 8; d *= 2) top = max(top, static_cast<uint32_t>(__shfl_xor(static_cast<int>(top), d)));
    if (slots[r] < 0) continue;
    const float amax = __builtin_bit_cast(float, top << 16);
    const bool bad = top >= 0x7F80u, dead = amax < kDeadBlock;
    const float sc = bad ? __builtin_bit_cast(float, 0x7FC00000u) : dead ? 0.0f : amax / 6.0f;
    uint32_t code = 0;
    if (!bad && !dead) {
      // 6 x / top against the levels.  Both are 8-bit numbers, so a quotient
      // that is not exactly half-way between two levels is at least 2^-11 away
      // from it; the 2^-16 on top moves exact halves outwards and nothing else.
      const float m = (6.0f / amax) * 1.0000152587890625f;
#pragma unroll
      for (int p = 0; p < 4; ++p) {
        const float u = __builtin_bit_cast(float, x[p] << 16) * m;
        const float y = __builtin_bit_cast(float, x[p] & 0xFFFF0000u) * m;
        // the first element goes to the high half of the byte
        switch (p) {
          case 0: code = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(code, y, u, 1.0f, 0); break;
          case 1: code = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(code, y, u, 1.0f, 1); break;
          case 2: code = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(code, y, u, 1.0f, 2); break;
          default: code = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(code, y, u, 1.0f, 3); break;
        }
      }
    }
    const int64_t vec = vec_of(c, slots[r], h);
    *reinterpret_cast<uint32_t*>((is_v ? c.v_codes : c.k_codes) + vec * (D / 2) + e / 2) = code;
    if ((e & 63) == 0) (is_v ? c.v_scale : c.k_scale)[vec * (D / 64) + e / 64] = sc;
  }
}

// ---- read back ---------------------------------------------------------------
// 8 elements a thread: one dword of patterns, four hardware conversions.
__global__ __launch_bounds__(256) void k_kv_dequantize(KVCache c, KVSeqs s, uint16_t* k_out, uint16_t* v_out, int fill,
                                                       int tt) {
  __shared__ int64_t slots[kAppendRows];
  __shared__ int seqs[kAppendRows];
  const int D = c.D, D8 = D / 8;
  const int t0 = blockIdx.x * tt, rows = min(tt, s.T - t0);
  for (int r = threadIdx.x >> 6; r < rows; r += 4) {
    const Place p = place_of(s, c, t0 + r);
    if ((threadIdx.x & 63) == 0) {
      slots[r] = p.slot;
      seqs[r] = p.seq;
    }
  }
  __syncthreads();
  const int per_head = rows * D8, total = 2 * c.Hkv * per_head;
  for (int i = blockIdx.y * 256 + threadIdx.x; i < total; i += 256 * gridDim.y) {
    const int hd = i / per_head, j = i - hd * per_head;
    const int r = j / D8, e = 8 * (j - r * D8);
    const bool is_v = hd >= c.Hkv;
    const int h = is_v ? hd - c.Hkv : hd;
    if (seqs[r] < 0 && !fill) continue;
    uint32_t x[4] = {0u, 0u, 0u, 0u};
    if (slots[r] >= 0) {
      const int64_t vec = vec_of(c, slots[r], h);
      const uint32_t code = *reinterpret_cast<const uint32_t*>((is_v ? c.v_codes : c.k_codes) + vec * (D / 2) + e / 2);
      const float sc = (is_v ? c.v_scale : c.k_scale)[vec * (D / 64) + e / 64];
      bf16x2_t l[4] = {__builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(code, 1.0f, 0),
                       __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(code, 1.0f, 1),
                       __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(code, 1.0f, 2),
                       __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(code, 1.0f, 3)};
#pragma unroll
      for (int p = 0; p < 4; ++p)
        x[p] = pack_bf16x2(static_cast<float>(l[p][1]) * sc, static_cast<float>(l[p][0]) * sc);
    }
    uint16_t* dst = (is_v ? v_out : k_out) + ((static_cast<int64_t>(t0) + r) * c.Hkv + h) * D + e;
    *reinterpret_cast<uint4*>(dst) = make_uint4(x[0], x[1], x[2], x[3]);
  }
}

// ---- attention over the cache --------------------------------------------------
// A unit is one sequence's tile of 16 * MT (query row, head) rows on one key
// head.  Scores come as S^T = K Q^T, so that a lane holds scores of ONE row
// (lane & 15) for the tokens 4g .. 4g+3 of a 16-token tile (g = lane >> 4):
// softmax needs two lane exchanges per maximum, and the weights are already in
// the operand layout of O^T = V^T P^T.  Patterns go from memory to registers
// and through the hardware conversion straight into matrix operands; the
// scale of a block multiplies the fp32 partial score (keys) or the weight
// (values), never an element.
constexpr int kStep = 128;           // tokens per workgroup step, 32 a wave

template <int D, int MT>
struct KVPart {                       // one worker's partial result of a unit
  static constexpr int kRows = 16 * MT;
  static constexpr size_t kFloats = static_cast<size_t>(kRows) * D + 2 * kRows;
};

struct SeqInfo {
  int first, n, len, tiles, steps;   // tiles of rows; steps per (tile, head)
};

template <int MT>
__device__ __forceinline__ SeqInfo seq_info(const KVSeqs& s, int b, int G, int cap) {
  SeqInfo i;
  seq_rows(s.offsets, b, s.T, i.first, i.n);
  i.len = s.lengths[b];
  const int seen = min(max(i.len, 0), cap);
  i.tiles = (i.n * G + 16 * MT - 1) / (16 * MT);
  i.steps = (seen + kStep - 1) / kStep;
  return i;
}

// Steps of the whole call, and the steps each worker takes.
template <int MT>
__device__ __forceinline__ void share(const KVSeqs& s, int Hkv, int G, int cap, int workers, int& total, int& per) {
  int sum = 0;
  for (int b0 = 0; b0 < s.B; b0 += 64) {
    const int b = b0 + (threadIdx.x & 63);
    if (b < s.B) {
      const SeqInfo i = seq_info<MT>(s, b, G, cap);
      sum += Hkv * i.tiles * i.steps;
    }
  }
  total = uniform(wave_sum(sum));
  per = max(1, (total + workers - 1) / workers);
}

template <int NB>
struct KVTile {                       // what one wave reads of 32 tokens
  uint2 k[2][NB];
  f32x4_t ks[2][NB];
  uint32_t v[2][NB][4];
  f32x4_t vs[2][NB];
  int ok;                             // bit u: 16-token tile u lies in a page
};

__device__ __forceinline__ bf16x8_t fp4_to_frag(uint32_t c) {
  const uint32_t a = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(c, 1.0f, 0));
  const uint32_t b = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(c, 1.0f, 1));
  const uint32_t d = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(c, 1.0f, 2));
  const uint32_t e = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(c, 1.0f, 3));
  return __builtin_bit_cast(bf16x8_t, u32x4_t{a, b, d, e});
}

template <int D, int MT>
__global__ __launch_bounds__(256) void k_kv_attention(KVCache c, KVSeqs s, const uint16_t* __restrict__ q,
                                                      int64_t q_stride, int Hq, float scale2,
                                                      uint16_t* __restrict__ out, float* __restrict__ ws) {
  constexpr int NB = D / 64, R = 16 * MT;
  __shared__ __align__(16) float lds[2 * (R * D + 2 * R)];
  const int G = Hq / c.Hkv, cap = s.width * c.page;
  const int lane = threadIdx.x & 63, wave = uniform(threadIdx.x >> 6);
  const int r16 = lane & 15, g = lane >> 4;
  int total, per;
  share<MT>(s, c.Hkv, G, cap, gridDim.x, total, per);
  int lo = min(static_cast<int64_t>(total), static_cast<int64_t>(blockIdx.x) * per);
  const int hi = min(total, lo + per);
  if (lo >= hi) return;
  const int begin = lo;

  // the sequence whose steps hold `lo`, and the steps before it
  int b = 0, base = 0;
  for (int b0 = 0; b0 < s.B; b0 += 64) {
    const int bb = b0 + lane;
    int st = 0;
    if (bb < s.B) {
      const SeqInfo i = seq_info<MT>(s, bb, G, cap);
      st = c.Hkv * i.tiles * i.steps;
    }
    const int incl = wave_scan(st);
    const uint64_t hit = __ballot(base + incl > lo);
    if (hit) {
      const int l = __builtin_ctzll(hit);
      b = b0 + l;
      base += __shfl(incl - st, l);
      break;
    }
    base += __shfl(incl, 63);
  }
  b = uniform(b);
  base = uniform(base);

  const uint32_t sel = r16 >= 8 ? 0x07030602u : 0x05010400u;

  while (lo < hi && b < s.B) {
    const SeqInfo si = seq_info<MT>(s, b, G, cap);
    const int n = uniform(si.n), len = uniform(si.len), ns = uniform(si.steps), first = uniform(si.first);
    const int units = c.Hkv * uniform(si.tiles);
    if (lo >= base + units * ns) {                 // nothing (left) of this sequence
      base += units * ns;
      ++b;
      continue;
    }
    const int u = (lo - base) / ns, s0 = lo - base - u * ns, s1 = min(ns, s0 + (hi - lo));
    const int rt = u / c.Hkv, h = u - rt * c.Hkv;
    const int32_t* pt = s.table + static_cast<int64_t>(b) * s.width;
    const int seen = min(max(len, 0), cap);

    // queries: row rt * R + 16 mt + (lane & 15), elements 16 g .. of each block, pairs swapped as the conversion
    // gives them
    bf16x8_t qf[MT][NB][2];
    int lim[MT];                                   // last token the row sees
    int low = seen - 1;                            // last token that every row sees
#pragma unroll
    for (int m = 0; m < MT; ++m) {
      const int row = rt * R + 16 * m + r16, j = row / G;
      const bool have = row < n * G;
      lim[m] = have ? min(len - n + j, seen - 1) : -1;
      const uint16_t* src = q + (first + (have ? j : 0)) * q_stride + (h * G + (have ? row - j * G : 0)) * D + 16 * g;
#pragma unroll
      for (int nb = 0; nb < NB; ++nb)
#pragma unroll
        for (int p = 0; p < 2; ++p) {
          u32x4_t w = *reinterpret_cast<const u32x4_t*>(src + 64 * nb + 8 * p);
#pragma unroll
          for (int x = 0; x < 4; ++x) w[x] = have ? __builtin_amdgcn_alignbit(w[x], w[x], 16) : 0u;
          qf[m][nb][p] = __builtin_bit_cast(bf16x8_t, w);
        }
    }
    // rows are in token order: the first row of the tile sees least
    low = min(low, len - n + rt * R / G);

    float mx[MT], sum[MT];
    f32x4_t acc[MT][NB][4];
#pragma unroll
    for (int m = 0; m < MT; ++m) {
      mx[m] = -INFINITY;
      sum[m] = 0.0f;
#pragma unroll
      for (int nb = 0; nb < NB; ++nb)
#pragma unroll
        for (int x = 0; x < 4; ++x) acc[m][nb][x] = f32x4_t{0.f, 0.f, 0.f, 0.f};
    }

    auto fetch = [&](int step, KVTile<NB>& t) __attribute__((always_inline)) {
      t.ok = 0;
#pragma unroll
      for (int w = 0; w < 2; ++w) {
        const int t0 = step * kStep + 32 * wave + 16 * w;
        int64_t pg = -1;
        if (t0 < seen) pg = pt[t0 / c.page];
        const bool ok = pg >= 0 && pg < c.P;
        t.ok |= static_cast<int>(ok) << w;
        if (!ok) pg = 0;                           // any page: its tokens are not seen
        const int64_t vec = (pg * c.Hkv + h) * c.page + t0 % c.page;
        const uint8_t* kc = c.k_codes + vec * (D / 2) + r16 * (D / 2) + 8 * g;
        const uint8_t* vc = c.v_codes + vec * (D / 2) + (4 * g) * (D / 2) + 4 * (r16 & 7);
        const float* ks = c.k_scale + (vec + 4 * g) * NB;
        const float* vs = c.v_scale + (vec + 4 * g) * NB;
#pragma unroll
        for (int nb = 0; nb < NB; ++nb) {
          t.k[w][nb] = *reinterpret_cast<const uint2*>(kc + 32 * nb);
          t.ks[w][nb] = *reinterpret_cast<const f32x4_t*>(ks + 4 * nb);
          t.vs[w][nb] = *reinterpret_cast<const f32x4_t*>(vs + 4 * nb);
#pragma unroll
          for (int i = 0; i < 4; ++i) t.v[w][nb][i] = *reinterpret_cast<const uint32_t*>(vc + i * (D / 2) + 32 * nb);
        }
      }
    };
    // scale of token 4g + i, block nb: floats [token][block]
    auto scale_of = [](const f32x4_t (&sv)[NB], int i, int nb) __attribute__((always_inline)) {
      return NB == 1 ? sv[0][i] : sv[(2 * i + nb) >> 2][(2 * i + nb) & 3];
    };

    auto step_of = [&](int step, const KVTile<NB>& t) __attribute__((always_inline)) {
      const int t0 = step * kStep + 32 * wave;
      // value patterns -> operands: bytes of 4 tokens together, then the two
      // 16-token tiles' patterns into one byte
      bf16x8_t vf[NB][4];
#pragma unroll
      for (int nb = 0; nb < NB; ++nb) {
        uint32_t y[2][2];
#pragma unroll
        for (int w = 0; w < 2; ++w) {
          const uint32_t a = perm(t.v[w][nb][1], t.v[w][nb][0], sel), d = perm(t.v[w][nb][3], t.v[w][nb][2], sel);
          y[w][0] = perm(d, a, 0x05040100u);
          y[w][1] = perm(d, a, 0x07060302u);
        }
#pragma unroll
        for (int p = 0; p < 2; ++p) {
          vf[nb][2 * p] = fp4_to_frag(bitsel(0x0F0F0F0Fu, y[0][p] >> 4, y[1][p]));
          vf[nb][2 * p + 1] = fp4_to_frag(bitsel(0x0F0F0F0Fu, y[0][p], y[1][p] << 4));
        }
      }
      bf16x8_t kf[2][NB][2];
#pragma unroll
      for (int w = 0; w < 2; ++w)
#pragma unroll
        for (int nb = 0; nb < NB; ++nb) {
          kf[w][nb][0] = fp4_to_frag(t.k[w][nb].x);
          kf[w][nb][1] = fp4_to_frag(t.k[w][nb].y);
        }
      const bool whole = t.ok == 3 && t0 + 31 <= low;
#pragma unroll
      for (int m = 0; m < MT; ++m) {
        float p[2][4];
        float top = -INFINITY;
#pragma unroll
        for (int w = 0; w < 2; ++w) {
          f32x4_t d[NB];
#pragma unroll
          for (int nb = 0; nb < NB; ++nb) {
            d[nb] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(kf[w][nb][0], qf[m][nb][0], f32x4_t{0.f, 0.f, 0.f, 0.f}, 0, 0, 0);
            d[nb] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(kf[w][nb][1], qf[m][nb][1], d[nb], 0, 0, 0);
          }
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            float x = d[0][i] * scale_of(t.ks[w], i, 0);
            if constexpr (NB == 2) x = __builtin_fmaf(d[1][i], scale_of(t.ks[w], i, 1), x);
            p[w][i] = x * scale2;
          }
        }
        if (!whole) {
#pragma unroll
          for (int w = 0; w < 2; ++w)
#pragma unroll
            for (int i = 0; i < 4; ++i)
              p[w][i] = ((t.ok >> w) & 1) && t0 + 16 * w + 4 * g + i <= lim[m] ? p[w][i] : -INFINITY;
        }
#pragma unroll
        for (int w = 0; w < 2; ++w)
#pragma unroll
          for (int i = 0; i < 4; ++i) top = fmaxf(top, p[w][i]);
        top = fmaxf(quad_max(top), mx[m]);
        const float ref = top == -INFINITY ? 0.0f : top;
        if (__any(top != mx[m])) {
          const float f = __builtin_amdgcn_exp2f(mx[m] - ref);
          sum[m] *= f;
#pragma unroll
          for (int nb = 0; nb < NB; ++nb)
#pragma unroll
            for (int x = 0; x < 4; ++x) acc[m][nb][x] *= f;
          mx[m] = top;
        }
        float ps = 0.0f;
#pragma unroll
        for (int w = 0; w < 2; ++w)
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            p[w][i] = __builtin_amdgcn_exp2f(p[w][i] - ref);
            ps += p[w][i];
          }
        sum[m] += ps;                              // this lane's tokens; the lanes of a row are added at the end
#pragma unroll
        for (int nb = 0; nb < NB; ++nb) {
          float x[2][4];
#pragma unroll
          for (int w = 0; w < 2; ++w)
#pragma unroll
            for (int i = 0; i < 4; ++i) {
              x[w][i] = p[w][i] * scale_of(t.vs[w], i, nb);
              // an unseen token's scale may be anything
              if (!whole)
                x[w][i] = ((t.ok >> w) & 1) && t0 + 16 * w + 4 * g + i <= lim[m] ? x[w][i] : 0.0f;
            }
          // rounded to bf16 for the matrix product: half a step of 2^-8 per weight
          const u32x4_t pw = {pack_bf16x2(x[0][0], x[1][0]), pack_bf16x2(x[0][1], x[1][1]),
                              pack_bf16x2(x[0][2], x[1][2]), pack_bf16x2(x[0][3], x[1][3])};
          const bf16x8_t pf = __builtin_bit_cast(bf16x8_t, pw);
#pragma unroll
          for (int x4 = 0; x4 < 4; ++x4)
            acc[m][nb][x4] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(vf[nb][x4], pf, acc[m][nb][x4], 0, 0, 0);
        }
      }
    };

    KVTile<NB> ta;
    for (int st = s0; st < s1; ++st) {
      fetch(st, ta);
      step_of(st, ta);
    }

    // join the four waves through LDS, two at a time
    // a row's 4 accumulators of one group are 4 neighbouring elements:
    // 64 nb + 8 ((4g + i) & 7) + 4 (g >> 1)
    float* const half_acc = lds;                                   // [2][R][D]
    float* const half_ms = lds + 2 * R * D;                        // [2][2][R]
#pragma unroll
    for (int m = 0; m < MT; ++m) sum[m] = quad_sum(sum[m]);
    for (int round = 0; round < 2; ++round) {
      const int senders = round == 0 ? 2 : 1;                      // waves 2, 3 -> 0, 1; then 1 -> 0
      __syncthreads();
      if (wave >= senders && wave < 2 * senders) {
        const int at = wave - senders;
#pragma unroll
        for (int m = 0; m < MT; ++m) {
          const int row = 16 * m + r16;
#pragma unroll
          for (int nb = 0; nb < NB; ++nb)
#pragma unroll
            for (int i = 0; i < 4; ++i) {
              const int e = 64 * nb + 8 * ((4 * g + i) & 7) + 4 * (g >> 1);
              *reinterpret_cast<f32x4_t*>(half_acc + (at * R + row) * D + (e ^ (4 * (r16 & 7)))) =
                  f32x4_t{acc[m][nb][0][i], acc[m][nb][1][i], acc[m][nb][2][i], acc[m][nb][3][i]};
            }
          if (g == 0) {
            half_ms[(2 * at) * R + row] = mx[m];
            half_ms[(2 * at + 1) * R + row] = sum[m];
          }
        }
      }
      __syncthreads();
      if (wave < senders) {
#pragma unroll
        for (int m = 0; m < MT; ++m) {
          const int row = 16 * m + r16;
          const float om = half_ms[(2 * wave) * R + row], os = half_ms[(2 * wave + 1) * R + row];
          const float top = fmaxf(mx[m], om), ref = top == -INFINITY ? 0.0f : top;
          const float fa = __builtin_amdgcn_exp2f(mx[m] - ref), fb = __builtin_amdgcn_exp2f(om - ref);
          mx[m] = top;
          sum[m] = sum[m] * fa + os * fb;
#pragma unroll
          for (int nb = 0; nb < NB; ++nb)
#pragma unroll
            for (int i = 0; i < 4; ++i) {
              const int e = 64 * nb + 8 * ((4 * g + i) & 7) + 4 * (g >> 1);
              const f32x4_t o = *reinterpret_cast<const f32x4_t*>(half_acc + (wave * R + row) * D + (e ^ (4 * (r16 & 7))));
#pragma unroll
              for (int x = 0; x < 4; ++x) acc[m][nb][x][i] = acc[m][nb][x][i] * fa + o[x] * fb;
            }
        }
      }
    }
    if (wave == 0) {
      const bool complete = s0 == 0 && s1 == ns;
      if (complete) {
#pragma unroll
        for (int m = 0; m < MT; ++m) {
          const int row = rt * R + 16 * m + r16, j = row / G;
          if (row >= n * G) continue;
          const float f = sum[m] == 0.0f ? 0.0f : 1.0f / sum[m];
          uint16_t* dst = out + ((static_cast<int64_t>(first) + j) * Hq + h * G + (row - j * G)) * D;
#pragma unroll
          for (int nb = 0; nb < NB; ++nb)
#pragma unroll
            for (int i = 0; i < 4; ++i) {
              const int e = 64 * nb + 8 * ((4 * g + i) & 7) + 4 * (g >> 1);
              *reinterpret_cast<uint2*>(dst + e) = make_uint2(pack_bf16x2(acc[m][nb][0][i] * f, acc[m][nb][1][i] * f),
                                                              pack_bf16x2(acc[m][nb][2][i] * f, acc[m][nb][3][i] * f));
            }
        }
      } else {
        float* part = ws + (2 * static_cast<size_t>(blockIdx.x) + (lo == begin ? 0 : 1)) * KVPart<D, MT>::kFloats;
#pragma unroll
        for (int m = 0; m < MT; ++m) {
          const int row = 16 * m + r16;
          if (rt * R + row >= n * G) continue;
          if (g == 0) {
            part[R * D + row] = mx[m];
            part[R * D + R + row] = sum[m];
          }
#pragma unroll
          for (int nb = 0; nb < NB; ++nb)
#pragma unroll
            for (int i = 0; i < 4; ++i) {
              const int e = 64 * nb + 8 * ((4 * g + i) & 7) + 4 * (g >> 1);
              *reinterpret_cast<f32x4_t*>(part + row * D + e) =
                  f32x4_t{acc[m][nb][0][i], acc[m][nb][1][i], acc[m][nb][2][i], acc[m][nb][3][i]};
            }
        }
      }
    }
    lo += s1 - s0;
  }
}

// Joins the partial results of a unit that several workers shared, in the
// workers' order; rows that see no key and rows outside every sequence are
// written here too.  One workgroup per (row, query head).
template <int D, int MT>
__global__ __launch_bounds__(256) void k_kv_join(KVCache c, KVSeqs s, int Hq, uint16_t* __restrict__ out,
                                                 const float* __restrict__ ws, int workers, int fill) {
  constexpr int R = 16 * MT, LP = D / 4, NG = 256 / LP;     // lanes per row, groups of workers
  __shared__ float red[NG][D + 4];
  const int G = Hq / c.Hkv, cap = s.width * c.page, t = blockIdx.x, hq = blockIdx.y;
  uint16_t* dst = out + (static_cast<int64_t>(t) * Hq + hq) * D;
  const int lane = threadIdx.x & 63;
  const int bb = uniform(seq_of(s.offsets, s.B, s.T, t));
  if (bb < 0) {
    if (fill && threadIdx.x < D / 2) reinterpret_cast<uint32_t*>(dst)[threadIdx.x] = 0u;
    return;
  }
  int total, per;
  share<MT>(s, c.Hkv, G, cap, workers, total, per);
  int before = 0;
  for (int b = lane; b < bb; b += 64) {
    const SeqInfo i = seq_info<MT>(s, b, G, cap);
    before += c.Hkv * i.tiles * i.steps;
  }
  before = uniform(wave_sum(before));
  const SeqInfo si = seq_info<MT>(s, bb, G, cap);
  if (si.steps == 0) {
    if (threadIdx.x < D / 2) reinterpret_cast<uint32_t*>(dst)[threadIdx.x] = 0u;
    return;
  }
  const int h = hq / G, row = (t - si.first) * G + (hq - h * G), rt = row / R, rr = row - rt * R;
  const int u0 = before + (rt * c.Hkv + h) * si.steps;
  const int w0 = u0 / per, w1 = (u0 + si.steps - 1) / per;
  if (w0 == w1) return;                                      // one worker wrote the result
  const int grp = threadIdx.x / LP, e = 4 * (threadIdx.x % LP);
  float m = -INFINITY, l = 0.0f;
  f32x4_t a = {0.f, 0.f, 0.f, 0.f};
  for (int w = w0 + grp; w <= w1; w += NG) {
    const float* part = ws + (2 * static_cast<size_t>(w) + (w * per >= u0 ? 0 : 1)) * KVPart<D, MT>::kFloats;
    const float om = part[R * D + rr], os = part[R * D + R + rr];
    const f32x4_t o = *reinterpret_cast<const f32x4_t*>(part + rr * D + e);
    const float top = fmaxf(m, om), ref = top == -INFINITY ? 0.0f : top;
    const float fa = __builtin_amdgcn_exp2f(m - ref), fb = __builtin_amdgcn_exp2f(om - ref);
    m = top;
    l = l * fa + os * fb;
#pragma unroll
    for (int x = 0; x < 4; ++x) a[x] = a[x] * fa + o[x] * fb;
  }
  *reinterpret_cast<f32x4_t*>(&red[grp][e]) = a;
  if (e == 0) {
    red[grp][D] = m;
    red[grp][D + 1] = l;
  }
  __syncthreads();
  if (threadIdx.x >= LP) return;
  m = red[0][D];
  l = red[0][D + 1];
  for (int k = 1; k < NG; ++k) {
    const float om = red[k][D], os = red[k][D + 1];
    const f32x4_t o = *reinterpret_cast<const f32x4_t*>(&red[k][e]);
    const float top = fmaxf(m, om), ref = top == -INFINITY ? 0.0f : top;
    const float fa = __builtin_amdgcn_exp2f(m - ref), fb = __builtin_amdgcn_exp2f(om - ref);
    m = top;
    l = l * fa + os * fb;
#pragma unroll
    for (int x = 0; x < 4; ++x) a[x] = a[x] * fa + o[x] * fb;
  }
  const float f = l == 0.0f ? 0.0f : 1.0f / l;
  *reinterpret_cast<uint2*>(dst + e) = make_uint2(pack_bf16x2(a[0] * f, a[1] * f), pack_bf16x2(a[2] * f, a[3] * f));
}

template <int D, int MT>
hipError_t attend(const KVAttnPlan& pl, const KVCache& c, const KVSeqs& s, const void* q, int64_t q_stride, int32_t Hq,
                  float scale, void* out, int fill, void* ws, hipStream_t stream) {
  // scores in units of log2: exp(x) = exp2(x log2 e)
  const float scale2 = scale * 1.44269504088896340736f;
  k_kv_attention<D, MT><<<pl.workers, 256, 0, stream>>>(c, s, static_cast<const uint16_t*>(q), q_stride, Hq, scale2,
                                                        static_cast<uint16_t*>(out), static_cast<float*>(ws));
  hipError_t e = hipGetLastError();
  if (e != hipSuccess) return e;
  k_kv_join<D, MT><<<dim3(s.T, Hq), 256, 0, stream>>>(c, s, Hq, static_cast<uint16_t*>(out),
                                                      static_cast<const float*>(ws), pl.workers, fill);
  return hipGetLastError();
}

}  // namespace

hipError_t launch_kv_append(const KVCache& c, const KVSeqs& s, const AppendArgs& a, hipStream_t stream) {
  const int tt = s.T >= 4096 ? kAppendRows : s.T >= 1024 ? 4 : 1;
  const int64_t items = static_cast<int64_t>((a.q ? a.Hq : 0) + 2 * c.Hkv) * tt * (c.D / 8);
  const int split = tt == 1 ? static_cast<int>((items + 255) / 256) : 1;
  k_kv_append<<<dim3((s.T + tt - 1) / tt, split), 256, 0, stream>>>(c, s, a, tt);
  return hipGetLastError();
}

hipError_t launch_kv_dequantize(const KVCache& c, const KVSeqs& s, void* k_out, void* v_out, int fill,
                                hipStream_t stream) {
  const int tt = s.T >= 4096 ? kAppendRows : s.T >= 1024 ? 4 : 1;
  const int64_t items = static_cast<int64_t>(2 * c.Hkv) * tt * (c.D / 8);
  const int split = tt == 1 ? static_cast<int>((items + 255) / 256) : 1;
  k_kv_dequantize<<<dim3((s.T + tt - 1) / tt, split), 256, 0, stream>>>(c, s, static_cast<uint16_t*>(k_out),
                                                                        static_cast<uint16_t*>(v_out), fill, tt);
  return hipGetLastError();
}

KVAttnPlan plan_kv_attention(int64_t T, int32_t B, int32_t Hq, int32_t Hkv, int32_t D, int cus) {
  KVAttnPlan pl;
  const int64_t G = Hq / Hkv;
  const int64_t mean = B > 0 ? (T * G + B - 1) / B : G;      // rows per sequence and key head
  pl.mt = mean <= 16 ? 1 : mean <= 32 ? 2 : 4;
  pl.workers = 2 * cus;
  pl.ws_bytes = 2 * static_cast<size_t>(pl.workers) * (16 * pl.mt * (D + 2)) * sizeof(float);
  return pl;
}

hipError_t launch_kv_attention(const KVAttnPlan& pl, const KVCache& c, const KVSeqs& s, const void* q, int64_t q_stride,
                               int32_t Hq, float scale, void* out, int fill, void* ws, hipStream_t stream) {
#define NF4_ATTEND(D_, MT_) \
  if (c.D == D_ && pl.mt == MT_) return attend<D_, MT_>(pl, c, s, q, q_stride, Hq, scale, out, fill, ws, stream)
  NF4_ATTEND(64, 1);
  NF4_ATTEND(64, 2);
  NF4_ATTEND(64, 4);
  NF4_ATTEND(128, 1);
  NF4_ATTEND(128, 2);
  NF4_ATTEND(128, 4);
#undef NF4_ATTEND
  return hipErrorInvalidValue;
}

}  // namespace nf4
