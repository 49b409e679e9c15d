// Paged key/value cache in 4 bits: append with position rotation, read back,
// and attention over it (nf4_attn.h).
#include "nf4_attn.hpp"

namespace nf4 {

namespace {

constexpr float kDeadBlock = 7.52316384526264e-37f;   // 2^-120

// Where a row lies in the cache.
struct Place {
  int seq, pos;         // seq < 0: the row is outside every sequence
  int64_t vec;          // (page * Hkv) * page size + place: head h adds h * page size; < 0: a hole
};

// Place of row t (the same t in the whole wave).
__device__ __forceinline__ Place place_of(const KVSeqs& s, const KVCache& c, int t) {
  Place p{seq_of(s.offsets, s.B, s.T, t), 0, -1};
  if (p.seq < 0) return p;
  const int end = s.offsets ? s.offsets[p.seq + 1] : t + 1;
  p.pos = s.lengths[p.seq] - end + t;
  const int i = p.pos / c.page;
  if (p.pos >= 0 && i < s.width) {
    const int64_t pg = s.table[static_cast<int64_t>(p.seq) * s.width + i];
    if (pg >= 0 && pg < c.P) p.vec = pg * c.Hkv * c.page + (p.pos - i * c.page);
  }
  return p;
}

// ---- append ----------------------------------------------------------------
// One workgroup takes TT consecutive rows (and, with TT == 1, 256 * 8 elements
// of them).  The sines and cosines of its rows are computed once in 64 bits into
// LDS; a thread keeps those of its 8 neighbouring elements for all heads, takes
// the elements' partners from another lane, and the 8 threads of a block of 64
// agree on its largest magnitude.  Bound by memory: 2 bytes in per
// element and 0.5 to 2.5 out.
template <int D, int TT>
__global__ __launch_bounds__(256) void k_kv_append(KVCache c, KVSeqs s, AppendArgs a) {
  constexpr int D8 = D / 8, kPer = TT * D8;
  __shared__ double2 turn[TT * 64];
  __shared__ int64_t vecs[TT];
  __shared__ int seqs[TT];
  const int half = a.half, t0 = blockIdx.x * TT, rows = min(TT, s.T - t0);
  for (int r = threadIdx.x >> 6; r < rows; r += 4) {
    const Place p = place_of(s, c, t0 + r);
    const int lane = threadIdx.x & 63;
    if (lane == 0) {
      vecs[r] = p.vec;
      seqs[r] = p.seq;
    }
    if (p.seq >= 0 && lane < half) {
      double sn, cs;
      sincos(static_cast<double>(p.pos) * static_cast<double>(a.inv_freq[lane]), &sn, &cs);
      turn[r * 64 + lane] = make_double2(cs, sn);
    }
  }
  __syncthreads();
  // a thread keeps its row and elements and goes over the heads
  const int j = threadIdx.x % kPer, r = j / D8, e = 8 * (j % D8);
  if (r >= rows) return;
  const int first_k = a.q ? a.Hq : 0, heads = first_k + 2 * c.Hkv, seq = seqs[r];
  const int64_t t = t0 + r, base = vecs[r];
  const bool turned = e < 2 * half, low = e < half;
  const int pair = a.interleaved ? e / 2 : low ? e : e - half;
  double2 cs[8];
  if (turned && seq >= 0) {
#pragma unroll
    for (int p = 0; p < 8; ++p) cs[p] = turn[r * 64 + min(pair + p, 63)];
  }
  constexpr int kHeads = 256 / kPer;
  auto source = [&](int hd) __attribute__((always_inline)) {
    return hd < first_k ? a.q + t * a.q_stride + hd * D
                        : hd < first_k + c.Hkv ? a.k + t * a.k_stride + (hd - first_k) * D
                                               : a.v + t * a.v_stride + (hd - first_k - c.Hkv) * D;
  };
  // kAhead heads are on their way while one is worked on
  constexpr int kAhead = 3;
  const int step = kHeads * gridDim.y, lane = threadIdx.x & 63, partner_lane = lane + (low ? half : -half) / 8;
  const int hd0 = blockIdx.y * kHeads + threadIdx.x / kPer;
  uint4 ring[kAhead];
  auto ask = [&](int i, uint4& to) __attribute__((always_inline)) {
    if (i < heads && seq >= 0) to = *reinterpret_cast<const uint4*>(source(i) + e);
  };
  auto work = [&](int hd, uint4& slot) __attribute__((always_inline)) {
    const bool is_q = hd < first_k, is_v = hd >= first_k + c.Hkv;
    const int h = is_q ? hd : is_v ? hd - first_k - c.Hkv : hd - first_k;
    uint16_t* dst = is_q ? a.q_out + (t * a.Hq + h) * D + e
                         : (!is_v && a.k_out) ? a.k_out + (t * c.Hkv + h) * D + e : nullptr;
    if (seq < 0) {
      if (dst && a.fill) *reinterpret_cast<uint4*>(dst) = make_uint4(0u, 0u, 0u, 0u);
      return;
    }
    uint32_t x[4] = {slot.x, slot.y, slot.z, slot.w};
    ask(hd + kAhead * step, slot);
    uint32_t o[4];
    if (!a.interleaved && half) {                               // the partners' elements lie in other lanes of the row
#pragma unroll
      for (int p = 0; p < 4; ++p) o[p] = __shfl(static_cast<int>(x[p]), partner_lane);
    }
    if (!is_v && turned) {
      if (a.interleaved) {
#pragma unroll
        for (int p = 0; p < 4; ++p) {
          const double u = static_cast<double>(__builtin_bit_cast(float, x[p] << 16));
          const double y = static_cast<double>(__builtin_bit_cast(float, x[p] & 0xFFFF0000u));
          x[p] = pack_bf16x2(static_cast<float>(u * cs[p].x - y * cs[p].y), static_cast<float>(y * cs[p].x + u * cs[p].y));
        }
      } else {
        const uint32_t flip = low ? 0x80000000u : 0u;           // a c - b s below, b c + a s above
        float z[8];
#pragma unroll
        for (int p = 0; p < 8; ++p) {
          const uint32_t mi = p & 1 ? x[p / 2] & 0xFFFF0000u : x[p / 2] << 16;
          const uint32_t ot = (p & 1 ? o[p / 2] & 0xFFFF0000u : o[p / 2] << 16) ^ flip;
          z[p] = static_cast<float>(static_cast<double>(__builtin_bit_cast(float, mi)) * cs[p].x +
                                    static_cast<double>(__builtin_bit_cast(float, ot)) * cs[p].y);
        }
#pragma unroll
        for (int p = 0; p < 4; ++p) x[p] = pack_bf16x2(z[2 * p], z[2 * p + 1]);
      }
    }
    if (dst) *reinterpret_cast<uint4*>(dst) = make_uint4(x[0], x[1], x[2], x[3]);
    if (is_q) return;
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
    if (base < 0) return;
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
    const int64_t vec = base + h * c.page;
    *reinterpret_cast<uint32_t*>((is_v ? c.v_codes : c.k_codes) + vec * (D / 2) + e / 2) = code;
    if ((e & 63) == 0) (is_v ? c.v_scale : c.k_scale)[vec * (D / 64) + e / 64] = sc;
  };
#pragma unroll
  for (int k = 0; k < kAhead; ++k) ask(hd0 + k * step, ring[k]);
  for (int hd = hd0; hd < heads; hd += kAhead * step) {
#pragma unroll
    for (int k = 0; k < kAhead; ++k)
      if (hd + k * step < heads) work(hd + k * step, ring[k]);
  }
}

// ---- read back ---------------------------------------------------------------
// 8 elements a thread: one dword of patterns, four hardware conversions.  Bound
// by memory: 17616 rows of 8 heads in 22 us (92 MB, 4.2 TB/s).
template <int D, int TT>
__global__ __launch_bounds__(256) void k_kv_dequantize(KVCache c, KVSeqs s, uint16_t* k_out, uint16_t* v_out, int fill) {
  constexpr int D8 = D / 8, kPer = TT * D8;
  __shared__ int64_t vecs[TT];
  __shared__ int seqs[TT];
  const int t0 = blockIdx.x * TT, rows = min(TT, s.T - t0);
  for (int r = threadIdx.x >> 6; r < rows; r += 4) {
    const Place p = place_of(s, c, t0 + r);
    if ((threadIdx.x & 63) == 0) {
      vecs[r] = p.vec;
      seqs[r] = p.seq;
    }
  }
  __syncthreads();
  const int total = 2 * c.Hkv * kPer;
  for (int i = blockIdx.y * 256 + threadIdx.x; i < total; i += 256 * gridDim.y) {
    const int hd = i / kPer, r = i % kPer / D8, e = 8 * (i % D8);
    if (r >= rows || (seqs[r] < 0 && !fill)) continue;
    const bool is_v = hd >= c.Hkv;
    const int h = is_v ? hd - c.Hkv : hd;
    uint32_t x[4] = {0u, 0u, 0u, 0u};
    const int64_t base = vecs[r];
    if (base >= 0) {
      const int64_t vec = base + h * c.page;
      const uint32_t code = *reinterpret_cast<const uint32_t*>((is_v ? c.v_codes : c.k_codes) + vec * (D / 2) + e / 2);
      const float sc = (is_v ? c.v_scale : c.k_scale)[vec * (D / 64) + e / 64];
      const bf16x2_t l[4] = {__builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(code, 1.0f, 0),
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
//
// Bound by memory: 4.5 bits an element (72 bytes a vector of 128), read once a
// unit.  131071 tokens, 32 heads on 8: 32 us for 151 MB (4.8 TB/s) and 4.4 us
// for the join; 64 sequences of up to 8192 tokens: 60 us for 302 MB.  About 250
// vector instructions per 32 tokens and wave.
constexpr int kStep = 128;           // tokens per workgroup step, 32 a wave
// Units of at most this many steps are taken whole, without a join.  One
// sequence, 32 heads on 8, whole and shared: 256 tokens 5.8 and 8.1 us, 512
// tokens 7.8 and 8.2, 1024 tokens 11.9 and 8.3.
constexpr int kSoloSteps = 4;
// Workgroups per compute unit that share the steps, all resident at once.  At
// D = 128 two fit: 131071 tokens, 32 heads on 8: 37 us with 2 (the join included),
// 42 with 3, 44 with 4; 64 sequences of up to 8192: 60, 67, 65.  At D = 64 four fit,
// and neither side wins everywhere: 64 such sequences, 64 heads on 8: 45 us with 2,
// 39 with 4; 131071 tokens, 8 heads on 2: 17 and 20.
constexpr int kWorkers = 2;
// Steps that starting and ending a unit counts as where the steps are dealt out
// (a start takes 1.7 us, an end 1.0, a step 1.3).  64 sequences of up to 8192
// tokens: 62 us with 2 and 3, 69 with 1, 73 with 0; 28 of 1081 tokens on 2 heads,
// one step a worker: 11.2 with 2, 10.8 with 0.
constexpr int kUnitCost = 2;
// Rows up to which the join gives each a workgroup (see k_kv_join's launch).
constexpr int64_t kWideRows = 1024;

template <int D, int MT>
struct KVPart {                       // one worker's partial result of a unit
  static constexpr int kRows = 16 * MT;
  static constexpr size_t kFloats = static_cast<size_t>(kRows) * D + 2 * kRows;
};

struct SeqInfo {
  int first, n, len, tiles, steps;   // tiles of rows; steps per (tile, head)
};

// All sequences as the kernels count them.  Lane l holds sequence l, the first
// 64 are read once.  Whole units are dealt out in `solo` calls, steps otherwise.
template <int MT>
struct Seqs {
  const KVSeqs& s;
  int Hkv, G, cap;
  bool solo;
  SeqInfo mine;
  __device__ __forceinline__ Seqs(const KVSeqs& s_, int Hkv_, int G_, int cap_, bool solo_)
      : s(s_), Hkv(Hkv_), G(G_), cap(cap_), solo(solo_) {
    mine = load(threadIdx.x & 63);
  }
  __device__ __forceinline__ SeqInfo load(int b) const {
    SeqInfo i{0, 0, 0, 0, 0};
    if (b < s.B) {
      seq_rows(s.offsets, b, s.T, i.first, i.n);
      i.len = s.lengths[b];
      i.tiles = (i.n * G + 16 * MT - 1) / (16 * MT);
      i.steps = (min(max(i.len, 0), cap) + kStep - 1) / kStep;
    }
    return i;
  }
  // of one unit: its steps come behind kUnitCost that stand for its start and end
  __device__ __forceinline__ int share(const SeqInfo& i) const { return solo ? 1 : i.steps > 0 ? i.steps + kUnitCost : 0; }
  __device__ __forceinline__ int weight(const SeqInfo& i) const { return wrap_mul(Hkv * i.tiles, share(i)); }
  __device__ __forceinline__ SeqInfo of_lane(int b0) const {    // sequence b0 + lane
    return b0 == 0 ? mine : load(b0 + (threadIdx.x & 63));
  }
  __device__ __forceinline__ SeqInfo get(int b) const {         // the same b in the whole wave
    if (b < 64) {
      return SeqInfo{__builtin_amdgcn_readlane(mine.first, b), __builtin_amdgcn_readlane(mine.n, b),
                     __builtin_amdgcn_readlane(mine.len, b), __builtin_amdgcn_readlane(mine.tiles, b),
                     __builtin_amdgcn_readlane(mine.steps, b)};
    }
    const SeqInfo i = load(b);
    return SeqInfo{uniform(i.first), uniform(i.n), uniform(i.len), uniform(i.tiles), uniform(i.steps)};
  }
  // Weight of all sequences and of those before `upto`.
  __device__ __forceinline__ void sums(int upto, int& total, int& before) const {
    int sum = 0, pre = 0;
    for (int b0 = 0; b0 < s.B; b0 += 64) {
      const int w = weight(of_lane(b0));
      sum = wrap_add(sum, w);
      if (b0 + static_cast<int>(threadIdx.x & 63) < upto) pre = wrap_add(pre, w);
    }
    total = wave_sum(sum);
    before = wave_sum(pre);
  }
  // The sequence that holds unit of weight `lo`, and the weight before it.
  __device__ __forceinline__ void find(int lo, int& b, int& base) const {
    b = s.B;
    base = 0;
    for (int b0 = 0; b0 < s.B; b0 += 64) {
      const int w = weight(of_lane(b0)), incl = wave_scan(w);
      const uint64_t hit = __ballot(wrap_add(base, incl) > lo);
      if (hit) {
        const int l = __builtin_ctzll(hit);
        b = b0 + l;
        base = wrap_add(base, __builtin_amdgcn_readlane(wrap_sub(incl, w), l));
        return;
      }
      base = wrap_add(base, __builtin_amdgcn_readlane(incl, 63));
    }
  }
};

// What one wave reads of 32 tokens, in LDS: the patterns of keys and values as
// they lie in their pages ([2 tiles][16 tokens][D / 2]) and the scales ([2][16]
// [D / 64]).  Each wave keeps kRing of these tiles, kRing - 1 on their way
// while it works on one, and copies only for itself: no barriers.
constexpr int kRing = 4;
template <int D>
struct KVTile {
  static constexpr int kCopies = D == 128 ? 6 : 3;              // copy instructions a tile
  uint8_t k[2][16 * D / 2], v[2][16 * D / 2];
  float ks[2][16 * D / 64], vs[2][16 * D / 64];
};

template <int N>
__device__ __forceinline__ void landed() {                     // all but this wave's last N copies
  asm volatile("s_waitcnt vmcnt(%0)" :: "n"(N) : "memory");
}

__device__ __forceinline__ bf16x8_t fp4_to_frag(uint32_t c) {
  const uint32_t a = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(c, 1.0f, 0));
  const uint32_t b = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(c, 1.0f, 1));
  const uint32_t d = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(c, 1.0f, 2));
  const uint32_t e = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(c, 1.0f, 3));
  return __builtin_bit_cast(bf16x8_t, u32x4_t{a, b, d, e});
}

template <int D, int MT>
__global__ __launch_bounds__(256, 2) void k_kv_attention(KVCache c, KVSeqs s, const uint16_t* __restrict__ q,
                                                      int64_t q_stride, int Hq, float scale2,
                                                      uint16_t* __restrict__ out, float* __restrict__ ws, bool solo,
                                                      int fill) {
  constexpr int NB = D / 64, R = 16 * MT, kCopies = KVTile<D>::kCopies;
  // the ring, and between segments the waves' results
  constexpr size_t kRingBytes = 4 * kRing * sizeof(KVTile<D>), kJoinBytes = 4 * (R * D + 2 * R) * sizeof(float);
  __shared__ __align__(1024) char shared[kRingBytes > kJoinBytes ? kRingBytes : kJoinBytes];
  float* const lds = reinterpret_cast<float*>(shared);
  const int G = Hq / c.Hkv, cap = s.width * c.page;
  const int lane = threadIdx.x & 63, wave = uniform(threadIdx.x >> 6);
  const int r16 = lane & 15, g = lane >> 4;
  const Seqs<MT> seqs(s, c.Hkv, G, cap, solo);
  int total, none;
  seqs.sums(0, total, none);
  const Deal deal(max(total, 0), gridDim.x);       // negative only where overlapping offsets overflow the counts
  int lo = deal.begin(blockIdx.x);
  const int hi = deal.begin(blockIdx.x + 1);
  if (solo && fill && s.offsets) {                 // rows outside every sequence: with a join, it writes them
    const int from = min(max(s.offsets[0], 0), s.T), to = min(max(s.offsets[s.B], from), s.T);
    for (int i = blockIdx.x; i < from + s.T - to; i += gridDim.x) {
      uint32_t* row = reinterpret_cast<uint32_t*>(out + static_cast<int64_t>(i < from ? i : to + (i - from)) * Hq * D);
      for (int e = threadIdx.x; e < Hq * D / 2; e += 256) row[e] = 0u;
    }
  }
  if (lo >= hi) return;
  const int begin = lo;

  int b, base;
  seqs.find(lo, b, base);
  const uint32_t sel = r16 >= 8 ? 0x07030602u : 0x05010400u;

  while (lo < hi && b < s.B) {
    const SeqInfo si = seqs.get(b);
    const int n = si.n, len = si.len, first = si.first, weight = seqs.weight(si);
    const int end = wrap_add(base, weight);
    if (lo >= end) {                               // nothing (left) of this sequence
      base = end;
      ++b;
      continue;
    }
    const int ns = si.steps, share = seqs.share(si);
    UnitAt at_unit;
    if (!unit_at(lo, hi, base, c.Hkv * si.tiles, share, at_unit)) return;   // only where overlapping offsets overflow the counts
    const int u = at_unit.u, from = at_unit.from, to = at_unit.to;
    const int s0 = solo ? 0 : max(0, from - kUnitCost), s1 = solo ? ns : to - kUnitCost;
    lo += to - from;
    if (!solo && s0 >= s1) continue;               // none of its steps
    const bool leading = lo - (to - from) == begin;
    const int rt = u / c.Hkv, h = u - rt * c.Hkv;
    // read by the scalar unit: nothing writes the table while the kernel runs
    typedef const __attribute__((address_space(4))) int32_t table_t;
    table_t* pt = (table_t*)(s.table + static_cast<int64_t>(b) * s.width);
    const int seen = min(max(len, 0), cap);
    const float room = headroom(seen);             // the same for all workers of the sequence

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

    // The wave's walk over the page table: index and place in the page of its
    // two 16-token tiles, and the pages read one step ahead of their use.
    KVTile<D>* const ring = reinterpret_cast<KVTile<D>*>(shared) + kRing * wave;
    int pi[2], po[2], ids[2], at = s0 * kStep + 32 * wave;
    const int page_q = kStep / c.page, page_r = kStep - page_q * c.page;
#pragma unroll
    for (int w = 0; w < 2; ++w) {
      pi[w] = (at + 16 * w) / c.page;
      po[w] = at + 16 * w - pi[w] * c.page;
    }
    auto look_up = [&]() __attribute__((always_inline)) {
#pragma unroll
      for (int w = 0; w < 2; ++w) ids[w] = at + 16 * w < seen ? pt[pi[w]] : -1;
    };
    uint32_t oks = 0;                              // bit 2 k + w: tile w of the step k steps back lies in a page
    auto fetch = [&](int slot) __attribute__((always_inline)) {
      oks <<= 2;
      int64_t vec[2];
#pragma unroll
      for (int w = 0; w < 2; ++w) {
        int64_t pg = ids[w];
        const bool ok = pg >= 0 && pg < c.P;
        oks |= static_cast<uint32_t>(ok) << w;
        if (!ok) pg = 0;                           // any page: its tokens are not seen
        vec[w] = (pg * c.Hkv + h) * c.page + po[w];
        pi[w] += page_q;
        po[w] += page_r;
        if (po[w] >= c.page) {
          po[w] -= c.page;
          ++pi[w];
        }
      }
      at += kStep;
      KVTile<D>& t = ring[slot];
      // one row tile a sequence: as a rule nobody else reads this (131071 tokens: 31.6
      // us, 33.8 without the hint; several row tiles lose 1 to 6 % with it).  Where
      // somebody does, the hint costs nothing: 64 sequences over the same 8192 tokens
      // 99.0 us with and without, one of 16 sequences with 33 rows 49.4 and 49.5
      constexpr bool kOnce = MT == 1;
      const uint32_t l16 = 16 * lane;
      const int64_t mine = lane < 32 ? vec[0] : vec[1];
      if constexpr (D == 128) {                    // 16 tokens' patterns are 1024 bytes, their scales 128
#pragma unroll
        for (int w = 0; w < 2; ++w) {
          copy16<kOnce>(l16, reinterpret_cast<const char*>(c.k_codes) + vec[w] * 64, lds_addr(t.k[w]));
          copy16<kOnce>(l16, reinterpret_cast<const char*>(c.v_codes) + vec[w] * 64, lds_addr(t.v[w]));
        }
        copy4<kOnce>(c.k_scale + mine * 2 + (lane & 31), lds_addr(t.ks));
        copy4<kOnce>(c.v_scale + mine * 2 + (lane & 31), lds_addr(t.vs));
      } else {                                     // 512 and 64 bytes
        copy16<kOnce>(c.k_codes + mine * 32 + 16 * (lane & 31), lds_addr(t.k));
        copy16<kOnce>(c.v_codes + mine * 32 + 16 * (lane & 31), lds_addr(t.v));
        const int64_t other = (lane & 16) ? vec[1] : vec[0];
        copy4<kOnce>((lane < 32 ? c.k_scale : c.v_scale) + other + (lane & 15), lds_addr(t.ks));
      }
    };

    auto step_of = [&](int step, int slot, uint32_t ok) __attribute__((always_inline)) {
      const KVTile<D>& t = ring[slot];
      const int t0 = step * kStep + 32 * wave;
      auto scale_of = [](const f32x4_t (&sv)[NB], int i, int nb) __attribute__((always_inline)) {
        return NB == 1 ? sv[0][i] : sv[(2 * i + nb) >> 2][(2 * i + nb) & 3];
      };
      const bool whole = ok == 3 && t0 + 31 <= low;
      float p[MT][2][4];
      {
        bf16x8_t kf[2][NB][2];
        f32x4_t ks[2][NB];                         // scales of tokens 4g .. 4g+3: floats [token][block]
#pragma unroll
        for (int w = 0; w < 2; ++w)
#pragma unroll
          for (int nb = 0; nb < NB; ++nb) {
            const uint2 x = *reinterpret_cast<const uint2*>(&t.k[w][r16 * (D / 2) + 8 * g + 32 * nb]);
            ks[w][nb] = *reinterpret_cast<const f32x4_t*>(&t.ks[w][4 * g * NB + 4 * nb]);
            kf[w][nb][0] = fp4_to_frag(x.x);
            kf[w][nb][1] = fp4_to_frag(x.y);
          }
#pragma unroll
        for (int m = 0; m < MT; ++m)
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
              p[m][w][i] = d[0][i] * scale_of(ks[w], i, 0);
              if constexpr (NB == 2) p[m][w][i] = __builtin_fmaf(d[1][i], scale_of(ks[w], i, 1), p[m][w][i]);
            }
          }
      }
      // keys first, then values: the operands of both at once would not fit
      if constexpr (MT > 1) __builtin_amdgcn_sched_barrier(0);
#pragma unroll
      for (int m = 0; m < MT; ++m) {
        if (!whole) {
#pragma unroll
          for (int w = 0; w < 2; ++w)
#pragma unroll
            for (int i = 0; i < 4; ++i)
              p[m][w][i] = ((ok >> w) & 1) && t0 + 16 * w + 4 * g + i <= lim[m] ? p[m][w][i] : -INFINITY;
        }
        float top = fmaxf(fmaxf(fmaxf(p[m][0][0], p[m][0][1]), p[m][0][2]), fmaxf(fmaxf(p[m][0][3], p[m][1][0]), p[m][1][1]));
        top = __builtin_fmaf(quad_max(fmaxf(fmaxf(top, p[m][1][2]), p[m][1][3])), scale2, room);
        // the maximum in use moves only when a score passes it by 2^kSlack
        if (__any(top > mx[m] + kSlack)) {
          const float to = fmaxf(top, mx[m]), f = to == -INFINITY ? 0.0f : __builtin_amdgcn_exp2f(mx[m] - to);
          sum[m] *= f;
#pragma unroll
          for (int nb = 0; nb < NB; ++nb)
#pragma unroll
            for (int x = 0; x < 4; ++x) acc[m][nb][x] *= f;
          mx[m] = to;
        }
        const float ref = mx[m] == -INFINITY ? 0.0f : mx[m];
        float ps[2] = {0.0f, 0.0f};
#pragma unroll
        for (int w = 0; w < 2; ++w)
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            p[m][w][i] = __builtin_amdgcn_exp2f(__builtin_fmaf(p[m][w][i], scale2, -ref));
            ps[w] += p[m][w][i];
          }
        sum[m] += ps[0] + ps[1];                   // this lane's tokens; the lanes of a row are added at the end
      }
      f32x4_t vs[2][NB];
#pragma unroll
      for (int w = 0; w < 2; ++w)
#pragma unroll
        for (int nb = 0; nb < NB; ++nb) vs[w][nb] = *reinterpret_cast<const f32x4_t*>(&t.vs[w][4 * g * NB + 4 * nb]);
#pragma unroll
      for (int nb = 0; nb < NB; ++nb) {
        // value patterns -> operands: bytes of 4 tokens together, then the two
        // 16-token tiles' patterns into one byte
        bf16x8_t vf[4];
        uint32_t y[2][2];
#pragma unroll
        for (int w = 0; w < 2; ++w) {
          uint32_t x[4];
#pragma unroll
          for (int i = 0; i < 4; ++i)
            x[i] = *reinterpret_cast<const uint32_t*>(&t.v[w][(4 * g + i) * (D / 2) + 4 * (r16 & 7) + 32 * nb]);
          const uint32_t lo4 = perm(x[1], x[0], sel), hi4 = perm(x[3], x[2], sel);
          y[w][0] = perm(hi4, lo4, 0x05040100u);
          y[w][1] = perm(hi4, lo4, 0x07060302u);
        }
#pragma unroll
        for (int b2 = 0; b2 < 2; ++b2) {
          vf[2 * b2] = fp4_to_frag(bitsel(0x0F0F0F0Fu, y[0][b2] >> 4, y[1][b2]));
          vf[2 * b2 + 1] = fp4_to_frag(bitsel(0x0F0F0F0Fu, y[0][b2], y[1][b2] << 4));
        }
#pragma unroll
        for (int m = 0; m < MT; ++m) {
          float x[2][4];
#pragma unroll
          for (int w = 0; w < 2; ++w)
#pragma unroll
            for (int i = 0; i < 4; ++i) x[w][i] = p[m][w][i] * scale_of(vs[w], i, nb);
          if (!whole) {                            // an unseen token's scale may be anything
#pragma unroll
            for (int w = 0; w < 2; ++w)
#pragma unroll
              for (int i = 0; i < 4; ++i)
                x[w][i] = ((ok >> w) & 1) && t0 + 16 * w + 4 * g + i <= lim[m] ? x[w][i] : 0.0f;
          }
          // rounded to bf16 for the matrix product: half a step of 2^-8 per weight
          const u32x4_t pw = {pack_bf16x2(x[0][0], x[1][0]), pack_bf16x2(x[0][1], x[1][1]),
                              pack_bf16x2(x[0][2], x[1][2]), pack_bf16x2(x[0][3], x[1][3])};
          const bf16x8_t pf = __builtin_bit_cast(bf16x8_t, pw);
#pragma unroll
          for (int x4 = 0; x4 < 4; ++x4)
            acc[m][nb][x4] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(vf[x4], pf, acc[m][nb][x4], 0, 0, 0);
        }
      }
    };

    look_up();
    // fill the ring, then one tile in for each one worked on
    for (int k = 0; k < kRing - 1 && s0 + k < s1; ++k) {
      fetch(k);
      look_up();
    }
    for (int st = s0, slot = 0; st < s1; ++st, slot = (slot + 1) % kRing) {
      // the slot that is filled next was read to the end in the last step
      asm volatile("s_waitcnt lgkmcnt(0)" ::: "memory");
      const int left = s1 - 1 - st;                              // tiles behind this one
      if (left >= kRing - 1) {
        fetch((slot + kRing - 1) % kRing);
        look_up();
        landed<(kRing - 1) * kCopies>();
      } else if (left == 2) {
        landed<2 * kCopies>();
      } else if (left == 1) {
        landed<kCopies>();
      } else {
        landed<0>();
      }
      const int back = min(left, kRing - 1);                     // steps fetched behind this one
      const uint32_t ok = (oks >> (2 * back)) & 3;
      if (ok) step_of(st, slot, ok);
    }

    // Join the four waves through LDS: all write, then every thread adds the
    // four values of its elements.  A row's 4 accumulators of one group are 4
    // neighbouring elements, 64 nb + 8 ((4g + i) & 7) + 4 (g >> 1); rows turn
    // their 16-byte chunks against each other's banks.
    __syncthreads();                                               // the ring is read to its end
    float* const ms = lds + 4 * R * D;                             // [wave][maximum, sum][R]
#pragma unroll
    for (int m = 0; m < MT; ++m) {
      const int row = 16 * m + r16;
      const float total_m = quad_sum(sum[m]);
#pragma unroll
      for (int nb = 0; nb < NB; ++nb)
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const int e = 64 * nb + 8 * ((4 * g + i) & 7) + 4 * (g >> 1);
          *reinterpret_cast<f32x4_t*>(lds + (wave * R + row) * D + (e ^ (4 * (r16 & 7)))) =
              f32x4_t{acc[m][nb][0][i], acc[m][nb][1][i], acc[m][nb][2][i], acc[m][nb][3][i]};
        }
      if (g == 0) {
        ms[(2 * wave) * R + row] = mx[m];
        ms[(2 * wave + 1) * R + row] = total_m;
      }
    }
    __syncthreads();
    const bool complete = s0 == 0 && s1 == ns;
    float* const part = ws + (2 * static_cast<size_t>(blockIdx.x) + (leading ? 0 : 1)) * KVPart<D, MT>::kFloats;
#pragma unroll
    for (int k = 0; k < R * D / 1024; ++k) {
      const int idx = k * 256 + threadIdx.x, row = idx / (D / 4), e = 4 * (idx % (D / 4));
      const int all = rt * R + row, j = all / G;
      if (all >= n * G) break;                                     // (rows only grow with k)
      float top = ms[row], f[4], l = 0.0f;
#pragma unroll
      for (int w = 1; w < 4; ++w) top = fmaxf(top, ms[(2 * w) * R + row]);
      const float ref = top == -INFINITY ? 0.0f : top;
      f32x4_t o = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
      for (int w = 0; w < 4; ++w) {
        f[w] = __builtin_amdgcn_exp2f(ms[(2 * w) * R + row] - ref);
        l = __builtin_fmaf(f[w], ms[(2 * w + 1) * R + row], l);
        const f32x4_t x = *reinterpret_cast<const f32x4_t*>(lds + (w * R + row) * D + (e ^ (4 * (row & 7))));
#pragma unroll
        for (int i = 0; i < 4; ++i) o[i] = __builtin_fmaf(f[w], x[i], o[i]);
      }
      if (complete) {
        const float y = l == 0.0f ? 0.0f : 1.0f / l;
        uint16_t* dst = out + ((static_cast<int64_t>(first) + j) * Hq + h * G + (all - j * G)) * D + e;
        *reinterpret_cast<uint2*>(dst) = make_uint2(pack_bf16x2(o[0] * y, o[1] * y), pack_bf16x2(o[2] * y, o[3] * y));
      } else {
        *reinterpret_cast<f32x4_t*>(part + row * D + e) = o;
        if (e == 0) {
          part[R * D + row] = top;
          part[R * D + R + row] = l;
        }
      }
    }
    __syncthreads();                                               // the results are read before the ring is filled again
  }
}

// Joins the partial results of a unit that several workers shared, in the
// workers' order; rows that see no key and rows outside every sequence are
// written here too.  A (row, query head) takes a workgroup where there are few
// of them (with many partial results each), a wave where there are many.
struct Partial {
  float m, l;
  f32x4_t a;
  __device__ __forceinline__ void add(float om, float os, const f32x4_t& o) {
    const float top = fmaxf(m, om), ref = top == -INFINITY ? 0.0f : top;
    const float fa = __builtin_amdgcn_exp2f(m - ref), fb = __builtin_amdgcn_exp2f(om - ref);
    m = top;
    l = l * fa + os * fb;
#pragma unroll
    for (int x = 0; x < 4; ++x) a[x] = a[x] * fa + o[x] * fb;
  }
};

template <int D, int MT, bool WIDE>
__global__ __launch_bounds__(256) void k_kv_join(KVCache c, KVSeqs s, int Hq, uint16_t* __restrict__ out,
                                                 const float* __restrict__ ws, int workers, int fill) {
  constexpr int R = 16 * MT, LP = D / 4, NG = (WIDE ? 256 : 64) / LP;   // lanes per row, groups of workers
  __shared__ float red[WIDE ? NG : 1][D + 4];
  const int G = Hq / c.Hkv, cap = s.width * c.page;
  const int tid = WIDE ? threadIdx.x : threadIdx.x & 63;
  const int64_t item = WIDE ? static_cast<int64_t>(blockIdx.x) : 4 * static_cast<int64_t>(blockIdx.x) + uniform(threadIdx.x >> 6);
  if (item >= static_cast<int64_t>(s.T) * Hq) return;
  const int t = static_cast<int>(item / Hq), hq = static_cast<int>(item - static_cast<int64_t>(t) * Hq);
  uint16_t* dst = out + item * D;
  const int bb = uniform(seq_of(s.offsets, s.B, s.T, t));
  if (bb < 0) {
    if (fill && tid < LP) *reinterpret_cast<uint2*>(dst + 4 * tid) = make_uint2(0u, 0u);
    return;
  }
  const Seqs<MT> seqs(s, c.Hkv, G, cap, false);
  int total, before;
  seqs.sums(bb, total, before);
  const Deal deal(max(total, 0), workers);
  const SeqInfo si = seqs.get(bb);
  if (si.steps == 0) {
    if (tid < LP) *reinterpret_cast<uint2*>(dst + 4 * tid) = make_uint2(0u, 0u);
    return;
  }
  const int h = hq / G, row = (t - si.first) * G + (hq - h * G), rt = row / R, rr = row - rt * R;
  SharedBy by;
  if (!shared_by(rt * c.Hkv + h, seqs.share(si), kUnitCost, before, total, deal, by)) return;   // as in k_kv_attention
  const int u0 = by.u0, w0 = by.w0, w1 = by.w1;
  if (w0 == w1) return;                                      // one worker wrote the result
  const int grp = tid / LP, e = 4 * (tid % LP);
  Partial p{-INFINITY, 0.0f, {0.f, 0.f, 0.f, 0.f}};
  constexpr int kAhead = 8;                                  // partial results asked for at once
  for (int w = w0 + grp; w <= w1; w += kAhead * NG) {
    float om[kAhead], os[kAhead];
    f32x4_t o[kAhead];
#pragma unroll
    for (int k = 0; k < kAhead; ++k) {
      const int wr = min(w + k * NG, w1);                    // the last one again behind the end, unused
      const float* part = ws + (2 * static_cast<size_t>(wr) + (deal.begin(wr) >= u0 ? 0 : 1)) * KVPart<D, MT>::kFloats;
      om[k] = part[R * D + rr];
      os[k] = part[R * D + R + rr];
      o[k] = *reinterpret_cast<const f32x4_t*>(part + rr * D + e);
    }
#pragma unroll
    for (int k = 0; k < kAhead; ++k)
      if (w + k * NG <= w1) p.add(om[k], os[k], o[k]);
  }
  if constexpr (WIDE) {
    *reinterpret_cast<f32x4_t*>(&red[grp][e]) = p.a;
    if (e == 0) {
      red[grp][D] = p.m;
      red[grp][D + 1] = p.l;
    }
    __syncthreads();
    if (grp > 0) return;
    for (int k = 1; k < NG; ++k) p.add(red[k][D], red[k][D + 1], *reinterpret_cast<const f32x4_t*>(&red[k][e]));
  } else {
#pragma unroll
    for (int d = LP; d < 64; d *= 2) {
      // both sides add the lower group's result first, so that they agree
      Partial q{__shfl_xor(p.m, d), __shfl_xor(p.l, d), {}};
#pragma unroll
      for (int x = 0; x < 4; ++x) q.a[x] = __shfl_xor(p.a[x], d);
      if (tid & d) {
        q.add(p.m, p.l, p.a);
        p = q;
      } else {
        p.add(q.m, q.l, q.a);
      }
    }
    if (grp > 0) return;
  }
  const float f = p.l == 0.0f ? 0.0f : 1.0f / p.l;
  *reinterpret_cast<uint2*>(dst + e) = make_uint2(pack_bf16x2(p.a[0] * f, p.a[1] * f), pack_bf16x2(p.a[2] * f, p.a[3] * f));
}

template <int D, int MT>
hipError_t attend(const KVAttnPlan& pl, const KVCache& c, const KVSeqs& s, const void* q, int64_t q_stride, int32_t Hq,
                  float scale, void* out, int fill, void* ws, hipStream_t stream) {
  // scores in units of log2: exp(x) = exp2(x log2 e)
  const float scale2 = scale * 1.44269504088896340736f;
  k_kv_attention<D, MT><<<static_cast<unsigned>(pl.workers), 256, 0, stream>>>(
      c, s, static_cast<const uint16_t*>(q), q_stride, Hq, scale2, static_cast<uint16_t*>(out), static_cast<float*>(ws),
      pl.solo, fill);
  const hipError_t e = hipGetLastError();
  if (e != hipSuccess || pl.solo) return e;
  const unsigned groups = static_cast<unsigned>(kv_join_groups(s.T, Hq));
  uint16_t* o = static_cast<uint16_t*>(out);
  const float* part = static_cast<const float*>(ws);
  // 80 rows of 40 heads, 4 or 5 partial results each: 8.1 us with a workgroup a
  // row, 4.8 with a wave; one row of 32 heads with 64 results: 4.4 with a workgroup
  if (static_cast<int64_t>(s.T) * Hq <= kWideRows)
    k_kv_join<D, MT, true><<<groups, 256, 0, stream>>>(c, s, Hq, o, part, static_cast<int>(pl.workers), fill);
  else
    k_kv_join<D, MT, false><<<groups, 256, 0, stream>>>(c, s, Hq, o, part, static_cast<int>(pl.workers), fill);
  return hipGetLastError();
}

}  // namespace

// Rows per workgroup: 4 share a cache line of scales and one start-up; fewer
// rows than would fill the machine are spread one by one over several
// workgroups.  17616 rows, 32 heads on 8: 102 us with 4, 106 with 8, 123 with 16
// (whose 1101 workgroups end in a nearly empty second round).
int rows_per_group(int64_t T) { return T >= 1024 ? 4 : 1; }

hipError_t launch_kv_append(const KVCache& c, const KVSeqs& s, const AppendArgs& a, hipStream_t stream) {
  const int tt = rows_per_group(s.T);
  const int64_t items = static_cast<int64_t>((a.q ? a.Hq : 0) + 2 * c.Hkv) * (c.D / 8);
  const dim3 grid((s.T + tt - 1) / tt, tt == 1 ? static_cast<unsigned>((items + 255) / 256) : 1);
#define NF4_APPEND(D_, TT_) \
  if (c.D == D_ && tt == TT_) k_kv_append<D_, TT_><<<grid, 256, 0, stream>>>(c, s, a)
  NF4_APPEND(64, 1);
  NF4_APPEND(64, 4);
  NF4_APPEND(128, 1);
  NF4_APPEND(128, 4);
#undef NF4_APPEND
  return hipGetLastError();
}

hipError_t launch_kv_dequantize(const KVCache& c, const KVSeqs& s, void* k_out, void* v_out, int fill,
                                hipStream_t stream) {
  const int tt = rows_per_group(s.T);
  const int64_t items = static_cast<int64_t>(2 * c.Hkv) * (c.D / 8);
  const dim3 grid((s.T + tt - 1) / tt, tt == 1 ? static_cast<unsigned>((items + 255) / 256) : 1);
  uint16_t *k = static_cast<uint16_t*>(k_out), *v = static_cast<uint16_t*>(v_out);
#define NF4_DEQUANTIZE(D_, TT_) \
  if (c.D == D_ && tt == TT_) k_kv_dequantize<D_, TT_><<<grid, 256, 0, stream>>>(c, s, k, v, fill)
  NF4_DEQUANTIZE(64, 1);
  NF4_DEQUANTIZE(64, 4);
  NF4_DEQUANTIZE(128, 1);
  NF4_DEQUANTIZE(128, 4);
#undef NF4_DEQUANTIZE
  return hipGetLastError();
}

int64_t kv_join_groups(int64_t T, int32_t Hq) { return T * Hq <= kWideRows ? T * Hq : (T * Hq + 3) / 4; }

KVAttnPlan plan_kv_attention(int64_t T, int32_t B, int32_t Hq, int32_t Hkv, int32_t D, int64_t tokens, int cus) {
  KVAttnPlan pl;
  const int64_t G = Hq / Hkv;
  const int64_t mean = B > 0 ? (T * G + B - 1) / B : G;      // rows per sequence and key head
  // 32 rows a unit where 16 do not hold a sequence's: 9 rows on 16 sequences of
  // up to 4099 tokens, heads 32 on 8: 63.5 us, with 64 rows a unit (registers for
  // one wave a SIMD only) 73.8
  pl.mt = mean <= 16 ? 1 : 2;
  const int64_t units = (T * G / (16 * pl.mt) + B) * Hkv, steps = (tokens + kStep - 1) / kStep;
  pl.solo = steps <= kSoloSteps;
  pl.workers = pl.solo ? (units > 0 ? units : 1) : kWorkers * cus;   // one even without sequences: rows outside are filled
  pl.steps = steps > 0 && units > INT64_MAX / steps ? INT64_MAX : units * (steps + kUnitCost);
  pl.ws_bytes = pl.solo ? 0 : 2 * static_cast<size_t>(pl.workers) * (16 * pl.mt * (D + 2)) * sizeof(float);
  return pl;
}

hipError_t launch_kv_attention(const KVAttnPlan& pl, const KVCache& c, const KVSeqs& s, const void* q, int64_t q_stride,
                               int32_t Hq, float scale, void* out, int fill, void* ws, hipStream_t stream) {
#define NF4_ATTEND(D_, MT_) \
  if (c.D == D_ && pl.mt == MT_) return attend<D_, MT_>(pl, c, s, q, q_stride, Hq, scale, out, fill, ws, stream)
  NF4_ATTEND(64, 1);
  NF4_ATTEND(64, 2);
  NF4_ATTEND(128, 1);
  NF4_ATTEND(128, 2);
#undef NF4_ATTEND
  return hipErrorInvalidValue;
}

}  // namespace nf4
