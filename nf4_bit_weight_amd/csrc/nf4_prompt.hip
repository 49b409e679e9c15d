// Causal attention over packed prompts, forward and backward (nf4_attn.h).
//
// All products run on 32x32x16 bf16 matrix instructions.  Each kernel keeps
// one operand's rows in registers (32 per wave) and streams tiles of 64 rows of
// the other two through LDS.  Scores are always formed with the register rows
// as the COLUMNS of the result, so that a lane holds scores of one register
// row (lane & 31) and, for the second product, the weights are already in operand
// layout: the contraction runs over the streamed rows in the order the first
// product left them (8 j + 4 (lane >> 5) + i), and the streamed tile is read
// transposed in that same order.
#include <type_traits>

#include "nf4_attn.hpp"
#include "nf4_internal.hpp"

namespace nf4 {

namespace {

typedef short s16x4_t __attribute__((ext_vector_type(4)));
typedef __attribute__((address_space(3))) s16x4_t lds_s16x4_t;

constexpr int kTile = 64;       // streamed rows per step
constexpr int kRows = 128;      // register rows per workgroup (32 a wave)
constexpr float kLog2e = 1.44269504088896340736f, kLn2 = 0.69314718055994530942f;

__device__ __forceinline__ void land() {                       // every copy has landed, for every wave
  asm volatile("s_waitcnt vmcnt(0) lgkmcnt(0)" ::: "memory");
  __builtin_amdgcn_s_barrier();
  asm volatile("" ::: "memory");
}

__device__ __forceinline__ void share_lds() {                  // LDS writes are seen by every wave; copies stay in flight
  asm volatile("s_waitcnt lgkmcnt(0)" ::: "memory");
  __builtin_amdgcn_s_barrier();
  asm volatile("" ::: "memory");
}

// LDS tile of 64 rows: [D / 32 slices of 32 elements][64 rows][64 bytes], the 16-byte chunk c of a row's slice at chunk c ^ ((row >> 2) & 3).
// Both reads are free of bank conflicts (16 bytes of 8 neighbouring rows; the
// transposed read's 32 bytes of 8 rows), and slice and row are immediate offsets
// from two lane addresses each.
//
// Copier copies rows row0 .. row0+63 of a sequence of n rows (the last row
// again behind the end; its scores are masked) into such a tile: an
// instruction copies 16 rows of one slice, 4 or 8 waves share the slices.
constexpr int kSlice = kTile * 64;                              // bytes
template <int D, int WAVES = 4>
struct Copier {
  static constexpr int kSlices = D / 32 / (WAVES / 4);          // of one wave
  uint32_t off, stride;                                         // bytes
  int row;
  __device__ __forceinline__ explicit Copier(int64_t stride_elems) {
    const int lane = threadIdx.x & 63;
    row = 16 * (uniform(threadIdx.x >> 6) & 3) + (lane >> 2);
    stride = static_cast<uint32_t>(stride_elems) * 2;
    off = 16 * ((lane & 3) ^ ((row >> 2) & 3));
  }
  __device__ __forceinline__ void operator()(const uint16_t* seq, int row0, int n, const void* tile) const {
    const int wave = uniform(threadIdx.x >> 6), first = WAVES == 4 ? 0 : kSlices * (wave >> 2);
    const char* base = reinterpret_cast<const char*>(seq) + static_cast<int64_t>(row0) * stride + 64 * first;
    const uint32_t lds = lds_addr(tile) + 1024 * (wave & 3) + kSlice * first;
    const uint32_t o = static_cast<uint32_t>(min(row, n - 1 - row0)) * stride + off;
#pragma unroll
    for (int i = 0; i < kSlices; ++i) copy16(o, base + 64 * i, lds + kSlice * i);
  }
};

// Lane addresses (bytes) of the two kinds of reads.
struct Offs {
  int row[2];               // row (lane & 31), chunks 2 ks + h of even and odd ks
  int tr[2];                // transposed: rows 4h + i (+ 8)
  __device__ __forceinline__ Offs() {
    const int lane = threadIdx.x & 63, l32 = lane & 31, h = lane >> 5;
#pragma unroll
    for (int p = 0; p < 2; ++p) row[p] = l32 * 64 + (((2 * p + h) ^ ((l32 >> 2) & 3)) << 4);
#pragma unroll
    for (int hi = 0; hi < 2; ++hi) {
      const int r = 4 * h + ((lane & 15) >> 2) + 8 * hi;
      const int col = 16 * ((lane >> 4) & 1) + 4 * (lane & 3);
      tr[hi] = r * 64 + (((col >> 3) ^ ((r >> 2) & 3)) << 4) + (col & 7) * 2;
    }
  }
};

// elements 16 ks + 8 h .. +7 of row 32 w + (lane & 31)
__device__ __forceinline__ bf16x8_t read_row(const char* tile, const Offs& o, int w, int ks) {
  return *reinterpret_cast<const bf16x8_t*>(tile + (ks >> 1) * kSlice + w * 2048 + o.row[ks & 1]);
}
__device__ __forceinline__ bf16x8_t read_tr_at(const char* lo, const char* hi) {
  const s16x4_t a = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_s16x4_t*)lo);
  const s16x4_t b = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_s16x4_t*)hi);
  const u32x2_t x = __builtin_bit_cast(u32x2_t, a), y = __builtin_bit_cast(u32x2_t, b);
  return __builtin_bit_cast(bf16x8_t, u32x4_t{x[0], x[1], y[0], y[1]});
}
// element 32 dt + (lane & 31) of rows 16 m + 4 h .. +3 and 16 m + 8 + 4 h .. +3
__device__ __forceinline__ bf16x8_t read_tr(const char* tile, const Offs& o, int m, int dt) {
  const char* p = tile + dt * kSlice + m * 1024;
  return read_tr_at(p + o.tr[0], p + o.tr[1]);
}
__device__ __forceinline__ f32x16_t mfma(bf16x8_t a, bf16x8_t b, f32x16_t c) {
  return __builtin_amdgcn_mfma_f32_32x32x16_bf16(a, b, c, 0, 0, 0);
}
__device__ __forceinline__ f32x16_t zero16() {
  f32x16_t z;
#pragma unroll
  for (int i = 0; i < 16; ++i) z[i] = 0.0f;
  return z;
}
// streamed row of result register r (within a 32-row tile), less 4 (lane >> 5)
__device__ __forceinline__ constexpr int reg_row(int r) { return 8 * (r / 4) + r % 4; }

// 8 weights of a 16-row slice, rounded once to bf16 (half a step of 2^-8 each)
__device__ __forceinline__ bf16x8_t pack8(const f32x16_t& p, int m) {
  return __builtin_bit_cast(bf16x8_t, u32x4_t{pack_bf16x2(p[8 * m], p[8 * m + 1]), pack_bf16x2(p[8 * m + 2], p[8 * m + 3]),
                                              pack_bf16x2(p[8 * m + 4], p[8 * m + 5]), pack_bf16x2(p[8 * m + 6], p[8 * m + 7])});
}

// What that rounding took from 8 values, itself rounded: the two together hold
// 16 bits of each.
__device__ __forceinline__ bf16x8_t rest8(const f32x16_t& p, int m, bf16x8_t high) {
  f32x16_t r;
#pragma unroll
  for (int i = 0; i < 8; ++i) r[i] = p[8 * m + i] - static_cast<float>(high[i]);
  return pack8(r, 0);
}

// The tiles of 128 rows of all sequences, heaviest first: a sequence of t tiles
// has one tile of each weight t, t-1, .. 1 (tiles of other rows that it works
// through).  The z-th is found by bisection over the weight w, with
// C(w) = sum_b max(0, t_b - w + 1) tiles of weight w or more.  False behind the
// last tile.
struct TileAt {
  int first, n, weight;
};
__device__ __forceinline__ bool find_tile(const PromptArgs& a, int z, TileAt& at) {
  const int lane = threadIdx.x & 63;
  auto tiles_of = [&](int b, int& f, int& n) __attribute__((always_inline)) {
    f = n = 0;
    if (b < a.B) seq_rows(a.offsets, b, a.T, f, n);
    return (n + kRows - 1) / kRows;
  };
  int f0, n0;
  const int t0 = tiles_of(lane, f0, n0);                        // the first 64 sequences stay in registers
  auto at_least = [&](int w) __attribute__((always_inline)) {
    int c = max(0, t0 - w + 1);
    for (int b = lane + 64; b < a.B; b += 64) {
      int f, n;
      c += max(0, tiles_of(b, f, n) - w + 1);
    }
    return uniform(wave_sum(c));
  };
  int lo = 1, hi = (a.T + kRows - 1) / kRows, above = 0;        // C(lo) > z once found, C(hi + 1) = above <= z
  if (a.B == 1) {
    lo = uniform(__shfl(t0, 0)) - z;
    if (lo < 1) return false;
    above = z;
  } else {
    if (at_least(1) <= z) return false;
    while (lo < hi) {
      const int mid = (lo + hi + 1) / 2, c = at_least(mid);
      if (c > z) {
        lo = mid;
      } else {
        hi = mid - 1;
        above = c;
      }
    }
  }
  int k = z - above;                                            // the k-th sequence with that many tiles
  for (int b0 = 0; b0 < a.B; b0 += 64) {
    int f = f0, n = n0;
    const int t = b0 == 0 ? t0 : tiles_of(b0 + lane, f, n);
    uint64_t has = __ballot(t >= lo);
    const int c = __popcll(has);
    if (k < c) {
      for (; k > 0; --k) has &= has - 1;
      const int l = __builtin_ctzll(has);
      at.first = uniform(__shfl(f, l));
      at.n = uniform(__shfl(n, l));
      at.weight = lo;
      return true;
    }
    k -= c;
  }
  return false;
}

// Rows outside every sequence, written as zeros: row `part` of every `parts`.
__device__ __forceinline__ void fill_rows(const PromptArgs& a, uint16_t* out, int heads, int head, int part, int parts) {
  if (!a.fill) return;
  const int first = min(max(a.offsets[0], 0), a.T), last = min(max(a.offsets[a.B], first), a.T);
  const int outside = first + a.T - last;
  for (int i = part; i < outside; i += parts) {
    const int64_t t = i < first ? i : last + (i - first);
    if (threadIdx.x < a.D / 2) reinterpret_cast<uint32_t*>(out + (t * heads + head) * a.D)[threadIdx.x] = 0u;
  }
}

// This thread's share of an LDS tile, read ahead; take_out then sets its
// elements that are infinite or NaN to zero, and *found if there were any (every
// thread of the workgroup takes part).
template <int D>
struct TileShare {
  static constexpr int kN = kTile * D * 2 / 4096;
  u32x4_t x[kN];
  __device__ __forceinline__ explicit TileShare(const char* tile) {
#pragma unroll
    for (int i = 0; i < kN; ++i) x[i] = reinterpret_cast<const u32x4_t*>(tile)[i * 256 + threadIdx.x];
  }
  __device__ __forceinline__ void take_out(char* tile, int* found) {
    uint32_t most = 0;                                          // largest magnitude: odd elements shifted up, even ones as they are
#pragma unroll
    for (int i = 0; i < kN; ++i)
#pragma unroll
      for (int k = 0; k < 4; ++k) most = max(most, max(x[i][k] & 0x7FFF0000u, x[i][k] << 16 & 0x7FFF0000u));
    if (most >= 0x7F800000u) {
#pragma unroll
      for (int i = 0; i < kN; ++i) {
#pragma unroll
        for (int k = 0; k < 4; ++k) {
          if ((x[i][k] & 0x7F80u) == 0x7F80u) x[i][k] &= 0xFFFF0000u;
          if ((x[i][k] & 0x7F800000u) == 0x7F800000u) x[i][k] &= 0xFFFFu;
        }
        reinterpret_cast<u32x4_t*>(tile)[i * 256 + threadIdx.x] = x[i];
      }
      *found = 1;
    }
    share_lds();
  }
};

// The results of one wave on their way out, 32 rows of D elements through its
// own part of LDS: a lane holds a row's elements in pieces of 4, and 32 rows with
// a piece each keep the memory busy several times as long as 4 whole rows.
// 16 sequences of 512 rows, 32 heads on 8 of 128: forward 74 us, 99 with 8-byte
// pieces; backward 227, 242 with them.
template <int D>
struct RowChunks {
  static constexpr int kChunks = D / 8;                         // of 16 bytes a row
  char* stage;
  __device__ __forceinline__ explicit RowChunks(char* s) : stage(s) {}
  // elements 32 dt + 16 p .. +15 of row (lane & 31): 4 h .. +3 of both halves of 8, two a dword
  __device__ __forceinline__ void put(int dt, int p, uint32_t (&x)[4]) const {
    const int lane = threadIdx.x & 63, row = lane & 31;
    halves(x);                                                  // now 8 neighbouring elements
    *reinterpret_cast<u32x4_t*>(stage + row * D * 2 + (((4 * dt + 2 * p + (lane >> 5)) ^ (row & (kChunks - 1))) << 4)) =
        u32x4_t{x[0], x[1], x[2], x[3]};
  }
  // and the other way: rows w0 .. w0+31 of a sequence of n (the last one again behind its end)
  __device__ __forceinline__ void fetch(const uint16_t* seq, int64_t stride, int w0, int n) const {
    const int top = min(w0, n - 1);
    const char* base = reinterpret_cast<const char*>(seq + top * stride);
#pragma unroll
    for (int i = 0; i < kChunks / 2; ++i) {
      const int at = 64 * i + static_cast<int>(threadIdx.x & 63), row = at / kChunks, ch = (at % kChunks) ^ (row & (kChunks - 1));
      copy16(static_cast<uint32_t>(min(row, n - 1 - top)) * static_cast<uint32_t>(2 * stride) + 16 * ch, base, lds_addr(stage + 1024 * i));
    }
  }
  __device__ __forceinline__ bf16x8_t read(int ks) const {      // elements 16 ks + 8 (lane >> 5) .. +7 of row (lane & 31)
    const int lane = threadIdx.x & 63, row = lane & 31;
    return *reinterpret_cast<const bf16x8_t*>(stage + row * D * 2 + (((2 * ks + (lane >> 5)) ^ (row & (kChunks - 1))) << 4));
  }
  __device__ __forceinline__ void store(uint16_t* dst, int64_t stride, int rows) const {
    __builtin_amdgcn_wave_barrier();
#pragma unroll
    for (int i = 0; i < kChunks / 2; ++i) {
      const int at = 64 * i + static_cast<int>(threadIdx.x & 63), row = at / kChunks, ch = at % kChunks;
      const u32x4_t x = *reinterpret_cast<const u32x4_t*>(stage + row * D * 2 + ((ch ^ (row & (kChunks - 1))) << 4));
      if (row < rows) *reinterpret_cast<u32x4_t*>(dst + row * stride + 8 * ch) = x;
    }
    __builtin_amdgcn_wave_barrier();
  }
};

// Heads of one key head next to each other in one XCD's queue (workgroups go
// round the 8 XCDs in order), so that they share its L2.
__device__ __forceinline__ int head_of(int x, int heads) { return heads % 8 == 0 ? (x % 8) * (heads / 8) + x / 8 : x; }

// ---- forward -------------------------------------------------------------------
// One workgroup: 128 query rows of one head, streaming keys and values.  Bound
// by the matrix and vector units together (a 64-key tile is 1024 cycles of
// products and about 900 of exponentials and sums a wave, two waves a SIMD):
// 8192 rows, 32 heads on 8 of 128: 488 to 548 us by the card, 1003 to 1127 TFLOP/s, where this card's
// library product of 8192 cubed reaches 1240.
template <int D>
__global__ __launch_bounds__(256, 2) void k_prompt_fwd(PromptArgs a, uint16_t* __restrict__ out,
                                                       uint16_t* __restrict__ rest, float* __restrict__ lse, int bound) {
  constexpr int KS = D / 16, DT = D / 32;
  __shared__ __align__(1024) char lds[2][2][kTile * D * 2];     // [buffer][keys, values]
  __shared__ int odd[2];                                        // of the tiles on the diagonal: values that are no numbers
  const int x = blockIdx.x % a.Hq, z = blockIdx.x / a.Hq;
  const int hq = head_of(x, a.Hq), hk = hq / (a.Hq / a.Hkv);
  fill_rows(a, out, a.Hq, hq, z, bound);
  if (rest) fill_rows(a, rest, a.Hq, hq, z, bound);
  TileAt at;
  if (!find_tile(a, z, at)) return;
  const int lane = threadIdx.x & 63, wave = uniform(threadIdx.x >> 6), l32 = lane & 31, h = lane >> 5;
  const int q0 = (at.weight - 1) * kRows, w0 = q0 + 32 * wave, qi = w0 + l32;
  const float c = a.scale * kLog2e;
  const Offs of;
  const Copier<D> ck(a.k_stride), cv(a.v_stride);
  const uint16_t* kb = a.k + at.first * a.k_stride + hk * D;
  const uint16_t* vb = a.v + at.first * a.v_stride + hk * D;
  const int tiles = (min(at.n, q0 + kRows) + kTile - 1) / kTile;
  const int whole = q0 / kTile;                                 // tiles that every row sees whole: an even number
  ck(kb, 0, at.n, lds[0][0]);
  // queries come through the second buffers, as whole rows too
  const RowChunks<D> qs(lds[1][wave >> 1] + (wave & 1) * 32 * D * 2);
  qs.fetch(a.q + at.first * a.q_stride + hq * D, a.q_stride, w0, at.n);
  bf16x8_t qf[KS];
  f32x16_t acc[DT];
#pragma unroll
  for (int dt = 0; dt < DT; ++dt) acc[dt] = zero16();
  const float room = headroom(at.n);
  float ref = -INFINITY, sum[2] = {0.0f, 0.0f};                 // ref: the maximum in use, times c, and room

  auto scores = [&](int j, f32x16_t (&s)[2]) __attribute__((always_inline)) {
    const char* kt = lds[j & 1][0];
    s[0] = zero16();
    s[1] = zero16();
#pragma unroll
    for (int ks = 0; ks < KS; ++ks)
#pragma unroll
      for (int w = 0; w < 2; ++w) s[w] = mfma(read_row(kt, of, w, ks), qf[ks], s[w]);
  };
  auto maximum = [&](const f32x16_t (&s)[2]) __attribute__((always_inline)) {
    float top = s[0][0];
#pragma unroll
    for (int r = 1; r < 31; r += 2) top = fmaxf(fmaxf(top, s[r / 16][r % 16]), s[(r + 1) / 16][(r + 1) % 16]);
    top = __builtin_fmaf(half_max(fmaxf(top, s[1][15])), c, room);
    if (__any(top > ref + kSlack)) {
      const float to = fmaxf(top, ref), f = to == -INFINITY ? 0.0f : __builtin_amdgcn_exp2f(ref - to);
      sum[0] *= f;
      sum[1] *= f;
#pragma unroll
      for (int dt = 0; dt < DT; ++dt)
#pragma unroll
        for (int r = 0; r < 16; ++r) acc[dt][r] *= f;
      ref = to;
    }
  };
  auto weigh = [&](int j, f32x16_t (&s)[2]) __attribute__((always_inline)) {
    const char* vt = lds[j & 1][1];
    const float m = ref == -INFINITY ? 0.0f : ref;
#pragma unroll
    for (int w = 0; w < 2; ++w) {
#pragma unroll
      for (int r = 0; r < 16; ++r) {
        s[w][r] = __builtin_amdgcn_exp2f(__builtin_fmaf(s[w][r], c, -m));
        sum[w] += s[w][r];
      }
#pragma unroll
      for (int mm = 0; mm < 2; ++mm) {
        const bf16x8_t pf = pack8(s[w], mm);
#pragma unroll
        for (int dt = 0; dt < DT; ++dt) acc[dt] = mfma(read_tr(vt, of, 2 * w + mm, dt), pf, acc[dt]);
      }
    }
  };

  // The scores of tile j+1 are formed while the weights of tile j are computed:
  // the two are independent, so matrix and vector instructions of one wave
  // overlap.  Keys therefore run one tile ahead of values.
  auto advance = [&](int j) __attribute__((always_inline)) {
    land();
    if (j + 2 < tiles) ck(kb, (j + 2) * kTile, at.n, lds[j & 1][0]);
    if (j + 1 < tiles) cv(vb, (j + 1) * kTile, at.n, lds[(j + 1) & 1][1]);
  };
  f32x16_t s0[2], s1[2];
  if (threadIdx.x < 2) odd[threadIdx.x] = 0;
  land();
  cv(vb, 0, at.n, lds[0][1]);
#pragma unroll
  for (int ks = 0; ks < KS; ++ks) qf[ks] = qs.read(ks);
  share_lds();
  if (1 < tiles) ck(kb, kTile, at.n, lds[1][0]);
  scores(0, s0);
  for (int j = 0; j < whole; j += 2) {
    advance(j);
    maximum(s0);
    scores(j + 1, s1);
    weigh(j, s0);
    advance(j + 1);
    maximum(s1);
    scores(j + 2, s0);
    weigh(j + 1, s1);
  }
  for (int j = whole; j < tiles; ++j) {                         // at most two, on the diagonal
    advance(j);
    // A value that is no number must not reach the rows before its token
    // through a weight of zero: it is taken out of the tile here and added to
    // the rows that see it below.
    TileShare<D> values(lds[j & 1][1]);
    const bool some = j * kTile <= w0 + 31;                     // else the tile lies behind every row of this wave
    if (some) {
#pragma unroll
      for (int w = 0; w < 2; ++w)
#pragma unroll
        for (int r = 0; r < 16; ++r)
          if (j * kTile + 32 * w + reg_row(r) + 4 * h > qi) s0[w][r] = -INFINITY;
      maximum(s0);
    }
    values.take_out(lds[j & 1][1], &odd[j - whole]);
    if (!some) continue;
    weigh(j, s0);
    if (odd[j - whole]) {
      for (int key = j * kTile; key < min(at.n, min(j * kTile + kTile, w0 + 32)); ++key) {
        const uint16_t* v = vb + key * a.v_stride + 4 * h;
#pragma unroll
        for (int dt = 0; dt < DT; ++dt)
#pragma unroll
          for (int r = 0; r < 16; ++r) {
            const uint32_t x = v[32 * dt + reg_row(r)];
            if ((x & 0x7F80u) == 0x7F80u && key <= qi) acc[dt][r] += __builtin_bit_cast(float, x << 16);
          }
      }
    }
    if (j + 1 < tiles) scores(j + 1, s0);
  }
  const float total = half_sum(sum[0] + sum[1]);
  const float f = 1.0f / total;                                 // every row sees itself
  if (lse && h == 0 && qi < at.n)
    lse[static_cast<int64_t>(hq) * a.T + at.first + qi] = (__builtin_amdgcn_logf(total) + ref) * kLn2;
  // the keys are read to their end: their buffers take the results
  char* const stage = lds[wave >> 1][0] + (wave & 1) * 32 * D * 2;
  u32x4_t left[DT][2];
#pragma unroll
  for (int dt = 0; dt < DT; ++dt)
#pragma unroll
    for (int p = 0; p < 2; ++p) {
      const RowChunks<D> to(stage);
      uint32_t o[4], r[4];
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const float y0 = acc[dt][8 * p + 2 * i] * f, y1 = acc[dt][8 * p + 2 * i + 1] * f;
        o[i] = pack_bf16x2(y0, y1);
        // what the rounding took, for the backward pass
        r[i] = pack_bf16x2(y0 - __builtin_bit_cast(float, o[i] << 16), y1 - __builtin_bit_cast(float, o[i] & 0xFFFF0000u));
      }
      to.put(dt, p, o);
      left[dt][p] = u32x4_t{r[0], r[1], r[2], r[3]};
    }
  const int64_t dst = (static_cast<int64_t>(at.first + w0) * a.Hq + hq) * D;
  RowChunks<D>(stage).store(out + dst, static_cast<int64_t>(a.Hq) * D, at.n - w0);
  if (rest) {
#pragma unroll
    for (int dt = 0; dt < DT; ++dt)
#pragma unroll
      for (int p = 0; p < 2; ++p) {
        uint32_t r[4] = {left[dt][p][0], left[dt][p][1], left[dt][p][2], left[dt][p][3]};
        RowChunks<D>(stage).put(dt, p, r);
      }
    RowChunks<D>(stage).store(rest + dst, static_cast<int64_t>(a.Hq) * D, at.n - w0);
  }
}

// ---- backward --------------------------------------------------------------------
struct GradArgs {
  const uint16_t *go, *out, *rest;
  int64_t go_stride;
  const float* lse;
  float* stat;              // [2][Hq][T]: lse log2(e) and -delta, grad_q's kernel to grad_k's
};

// grad_q: a wave keeps 32 query rows and streams keys and values.
//   delta = dO . O, P = exp(scale S - lse), dS = P (dO V^T - delta), grad_q = scale dS K
// 9195 rows in 6 sequences, 32 heads on 8 of 128: 221 to 231 us (3 products, 845
// TFLOP/s and more), 7 of them for what rounding took on the diagonal; with S and dP
// formed together, one product each in turn, 16 more.
template <int D>
__global__ __launch_bounds__(256, 2) void k_prompt_bwd_q(PromptArgs a, GradArgs g, uint16_t* __restrict__ gq, int bound) {
  constexpr int KS = D / 16, DT = D / 32;
  __shared__ __align__(1024) char lds[2][2][kTile * D * 2];
  const int x = blockIdx.x % a.Hq, z = blockIdx.x / a.Hq;
  const int hq = head_of(x, a.Hq), hk = hq / (a.Hq / a.Hkv);
  fill_rows(a, gq, a.Hq, hq, z, bound);
  TileAt at;
  if (!find_tile(a, z, at)) return;
  const int lane = threadIdx.x & 63, wave = uniform(threadIdx.x >> 6), l32 = lane & 31, h = lane >> 5;
  const int q0 = (at.weight - 1) * kRows, w0 = q0 + 32 * wave, qi = w0 + l32;
  const float c = a.scale * kLog2e;
  const Offs of;
  const Copier<D> ck(a.k_stride), cv(a.v_stride);
  const uint16_t* kb = a.k + at.first * a.k_stride + hk * D;
  const uint16_t* vb = a.v + at.first * a.v_stride + hk * D;
  const int tiles = (min(at.n, q0 + kRows) + kTile - 1) / kTile;
  const int whole = q0 / kTile;                                 // tiles that every row sees whole
  ck(kb, 0, at.n, lds[0][0]);
  cv(vb, 0, at.n, lds[0][1]);

  const int64_t t = static_cast<int64_t>(at.first) + min(qi, at.n - 1);
  bf16x8_t qf[KS], gf[KS];
  float delta = 0.0f;
  {
    const uint16_t* qs = a.q + t * a.q_stride + hq * D + 8 * h;
    const uint16_t* gs = g.go + t * g.go_stride + hq * D + 8 * h;
    const int64_t os = (t * a.Hq + hq) * D + 8 * h;
#pragma unroll
    for (int ks = 0; ks < KS; ++ks) {
      qf[ks] = *reinterpret_cast<const bf16x8_t*>(qs + 16 * ks);
      gf[ks] = *reinterpret_cast<const bf16x8_t*>(gs + 16 * ks);
    }
#pragma unroll
    for (int ks = 0; ks < KS; ++ks) {
      const bf16x8_t o = *reinterpret_cast<const bf16x8_t*>(g.out + os + 16 * ks);
#pragma unroll
      for (int i = 0; i < 8; ++i) delta = __builtin_fmaf(static_cast<float>(gf[ks][i]), static_cast<float>(o[i]), delta);
    }
    if (g.rest) {
#pragma unroll
      for (int ks = 0; ks < KS; ++ks) {
        const bf16x8_t o = *reinterpret_cast<const bf16x8_t*>(g.rest + os + 16 * ks);
#pragma unroll
        for (int i = 0; i < 8; ++i) delta = __builtin_fmaf(static_cast<float>(gf[ks][i]), static_cast<float>(o[i]), delta);
      }
    }
  }
  delta = half_sum(delta);
  const int64_t st = static_cast<int64_t>(hq) * a.T + t;
  const float ls = g.lse[st] * kLog2e;
  if (qi < at.n && h == 0) {
    g.stat[st] = ls;
    g.stat[static_cast<int64_t>(a.Hq) * a.T + st] = -delta;
  }
  f32x16_t acc[DT];
#pragma unroll
  for (int dt = 0; dt < DT; ++dt) acc[dt] = zero16();

  struct Pair {
    f32x16_t s, dp;
  };
  auto scores = [&](int j, int w, Pair& p) __attribute__((always_inline)) {
    const char* kt = lds[j & 1][0];
    const char* vt = lds[j & 1][1];
    p.s = zero16();
    p.dp = zero16();
#pragma unroll
    for (int ks = 0; ks < KS; ++ks) p.s = mfma(read_row(kt, of, w, ks), qf[ks], p.s);
#pragma unroll
    for (int ks = 0; ks < KS; ++ks) p.dp = mfma(read_row(vt, of, w, ks), gf[ks], p.dp);
  };
  auto apply = [&](int j, int w, Pair& p, auto masked) __attribute__((always_inline)) {
    const char* kt = lds[j & 1][0];
#pragma unroll
    for (int r = 0; r < 16; ++r) {
      p.s[r] = __builtin_amdgcn_exp2f(__builtin_fmaf(p.s[r], c, -ls)) * (p.dp[r] - delta);
      if constexpr (decltype(masked)::value)
        if (j * kTile + 32 * w + reg_row(r) + 4 * h > qi) p.s[r] = 0.0f;
    }
    // the first row sees one key: its weight is 1 whatever the score, the score's
    // gradient zero, not what two orders of the same sum differ by (a NaN stays)
    if constexpr (decltype(masked)::value)
      if (qi == 0) p.s[0] *= 0.0f;
#pragma unroll
    for (int m = 0; m < 2; ++m) {
      const bf16x8_t pf = pack8(p.s, m);
#pragma unroll
      for (int dt = 0; dt < DT; ++dt) acc[dt] = mfma(read_tr(kt, of, 2 * w + m, dt), pf, acc[dt]);
      // on the diagonal, where a row's few score gradients cancel each other
      // (they sum to zero), with what the rounding took
      if constexpr (decltype(masked)::value) {
        const bf16x8_t rf = rest8(p.s, m, pf);
#pragma unroll
        for (int dt = 0; dt < DT; ++dt) acc[dt] = mfma(read_tr(kt, of, 2 * w + m, dt), rf, acc[dt]);
      }
    }
  };
  auto step = [&](int j, auto masked) __attribute__((always_inline)) {
    land();
    if (j + 1 < tiles) {
      ck(kb, (j + 1) * kTile, at.n, lds[(j + 1) & 1][0]);
      cv(vb, (j + 1) * kTile, at.n, lds[(j + 1) & 1][1]);
    }
    if (decltype(masked)::value && j * kTile > w0 + 31) return;  // behind every row of this wave
    Pair p0, p1;
    scores(j, 0, p0);
    scores(j, 1, p1);
    apply(j, 0, p0, masked);
    apply(j, 1, p1, masked);
  };
  for (int j = 0; j < whole; ++j) step(j, std::false_type{});
  for (int j = whole; j < tiles; ++j) step(j, std::true_type{});  // at most two, on the diagonal
  // out through the buffers that the last tile does not use
  const RowChunks<D> to(lds[tiles & 1][wave >> 1] + (wave & 1) * 32 * D * 2);
#pragma unroll
  for (int dt = 0; dt < DT; ++dt)
#pragma unroll
    for (int p = 0; p < 2; ++p) {
      uint32_t x[4];
#pragma unroll
      for (int i = 0; i < 4; ++i) x[i] = pack_bf16x2(acc[dt][8 * p + 2 * i] * a.scale, acc[dt][8 * p + 2 * i + 1] * a.scale);
      to.put(dt, p, x);
    }
  to.store(gq + (static_cast<int64_t>(at.first + w0) * a.Hq + hq) * D, static_cast<int64_t>(a.Hq) * D, at.n - w0);
}

// grad_k and grad_v: a workgroup of 8 waves keeps 128 keys with their values
// and streams the queries and output gradients of every query head of the
// group, in order, in tiles of 64 rows.
//   grad_v = P^T dO, grad_k = scale dS^T Q
// Two waves share 32 keys.  First each forms P and dS of its half of the tile's
// rows and leaves them in LDS (bf16); then each multiplies the whole tile into
// its half of the elements of grad_v and grad_k.  So the sums of a wave take 64
// registers, not 128, and two waves fit a SIMD, one's exponentials under the
// other's products.  9195 rows in 6 sequences, 32 heads on 8 of 128: 317 to 325
// us (4 products, 800 TFLOP/s and more), 17 of them for what rounding took on the diagonal;
// 4 waves that keep all sums, one a SIMD, took 360 without that.
// Where the tiles alone leave compute units idle, the heads of a group are
// split over `parts` workgroups, whose fp32 sums k_prompt_join adds in order.
template <int D>
__global__ __launch_bounds__(512, 2) void k_prompt_bwd_kv(PromptArgs a, GradArgs g, uint16_t* __restrict__ gk,
                                                          uint16_t* __restrict__ gv, float* __restrict__ part, int parts,
                                                          int bound) {
  constexpr int KS = D / 16, DT = D / 64;                       // 32-element tiles of a wave's half
  __shared__ __align__(1024) char lds[2][2][kTile * D * 2];     // [buffer][queries, output gradients]
  __shared__ __align__(1024) char weights[3][kRows * kTile * 2];   // [P, dS, what rounding took from dS][key][row of the tile]
  __shared__ __align__(256) float stat[2][2][kTile];            // [buffer][lse, -delta]
  const int x = blockIdx.x % (a.Hkv * parts), z = blockIdx.x / (a.Hkv * parts);
  const int hk = head_of(x / parts, a.Hkv), pt = x % parts;
  const int g0 = a.Hq / a.Hkv * pt / parts, G = a.Hq / a.Hkv * (pt + 1) / parts - g0;   // heads g0 .. g0+G-1 of the group
  const int h0 = hk * (a.Hq / a.Hkv) + g0;
  if (pt == 0) {
    fill_rows(a, gk, a.Hkv, hk, z, bound);
    fill_rows(a, gv, a.Hkv, hk, z, bound);
  }
  TileAt at;
  if (!find_tile(a, z, at)) return;
  const int lane = threadIdx.x & 63, wave = uniform(threadIdx.x >> 6), l32 = lane & 31, h = lane >> 5;
  const int kg = wave & 3, hf = wave >> 2;
  const int k0 = ((at.n + kRows - 1) / kRows - at.weight) * kRows, w0 = k0 + 32 * kg, ki = w0 + l32;
  const float c = a.scale * kLog2e;
  const Offs of;
  int tr[2];                                                    // transposed reads in natural order: rows 8h + i (+ 4)
#pragma unroll
  for (int hi = 0; hi < 2; ++hi) {
    const int r = 8 * h + ((lane & 15) >> 2) + 4 * hi, col = 16 * ((lane >> 4) & 1) + 4 * (lane & 3);
    tr[hi] = r * 64 + (((col >> 3) ^ ((r >> 2) & 3)) << 4) + (col & 7) * 2 + hf * DT * kSlice;
  }
  const int wrow = (32 * kg + l32) * 128;                       // this lane's key in `weights`: 16-byte chunk q / 8 at chunk ^ (key & 7)
  const Copier<D, 8> cq(a.q_stride), cg(g.go_stride);
  const int j0 = k0 / kTile;                                    // first query tile that sees these keys
  const int per = (at.n + kTile - 1) / kTile - j0;
  const uint16_t* qb = a.q + at.first * a.q_stride + h0 * D;
  const uint16_t* gb = g.go + at.first * g.go_stride + h0 * D;
  auto copy_step = [&](int buf, int i, int j) __attribute__((always_inline)) {
    cq(qb + i * D, j * kTile, at.n, lds[buf][0]);
    cg(gb + i * D, j * kTile, at.n, lds[buf][1]);
    if (wave < 2) {
      const int64_t row = (static_cast<int64_t>(wave) * a.Hq + h0 + i) * a.T + at.first + min(j * kTile + lane, at.n - 1);
      copy4(g.stat + row, lds_addr(stat[buf][wave]));
    }
  };

  const int64_t t = static_cast<int64_t>(at.first) + min(ki, at.n - 1);
  bf16x8_t kf[KS], vf[KS];
#pragma unroll
  for (int ks = 0; ks < KS; ++ks) {
    kf[ks] = *reinterpret_cast<const bf16x8_t*>(a.k + t * a.k_stride + hk * D + 8 * h + 16 * ks);
    vf[ks] = *reinterpret_cast<const bf16x8_t*>(a.v + t * a.v_stride + hk * D + 8 * h + 16 * ks);
  }
  f32x16_t ak[DT], av[DT];
#pragma unroll
  for (int dt = 0; dt < DT; ++dt) {
    ak[dt] = zero16();
    av[dt] = zero16();
  }

  auto weigh = [&](int buf, int j, auto masked) __attribute__((always_inline)) {
    const char* qt = lds[buf][0];
    const char* gt = lds[buf][1];
    f32x16_t s = zero16(), dp;                                  // dP starts from -delta
#pragma unroll
    for (int b = 0; b < 4; ++b) {
      const f32x4_t dl = *reinterpret_cast<const f32x4_t*>(&stat[buf][1][32 * hf + 8 * b + 4 * h]);
#pragma unroll
      for (int i = 0; i < 4; ++i) dp[4 * b + i] = dl[i];
    }
#pragma unroll
    for (int ks = 0; ks < KS; ++ks) s = mfma(read_row(qt, of, hf, ks), kf[ks], s);
#pragma unroll
    for (int ks = 0; ks < KS; ++ks) dp = mfma(read_row(gt, of, hf, ks), vf[ks], dp);
#pragma unroll
    for (int b = 0; b < 4; ++b) {
      const f32x4_t ls = *reinterpret_cast<const f32x4_t*>(&stat[buf][0][32 * hf + 8 * b + 4 * h]);
      float p[4], ds[4];
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const int r = 4 * b + i;
        p[i] = __builtin_amdgcn_exp2f(__builtin_fmaf(s[r], c, -ls[i]));
        ds[i] = p[i] * dp[r];
        if constexpr (decltype(masked)::value) {
          const int q = j * kTile + 32 * hf + reg_row(r) + 4 * h;
          if (q < ki || q >= at.n) p[i] = ds[i] = 0.0f;
          if (r == 0 && q == 0) ds[i] *= 0.0f;                  // as in grad_q's kernel
        }
      }
      const int at_q = wrow + (((4 * hf + b) ^ (l32 & 7)) << 4) + 8 * h;
      *reinterpret_cast<uint2*>(weights[0] + at_q) = make_uint2(pack_bf16x2(p[0], p[1]), pack_bf16x2(p[2], p[3]));
      const uint2 high = make_uint2(pack_bf16x2(ds[0], ds[1]), pack_bf16x2(ds[2], ds[3]));
      *reinterpret_cast<uint2*>(weights[1] + at_q) = high;
      if constexpr (decltype(masked)::value)                    // as in grad_q's kernel
        *reinterpret_cast<uint2*>(weights[2] + at_q) =
            make_uint2(pack_bf16x2(ds[0] - __builtin_bit_cast(float, high.x << 16), ds[1] - __builtin_bit_cast(float, high.x & 0xFFFF0000u)),
                       pack_bf16x2(ds[2] - __builtin_bit_cast(float, high.y << 16), ds[3] - __builtin_bit_cast(float, high.y & 0xFFFF0000u)));
    }
  };
  auto gather = [&](int buf, int w, auto masked) __attribute__((always_inline)) {
#pragma unroll
    for (int m = 2 * w; m < 2 * w + 2; ++m) {
      const int at_q = wrow + (((2 * m + h) ^ (l32 & 7)) << 4);
      const bf16x8_t pf = *reinterpret_cast<const bf16x8_t*>(weights[0] + at_q);
      const bf16x8_t sf = *reinterpret_cast<const bf16x8_t*>(weights[1] + at_q);
#pragma unroll
      for (int dt = 0; dt < DT; ++dt) {
        const char* q = lds[buf][0] + m * 1024 + dt * kSlice;
        const char* o = lds[buf][1] + m * 1024 + dt * kSlice;
        av[dt] = mfma(read_tr_at(o + tr[0], o + tr[1]), pf, av[dt]);
        const bf16x8_t qf = read_tr_at(q + tr[0], q + tr[1]);
        ak[dt] = mfma(qf, sf, ak[dt]);
        if constexpr (decltype(masked)::value)
          ak[dt] = mfma(qf, *reinterpret_cast<const bf16x8_t*>(weights[2] + at_q), ak[dt]);
      }
    }
  };

  // First the tiles that some key does not see whole (two on the diagonal,
  // one that the sequence's end cuts), then all others: one kind of step a
  // loop, so that the sums stay where they are.
  const int edge = at.n % kTile && per > 2 ? 1 : 0, front = min(per, 2), inner = per - front - edge;
  auto sweep = [&](int count, int first, auto masked) __attribute__((always_inline)) {
    // `count` tiles a head: j0 + first .., the cut one last in the first sweep
    int i = 0, k = 0;
    auto tile_of = [&](int kk) { return decltype(masked)::value && kk == front ? j0 + per - 1 : j0 + first + kk; };
    const int steps = count * G;
    if (steps == 0) return;
    copy_step(0, 0, tile_of(0));
    for (int st = 0; st < steps; ++st) {
      const int j = tile_of(k), buf = st & 1;
      if (++k == count) {
        k = 0;
        ++i;
      }
      land();
      if (st + 1 < steps) copy_step(buf ^ 1, i, tile_of(k));
      // rows before every key of a wave have no weights: neither formed nor read
      if (!decltype(masked)::value || j * kTile + 32 * hf + 31 >= w0) weigh(buf, j, masked);
      share_lds();
#pragma unroll
      for (int w = 0; w < 2; ++w)
        if (!decltype(masked)::value || j * kTile + 32 * w + 31 >= w0) gather(buf, w, masked);
    }
    land();                                                     // the tiles are free again
  };
  sweep(front + edge, 0, std::true_type{});
  sweep(inner, front, std::false_type{});
  if (parts > 1) {
    if (ki >= at.n) return;
    const int64_t at_out = (t * a.Hkv + hk) * D + 32 * DT * hf + 4 * h;
    const int64_t set = static_cast<int64_t>(a.T) * a.Hkv * D;
    float* dst = part + 2 * pt * set + at_out;
#pragma unroll
    for (int dt = 0; dt < DT; ++dt)
#pragma unroll
      for (int b = 0; b < 4; ++b) {
        *reinterpret_cast<f32x4_t*>(dst + 32 * dt + 8 * b) = f32x4_t{ak[dt][4 * b], ak[dt][4 * b + 1], ak[dt][4 * b + 2], ak[dt][4 * b + 3]};
        *reinterpret_cast<f32x4_t*>(dst + set + 32 * dt + 8 * b) = f32x4_t{av[dt][4 * b], av[dt][4 * b + 1], av[dt][4 * b + 2], av[dt][4 * b + 3]};
      }
    return;
  }
  const RowChunks<D / 2> to(lds[0][0] + wave * 32 * D);           // a wave's half rows
  const int64_t dst = (static_cast<int64_t>(at.first + w0) * a.Hkv + hk) * D + 32 * DT * hf;
  auto leave = [&](const f32x16_t (&x)[DT], float f, uint16_t* grad) __attribute__((always_inline)) {
#pragma unroll
    for (int dt = 0; dt < DT; ++dt)
#pragma unroll
      for (int p = 0; p < 2; ++p) {
        uint32_t y[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) y[i] = pack_bf16x2(x[dt][8 * p + 2 * i] * f, x[dt][8 * p + 2 * i + 1] * f);
        to.put(dt, p, y);
      }
    to.store(grad + dst, static_cast<int64_t>(a.Hkv) * D, at.n - w0);
  };
  leave(ak, a.scale, gk);
  leave(av, 1.0f, gv);
}

// Adds the parts of grad_k and grad_v in order; rows outside every sequence
// have none.  Four elements a thread.
__global__ __launch_bounds__(256) void k_prompt_join(PromptArgs a, const float* __restrict__ part, int parts,
                                                     uint16_t* __restrict__ gk, uint16_t* __restrict__ gv) {
  const int first = min(max(a.offsets[0], 0), a.T), last = min(max(a.offsets[a.B], first), a.T);
  const int64_t row = static_cast<int64_t>(a.Hkv) * a.D, set = a.T * row;
  for (int64_t i = 4 * (static_cast<int64_t>(blockIdx.x) * 256 + threadIdx.x) + first * row; i < last * row;
       i += static_cast<int64_t>(gridDim.x) * 1024) {
    f32x4_t k = *reinterpret_cast<const f32x4_t*>(part + i), v = *reinterpret_cast<const f32x4_t*>(part + set + i);
    for (int p = 1; p < parts; ++p) {
      const f32x4_t x = *reinterpret_cast<const f32x4_t*>(part + 2 * p * set + i);
      const f32x4_t y = *reinterpret_cast<const f32x4_t*>(part + (2 * p + 1) * set + i);
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        k[e] += x[e];
        v[e] += y[e];
      }
    }
    *reinterpret_cast<uint2*>(gk + i) = make_uint2(pack_bf16x2(k[0] * a.scale, k[1] * a.scale), pack_bf16x2(k[2] * a.scale, k[3] * a.scale));
    *reinterpret_cast<uint2*>(gv + i) = make_uint2(pack_bf16x2(v[0], v[1]), pack_bf16x2(v[2], v[3]));
  }
}

// Most tiles that T rows in B sequences can make.
int64_t tile_bound(int64_t T, int32_t B) { return T / kRows + B + 1; }

// Floats of the rows' statistics, rounded up to 16 bytes.
int64_t stat_floats(int64_t T, int32_t Hq) { return (2 * T * Hq + 3) / 4 * 4; }

// Workgroups over which the heads of a group are split: as many as bring the
// launch to one workgroup per compute unit, the rows counted as one sequence's
// (lengths are on the device).  Unsplit, a small training step (5 sequences up
// to 203 rows, 8 heads on 2 of 64) takes 42 us backward, split 26.  Many short sequences
// have more tiles than that and gain nothing by the split (16 of 60 rows, 40 heads
// on 8 of 128: 54 us, 39 unsplit; 64 of 8 rows, 32 heads on 8: 92 and 62); with a
// tile counted for each sequence others lose (8 of up to 400 rows, 32 heads on 8: 75
// us, 91 so; 40 of 200 rows, 7 heads on 1: 75 and 83).
int head_parts(int64_t T, int32_t Hq, int32_t Hkv, int cus) {
  const int64_t tiles = (T / kRows + 1) * Hkv;
  const int64_t want = cus / tiles;
  return static_cast<int>(want < 1 ? 1 : want > Hq / Hkv ? Hq / Hkv : want);
}

template <int D>
hipError_t forward(const PromptArgs& a, void* out, void* rest, float* lse, hipStream_t stream) {
  const int bound = static_cast<int>(tile_bound(a.T, a.B));
  k_prompt_fwd<D><<<static_cast<unsigned>(bound) * a.Hq, 256, 0, stream>>>(a, static_cast<uint16_t*>(out),
                                                                          static_cast<uint16_t*>(rest), lse, bound);
  return hipGetLastError();
}

template <int D>
hipError_t backward(const PromptArgs& a, const GradArgs& g, void* gq, void* gk, void* gv, hipStream_t stream) {
  const int bound = static_cast<int>(tile_bound(a.T, a.B));
  k_prompt_bwd_q<D><<<static_cast<unsigned>(bound) * a.Hq, 256, 0, stream>>>(a, g, static_cast<uint16_t*>(gq), bound);
  hipError_t e = hipGetLastError();
  if (e != hipSuccess) return e;
  const int parts = head_parts(a.T, a.Hq, a.Hkv, device_cu_count());
  float* part = g.stat + stat_floats(a.T, a.Hq);
  k_prompt_bwd_kv<D><<<static_cast<unsigned>(bound) * a.Hkv * parts, 512, 0, stream>>>(
      a, g, static_cast<uint16_t*>(gk), static_cast<uint16_t*>(gv), part, parts, bound);
  e = hipGetLastError();
  if (e != hipSuccess || parts == 1) return e;
  const int64_t groups = (static_cast<int64_t>(a.T) * a.Hkv * D / 4 + 255) / 256;
  k_prompt_join<<<static_cast<unsigned>(groups < 2048 ? groups : 2048), 256, 0, stream>>>(
      a, part, parts, static_cast<uint16_t*>(gk), static_cast<uint16_t*>(gv));
  return hipGetLastError();
}

}  // namespace

hipError_t launch_prompt_fwd(const PromptArgs& a, void* out, void* rest, float* lse, hipStream_t stream) {
  return a.D == 128 ? forward<128>(a, out, rest, lse, stream) : forward<64>(a, out, rest, lse, stream);
}

hipError_t launch_prompt_bwd(const PromptArgs& a, const void* grad_out, int64_t grad_stride, const void* out,
                             const void* rest, const float* lse, void* grad_q, void* grad_k, void* grad_v, void* ws,
                             hipStream_t stream) {
  const GradArgs g{static_cast<const uint16_t*>(grad_out), static_cast<const uint16_t*>(out),
                   static_cast<const uint16_t*>(rest), grad_stride, lse, static_cast<float*>(ws)};
  return a.D == 128 ? backward<128>(a, g, grad_q, grad_k, grad_v, stream) : backward<64>(a, g, grad_q, grad_k, grad_v, stream);
}

size_t prompt_bwd_ws_bytes(int64_t T, int32_t Hq, int32_t Hkv, int32_t D) {
  const int parts = head_parts(T, Hq, Hkv, device_cu_count());
  const int64_t sums = parts > 1 ? 2 * parts * T * Hkv * D : 0;
  return static_cast<size_t>(stat_floats(T, Hq) + sums) * sizeof(float);
}

}  // namespace nf4
