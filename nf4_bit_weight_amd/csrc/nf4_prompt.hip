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
#include "nf4_attn.hpp"

namespace nf4 {

namespace {

typedef short s16x4_t __attribute__((ext_vector_type(4)));
typedef __attribute__((address_space(3))) void lds_void_t;
typedef __attribute__((address_space(3))) s16x4_t lds_s16x4_t;

constexpr int kTile = 64;       // streamed rows per step
constexpr int kRows = 128;      // register rows per workgroup (32 a wave)
constexpr float kLog2e = 1.44269504088896340736f, kLn2 = 0.69314718055994530942f;

// Copies straight into LDS, invisible to the compiler's own waits; the kernel
// waits for them itself (vm_wait).  The LDS address is uniform, lane i lands
// 16 i (4 i) bytes behind it.
__device__ __forceinline__ void dma_b128(const void* src, uint32_t lds) {
  asm volatile("s_nop 0\n\tglobal_load_lds_dwordx4 %0, off" :: "v"(src), "{m0}"(lds) : "memory");
}
__device__ __forceinline__ void dma_b32(const void* src, uint32_t lds) {
  asm volatile("s_nop 0\n\tglobal_load_lds_dword %0, off" :: "v"(src), "{m0}"(lds) : "memory");
}
__device__ __forceinline__ uint32_t lds_addr(const void* p) {
  return static_cast<uint32_t>(reinterpret_cast<uintptr_t>((const lds_void_t*)p));
}
__device__ __forceinline__ void land() {                       // every copy has landed, for every wave
  asm volatile("s_waitcnt vmcnt(0) lgkmcnt(0)" ::: "memory");
  __builtin_amdgcn_s_barrier();
  asm volatile("" ::: "memory");
}

// LDS tile [64][D]: the 16-byte chunk c of row r lies at chunk c ^ turn(r).  Both
// reads are free of bank conflicts: 16 bytes of 8 neighbouring rows, and the
// transposed read's 32 bytes of 8 rows.
template <int D>
__device__ __forceinline__ int turn(int r) {
  return D == 128 ? 2 * (r & 7) + ((r >> 3) & 1) : 2 * ((r >> 1) & 3) + ((r >> 3) & 1);
}

// Copies rows row0 .. row0+63 of a sequence of n rows (the last row again
// behind the end; its scores are masked) into an LDS tile.
template <int D>
__device__ __forceinline__ void copy_tile(const uint16_t* base, int64_t stride, int row0, int n, const void* tile) {
  constexpr int C = D / 8, N = kTile * C / 256;
  const int wave = uniform(threadIdx.x >> 6), lane = threadIdx.x & 63;
#pragma unroll
  for (int i = 0; i < N; ++i) {
    const int k = (i * 4 + wave) * 64 + lane, r = k / C, c = (k % C) ^ turn<D>(r);
    dma_b128(base + min(row0 + r, n - 1) * stride + 8 * c, lds_addr(tile) + (i * 4 + wave) * 1024);
  }
}

// Lane offsets (bytes) of the two kinds of reads.
template <int D>
struct Offs {
  int row[D / 16];          // chunk 2 ks + h of row (lane & 31)
  int tr[D / 32][2];        // transposed: rows 4h + i (+ 8), elements 32 dt + ..
  __device__ __forceinline__ Offs() {
    const int lane = threadIdx.x & 63, l32 = lane & 31, h = lane >> 5;
#pragma unroll
    for (int ks = 0; ks < D / 16; ++ks) row[ks] = l32 * D * 2 + (((2 * ks + h) ^ turn<D>(l32)) << 4);
#pragma unroll
    for (int dt = 0; dt < D / 32; ++dt)
#pragma unroll
      for (int hi = 0; hi < 2; ++hi) {
        const int r = 4 * h + ((lane & 15) >> 2) + 8 * hi;
        const int col = 32 * dt + 16 * ((lane >> 4) & 1) + 4 * (lane & 3);
        tr[dt][hi] = r * D * 2 + (((col >> 3) ^ turn<D>(r)) << 4) + (col & 7) * 2;
      }
  }
};

__device__ __forceinline__ bf16x8_t read_row(const char* p) { return *reinterpret_cast<const bf16x8_t*>(p); }
__device__ __forceinline__ bf16x8_t read_tr(const char* lo, const char* hi) {
  const s16x4_t a = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_s16x4_t*)lo);
  const s16x4_t b = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_s16x4_t*)hi);
  const u32x2_t x = __builtin_bit_cast(u32x2_t, a), y = __builtin_bit_cast(u32x2_t, b);
  return __builtin_bit_cast(bf16x8_t, u32x4_t{x[0], x[1], y[0], y[1]});
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

// The z-th tile of `rows` rows, counted over all sequences; false behind the last.
struct TileAt {
  int first, n, tile;
};
__device__ __forceinline__ int count_tiles(const PromptArgs& a, int rows) {
  int sum = 0;
  for (int b = threadIdx.x & 63; b < a.B; b += 64) {
    int f, n;
    seq_rows(a.offsets, b, a.T, f, n);
    sum += (n + rows - 1) / rows;
  }
  return uniform(wave_sum(sum));
}
__device__ __forceinline__ bool find_tile(const PromptArgs& a, int rows, int z, TileAt& at) {
  int base = 0;
  const int lane = threadIdx.x & 63;
  for (int b0 = 0; b0 < a.B; b0 += 64) {
    int f = 0, n = 0;
    if (b0 + lane < a.B) seq_rows(a.offsets, b0 + lane, a.T, f, n);
    const int tiles = (n + rows - 1) / rows, incl = wave_scan(tiles);
    const uint64_t hit = __ballot(base + incl > z);
    if (hit) {
      const int l = __builtin_ctzll(hit);
      at.first = uniform(__shfl(f, l));
      at.n = uniform(__shfl(n, l));
      at.tile = uniform(z - base - __shfl(incl - tiles, l));
      return true;
    }
    base += __shfl(incl, 63);
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

// Heads of one key head next to each other in one XCD's queue (workgroups go
// round the 8 XCDs in order), so that they share its L2.
__device__ __forceinline__ int head_of(int x, int heads) { return heads % 8 == 0 ? (x % 8) * (heads / 8) + x / 8 : x; }

// ---- forward -------------------------------------------------------------------
template <int D>
__global__ __launch_bounds__(256, 2) void k_prompt_fwd(PromptArgs a, uint16_t* __restrict__ out, float* __restrict__ lse,
                                                       int bound) {
  constexpr int KS = D / 16, DT = D / 32;
  __shared__ __align__(1024) char lds[2][2][kTile * D * 2];     // [buffer][keys, values]
  const int x = blockIdx.x % a.Hq, z = blockIdx.x / a.Hq;
  const int hq = head_of(x, a.Hq), hk = hq / (a.Hq / a.Hkv);
  fill_rows(a, out, a.Hq, hq, z, bound);
  const int total = count_tiles(a, kRows);
  TileAt at;
  // long rows of keys first
  if (z >= total || !find_tile(a, kRows, total - 1 - z, at)) return;
  const int lane = threadIdx.x & 63, wave = uniform(threadIdx.x >> 6), l32 = lane & 31, h = lane >> 5;
  const int w0 = at.tile * kRows + 32 * wave, qi = w0 + l32;
  const float c = a.scale * kLog2e;
  const Offs<D> of;

  const uint16_t* kb = a.k + at.first * a.k_stride + hk * D;
  const uint16_t* vb = a.v + at.first * a.v_stride + hk * D;
  copy_tile<D>(kb, a.k_stride, 0, at.n, lds[0][0]);
  copy_tile<D>(vb, a.v_stride, 0, at.n, lds[0][1]);

  bf16x8_t qf[KS];
  {
    const uint16_t* src = a.q + (static_cast<int64_t>(at.first) + min(qi, at.n - 1)) * a.q_stride + hq * D + 8 * h;
#pragma unroll
    for (int ks = 0; ks < KS; ++ks) qf[ks] = *reinterpret_cast<const bf16x8_t*>(src + 16 * ks);
  }
  f32x16_t acc[DT];
#pragma unroll
  for (int dt = 0; dt < DT; ++dt) acc[dt] = zero16();
  float mx = -INFINITY, sum = 0.0f;

  const int tiles = (min(at.n, at.tile * kRows + kRows) + kTile - 1) / kTile;
  for (int j = 0; j < tiles; ++j) {
    land();
    if (j + 1 < tiles) {
      copy_tile<D>(kb, a.k_stride, (j + 1) * kTile, at.n, lds[(j + 1) & 1][0]);
      copy_tile<D>(vb, a.v_stride, (j + 1) * kTile, at.n, lds[(j + 1) & 1][1]);
    }
    if (j * kTile > w0 + 31) continue;                          // behind every row of this wave
    const char* kt = lds[j & 1][0];
    const char* vt = lds[j & 1][1];
    f32x16_t s[2] = {zero16(), zero16()};
#pragma unroll
    for (int ks = 0; ks < KS; ++ks)
#pragma unroll
      for (int w = 0; w < 2; ++w) s[w] = mfma(read_row(kt + of.row[ks] + 32 * w * D * 2), qf[ks], s[w]);
    if (j * kTile + kTile - 1 > w0) {
#pragma unroll
      for (int w = 0; w < 2; ++w)
#pragma unroll
        for (int r = 0; r < 16; ++r)
          if (j * kTile + 32 * w + reg_row(r) + 4 * h > qi) s[w][r] = -INFINITY;
    }
    float top = mx;
#pragma unroll
    for (int w = 0; w < 2; ++w)
#pragma unroll
      for (int r = 0; r < 16; ++r) top = fmaxf(top, s[w][r]);
    top = half_max(top);
    const float ref = top == -INFINITY ? 0.0f : top * c;
    if (__any(top != mx)) {
      const float f = __builtin_amdgcn_exp2f(__builtin_fmaf(mx, c, -ref));
      sum *= f;
#pragma unroll
      for (int dt = 0; dt < DT; ++dt)
#pragma unroll
        for (int r = 0; r < 16; ++r) acc[dt][r] *= f;
      mx = top;
    }
#pragma unroll
    for (int w = 0; w < 2; ++w)
#pragma unroll
      for (int r = 0; r < 16; ++r) {
        s[w][r] = __builtin_amdgcn_exp2f(__builtin_fmaf(s[w][r], c, -ref));
        sum += s[w][r];
      }
#pragma unroll
    for (int w = 0; w < 2; ++w)
#pragma unroll
      for (int m = 0; m < 2; ++m) {
        const bf16x8_t pf = pack8(s[w], m);
#pragma unroll
        for (int dt = 0; dt < DT; ++dt) {
          const char* p = vt + (32 * w + 16 * m) * D * 2;
          acc[dt] = mfma(read_tr(p + of.tr[dt][0], p + of.tr[dt][1]), pf, acc[dt]);
        }
      }
  }
  sum = half_sum(sum);
  if (qi >= at.n) return;
  const float f = 1.0f / sum;                                   // every row sees itself
  const int64_t t = static_cast<int64_t>(at.first) + qi;
  if (lse && h == 0) lse[static_cast<int64_t>(hq) * a.T + t] = (__builtin_amdgcn_logf(sum) + mx * c) * kLn2;
  uint16_t* dst = out + (t * a.Hq + hq) * D + 4 * h;
#pragma unroll
  for (int dt = 0; dt < DT; ++dt)
#pragma unroll
    for (int b = 0; b < 4; ++b)
      *reinterpret_cast<uint2*>(dst + 32 * dt + 8 * b) =
          make_uint2(pack_bf16x2(acc[dt][4 * b] * f, acc[dt][4 * b + 1] * f),
                     pack_bf16x2(acc[dt][4 * b + 2] * f, acc[dt][4 * b + 3] * f));
}

// ---- backward --------------------------------------------------------------------
// delta[hq][t] = grad_out[t, hq] . out[t, hq], in fp32: D / 8 lanes a row.
template <int D>
__global__ __launch_bounds__(256) void k_prompt_delta(PromptArgs a, const uint16_t* __restrict__ go, int64_t go_stride,
                                                      const uint16_t* __restrict__ out, float* __restrict__ delta) {
  constexpr int L = D / 8;
  const int64_t rows = static_cast<int64_t>(a.T) * a.Hq;
  for (int64_t i = (static_cast<int64_t>(blockIdx.x) * 256 + threadIdx.x) / L; i < rows;
       i += static_cast<int64_t>(gridDim.x) * 256 / L) {
    const int64_t t = i / a.Hq;
    const int hq = static_cast<int>(i - t * a.Hq), e = 8 * (threadIdx.x % L);
    const u32x4_t x = *reinterpret_cast<const u32x4_t*>(go + t * go_stride + hq * D + e);
    const u32x4_t y = *reinterpret_cast<const u32x4_t*>(out + i * D + e);
    float s = 0.0f;
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      s = __builtin_fmaf(__builtin_bit_cast(float, x[k] << 16), __builtin_bit_cast(float, y[k] << 16), s);
      s = __builtin_fmaf(__builtin_bit_cast(float, x[k] & 0xFFFF0000u), __builtin_bit_cast(float, y[k] & 0xFFFF0000u), s);
    }
#pragma unroll
    for (int d = 1; d < L; d *= 2) s += __shfl_xor(s, d);
    if (e == 0) delta[static_cast<int64_t>(hq) * a.T + t] = s;
  }
}

// grad_q: a wave keeps 32 query rows and streams keys and values.
//   P = exp(scale S - lse), dS = P (dP - delta), grad_q = scale dS K
template <int D>
__global__ __launch_bounds__(256, 2) void k_prompt_bwd_q(PromptArgs a, const uint16_t* __restrict__ go, int64_t go_stride,
                                                         const float* __restrict__ lse, const float* __restrict__ delta,
                                                         uint16_t* __restrict__ gq, int bound) {
  constexpr int KS = D / 16, DT = D / 32;
  __shared__ __align__(1024) char lds[2][2][kTile * D * 2];
  const int x = blockIdx.x % a.Hq, z = blockIdx.x / a.Hq;
  const int hq = head_of(x, a.Hq), hk = hq / (a.Hq / a.Hkv);
  fill_rows(a, gq, a.Hq, hq, z, bound);
  const int total = count_tiles(a, kRows);
  TileAt at;
  if (z >= total || !find_tile(a, kRows, total - 1 - z, at)) return;
  const int lane = threadIdx.x & 63, wave = uniform(threadIdx.x >> 6), l32 = lane & 31, h = lane >> 5;
  const int w0 = at.tile * kRows + 32 * wave, qi = w0 + l32;
  const float c = a.scale * kLog2e;
  const Offs<D> of;
  const uint16_t* kb = a.k + at.first * a.k_stride + hk * D;
  const uint16_t* vb = a.v + at.first * a.v_stride + hk * D;
  copy_tile<D>(kb, a.k_stride, 0, at.n, lds[0][0]);
  copy_tile<D>(vb, a.v_stride, 0, at.n, lds[0][1]);

  const int64_t t = static_cast<int64_t>(at.first) + min(qi, at.n - 1);
  bf16x8_t qf[KS], gf[KS];
#pragma unroll
  for (int ks = 0; ks < KS; ++ks) {
    qf[ks] = *reinterpret_cast<const bf16x8_t*>(a.q + t * a.q_stride + hq * D + 8 * h + 16 * ks);
    gf[ks] = *reinterpret_cast<const bf16x8_t*>(go + t * go_stride + hq * D + 8 * h + 16 * ks);
  }
  const float ls = lse[static_cast<int64_t>(hq) * a.T + t] * kLog2e, dl = delta[static_cast<int64_t>(hq) * a.T + t];
  f32x16_t acc[DT];
#pragma unroll
  for (int dt = 0; dt < DT; ++dt) acc[dt] = zero16();

  const int tiles = (min(at.n, at.tile * kRows + kRows) + kTile - 1) / kTile;
  for (int j = 0; j < tiles; ++j) {
    land();
    if (j + 1 < tiles) {
      copy_tile<D>(kb, a.k_stride, (j + 1) * kTile, at.n, lds[(j + 1) & 1][0]);
      copy_tile<D>(vb, a.v_stride, (j + 1) * kTile, at.n, lds[(j + 1) & 1][1]);
    }
#pragma unroll
    for (int w = 0; w < 2; ++w) {
      const int k0 = j * kTile + 32 * w;
      if (k0 > w0 + 31) continue;
      const char* kt = lds[j & 1][0] + 32 * w * D * 2;
      const char* vt = lds[j & 1][1] + 32 * w * D * 2;
      f32x16_t s = zero16(), dp = zero16();
#pragma unroll
      for (int ks = 0; ks < KS; ++ks) {
        s = mfma(read_row(kt + of.row[ks]), qf[ks], s);
        dp = mfma(read_row(vt + of.row[ks]), gf[ks], dp);
      }
#pragma unroll
      for (int r = 0; r < 16; ++r) s[r] = __builtin_amdgcn_exp2f(__builtin_fmaf(s[r], c, -ls)) * (dp[r] - dl);
      if (k0 + 31 > w0) {
#pragma unroll
        for (int r = 0; r < 16; ++r)
          if (k0 + reg_row(r) + 4 * h > qi) s[r] = 0.0f;
      }
#pragma unroll
      for (int m = 0; m < 2; ++m) {
        const bf16x8_t pf = pack8(s, m);
#pragma unroll
        for (int dt = 0; dt < DT; ++dt) {
          const char* p = kt + 16 * m * D * 2;
          acc[dt] = mfma(read_tr(p + of.tr[dt][0], p + of.tr[dt][1]), pf, acc[dt]);
        }
      }
    }
  }
  if (qi >= at.n) return;
  uint16_t* dst = gq + (t * a.Hq + hq) * D + 4 * h;
#pragma unroll
  for (int dt = 0; dt < DT; ++dt)
#pragma unroll
    for (int b = 0; b < 4; ++b)
      *reinterpret_cast<uint2*>(dst + 32 * dt + 8 * b) =
          make_uint2(pack_bf16x2(acc[dt][4 * b] * a.scale, acc[dt][4 * b + 1] * a.scale),
                     pack_bf16x2(acc[dt][4 * b + 2] * a.scale, acc[dt][4 * b + 3] * a.scale));
}

// grad_k and grad_v: a wave keeps 32 keys with their values and streams the
// queries and output gradients of every query head of the group, in order.
//   grad_v = P^T dO, grad_k = scale dS^T Q
template <int D>
__global__ __launch_bounds__(256, 1) void k_prompt_bwd_kv(PromptArgs a, const uint16_t* __restrict__ go, int64_t go_stride,
                                                          const float* __restrict__ lse, const float* __restrict__ delta,
                                                          uint16_t* __restrict__ gk, uint16_t* __restrict__ gv, int bound) {
  constexpr int KS = D / 16, DT = D / 32;
  __shared__ __align__(1024) char lds[2][2][kTile * D * 2];     // [buffer][queries, output gradients]
  __shared__ __align__(256) float stat[2][2][kTile];            // [buffer][lse, delta]
  const int x = blockIdx.x % a.Hkv, z = blockIdx.x / a.Hkv, G = a.Hq / a.Hkv;
  const int hk = head_of(x, a.Hkv);
  fill_rows(a, gk, a.Hkv, hk, z, bound);
  fill_rows(a, gv, a.Hkv, hk, z, bound);
  TileAt at;
  if (!find_tile(a, kRows, z, at)) return;
  const int lane = threadIdx.x & 63, wave = uniform(threadIdx.x >> 6), l32 = lane & 31, h = lane >> 5;
  const int w0 = at.tile * kRows + 32 * wave, ki = w0 + l32;
  const float c = a.scale * kLog2e;
  const Offs<D> of;
  const int q0 = at.tile * kRows / kTile;                       // first query tile that sees these keys
  const int per = (at.n + kTile - 1) / kTile - q0, steps = per * G;
  auto copy_step = [&](int st) __attribute__((always_inline)) {
    const int hq = hk * G + st / per, j = q0 + st % per, buf = st & 1;
    copy_tile<D>(a.q + at.first * a.q_stride + hq * D, a.q_stride, j * kTile, at.n, lds[buf][0]);
    copy_tile<D>(go + at.first * go_stride + hq * D, go_stride, j * kTile, at.n, lds[buf][1]);
    if (wave < 2) {
      const int64_t row = static_cast<int64_t>(hq) * a.T + at.first + min(j * kTile + lane, at.n - 1);
      dma_b32((wave == 0 ? lse : delta) + row, lds_addr(stat[buf][wave]));
    }
  };
  copy_step(0);

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

  for (int st = 0; st < steps; ++st) {
    land();
    if (st + 1 < steps) copy_step(st + 1);
    const int j = q0 + st % per;
#pragma unroll
    for (int w = 0; w < 2; ++w) {
      const int r0 = j * kTile + 32 * w;
      if (r0 + 31 < w0) continue;                               // before every key of this wave
      const char* qt = lds[st & 1][0] + 32 * w * D * 2;
      const char* gt = lds[st & 1][1] + 32 * w * D * 2;
      f32x16_t s = zero16(), dp = zero16();
#pragma unroll
      for (int ks = 0; ks < KS; ++ks) {
        s = mfma(read_row(qt + of.row[ks]), kf[ks], s);
        dp = mfma(read_row(gt + of.row[ks]), vf[ks], dp);
      }
#pragma unroll
      for (int b = 0; b < 4; ++b) {
        const f32x4_t ls = *reinterpret_cast<const f32x4_t*>(&stat[st & 1][0][32 * w + 8 * b + 4 * h]);
        const f32x4_t dl = *reinterpret_cast<const f32x4_t*>(&stat[st & 1][1][32 * w + 8 * b + 4 * h]);
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const int r = 4 * b + i;
          s[r] = __builtin_amdgcn_exp2f(__builtin_fmaf(s[r], c, -ls[i] * kLog2e));
          dp[r] = s[r] * (dp[r] - dl[i]);
        }
      }
      if (r0 < w0 + 31 || r0 + 32 > at.n) {
#pragma unroll
        for (int r = 0; r < 16; ++r) {
          const int q = r0 + reg_row(r) + 4 * h;
          if (q < ki || q >= at.n) {
            s[r] = 0.0f;
            dp[r] = 0.0f;
          }
        }
      }
#pragma unroll
      for (int m = 0; m < 2; ++m) {
        const bf16x8_t pf = pack8(s, m), sf = pack8(dp, m);
#pragma unroll
        for (int dt = 0; dt < DT; ++dt) {
          const char* g = gt + 16 * m * D * 2;
          const char* q = qt + 16 * m * D * 2;
          av[dt] = mfma(read_tr(g + of.tr[dt][0], g + of.tr[dt][1]), pf, av[dt]);
          ak[dt] = mfma(read_tr(q + of.tr[dt][0], q + of.tr[dt][1]), sf, ak[dt]);
        }
      }
    }
  }
  if (ki >= at.n) return;
  uint16_t* dk = gk + (t * a.Hkv + hk) * D + 4 * h;
  uint16_t* dv = gv + (t * a.Hkv + hk) * D + 4 * h;
#pragma unroll
  for (int dt = 0; dt < DT; ++dt)
#pragma unroll
    for (int b = 0; b < 4; ++b) {
      *reinterpret_cast<uint2*>(dk + 32 * dt + 8 * b) =
          make_uint2(pack_bf16x2(ak[dt][4 * b] * a.scale, ak[dt][4 * b + 1] * a.scale),
                     pack_bf16x2(ak[dt][4 * b + 2] * a.scale, ak[dt][4 * b + 3] * a.scale));
      *reinterpret_cast<uint2*>(dv + 32 * dt + 8 * b) =
          make_uint2(pack_bf16x2(av[dt][4 * b], av[dt][4 * b + 1]), pack_bf16x2(av[dt][4 * b + 2], av[dt][4 * b + 3]));
    }
}

// Most tiles that T rows in B sequences can make.
int64_t tile_bound(const PromptArgs& a) { return a.T / kRows + a.B + 1; }

template <int D>
hipError_t forward(const PromptArgs& a, void* out, float* lse, hipStream_t stream) {
  const int bound = static_cast<int>(tile_bound(a));
  k_prompt_fwd<D><<<static_cast<unsigned>(bound) * a.Hq, 256, 0, stream>>>(a, static_cast<uint16_t*>(out), lse, bound);
  return hipGetLastError();
}

template <int D>
hipError_t backward(const PromptArgs& a, const void* grad_out, int64_t go_stride, const void* out, const float* lse,
                    void* gq, void* gk, void* gv, void* ws, hipStream_t stream) {
  const int bound = static_cast<int>(tile_bound(a));
  float* delta = static_cast<float*>(ws);
  const uint16_t* go = static_cast<const uint16_t*>(grad_out);
  const int64_t groups = (static_cast<int64_t>(a.T) * a.Hq * (D / 8) + 255) / 256;
  k_prompt_delta<D><<<static_cast<unsigned>(groups < 4096 ? groups : 4096), 256, 0, stream>>>(
      a, go, go_stride, static_cast<const uint16_t*>(out), delta);
  hipError_t e = hipGetLastError();
  if (e != hipSuccess) return e;
  k_prompt_bwd_kv<D><<<static_cast<unsigned>(bound) * a.Hkv, 256, 0, stream>>>(
      a, go, go_stride, lse, delta, static_cast<uint16_t*>(gk), static_cast<uint16_t*>(gv), bound);
  e = hipGetLastError();
  if (e != hipSuccess) return e;
  k_prompt_bwd_q<D><<<static_cast<unsigned>(bound) * a.Hq, 256, 0, stream>>>(a, go, go_stride, lse, delta,
                                                                            static_cast<uint16_t*>(gq), bound);
  return hipGetLastError();
}

}  // namespace

hipError_t launch_prompt_fwd(const PromptArgs& a, void* out, float* lse, hipStream_t stream) {
  return a.D == 128 ? forward<128>(a, out, lse, stream) : forward<64>(a, out, lse, stream);
}

hipError_t launch_prompt_bwd(const PromptArgs& a, const void* grad_out, int64_t grad_stride, const void* out,
                             const float* lse, void* grad_q, void* grad_k, void* grad_v, void* ws, hipStream_t stream) {
  return a.D == 128 ? backward<128>(a, grad_out, grad_stride, out, lse, grad_q, grad_k, grad_v, ws, stream)
                    : backward<64>(a, grad_out, grad_stride, out, lse, grad_q, grad_k, grad_v, ws, stream);
}

}  // namespace nf4
