// Products in 8-bit integers with a scale for each token and each channel
// (nf4_int8.h).
#include <cmath>

#include <type_traits>

#include "nf4_attn.hpp"
#include "nf4_device.hpp"
#include "nf4_int8.hpp"
#include "nf4_internal.hpp"

namespace nf4 {

namespace {

typedef int i32x4_t __attribute__((ext_vector_type(4)));
typedef int i32x16_t __attribute__((ext_vector_type(16)));

__device__ __forceinline__ float as_float(uint16_t b) { return __builtin_bit_cast(float, static_cast<uint32_t>(b) << 16); }
__device__ __forceinline__ float value(const float* p) { return *p; }
__device__ __forceinline__ float value(const uint16_t* p) { return as_float(*p); }
__device__ __forceinline__ void put(float* p, float v) { *p = v; }
__device__ __forceinline__ void put(uint16_t* p, float v) { *p = to_bf16(v); }

// LDS written by some lanes of a wave is read by others of the same wave.
__device__ __forceinline__ void wave_sync() {
  __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
  __builtin_amdgcn_wave_barrier();
}

// ---- rows of integers --------------------------------------------------------------

// The integer nearest to 127 x / top, half-way to even, in the low byte.  A
// rounded quotient is at most one off; the rest 127 x - q top then says on which
// side of the middle x lies.  It is exact: for bf16 every term has at most 15
// bits and the rest fits 24, for fp32 it is taken in 64 bits (7 + 24).  (All over 128:
// 127 times the largest number is none.)
// Adding 1.5 * 2^23 rounds to an integer, which then stands in the low bits.
template <typename T>
__device__ __forceinline__ uint32_t nearest(float x, float top, float inverse) {
  constexpr float kInt = 12582912.0f;
  const float t = fmaf(x, inverse, kInt), q = t - kInt;
  const uint32_t i = __builtin_bit_cast(uint32_t, t);
  using R = std::conditional_t<sizeof(T) == 2, float, double>;
  const R unit = static_cast<R>(top) * static_cast<R>(0x1p-7), half = static_cast<R>(0.5) * unit;
  const R rest = fma(-static_cast<R>(q), unit, static_cast<R>(127 * 0x1p-7) * static_cast<R>(x));
  const bool odd = (i & 1) != 0;
  return i + (rest > half || (rest == half && odd)) - (rest < -half || (rest == -half && odd));
}

// Elements i .. i + 7 of a row of K, zeros behind it; VEC: rows are 16-byte aligned.
template <bool VEC, typename T>
__device__ __forceinline__ void load8(const T* row, int i, int K, float (&f)[8]) {
  if (VEC && i + 8 <= K) {
    if constexpr (sizeof(T) == 4) {
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        const f32x4_t v = *reinterpret_cast<const f32x4_t*>(row + i + 4 * h);
#pragma unroll
        for (int e = 0; e < 4; ++e) f[4 * h + e] = v[e];
      }
    } else {
      const u32x4_t v = *reinterpret_cast<const u32x4_t*>(row + i);
#pragma unroll
      for (int e = 0; e < 8; ++e) f[e] = as_float(static_cast<uint16_t>(v[e / 2] >> (16 * (e & 1))));
    }
  } else {
#pragma unroll
    for (int e = 0; e < 8; ++e) f[e] = i + e < K ? value(row + i + e) : 0.0f;
  }
}

// The largest magnitude as an integer: of bit patterns without a sign, infinity
// and NaN are the largest.
__device__ __forceinline__ uint32_t largest_of(const float (&v)[8], uint32_t top_bits) {
#pragma unroll
  for (int e = 0; e < 8; ++e) top_bits = max(top_bits, __builtin_bit_cast(uint32_t, v[e]) & 0x7FFFFFFFu);
  return top_bits;
}
// over the 16 lanes of a row, in lane moves of the vector unit (quad_perm twice, row_half_mirror, row_mirror)
template <int MOVE>
__device__ __forceinline__ uint32_t moved_max(uint32_t v) {
  const uint32_t o = static_cast<uint32_t>(__builtin_amdgcn_update_dpp(0, static_cast<int>(v), MOVE, 0xF, 0xF, true));
  return o > v ? o : v;
}
__device__ __forceinline__ uint32_t row_max(uint32_t v) {
  return moved_max<0x140>(moved_max<0x141>(moved_max<0x4E>(moved_max<0xB1>(v))));
}
__device__ __forceinline__ uint32_t wave_max(uint32_t v) {
  const int m = static_cast<int>(row_max(v));                  // (below 2^31)
  return static_cast<uint32_t>(max(max(__builtin_amdgcn_readlane(m, 0), __builtin_amdgcn_readlane(m, 16)),
                                   max(__builtin_amdgcn_readlane(m, 32), __builtin_amdgcn_readlane(m, 48))));
}
struct RowScale {
  float top, inverse, scale;
  bool live;
};
__device__ __forceinline__ RowScale row_scale(uint32_t top_bits) {
  const float top = __builtin_bit_cast(float, top_bits);
  const bool bad = top_bits >= 0x7F800000u, live = !bad && top >= 0x1p-119f;
  return {top, 127.0f / top, bad ? NAN : live ? top / 127.0f : 0.0f, live};
}
template <typename T>
__device__ __forceinline__ u32x2_t round8(const float (&v)[8], const RowScale& sc) {
  u32x2_t o = {0, 0};
  if (sc.live) {
    uint32_t b[8];
#pragma unroll
    for (int e = 0; e < 8; ++e) b[e] = nearest<T>(v[e], sc.top, sc.inverse);
#pragma unroll
    for (int h = 0; h < 2; ++h)
      o[h] = perm(perm(b[4 * h + 3], b[4 * h + 2], 0x0C0C0400u), perm(b[4 * h + 1], b[4 * h], 0x0C0C0400u), 0x05040100u);
  }
  return o;
}

// A workgroup a row.  Up to 2048 J elements stay in registers between the search
// for the largest and the rounding; J = 0 reads the row twice.
// (2048 x 5120 bf16, 31 MB: 20.4 us with one element a load, 10.1 to 12.4 so; at a copy's rate the
// bytes take 6.2.  All those rows are in work at once, and each is read whole, waited for, and only
// then written, so that little reading and writing overlaps.)
template <typename T, int J, bool VEC>
__global__ __launch_bounds__(256) void k_quantize(const T* x, int64_t stride, int K, int pitch, int8_t* q, float* scale) {
  __shared__ uint32_t s_top[4];
  const int64_t r = blockIdx.x;
  const T* row = x + r * stride;
  constexpr int kKept = J > 0 ? J : 1;
  float f[kKept][8];
  uint32_t top_bits = 0;
  if constexpr (J > 0) {
#pragma unroll
    for (int j = 0; j < J; ++j) load8<VEC>(row, (j * 256 + threadIdx.x) * 8, K, f[j]);
#pragma unroll
    for (int j = 0; j < J; ++j) top_bits = largest_of(f[j], top_bits);
  } else {
    for (int i = threadIdx.x * 8; i < K; i += 2048) {
      load8<VEC>(row, i, K, f[0]);
      top_bits = largest_of(f[0], top_bits);
    }
  }
  top_bits = wave_max(top_bits);
  if ((threadIdx.x & 63) == 0) s_top[threadIdx.x >> 6] = top_bits;
  __syncthreads();
  const RowScale sc = row_scale(max(max(s_top[0], s_top[1]), max(s_top[2], s_top[3])));
  auto put8 = [&](const float (&v)[8], int i) {
    if (i < pitch) *reinterpret_cast<u32x2_t*>(q + r * pitch + i) = round8<T>(v, sc);
  };
  if constexpr (J > 0) {
#pragma unroll
    for (int j = 0; j < J; ++j) put8(f[j], (j * 256 + threadIdx.x) * 8);
  } else {
    for (int i = threadIdx.x * 8; i < pitch; i += 2048) {
      load8<VEC>(row, i, K, f[0]);
      put8(f[0], i);
    }
  }
  if (threadIdx.x == 0) scale[r] = sc.scale;
}

template <typename T, bool VEC>
hipError_t launch_quantize_t(const T* x, int64_t stride, int64_t M, int K, int pitch, int8_t* q, float* scale, hipStream_t stream) {
  auto go = [&](auto kernel) {
    kernel<<<static_cast<uint32_t>(M), 256, 0, stream>>>(x, stride, K, pitch, q, scale);
    return hipGetLastError();
  };
  if (pitch <= 2048) return go(k_quantize<T, 1, VEC>);
  if (pitch <= 4096) return go(k_quantize<T, 2, VEC>);
  if (pitch <= 8192) return go(k_quantize<T, 4, VEC>);
  if (pitch <= 16384) return go(k_quantize<T, 8, VEC>);
  return go(k_quantize<T, 0, VEC>);
}

// ---- the product -------------------------------------------------------------------

// The rows of row tile mt (as in nf4_gemm.hip: the experts' tiles one expert
// after another, found by every wave on its own).  Behind them come the tiles of
// the rows that belong to nobody: e == E.
struct RowTile {
  int64_t first, end;
  int e;
};
template <int BM>
__device__ __forceinline__ RowTile row_tile(const Int8Args& a, int mt) {
  if (!a.offsets) return {static_cast<int64_t>(mt) * BM, a.M, 0};
  const int lane = static_cast<int>(threadIdx.x & 63), M = static_cast<int>(a.M);
  int before = 0;
  for (int e0 = 0; e0 <= a.E; e0 += 64) {
    const int e = e0 + lane;
    int lo = 0, hi = 0;
    if (e <= a.E) {
      lo = a.offsets[e];
      hi = e < a.E ? a.offsets[e + 1] : M;
      lo = min(max(lo, 0), M);
      hi = min(max(hi, lo), M);
    }
    const int tiles = (hi - lo + BM - 1) / BM, incl = wave_scan(tiles), at = before + incl - tiles;
    const unsigned long long hit = __ballot(mt >= at && mt < before + incl);
    if (hit) {
      const int l = uniform(__ffsll(static_cast<long long>(hit)) - 1);
      return {__builtin_amdgcn_readlane(lo, l) + static_cast<int64_t>(mt - __builtin_amdgcn_readlane(at, l)) * BM,
              __builtin_amdgcn_readlane(hi, l), e0 + l};
    }
    before += __builtin_amdgcn_readlane(incl, 63);
  }
  return {0, 0, 0};
}
// Bound on the row tiles of M rows.
int64_t row_tiles(const Int8Args& a, int bm) {
  return a.offsets ? a.M / bm + (a.E < a.M ? a.E : a.M) + 1 : (a.M + bm - 1) / bm;
}

__device__ __forceinline__ int64_t row_of(const Int8Args& a, int64_t r) {
  if (!a.tokens) return r;
  const int64_t t = a.tokens[r];
  return t < 0 ? 0 : t < a.x_rows ? t : a.x_rows - 1;
}

// A step's piece of a tile's rows in LDS: rows of BK = 128 bytes with 16-byte unit u of
// row r at unit u ^ ((r >> 1) & 7), or of 64 bytes, u at u ^ ((r >> 2) & 3).  Sixteen
// neighbouring rows then hold the same unit in all 64 banks.
template <int BK>
__device__ __forceinline__ int unit_at(int r, int u) {
  return BK == 128 ? u ^ ((r >> 1) & 7) : u ^ ((r >> 2) & 3);
}

// The result of a wave is WM x WN, of 32 x 32 blocks whose lanes hold row lane & 31 and
// columns 8 (i / 4) + 4 half + i % 4.
template <int BM_, int BN_, int WX_, int WY_, int BK_, int NS_>
struct Tile {
  static constexpr int BM = BM_, BN = BN_, WX = WX_, WY = WY_;
  static constexpr int kWaves = WX * WY, WM = BM / WX, WN = BN / WY, MI = WM / 32, NI = WN / 32;
  static constexpr int BK = BK_, NS = NS_;                      // bytes of a row in one step, steps in LDS
  static constexpr int kStage = (BM + BN) * BK;                // bytes of one step
  static constexpr int kRows = 1024 / BK;                      // rows of one copy
  static constexpr int IX = BM / kRows / kWaves, IW = BN / kRows / kWaves;       // copies of a wave
  static constexpr int kLds = NS * kStage;
  static constexpr int kOut = kWaves * 32 * (WN * 4 + 16);       // 32 rows of each wave's result
  static constexpr int kAfter = kOut + (BM + 2 * BN) * 4;        // and the scales
  static constexpr int kBytes = kLds > kAfter ? kLds : kAfter;
};

// What bounds it: 2048 x 27648 x 5120 in 256 x 256 takes 295 us, 1963 TOP/s (a library product of
// the same integers, without scales, 306); the matrix units are busy 48 % of the time at the 1.9 GHz that
// they leave the card under this load.  512 tokens of 8 of 64 experts, 1024 x 2048 each, in 64 x 64: 41 us, of which the bytes
// would take 29.  Neither they (114 MB moved, 2.8 TB/s) nor the matrix units (busy 12 %) bound it but
// the tiles: the experts hold 4 to 251 rows, 36 of their 100 row tiles read a weight again and 37 hold at
// most 32 rows, and 1600 workgroups on 512 places are three rounds and an eighth of one.
template <typename T, typename Y>
__global__ __launch_bounds__(64 * T::kWaves, 1) void k_tile(Int8Args a, int m_tiles, int n_tiles) {
  constexpr int BM = T::BM, BN = T::BN, MI = T::MI, NI = T::NI, IX = T::IX, IW = T::IW;
  extern __shared__ __attribute__((aligned(16))) char lds[];
  int mt, nt;
  if (a.offsets) {
    // an expert's column tiles side by side on one XCD, the row tiles dealt to the XCDs in turn
    const int idx = blockIdx.x >> 3;
    nt = idx % n_tiles;
    mt = idx / n_tiles * 8 + (blockIdx.x & 7);
  } else {
    // every XCD a run of tiles, the row tiles of one weight tile side by side
    const int t = gridDim.x, xcd = blockIdx.x & 7, q = t >> 3, r = t & 7;
    const int id = xcd * q + (xcd < r ? xcd : r) + (blockIdx.x >> 3);
    mt = id % m_tiles;
    nt = id / m_tiles;
  }
  const RowTile rt = row_tile<BM>(a, mt);
  if (rt.first >= rt.end) return;
  const int64_t n0 = static_cast<int64_t>(nt) * BN;
  Y* y = static_cast<Y*>(a.y);
  if (a.offsets && rt.e == a.E) {
    if (a.fill)
      for (int i = threadIdx.x; i < BM * BN; i += 64 * T::kWaves) {
        const int64_t m = rt.first + i / BN, n = n0 + i % BN;
        if (m < rt.end && n < a.N) put(y + m * a.N + n, 0.0f);
      }
    return;
  }
  const int lane = threadIdx.x & 63, wave = uniform(threadIdx.x >> 6), half = lane >> 5;
  const int wx = wave % T::WX, wy = wave / T::WX;

  // Where this lane's copies come from.  A copy lands 1024 bytes in order, so the
  // lane reads the unit that belongs at its place.
  constexpr int BK = T::BK, NS = T::NS, kUnits = BK / 16, C = IX + IW;
  const char *xs[IX], *ws[IW];
#pragma unroll
  for (int i = 0; i < IX; ++i) {
    const int r = T::kRows * (wave * IX + i) + lane / kUnits;
    xs[i] = reinterpret_cast<const char*>(a.x) + row_of(a, min(rt.first + r, rt.end - 1)) * a.pitch + 16 * unit_at<BK>(r, lane % kUnits);
  }
#pragma unroll
  for (int i = 0; i < IW; ++i) {
    const int r = T::kRows * (wave * IW + i) + lane / kUnits;
    ws[i] = reinterpret_cast<const char*>(a.q) + (rt.e * a.N + min(n0 + r, a.N - 1)) * a.pitch + 16 * unit_at<BK>(r, lane % kUnits);
  }
  // Scales and bias are on their way while the products run: a thread fetches one row's or column's.
  static_assert(BM + BN <= 64 * T::kWaves, "one scale a thread");
  // Its row's number comes with those of the copies, and the scale itself is asked for behind the first of
  // them: 512 tokens of 8 of 64 experts 47.0 -> 45.5 us where the copies waited for both.
  const int tid = static_cast<int>(threadIdx.x);
  const int64_t scale_row = row_of(a, min(rt.first + min(tid, BM - 1), rt.end - 1)), scale_n = min(n0 + max(tid - BM, 0), a.N - 1);
  const uint32_t base = lds_addr(lds);
  auto copy = [&](uint32_t stage, int i) {                     // i-th of C
    if (i < IX) {
      copy16(xs[i], base + stage + (wave * IX + i) * 1024);
      xs[i] += BK;
    } else {
      copy16(ws[i - IX], base + stage + BM * BK + (wave * IW + i - IX) * 1024);
      ws[i - IX] += BK;
    }
  };
  const int steps = static_cast<int>(a.pitch / BK);
  i32x16_t acc[MI][NI] = {};
  constexpr int S = BK / 32, R = MI + NI;                      // pieces of 32 bytes in a step, fragments of a piece
  static_assert(S % 2 == 0, "the two sets of fragments change places with every piece");
  i32x4_t fx[2][MI], fw[2][NI];
  // this lane's units of a 32-row block, by piece
  int at[S];
#pragma unroll
  for (int s = 0; s < S; ++s) at[s] = (lane & 31) * BK + 16 * unit_at<BK>(lane & 31, 2 * s + half);
  auto read = [&](uint32_t stage, int s, int set, int i) {     // i-th of R
    const char* tile = lds + stage + at[s];
    if (i < MI) fx[set][i] = *reinterpret_cast<const i32x4_t*>(tile + (wx * T::WM + 32 * i) * BK);
    else fw[set][i - MI] = *reinterpret_cast<const i32x4_t*>(tile + (BM + wy * T::WN + 32 * (i - MI)) * BK);
  };

  // Copies run NS - 1 steps ahead.  Before the last piece of step k is multiplied, step k + 1
  // has landed, for every wave, and every wave is done with step k - 1; from there the
  // first fragments of step k + 1 are read, and step k - 1 + NS is copied over step k - 1.
  // Still in flight are the copies of the steps behind k + 1.
  auto landed = [](bool later) {
    if (later) asm volatile("s_waitcnt vmcnt(%0)\n\ts_barrier" :: "n"((NS - 3) * C) : "memory");
    else asm volatile("s_waitcnt vmcnt(0)\n\ts_barrier" ::: "memory");
  };
  const int ahead = min(steps, NS - 1);
  for (int k = 0; k < ahead; ++k)
#pragma unroll
    for (int i = 0; i < C; ++i) copy(k * T::kStage, i);
  const float early_scale = *(tid < BM ? a.x_scale + scale_row : a.scale + rt.e * a.N + scale_n);
  const float early_bias = a.bias ? a.bias[scale_n] : 0.0f;
  if (steps > 0) {
    if (steps >= NS - 1) asm volatile("s_waitcnt vmcnt(%0)\n\ts_barrier" :: "n"((NS - 2) * C) : "memory");
    else landed(false);
#pragma unroll
    for (int i = 0; i < R; ++i) read(0, 0, 0, i);
  }
  uint32_t stage = 0, before = T::kLds - T::kStage, older = 0;
  // One step, without a branch: the compiler's waits for the fragments are exact only then.
  // The copies of a step are dealt over the pieces from that barrier to the next: the
  // first of them behind it, `rest` in the following step.
  auto step = [&](auto more_steps, auto fetch, auto rest) {
    const uint32_t next = stage + T::kStage == T::kLds ? 0 : stage + T::kStage;
#pragma unroll
    for (int s = 0; s < S; ++s) {
      constexpr int P = MI * NI;                                // products of a piece
      const int set = s & 1;
      const bool last = s == S - 1, more = !last || more_steps;
      if (last && more_steps) landed(fetch);
#pragma unroll
      for (int m = 0; m < P; ++m) {
        // between the products: the next fragments first, then copies
        constexpr int kReads = 2 * P >= R ? 2 : R, kBusy = (R + kReads - 1) / kReads, kLast = kBusy < P ? kBusy : P - 1;
        constexpr int kRest = P - kLast, kPart = (C + S - 1) / S;               // copies of a piece
        if (more)
#pragma unroll
          for (int i = m * kReads; i < (m + 1) * kReads && i < R; ++i) read(last ? next : stage, (s + 1) % S, set ^ 1, i);
        const int part = last ? 0 : (s + 1) * kPart;
        if (m >= kLast && (last ? fetch : rest))
#pragma unroll
          for (int i = (m - kLast) * kPart / kRest; i < (m - kLast + 1) * kPart / kRest && part + i < C; ++i)
            copy(last ? before : older, part + i);
        acc[m / NI][m % NI] = __builtin_amdgcn_mfma_i32_32x32x32_i8(fw[set][m % NI], fx[set][m / NI], acc[m / NI][m % NI], 0, 0, 0);
        __builtin_amdgcn_sched_barrier(0);
      }
    }
    older = before;
    before = stage;
    stage = next;
  };
  constexpr std::true_type yes{};
  constexpr std::false_type no{};
  int k = 0;
  if (NS - 1 < steps) {
    step(yes, yes, no);
    for (k = 1; k + NS - 1 < steps; ++k) step(yes, yes, yes);
    step(yes, no, yes);
    ++k;
  }
  for (; k + 1 < steps; ++k) step(yes, no, no);
  if (k < steps) step(no, no, no);

  // Out through LDS, 32 rows of a wave at a time, so that whole runs of columns are written.
  constexpr int kPitch = T::WN * sizeof(Y) + 16;
  static_assert(T::kWaves * 32 * kPitch <= T::kBytes, "the result's rows fit the stages");
  __syncthreads();
  float* s_scale = reinterpret_cast<float*>(lds + T::kOut);     // of BM rows, BN columns; then the columns' bias
  if (threadIdx.x < BM + BN) s_scale[threadIdx.x] = early_scale;
  if (threadIdx.x >= BM && threadIdx.x < BM + BN) s_scale[BN + threadIdx.x] = early_bias;
  __syncthreads();
  char* mine = lds + wave * 32 * kPitch;
  const int64_t n_wave = n0 + wy * T::WN;
  constexpr int kVec = 16 / sizeof(Y), kLanes = T::WN / kVec;   // lanes that write one row
  const bool whole = a.N % kVec == 0;
#pragma unroll
  for (int i = 0; i < MI; ++i) {
    const int64_t m0 = rt.first + wx * T::WM + 32 * i;
    const float xsc = s_scale[wx * T::WM + 32 * i + (lane & 31)];
#pragma unroll
    for (int j = 0; j < NI; ++j)
#pragma unroll
      for (int g = 0; g < 4; ++g) {
        const float* col = s_scale + BM + wy * T::WN + 32 * j + 8 * g + 4 * half;
        const f32x4_t sc = *reinterpret_cast<const f32x4_t*>(col), b = *reinterpret_cast<const f32x4_t*>(col + BN);
        float v[4];
#pragma unroll
        for (int e = 0; e < 4; ++e) v[e] = static_cast<float>(acc[i][j][4 * g + e]) * sc[e] * xsc + b[e];
        char* to = mine + (lane & 31) * kPitch + (32 * j + 8 * g + 4 * half) * sizeof(Y);
        if constexpr (sizeof(Y) == 4) *reinterpret_cast<f32x4_t*>(to) = f32x4_t{v[0], v[1], v[2], v[3]};
        else *reinterpret_cast<u32x2_t*>(to) = u32x2_t{pack_bf16x2(v[0], v[1]), pack_bf16x2(v[2], v[3])};
      }
    wave_sync();
    for (int r = lane / kLanes; r < 32; r += 64 / kLanes) {
      const int c = lane % kLanes * kVec;
      const u32x4_t v = *reinterpret_cast<const u32x4_t*>(mine + r * kPitch + c * sizeof(Y));
      if (m0 + r >= rt.end || n_wave + c >= a.N) continue;
      Y* to = y + (m0 + r) * a.N + n_wave + c;
      if (whole) {
        *reinterpret_cast<u32x4_t*>(to) = v;
      } else {
        const Y* one = reinterpret_cast<const Y*>(mine + r * kPitch) + c;
        for (int e = 0; e < kVec && n_wave + c + e < a.N; ++e) to[e] = one[e];
      }
    }
    wave_sync();
  }
}

// ---- few rows ----------------------------------------------------------------------

// The weight goes from memory straight into the operands of the products, read once; what
// bounds the kernel are the bytes in flight.  A workgroup's 8 waves take 16 NT channels
// each, or share them over the contraction (every kw-th piece of 128 bytes), and join in LDS.
// Up to 16 MT rows of x stand in the other operand.  (1 x 4096 x 4096 from bf16: 6.2 us, of which the
// bytes take 3.4 and the launch about 2.)
// FUSED: x comes in its own type, few enough bytes (kFusedBytes) for each workgroup to
// quantise all of it into LDS while its first weights are on their way: one launch.
constexpr int kFusedBytes = 16384;
struct FusedX {
  const void* x;
  int64_t stride;
  int K;
  bool bf16, vec;
};

template <int MT, int NT, int U, int EU, bool FUSED, typename Y>
__global__ __launch_bounds__(512, EU) void k_stream(Int8Args a, FusedX fx, int m_tiles, int n_tiles, int kw) {
  extern __shared__ __attribute__((aligned(16))) char lds[];
  constexpr int BM = 16 * MT;
  const int mt = static_cast<int>(blockIdx.x % m_tiles), nt = static_cast<int>(blockIdx.x / m_tiles);
  const int64_t m0 = static_cast<int64_t>(mt) * BM;
  const int lane = threadIdx.x & 63, wave = uniform(threadIdx.x >> 6);
  const int nw = 8 / kw, wn = wave / kw, wk = wave % kw;        // groups of channels, this wave's, its share of K
  const int64_t n0 = (static_cast<int64_t>(nt) * nw + wn) * 16 * NT;
  Y* y = static_cast<Y*>(a.y);
  const int blocks = static_cast<int>(a.pitch / 128), row = lane & 15, part = lane >> 4;
  const char *wp[NT], *xp[MT];
  int xat[MT];
#pragma unroll
  for (int j = 0; j < NT; ++j)
    wp[j] = reinterpret_cast<const char*>(a.q) + min(n0 + 16 * j + row, a.N - 1) * a.pitch + 16 * part;
  const int lds_pitch = static_cast<int>(a.pitch) + 16;
#pragma unroll
  for (int i = 0; i < MT; ++i) {
    const int64_t r = min(m0 + 16 * i + row, a.M - 1);
    if constexpr (FUSED) xat[i] = static_cast<int>(r) * lds_pitch + 16 * part;
    else xp[i] = reinterpret_cast<const char*>(a.x) + r * a.pitch + 16 * part;
  }

  i32x4_t w[2][U][NT][2], x[2][U][FUSED ? 1 : MT][2];
  auto load = [&](int set, int b) {
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const int64_t at = static_cast<int64_t>(min(b + u * kw, blocks - 1)) * 128;
#pragma unroll
      for (int h = 0; h < 2; ++h) {
#pragma unroll
        for (int j = 0; j < NT; ++j) w[set][u][j][h] = *reinterpret_cast<const i32x4_t*>(wp[j] + at + 64 * h);
        if constexpr (!FUSED)
#pragma unroll
          for (int i = 0; i < MT; ++i) x[set][u][i][h] = *reinterpret_cast<const i32x4_t*>(xp[i] + at + 64 * h);
      }
    }
  };
  i32x4_t acc[MT][NT] = {};
  auto multiply = [&](int set, int b) {
#pragma unroll
    for (int u = 0; u < U; ++u) {
      if (b + u * kw >= blocks) break;
#pragma unroll
      for (int h = 0; h < 2; ++h)
#pragma unroll
        for (int i = 0; i < MT; ++i) {
          i32x4_t xv;
          if constexpr (FUSED) xv = *reinterpret_cast<const i32x4_t*>(lds + xat[i] + (b + u * kw) * 128 + 64 * h);
          else xv = x[set][u][i][h];
#pragma unroll
          for (int j = 0; j < NT; ++j) acc[i][j] = __builtin_amdgcn_mfma_i32_16x16x64_i8(w[set][u][j][h], xv, acc[i][j], 0, 0, 0);
        }
    }
  };

  float* s_scale = reinterpret_cast<float*>(lds + (FUSED ? a.x_rows * lds_pitch : 0));
  if constexpr (!FUSED) {
    if (blocks > 0) load(0, wk);
  } else {
    // 8 elements at a time, at most kFusedBytes / 8 of them; 16 neighbouring lanes are in one row
    constexpr int kMost = kFusedBytes / 8 / 512;
    const int vecs = static_cast<int>(a.pitch / 8), all = static_cast<int>(a.x_rows) * vecs;
    uint32_t* s_top = reinterpret_cast<uint32_t*>(s_scale);
    for (int i = threadIdx.x; i < a.x_rows; i += 512) s_top[i] = 0;
    __syncthreads();
    auto body = [&](auto type, auto vec) {
      using T = decltype(type);
      float f[kMost][8];
      int at[kMost], of[kMost];
#pragma unroll
      for (int j = 0; j < kMost; ++j) {
        const int v = j * 512 + threadIdx.x;
        of[j] = v < all ? v / vecs : -1;
        at[j] = (v - of[j] * vecs) * 8;
        if (of[j] >= 0) load8<vec>(static_cast<const T*>(fx.x) + of[j] * fx.stride, at[j], fx.K, f[j]);
      }
      // loads come back in order: the weights behind x, so that x can be waited for alone
      __builtin_amdgcn_sched_barrier(0);
      load(0, wk);
      __builtin_amdgcn_sched_barrier(0);
#pragma unroll
      for (int j = 0; j < kMost; ++j) {
        if (of[j] < 0) continue;
        const uint32_t top = row_max(largest_of(f[j], 0));
        if ((lane & 15) == 0) atomicMax(&s_top[of[j]], top);    // (the largest of integers: in any order)
      }
      __syncthreads();
      float scale[kMost];
#pragma unroll
      for (int j = 0; j < kMost; ++j) {
        if (of[j] < 0) continue;
        const RowScale sc = row_scale(s_top[of[j]]);
        scale[j] = sc.scale;
        *reinterpret_cast<u32x2_t*>(lds + of[j] * lds_pitch + at[j]) = round8<T>(f[j], sc);
      }
      __syncthreads();
#pragma unroll
      for (int j = 0; j < kMost; ++j)
        if (of[j] >= 0 && at[j] == 0) s_scale[of[j]] = scale[j];
    };
    if (fx.bf16) fx.vec ? body(uint16_t{}, std::true_type{}) : body(uint16_t{}, std::false_type{});
    else fx.vec ? body(float{}, std::true_type{}) : body(float{}, std::false_type{});
    __syncthreads();
  }
  for (int b = wk; b < blocks; b += 2 * U * kw) {
    if (b + U * kw < blocks) load(1, b + U * kw);
    multiply(0, b);
    if (b + 2 * U * kw < blocks) load(0, b + 2 * U * kw);
    if (b + U * kw < blocks) multiply(1, b + U * kw);
  }

  // Join: lane (m = lane & 15, channels 4 (lane >> 4) + i) of every wave.  (Sums of
  // integers: their order does not matter.)
  i32x4_t* s_acc = reinterpret_cast<i32x4_t*>(lds + (FUSED ? (a.x_rows * (lds_pitch + 4) + 15) / 16 * 16 : 0));
  constexpr int kTiles = MT * NT;
  if (kw > 1) {
#pragma unroll
    for (int i = 0; i < MT; ++i)
#pragma unroll
      for (int j = 0; j < NT; ++j) s_acc[(wave * kTiles + i * NT + j) * 64 + lane] = acc[i][j];
    __syncthreads();
  }
#pragma unroll
  for (int t = 0; t < kTiles; ++t) {
    if (t % kw != wk) continue;                                 // the group's waves share its tiles
    i32x4_t sum = acc[t / NT][t % NT];
    if (kw > 1) {
      sum = i32x4_t{0, 0, 0, 0};
      for (int k = 0; k < kw; ++k) sum += s_acc[((wn * kw + k) * kTiles + t) * 64 + lane];
    }
    const int64_t m = m0 + 16 * (t / NT) + row, n = n0 + 16 * (t % NT) + 4 * part;
    if (m >= a.M || n >= a.N) continue;
    float xsc;
    if constexpr (FUSED) xsc = s_scale[m];
    else xsc = a.x_scale[m];
    float v[4];
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      const int64_t c = min(n + e, a.N - 1);
      v[e] = static_cast<float>(sum[e]) * a.scale[c] * xsc + (a.bias ? a.bias[c] : 0.0f);
    }
    Y* to = y + m * a.N + n;
    if (a.N % 4 == 0) {
      if constexpr (sizeof(Y) == 4) *reinterpret_cast<f32x4_t*>(to) = f32x4_t{v[0], v[1], v[2], v[3]};
      else *reinterpret_cast<u32x2_t*>(to) = u32x2_t{pack_bf16x2(v[0], v[1]), pack_bf16x2(v[2], v[3])};
    } else {
#pragma unroll
      for (int e = 0; e < 4; ++e)
        if (n + e < a.N) put(to + e, v[e]);
    }
  }
}

// Waves that share a workgroup's contraction.
int stream_split(const Int8Args& a) {
  const int blocks = static_cast<int>(a.pitch / 128);
  return blocks >= 8 ? 8 : blocks >= 4 ? 4 : blocks >= 2 ? 2 : 1;
}

template <int MT, int NT, int U, int EU>
hipError_t launch_stream(const Int8Args& a, const FusedX* fx, hipStream_t stream) {
  const int kw = stream_split(a);
  const int64_t m_tiles = row_tiles(a, 16 * MT), cols = 8 / kw * 16 * NT, n_tiles = (a.N + cols - 1) / cols;
  const size_t held = fx ? (a.x_rows * (a.pitch + 20) + 15) / 16 * 16 : 0, bytes = held + (kw > 1 ? 8 * MT * NT * 1024 : 0);
  auto go = [&](auto kernel) {
    constexpr auto launch = decltype(kernel)::launch;
    allow_lds<launch>();
    launch<<<static_cast<uint32_t>(m_tiles * n_tiles), 512, bytes, stream>>>(a, fx ? *fx : FusedX{}, static_cast<int>(m_tiles),
                                                                              static_cast<int>(n_tiles), kw);
    return hipGetLastError();
  };
  if (fx) return a.bf16 ? go(Kernel<k_stream<MT, NT, U, EU, true, uint16_t>>{}) : go(Kernel<k_stream<MT, NT, U, EU, true, float>>{});
  return a.bf16 ? go(Kernel<k_stream<MT, NT, U, EU, false, uint16_t>>{}) : go(Kernel<k_stream<MT, NT, U, EU, false, float>>{});
}

template <typename T>
hipError_t launch_tile(const Int8Args& a, hipStream_t stream) {
  int64_t m_tiles = row_tiles(a, T::BM);
  const int64_t n_tiles = (a.N + T::BN - 1) / T::BN;
  if (a.offsets) m_tiles = (m_tiles + 7) / 8 * 8;
  auto go = [&](auto kernel) {
    constexpr auto launch = decltype(kernel)::launch;
    allow_lds<launch>();
    launch<<<static_cast<uint32_t>(m_tiles * n_tiles), 64 * T::kWaves, T::kBytes, stream>>>(a, static_cast<int>(m_tiles), static_cast<int>(n_tiles));
    return hipGetLastError();
  };
  return a.bf16 ? go(Kernel<k_tile<T, uint16_t>>{}) : go(Kernel<k_tile<T, float>>{});
}

}  // namespace

hipError_t launch_int8_quantize(const void* x, bool bf16, int64_t stride, int64_t M, int64_t K, int8_t* q, float* scale,
                                hipStream_t stream) {
  const int pitch = static_cast<int>(int8_row_bytes(K)), n = static_cast<int>(K);
  const bool vec = (reinterpret_cast<uintptr_t>(x) & 15) == 0 && (M == 1 || stride * (bf16 ? 2 : 4) % 16 == 0);
  if (bf16) {
    const uint16_t* p = static_cast<const uint16_t*>(x);
    return vec ? launch_quantize_t<uint16_t, true>(p, stride, M, n, pitch, q, scale, stream)
               : launch_quantize_t<uint16_t, false>(p, stride, M, n, pitch, q, scale, stream);
  }
  const float* p = static_cast<const float*>(x);
  return vec ? launch_quantize_t<float, true>(p, stride, M, n, pitch, q, scale, stream)
             : launch_quantize_t<float, false>(p, stride, M, n, pitch, q, scale, stream);
}

namespace {

using Tile64 = Tile<64, 64, 2, 2, 128, 5>;
using Tile128x64 = Tile<128, 64, 4, 2, 128, 6>;
using Tile128 = Tile<128, 128, 2, 4, 128, 5>;
using Tile128Pair = Tile<128, 128, 2, 4, 64, 5>;               // two workgroups a compute unit
using Tile256x128 = Tile<256, 128, 4, 2, 64, 6>;
using Tile256 = Tile<256, 256, 2, 4, 64, 5>;

// Which kernel takes the call, by the rounds of its tiles over the chip and what a
// round costs (a.pitch counts for all of them alike).  Costs of a round beside each other, from
// 4096-wide x on one card, with its quantising; behind them the products alone, on another card:
//   64 x 64      13   256 x 4096   12.7 us  11.1    128 x 128   33   1024 x 4096  24.5 us  21.3
//   128 x 64     20   512 x 4096   16.4 us  14.7    256 x 128   63   2048 x 4096  42.5 us  40.9
//   256 x 256    96   4096 x 4096  65 us  62.4 (2200 TOP/s; 94 us in 128 x 128, 82 in 256 x 128)
// Small sizes keep the chip busy only in small tiles (512 x 4096: 128 x 64 14.7 us, 128 x
// 128 16.5, 256 x 256 41), large ones reread too much in them.  No choice cuts the contraction: from
// 65 rows on a product of few channels leaves most of the chip idle (128 x 1024 x 4096: 32 workgroups, 9.5 us;
// 128 x 4096 x 14336: 128 of them, 25.5 us, of which the bytes take 12.7).  Grouped calls do not know their
// tiles here: a part of a tile is lost for every expert.  Their costs are of rounds of experts' tiles,
// which read other weights each: 512 tokens of 2 of 8 experts 14336 wide take 146 us in 128 x 128, 166 in
// the 64 x 64 that the costs of the plain product choose.
struct TileShape {
  int bm, bn, cost;
};
constexpr TileShape kShapes[] = {{64, 64, 13}, {128, 64, 20}, {128, 128, 33}, {256, 128, 63}, {256, 256, 96}};
constexpr TileShape kGroupedShapes[] = {{64, 64, 17}, {0, 0, 0}, {128, 128, 40}, {0, 0, 0}, {256, 256, 97}};

int best_shape(const Int8Args& a, int cus) {
  int best = 0;
  double least = 0.0;
  for (int i = 0; i < 5; ++i) {
    const TileShape& t = a.offsets ? kGroupedShapes[i] : kShapes[i];
    if (!t.bm) continue;
    double rows = static_cast<double>((a.M + t.bm - 1) / t.bm);
    if (a.offsets) {
      const double experts = static_cast<double>(a.E < a.M ? a.E : a.M), each = static_cast<double>(a.M) / experts / t.bm + 0.5;
      rows = experts * (each < 1.1 ? 1.1 : each);
    }
    const double cost = std::ceil(rows * static_cast<double>((a.N + t.bn - 1) / t.bn) / cus) * t.cost;
    if (i == 0 || cost < least) best = i, least = cost;
  }
  return best;
}

// The few-row kernel reads its weights once for 16 or 32 rows, straight from memory, and cuts K
// eight ways: it takes up to 16 rows (1 x 4096 x 4096: 6.2 us for 9.5 in tiles, without quantising), and
// up to 64 where tiles would fill less than half of the chip (32 x 4096 x 4096: 8.4 for 9.7; 64 x 1024 x
// 4096: 6.4 for 9.4, x 14336: 15.4 for 25.2; 64 x 2048 x 4096: 8.4 for 9.6; not 32 x 14336 x 4096: 17.7 for
// 11.7).  Where this is not the faster one: above 32 rows, whose weights it reads twice, from 4096 channels on
// (64 x 4096 x 4096: 12.4 for 9.9, 64 x 8000 x 4096: 19.6 for 10.0), and in the largest products (16 x 14336 x 4096:
// 12.6 for 11.4, 32 x 5120 x 27648: 76.9 for 60.9).
bool few_rows(const Int8Args& a, int cus) {
  if (a.offsets) return false;
  return a.M <= 16 || (a.M <= 64 && (a.N + 63) / 64 < cus / 2);
}
// Channels and rows of a workgroup: the most that leave seven eighths of the chip busy
// (4096 channels: 16 a workgroup, 6.1 us for 7.7 with 32; 14336: 64, 15.6 for 21.3 with 16 at 16 rows).
hipError_t launch_few_rows(const Int8Args& a, const FusedX* fx, int cus, hipStream_t stream) {
  const int groups = 8 / stream_split(a);
  auto fills = [&](int mt, int nt) {
    return row_tiles(a, 16 * mt) * ((a.N + 16 * nt * groups - 1) / (16 * nt * groups)) * 8 >= static_cast<int64_t>(cus) * 7;
  };
  if (a.M > 16) {
    if (fills(2, 2)) return launch_stream<2, 2, 1, 4>(a, fx, stream);
    if (fills(2, 1)) return launch_stream<2, 1, 2, 1>(a, fx, stream);
    return launch_stream<1, 1, 2, 1>(a, fx, stream);
  }
  if (fills(1, 4)) return launch_stream<1, 4, 1, 4>(a, fx, stream);
  if (fills(1, 2)) return launch_stream<1, 2, 2, 1>(a, fx, stream);
  return launch_stream<1, 1, 2, 1>(a, fx, stream);
}

}  // namespace

// One launch pays while the x that every workgroup quantises for itself is small: one
// row (1 x 4096 x 4096: 6.8 us for 9.7 in two), or two of 4096 (7.7 for 9.7; four: 11.0 for 9.7).
bool int8_fused(const Int8Args& a) {
  if (a.pitch == 0 || a.x_rows * a.pitch > (a.x_rows == 1 ? kFusedBytes : kFusedBytes / 2)) return false;
  return few_rows(a, device_cu_count());
}

hipError_t launch_int8_matmul(const Int8Args& a, const Int8Source* source, hipStream_t stream) {
  const int cus = device_cu_count();
  if (few_rows(a, cus)) {
    if (!source) return launch_few_rows(a, nullptr, cus, stream);
    const int64_t size = source->bf16 ? 2 : 4;
    const bool vec = (reinterpret_cast<uintptr_t>(source->x) & 15) == 0 && (a.x_rows == 1 || source->stride * size % 16 == 0);
    const FusedX fx{source->x, source->stride, source->K, source->bf16, vec};
    return launch_few_rows(a, &fx, cus, stream);
  }
  switch (best_shape(a, cus)) {
    case 0: return launch_tile<Tile64>(a, stream);
    case 1: return launch_tile<Tile128x64>(a, stream);
    case 2: return a.offsets ? launch_tile<Tile128Pair>(a, stream) : launch_tile<Tile128>(a, stream);
    case 3: return launch_tile<Tile256x128>(a, stream);
    default: return launch_tile<Tile256>(a, stream);
  }
}

// Workgroups of the call with the most.
bool int8_launchable(int64_t M, int64_t N, int32_t E) {
  Int8Args a{};
  const int32_t none = 0;
  a.M = M, a.N = N, a.E = E, a.offsets = E ? &none : nullptr;
  return (row_tiles(a, 64) + 8) * ((N + 63) / 64) <= UINT32_MAX / 512;
}

}  // namespace nf4
