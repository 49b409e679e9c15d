// Products in 8-bit integers with a scale for each token and each channel
// (nf4_int8.h).
#include <cmath>

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

// ---- rows of integers --------------------------------------------------------------

// The integer nearest to 127 x / top, half-way to even.  A rounded quotient is at
// most one off; 127 x - q top then says on which side of the middle x lies.  In 64
// bits both products are exact (7 + 24 bits).
__device__ __forceinline__ int nearest(float x, float top, float inverse) {
  float q = rintf(x * inverse);
  const double rest = fma(-static_cast<double>(q), static_cast<double>(top), 127.0 * static_cast<double>(x));
  const double half = 0.5 * static_cast<double>(top);
  const bool odd = (static_cast<int>(q) & 1) != 0;
  if (rest > half || (rest == half && odd)) q += 1.0f;
  else if (rest < -half || (rest == -half && odd)) q -= 1.0f;
  return static_cast<int>(q);
}

// A workgroup a row.
template <typename T>
__global__ __launch_bounds__(256) void k_quantize(const T* x, int64_t stride, int64_t K, int64_t pitch, int8_t* q, float* scale) {
  __shared__ float s_top[4];
  __shared__ int s_bad[4];
  const T* row = x + blockIdx.x * stride;
  int8_t* out = q + blockIdx.x * pitch;
  float top = 0.0f;
  bool bad = false;
  for (int64_t i = threadIdx.x; i < K; i += 256) {
    const float v = fabsf(value(row + i));
    bad |= !(v < INFINITY);
    top = fmaxf(top, v);
  }
#pragma unroll
  for (int m = 1; m < 64; m <<= 1) top = fmaxf(top, __shfl_xor(top, m, 64));
  const bool any = __ballot(bad) != 0;
  if ((threadIdx.x & 63) == 0) s_top[threadIdx.x >> 6] = top, s_bad[threadIdx.x >> 6] = any;
  __syncthreads();
  top = fmaxf(fmaxf(s_top[0], s_top[1]), fmaxf(s_top[2], s_top[3]));
  bad = s_bad[0] | s_bad[1] | s_bad[2] | s_bad[3];
  const bool live = !bad && top >= 0x1p-119f;
  const float inverse = 127.0f / top;
  for (int64_t i = threadIdx.x; i < pitch; i += 256)
    out[i] = live && i < K ? static_cast<int8_t>(nearest(value(row + i), top, inverse)) : 0;
  if (threadIdx.x == 0) scale[blockIdx.x] = bad ? NAN : live ? top / 127.0f : 0.0f;
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
  const int lane = static_cast<int>(threadIdx.x & 63);
  int before = 0;
  for (int e0 = 0; e0 <= a.E; e0 += 64) {
    const int e = e0 + lane;
    int64_t lo = 0, hi = 0;
    if (e <= a.E) {
      lo = a.offsets[e];
      hi = e < a.E ? a.offsets[e + 1] : a.M;
      lo = lo < 0 ? 0 : (lo > a.M ? a.M : lo);
      hi = hi < lo ? lo : (hi > a.M ? a.M : hi);
    }
    const int tiles = static_cast<int>((hi - lo + BM - 1) / BM);
    int incl = tiles;
#pragma unroll
    for (int d = 1; d < 64; d <<= 1) {
      const int o = __shfl_up(incl, d, 64);
      if (lane >= d) incl += o;
    }
    const int at = before + incl - tiles;
    const unsigned long long hit = __ballot(mt >= at && mt < before + incl);
    if (hit) {
      const int l = __ffsll(static_cast<long long>(hit)) - 1;
      return {__shfl(lo, l, 64) + static_cast<int64_t>(mt - __shfl(at, l, 64)) * BM, __shfl(hi, l, 64), e0 + l};
    }
    before += __shfl(incl, 63, 64);
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

constexpr int kBK = 128;                                       // bytes of a row in one step
// 16-byte unit u of row r of a tile stands at unit u ^ ((r >> 1) & 7).
__device__ __forceinline__ int swz(int r, int u) { return r * kBK + ((u ^ ((r >> 1) & 7)) << 4); }

// 64 x 64 of y: four waves, each 32 x 32.
template <typename Y>
__global__ __launch_bounds__(256) void k_tile(Int8Args a) {
  __shared__ __attribute__((aligned(16))) char s_x[64 * kBK], s_w[64 * kBK];
  const RowTile rt = row_tile<64>(a, blockIdx.y);
  if (rt.first >= rt.end) return;
  const int64_t n0 = static_cast<int64_t>(blockIdx.x) * 64;
  Y* y = static_cast<Y*>(a.y);
  if (rt.e == a.E && a.offsets) {
    if (a.fill)
      for (int i = threadIdx.x; i < 64 * 64; i += 256) {
        const int64_t m = rt.first + i / 64, n = n0 + i % 64;
        if (m < rt.end && n < a.N) put(y + m * a.N + n, 0.0f);
      }
    return;
  }
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6, half = lane >> 5;
  const int wm = 32 * (wave & 1), wn = 32 * (wave >> 1);
  const int r = threadIdx.x >> 2, u = 2 * (threadIdx.x & 3);    // this thread copies two units of a row of each tile
  const int64_t xm = row_of(a, min(rt.first + r, rt.end - 1));
  const int8_t* xp = a.x + xm * a.pitch + 16 * u;
  const int8_t* wp = a.q + (rt.e * a.N + min(n0 + r, a.N - 1)) * a.pitch + 16 * u;
  i32x16_t acc = {};
  for (int64_t k = 0; k < a.pitch; k += kBK) {
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      *reinterpret_cast<i32x4_t*>(s_x + swz(r, u + i)) = *reinterpret_cast<const i32x4_t*>(xp + k + 16 * i);
      *reinterpret_cast<i32x4_t*>(s_w + swz(r, u + i)) = *reinterpret_cast<const i32x4_t*>(wp + k + 16 * i);
    }
    __syncthreads();
#pragma unroll
    for (int s = 0; s < 4; ++s) {
      const i32x4_t xv = *reinterpret_cast<const i32x4_t*>(s_x + swz(wm + (lane & 31), 2 * s + half));
      const i32x4_t wv = *reinterpret_cast<const i32x4_t*>(s_w + swz(wn + (lane & 31), 2 * s + half));
      acc = __builtin_amdgcn_mfma_i32_32x32x32_i8(xv, wv, acc, 0, 0, 0);
    }
    __syncthreads();
  }
  // a lane holds rows 8 (i / 4) + 4 half + i % 4 of column lane & 31
  const int64_t n = n0 + wn + (lane & 31);
  if (n >= a.N) return;
  const float sw = a.scale[rt.e * a.N + n], b = a.bias ? a.bias[n] : 0.0f;
#pragma unroll
  for (int i = 0; i < 16; ++i) {
    const int64_t m = rt.first + wm + 8 * (i / 4) + 4 * half + i % 4;
    if (m < rt.end) put(y + m * a.N + n, static_cast<float>(acc[i]) * sw * a.x_scale[row_of(a, m)] + b);
  }
}

}  // namespace

hipError_t launch_int8_quantize(const void* x, bool bf16, int64_t stride, int64_t M, int64_t K, int8_t* q, float* scale,
                                hipStream_t stream) {
  const int64_t pitch = int8_row_bytes(K);
  if (bf16) k_quantize<<<M, 256, 0, stream>>>(static_cast<const uint16_t*>(x), stride, K, pitch, q, scale);
  else k_quantize<<<M, 256, 0, stream>>>(static_cast<const float*>(x), stride, K, pitch, q, scale);
  return hipGetLastError();
}

hipError_t launch_int8_matmul(const Int8Args& a, hipStream_t stream) {
  const dim3 grid(static_cast<uint32_t>((a.N + 63) / 64), static_cast<uint32_t>(row_tiles(a, 64)));
  if (a.bf16) k_tile<uint16_t><<<grid, 256, 0, stream>>>(a);
  else k_tile<float><<<grid, 256, 0, stream>>>(a);
  return hipGetLastError();
}

}  // namespace nf4
