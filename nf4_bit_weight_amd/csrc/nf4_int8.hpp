// Launch interface of the products in 8-bit integers (nf4_int8.hip), between the
// C ABI of nf4_int8.h and the kernels.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

namespace nf4 {

constexpr int64_t int8_row_bytes(int64_t K) { return (K + 127) / 128 * 128; }

struct Int8Args {
  const int8_t* x;           // rows of `pitch` bytes, 16-byte aligned
  const float* x_scale;
  int64_t x_rows;
  const int32_t* tokens;     // NULL: row r reads row r
  const int32_t* offsets;    // NULL: one weight for all rows
  int32_t E;
  int64_t M, N, pitch;       // pitch = int8_row_bytes(K)
  const int8_t* q;
  const float* scale;
  const float* bias;
  void* y;
  bool bf16, fill;
};

hipError_t launch_int8_quantize(const void* x, bool bf16, int64_t stride, int64_t M, int64_t K, int8_t* q, float* scale,
                                hipStream_t stream);
// x before it is quantised
struct Int8Source {
  const void* x;
  bool bf16;
  int64_t stride;
  int32_t K;
};
bool int8_launchable(int64_t M, int64_t N, int32_t E);
// Whether the product quantises x itself (source given; a.x and a.x_scale are not read).
bool int8_fused(const Int8Args& a);
hipError_t launch_int8_matmul(const Int8Args& a, const Int8Source* source, hipStream_t stream);

}  // namespace nf4
