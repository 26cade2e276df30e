// E4M3 values with one FP32 scale for a vector of them (a block of 128 columns
// of a row, a token's head): scale = max(max |v| / 448, 2^-100), q = e4m3(v / scale).
//
// The floor keeps the scale and its reciprocal normal numbers, and the scale of
// a vector of zeros small beside any other. A vector that holds an infinity or
// a NaN gets that as its scale, so all of it decodes to NaN.
#pragma once

#include <cuda_runtime.h>
#include <stdint.h>

namespace afd {

constexpr float kE4m3Max = 448.f;
constexpr float kSmallestScale = 7.888609052210118e-31f;  // 2^-100

// The largest magnitude as bits, which order NaN above infinity above the rest.
__device__ __forceinline__ uint32_t absmax8(const float (&v)[8]) {
  uint32_t m = 0;
#pragma unroll
  for (int e = 0; e < 8; ++e) m = max(m, __float_as_uint(v[e]) & 0x7fffffffu);
  return m;
}

// ... over groups of LANES lanes.
template <int LANES>
__device__ __forceinline__ uint32_t lanes_absmax(uint32_t m) {
#pragma unroll
  for (int d = LANES / 2; d; d >>= 1) m = max(m, __shfl_xor_sync(0xffffffffu, m, d));
  return m;
}

// (A product with 1 / 448: at most a step of FP32 from the quotient.)
__device__ __forceinline__ float block_scale(uint32_t absmax) {
  const float s = __uint_as_float(absmax) * (1.f / kE4m3Max);
  return s < kSmallestScale ? kSmallestScale : s;  // (a NaN stays)
}

// Two floats rounded to nearest even E4M3 (448 at most), `lo` in the low byte.
__device__ __forceinline__ uint32_t pack_e4m3(float lo, float hi) {
  uint16_t r;
  asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(r) : "f"(hi), "f"(lo));
  return r;
}

// v / scale as v * (1 / scale), at most 2^-23 off. That moves a value in a hundred
// thousand to its E4M3 neighbour, for values that are FP32 results; quotients of
// BF16 values often lie on a tie (one in a few hundred), so those are divided.
__device__ __forceinline__ uint2 to_e4m3x8(const float (&v)[8], float inv) {
  return make_uint2(pack_e4m3(v[0] * inv, v[1] * inv) | pack_e4m3(v[2] * inv, v[3] * inv) << 16,
                    pack_e4m3(v[4] * inv, v[5] * inv) | pack_e4m3(v[6] * inv, v[7] * inv) << 16);
}

__device__ __forceinline__ uint2 divided_e4m3x8(const float (&v)[8], float scale) {
  return make_uint2(pack_e4m3(v[0] / scale, v[1] / scale) | pack_e4m3(v[2] / scale, v[3] / scale) << 16,
                    pack_e4m3(v[4] / scale, v[5] / scale) | pack_e4m3(v[6] / scale, v[7] / scale) << 16);
}

}  // namespace afd
