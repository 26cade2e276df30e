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

__device__ __forceinline__ uint2 divided_e4m3x8(const float (&v)[8], float scale) {
  return make_uint2(pack_e4m3(v[0] / scale, v[1] / scale) | pack_e4m3(v[2] / scale, v[3] / scale) << 16,
                    pack_e4m3(v[4] / scale, v[5] / scale) | pack_e4m3(v[6] / scale, v[7] / scale) << 16);
}

// The same quotients where eight divisions cost more than the rest: the product with
// the rounded reciprocal, corrected by its remainder, which an FMA gives exactly, is the
// rounded quotient (P. W. Markstein, Computation of elementary functions on the IBM RISC
// System/6000 processor, IBM J. Res. Dev. 34, 1990). The remainder is exact while its
// last digit, the quotient's times the scale's, is 2^-149 or more: from scales of 2^-92 on,
// as quotients below 2^-10 all go to zero. Where the scale is below 2^-90 both sides are
// multiplied by 2^64.
// Norm of 4,096 rows of 4,096: 24.3 us, 27.9 with divisions, 25.9 with divisions for the
// small scales alone; 23.9 with the product alone, which put one value in 40,000 on the
// wrong side of a border.
__device__ __forceinline__ uint2 quotient_e4m3x8(const float (&v)[8], float scale) {
  const float up = scale < 8.077935669463161e-28f ? 18446744073709551616.f : 1.f;
  const float s = scale * up, inv = 1.f / s;
  float q[8];
#pragma unroll
  for (int e = 0; e < 8; ++e) {
    const float y = v[e] * up, near = y * inv;
    q[e] = fmaf(-fmaf(near, s, -y), inv, near);  // (so ordered, a zero keeps its sign)
  }
  return make_uint2(pack_e4m3(q[0], q[1]) | pack_e4m3(q[2], q[3]) << 16, pack_e4m3(q[4], q[5]) | pack_e4m3(q[6], q[7]) << 16);
}

}  // namespace afd
