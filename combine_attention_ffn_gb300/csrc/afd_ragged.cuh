// Rows grouped by expert (afd_recv): expert l's rows are
// [align_up(ends[l-1], alpha), ends[l]), ends[-1] = 0.
#pragma once

#include <stdint.h>

#include "afd_internal.cuh"

namespace afd {

// Start of a group given the end of the one before it, both clamped to the
// number of rows (so that no bad end reaches past the buffers, and the
// rounding up cannot pass 32 bits: num_rows + alpha <= INT32_MAX).
__device__ __forceinline__ int group_start(int end_before, int alpha, int num_rows) {
  const int e = min(max(end_before, 0), num_rows);
  return (alpha & (alpha - 1)) == 0 ? (e + alpha - 1) & -alpha : (e + alpha - 1) / alpha * alpha;
}

__device__ __forceinline__ int group_end(int end, int num_rows) { return min(max(end, 0), num_rows); }

// 16 bytes of BF16 as eight floats and back.
__device__ __forceinline__ void bf16x8_to_float(const uint4& v, float (&f)[8]) {
  const uint32_t u[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    f[2 * i] = __uint_as_float(u[i] << 16);
    f[2 * i + 1] = __uint_as_float(u[i] & 0xffff0000u);
  }
}

// Two floats rounded to nearest even, `lo` in the low half.
__device__ __forceinline__ uint32_t pack_bf16(float lo, float hi) {
  uint32_t r;
  asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
  return r;
}

__device__ __forceinline__ uint4 float_to_bf16x8(const float (&f)[8]) {
  return make_uint4(pack_bf16(f[0], f[1]), pack_bf16(f[2], f[3]), pack_bf16(f[4], f[5]), pack_bf16(f[6], f[7]));
}

// silu(g) * u = g * u / (1 + exp(-g)), with t = exp(-|g|) <= 1 so that nothing
// overflows on the way: 1 / (1 + t) or t / (1 + t). The fast exponential errs
// by about 2^-21 + |g| 2^-24 relative, far below the BF16 rounding that follows.
__device__ __forceinline__ float silu_mul(float g, float u) {
  const float t = __expf(-fabsf(g));
  return __fdividef(g >= 0.0f ? g : g * t, 1.0f + t) * u;
}

}  // namespace afd
