// afd_grouped_linear: the experts' matrix product over received rows.

#include <cuda_runtime.h>
#include <stdint.h>

#include <climits>

#include "afd.h"
#include "afd_device.cuh"
#include "afd_pointers.cuh"
#include "afd_ragged.cuh"

namespace {

struct ExpertParams {
  const uint8_t* x;
  int64_t x_stride;
  const float* x_scale;
  const uint8_t* w;
  const float* w_scale;
  const int32_t* ends;
  int32_t G, alpha, R, K, N, gated;
  uint16_t* out;
  int64_t out_stride;
  int32_t* error;
};

template <bool FP8>
__device__ __forceinline__ float element(const uint8_t* p, int64_t i) {
  if (FP8) {
    uint32_t h;
    asm("{ .reg .b16 t; cvt.u16.u32 t, %1; cvt.rn.f16x2.e4m3x2 %0, t; }" : "=r"(h) : "r"((uint32_t)p[i]));
    float f;
    asm("{ .reg .b16 lo, hi; mov.b32 {lo, hi}, %1; cvt.f32.f16 %0, lo; }" : "=f"(f) : "r"(h));
    return f;
  }
  return __uint_as_float((uint32_t) reinterpret_cast<const uint16_t*>(p)[i] << 16);
}

// 64 rows x 64 columns a block, 4 x 4 sums a thread, 32 of K at a time.
template <bool FP8>
__global__ void __launch_bounds__(256) grouped_simple_kernel(const ExpertParams p) {
  __shared__ float xs[32][65], ws[2][32][65];
  const int n0 = blockIdx.x * 64, g = blockIdx.y;
  const int start = g ? afd::group_start(p.ends[g - 1], p.alpha, p.R) : 0, end = afd::group_end(p.ends[g], p.R);
  const int W = p.gated ? 2 * p.N : p.N, halves = p.gated ? 2 : 1;
  const int tx = threadIdx.x & 15, ty = threadIdx.x >> 4;
  for (int r0 = start + blockIdx.z * 64; r0 < end; r0 += gridDim.z * 64) {
    float acc[2][4][4] = {};
    for (int k0 = 0; k0 < p.K; k0 += 32) {
      for (int i = threadIdx.x; i < 64 * 32; i += 256) {
        const int k = k0 + (i & 31), r = r0 + (i >> 5), n = n0 + (i >> 5);
        float v = 0.f;
        if (k < p.K && r < end) {
          v = element<FP8>(p.x, r * p.x_stride + k);
          if (FP8) v *= p.x_scale[(int64_t)r * (p.K / 128) + k / 128];
        }
        xs[i & 31][i >> 5] = v;
        for (int h = 0; h < halves; ++h) {
          float u = 0.f;
          if (k < p.K && n < p.N) {
            const int64_t row = (int64_t)g * W + h * p.N + n;
            u = element<FP8>(p.w, row * p.K + k);
            if (FP8) u *= p.w_scale[row / 128 * (p.K / 128) + k / 128];
          }
          ws[h][i & 31][i >> 5] = u;
        }
      }
      __syncthreads();
      for (int k = 0; k < 32; ++k)
        for (int h = 0; h < halves; ++h)
          for (int i = 0; i < 4; ++i)
            for (int j = 0; j < 4; ++j) acc[h][i][j] = fmaf(xs[k][ty * 4 + i], ws[h][k][tx * 4 + j], acc[h][i][j]);
      __syncthreads();
    }
    for (int i = 0; i < 4; ++i)
      for (int j = 0; j < 4; ++j) {
        const int r = r0 + ty * 4 + i, n = n0 + tx * 4 + j;
        if (r < end && n < p.N)
          p.out[r * p.out_stride + n] =
              (uint16_t)afd::pack_bf16(p.gated ? afd::silu_mul(acc[0][i][j], acc[1][i][j]) : acc[0][i][j], 0.f);
      }
  }
}

// Device memory of the current device (bulk copies read it).
bool on_device(const void* p, int dev) {
  cudaPointerAttributes a = {};
  if (cudaPointerGetAttributes(&a, p) != cudaSuccess) {
    cudaGetLastError();
    return false;
  }
  return a.type == cudaMemoryTypeDevice && a.device == dev;
}

}  // namespace

extern "C" AFD_API afd_status afd_grouped_linear(const void* x, int64_t x_stride, const float* x_scale,
                                                 const void* weight, const float* weight_scale, const int32_t* ends,
                                                 int32_t num_groups, int32_t expert_alignment, int64_t num_rows,
                                                 int32_t in_features, int32_t out_features, int32_t dtype,
                                                 int32_t gated, void* out, int64_t out_stride, int32_t* error,
                                                 afd_stream stream) {
  const int K = in_features, N = out_features;
  const bool fp8 = dtype == AFD_FP8_E4M3;
  if (dtype != AFD_BF16 && !fp8) return AFD_ERR_ARG;
  if (num_groups < 1 || expert_alignment < 1 || num_rows < 0 || K < 1 || N < 1 || (gated != 0 && gated != 1))
    return AFD_ERR_ARG;
  if (x_stride < K || out_stride < N || !weight || !ends || fp8 != (weight_scale != nullptr)) return AFD_ERR_ARG;
  if (num_rows > 0 && (!x || !out || fp8 != (x_scale != nullptr))) return AFD_ERR_ARG;
  const int elt = fp8 ? 1 : 2;
  if (num_groups > afd::kMaxExperts || num_rows > INT32_MAX - (int64_t)expert_alignment || N > (1 << 24) || K > (1 << 24))
    return AFD_ERR_UNSUPPORTED;
  if (K * elt % 16 || x_stride * elt % 16 || (fp8 && (K % 128 || N % 128))) return AFD_ERR_UNSUPPORTED;
  if (num_rows == 0) return AFD_OK;
  if (!afd::aligned_to(x, 16) || !afd::aligned_to(weight, 16)) return AFD_ERR_UNSUPPORTED;
  if (!afd::aligned_to(x_scale, 4) || !afd::aligned_to(weight_scale, 4) || !afd::aligned_to(ends, 4) ||
      !afd::aligned_to(out, 2) || !afd::aligned_to(error, 4))
    return AFD_ERR_ARG;
  int dev = -1;
  if (cudaGetDevice(&dev) != cudaSuccess) return AFD_ERR_CUDA;
  if (!on_device(x, dev) || !on_device(weight, dev) || !on_device(ends, dev) || !on_device(out, dev) ||
      (fp8 && (!on_device(x_scale, dev) || !on_device(weight_scale, dev))) || (error && !on_device(error, dev)))
    return AFD_ERR_ARG;
  ExpertParams p = {static_cast<const uint8_t*>(x), x_stride, x_scale, static_cast<const uint8_t*>(weight), weight_scale,
                    ends, num_groups, expert_alignment, (int32_t)num_rows, K, N, gated,
                    static_cast<uint16_t*>(out), out_stride, error};
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((N + 63) / 64, num_groups, 4);
  cfg.blockDim = dim3(256);
  cfg.stream = reinterpret_cast<cudaStream_t>(stream);
  const cudaError_t e = fp8 ? cudaLaunchKernelEx(&cfg, grouped_simple_kernel<true>, p)
                            : cudaLaunchKernelEx(&cfg, grouped_simple_kernel<false>, p);
  return e == cudaSuccess ? AFD_OK : AFD_ERR_CUDA;
}
