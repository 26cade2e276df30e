// afd_norm_rows: the rows a source dispatches, from its residual stream: the
// residual's addition, the root-mean-square norm, and the rows in BF16 (for the
// router and BF16 exchanges) and in E4M3 with block-128 scales (FP8 exchanges).
//
//   r = x + residual,  y = r rsqrt(mean(r^2) + eps) weight,
//   scale_b = max(max |y_b| / 448, 2^-100),  q = e4m3(y / scale_b)
//
// One pass: a block holds a row in registers between the sum of squares and
// the products, so each input is read and each output written once, which is
// what bounds it for many rows: 4,096 of 4,096 columns (151.5 MB) in 24.3 us, 6.2
// TB/s, against 22.6 at the copy's rate. Decode steps are a launch and two trips to
// memory: one row of 2,048 1.7 us, 128 of 7,168 2.1. Two groups of eight columns a
// thread above 2,048 columns (against 25.2 us then, one took 27.6 and four 24.8, but
// 2.3 for the 128 rows).

#include <cuda_runtime.h>
#include <stdint.h>

#include "afd.h"
#include "afd_device.cuh"
#include "afd_e4m3.cuh"
#include "afd_pointers.cuh"
#include "afd_ragged.cuh"

namespace {

struct NormParams {
  const uint16_t* x;
  int64_t x_stride;
  const uint16_t* residual;
  int64_t residual_stride;
  const uint16_t* weight;
  float eps;
  int32_t T, H;
  uint16_t* residual_out;
  int64_t residual_out_stride;
  uint16_t* out;
  int64_t out_stride;
  uint8_t* q;      // [T][H]
  float* q_scale;  // [T][H / 128]
};

// Threads of a block at most, and the widest row a block holds.
constexpr int norm_threads(int vpt) { return vpt == 1 ? 256 : 512; }
constexpr int kMaxWidth = 8 * 8 * norm_threads(8);

// The block's sum, the same for every thread.
__device__ __forceinline__ float block_sum(float v, float* part) {
#pragma unroll
  for (int d = 16; d; d >>= 1) v += __shfl_xor_sync(0xffffffffu, v, d);
  const int warps = blockDim.x >> 5;
  if ((threadIdx.x & 31) == 0) part[threadIdx.x >> 5] = v;
  __syncthreads();
  float sum = (threadIdx.x & 31) < warps ? part[threadIdx.x & 31] : 0.f;
#pragma unroll
  for (int d = 16; d; d >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, d);
  return sum;
}

// A block per row, VPT groups of eight columns a thread.
template <int VPT>
__global__ void __launch_bounds__(norm_threads(VPT)) norm_rows_kernel(const NormParams p) {
  __shared__ float part[32];
  afd::pdl_wait();
  afd::pdl_launch_dependents();
  const int64_t t = blockIdx.x;
  float r[VPT][8];
  uint4 wv[VPT];
  float sum = 0.f;
  uint4 xv[VPT], rv[VPT];
#pragma unroll
  for (int i = 0; i < VPT; ++i) {
    const int c = (i * blockDim.x + threadIdx.x) * 8;
    if (c >= p.H) continue;
    xv[i] = afd::ld_before_write(reinterpret_cast<const uint4*>(p.x + t * p.x_stride + c));  // (an output may lie there)
    if (p.residual) rv[i] = afd::ld_before_write(reinterpret_cast<const uint4*>(p.residual + t * p.residual_stride + c));
    wv[i] = *reinterpret_cast<const uint4*>(p.weight + c);
  }
#pragma unroll
  for (int i = 0; i < VPT; ++i) {
    const int c = (i * blockDim.x + threadIdx.x) * 8;
#pragma unroll
    for (int e = 0; e < 8; ++e) r[i][e] = 0.f;
    if (c >= p.H) continue;
    afd::bf16x8_to_float(xv[i], r[i]);
    if (p.residual) {
      float a[8];
      afd::bf16x8_to_float(rv[i], a);
#pragma unroll
      for (int e = 0; e < 8; ++e) r[i][e] += a[e];
    }
    if (p.residual_out)
      *reinterpret_cast<uint4*>(p.residual_out + t * p.residual_out_stride + c) = afd::float_to_bf16x8(r[i]);
#pragma unroll
    for (int e = 0; e < 8; ++e) sum = fmaf(r[i][e], r[i][e], sum);
  }
  const float f = rsqrtf(block_sum(sum, part) / (float)p.H + p.eps);
#pragma unroll
  for (int i = 0; i < VPT; ++i) {
    const int c = (i * blockDim.x + threadIdx.x) * 8;
    const bool in = c < p.H;
    float y[8] = {};
    if (in) {
      float w[8];
      afd::bf16x8_to_float(wv[i], w);
#pragma unroll
      for (int e = 0; e < 8; ++e) y[e] = r[i][e] * f * w[e];
      if (p.out) *reinterpret_cast<uint4*>(p.out + t * p.out_stride + c) = afd::float_to_bf16x8(y);
    }
    if (p.q) {  // a block of 128 columns is 16 lanes' (H is a multiple of 128 then)
      const float scale = afd::block_scale(afd::lanes_absmax<16>(afd::absmax8(y)));
      if (in) {
        *reinterpret_cast<uint2*>(p.q + t * p.H + c) = afd::quotient_e4m3x8(y, scale);
        if ((threadIdx.x & 15) == 0) p.q_scale[t * (p.H / 128) + c / 128] = scale;
      }
    }
  }
}

// Rows of any width and alignment, two passes over them.
__global__ void __launch_bounds__(256) norm_rows_any_kernel(const NormParams p) {
  __shared__ float part[32];
  afd::pdl_wait();
  afd::pdl_launch_dependents();
  const int64_t t = blockIdx.x;
  const uint16_t* x = p.x + t * p.x_stride;
  const uint16_t* residual = p.residual ? p.residual + t * p.residual_stride : nullptr;
  auto at = [&](int c) {
    float v = __uint_as_float((uint32_t)x[c] << 16);
    if (residual) v += __uint_as_float((uint32_t)residual[c] << 16);
    return v;
  };
  float sum = 0.f;
  for (int c = threadIdx.x; c < p.H; c += blockDim.x) {
    const float v = at(c);
    sum = fmaf(v, v, sum);
  }
  const float f = rsqrtf(block_sum(sum, part) / (float)p.H + p.eps);
  for (int c = threadIdx.x; c < p.H; c += blockDim.x) {
    const float v = at(c);  // (before this column's outputs, which may lie there)
    if (p.residual_out) p.residual_out[t * p.residual_out_stride + c] = (uint16_t)afd::pack_bf16(v, 0.f);
    const float y = v * f * __uint_as_float((uint32_t)p.weight[c] << 16);
    if (p.out) p.out[t * p.out_stride + c] = (uint16_t)afd::pack_bf16(y, 0.f);
  }
}

template <int VPT>
cudaError_t launch_norm(const NormParams& p, cudaStream_t stream) {
  const int vecs = (p.H / 8 + VPT - 1) / VPT;
  return afd::launch_dependent(norm_rows_kernel<VPT>, p.T, (vecs + 31) / 32 * 32, 0, stream, p);
}

// Whether an array of rows can be read 16 bytes at a time.
bool vector_rows(const void* p, int64_t stride) { return !p || (stride % 8 == 0 && afd::aligned_to(p, 16)); }

}  // namespace

extern "C" AFD_API afd_status afd_norm_rows(const void* x, int64_t x_stride, const void* residual, int64_t residual_stride,
                                            const void* weight, float eps, int64_t num_rows, int32_t features,
                                            void* residual_out, int64_t residual_out_stride, void* out, int64_t out_stride,
                                            void* fp8_out, float* scale_out, afd_stream stream) {
  const int H = features;
  if (num_rows < 0 || H < 1 || x_stride < H || (residual && residual_stride < H) ||
      (residual_out && residual_out_stride < H) || (out && out_stride < H) || !(eps >= 0.f))
    return AFD_ERR_ARG;
  if (!fp8_out != !scale_out || (residual_out && !residual)) return AFD_ERR_ARG;
  if (num_rows > afd::kMaxRows || H > afd::kMaxFeatures || (fp8_out && (H % 128 || H > kMaxWidth)))
    return AFD_ERR_UNSUPPORTED;
  if (num_rows == 0) return AFD_OK;
  if (!x || !weight || (!out && !fp8_out && !residual_out)) return AFD_ERR_ARG;
  if (!afd::aligned_to(x, 2) || !afd::aligned_to(residual, 2) || !afd::aligned_to(weight, 2) ||
      !afd::aligned_to(residual_out, 2) || !afd::aligned_to(out, 2) || !afd::aligned_to(scale_out, 4))
    return AFD_ERR_ARG;
  const bool vec = H % 8 == 0 && H <= kMaxWidth && vector_rows(x, x_stride) && vector_rows(residual, residual_stride) &&
                   vector_rows(weight, 0) && vector_rows(residual_out, residual_out_stride) && vector_rows(out, out_stride);
  if (fp8_out && (!vec || !afd::aligned_to(fp8_out, 8))) return AFD_ERR_UNSUPPORTED;
  NormParams p = {};
  p.x_stride = x_stride, p.residual_stride = residual_stride, p.eps = eps, p.T = (int32_t)num_rows, p.H = H;
  p.residual_out_stride = residual_out_stride, p.out_stride = out_stride;
  if (!afd::device_view(static_cast<const uint16_t*>(x), &p.x) ||
      (residual && !afd::device_view(static_cast<const uint16_t*>(residual), &p.residual)) ||
      !afd::device_view(static_cast<const uint16_t*>(weight), &p.weight) ||
      (residual_out && !afd::device_view(static_cast<uint16_t*>(residual_out), &p.residual_out)) ||
      (out && !afd::device_view(static_cast<uint16_t*>(out), &p.out)) ||
      (fp8_out && (!afd::device_view(static_cast<uint8_t*>(fp8_out), &p.q) || !afd::device_view(scale_out, &p.q_scale))))
    return AFD_ERR_ARG;
  cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
  cudaError_t e;
  if (!vec) e = afd::launch_dependent(norm_rows_any_kernel, p.T, 256, 0, s, p);
  else if (H <= 8 * norm_threads(1)) e = launch_norm<1>(p, s);
  else if (H <= 2 * 8 * norm_threads(2)) e = launch_norm<2>(p, s);
  else if (H <= 4 * 8 * norm_threads(4)) e = launch_norm<4>(p, s);
  else e = launch_norm<8>(p, s);
  return e == cudaSuccess ? AFD_OK : AFD_ERR_CUDA;
}
