// Row operators of a worker between its products: the gated activation
// (afd_gated_rows) and the low-rank adapters of many requests
// (afd_adapter_add).

#include <cuda_runtime.h>
#include <stdint.h>

#include <climits>

#include "afd.h"
#include "afd_device.cuh"
#include "afd_pointers.cuh"
#include "afd_ragged.cuh"

namespace {

// ---------------------------------------------------------- gated activation
struct GatedParams {
  const uint16_t* h;
  int64_t h_stride;
  const int32_t* ends;
  int32_t G, alpha, R, N;
  uint16_t* out;
  int64_t out_stride;
};

__device__ __forceinline__ float bf16_at(const uint16_t* p) { return __uint_as_float((uint32_t)*p << 16); }

// A warp per row; VEC: rows and halves start on 16-byte boundaries.
template <bool VEC>
__global__ void __launch_bounds__(256) gated_rows_kernel(const GatedParams p) {
  __shared__ int sh_end[afd::kMaxExperts];
  for (int g = threadIdx.x; g < p.G; g += blockDim.x) sh_end[g] = afd::group_end(p.ends[g], p.R);
  __syncthreads();
  const int lane = threadIdx.x & 31;
  const int warps = gridDim.x * (blockDim.x >> 5);
  const int limit = sh_end[p.G - 1];
  for (int r = blockIdx.x * (blockDim.x >> 5) + (threadIdx.x >> 5); r < limit; r += warps) {
    // the first group that ends behind this row
    int lo = 0, hi = p.G - 1;
    while (lo < hi) {
      const int mid = (lo + hi) >> 1;
      if (sh_end[mid] > r) hi = mid; else lo = mid + 1;
    }
    if (r < (lo ? afd::group_start(sh_end[lo - 1], p.alpha, p.R) : 0)) continue;  // padding
    const uint16_t* gate = p.h + r * p.h_stride;
    const uint16_t* up = gate + p.N;
    uint16_t* out = p.out + r * p.out_stride;
    if (VEC) {
      for (int c = lane * 8; c < p.N; c += 256) {
        float g[8], u[8];
        afd::bf16x8_to_float(*reinterpret_cast<const uint4*>(gate + c), g);
        afd::bf16x8_to_float(*reinterpret_cast<const uint4*>(up + c), u);
#pragma unroll
        for (int i = 0; i < 8; ++i) g[i] = afd::silu_mul(g[i], u[i]);
        *reinterpret_cast<uint4*>(out + c) = afd::float_to_bf16x8(g);
      }
    } else {
      for (int c = lane; c < p.N; c += 32)
        out[c] = (uint16_t)afd::pack_bf16(afd::silu_mul(bf16_at(gate + c), bf16_at(up + c)), 0.f);
    }
  }
}

// ------------------------------------------------------------------ adapters
struct AdapterParams {
  const uint16_t* base;
  int64_t base_stride;
  const uint16_t* x;
  int64_t x_stride;
  const uint16_t* down;
  const uint16_t* up;
  const int32_t* token_slots;
  const float* scales;
  const int32_t* row_src;
  const int32_t* ends;
  int32_t G, top_k, R, tokens, S, rank, K, N;
  uint16_t* out;
  int64_t out_stride;
};

// A block per row: the rank dot products over x by one warp each, then the
// output's columns by the block's threads.
__global__ void __launch_bounds__(256) adapter_rows_kernel(const AdapterParams p) {
  __shared__ float low[64];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int limit = p.row_src ? afd::group_end(p.ends[p.G - 1], p.R) : p.R;
  for (int r = blockIdx.x; r < limit; r += gridDim.x) {
    int t = r;
    if (p.row_src) {
      const int src = p.row_src[r];
      t = src < 0 ? -1 : src / p.top_k;
      if (t < 0 || t >= p.tokens) continue;
    }
    const int a = p.token_slots[t];
    const bool has = a >= 0 && a < p.S;
    if (has) {
      const uint16_t* x = p.x + r * p.x_stride;
      for (int j = warp; j < p.rank; j += 8) {
        const uint16_t* d = p.down + ((int64_t)a * p.rank + j) * p.K;
        float sum = 0.f;
        for (int c = lane; c < p.K; c += 32) sum = fmaf(bf16_at(x + c), bf16_at(d + c), sum);
        for (int s = 16; s; s >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, s);
        if (lane == 0) low[j] = sum * p.scales[a];
      }
    }
    __syncthreads();
    for (int n = threadIdx.x; n < p.N; n += blockDim.x) {
      float sum = 0.f;
      if (has) {
        const uint16_t* u = p.up + ((int64_t)a * p.N + n) * p.rank;
        for (int j = 0; j < p.rank; ++j) sum = fmaf(low[j], bf16_at(u + j), sum);
      }
      p.out[r * p.out_stride + n] = (uint16_t)afd::pack_bf16(bf16_at(p.base + r * p.base_stride + n) + sum, 0.f);
    }
    __syncthreads();
  }
}

int sm_count() {
  int dev = 0, n = 0;
  if (cudaGetDevice(&dev) != cudaSuccess || cudaDeviceGetAttribute(&n, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess)
    return 0;
  return n;
}

}  // namespace

extern "C" {

AFD_API afd_status afd_gated_rows(const void* h, int64_t h_stride, const int32_t* ends, int32_t num_groups,
                                  int32_t expert_alignment, int64_t num_rows, int32_t features, void* out,
                                  int64_t out_stride, afd_stream stream) {
  if (num_groups < 1 || expert_alignment < 1 || num_rows < 0 || features < 1 || !ends) return AFD_ERR_ARG;
  if (h_stride < 2 * (int64_t)features || out_stride < features) return AFD_ERR_ARG;
  if (num_groups > afd::kMaxExperts || num_rows > INT32_MAX - (int64_t)expert_alignment) return AFD_ERR_UNSUPPORTED;
  if (num_rows == 0) return AFD_OK;
  if (!h || !out) return AFD_ERR_ARG;
  GatedParams p = {nullptr, h_stride, nullptr, num_groups, expert_alignment, (int32_t)num_rows, features, nullptr, out_stride};
  if (!afd::device_view(static_cast<const uint16_t*>(h), &p.h) || !afd::device_view(ends, &p.ends) ||
      !afd::device_view(static_cast<uint16_t*>(out), &p.out))
    return AFD_ERR_ARG;
  if (!afd::aligned_to(p.h, 2) || !afd::aligned_to(p.out, 2) || !afd::aligned_to(p.ends, 4)) return AFD_ERR_ARG;
  const int sms = sm_count();
  if (sms < 1) return AFD_ERR_CUDA;
  const bool vec = features % 8 == 0 && h_stride % 8 == 0 && out_stride % 8 == 0 && afd::aligned_to(p.h, 16) &&
                   afd::aligned_to(p.out, 16);
  cudaLaunchConfig_t cfg = {};
  const int64_t blocks = (num_rows + 7) / 8;
  cfg.gridDim = dim3((unsigned)(blocks < sms * 8 ? blocks : sms * 8));
  cfg.blockDim = dim3(256);
  cfg.stream = reinterpret_cast<cudaStream_t>(stream);
  const cudaError_t e = vec ? cudaLaunchKernelEx(&cfg, gated_rows_kernel<true>, p)
                            : cudaLaunchKernelEx(&cfg, gated_rows_kernel<false>, p);
  return e == cudaSuccess ? AFD_OK : AFD_ERR_CUDA;
}

AFD_API afd_status afd_adapter_add(const void* base, int64_t base_stride, const void* x, int64_t x_stride,
                                   const void* down, const void* up, const int32_t* token_slots, const float* scales,
                                   const int32_t* row_src, const int32_t* ends, int32_t num_groups, int32_t top_k,
                                   int64_t num_rows, int32_t num_tokens, int32_t num_slots, int32_t rank,
                                   int32_t in_features, int32_t out_features, void* out, int64_t out_stride,
                                   afd_stream stream) {
  if (num_rows < 0 || num_tokens < 0 || num_slots < 1 || rank < 1 || in_features < 1 || out_features < 1)
    return AFD_ERR_ARG;
  if (base_stride < out_features || out_stride < out_features || x_stride < in_features) return AFD_ERR_ARG;
  if (row_src ? (!ends || num_groups < 1 || top_k < 1) : num_tokens < num_rows) return AFD_ERR_ARG;
  if (rank != 8 && rank != 16 && rank != 32 && rank != 64) return AFD_ERR_UNSUPPORTED;
  if (in_features % 16 || out_features % 8 || base_stride % 8 || out_stride % 8 || x_stride % 8 || num_rows > INT32_MAX)
    return AFD_ERR_UNSUPPORTED;
  if (num_rows == 0) return AFD_OK;
  if (!base || !x || !down || !up || !token_slots || !scales || !out) return AFD_ERR_ARG;
  AdapterParams p = {};
  p.base_stride = base_stride, p.x_stride = x_stride, p.out_stride = out_stride;
  p.G = num_groups, p.top_k = top_k, p.R = (int32_t)num_rows, p.tokens = num_tokens, p.S = num_slots, p.rank = rank;
  p.K = in_features, p.N = out_features;
  if (!afd::device_view(static_cast<const uint16_t*>(base), &p.base) ||
      !afd::device_view(static_cast<const uint16_t*>(x), &p.x) ||
      !afd::device_view(static_cast<const uint16_t*>(down), &p.down) ||
      !afd::device_view(static_cast<const uint16_t*>(up), &p.up) || !afd::device_view(token_slots, &p.token_slots) ||
      !afd::device_view(scales, &p.scales) || !afd::device_view(static_cast<uint16_t*>(out), &p.out) ||
      (row_src && (!afd::device_view(row_src, &p.row_src) || !afd::device_view(ends, &p.ends))))
    return AFD_ERR_ARG;
  if (!afd::aligned_to(p.token_slots, 4) || !afd::aligned_to(p.scales, 4) || !afd::aligned_to(p.row_src, 4) ||
      !afd::aligned_to(p.ends, 4))
    return AFD_ERR_ARG;
  if (!afd::aligned_to(p.base, 16) || !afd::aligned_to(p.x, 16) || !afd::aligned_to(p.down, 16) ||
      !afd::aligned_to(p.up, 16) || !afd::aligned_to(p.out, 16))
    return AFD_ERR_UNSUPPORTED;
  const int sms = sm_count();
  if (sms < 1) return AFD_ERR_CUDA;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)(num_rows < sms * 8 ? num_rows : sms * 8));
  cfg.blockDim = dim3(256);
  cfg.stream = reinterpret_cast<cudaStream_t>(stream);
  return cudaLaunchKernelEx(&cfg, adapter_rows_kernel, p) == cudaSuccess ? AFD_OK : AFD_ERR_CUDA;
}

}  // extern "C"
