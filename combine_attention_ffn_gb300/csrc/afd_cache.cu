// afd_cache_write: new tokens' rotary positions and their way into a paged
// cache, in BF16 or as E4M3 with one FP32 scale for each token and head.
//
//   angle_i = position * inv_freq_i; pair i of a head's columns (i and pairs + i,
//   or 2i and 2i + 1): (a cos - b sin, b cos + a sin) * factor
//
// Angles are products and remainders in FP64 (a position of a million leaves
// FP32 two digits of the angle), once for each token and pair of a block; sine
// and cosine of the remainder, at most pi, and the rotation are FP32. A block
// takes some of a token's heads, a thread eight columns of one at a time. What
// bounds many tokens is the traffic: queries read and written, keys and values
// read and written once.

#include <cuda_runtime.h>
#include <stdint.h>

#include "afd.h"
#include "afd_cache.cuh"
#include "afd_device.cuh"
#include "afd_e4m3.cuh"
#include "afd_pointers.cuh"
#include "afd_ragged.cuh"

namespace {

struct WriteParams {
  const uint16_t* q;
  int64_t q_stride;
  const uint16_t* k;
  int64_t k_stride;
  const uint16_t* v;
  int64_t v_stride;
  const int64_t* positions;
  const int64_t* slots;
  const float* inv_freq;
  int32_t pairs, interleaved;
  float factor;
  int32_t T, Hq, Hkv, splits;
  afd::CacheParams cache;
  uint16_t* q_out;
  int64_t q_out_stride;
};

constexpr int kWriteThreads = 256;
constexpr int kMaxPairs = 64;

// Sine and cosine of position * freq.
__device__ __forceinline__ float2 rotation(int64_t position, float freq, float factor) {
  const double angle = (double)position * (double)freq;
  const double turns = rint(angle * 0.15915494309189533577);
  // 2 pi in two parts, so that the remainder keeps what the product holds
  const double rest = fma(turns, -2.4492935982947064e-16, fma(turns, -6.283185307179586, angle));
  float s, c;
  sincosf((float)rest, &s, &c);
  return make_float2(c * factor, s * factor);
}

template <int D, bool FP8>
__global__ void __launch_bounds__(kWriteThreads) cache_write_kernel(const WriteParams p) {
  __shared__ float2 turn[kMaxPairs];
  constexpr int L = D / 8;  // lanes of a head
  afd::pdl_wait();
  afd::pdl_launch_dependents();
  const int t = blockIdx.x / p.splits, part = blockIdx.x % p.splits;
  const int heads = p.Hq + 2 * p.Hkv;
  const int vecs = heads * L;
  // a whole number of warps' worth of a token's groups each
  const int each = ((vecs + p.splits - 1) / p.splits + 31) & ~31;
  const int lo = part * each, hi = min(vecs, lo + each);
  if (lo >= hi) return;
  const int64_t slot = p.slots[t];
  const bool kept = slot >= 0 && slot < (int64_t)p.cache.pages * p.cache.page_size;
  const int64_t page = kept ? (uint32_t)slot / (uint32_t)p.cache.page_size : 0;
  const int in_page = kept ? (int)((uint32_t)slot % (uint32_t)p.cache.page_size) : 0;
  if ((int)threadIdx.x < p.pairs) turn[threadIdx.x] = rotation(p.positions[t], p.inv_freq[threadIdx.x], p.factor);
  __syncthreads();
  for (int i0 = lo; i0 < hi; i0 += kWriteThreads) {
    const int i = i0 + threadIdx.x;
    const bool in = i < hi;
    const int head = in ? i / L : 0, c = i % L * 8;
    const uint16_t* from = head < p.Hq ? p.q + t * p.q_stride + head * D
                           : head < p.Hq + p.Hkv ? p.k + t * p.k_stride + (head - p.Hq) * D
                                                 : p.v + t * p.v_stride + (head - p.Hq - p.Hkv) * D;
    const bool turned = head < p.Hq + p.Hkv && c < 2 * p.pairs;
    float f[8] = {};
    if (in) {
      afd::bf16x8_to_float(afd::ld_before_write(reinterpret_cast<const uint4*>(from + c)), f);  // (q_out may be q)
      if (turned) {
        if (p.interleaved) {
#pragma unroll
          for (int e = 0; e < 8; e += 2) {
            const int pair = (c + e) / 2;
            if (pair < p.pairs) {
              const float2 w = turn[pair];
              const float a = f[e], b = f[e + 1];
              f[e] = a * w.x - b * w.y;
              f[e + 1] = b * w.x + a * w.y;
            }
          }
        } else {
#pragma unroll
          for (int e = 0; e < 8; ++e) {
            const int col = c + e;
            if (col < 2 * p.pairs) {
              const bool first = col < p.pairs;
              const float2 w = turn[first ? col : col - p.pairs];
              const float other = __uint_as_float((uint32_t)from[first ? col + p.pairs : col - p.pairs] << 16);
              f[e] = f[e] * w.x + (first ? -other : other) * w.y;
            }
          }
        }
      }
    }
    __syncwarp();  // the warp has read the heads that it now writes
    const bool key = head >= p.Hq && head < p.Hq + p.Hkv;
    const int h = key ? head - p.Hq : head - p.Hq - p.Hkv;
    float scale = 1.f;
    if (FP8) scale = afd::block_scale(afd::lanes_absmax<L>(afd::absmax8(f)));
    if (!in) continue;
    if (head < p.Hq) {
      *reinterpret_cast<uint4*>(p.q_out + t * p.q_out_stride + head * D + c) = afd::float_to_bf16x8(f);
    } else if (kept) {
      const int64_t row = (int64_t)h * p.cache.page_size + in_page;
      uint8_t* to = key ? p.cache.k + page * p.cache.k_page_units * 64 : p.cache.v + page * p.cache.v_page_units * 64;
      if (FP8) {
        *reinterpret_cast<uint2*>(to + row * D + c) = afd::to_e4m3x8(f, 1.f / scale);
        if (c == 0) (key ? p.cache.k_scale : p.cache.v_scale)[page * p.Hkv * p.cache.page_size + row] = scale;
      } else {
        *reinterpret_cast<uint4*>(to + (row * D + c) * 2) = afd::float_to_bf16x8(f);
      }
    }
  }
}

}  // namespace

extern "C" AFD_API afd_status afd_cache_write(const void* q, int64_t q_stride, const void* k, int64_t k_stride,
                                              const void* v, int64_t v_stride, const int64_t* positions,
                                              const int64_t* slots, const float* inv_freq, int32_t rotary_pairs,
                                              int32_t interleaved, float factor, int64_t num_tokens,
                                              int32_t num_q_heads, const afd_cache* cache, void* q_out,
                                              int64_t q_out_stride, afd_stream stream) {
  if (num_tokens < 0 || num_q_heads < 0 || rotary_pairs < 0 || (interleaved != 0 && interleaved != 1)) return AFD_ERR_ARG;
  const afd_status checked = afd::check_cache(cache);
  if (checked != AFD_OK) return checked;
  const int D = cache->head_dim, Hq = num_q_heads, Hkv = cache->num_kv_heads;
  if (2 * (int64_t)rotary_pairs > D || (num_q_heads > 0 && (q_stride < (int64_t)Hq * D || q_out_stride < (int64_t)Hq * D)) ||
      k_stride < (int64_t)Hkv * D || v_stride < (int64_t)Hkv * D)
    return AFD_ERR_ARG;
  if (num_tokens > afd::kMaxRows || Hq > afd::kMaxHeads || (Hq > 0 && (q_stride % 8 || q_out_stride % 8)) || k_stride % 8 ||
      v_stride % 8)
    return AFD_ERR_UNSUPPORTED;
  if (num_tokens == 0) return AFD_OK;
  if ((Hq > 0 && (!q || !q_out)) || !k || !v || !slots || (rotary_pairs > 0 && (!positions || !inv_freq))) return AFD_ERR_ARG;
  if (!afd::aligned_to(slots, 8) || !afd::aligned_to(positions, 8) || !afd::aligned_to(inv_freq, 4)) return AFD_ERR_ARG;
  if (!afd::aligned_to(q, 16) || !afd::aligned_to(q_out, 16) || !afd::aligned_to(k, 16) || !afd::aligned_to(v, 16))
    return AFD_ERR_UNSUPPORTED;
  WriteParams p = {};
  p.q_stride = q_stride, p.k_stride = k_stride, p.v_stride = v_stride, p.q_out_stride = q_out_stride;
  p.pairs = rotary_pairs, p.interleaved = interleaved, p.factor = factor;
  p.T = (int32_t)num_tokens, p.Hq = Hq, p.Hkv = Hkv;
  if ((Hq > 0 && (!afd::device_view(static_cast<const uint16_t*>(q), &p.q) ||
                  !afd::device_view(static_cast<uint16_t*>(q_out), &p.q_out))) ||
      !afd::device_view(static_cast<const uint16_t*>(k), &p.k) || !afd::device_view(static_cast<const uint16_t*>(v), &p.v) ||
      !afd::device_view(slots, &p.slots) || !afd::view_cache(cache, &p.cache) ||
      (rotary_pairs > 0 && (!afd::device_view(positions, &p.positions) || !afd::device_view(inv_freq, &p.inv_freq))))
    return AFD_ERR_ARG;
  int dev = -1, sms = 0;
  if (cudaGetDevice(&dev) != cudaSuccess || cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess)
    return AFD_ERR_CUDA;
  // Few tokens: several blocks share a token, so that no thread takes its
  // groups of columns in turn while SMs are idle.
  const int rounds = ((Hq + 2 * Hkv) * (D / 8) + kWriteThreads - 1) / kWriteThreads;
  const int64_t spread = (2 * (int64_t)sms + p.T - 1) / p.T;
  p.splits = (int32_t)(spread < rounds ? spread : rounds);
  const int64_t grid = (int64_t)p.T * p.splits;
  if (grid > INT32_MAX) return AFD_ERR_UNSUPPORTED;
  cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
  const bool fp8 = cache->dtype == AFD_FP8_E4M3;
  auto kernel = D == 64 ? (fp8 ? cache_write_kernel<64, true> : cache_write_kernel<64, false>)
                        : (fp8 ? cache_write_kernel<128, true> : cache_write_kernel<128, false>);
  return afd::launch_dependent(kernel, grid, kWriteThreads, 0, s, p) == cudaSuccess ? AFD_OK : AFD_ERR_CUDA;
}
