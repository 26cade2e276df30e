// afd_cache_write: new tokens' rotary positions and their way into a paged
// cache, in BF16 or as E4M3 with one FP32 scale for each token and head.
//
//   angle_i = position * inv_freq_i; pair i of a head's columns (i and pairs + i,
//   or 2i and 2i + 1): (a cos - b sin, b cos + a sin) * factor
//
// Angles are products and remainders in FP64 (a position of a million leaves
// FP32 two digits of the angle), once for each token and pair; sine and cosine of
// the remainder, at most pi, and the rotation are FP32. A block takes some tokens,
// or some of a token's heads where there are few; a thread has eight columns of
// every so many heads, so it holds its sines and cosines in registers through a
// token (looked up and chosen for every group of columns, 8,192 tokens took 83 us).
// What bounds many tokens is the traffic, queries read and written, keys and values
// read and written once, with half of the issue slots: 314 MB in 57 us, 5.5 TB/s.
// A decode step is a chain of latencies: 2.4 us for a token, 4.4 for 128.

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
  int32_t T, Hq, Hkv;
  int32_t blocks;        // that share the tokens
  int32_t splits, each;  // blocks that share a token's heads, and the heads of each
  afd::CacheParams cache;
  uint16_t* q_out;
  int64_t q_out_stride;
};

constexpr int kWriteThreads = 256;  // of a block at most
// Blocks of an SM, of many tokens, and of all SMs two of few. 8,192 tokens (64 query
// heads, 8 KV heads, E4M3): 55.9 us; four 55.3, five 56.8, six 57.9; 128 tokens,
// where registers and not their number count: 4.2, 4.8, 6.0 and 6.3 (all before the
// values were divided by their scale, which takes 1 and 0.2 us more).
constexpr int kWriteBlocks = 3;
constexpr int kAhead = 4;           // groups of eight columns of a thread in flight
constexpr int kMaxTokens = 8;       // whose sines and cosines a block finds in one go
constexpr uint32_t kNowhere = 0xffffffffu;
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

// How a head's columns turn: not at all, (2i, 2i + 1) with a multiple of four
// pairs, (i, pairs + i) with one of eight, or either with another number of them.
enum { kStill, kInterleaved, kHalves, kUneven };

// Eight columns of a head turned. `raw` are the columns as they lie there, `from`
// the head's address, `partner` the lane that has their partners (kHalves).
template <int MODE>
__device__ __forceinline__ void turn_columns(const uint4& raw, const uint16_t* from, int c, int pairs, bool interleaved,
                                             int partner, const float (&cosine)[8], const float (&sine)[8], float (&f)[8]) {
  afd::bf16x8_to_float(raw, f);
  if (MODE == kStill) return;
  float other[8] = {};
  if (MODE == kInterleaved) {
#pragma unroll
    for (int e = 0; e < 8; ++e) other[e] = f[e ^ 1];
  } else if (MODE == kHalves) {
    afd::bf16x8_to_float(make_uint4(__shfl_sync(0xffffffffu, raw.x, partner), __shfl_sync(0xffffffffu, raw.y, partner),
                                    __shfl_sync(0xffffffffu, raw.z, partner), __shfl_sync(0xffffffffu, raw.w, partner)), other);
  } else if (from) {
#pragma unroll 1
    for (int e = 0; e < 8 && c + e < 2 * pairs; ++e) {
      const int col = c + e;
      other[e] = __uint_as_float((uint32_t)from[interleaved ? col ^ 1 : col < pairs ? col + pairs : col - pairs] << 16);
    }
  }
  if (c >= 2 * pairs) return;
#pragma unroll
  for (int e = 0; e < 8; ++e) {
    const float y = f[e] * cosine[e] + other[e] * sine[e];
    f[e] = MODE == kUneven && c + e >= 2 * pairs ? f[e] : y;
  }
}

template <int D, bool FP8, int MODE>
__global__ void __launch_bounds__(kWriteThreads, kWriteBlocks) cache_write_kernel(const WriteParams p) {
  __shared__ float2 turn[kMaxTokens][kMaxPairs];
  __shared__ uint32_t page_of[kMaxTokens], place_of[kMaxTokens];  // kNowhere: not kept
  constexpr int L = D / 8;  // lanes of a head
  afd::pdl_wait();
  afd::pdl_launch_dependents();
  const int block = blockIdx.x / p.splits, part = blockIdx.x - block * p.splits;
  const int t0 = (int)((int64_t)p.T * block / p.blocks), t1 = (int)((int64_t)p.T * (block + 1) / p.blocks);
  // The block's heads, counted through queries, keys and values.
  const int h0 = part * p.each, h1 = min(p.Hq + 2 * p.Hkv, h0 + p.each);
  const int q1 = min(h1, p.Hq), kv0 = max(h0, p.Hq);
  const int c = threadIdx.x % L * 8, mine = threadIdx.x / L;
  const int step = blockDim.x / L;  // heads that the block takes at a time
  const int partner = (threadIdx.x & 31) + (c < p.pairs ? p.pairs : -p.pairs) / 8;
#pragma unroll 1
  for (int t = t0; t < t1; ++t) {
    const int at = (t - t0) % kMaxTokens;
    // The first rows are on their way while the block finds its sines and cosines.
    const uint16_t* q = p.q + t * p.q_stride + (h0 + mine) * D + c;
    uint4 raw[kAhead], kv = make_uint4(0, 0, 0, 0);
    auto fetch = [&](int r0) {
#pragma unroll
      for (int u = 0; u < kAhead; ++u)
        raw[u] = r0 + u * step + mine < q1 ? afd::ld_before_write(reinterpret_cast<const uint4*>(q + u * step * D))
                                           : make_uint4(0, 0, 0, 0);  // (q_out may be q)
    };
    auto kv_source = [&](int head) {
      return head < p.Hq + p.Hkv ? p.k + t * p.k_stride + (head - p.Hq) * D : p.v + t * p.v_stride + (head - p.Hq - p.Hkv) * D;
    };
    fetch(h0);
    if (kv0 + mine < h1) kv = afd::ld_once(reinterpret_cast<const uint4*>(kv_source(kv0 + mine) + c));
    if (at == 0) {
      const int tokens = min(t1 - t, kMaxTokens);
      __syncthreads();  // (the last tokens' have been read)
      for (int i = threadIdx.x; i < tokens; i += blockDim.x) {
        const int64_t slot = p.slots[t + i];
        const bool kept = slot >= 0 && slot < (int64_t)p.cache.pages * p.cache.page_size;
        const uint32_t page = kept ? (uint32_t)slot / (uint32_t)p.cache.page_size : kNowhere;
        page_of[i] = page;
        place_of[i] = kept ? (uint32_t)slot - page * (uint32_t)p.cache.page_size : 0;
      }
      if (MODE != kStill)
        for (int i = threadIdx.x; i < tokens * p.pairs; i += blockDim.x) {
          const int tok = i / p.pairs, pair = i - tok * p.pairs;
          turn[tok][pair] = rotation(p.positions[t + tok], p.inv_freq[pair], p.factor);
        }
      __syncthreads();
    }
    float cosine[8], sine[8];  // of this thread's columns, sines with their signs
    if (MODE != kStill) {
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        const int col = c + e;
        const bool paired = MODE == kInterleaved || (MODE == kUneven && p.interleaved);
        const bool second = paired ? e & 1 : col >= p.pairs;
        const int pair = paired ? col / 2 : second ? col - p.pairs : col;
        const float2 w = turn[at][min(pair, p.pairs - 1)];
        cosine[e] = w.x, sine[e] = second ? w.y : -w.y;
      }
    }
    uint16_t* out = p.q_out + t * p.q_out_stride + (h0 + mine) * D + c;
#pragma unroll 1
    for (int r0 = h0; r0 < q1;) {
#pragma unroll
      for (int u = 0; u < kAhead; ++u) {
        if (r0 + u * step >= q1) break;  // (the whole block)
        float f[8];
        const bool in = r0 + u * step + mine < q1;
        turn_columns<MODE>(raw[u], in ? q - c + u * step * D : nullptr, c, p.pairs, p.interleaved, partner, cosine, sine, f);
        if (MODE == kUneven) __syncwarp();  // the warp has read the heads that it now writes
        if (in) *reinterpret_cast<uint4*>(out + u * step * D) = afd::float_to_bf16x8(f);
      }
      r0 += kAhead * step;
      if (r0 >= q1) break;
      q += kAhead * step * D, out += kAhead * step * D;
      fetch(r0);
    }
#pragma unroll 1
    for (int r0 = kv0; r0 < h1; r0 += step) {
      const int head = r0 + mine;
      const bool in = head < h1, key = head < p.Hq + p.Hkv;
      if (r0 > kv0) kv = in ? afd::ld_once(reinterpret_cast<const uint4*>(kv_source(head) + c)) : make_uint4(0, 0, 0, 0);
      float f[8], still[8];
      turn_columns<MODE>(kv, in && key ? kv_source(head) : nullptr, c, p.pairs, p.interleaved, partner, cosine, sine, f);
      afd::bf16x8_to_float(kv, still);
#pragma unroll
      for (int e = 0; e < 8; ++e) f[e] = key ? f[e] : still[e];
      float scale = 1.f;
      if (FP8) scale = afd::block_scale(afd::lanes_absmax<L>(afd::absmax8(f)));
      const uint32_t page = page_of[at];
      if (!in || page == kNowhere) continue;
      const int64_t row = (int64_t)(head - p.Hq - (key ? 0 : p.Hkv)) * p.cache.page_size + place_of[at];
      uint8_t* to = key ? p.cache.k + (uint64_t)page * p.cache.k_page_units * 64 : p.cache.v + (uint64_t)page * p.cache.v_page_units * 64;
      if (FP8) {
        *reinterpret_cast<uint2*>(to + row * D + c) = afd::divided_e4m3x8(f, scale);
        if (c == 0) (key ? p.cache.k_scale : p.cache.v_scale)[(int64_t)page * p.Hkv * p.cache.page_size + row] = scale;
      } else {
        *reinterpret_cast<uint4*>(to + (row * D + c) * 2) = afd::float_to_bf16x8(f);
      }
    }
  }
}

template <int D, bool FP8>
cudaError_t launch_write(const WriteParams& p, int64_t grid, int threads, cudaStream_t s) {
  auto kernel = p.pairs == 0 ? cache_write_kernel<D, FP8, kStill>
                : p.pairs % (p.interleaved ? 4 : 8) ? cache_write_kernel<D, FP8, kUneven>
                : p.interleaved ? cache_write_kernel<D, FP8, kInterleaved> : cache_write_kernel<D, FP8, kHalves>;
  return afd::launch_dependent(kernel, grid, threads, 0, s, p);
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
  // Many tokens: as many blocks as there is room for, with the same number each.
  // Few: several blocks share a token, so that no head waits for another while SMs
  // are idle.
  const int heads = Hq + 2 * Hkv, L = D / 8;
  p.blocks = (int32_t)(p.T < kWriteBlocks * (int64_t)sms ? p.T : kWriteBlocks * (int64_t)sms);
  const int spread = (2 * sms + p.blocks - 1) / p.blocks, most = (heads * L + 127) / 128;
  p.splits = spread < most ? spread : most;
  p.each = (heads + p.splits - 1) / p.splits;
  const int need = (p.each * L + 31) & ~31, threads = need < kWriteThreads ? need : kWriteThreads;
  const int64_t grid = (int64_t)p.blocks * p.splits;
  cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
  const bool fp8 = cache->dtype == AFD_FP8_E4M3;
  const cudaError_t e = D == 64 ? (fp8 ? launch_write<64, true>(p, grid, threads, s) : launch_write<64, false>(p, grid, threads, s))
                                : (fp8 ? launch_write<128, true>(p, grid, threads, s) : launch_write<128, false>(p, grid, threads, s));
  return e == cudaSuccess ? AFD_OK : AFD_ERR_CUDA;
}
