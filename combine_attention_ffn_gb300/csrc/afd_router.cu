// afd_route_topk: the router's top-k in the form a dispatch takes.
//
// One warp per token; lane i holds the logits of experts i, i + 32, ... in
// registers. A selection round takes the warp's largest key with one
// redux.sync over order-preserving 32-bit images of the keys and the lowest
// index among its holders with a second one, so k rounds cost 2k warp
// reductions and no shared memory. The work is a few KB per token: a decode
// step is bound by the launch, a prefill bucket by the latency of one warp's
// rounds, which is why tokens take a warp each and not a block: 2.3 us for one
// token of 128 experts, 3.4 us for 2,048, with a bias 3.1 to 3.4 and 4.5 to 6.4
// (softmax scores and a bias of zeros, whose keys crowd: 8.9).
//
// Softmax and sigmoid are monotone, so without a bias the logits themselves
// are the keys, exactly. With a bias the keys score + bias are computed in
// FP32 first; where neighbouring keys lie closer together than those sums'
// error, the experts in question are put in order by 64-bit keys, one a lane
// (rare: gaps are of the order of 1e-2, the error of 1e-6; the one token of a
// bucket that needs it adds 2 us with sigmoid scores and 4 with softmax). The
// rounds leave that question to a look at all slots after the last one (asked
// in every round, 2,048 tokens took 8 us).

#include <cuda_runtime.h>
#include <float.h>
#include <stdint.h>

#include "afd.h"
#include "afd_device.cuh"
#include "afd_pointers.cuh"

namespace {

constexpr int kRouterWarps = 4;  // tokens per block
constexpr unsigned kFull = 0xffffffffu;

struct RouterParams {
  const void* logits;
  int64_t row_stride;
  const float* bias;
  const int32_t* live;
  int32_t T, E, K;
  int32_t sigmoid, renormalize;
  float scale;
  int64_t* ids;
  float* weights;
};

// Order-preserving image of a finite or +infinite value; 0 is left for "not
// selectable" (the image of -infinity is 0x007fffff).
__device__ __forceinline__ uint32_t order_image(float v) {
  const uint32_t b = __float_as_uint(v + 0.0f);  // -0 and +0 are equal
  return (b & 0x80000000u) ? ~b : b | 0x80000000u;
}

__device__ __forceinline__ float from_image(uint32_t u) {
  return __uint_as_float((u & 0x80000000u) ? u & 0x7fffffffu : ~u);
}

__device__ __forceinline__ float warp_sum(float v) {
#pragma unroll
  for (int d = 16; d; d >>= 1) v += __shfl_xor_sync(kFull, v, d);
  return v;
}

__device__ __forceinline__ double warp_sum(double v) {
#pragma unroll
  for (int d = 16; d; d >>= 1) v += __shfl_xor_sync(kFull, v, d);
  return v;
}

// The largest FP32 distance at which two computed keys may be out of order:
// twice the error of a score plus that of the two additions (2^-23 of the larger
// key, taken twice). Softmax (exp, the sum of up to 1,024, the quotient): below
// 2^-17 relative. Sigmoid: exp 2^-22 and two roundings, below 2^-21 even where
// the score is subnormal.
__device__ __forceinline__ float key_slack(bool sigmoid, float pa, float pb, float ka, float kb) {
  return (sigmoid ? 1.5e-6f : 1.6e-5f) * fmaxf(pa, pb) + 2.4e-7f * fmaxf(fabsf(ka), fabsf(kb));
}

// Selection with keys in 64 bits, for more than 32 keys that lie close
// together; every lane returns in `mine` the expert of
// slot `lane` (-1: none) and in `logit` its logit.
template <int PER>
__device__ __noinline__ void select_exact(const float (&l)[PER], const RouterParams& p, float top, int lane,
                                          int* mine, float* logit) {
  double inv = 1.0;
  if (!p.sigmoid) {
    double sum = 0.0;
    for (int j = 0; j < PER; ++j)
      if (l[j] != -INFINITY) sum += exp((double)l[j] - (double)top);
    inv = warp_sum(sum);
  }
  uint32_t taken = 0;
  *mine = -1;
  *logit = 0.f;
  for (int k = 0; k < p.K; ++k) {
    double best = -INFINITY;
    float best_logit = 0.f;
    int at = INT32_MAX;
    for (int j = 0; j < PER; ++j) {
      if (l[j] == -INFINITY || ((taken >> j) & 1u)) continue;
      const double s = p.sigmoid ? 1.0 / (1.0 + exp(-(double)l[j])) : exp((double)l[j] - (double)top) / inv;
      const double key = s + (double)p.bias[lane + 32 * j];
      if (at == INT32_MAX || key > best) best = key, best_logit = l[j], at = lane + 32 * j;
    }
    for (int d = 16; d; d >>= 1) {
      const double ob = __shfl_xor_sync(kFull, best, d);
      const float ol = __shfl_xor_sync(kFull, best_logit, d);
      const int oa = __shfl_xor_sync(kFull, at, d);
      if (oa != INT32_MAX && (at == INT32_MAX || ob > best || (ob == best && oa < at)))
        best = ob, best_logit = ol, at = oa;
    }
    if (at == INT32_MAX) break;
    if ((at & 31) == lane) taken |= 1u << (at >> 5);
    if (lane == k) *mine = at, *logit = best_logit;
  }
}

// Puts the first `found` lanes' experts in the order of their 64-bit keys.
template <int PER>
__device__ __noinline__ void order_exact(const float (&l)[PER], const RouterParams& p, float top, int lane, int found,
                                         int* mine, float* logit) {
  double sum = 1.0;
  if (!p.sigmoid) {
    sum = 0.0;
    for (int j = 0; j < PER; ++j)
      if (l[j] != -INFINITY) sum += exp((double)l[j] - (double)top);
    sum = warp_sum(sum);
  }
  double key = -INFINITY;
  if (lane < found) {
    const double v = *logit;
    key = (p.sigmoid ? 1.0 / (1.0 + exp(-v)) : exp(v - (double)top) / sum) + (double)p.bias[*mine];
  }
  int rank = 0;
  for (int j = 0; j < found; ++j) {
    const double other = __shfl_sync(kFull, key, j);
    const int id = __shfl_sync(kFull, *mine, j);
    rank += other > key || (other == key && id < *mine);
  }
  int id = -1;
  float v = 0.f;
  for (int j = 0; j < found; ++j) {
    const int r = __shfl_sync(kFull, rank, j), i = __shfl_sync(kFull, *mine, j);
    const float x = __shfl_sync(kFull, *logit, j);
    if (r == lane) id = i, v = x;
  }
  *mine = id;
  *logit = v;
}

template <int PER, bool BF16>
__global__ void __launch_bounds__(kRouterWarps * 32) route_topk_kernel(const RouterParams p) {
  afd::pdl_wait();
  afd::pdl_launch_dependents();
  const int lane = threadIdx.x & 31;
  const int t = blockIdx.x * kRouterWarps + (threadIdx.x >> 5);
  if (t >= p.T) return;
  int mine = -1;        // lane k: the expert of slot k ...
  float score = 0.f;    // ... and its score
  float total = 0.f;    // sum of the selected scores
  if (!p.live || t < *p.live) {
    // Logits; NaN, -infinity, a NaN or -infinite bias and columns past E
    // become -infinity (never selected), +infinity the largest finite value.
    float l[PER];
    uint32_t key[PER];
    float top = -INFINITY;
#pragma unroll
    for (int j = 0; j < PER; ++j) {
      const int e = lane + 32 * j;
      float v = -INFINITY;
      if (e < p.E) {
        if (BF16)
          v = __uint_as_float((uint32_t)reinterpret_cast<const uint16_t*>(p.logits)[t * p.row_stride + e] << 16);
        else
          v = reinterpret_cast<const float*>(p.logits)[t * p.row_stride + e];
        if (v != v) v = -INFINITY;
        if (p.bias) {
          const float b = p.bias[e];
          if (b != b || b == -INFINITY) v = -INFINITY;
        }
      }
      l[j] = fminf(v, FLT_MAX);
      top = fmaxf(top, l[j]);
    }
#pragma unroll
    for (int d = 16; d; d >>= 1) top = fmaxf(top, __shfl_xor_sync(kFull, top, d));
    float inv = 1.f;
    if (!p.sigmoid && (p.bias || !p.renormalize)) {
      float sum = 0.f;
#pragma unroll
      for (int j = 0; j < PER; ++j)
        if (l[j] != -INFINITY) sum += expf(l[j] - top);
      inv = 1.f / warp_sum(sum);
    }
    // Scores: with renormalised softmax the sum over all experts cancels.
    auto score_of = [&](float v) { return p.sigmoid ? 1.f / (1.f + expf(-v)) : expf(v - top) * inv; };
#pragma unroll
    for (int j = 0; j < PER; ++j) {
      key[j] = 0;
      if (l[j] == -INFINITY) continue;
      const float k = p.bias ? score_of(l[j]) + p.bias[lane + 32 * j] : l[j];
      key[j] = order_image(k);
    }
    // A round: the expert with the largest key, which it loses, and its logit.
    auto pick = [&](int* expert, float* value) {
      uint32_t best = 0;
#pragma unroll
      for (int j = 0; j < PER; ++j) best = max(best, key[j]);
      best = __reduce_max_sync(kFull, best);
      if (best == 0) return best;
      uint32_t at = 0xffffffffu;
#pragma unroll
      for (int j = PER - 1; j >= 0; --j)
        if (key[j] == best) at = lane + 32 * j;
      at = __reduce_min_sync(kFull, at);
      float v = 0.f;
#pragma unroll
      for (int j = 0; j < PER; ++j)
        if ((int)at == lane + 32 * j) v = l[j], key[j] = 0;
      *expert = (int)at;
      *value = __shfl_sync(kFull, v, at & 31);
      return best;
    };
    float logit = 0.f, kept = 0.f;  // lane k: the logit and the key of slot k
    int found = 0;
    for (; found < p.K; ++found) {
      int at;
      float v;
      const uint32_t best = pick(&at, &v);
      if (best == 0) break;
      if (lane == found) mine = at, logit = v, kept = from_image(best);
    }
    if (p.bias) {
      // Whether two keys are too close to tell (a score is at most 1, which
      // spares most tokens its second reckoning).
      auto near = [&](float va, int ea, float ka, float vb, int eb, float kb) {
        if (ka - kb > key_slack(p.sigmoid, 1.f, 1.f, ka, kb)) return false;
        if (va == vb && p.bias[ea] == p.bias[eb]) return false;
        return !(ka - kb > key_slack(p.sigmoid, score_of(va), score_of(vb), ka, kb));
      };
      // The rounds go on until no expert that is left can belong to the first K:
      // none has a key near enough to one of theirs for the largest score that
      // is left (1 at first, which most tokens' gap exceeds). The next key alone
      // does not tell: behind one that is apart, or equal to the last slot's,
      // one with a larger score, and so a larger error, may follow.
      bool over = false;
      float left = -1.f, own = 0.f;
      auto apart = [&](float score_left, float score_own, float k) {
        return __all_sync(kFull, lane >= p.K || kept - k > key_slack(p.sigmoid, score_left, score_own, kept, k));
      };
      while (found >= p.K) {
        int at;
        float v;
        const uint32_t best = pick(&at, &v);
        if (best == 0) break;
        const float k = from_image(best);
        if (apart(1.f, 1.f, k)) break;
        if (left < 0.f) {
          float most = v;
#pragma unroll
          for (int j = 0; j < PER; ++j)
            if (key[j]) most = fmaxf(most, l[j]);
#pragma unroll
          for (int d = 16; d; d >>= 1) most = fmaxf(most, __shfl_xor_sync(kFull, most, d));
          left = score_of(most);
          if (lane < p.K) own = score_of(logit);
        }
        if (apart(left, own, k)) break;
        // Of equal experts (the same logit and bias) the first K will do.
        const float b = p.bias[at];
        if (__popc(__ballot_sync(kFull, lane < found && logit == v && p.bias[max(mine, 0)] == b)) >= p.K) {
#pragma unroll
          for (int j = 0; j < PER; ++j)
            if (key[j] && l[j] == v && p.bias[lane + 32 * j] == b) key[j] = 0;
          continue;
        }
        over = found == 32;
        if (over) break;
        if (lane == found) mine = at, logit = v, kept = k;
        ++found;
      }
      // If any two are near without being equal, two neighbours are.
      const float va = __shfl_up_sync(kFull, logit, 1), ka = __shfl_up_sync(kFull, kept, 1);
      const int ea = __shfl_up_sync(kFull, mine, 1);
      const bool close = __any_sync(kFull, lane > 0 && lane < found && near(va, ea, ka, logit, mine, kept));
      if (over)
        select_exact<PER>(l, p, top, lane, &mine, &logit);
      else if (close)
        order_exact<PER>(l, p, top, lane, found, &mine, &logit);
    }
    if (lane >= p.K) mine = -1;
    if (p.renormalize) {
      // A factor common to the selected scores cancels: exp(-top) of softmax,
      // and for sigmoid(v) = exp(min(v, 0)) / (1 + exp(-|v|)) that of the
      // largest exponent, so that small scores do not underflow first.
      float v = mine < 0 ? -INFINITY : p.sigmoid ? fminf(logit, 0.f) : logit;
      float m = v;
#pragma unroll
      for (int d = 16; d; d >>= 1) m = fmaxf(m, __shfl_xor_sync(kFull, m, d));
      if (mine >= 0) score = p.sigmoid ? expf(v - m) / (1.f + expf(-fabsf(logit))) : expf(v - m);
      total = warp_sum(score);
    } else if (mine >= 0) {
      score = score_of(logit);
    }
  }
  if (lane < p.K) {
    const float w = p.renormalize && mine >= 0 ? score / total : score;
    p.ids[(int64_t)t * p.K + lane] = mine;
    p.weights[(int64_t)t * p.K + lane] = p.scale * w;
  }
}

template <int PER>
cudaError_t launch_router(const RouterParams& p, bool bf16, cudaStream_t stream) {
  const int grid = (p.T + kRouterWarps - 1) / kRouterWarps;
  return bf16 ? afd::launch_dependent(route_topk_kernel<PER, true>, grid, kRouterWarps * 32, 0, stream, p)
              : afd::launch_dependent(route_topk_kernel<PER, false>, grid, kRouterWarps * 32, 0, stream, p);
}

}  // namespace

extern "C" AFD_API afd_status afd_route_topk(const void* logits, int32_t logits_dtype, int64_t row_stride,
                                             const float* bias, const int32_t* live_tokens, int32_t num_tokens,
                                             int32_t num_experts, int32_t top_k, int32_t scoring,
                                             int32_t renormalize, float scale, int64_t* ids, float* weights,
                                             afd_stream stream) {
  const int T = num_tokens, E = num_experts, K = top_k;
  if (T < 0 || E < 1 || K < 1 || K > E || K > 32 || row_stride < E) return AFD_ERR_ARG;
  if (T > 0 && (!logits || !ids || !weights)) return AFD_ERR_ARG;
  if (logits_dtype != AFD_BF16 && logits_dtype != AFD_FP32) return AFD_ERR_ARG;
  if (scoring != AFD_SCORE_SOFTMAX && scoring != AFD_SCORE_SIGMOID) return AFD_ERR_ARG;
  if (renormalize != 0 && renormalize != 1) return AFD_ERR_ARG;
  if (E > 1024 || T > afd::kMaxRows) return AFD_ERR_UNSUPPORTED;
  if (T == 0) return AFD_OK;
  RouterParams p = {logits, row_stride, bias, live_tokens, T, E, K, scoring == AFD_SCORE_SIGMOID, renormalize,
                    scale, ids, weights};
  const uint8_t* l8 = nullptr;
  if (!afd::device_view(static_cast<const uint8_t*>(logits), &l8) || !afd::device_view(ids, &p.ids) ||
      !afd::device_view(weights, &p.weights) || (bias && !afd::device_view(bias, &p.bias)) ||
      (live_tokens && !afd::device_view(live_tokens, &p.live)))
    return AFD_ERR_ARG;
  if (!afd::aligned_to(l8, logits_dtype == AFD_BF16 ? 2 : 4) || !afd::aligned_to(p.ids, 8) ||
      !afd::aligned_to(p.weights, 4) || !afd::aligned_to(p.bias, 4) || !afd::aligned_to(p.live, 4))
    return AFD_ERR_ARG;
  p.logits = l8;
  const bool bf16 = logits_dtype == AFD_BF16;
  cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
  cudaError_t e;
  if (E <= 32) e = launch_router<1>(p, bf16, s);
  else if (E <= 64) e = launch_router<2>(p, bf16, s);
  else if (E <= 128) e = launch_router<4>(p, bf16, s);
  else if (E <= 256) e = launch_router<8>(p, bf16, s);
  else if (E <= 512) e = launch_router<16>(p, bf16, s);
  else e = launch_router<32>(p, bf16, s);
  return e == cudaSuccess ? AFD_OK : AFD_ERR_CUDA;
}
