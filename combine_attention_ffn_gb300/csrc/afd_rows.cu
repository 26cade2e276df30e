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

// Low-rank adapters. A cluster of four CTAs takes 64 rows at a time; the rows'
// adapters are found first (their distinct slots and which 16-row tiles hold
// them), then
//   down: t = down[a] x for every row, K split over the cluster's CTAs and four
//         warps in each, the parts joined through distributed shared memory in
//         a fixed order;
//   up:   out = base + (scale t) up[a], the columns split the same way.
// Both products run for every slot of a 16-row tile, and each row keeps its own
// slot's (by selection, not by zeros: an adapter that holds an infinity must
// not reach another request's rows). The operands go from global memory
// straight into registers: the order of K (and of the output's columns) inside
// a fragment is free as long as both sides agree, so a thread takes eight
// neighbouring values, 16 bytes at a time.
// What bounds it is the traffic of x, base and out (about 6 bytes a column and
// row against 2 rank flops): mma.sync's rate is enough, and its row masks and
// register operands spare the copies through shared memory and TMEM.
// t is FP32; for the up product it is split into two BF16 (16 bits and more).
constexpr int kAdRows = 64;
constexpr int kAdCtas = 4;      // a cluster's CTAs
constexpr int kAdParts = 4;     // warps of a CTA that share 32 rows
constexpr int kAdSplit = kAdCtas * kAdParts;
constexpr int kAdThreads = 256;

__device__ __forceinline__ void mma_16816(float (&c)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3,
                                          uint32_t b0, uint32_t b1) {
  asm("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, {%0, %1, %2, %3};"
      : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

__device__ __forceinline__ float2 ld_cluster2(const float* p, uint32_t rank) {
  uint32_t a = (uint32_t)__cvta_generic_to_shared(p);
  float2 v;
  asm volatile("mapa.shared::cluster.u32 %0, %0, %1;" : "+r"(a) : "r"(rank));
  asm volatile("ld.shared::cluster.v2.f32 {%0, %1}, [%2];" : "=f"(v.x), "=f"(v.y) : "r"(a) : "memory");
  return v;
}

template <int RANK>
struct AdapterShared {
  static constexpr int kPad = RANK + 4;    // FP32 row
  static constexpr int kPadH = RANK + 8;   // BF16 row
  alignas(16) float part[kAdParts][kAdRows][kPad];
  alignas(16) uint16_t hi[kAdRows][kPadH], lo[kAdRows][kPadH];
  int slot[kAdRows];             // the row's adapter, -1 none, -2 not a row
  int list[kAdRows], mask[kAdRows];  // distinct adapters and the 16-row tiles that hold them
  int count, rows;               // adapters of this tile; whether it has any row
};

template <int RANK>
__global__ void __cluster_dims__(kAdCtas, 1, 1) __launch_bounds__(kAdThreads, RANK <= 32 ? 2 : 1)
    adapter_kernel(const AdapterParams p) {
  using Sh = AdapterShared<RANK>;
  extern __shared__ __align__(16) uint8_t ad_smem[];
  Sh& sh = *reinterpret_cast<Sh*>(ad_smem);
  constexpr int NT = RANK / 8;                        // 8-column tiles of the down product
  constexpr int U = RANK <= 32 ? 4 : 2;               // K chunks of 32 loaded together
  constexpr int EL = RANK >= 32 ? 8 : RANK / 4;       // rank values a thread takes at a time
  constexpr int CH = RANK >= 32 ? RANK / 32 : 1;      // ... and how often
  constexpr int STEPS = EL == 8 ? 2 : 1;              // products per chunk
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int g = lane >> 2, tig = lane & 3;
  const int wr = warp & 1, wk = warp >> 1;            // half of the rows; part of K and of the columns
  const int cta = blockIdx.x % kAdCtas, cluster = blockIdx.x / kAdCtas, clusters = gridDim.x / kAdCtas;
  const int part = cta * kAdParts + wk;
  const int limit = p.row_src ? afd::group_end(p.ends[p.G - 1], p.R) : p.R;
  const int chunks = (p.K + 31) >> 5, groups = (p.N + 31) >> 5;
  bool open = false;  // this CTA has told the cluster that it has read its parts, and not waited yet

  for (int64_t r0 = (int64_t)cluster * kAdRows; r0 < limit; r0 += (int64_t)clusters * kAdRows) {
    // ------------------------------------------------------ the rows' adapters
    __syncthreads();
    int mine = -2;
    if (threadIdx.x < kAdRows) {
      const int64_t r = r0 + threadIdx.x;
      if (r < limit) {
        int t = (int)r;
        if (p.row_src) {
          const int src = p.row_src[r];
          t = src < 0 ? -1 : src / p.top_k;
        }
        if (t >= 0 && t < p.tokens) {
          mine = p.token_slots[t];
          if (mine < 0 || mine >= p.S) mine = -1;
        }
      }
      sh.slot[threadIdx.x] = mine;
      sh.mask[threadIdx.x] = 0;
    }
    const int any = __syncthreads_or(mine > -2);
    if (!any) continue;  // the same in every CTA of the cluster
    // The distinct adapters: those of the first 32 rows, then what the others add.
    int at = -1;
#pragma unroll
    for (int w = 0; w < kAdRows / 32; ++w) {
      if (warp == w) {
        const int before = w ? sh.count : 0;
        for (int i = 0; i < before; ++i)
          if (sh.list[i] == mine) at = i;
        const unsigned same = __match_any_sync(0xffffffffu, mine);
        const int leader = __ffs(same) - 1;
        const unsigned opens = __ballot_sync(0xffffffffu, mine >= 0 && at < 0 && lane == leader);
        if (mine >= 0 && at < 0) at = before + __popc(opens & ((1u << leader) - 1));
        if (mine >= 0 && (opens >> lane & 1)) sh.list[at] = mine;
        if (lane == 0) sh.count = before + __popc(opens);
        if (mine >= 0) atomicOr(&sh.mask[at], 1 << (threadIdx.x >> 4));
      }
      __syncthreads();
    }
    const int count = sh.count;
    int slot[2][2];  // of this thread's rows: [16-row tile][g / g + 8]
#pragma unroll
    for (int s = 0; s < 2; ++s)
#pragma unroll
      for (int h = 0; h < 2; ++h) slot[s][h] = sh.slot[32 * wr + 16 * s + 8 * h + g];

    if (count) {
      // ---------------------------------------------------------------- down
      float acc[2][NT][4];
#pragma unroll
      for (int s = 0; s < 2; ++s)
#pragma unroll
        for (int n = 0; n < NT; ++n)
#pragma unroll
          for (int i = 0; i < 4; ++i) acc[s][n][i] = 0.f;
      for (int c0 = part; c0 < chunks; c0 += U * kAdSplit) {
        uint4 xv[U][2][2];
#pragma unroll
        for (int u = 0; u < U; ++u) {
          const int k = (c0 + u * kAdSplit) * 32 + tig * 8;
#pragma unroll
          for (int s = 0; s < 2; ++s)
#pragma unroll
            for (int h = 0; h < 2; ++h)
              xv[u][s][h] = k < p.K && slot[s][h] >= 0
                                ? afd::ld_once(reinterpret_cast<const uint4*>(
                                      p.x + (r0 + 32 * wr + 16 * s + 8 * h + g) * p.x_stride + k))
                                : make_uint4(0, 0, 0, 0);
        }
        for (int d = 0; d < count; ++d) {
          const int m = sh.mask[d] >> (2 * wr) & 3;
          if (!m) continue;
          const int a = sh.list[d];
#pragma unroll
          for (int n = 0; n < NT; ++n) {
            float v[2][4] = {};
#pragma unroll
            for (int u = 0; u < U; ++u) {
              const int k = (c0 + u * kAdSplit) * 32 + tig * 8;
              const uint4 b = k < p.K ? __ldg(reinterpret_cast<const uint4*>(p.down + ((int64_t)a * RANK + n * 8 + g) * p.K + k))
                                      : make_uint4(0, 0, 0, 0);
#pragma unroll
              for (int s = 0; s < 2; ++s) {
                if (!(m >> s & 1)) continue;
                const uint4 &x0 = xv[u][s][0], &x1 = xv[u][s][1];
                mma_16816(v[s], x0.x, x1.x, x0.y, x1.y, b.x, b.y);
                mma_16816(v[s], x0.z, x1.z, x0.w, x1.w, b.z, b.w);
              }
            }
#pragma unroll
            for (int s = 0; s < 2; ++s)
#pragma unroll
              for (int h = 0; h < 2; ++h)
                if (slot[s][h] == a) {
                  acc[s][n][2 * h] += v[s][2 * h];
                  acc[s][n][2 * h + 1] += v[s][2 * h + 1];
                }
          }
        }
      }
      if (open) {  // the others have read the last tile's parts
        asm volatile("barrier.cluster.wait.acquire.aligned;" ::: "memory");
        open = false;
      }
#pragma unroll
      for (int s = 0; s < 2; ++s)
#pragma unroll
        for (int n = 0; n < NT; ++n)
#pragma unroll
          for (int h = 0; h < 2; ++h)
            *reinterpret_cast<float2*>(&sh.part[wk][32 * wr + 16 * s + 8 * h + g][8 * n + 2 * tig]) =
                make_float2(acc[s][n][2 * h], acc[s][n][2 * h + 1]);
      __syncthreads();
      for (int i = threadIdx.x; i < kAdRows * RANK / 2; i += kAdThreads) {
        const int r = i / (RANK / 2), c = i % (RANK / 2) * 2;
        float2 t = *reinterpret_cast<const float2*>(&sh.part[0][r][c]);
#pragma unroll
        for (int w = 1; w < kAdParts; ++w) {
          const float2 v = *reinterpret_cast<const float2*>(&sh.part[w][r][c]);
          t.x += v.x, t.y += v.y;
        }
        *reinterpret_cast<float2*>(&sh.part[0][r][c]) = t;
      }
      asm volatile("barrier.cluster.arrive.release.aligned;\nbarrier.cluster.wait.acquire.aligned;" ::: "memory");
      for (int i = threadIdx.x; i < kAdRows * RANK / 2; i += kAdThreads) {
        const int r = i / (RANK / 2), c = i % (RANK / 2) * 2;
        float2 t = make_float2(0.f, 0.f);
#pragma unroll
        for (int w = 0; w < kAdCtas; ++w) {
          const float2 v = ld_cluster2(&sh.part[0][r][c], w);
          t.x += v.x, t.y += v.y;
        }
        const float scale = sh.slot[r] >= 0 ? p.scales[sh.slot[r]] : 0.f;
        t.x *= scale, t.y *= scale;
        // (an infinite product stays one: nothing is left of it then)
        const uint32_t hi = afd::pack_bf16(t.x, t.y);
        *reinterpret_cast<uint32_t*>(&sh.hi[r][c]) = hi;
        *reinterpret_cast<uint32_t*>(&sh.lo[r][c]) =
            afd::pack_bf16(isinf(t.x) ? 0.f : t.x - __uint_as_float(hi << 16),
                           isinf(t.y) ? 0.f : t.y - __uint_as_float(hi & 0xffff0000u));
      }
      asm volatile("barrier.cluster.arrive.release.aligned;" ::: "memory");
      open = true;
      __syncthreads();
    }

    // -------------------------------------------------------------------- up
    uint32_t th[2][2][CH][EL / 2], tl[2][2][CH][EL / 2];  // [tile][g / g + 8]
#pragma unroll
    for (int s = 0; s < 2; ++s)
#pragma unroll
      for (int h = 0; h < 2; ++h)
#pragma unroll
        for (int q = 0; q < CH; ++q)
#pragma unroll
          for (int e = 0; e < EL / 2; ++e) {
            const int r = 32 * wr + 16 * s + 8 * h + g, c = q * 32 + tig * EL + 2 * e;
            th[s][h][q][e] = slot[s][h] >= 0 ? *reinterpret_cast<const uint32_t*>(&sh.hi[r][c]) : 0u;
            tl[s][h][q][e] = slot[s][h] >= 0 ? *reinterpret_cast<const uint32_t*>(&sh.lo[r][c]) : 0u;
          }
    for (int gi = part; gi < groups; gi += kAdSplit) {
      const int n0 = gi * 32;
      const bool in = n0 + tig * 8 < p.N;  // this thread's eight output columns
      uint4 bv[2][2];
#pragma unroll
      for (int s = 0; s < 2; ++s)
#pragma unroll
        for (int h = 0; h < 2; ++h)
          if (in && slot[s][h] > -2)
            bv[s][h] = *reinterpret_cast<const uint4*>(p.base + (r0 + 32 * wr + 16 * s + 8 * h + g) * p.base_stride + n0 + tig * 8);
      float acc[2][4][4];  // [row tile][column tile]
#pragma unroll
      for (int s = 0; s < 2; ++s)
#pragma unroll
        for (int i = 0; i < 4; ++i)
#pragma unroll
          for (int e = 0; e < 4; ++e) acc[s][i][e] = 0.f;
      for (int d = 0; d < count; ++d) {
        const int m = sh.mask[d] >> (2 * wr) & 3;
        if (!m) continue;
        const int a = sh.list[d];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          // column tile i holds columns 8 j + 2 i and 8 j + 2 i + 1, so that a
          // thread ends with eight neighbouring ones
          const int n = n0 + (g >> 1) * 8 + 2 * i + (g & 1);
          const uint16_t* up = p.up + ((int64_t)a * p.N + n) * RANK + tig * EL;
          float v[2][4] = {};
#pragma unroll
          for (int q = 0; q < CH; ++q) {
            uint32_t b[EL / 2];
            if (EL == 8) {
              const uint4 v = n < p.N ? __ldg(reinterpret_cast<const uint4*>(up + q * 32)) : make_uint4(0, 0, 0, 0);
              b[0] = v.x, b[1 % (EL / 2)] = v.y, b[2 % (EL / 2)] = v.z, b[3 % (EL / 2)] = v.w;
            } else if (EL == 4) {
              const uint2 v = n < p.N ? __ldg(reinterpret_cast<const uint2*>(up)) : make_uint2(0, 0);
              b[0] = v.x, b[1 % (EL / 2)] = v.y;
            } else {
              b[0] = n < p.N ? __ldg(reinterpret_cast<const uint32_t*>(up)) : 0u;
            }
#pragma unroll
            for (int s = 0; s < 2; ++s) {
              if (!(m >> s & 1)) continue;
#pragma unroll
              for (int st = 0; st < STEPS; ++st) {
                const int e0 = 2 * st, e1 = EL == 2 ? 0 : 2 * st + 1;
                const bool two = EL != 2;  // rank 8 fills half of a product's K
                mma_16816(v[s], th[s][0][q][e0], th[s][1][q][e0], two ? th[s][0][q][e1] : 0u, two ? th[s][1][q][e1] : 0u,
                          b[e0], two ? b[e1] : 0u);
                mma_16816(v[s], tl[s][0][q][e0], tl[s][1][q][e0], two ? tl[s][0][q][e1] : 0u, two ? tl[s][1][q][e1] : 0u,
                          b[e0], two ? b[e1] : 0u);
              }
            }
          }
#pragma unroll
          for (int s = 0; s < 2; ++s)
#pragma unroll
            for (int h = 0; h < 2; ++h)
              if (slot[s][h] == a) acc[s][i][2 * h] = v[s][2 * h], acc[s][i][2 * h + 1] = v[s][2 * h + 1];
        }
      }
#pragma unroll
      for (int s = 0; s < 2; ++s)
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          if (!in || slot[s][h] <= -2) continue;
          uint4 o = bv[s][h];
          if (slot[s][h] >= 0) {
            float f[8];
            afd::bf16x8_to_float(o, f);
#pragma unroll
            for (int i = 0; i < 4; ++i) {
              f[2 * i] += acc[s][i][2 * h];
              f[2 * i + 1] += acc[s][i][2 * h + 1];
            }
            o = afd::float_to_bf16x8(f);
          }
          *reinterpret_cast<uint4*>(p.out + (r0 + 32 * wr + 16 * s + 8 * h + g) * p.out_stride + n0 + tig * 8) = o;
        }
    }
  }
  if (open) asm volatile("barrier.cluster.wait.acquire.aligned;" ::: "memory");
}

template <int RANK>
cudaError_t launch_adapters(const AdapterParams& p, int sms, cudaStream_t stream) {
  constexpr int kSmem = sizeof(AdapterShared<RANK>);
  const cudaError_t e = cudaFuncSetAttribute(adapter_kernel<RANK>, cudaFuncAttributeMaxDynamicSharedMemorySize, kSmem);
  if (e != cudaSuccess) return e;
  const int tiles = (int)(((int64_t)p.R + kAdRows - 1) / kAdRows);
  const int most = sms * (RANK <= 32 ? 2 : 1) / kAdCtas;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)((tiles < most ? tiles : most) * kAdCtas));
  cfg.blockDim = dim3(kAdThreads);
  cfg.dynamicSmemBytes = kSmem;
  cfg.stream = stream;
  return cudaLaunchKernelEx(&cfg, adapter_kernel<RANK>, p);
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
  cudaStream_t st = reinterpret_cast<cudaStream_t>(stream);
  const cudaError_t e = rank == 8    ? launch_adapters<8>(p, sms, st)
                        : rank == 16 ? launch_adapters<16>(p, sms, st)
                        : rank == 32 ? launch_adapters<32>(p, sms, st)
                                     : launch_adapters<64>(p, sms, st);
  return e == cudaSuccess ? AFD_OK : AFD_ERR_CUDA;
}

}  // extern "C"
