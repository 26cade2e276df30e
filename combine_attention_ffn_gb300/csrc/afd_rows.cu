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
  int32_t* first;  // workspace: where each adapter's rows start in `order`, [S + 2]
  int32_t* order;  // workspace: the live rows by adapter, [R]
};

// Low-rank adapters, in two launches. The first groups the rows by adapter
// (a request's rows are spread over every expert's range, so rows that follow
// one another mostly differ in theirs): a permutation of the live rows, sorted
// by adapter, and where each adapter starts. In the second a cluster of four
// CTAs takes up to 64 rows of one adapter at a time:
//   down: t = down[a] x, K split over the cluster's CTAs and four warps in
//         each, the parts joined through distributed shared memory in a fixed
//         order;
//   up:   out = base + (scale t) up[a], the columns split the same way.
// The operands go from global memory straight into registers: the order of K
// (and of the output's columns) inside a fragment is free as long as both
// sides agree, so a thread takes eight neighbouring values, 16 bytes at a time.
// What bounds it is the traffic of x, base and out (about 6 bytes a column and
// row against 2 rank flops): mma.sync's rate is enough, and its register
// operands spare the copies through shared memory and TMEM. A product's rows
// do not mix, so neither the order of the rows inside a group nor what another
// request's adapter holds reaches a result.
// t is FP32; for the up product it is split into two BF16 (16 bits and more).
constexpr int kMaxSlots = 1024;
constexpr int kGroupCtas = 8;
constexpr int kGroupThreads = 1024;
constexpr int kAdRows = 64;
constexpr int kAdCtas = 4;      // a cluster's CTAs
constexpr int kAdParts = 4;     // warps of a CTA that share 32 rows
constexpr int kAdSplit = kAdCtas * kAdParts;
constexpr int kAdThreads = 256;

// The group of a row: its adapter, S for none, -1 for what is not a row.
__device__ __forceinline__ int row_group(const AdapterParams& p, int r) {
  int t = r;
  if (p.row_src) {
    const int src = p.row_src[r];
    if (src < 0) return -1;
    t = src / p.top_k;
  }
  if (t >= p.tokens) return -1;
  const int a = p.token_slots[t];
  return a >= 0 && a < p.S ? a : p.S;
}

__device__ __forceinline__ uint32_t remote(const void* p, uint32_t rank) {
  uint32_t a = (uint32_t)__cvta_generic_to_shared(p);
  asm volatile("mapa.shared::cluster.u32 %0, %0, %1;" : "+r"(a) : "r"(rank));
  return a;
}

__device__ __forceinline__ void cluster_sync() {
  asm volatile("barrier.cluster.arrive.release.aligned;\nbarrier.cluster.wait.acquire.aligned;" ::: "memory");
}

// One cluster: counts per adapter and CTA, their prefix, then every row's
// place. Inside a group the order is that of the atomics; no result depends
// on it.
__global__ void __cluster_dims__(kGroupCtas, 1, 1) __launch_bounds__(kGroupThreads) adapter_group_kernel(const AdapterParams p) {
  __shared__ int count[kMaxSlots + 1], cursor[kMaxSlots + 1];
  __shared__ int warp_total[kGroupThreads / 32];
  afd::pdl_launch_dependents();
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const uint32_t cta = blockIdx.x;
  const int groups = p.S + 1;
  const int limit = p.row_src ? afd::group_end(p.ends[p.G - 1], p.R) : p.R;
  const int share = ((limit + kGroupCtas - 1) / kGroupCtas + 31) & ~31;
  const int64_t lo = (int64_t)cta * share, hi = lo + share < limit ? lo + share : limit;
  for (int g = threadIdx.x; g < groups; g += kGroupThreads) count[g] = 0;
  __syncthreads();
  for (int64_t r0 = lo + 32 * warp; r0 < hi; r0 += kGroupThreads) {
    const int g = r0 + lane < hi ? row_group(p, (int)r0 + lane) : -1;
    const unsigned same = __match_any_sync(0xffffffffu, g);
    if (g >= 0 && lane == __ffs(same) - 1) atomicAdd(&count[g], __popc(same));
  }
  cluster_sync();
  // a thread takes `each` neighbouring groups of the prefix sum
  const int each = (groups + kGroupThreads - 1) / kGroupThreads;
  int total[2] = {0, 0}, before[2] = {0, 0};  // each <= 2
  for (int i = 0; i < each; ++i) {
    const int g = threadIdx.x * each + i;
    if (g >= groups) break;
#pragma unroll
    for (uint32_t c = 0; c < kGroupCtas; ++c) {
      int v;
      asm volatile("ld.shared::cluster.s32 %0, [%1];" : "=r"(v) : "r"(remote(&count[g], c)) : "memory");
      total[i] += v;
      if (c < cta) before[i] += v;
    }
  }
  int run = afd::warp_inclusive_scan(total[0] + total[1]);
  if (lane == 31) warp_total[warp] = run;
  __syncthreads();
  if (warp == 0) {
    const int t = warp_total[lane];
    warp_total[lane] = afd::warp_inclusive_scan(t) - t;
  }
  __syncthreads();
  run += warp_total[warp] - total[0] - total[1];
  for (int i = 0; i < each; ++i) {
    const int g = threadIdx.x * each + i;
    if (g >= groups) break;
    cursor[g] = run + before[i];
    if (cta == 0) p.first[g] = run;
    run += total[i];
    if (cta == 0 && g == groups - 1) p.first[groups] = run;
  }
  __syncthreads();
  for (int64_t r0 = lo + 32 * warp; r0 < hi; r0 += kGroupThreads) {
    const int g = r0 + lane < hi ? row_group(p, (int)r0 + lane) : -1;
    const unsigned same = __match_any_sync(0xffffffffu, g);
    int at = 0;
    if (g >= 0 && lane == __ffs(same) - 1) at = atomicAdd(&cursor[g], __popc(same));
    at = __shfl_sync(0xffffffffu, at, __ffs(same) - 1) + __popc(same & ((1u << lane) - 1));
    if (g >= 0) p.order[at] = (int)r0 + lane;
  }
  cluster_sync();  // nobody leaves while its counts may be read
}

__device__ __forceinline__ void mma_16816(float (&c)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3,
                                          uint32_t b0, uint32_t b1) {
  asm("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, {%0, %1, %2, %3};"
      : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

template <int RANK>
struct AdapterShared {
  static constexpr int kPad = RANK + 4;    // FP32 row
  static constexpr int kPadH = RANK + 8;   // BF16 row
  alignas(16) float part[kAdParts][kAdRows][kPad];
  alignas(16) uint16_t hi[kAdRows][kPadH], lo[kAdRows][kPadH];
  int first[kMaxSlots + 2];       // of the order: where each group starts
  int first_tile[kMaxSlots + 2];
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
  const int chunks = (p.K + 31) >> 5, col_groups = (p.N + 31) >> 5;
  bool open = false;  // this CTA has told the cluster that it has read its parts, and not waited yet

  afd::pdl_wait();  // the grouping
  for (int i = threadIdx.x; i < p.S + 2; i += kAdThreads) sh.first[i] = p.first[i];
  __syncthreads();
  if (warp == 0) {
    int carry = 0;
    for (int i0 = 0; i0 <= p.S; i0 += 32) {
      const int i = i0 + lane;
      const int t = i <= p.S ? (sh.first[i + 1] - sh.first[i] + kAdRows - 1) / kAdRows : 0;
      const int incl = afd::warp_inclusive_scan(t);
      if (i <= p.S) sh.first_tile[i] = carry + incl - t;
      carry += __shfl_sync(0xffffffffu, incl, 31);
    }
    if (lane == 0) sh.first_tile[p.S + 1] = carry;
  }
  __syncthreads();
  const int tiles = sh.first_tile[p.S + 1];

  for (int t = cluster; t < tiles; t += clusters) {
    int a = 0;  // the last group that starts at or before this tile
    for (int hi = p.S; a < hi;) {
      const int mid = (a + hi + 1) >> 1;
      if (sh.first_tile[mid] <= t) a = mid; else hi = mid - 1;
    }
    const int at = sh.first[a] + (t - sh.first_tile[a]) * kAdRows, end = sh.first[a + 1];
    int64_t row[2][2];  // of this thread: [16-row tile][g / g + 8]; -1: none
#pragma unroll
    for (int s = 0; s < 2; ++s)
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        const int i = at + 32 * wr + 16 * s + 8 * h + g;
        row[s][h] = i < end ? p.order[i] : -1;
      }
    const bool adapt = a < p.S;  // the last group has no adapter: its rows are copied

    if (adapt) {
      // ---------------------------------------------------------------- down
      float acc[2][NT][4];
#pragma unroll
      for (int s = 0; s < 2; ++s)
#pragma unroll
        for (int n = 0; n < NT; ++n)
#pragma unroll
          for (int i = 0; i < 4; ++i) acc[s][n][i] = 0.f;
      const uint16_t* down = p.down + ((int64_t)a * RANK + g) * p.K;
      for (int c0 = part; c0 < chunks; c0 += U * kAdSplit) {
        uint4 xv[U][2][2];
#pragma unroll
        for (int u = 0; u < U; ++u) {
          const int k = (c0 + u * kAdSplit) * 32 + tig * 8;
#pragma unroll
          for (int s = 0; s < 2; ++s)
#pragma unroll
            for (int h = 0; h < 2; ++h)
              xv[u][s][h] = k < p.K && row[s][h] >= 0
                                ? afd::ld_once(reinterpret_cast<const uint4*>(p.x + row[s][h] * p.x_stride + k))
                                : make_uint4(0, 0, 0, 0);
        }
#pragma unroll
        for (int u = 0; u < U; ++u) {
          const int k = (c0 + u * kAdSplit) * 32 + tig * 8;
#pragma unroll
          for (int n = 0; n < NT; ++n) {
            const uint4 b = k < p.K ? __ldg(reinterpret_cast<const uint4*>(down + (int64_t)n * 8 * p.K + k)) : make_uint4(0, 0, 0, 0);
#pragma unroll
            for (int s = 0; s < 2; ++s) {
              const uint4 &x0 = xv[u][s][0], &x1 = xv[u][s][1];
              mma_16816(acc[s][n], x0.x, x1.x, x0.y, x1.y, b.x, b.y);
              mma_16816(acc[s][n], x0.z, x1.z, x0.w, x1.w, b.z, b.w);
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
        float2 v = *reinterpret_cast<const float2*>(&sh.part[0][r][c]);
#pragma unroll
        for (int w = 1; w < kAdParts; ++w) {
          const float2 o = *reinterpret_cast<const float2*>(&sh.part[w][r][c]);
          v.x += o.x, v.y += o.y;
        }
        *reinterpret_cast<float2*>(&sh.part[0][r][c]) = v;
      }
      cluster_sync();
      const float scale = p.scales[a];
      for (int i = threadIdx.x; i < kAdRows * RANK / 2; i += kAdThreads) {
        const int r = i / (RANK / 2), c = i % (RANK / 2) * 2;
        float2 v = make_float2(0.f, 0.f);
#pragma unroll
        for (int w = 0; w < kAdCtas; ++w) {
          float2 o;
          asm volatile("ld.shared::cluster.v2.f32 {%0, %1}, [%2];" : "=f"(o.x), "=f"(o.y) : "r"(remote(&sh.part[0][r][c], w)) : "memory");
          v.x += o.x, v.y += o.y;
        }
        v.x *= scale, v.y *= scale;
        const uint32_t hi = afd::pack_bf16(v.x, v.y);
        *reinterpret_cast<uint32_t*>(&sh.hi[r][c]) = hi;
        // (an infinite product leaves no rest)
        *reinterpret_cast<uint32_t*>(&sh.lo[r][c]) =
            afd::pack_bf16(isinf(v.x) ? 0.f : v.x - __uint_as_float(hi << 16),
                           isinf(v.y) ? 0.f : v.y - __uint_as_float(hi & 0xffff0000u));
      }
      asm volatile("barrier.cluster.arrive.release.aligned;" ::: "memory");
      open = true;
      __syncthreads();
    }

    // -------------------------------------------------------------------- up
    uint32_t th[2][2][CH][EL / 2], tl[2][2][CH][EL / 2];  // [tile][g / g + 8]
    if (adapt) {
#pragma unroll
      for (int s = 0; s < 2; ++s)
#pragma unroll
        for (int h = 0; h < 2; ++h)
#pragma unroll
          for (int q = 0; q < CH; ++q)
#pragma unroll
            for (int e = 0; e < EL / 2; ++e) {
              const int r = 32 * wr + 16 * s + 8 * h + g, c = q * 32 + tig * EL + 2 * e;
              th[s][h][q][e] = *reinterpret_cast<const uint32_t*>(&sh.hi[r][c]);
              tl[s][h][q][e] = *reinterpret_cast<const uint32_t*>(&sh.lo[r][c]);
            }
    }
    for (int gi = part; gi < col_groups; gi += kAdSplit) {
      const int n0 = gi * 32;
      const bool in = n0 + tig * 8 < p.N;  // this thread's eight output columns
      uint4 bv[2][2];
#pragma unroll
      for (int s = 0; s < 2; ++s)
#pragma unroll
        for (int h = 0; h < 2; ++h)
          if (in && row[s][h] >= 0) bv[s][h] = *reinterpret_cast<const uint4*>(p.base + row[s][h] * p.base_stride + n0 + tig * 8);
      if (adapt) {
        float acc[2][4][4];  // [row tile][column tile]
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          // column tile i holds columns 8 j + 2 i and 8 j + 2 i + 1, so that a
          // thread ends with eight neighbouring ones
          const int n = n0 + (g >> 1) * 8 + 2 * i + (g & 1);
          const uint16_t* up = p.up + ((int64_t)a * p.N + n) * RANK + tig * EL;
#pragma unroll
          for (int s = 0; s < 2; ++s)
#pragma unroll
            for (int e = 0; e < 4; ++e) acc[s][i][e] = 0.f;
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
            for (int s = 0; s < 2; ++s)
#pragma unroll
              for (int st = 0; st < STEPS; ++st) {
                const int e0 = 2 * st, e1 = EL == 2 ? 0 : 2 * st + 1;
                const bool two = EL != 2;  // rank 8 fills half of a product's K
                mma_16816(acc[s][i], th[s][0][q][e0], th[s][1][q][e0], two ? th[s][0][q][e1] : 0u, two ? th[s][1][q][e1] : 0u,
                          b[e0], two ? b[e1] : 0u);
                mma_16816(acc[s][i], tl[s][0][q][e0], tl[s][1][q][e0], two ? tl[s][0][q][e1] : 0u, two ? tl[s][1][q][e1] : 0u,
                          b[e0], two ? b[e1] : 0u);
              }
          }
        }
#pragma unroll
        for (int s = 0; s < 2; ++s)
#pragma unroll
          for (int h = 0; h < 2; ++h) {
            float f[8];
            afd::bf16x8_to_float(bv[s][h], f);
#pragma unroll
            for (int i = 0; i < 4; ++i) {
              f[2 * i] += acc[s][i][2 * h];
              f[2 * i + 1] += acc[s][i][2 * h + 1];
            }
            bv[s][h] = afd::float_to_bf16x8(f);
          }
      }
#pragma unroll
      for (int s = 0; s < 2; ++s)
#pragma unroll
        for (int h = 0; h < 2; ++h)
          if (in && row[s][h] >= 0) *reinterpret_cast<uint4*>(p.out + row[s][h] * p.out_stride + n0 + tig * 8) = bv[s][h];
    }
  }
  if (open) asm volatile("barrier.cluster.wait.acquire.aligned;" ::: "memory");
}

template <int RANK>
cudaError_t launch_adapters(const AdapterParams& p, int sms, cudaStream_t stream) {
  constexpr int kSmem = sizeof(AdapterShared<RANK>);
  cudaError_t e = cudaFuncSetAttribute(adapter_kernel<RANK>, cudaFuncAttributeMaxDynamicSharedMemorySize, kSmem);
  if (e != cudaSuccess) return e;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(kGroupCtas);
  cfg.blockDim = dim3(kGroupThreads);
  cfg.stream = stream;
  e = cudaLaunchKernelEx(&cfg, adapter_group_kernel, p);
  if (e != cudaSuccess) return e;
  // a tile holds rows of one adapter: at most one tile more than full ones per group
  const int64_t tiles = (int64_t)p.R / kAdRows + (p.S + 1 < p.R ? p.S + 1 : p.R);
  const int64_t most = sms * (RANK <= 32 ? 2 : 1) / kAdCtas;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.gridDim = dim3((unsigned)((tiles < most ? tiles : most) * kAdCtas));
  cfg.blockDim = dim3(kAdThreads);
  cfg.dynamicSmemBytes = kSmem;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
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

AFD_API int64_t afd_adapter_workspace_bytes(int64_t num_rows, int32_t num_slots) {
  return num_rows < 0 || num_slots < 1 ? -1 : (num_rows + num_slots + 2) * (int64_t)sizeof(int32_t);
}

AFD_API afd_status afd_adapter_add(const void* base, int64_t base_stride, const void* x, int64_t x_stride,
                                   const void* down, const void* up, const int32_t* token_slots, const float* scales,
                                   const int32_t* row_src, const int32_t* ends, int32_t num_groups, int32_t top_k,
                                   int64_t num_rows, int32_t num_tokens, int32_t num_slots, int32_t rank,
                                   int32_t in_features, int32_t out_features, void* out, int64_t out_stride,
                                   void* workspace, int64_t workspace_bytes, afd_stream stream) {
  if (num_rows < 0 || num_tokens < 0 || num_slots < 1 || rank < 1 || in_features < 1 || out_features < 1)
    return AFD_ERR_ARG;
  if (base_stride < out_features || out_stride < out_features || x_stride < in_features) return AFD_ERR_ARG;
  if (row_src ? (!ends || num_groups < 1 || top_k < 1) : num_tokens < num_rows) return AFD_ERR_ARG;
  if (rank != 8 && rank != 16 && rank != 32 && rank != 64) return AFD_ERR_UNSUPPORTED;
  if (in_features % 16 || out_features % 8 || base_stride % 8 || out_stride % 8 || x_stride % 8 ||
      num_rows > INT32_MAX - kAdRows || num_slots > kMaxSlots)
    return AFD_ERR_UNSUPPORTED;
  if (num_rows == 0) return AFD_OK;
  if (!base || !x || !down || !up || !token_slots || !scales || !out || !workspace) return AFD_ERR_ARG;
  if (workspace_bytes < afd_adapter_workspace_bytes(num_rows, num_slots)) return AFD_ERR_ARG;
  AdapterParams p = {};
  p.base_stride = base_stride, p.x_stride = x_stride, p.out_stride = out_stride;
  p.G = num_groups, p.top_k = top_k, p.R = (int32_t)num_rows, p.tokens = num_tokens, p.S = num_slots, p.rank = rank;
  p.K = in_features, p.N = out_features;
  if (!afd::device_view(static_cast<const uint16_t*>(base), &p.base) ||
      !afd::device_view(static_cast<const uint16_t*>(x), &p.x) ||
      !afd::device_view(static_cast<const uint16_t*>(down), &p.down) ||
      !afd::device_view(static_cast<const uint16_t*>(up), &p.up) || !afd::device_view(token_slots, &p.token_slots) ||
      !afd::device_view(scales, &p.scales) || !afd::device_view(static_cast<uint16_t*>(out), &p.out) ||
      !afd::device_view(static_cast<int32_t*>(workspace), &p.first) ||
      (row_src && (!afd::device_view(row_src, &p.row_src) || !afd::device_view(ends, &p.ends))))
    return AFD_ERR_ARG;
  p.order = p.first + num_slots + 2;
  if (!afd::aligned_to(p.first, 4) || !afd::aligned_to(p.token_slots, 4) || !afd::aligned_to(p.scales, 4) || !afd::aligned_to(p.row_src, 4) ||
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
