// Row operators of a worker between its products: the gated activation
// (afd_gated_rows) and the low-rank adapters of many requests
// (afd_adapter_add).

#include <cuda_fp16.h>
#include <cuda_runtime.h>
#include <stdint.h>

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

// A warp per row, four 16-byte groups of either half in flight; VEC: rows and
// halves start on 16-byte boundaries. Bound by DRAM: 16.4 K rows of 2 x 1024 in
// 18 us, 5.6 TB/s (20 us with one group in flight).
template <bool VEC>
__global__ void __launch_bounds__(256) gated_rows_kernel(const GatedParams p) {
  __shared__ int sh_end[afd::kMaxExperts];
  afd::pdl_wait();
  afd::pdl_launch_dependents();
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
      // four column groups' loads in flight at a time
      for (int c0 = lane * 8; c0 < p.N; c0 += 4 * 256) {
        uint4 gv[4], uv[4];
#pragma unroll
        for (int i = 0; i < 4; ++i)
          if (c0 + 256 * i < p.N) {
            gv[i] = afd::ld_before_write(reinterpret_cast<const uint4*>(gate + c0 + 256 * i));  // `out` may be there
            uv[i] = afd::ld_once(reinterpret_cast<const uint4*>(up + c0 + 256 * i));
          }
#pragma unroll
        for (int i = 0; i < 4; ++i)
          if (c0 + 256 * i < p.N) {
            float g[8], u[8];
            afd::bf16x8_to_float(gv[i], g);
            afd::bf16x8_to_float(uv[i], u);
#pragma unroll
            for (int j = 0; j < 8; ++j) g[j] = afd::silu_mul(g[j], u[j]);
            *reinterpret_cast<uint4*>(out + c0 + 256 * i) = afd::float_to_bf16x8(g);
          }
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
  const uint8_t* x;       // BF16, or E4M3 with x_scale
  int64_t x_stride;       // bytes
  const float* x_scale;   // [R][K / 128]
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
  uint16_t *t_hi, *t_lo;  // workspace: scale * down[a] x of each of them, [R][rank]
};

// The group of a row: its adapter, S for none, -1 for what is not a row.
__device__ __forceinline__ int token_group(const AdapterParams& p, int src) {
  const int t = src < 0 ? -1 : p.row_src ? src / p.top_k : src;
  if (t < 0 || t >= p.tokens) return -1;
  const int a = p.token_slots[t];
  return a >= 0 && a < p.S ? a : p.S;
}
__device__ __forceinline__ int row_group(const AdapterParams& p, int r) {
  return token_group(p, p.row_src ? p.row_src[r] : r);
}

// Four E4M3 values as two pairs of BF16 (exact).
__device__ __forceinline__ void e4m3_to_bf16(uint32_t v, uint32_t& lo, uint32_t& hi) {
  uint32_t a, b;
  asm("{\n.reg .b16 l, h;\nmov.b32 {l, h}, %2;\ncvt.rn.f16x2.e4m3x2 %0, l;\ncvt.rn.f16x2.e4m3x2 %1, h;\n}" : "=r"(a), "=r"(b) : "r"(v));
  const float2 x = __half22float2(*reinterpret_cast<const __half2*>(&a)), y = __half22float2(*reinterpret_cast<const __half2*>(&b));
  lo = afd::pack_bf16(x.x, x.y);
  hi = afd::pack_bf16(y.x, y.y);
}

// The generic address of this shared address in another CTA of the cluster.
template <typename T>
__device__ __forceinline__ T* remote(T* p, uint32_t rank) {
  uint64_t a;
  asm("mapa.u64 %0, %1, %2;" : "=l"(a) : "l"(p), "r"(rank));
  return reinterpret_cast<T*>(a);
}

__device__ __forceinline__ void cluster_sync() {
  asm volatile("barrier.cluster.arrive.release.aligned;\nbarrier.cluster.wait.acquire.aligned;" ::: "memory");
}

// Low-rank adapters of few rows (a decode step): a cluster of `ctas` blocks per
// row, in one launch and without a workspace. The blocks share the K columns of
// the rank's dot products and leave each other their parts, then share the
// columns of the result; a lane reads 16 bytes of an adapter at a time, next to
// its neighbour's. With few rows a call is a chain of latencies (2.9 us for one
// row of 2048 columns, rank 16; 9.7 us by the three launches below), with many
// every row reads its adapter from L2 again. Blocks of a cluster, 2048 columns,
// rank 16: with 16 rows 8 take 3.2 us, 4 3.3, 2 4.2 and 1 5.9; with 64 rows 4.6,
// 3.6, 4.3 and 6.1; with 128 8.4, 4.9, 5.0 and 6.2; with 512 30, 16, 11.2 and
// 10.3, padded to 128 rows a group 13.8, 10.6, 9.3 and 12.2. So 8 up to 32 rows,
// 4 up to 64 and 2 beyond. Four blocks share an SM up to rank 16 (256 rows: 6.7
// us, with three 8.9; five at rank 8 5.5, with four 5.0), two above (rank 32, 128
// rows: 6.4, with three 7.7).
// Rows are dealt to the clusters one by one, as the live ones of a padded layout
// sit next to each other, and to an odd number of clusters, as groups start at
// multiples of a power of two (the padded 512 rows in 304 clusters: 13.5 us, in
// 303: 9.1). A cluster looks 32 of its rows up at a time.
constexpr int kRowCtas = 8, kRowThreads = 256;

template <int RANK, bool FP8>
__global__ void __launch_bounds__(kRowThreads, RANK <= 16 ? 4 : 2) adapter_rows_kernel(const AdapterParams p, const int ctas) {
  __shared__ float part[2][kRowCtas][RANK];
  __shared__ __align__(16) float low[RANK];
  constexpr int JW = RANK / 8;                          // dot products of a warp
  constexpr int L = RANK / 8;                           // lanes of a column's up row
  constexpr int COLS = kRowThreads / L;                 // columns a block takes in one go
  constexpr int U = 4;                                  // times it, loaded together
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int cta = blockIdx.x % ctas;
  const int64_t cluster = blockIdx.x / ctas, clusters = gridDim.x / ctas;
  cluster_sync();  // the others have started: their shared memory may be written
  afd::pdl_wait();
  afd::pdl_launch_dependents();
  const int limit = p.row_src ? afd::group_end(p.ends[p.G - 1], p.R) : p.R;
  const bool in_place = p.out == p.base && p.out_stride == p.base_stride;
  int turn = 0;
  for (int64_t i0 = cluster; i0 < limit; i0 += 32 * clusters) {
    const int64_t mine = i0 + (int64_t)lane * clusters;
    const int group = mine < limit ? row_group(p, (int)mine) : -1;
    unsigned todo = __ballot_sync(0xffffffffu, group >= 0 && !(group == p.S && in_place));
    for (; todo; todo &= todo - 1) {
      const int which = __ffs(todo) - 1;
      const int64_t r = i0 + (int64_t)which * clusters;
      const int a = __shfl_sync(0xffffffffu, group, which);
      const uint16_t* base = p.base + r * p.base_stride;
      uint16_t* out = p.out + r * p.out_stride;
      if (a == p.S) {  // no adapter
        for (int c = (cta * kRowThreads + threadIdx.x) * 8; c < p.N; c += ctas * kRowThreads * 8)
          *reinterpret_cast<uint4*>(out + c) = *reinterpret_cast<const uint4*>(base + c);
        continue;
      }
      const uint8_t* x = p.x + r * p.x_stride;
      const uint16_t* down = p.down + (int64_t)a * RANK * p.K;
      const uint16_t* up = p.up + (int64_t)a * p.N * RANK + threadIdx.x % L * 8;
      // The first columns' operands are on their way while the dot products run.
      const int c0 = cta * COLS + threadIdx.x / L;
      uint4 uv[U];
      uint16_t bv[U];
      auto fetch = [&](int c) {
#pragma unroll
        for (int u = 0; u < U; ++u) {
          const int col = c + u * ctas * COLS;
          uv[u] = col < p.N ? __ldg(reinterpret_cast<const uint4*>(up + (int64_t)col * RANK)) : make_uint4(0, 0, 0, 0);
          bv[u] = col < p.N ? base[col] : 0;
        }
      };
      fetch(c0);
      float sum[JW] = {};
#pragma unroll 1
      for (int k = (cta * 32 + lane) * 8; k < p.K; k += ctas * 32 * 8) {
        uint4 xv, dv[JW];
        float xs = 1.f;
        if (FP8) {
          const uint2 q = *reinterpret_cast<const uint2*>(x + k);
          e4m3_to_bf16(q.x, xv.x, xv.y);
          e4m3_to_bf16(q.y, xv.z, xv.w);
          xs = p.x_scale[r * (p.K / 128) + k / 128];
        } else {
          xv = *reinterpret_cast<const uint4*>(x + 2 * k);
        }
#pragma unroll
        for (int j = 0; j < JW; ++j)
          dv[j] = __ldg(reinterpret_cast<const uint4*>(down + (int64_t)(warp + 8 * j) * p.K + k));
        float xf[8];
        afd::bf16x8_to_float(xv, xf);
        if (FP8)
#pragma unroll
          for (int e = 0; e < 8; ++e) xf[e] *= xs;
#pragma unroll
        for (int j = 0; j < JW; ++j) {
          float df[8];
          afd::bf16x8_to_float(dv[j], df);
#pragma unroll
          for (int e = 0; e < 8; ++e) sum[j] = fmaf(xf[e], df[e], sum[j]);
        }
      }
      const float scale = p.scales[a];
#pragma unroll
      for (int j = 0; j < JW; ++j) {
#pragma unroll
        for (int d = 16; d; d >>= 1) sum[j] += __shfl_xor_sync(0xffffffffu, sum[j], d);
        if (lane < ctas) *remote(&part[turn][cta][warp + 8 * j], lane) = sum[j];
      }
      cluster_sync();
      if (threadIdx.x < RANK) {
        float t = 0.f;
#pragma unroll
        for (int i = 0; i < kRowCtas; ++i)
          if (i < ctas) t += part[turn][i][threadIdx.x];
        low[threadIdx.x] = t * scale;
      }
      // The other half of `part` is written next; this one again only after the
      // cluster's next barrier, which comes after these reads.
      turn ^= 1;
      __syncthreads();
      float t[8];
#pragma unroll
      for (int e = 0; e < 8; ++e) t[e] = low[threadIdx.x % L * 8 + e];
      for (int c = c0;;) {
#pragma unroll
        for (int u = 0; u < U; ++u) {
          const int col = c + u * ctas * COLS;
          float f[8], add = 0.f;
          afd::bf16x8_to_float(uv[u], f);
#pragma unroll
          for (int e = 0; e < 8; ++e) add = fmaf(t[e], f[e], add);
#pragma unroll
          for (int d = 1; d < L; d <<= 1) add += __shfl_xor_sync(0xffffffffu, add, d);
          if (threadIdx.x % L == 0 && col < p.N)
            out[col] = (uint16_t)afd::pack_bf16(__uint_as_float((uint32_t)bv[u] << 16) + add, 0.f);
        }
        c += U * ctas * COLS;
        if (c - threadIdx.x / L >= p.N) break;  // (the same for the whole block)
        fetch(c);
      }
    }
  }
  cluster_sync();  // nobody leaves while its shared memory may be written
}

// Low-rank adapters of many rows, in three launches that follow each other by
// programmatic dependent launch.
//   group: the live rows sorted by adapter (a request's rows are spread over
//          every expert's range, so rows that follow one another mostly differ
//          in theirs), and where each adapter starts; rows without one last.
//   down:  t = scale * down[a] x for 16 rows of one adapter a block, K split
//          over its eight warps and joined in a fixed order. Then the blocks
//          copy the rows without an adapter (not in place): few blocks have a
//          tile more than the others, and the copies fill the rest.
//   up:    out = base + up[a] t for 16 rows and some of the columns a warp, 32
//          columns at a time with the next ones' operands on their way.
// What bounds it is the traffic of x, base and out (about 6 bytes a column and
// row against 2 rank flops), which down and up stream with many small blocks
// in flight. mma.sync's rate is enough, and its register operands spare TMEM
// and the layout it wants: the order of K (and of the output's columns) inside
// a fragment is free as long as both sides agree, so a thread takes eight
// neighbouring values, 16 bytes at a time. A product's rows do not mix, so
// neither the order of the rows inside a group nor what another request's
// adapter holds reaches a result.
// t is FP32; between the two it is kept as two BF16 (16 bits and more).
// Measured with 16.4 K rows, K = N = 2048, rank 32, eight adapters, two rows in
// three with one: 47.5 us (7 + 20 + 17 and the launches) against a floor of 27;
// without the grouping, 64 neighbouring rows at a time, 192 us.
constexpr int kFewRows = 512;
constexpr int64_t kFewRowsBytes = (int64_t)64 << 20;
constexpr int kMaxSlots = 1023;    // and the rows without one: a thread of the grouping each
constexpr int kGroupCtas = 8;
constexpr int kGroupThreads = 1024;
constexpr int kGroupKeep = 4;      // rows of a thread whose group it remembers
constexpr int kDownRows = 16;      // rows of a block
constexpr int kDownWarps = 8;      // ... whose warps share K
constexpr int kUpRows = 64;        // rows of a tile: 16 for each of four warps
constexpr int kUpThreads = 256;
// K chunks of a warp in flight, and column groups. At rank 64 so few that two
// blocks share an SM (2,048 tokens a source: 71 us, with 3 and 4 stages and one
// block 85, both before the grouping's loads overlapped); at rank 32 3 and 4 take
// 50.5 us, 2 and 2 52.4, 4 and 4 53.
constexpr int down_stages(int rank) { return rank <= 32 ? 3 : 2; }
constexpr int up_stages(int rank) { return rank <= 32 ? 4 : 2; }

// One cluster: counts per group and CTA, their prefix, then every row's place.
// Inside a group the order is that of the atomics; no result depends on it.
__global__ void __cluster_dims__(kGroupCtas, 1, 1) __launch_bounds__(kGroupThreads) adapter_group_kernel(const AdapterParams p) {
  __shared__ int count[kMaxSlots + 1], cursor[kMaxSlots + 1];
  __shared__ int warp_total[kGroupThreads / 32];
  afd::pdl_wait();
  afd::pdl_launch_dependents();
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const uint32_t cta = blockIdx.x;
  const int groups = p.S + 1;  // at most kGroupThreads
  // Rows go to the CTAs 1024 at a time, whatever the last end is: the first
  // ones' row_src and that end are on their way together (a contiguous share
  // each, known after the end only: 1.3 us more).
  constexpr int kStep = kGroupCtas * kGroupThreads;
  const int64_t lo = (int64_t)cta * kGroupThreads;
  int keep[kGroupKeep];
#pragma unroll
  for (int i = 0; i < kGroupKeep; ++i) {
    const int64_t r = lo + i * kStep + threadIdx.x;
    keep[i] = r >= p.R ? -1 : p.row_src ? p.row_src[r] : (int)r;
  }
  const int limit = p.row_src ? afd::group_end(p.ends[p.G - 1], p.R) : p.R;
  for (int g = threadIdx.x; g < groups; g += kGroupThreads) count[g] = 0;
  __syncthreads();
  // The first rows' groups stay in registers, all their loads in flight at once.
#pragma unroll
  for (int i = 0; i < kGroupKeep; ++i)
    keep[i] = lo + i * kStep + threadIdx.x < limit ? token_group(p, keep[i]) : -1;
  auto tally = [&](int g) {
    const unsigned same = __match_any_sync(0xffffffffu, g);
    if (g >= 0 && lane == __ffs(same) - 1) atomicAdd(&count[g], __popc(same));
  };
#pragma unroll
  for (int i = 0; i < kGroupKeep; ++i) tally(keep[i]);
  const int64_t rest = lo + kGroupKeep * kStep + 32 * warp;
  for (int64_t r0 = rest; r0 < limit; r0 += kStep) tally(r0 + lane < limit ? row_group(p, (int)r0 + lane) : -1);
  cluster_sync();
  // a thread per group of the prefix sum
  const int g = threadIdx.x;
  int total = 0, before = 0;
  if (g < groups) {
#pragma unroll
    for (uint32_t c = 0; c < kGroupCtas; ++c) {
      const int v = *remote(&count[g], c);
      total += v;
      if (c < cta) before += v;
    }
  }
  int run = afd::warp_inclusive_scan(total);
  if (lane == 31) warp_total[warp] = run;
  __syncthreads();
  if (warp == 0) {
    const int t = warp_total[lane];
    warp_total[lane] = afd::warp_inclusive_scan(t) - t;
  }
  __syncthreads();
  run += warp_total[warp] - total;
  if (g < groups) {
    cursor[g] = run + before;
    if (cta == 0) {
      p.first[g] = run;
      if (g == groups - 1) p.first[groups] = run + total;
    }
  }
  __syncthreads();
  auto place = [&](int g, int64_t r) {
    const unsigned same = __match_any_sync(0xffffffffu, g);
    int at = 0;
    if (g >= 0 && lane == __ffs(same) - 1) at = atomicAdd(&cursor[g], __popc(same));
    at = __shfl_sync(0xffffffffu, at, __ffs(same) - 1) + __popc(same & ((1u << lane) - 1));
    if (g >= 0) p.order[at] = (int)r;
  };
#pragma unroll
  for (int i = 0; i < kGroupKeep; ++i) place(keep[i], lo + i * kStep + threadIdx.x);
  for (int64_t r0 = rest; r0 < limit; r0 += kStep) place(r0 + lane < limit ? row_group(p, (int)r0 + lane) : -1, r0 + lane);
  cluster_sync();  // nobody leaves while its counts may be read
}

__device__ __forceinline__ void mma_16816(float (&c)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3,
                                          uint32_t b0, uint32_t b1) {
  asm("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, {%0, %1, %2, %3};"
      : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

// Where the groups start, in rows and in tiles of ROWS rows (of the first
// `groups` groups).
struct GroupTable {
  int* first;
  int* first_tile;
};

// In dynamic shared memory, behind what a block needs besides.
constexpr size_t table_bytes(int slots) { return 2 * sizeof(int) * (slots + 2); }
__device__ __forceinline__ GroupTable table_at(void* p, int slots) {
  int* first = static_cast<int*>(p);
  return {first, first + slots + 2};
}

template <int ROWS>
__device__ __forceinline__ int load_groups(const AdapterParams& p, const GroupTable& sh, int groups) {
  const int lane = threadIdx.x & 31;
  for (int i = threadIdx.x; i <= groups; i += blockDim.x) sh.first[i] = p.first[i];
  __syncthreads();
  if (threadIdx.x < 32) {
    int carry = 0;
    for (int i0 = 0; i0 < groups; i0 += 32) {
      const int i = i0 + lane;
      const int t = i < groups ? (sh.first[i + 1] - sh.first[i] + ROWS - 1) / ROWS : 0;
      const int incl = afd::warp_inclusive_scan(t);
      if (i < groups) sh.first_tile[i] = carry + incl - t;
      carry += __shfl_sync(0xffffffffu, incl, 31);
    }
    if (lane == 0) sh.first_tile[groups] = carry;
  }
  __syncthreads();
  return sh.first_tile[groups];
}

// The group of tile t: the last one that starts at or before it.
__device__ __forceinline__ int tile_group(const GroupTable& sh, int groups, int t) {
  int a = 0;
  for (int hi = groups - 1; a < hi;) {
    const int mid = (a + hi + 1) >> 1;
    if (sh.first_tile[mid] <= t) a = mid; else hi = mid - 1;
  }
  return a;
}

// Asynchronous copies of BYTES (4, 8 or 16) into shared memory; nothing is
// read where `in` is false, and zeros are written.
template <int BYTES>
__device__ __forceinline__ void copy_async(void* dst, const void* src, bool in) {
  const uint32_t d = (uint32_t)__cvta_generic_to_shared(dst);
  const int n = in ? BYTES : 0;
  if (BYTES == 16)
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(d), "l"(src), "r"(n) : "memory");
  else
    asm volatile("cp.async.ca.shared.global [%0], [%1], %2, %3;" ::"r"(d), "l"(src), "n"(BYTES), "r"(n) : "memory");
}

// Operands of one 32-wide K chunk on their way: every thread copies exactly
// what it uses itself, so no other thread has to be waited for.
template <bool FP8>
struct DownRows;
template <>
struct DownRows<false> {
  uint4 x[2][32];  // rows g / g + 8: eight values
};
template <>
struct DownRows<true> {
  uint2 x[2][32];
  float scale[2][32];  // of the rows' block
};

template <int RANK, bool FP8>
struct alignas(16) DownStage : DownRows<FP8> {
  alignas(16) uint4 down[RANK / 8][32];  // rank rows 8 n + g
};

template <int RANK, bool FP8>
struct DownShared {
  static constexpr int kPad = RANK + 4;
  union {
    DownStage<RANK, FP8> stage[kDownWarps][down_stages(RANK)];
    float part[kDownWarps][kDownRows][kPad];  // once the products are done
  };
};

// What of v is rounded to BF16 first: a finite number above the largest BF16
// gives that one (rounded up it were infinite, and the rest minus infinity).
__device__ __forceinline__ float high_part(float v) {
  const float most = __uint_as_float(0x7f7f0000u);
  return fabsf(v) > most && !isinf(v) ? copysignf(most, v) : v;
}

template <int RANK, bool FP8>
__global__ void __launch_bounds__(kDownWarps * 32) adapter_down_kernel(const AdapterParams p) {
  extern __shared__ __align__(16) uint8_t ad_smem[];
  DownShared<RANK, FP8>& sh = *reinterpret_cast<DownShared<RANK, FP8>*>(ad_smem);
  constexpr int NT = RANK / 8;             // 8-column tiles of the product
  constexpr int kStages = down_stages(RANK);
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int g = lane >> 2, tig = lane & 3;
  const int chunks = (p.K + 31) >> 5;
  DownStage<RANK, FP8>* stage = sh.stage[warp];
  const GroupTable groups = table_at(&sh + 1, p.S);
  afd::pdl_wait();
  afd::pdl_launch_dependents();
  const int tiles = load_groups<kDownRows>(p, groups, p.S);
  for (int t = blockIdx.x; t < tiles; t += gridDim.x) {
    const int a = tile_group(groups, p.S, t);
    const int at = groups.first[a] + (t - groups.first_tile[a]) * kDownRows, end = groups.first[a + 1];
    const uint8_t* x[2];  // this thread's rows: g / g + 8
    const float* xs[2];
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      const int i = at + 8 * h + g;
      const int64_t r = i < end ? p.order[i] : -1;
      x[h] = r >= 0 ? p.x + r * p.x_stride : nullptr;
      xs[h] = FP8 && r >= 0 ? p.x_scale + r * (p.K / 128) : nullptr;
    }
    const uint16_t* down = p.down + ((int64_t)a * RANK + g) * p.K;
    auto fetch = [&](int i) {  // this warp's i-th chunk
      const int c = warp + i * kDownWarps;
      if (c < chunks) {
        DownStage<RANK, FP8>& st = stage[i % kStages];
        const int k = c * 32 + tig * 8;
        const bool in = k < p.K;
#pragma unroll
        for (int n = 0; n < NT; ++n) copy_async<16>(&st.down[n][lane], in ? down + (int64_t)n * 8 * p.K + k : p.down, in);
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          const bool live = in && x[h];
          copy_async<FP8 ? 8 : 16>(&st.x[h][lane], live ? x[h] + k * (FP8 ? 1 : 2) : p.x, live);
          if constexpr (FP8) copy_async<4>(&st.scale[h][lane], live ? xs[h] + k / 128 : p.x_scale, live);
        }
      }
      asm volatile("cp.async.commit_group;" ::: "memory");
    };
#pragma unroll
    for (int i = 0; i < kStages - 1; ++i) fetch(i);
    float acc[NT][4];
#pragma unroll
    for (int n = 0; n < NT; ++n)
#pragma unroll
      for (int i = 0; i < 4; ++i) acc[n][i] = 0.f;
    for (int i = 0; warp + i * kDownWarps < chunks; ++i) {
      fetch(i + kStages - 1);
      asm volatile("cp.async.wait_group %0;" ::"n"(kStages - 1) : "memory");
      const DownStage<RANK, FP8>& st = stage[i % kStages];
      uint32_t x0[4], x1[4];
      const auto v0 = st.x[0][lane], v1 = st.x[1][lane];
      if constexpr (FP8) {
        e4m3_to_bf16(v0.x, x0[0], x0[1]);
        e4m3_to_bf16(v0.y, x0[2], x0[3]);
        e4m3_to_bf16(v1.x, x1[0], x1[1]);
        e4m3_to_bf16(v1.y, x1[2], x1[3]);
      } else {
        x0[0] = v0.x, x0[1] = v0.y, x0[2] = v0.z, x0[3] = v0.w;
        x1[0] = v1.x, x1[1] = v1.y, x1[2] = v1.z, x1[3] = v1.w;
      }
#pragma unroll
      for (int n = 0; n < NT; ++n) {
        const uint4 b = st.down[n][lane];
        if constexpr (FP8) {
          // a chunk lies in one block of 128: its product takes the rows' scales
          float v[4] = {};
          mma_16816(v, x0[0], x1[0], x0[1], x1[1], b.x, b.y);
          mma_16816(v, x0[2], x1[2], x0[3], x1[3], b.z, b.w);
#pragma unroll
          for (int e = 0; e < 4; ++e) acc[n][e] = fmaf(v[e], st.scale[e >> 1][lane], acc[n][e]);
        } else {
          mma_16816(acc[n], x0[0], x1[0], x0[1], x1[1], b.x, b.y);
          mma_16816(acc[n], x0[2], x1[2], x0[3], x1[3], b.z, b.w);
        }
      }
    }
    asm volatile("cp.async.wait_all;" ::: "memory");
    __syncthreads();
#pragma unroll
    for (int n = 0; n < NT; ++n)
#pragma unroll
      for (int h = 0; h < 2; ++h)
        *reinterpret_cast<float2*>(&sh.part[warp][8 * h + g][8 * n + 2 * tig]) = make_float2(acc[n][2 * h], acc[n][2 * h + 1]);
    __syncthreads();
    const float scale = p.scales[a];
    for (int i = threadIdx.x; i < kDownRows * RANK / 2; i += kDownWarps * 32) {
      const int r = i / (RANK / 2), c = i % (RANK / 2) * 2;
      if (at + r >= end) continue;
      float2 v = make_float2(0.f, 0.f);
#pragma unroll
      for (int w = 0; w < kDownWarps; ++w) {
        const float2 o = *reinterpret_cast<const float2*>(&sh.part[w][r][c]);
        v.x += o.x, v.y += o.y;
      }
      v.x *= scale, v.y *= scale;
      const uint32_t hi = afd::pack_bf16(high_part(v.x), high_part(v.y));
      // (an infinite product leaves no rest)
      const uint32_t lo = afd::pack_bf16(isinf(v.x) ? 0.f : v.x - __uint_as_float(hi << 16),
                                         isinf(v.y) ? 0.f : v.y - __uint_as_float(hi & 0xffff0000u));
      const int64_t o = (int64_t)(at + r) * RANK + c;
      *reinterpret_cast<uint32_t*>(p.t_hi + o) = hi;
      *reinterpret_cast<uint32_t*>(p.t_lo + o) = lo;
    }
    __syncthreads();
  }
  if (p.out == p.base && p.out_stride == p.base_stride) return;
  // Rows without an adapter, a row a warp, from the last block on: the first
  // ones may have had a tile more.
  const int plain = groups.first[p.S], plain_end = p.first[p.S + 1];
  for (int i = plain + (int)(gridDim.x - 1 - blockIdx.x) * kDownWarps + warp; i < plain_end; i += gridDim.x * kDownWarps) {
    const int64_t r = p.order[i];
    const uint16_t* from = p.base + r * p.base_stride;
    uint16_t* to = p.out + r * p.out_stride;
    for (int c0 = lane * 8; c0 < p.N; c0 += 4 * 256) {
      uint4 v[4];
#pragma unroll
      for (int j = 0; j < 4; ++j)
        if (c0 + 256 * j < p.N) v[j] = afd::ld_once(reinterpret_cast<const uint4*>(from + c0 + 256 * j));
#pragma unroll
      for (int j = 0; j < 4; ++j)
        if (c0 + 256 * j < p.N) *reinterpret_cast<uint4*>(to + c0 + 256 * j) = v[j];
    }
  }
}

// EL rank values (EL / 2 words) of a thread.
template <int EL>
__device__ __forceinline__ void load_rank(const uint16_t* q, bool in, uint32_t (&v)[EL / 2]) {
  if (EL == 8) {
    const uint4 w = in ? *reinterpret_cast<const uint4*>(q) : make_uint4(0, 0, 0, 0);
    v[0] = w.x, v[1 % (EL / 2)] = w.y, v[2 % (EL / 2)] = w.z, v[3 % (EL / 2)] = w.w;
  } else if (EL == 4) {
    const uint2 w = in ? *reinterpret_cast<const uint2*>(q) : make_uint2(0, 0);
    v[0] = w.x, v[1 % (EL / 2)] = w.y;
  } else {
    v[0] = in ? *reinterpret_cast<const uint32_t*>(q) : 0u;
  }
}

// Operands of one 32-column group on their way: every thread copies exactly
// what it uses itself, so no other thread has to be waited for.
template <int RANK>
struct UpStage {
  static constexpr int EL = RANK >= 32 ? 8 : RANK / 4;  // rank values a thread takes at a time
  static constexpr int CH = RANK >= 32 ? RANK / 32 : 1;  // ... and how often
  uint4 base[2][32];                                    // rows g / g + 8
  struct alignas(EL * 2) { uint32_t v[EL / 2]; } up[4][CH][32];
};

template <int RANK>
struct UpShared {
  alignas(16) UpStage<RANK> stage[kUpThreads / 32][up_stages(RANK)];
};

template <int RANK>
__global__ void __launch_bounds__(kUpThreads, 2) adapter_up_kernel(const AdapterParams p) {
  extern __shared__ __align__(16) uint8_t ad_smem[];
  UpShared<RANK>& sh = *reinterpret_cast<UpShared<RANK>*>(ad_smem);
  constexpr int EL = UpStage<RANK>::EL, CH = UpStage<RANK>::CH;
  constexpr int STEPS = EL == 8 ? 2 : 1;              // products per chunk
  constexpr int kStages = up_stages(RANK);
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int g = lane >> 2, tig = lane & 3;
  const int col_groups = (p.N + 31) >> 5, slots = gridDim.x * (kUpThreads / 32);
  UpStage<RANK>* stage = sh.stage[warp];
  const GroupTable groups = table_at(&sh + 1, p.S);
  afd::pdl_wait();
  afd::pdl_launch_dependents();
  const int tiles = load_groups<kUpRows>(p, groups, p.S);
  // The columns are split so far that every warp has something to do.
  const int want = max(1, min(col_groups, slots / max(4 * tiles, 1)));
  const int each = (col_groups + want - 1) / want, parts = (col_groups + each - 1) / each;
  const int64_t items = (int64_t)tiles * parts * 4;
  for (int64_t item = (int64_t)blockIdx.x * (kUpThreads / 32) + warp; item < items; item += slots) {
    const int quarter = (int)(item & 3);
    const int t = (int)((item >> 2) / parts), part = (int)((item >> 2) % parts);
    const int a = tile_group(groups, p.S, t);
    const int at = groups.first[a] + (t - groups.first_tile[a]) * kUpRows + 16 * quarter, end = groups.first[a + 1];
    if (at >= end) continue;
    const int g0 = part * each, g1 = min(g0 + each, col_groups);
    const uint16_t* base[2];  // this thread's rows at its first column: g / g + 8
    uint16_t* out[2];
    uint32_t th[2][CH][EL / 2], tl[2][CH][EL / 2];
    bool live[2];
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      const int i = at + 8 * h + g;
      live[h] = i < end;
      const int64_t r = live[h] ? p.order[i] : 0;
      base[h] = p.base + r * p.base_stride + tig * 8;
      out[h] = p.out + r * p.out_stride + tig * 8;
    }
    // column tile i holds columns 8 j + 2 i and 8 j + 2 i + 1, so that a thread
    // ends with eight neighbouring ones
    const int col = (g >> 1) * 8 + (g & 1);
    const uint16_t* up = p.up + ((int64_t)a * p.N + col) * RANK + tig * EL;
    auto fetch = [&](int gi) {
      if (gi < g1) {
        UpStage<RANK>& st = stage[gi % kStages];
        const int n0 = gi * 32;
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          const bool in = live[h] && n0 + tig * 8 < p.N;
          copy_async<16>(&st.base[h][lane], in ? base[h] + n0 : p.base, in);
        }
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const bool in = n0 + col + 2 * i < p.N;
#pragma unroll
          for (int q = 0; q < CH; ++q)
            copy_async<2 * EL>(&st.up[i][q][lane], in ? up + (int64_t)(n0 + 2 * i) * RANK + q * 32 : p.up, in);
        }
      }
      asm volatile("cp.async.commit_group;" ::: "memory");
    };
#pragma unroll
    for (int i = 0; i < kStages - 1; ++i) fetch(g0 + i);
#pragma unroll
    for (int h = 0; h < 2; ++h)
#pragma unroll
      for (int q = 0; q < CH; ++q) {
        const int64_t o = (int64_t)(at + 8 * h + g) * RANK + q * 32 + tig * EL;
        load_rank<EL>(p.t_hi + o, live[h], th[h][q]);
        load_rank<EL>(p.t_lo + o, live[h], tl[h][q]);
      }
    for (int gi = g0; gi < g1; ++gi) {
      fetch(gi + kStages - 1);
      asm volatile("cp.async.wait_group %0;" ::"n"(kStages - 1) : "memory");
      const UpStage<RANK>& st = stage[gi % kStages];
      const int n0 = gi * 32;
      uint4 bv[2] = {st.base[0][lane], st.base[1][lane]};
      float acc[4][4];  // [column tile]
#pragma unroll
      for (int i = 0; i < 4; ++i) {
#pragma unroll
        for (int e = 0; e < 4; ++e) acc[i][e] = 0.f;
#pragma unroll
        for (int q = 0; q < CH; ++q) {
          const auto b = st.up[i][q][lane];
#pragma unroll
          for (int s = 0; s < STEPS; ++s) {
            const int e0 = 2 * s, e1 = EL == 2 ? 0 : 2 * s + 1;
            const bool two = EL != 2;  // rank 8 fills half of a product's K
            mma_16816(acc[i], th[0][q][e0], th[1][q][e0], two ? th[0][q][e1] : 0u, two ? th[1][q][e1] : 0u, b.v[e0],
                      two ? b.v[e1] : 0u);
            mma_16816(acc[i], tl[0][q][e0], tl[1][q][e0], two ? tl[0][q][e1] : 0u, two ? tl[1][q][e1] : 0u, b.v[e0],
                      two ? b.v[e1] : 0u);
          }
        }
      }
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        float f[8];
        afd::bf16x8_to_float(bv[h], f);
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          f[2 * i] += acc[i][2 * h];
          f[2 * i + 1] += acc[i][2 * h + 1];
        }
        bv[h] = afd::float_to_bf16x8(f);
      }
#pragma unroll
      for (int h = 0; h < 2; ++h)
        if (live[h] && n0 + tig * 8 < p.N) *reinterpret_cast<uint4*>(out[h] + n0) = bv[h];
    }
    asm volatile("cp.async.wait_all;" ::: "memory");
  }
}

template <int RANK, bool FP8>
cudaError_t launch_adapters(const AdapterParams& p, int device, int sms, cudaStream_t stream) {
  constexpr int kDownBase = sizeof(DownShared<RANK, FP8>), kUpBase = sizeof(UpShared<RANK>);
  static std::atomic<uint64_t> down_set{0}, up_set{0};
  cudaError_t e = afd::allow_shared(adapter_up_kernel<RANK>, kUpBase + (int)table_bytes(kMaxSlots), device, up_set);
  if (e == cudaSuccess)
    e = afd::allow_shared(adapter_down_kernel<RANK, FP8>, kDownBase + (int)table_bytes(kMaxSlots), device, down_set);
  if (e != cudaSuccess) return e;
  const int down_smem = kDownBase + (int)table_bytes(p.S), up_smem = kUpBase + (int)table_bytes(p.S);
  const int down_fit = 227 * 1024 / (down_smem + 1024), up_fit = 227 * 1024 / (up_smem + 1024);  // blocks of an SM
  e = afd::launch_dependent(adapter_group_kernel, kGroupCtas, kGroupThreads, 0, stream, p);
  if (e != cudaSuccess) return e;
  // A tile holds rows of one group: at most one partial tile for each. Blocks
  // beyond what fits at once would only queue, so each takes several tiles.
  const int64_t down = (int64_t)p.R / kDownRows + (p.S < p.R ? p.S : p.R);
  const int64_t up = (p.R / kUpRows + (p.S < p.R ? p.S : p.R)) * (((int64_t)p.N + 31) / 32);
  const int64_t down_most = (int64_t)sms * (down_fit < 4 ? down_fit : 4), up_most = (int64_t)sms * (up_fit < 2 ? up_fit : 2);
  e = afd::launch_dependent(adapter_down_kernel<RANK, FP8>, down < down_most ? down : down_most, kDownWarps * 32, down_smem, stream, p);
  if (e != cudaSuccess) return e;
  return afd::launch_dependent(adapter_up_kernel<RANK>, up < up_most ? up : up_most, kUpThreads, up_smem, stream, p);
}

// Whether a cluster per row does; `rows` is the most rows that can be live. The
// row kernel reads rows * rank * (K + N) * 2 bytes of adapters from L2. The three
// launches read far less, but a tile's rank * K * 2 bytes by one block, at about
// a 64th of the rate of all. Rank 16, K = N = 2048: 128 rows (16 MiB) 4.9 against
// 10.5 us, 256 (32) 6.7 against 10.8, 512 (64) 11.2 against 11.7, padded to 128
// rows a group 9.3 against 11.0; rank 64: 128 rows (64 of 80) 9.6 against 14.2,
// 256 (128) 17.6 against 14.7. K = 7168, rank 16: 128 rows (36 of 78) 7.5 against
// 13.6, 512 (144) 19.0 against 15.0; rank 64: 64 rows (72 of 120) 10.0 against
// 21.5, 256 (288) 29.6 against 22.7. Rank 8 stops at 512 rows: 7.7 against 11.1
// (32 MiB), where 256 took 5.0. One launch in place of three and no workspace
// also take 12 us less of the caller's time.
bool few_rows(int64_t rows, int32_t rank, int32_t in_features, int32_t out_features) {
  const int64_t k = (int64_t)rank * in_features * 2, n = (int64_t)rank * out_features * 2;
  return rows <= kFewRows && rows * (k + n) <= kFewRowsBytes + 64 * k;
}

int64_t live_rows_bound(int64_t num_rows, int32_t num_tokens, int32_t top_k) {
  const int64_t routes = (int64_t)num_tokens * top_k;  // (top_k 0: rows are tokens)
  return top_k > 0 && routes < num_rows ? routes : num_rows;
}

// `few`: the most rows that can be live, where a cluster per row does; else 0.
template <int RANK, bool FP8>
cudaError_t launch_adapters_of(const AdapterParams& p, int few, int device, int sms, cudaStream_t stream) {
  if (!few) return launch_adapters<RANK, FP8>(p, device, sms, stream);
  const int ctas = few <= 32 ? 8 : few <= 64 ? 4 : 2;
  const int64_t most = (sms * (RANK <= 16 ? 4 : 2) / ctas - 1) | 1;
  return afd::launch_clusters(adapter_rows_kernel<RANK, FP8>, (p.R < most ? p.R : most) * ctas, kRowThreads, ctas, 0,
                              stream, p, ctas);
}

template <bool FP8>
cudaError_t launch_adapters_rank(const AdapterParams& p, int few, int device, int sms, cudaStream_t stream) {
  switch (p.rank) {
    case 8: return launch_adapters_of<8, FP8>(p, few, device, sms, stream);
    case 16: return launch_adapters_of<16, FP8>(p, few, device, sms, stream);
    case 32: return launch_adapters_of<32, FP8>(p, few, device, sms, stream);
    default: return launch_adapters_of<64, FP8>(p, few, device, sms, stream);
  }
}

// Bytes of the groups' starts and the order, up to a 16-byte boundary.
int64_t adapter_table_bytes(int64_t rows, int32_t slots) { return (rows + slots + 2 + 3) / 4 * 16; }

int64_t adapter_workspace(int64_t rows, int32_t slots, int32_t rank) {
  return adapter_table_bytes(rows, slots) + 2 * rows * rank * (int64_t)sizeof(uint16_t);
}

int sm_count(int device) {
  int n = 0;
  return cudaDeviceGetAttribute(&n, cudaDevAttrMultiProcessorCount, device) == cudaSuccess ? n : 0;
}

}  // namespace

extern "C" {

AFD_API afd_status afd_gated_rows(const void* h, int64_t h_stride, const int32_t* ends, int32_t num_groups,
                                  int32_t expert_alignment, int64_t num_rows, int32_t features, void* out,
                                  int64_t out_stride, afd_stream stream) {
  if (num_groups < 1 || expert_alignment < 1 || num_rows < 0 || features < 1 || !ends) return AFD_ERR_ARG;
  if (h_stride < 2 * (int64_t)features || out_stride < features) return AFD_ERR_ARG;
  if (num_groups > afd::kMaxExperts || num_rows > afd::kMaxRows - expert_alignment || features > afd::kMaxFeatures)
    return AFD_ERR_UNSUPPORTED;
  if (num_rows == 0) return AFD_OK;
  if (!h || !out) return AFD_ERR_ARG;
  GatedParams p = {nullptr, h_stride, nullptr, num_groups, expert_alignment, (int32_t)num_rows, features, nullptr, out_stride};
  if (!afd::device_view(static_cast<const uint16_t*>(h), &p.h) || !afd::device_view(ends, &p.ends) ||
      !afd::device_view(static_cast<uint16_t*>(out), &p.out))
    return AFD_ERR_ARG;
  if (!afd::aligned_to(p.h, 2) || !afd::aligned_to(p.out, 2) || !afd::aligned_to(p.ends, 4)) return AFD_ERR_ARG;
  int dev = -1;
  if (cudaGetDevice(&dev) != cudaSuccess) return AFD_ERR_CUDA;
  const int sms = sm_count(dev);
  if (sms < 1) return AFD_ERR_CUDA;
  const bool vec = features % 8 == 0 && h_stride % 8 == 0 && out_stride % 8 == 0 && afd::aligned_to(p.h, 16) &&
                   afd::aligned_to(p.out, 16);
  const int64_t blocks = (num_rows + 7) / 8, grid = blocks < sms * 8 ? blocks : sms * 8;
  cudaStream_t st = reinterpret_cast<cudaStream_t>(stream);
  const cudaError_t e = vec ? afd::launch_dependent(gated_rows_kernel<true>, grid, 256, 0, st, p)
                            : afd::launch_dependent(gated_rows_kernel<false>, grid, 256, 0, st, p);
  return e == cudaSuccess ? AFD_OK : AFD_ERR_CUDA;
}

AFD_API int64_t afd_adapter_workspace_bytes(int64_t num_rows, int32_t num_tokens, int32_t top_k, int32_t num_slots,
                                            int32_t rank, int32_t in_features, int32_t out_features) {
  if (num_rows < 0 || num_tokens < 0 || top_k < 0 || num_slots < 1 || rank < 1 || in_features < 1 || out_features < 1)
    return -1;
  if (few_rows(live_rows_bound(num_rows, num_tokens, top_k), rank, in_features, out_features)) return 0;
  return adapter_workspace(num_rows, num_slots, rank);
}

AFD_API afd_status afd_adapter_add(const void* base, int64_t base_stride, const void* x, int64_t x_stride,
                                   const float* x_scale, const void* down, const void* up, const int32_t* token_slots, const float* scales,
                                   const int32_t* row_src, const int32_t* ends, int32_t num_groups, int32_t top_k,
                                   int64_t num_rows, int32_t num_tokens, int32_t num_slots, int32_t rank,
                                   int32_t in_features, int32_t out_features, void* out, int64_t out_stride,
                                   void* workspace, int64_t workspace_bytes, afd_stream stream) {
  if (num_rows < 0 || num_tokens < 0 || num_slots < 1 || rank < 1 || in_features < 1 || out_features < 1)
    return AFD_ERR_ARG;
  if (base_stride < out_features || out_stride < out_features || x_stride < in_features) return AFD_ERR_ARG;
  if (row_src ? (!ends || num_groups < 1 || top_k < 1) : num_tokens < num_rows) return AFD_ERR_ARG;
  if (rank != 8 && rank != 16 && rank != 32 && rank != 64) return AFD_ERR_UNSUPPORTED;
  const bool fp8 = x_scale != nullptr;
  if (in_features % (fp8 ? 128 : 16) || out_features % 8 || base_stride % 8 || out_stride % 8 || x_stride % (fp8 ? 16 : 8) ||
      num_rows > afd::kMaxRows || num_slots > kMaxSlots || in_features > afd::kMaxFeatures ||
      out_features > afd::kMaxFeatures)
    return AFD_ERR_UNSUPPORTED;
  if (num_rows == 0 || num_tokens == 0) return AFD_OK;
  if (!base || !x || !down || !up || !token_slots || !scales || !out) return AFD_ERR_ARG;
  const int64_t live = live_rows_bound(num_rows, num_tokens, row_src ? top_k : 0);
  const bool few = few_rows(live, rank, in_features, out_features);
  if (!few && (!workspace || workspace_bytes < adapter_workspace(num_rows, num_slots, rank))) return AFD_ERR_ARG;
  AdapterParams p = {};
  p.base_stride = base_stride, p.x_stride = x_stride * (fp8 ? 1 : 2), p.out_stride = out_stride;
  p.G = num_groups, p.top_k = top_k, p.R = (int32_t)num_rows, p.tokens = num_tokens, p.S = num_slots, p.rank = rank;
  p.K = in_features, p.N = out_features;
  if (!afd::device_view(static_cast<const uint16_t*>(base), &p.base) ||
      !afd::device_view(static_cast<const uint8_t*>(x), &p.x) || (fp8 && !afd::device_view(x_scale, &p.x_scale)) ||
      !afd::device_view(static_cast<const uint16_t*>(down), &p.down) ||
      !afd::device_view(static_cast<const uint16_t*>(up), &p.up) || !afd::device_view(token_slots, &p.token_slots) ||
      !afd::device_view(scales, &p.scales) || !afd::device_view(static_cast<uint16_t*>(out), &p.out) ||
      (!few && !afd::device_view(static_cast<int32_t*>(workspace), &p.first)) ||
      (row_src && (!afd::device_view(row_src, &p.row_src) || !afd::device_view(ends, &p.ends))))
    return AFD_ERR_ARG;
  if (!few) {
    p.order = p.first + num_slots + 2;
    p.t_hi = reinterpret_cast<uint16_t*>(reinterpret_cast<uint8_t*>(p.first) + adapter_table_bytes(num_rows, num_slots));
    p.t_lo = p.t_hi + num_rows * rank;
  }
  if (!afd::aligned_to(p.first, 16) || !afd::aligned_to(p.token_slots, 4) || !afd::aligned_to(p.scales, 4) ||
      !afd::aligned_to(p.x_scale, 4) || !afd::aligned_to(p.row_src, 4) || !afd::aligned_to(p.ends, 4))
    return AFD_ERR_ARG;
  if (!afd::aligned_to(p.base, 16) || !afd::aligned_to(p.x, 16) || !afd::aligned_to(p.down, 16) ||
      !afd::aligned_to(p.up, 16) || !afd::aligned_to(p.out, 16))
    return AFD_ERR_UNSUPPORTED;
  int dev = -1;
  if (cudaGetDevice(&dev) != cudaSuccess) return AFD_ERR_CUDA;
  const int sms = sm_count(dev);
  if (sms < 1) return AFD_ERR_CUDA;
  cudaStream_t st = reinterpret_cast<cudaStream_t>(stream);
  const int rows = few ? (int)live : 0;
  const cudaError_t e = fp8 ? launch_adapters_rank<true>(p, rows, dev, sms, st) : launch_adapters_rank<false>(p, rows, dev, sms, st);
  return e == cudaSuccess ? AFD_OK : AFD_ERR_CUDA;
}

}  // extern "C"
