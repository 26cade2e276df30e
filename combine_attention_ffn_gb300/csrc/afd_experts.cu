// afd_grouped_linear: the experts' matrix product over received rows, on the
// fifth-generation tensor cores.
//
// The product is computed transposed, out^T = W x^T: a pair of CTAs holds 256
// weight rows (the products' M, 128 a CTA) against up to 256 received rows
// (their N, any multiple of 32). An expert's rows are cut into equal tiles, so
// a ragged expert wastes at most 31 columns a tile, where rows as M would be
// padded to 128 or 256 (a prefill bucket has 256 +- 16 rows an expert), and a
// decode step streams the touched experts' weights past a 32-column product.
// Each CTA of a pair loads its 128 weight rows and half the received rows, and
// the tensor cores read both halves: half the L2 traffic of single CTAs.
//
// Persistent pairs walk the tiles (expert, weight tile, row tile) with these
// roles per CTA: warp 0 loads by tiled bulk copies (K blocks of 128 bytes, a
// ring of stages), warp 1 of the even CTA issues the products, sixteen warps
// drain the accumulators, which take turns in TMEM (two of 256 columns, or more
// and narrower ones where the widest tile is narrower): the next tile's
// products run while the last one's are stored.
//
// Tiles are dealt out once, widest experts first and back and forth over the
// pairs: on a prefill bucket the pair with the most work has 1.04 times the
// mean, dealt in the experts' order 1.09 to 1.14 times.
//
// Gated: a bulk copy with dimensions (k, half, row) interleaves gate and up
// rows in shared memory, so the two sums of an output sit in neighbouring
// lanes and one shuffle brings them together.
//
// What bounds it, measured (16.4 K rows of 64 experts, K 2048, 2 x 1024 weight
// rows, gated, BF16: 116 us): no one thing. 1.35 GB come from L2 at 11.6 TB/s,
// 640 MB from DRAM at 5.5 TB/s, the tensor pipes are 55% busy; without any row
// loads it takes 106 us, without stores 108. A decode step (one token a source)
// streams the touched experts' weights: 8 in 15.4 us, 9 in 16.4 at 4.6 TB/s.
// One lane alone in the loops of the loading and issuing warps, as a first form
// had it, took 100 clocks an issue and 150 us.
//
// FP8: each 128-wide K block has scales of its own, so it gets an accumulator
// of its own; the draining warps add it, scaled, to FP32 sums in registers:
// one multiply-add a value, with x_scale * weight_scale multiplied once per
// row and block by warps 2 and 3, which keep a ring of them in shared memory.
// 64 sums a thread need more than an even share of the registers, so the
// other warps hand some of theirs over. With many rows (the shape above: 108 us
// against a floor of 50) the hand-over bounds it: issue slots are 56% busy, the
// tensor pipes 27%, and with two accumulators in TMEM a block's products wait
// until all draining warps have added the one before the last. Eight warps with
// twice the sums took 128 us.

#include <cuda.h>
#include <cuda_runtime.h>
#include <stdint.h>

#include <atomic>

#include "afd.h"
#include "afd_device.cuh"
#include "afd_pointers.cuh"
#include "afd_ragged.cuh"
#include "afd_tcgen05.cuh"

namespace {

constexpr int kPairRows = 256;    // weight rows of a tile (two CTAs)
constexpr int kCtaRows = 128;
constexpr int kTileRows = 256;    // received rows of a tile, at most
constexpr int kBlockBytes = 128;  // bytes of K per stage and row
constexpr int kHalfBytes = kCtaRows * kBlockBytes;  // a stage's weight rows
constexpr int kRingBytes = 6 * 2 * kHalfBytes;      // six stages of the widest tiles, or more of narrower ones
constexpr int kMaxStages = 8;  // (ten: the same for BF16, 3% slower for FP8 with few rows)
constexpr int kDrainWarps = 16;
constexpr int kDrainParts = kDrainWarps / 4;  // warps that share 32 lanes of TMEM, 16 columns each in turn
constexpr int kThreads = 128 + 32 * kDrainWarps;
constexpr int kColumns = 512;     // all of TMEM
constexpr int kMaxBufs = 8;       // accumulators in it, at most
constexpr int kClasses = kTileRows / 32;  // tile widths
constexpr int kListed = 64;       // tiles of a pair that are looked up before the roles start
constexpr int kColStep = 32;      // received rows of a product come in multiples of this
constexpr int kRowMaps = 8;       // boxes of 16, 32, .. 128 received rows: one copy a stage, whatever the tile
constexpr int kScaleStages = 8;   // ring of scales (FP8)
constexpr int kScaleThreads = 64; // warps 2 and 3
constexpr int kScaleRows = kTileRows / kScaleThreads;
constexpr int kScaleAhead = 4;    // blocks whose scales are loaded together
// Registers a thread after the hand-over (FP8): 128 x 64 + 512 x 104, at most
// what the block is launched with (checked before the first launch).
constexpr int kFrontRegs = 64, kDrainRegs = 104;

struct Maps {
  CUtensorMap w;
  CUtensorMap x[kRowMaps];
};

struct ExpertParams {
  const float* x_scale;
  const float* w_scale;
  const int32_t* ends;
  int32_t G, alpha, R, K, N;
  int32_t m_tiles;   // weight tiles of an expert
  int32_t k_blocks;
  int32_t vec;       // out takes 4-byte stores of two columns
  uint16_t* out;
  int64_t out_stride;
  int32_t* error;
  int64_t wait_cycles;  // of every wait, at most; 0: give up without one
};

struct alignas(16) BlockScales {
  float s[2][kTileRows + 4];  // [gate / up][received row]; plain uses the first
};

struct alignas(16) Tile {
  int group, m, row, rows;
  __device__ __forceinline__ int cols() const { return (rows + kColStep - 1) & -kColStep; }
};

struct Shared {
  alignas(8) uint64_t full[kMaxStages], empty[kMaxStages];
  uint64_t drain_full[kMaxBufs];  // an accumulator's products are complete
  uint64_t drained[kMaxBufs];     // this CTA's warps have read it
  uint64_t peer_drained[kMaxBufs];  // ... and the other CTA's (used in the even one)
  uint64_t scale_full[kScaleStages], scale_empty[kScaleStages];
  uint32_t tmem;
  int gave_up;
  int widest, mixed;               // widest tile, and whether there are others
  int end[afd::kMaxExperts];
  int first_tile[afd::kMaxExperts + 1];  // by position in `order`
  uint16_t order[afd::kMaxExperts];      // the groups, widest tiles first
  uint16_t class_count[afd::kMaxExperts / 32][kClasses + 1];
  Tile list[kListed];                    // this pair's first tiles
  BlockScales scale[kScaleStages];
};

constexpr size_t kSmem = 1024 + kRingBytes + sizeof(Shared);
static_assert(kSmem <= 232448, "shared memory of one CTA");

__device__ __forceinline__ int row_tiles(int count) { return (count + kTileRows - 1) / kTileRows; }

// Width of a group's tiles: its rows in equal parts, whole column steps.
__device__ __forceinline__ int tile_width(int count) {
  const int n = row_tiles(count);
  return n ? ((count + n - 1) / n + kColStep - 1) & -kColStep : 0;
}

__device__ __forceinline__ int group_count(const Shared& sh, const ExpertParams& p, int g) {
  return max(sh.end[g] - (g ? afd::group_start(sh.end[g - 1], p.alpha, p.R) : 0), 0);
}

// Tile `t` of this pair's turn: every second turn goes back over the pairs.
__device__ __forceinline__ int dealt(int turn, int pair, int pairs) {
  return turn * pairs + (turn & 1 ? pairs - 1 - pair : pair);
}

__device__ __forceinline__ Tile find_tile(const Shared& sh, const ExpertParams& p, int t) {
  int lo = 0, hi = p.G - 1;  // the last group whose first tile is at or before t, skipping empty ones
  while (lo < hi) {
    const int mid = (lo + hi + 1) >> 1;
    if (sh.first_tile[mid] <= t) lo = mid; else hi = mid - 1;
  }
  Tile tile;
  tile.group = sh.mixed ? sh.order[lo] : lo;
  const int start = tile.group ? afd::group_start(sh.end[tile.group - 1], p.alpha, p.R) : 0;
  const int count = sh.end[tile.group] - start, n = row_tiles(count), width = tile_width(count);
  const int i = t - sh.first_tile[lo];
  tile.m = i / n;
  const int off = (i - tile.m * n) * width;
  tile.row = start + off;
  tile.rows = min(width, count - off);  // at least 1: (n - 1) * width < count
  return tile;
}

// The tile of this pair's turn; false: it has none.
__device__ __forceinline__ bool next_tile(const Shared& sh, const ExpertParams& p, int turn, int pair, int pairs, int tiles,
                                          Tile* tile) {
  const int t = dealt(turn, pair, pairs);
  if (t >= tiles) return false;
  *tile = turn < kListed ? sh.list[turn] : find_tile(sh, p, t);
  return true;
}

// Where a lane stores: two neighbouring columns of every second (plain) or
// fourth (gated) row, or with other strides one column.
struct Out {
  uint16_t* at;      // the lane's column in its first row of the tile
  int64_t step;      // elements from one of its rows to the next
  int row;           // its first row in a chunk
  bool in;           // its columns exist
  uint32_t select;   // which halves of two lanes' pairs it stores
};

template <bool GATED>
__device__ __forceinline__ Out lane_out(const ExpertParams& p, const Tile& tile, int n0, int lane) {
  Out o;
  const int odd = lane & 1, upper = lane >> 1 & 1;
  const int n = n0 + (GATED ? lane >> 1 : lane);
  const int side = GATED ? upper : odd;
  o.row = GATED ? (p.vec ? 2 * upper + odd : odd) : (p.vec ? odd : 0);
  o.step = p.out_stride * (GATED ? (p.vec ? 4 : 2) : (p.vec ? 2 : 1));
  o.in = n < p.N;
  o.select = side ? 0x3276 : 0x5410;
  o.at = p.out + (int64_t)(tile.row + o.row) * p.out_stride + (p.vec ? n & ~1 : n);
  return o;
}

// Stores 16 received rows x 32 lanes of sums: lane = weight row, v[i] = row i.
// Rows are exchanged between neighbouring lanes in pairs, so that each lane
// completes one output of two (gated), then stores two columns at a time.
template <bool GATED>
__device__ __forceinline__ void store16(const ExpertParams& p, const Tile& tile, const Out& o, int c0, int lane,
                                        const float (&v)[16]) {
  const int left = o.in ? tile.rows - c0 - o.row : 0;
  uint16_t* at = o.at + c0 * p.out_stride;
  if (GATED) {
    const bool odd = lane & 1;
    float a[8];  // outputs of row 2 i + odd
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const float mine = odd ? v[2 * i + 1] : v[2 * i];
      const float other = __shfl_xor_sync(0xffffffffu, odd ? v[2 * i] : v[2 * i + 1], 1);
      a[i] = afd::silu_mul(odd ? other : mine, odd ? mine : other);
    }
    if (p.vec) {
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const uint32_t two = afd::pack_bf16(a[2 * i], a[2 * i + 1]);
        const uint32_t out = __byte_perm(two, __shfl_xor_sync(0xffffffffu, two, 2), o.select);
        if (4 * i < left) *reinterpret_cast<uint32_t*>(at) = out;
        at += o.step;
      }
    } else {
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        if (2 * i < left) *at = (uint16_t)afd::pack_bf16(a[i], 0.f);
        at += o.step;
      }
    }
  } else if (p.vec) {
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const uint32_t two = afd::pack_bf16(v[2 * i], v[2 * i + 1]);
      const uint32_t out = __byte_perm(two, __shfl_xor_sync(0xffffffffu, two, 1), o.select);
      if (2 * i < left) *reinterpret_cast<uint32_t*>(at) = out;
      at += o.step;
    }
  } else {
#pragma unroll
    for (int i = 0; i < 16; ++i) {
      if (i < left) *at = (uint16_t)afd::pack_bf16(v[i], 0.f);
      at += o.step;
    }
  }
}

// The ring of stages. Narrow tiles leave room for more of them: with six a
// decode step of 128 skewed tokens took 3% longer than with eight.
struct Ring {
  int stages, bytes;         // of a stage: weight rows, then half the widest tile's received rows
  uint32_t count = 0;        // stages passed so far
  int slot = 0;
  uint32_t phase = 0;
  __device__ __forceinline__ explicit Ring(int widest)
      : stages(min(kMaxStages, kRingBytes / (kHalfBytes + widest / 2 * kBlockBytes))), bytes(kHalfBytes + widest / 2 * kBlockBytes) {}
  __device__ __forceinline__ void advance() {
    ++count;
    if (++slot == stages) slot = 0, phase ^= 1;
  }
  // Calls wait(slot, parity) for the last stages passed, oldest first.
  template <typename F>
  __device__ __forceinline__ void last(F wait) const {
    for (uint32_t i = count > (uint32_t)stages ? count - stages : 0; i < count; ++i) wait(i % stages, i / stages & 1);
  }
};

// The accumulators' turns: unit u uses buffer u & (bufs - 1).
struct Turns {
  uint32_t tmem, full, drained;  // addresses of buffer 0
  int shift;                     // log2 bufs
  int cols;                      // columns of a buffer
  __device__ __forceinline__ uint32_t buf(uint32_t unit) const { return unit & ((1u << shift) - 1); }
  __device__ __forceinline__ uint32_t phase(uint32_t unit) const { return unit >> shift & 1; }
};

// One tile's FP8 blocks: every block's products, scaled, into FP32 sums in
// registers, then the store. The number of steps is a constant: a sum that a
// branch may or may not add to is moved twice a step.
template <bool GATED, int STEPS>
__device__ __forceinline__ bool drain_blocks(const ExpertParams& p, Shared& sh, const Tile& tile, const Turns& turns,
                                             const Out& out, int h, int lane, uint32_t& unit) {
  const uint32_t scale_full = afd::smem_u32(sh.scale_full), scale_empty = afd::smem_u32(sh.scale_empty);
  float sum[STEPS + 1][16];
#pragma unroll
  for (int i = 0; i < STEPS; ++i)
#pragma unroll
    for (int j = 0; j < 16; ++j) sum[i][j] = 0.f;
  for (int kb = 0; kb < p.k_blocks; ++kb, ++unit) {
    const uint32_t s = unit % kScaleStages, b = turns.buf(unit);
    if (!afd::mbar_wait(scale_full + 8 * s, (unit / kScaleStages) & 1, &sh.gave_up, p.wait_cycles) ||
        !afd::mbar_wait(turns.full + 8 * b, turns.phase(unit), &sh.gave_up, p.wait_cycles))
      return false;
    afd::tcgen05_fence_after();
    const uint32_t acc = turns.tmem + b * turns.cols + 16 * h;
    const float* sc = sh.scale[s].s[GATED ? lane & 1 : 0] + 16 * h;
#pragma unroll
    for (int i = 0; i < STEPS; ++i) {
      const int c = 16 * kDrainParts * i;
      float v[16];
      afd::tmem_load16(acc + c, v);
#pragma unroll
      for (int j = 0; j < 16; j += 4) {
        const float4 s4 = *reinterpret_cast<const float4*>(sc + c + j);
        sum[i][j] = fmaf(v[j], s4.x, sum[i][j]);
        sum[i][j + 1] = fmaf(v[j + 1], s4.y, sum[i][j + 1]);
        sum[i][j + 2] = fmaf(v[j + 2], s4.z, sum[i][j + 2]);
        sum[i][j + 3] = fmaf(v[j + 3], s4.w, sum[i][j + 3]);
      }
    }
    afd::tcgen05_fence_before();
    __syncwarp();
    if (lane == 0) {
      afd::mbar_arrive(turns.drained + 8 * b);
      afd::mbar_arrive(scale_empty + 8 * s);
    }
  }
#pragma unroll
  for (int i = 0; i < STEPS; ++i) store16<GATED>(p, tile, out, 16 * (kDrainParts * i + h), lane, sum[i]);
  return true;
}

template <bool FP8, bool GATED>
__global__ void __cluster_dims__(2, 1, 1) __launch_bounds__(kThreads, 1)
    grouped_linear_kernel(const __grid_constant__ Maps maps, const ExpertParams p) {
  extern __shared__ uint8_t smem_raw[];
  const uint32_t smem = (afd::smem_u32(smem_raw) + 1023) & ~1023u;
  Shared& sh = *reinterpret_cast<Shared*>(smem_raw + (smem - afd::smem_u32(smem_raw)) + kRingBytes);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const uint32_t rank = afd::cluster_rank();
  const int pair = blockIdx.x >> 1, pairs = gridDim.x >> 1;
  const uint32_t full = afd::smem_u32(sh.full), empty = afd::smem_u32(sh.empty);
  const uint32_t drain_full = afd::smem_u32(sh.drain_full), drained = afd::smem_u32(sh.drained);
  const uint32_t peer_drained = afd::smem_u32(sh.peer_drained);
  const uint32_t scale_full = afd::smem_u32(sh.scale_full), scale_empty = afd::smem_u32(sh.scale_empty);

  if (warp == 0 && lane == 0) {
    for (int i = 0; i < kMaxStages; ++i) {
      afd::mbar_init(full + 8 * i, 1);
      afd::mbar_init(empty + 8 * i, 1);
    }
    for (int i = 0; i < kMaxBufs; ++i) {
      afd::mbar_init(drain_full + 8 * i, 1);
      afd::mbar_init(drained + 8 * i, kDrainWarps);
      afd::mbar_init(peer_drained + 8 * i, 1);
    }
    for (int i = 0; FP8 && i < kScaleStages; ++i) {
      afd::mbar_init(scale_full + 8 * i, kScaleThreads);
      afd::mbar_init(scale_empty + 8 * i, kDrainWarps);
    }
    sh.gave_up = p.wait_cycles == 0;
    asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
  }
  if (warp == 1) afd::tmem_alloc_pair(afd::smem_u32(&sh.tmem), kColumns);
  // Up to here nothing of another kernel's has been touched.
  afd::pdl_wait();
  afd::pdl_launch_dependents();
  // every group's end, then the prefix sums of the groups' tiles
  for (int g = threadIdx.x; g < p.G; g += kThreads) sh.end[g] = afd::group_end(p.ends[g], p.R);
  __syncthreads();
  if (warp == 2) {
    int widest = 0, narrowest = kTileRows, carry = 0;
    for (int g0 = 0; g0 < p.G; g0 += 32) {
      const int g = g0 + lane, count = g < p.G ? group_count(sh, p, g) : 0;
      const int w = tile_width(count), n = row_tiles(count) * p.m_tiles;
      widest = max(widest, w);
      if (w) narrowest = min(narrowest, w);
      const int incl = afd::warp_inclusive_scan(n);
      if (g < p.G) sh.first_tile[g] = carry + incl - n;
      carry += __shfl_sync(0xffffffffu, incl, 31);
    }
    widest = __reduce_max_sync(0xffffffffu, widest);
    narrowest = __reduce_min_sync(0xffffffffu, narrowest);
    if (lane == 0) {
      sh.widest = max(widest, kColStep);
      sh.mixed = narrowest < widest;
      sh.first_tile[p.G] = carry;
    }
  }
  __syncthreads();
  if (sh.mixed) {
    // A stable counting sort of the groups by width: counts of 32 groups and
    // class, their prefix with the widest class first, then the places.
    for (int c = warp; c * 32 < p.G; c += kThreads / 32) {
      const int g = c * 32 + lane;
      const int k = g < p.G ? kClasses - tile_width(group_count(sh, p, g)) / kColStep : -1;  // 0: widest
      int place = 0;
      for (int i = 0; i <= kClasses; ++i) {
        const unsigned m = __ballot_sync(0xffffffffu, k == i);
        if (k == i) place = __popc(m & ((1u << lane) - 1));
        if (lane == i) sh.class_count[c][i] = (uint16_t)__popc(m);
      }
      if (g < p.G) sh.first_tile[g] = k << 16 | place;  // kept until the places are known
    }
    __syncthreads();
    if (warp == 2) {
      int carry = 0;
      for (int i = 0; i <= kClasses; ++i) {
        const int n = lane * 32 < p.G ? sh.class_count[lane][i] : 0;
        const int incl = afd::warp_inclusive_scan(n);
        if (lane * 32 < p.G) sh.class_count[lane][i] = (uint16_t)(carry + incl - n);
        carry += __shfl_sync(0xffffffffu, incl, 31);
      }
    }
    __syncthreads();
    for (int g = threadIdx.x; g < p.G; g += kThreads) {
      const int v = sh.first_tile[g];
      sh.order[sh.class_count[g >> 5][v >> 16] + (v & 0xffff)] = (uint16_t)g;
    }
    __syncthreads();
    if (warp == 2) {
      int carry = 0;
      for (int i0 = 0; i0 < p.G; i0 += 32) {
        const int i = i0 + lane;
        const int n = i < p.G ? row_tiles(group_count(sh, p, sh.order[i])) * p.m_tiles : 0;
        const int incl = afd::warp_inclusive_scan(n);
        if (i < p.G) sh.first_tile[i] = carry + incl - n;
        carry += __shfl_sync(0xffffffffu, incl, 31);
      }
    }
    __syncthreads();
  }
  const int tiles = sh.first_tile[p.G];
  if (threadIdx.x < kListed) {
    const int t = dealt(threadIdx.x, pair, pairs);
    if (t < tiles) sh.list[threadIdx.x] = find_tile(sh, p, t);
  }
  afd::tcgen05_fence_before();
  __syncthreads();
  afd::cluster_sync_all();
  afd::tcgen05_fence_after();
  const uint32_t tmem = sh.tmem;
  volatile int* gave_up = &sh.gave_up;
  // as many accumulators of the widest tile's columns (a power of two) as fit
  const int wide = 32 - __clz(sh.widest - 1);
  const int buf_shift = min(wide < 6 ? 3 : 9 - wide, 3);
  const Turns turns = {tmem, drain_full, drained, buf_shift, kColumns >> buf_shift};

  if (warp < 4) {
    if (FP8) asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(kFrontRegs));
    if (warp == 0) {
      // ---------------------------------------------------------------- loads
      // The whole warp walks the loop and one elected lane issues: with a single
      // lane in it the compiler cannot keep the operands in uniform registers,
      // and an issue takes 100 clocks and more.
      // Weights read once leave L2 first (with one priority for all a decode step
      // takes 4% longer). The rest keeps the normal one: evict-last would gain
      // 0.5% here and hold its lines against whatever runs next.
      uint64_t keep, once;
      asm("createpolicy.fractional.L2::evict_normal.b64 %0, 1.0;" : "=l"(keep));
      asm("createpolicy.fractional.L2::evict_first.b64 %0, 1.0;" : "=l"(once));
      const uint32_t lead_full = afd::map_to_rank(full, 0);
      Ring ring(sh.widest);
      bool ok = p.wait_cycles != 0;
      Tile tile;
      for (int turn = 0; ok && next_tile(sh, p, turn, pair, pairs, tiles, &tile); ++turn) {
        const int half = tile.cols() >> 1;
        const int row = tile.row + (int)rank * half;
        const uint32_t bytes = 2 * (kHalfBytes + half * kBlockBytes);
        const CUtensorMap* x_map = &maps.x[half / 16 - 1];
        // this weight tile is read again if the expert has more row tiles
        const uint64_t w_policy = tile.rows == group_count(sh, p, tile.group) ? once : keep;
        const int w_row = GATED ? tile.m * (kPairRows / 2) + (int)rank * (kCtaRows / 2) : tile.m * kPairRows + (int)rank * kCtaRows;
        for (int kb = 0; kb < p.k_blocks; ++kb, ring.advance()) {
          const int s = ring.slot;
          if (!(ok = afd::mbar_wait(empty + 8 * s, ring.phase ^ 1, gave_up, p.wait_cycles))) break;
          const uint32_t a = smem + s * ring.bytes, b = a + kHalfBytes, bar = lead_full + 8 * s;
          const int k = kb * (FP8 ? 128 : 64);
          if (afd::elect_one()) {
            if (rank == 0) afd::mbar_expect(full + 8 * s, bytes);
            if (GATED)
              afd::tma_load_4d(a, &maps.w, bar, k, 0, w_row, tile.group, w_policy);
            else
              afd::tma_load_3d(a, &maps.w, bar, k, w_row, tile.group, w_policy);
            afd::tma_load_2d(b, x_map, bar, k, row, keep);
          }
          __syncwarp();
        }
      }
      // The pair's last products have read this CTA's operands.
      ring.last([&](int slot, uint32_t parity) { ok = ok && afd::mbar_wait(empty + 8 * slot, parity, gave_up, p.wait_cycles); });
      if (!ok && rank == 0) {
        // Copies in flight count on this CTA's barriers: wait for the last ring of them.
        ring.last([&](int slot, uint32_t parity) {
          const long long t0 = clock64();
          while (!afd::mbar_try(full + 8 * slot, parity) && clock64() - t0 < 2000000) {
          }
        });
      }
      __syncwarp();
    } else if (warp == 1) {
      // ------------------------------------------------------------- products
      if (rank == 0) {
        Ring ring(sh.widest);
        uint32_t unit = 0;
        bool ok = p.wait_cycles != 0;
        Tile tile;
        for (int turn = 0; ok && next_tile(sh, p, turn, pair, pairs, tiles, &tile); ++turn) {
          const uint32_t idesc = afd::instr_desc(FP8, kPairRows, tile.cols());
          for (int kb = 0; kb < p.k_blocks; ++kb, ring.advance()) {
            const bool opens = FP8 || kb == 0, closes = FP8 || kb == p.k_blocks - 1;
            if (opens) {
              const uint32_t buf = turns.buf(unit), ph = turns.phase(unit) ^ 1;
              ok = afd::mbar_wait(drained + 8 * buf, ph, gave_up, p.wait_cycles) && afd::mbar_wait(peer_drained + 8 * buf, ph, gave_up, p.wait_cycles);
              if (!ok) break;
            }
            const int s = ring.slot;
            if (!(ok = afd::mbar_wait(full + 8 * s, ring.phase, gave_up, p.wait_cycles))) break;
            afd::tcgen05_fence_after();
            const uint64_t a = afd::operand_desc(smem + s * ring.bytes);
            const uint64_t b = afd::operand_desc(smem + s * ring.bytes + kHalfBytes);
            const uint32_t d = tmem + turns.buf(unit) * turns.cols;
            if (afd::elect_one()) {
#pragma unroll
              for (int i = 0; i < 4; ++i)  // 32 bytes of K each
                afd::mma_pair<FP8>(d, a + 2 * i, b + 2 * i, idesc, !(opens && i == 0));
              afd::mma_commit_pair(empty + 8 * s);
              if (closes) afd::mma_commit_pair(drain_full + 8 * turns.buf(unit));
            }
            __syncwarp();
            if (closes) ++unit;
          }
        }
      } else {
        // The odd CTA's warp passes on that its accumulators are read: one
        // arrival across the pair instead of one for every draining warp.
        const uint32_t lead = afd::map_to_rank(peer_drained, 0);
        uint32_t unit = 0;
        bool ok = p.wait_cycles != 0;
        for (int turn = 0; ok && dealt(turn, pair, pairs) < tiles; ++turn) {
          for (int kb = 0; kb < (FP8 ? p.k_blocks : 1); ++kb, ++unit) {
            const uint32_t buf = turns.buf(unit);
            if (!(ok = afd::mbar_wait(drained + 8 * buf, turns.phase(unit), gave_up, p.wait_cycles))) break;
            if (lane == 0) afd::mbar_arrive_cluster(lead + 8 * buf);
          }
        }
      }
      __syncwarp();
    } else {
      // --------------------------------------------------------------- scales
      if (FP8) {
        const int u = threadIdx.x - 64;
        const int64_t w_rows = (int64_t)(GATED ? 2 : 1) * p.N / 128;
        uint32_t it = 0;
        bool ok = p.wait_cycles != 0;
        Tile tile;
        for (int turn = 0; ok && next_tile(sh, p, turn, pair, pairs, tiles, &tile); ++turn) {
          const float* xs = p.x_scale + (int64_t)(tile.row + u) * p.k_blocks;
          // the weight block of this CTA's rows (the last one for rows past N, which are not stored)
          const int f = GATED ? tile.m * (kPairRows / 2) + (int)rank * (kCtaRows / 2) : tile.m * kPairRows + (int)rank * kCtaRows;
          const float* wg = p.w_scale + (tile.group * w_rows + min(f, p.N - 1) / 128) * p.k_blocks;
          const float* wu = wg + (int64_t)(p.N / 128) * p.k_blocks;
          // kScaleAhead blocks are loaded at a time; the ring is twice as long,
          // so the loads of the next ones overlap the use of these
          for (int kb0 = 0; ok && kb0 < p.k_blocks; kb0 += kScaleAhead) {
            float x[kScaleAhead][kScaleRows], w[kScaleAhead][2];
#pragma unroll
            for (int j = 0; j < kScaleAhead; ++j) {
              const int kb = min(kb0 + j, p.k_blocks - 1);
              w[j][0] = wg[kb];
              w[j][1] = GATED ? wu[kb] : 0.f;
#pragma unroll
              for (int i = 0; i < kScaleRows; ++i)
                x[j][i] = u + kScaleThreads * i < tile.rows ? xs[(int64_t)kScaleThreads * i * p.k_blocks + kb] : 0.f;
            }
#pragma unroll
            for (int j = 0; j < kScaleAhead; ++j) {
              if (ok && kb0 + j < p.k_blocks) {
                const uint32_t s = it % kScaleStages, ph = (it / kScaleStages) & 1;
                ok = afd::mbar_wait(scale_empty + 8 * s, ph ^ 1, gave_up, p.wait_cycles);
                if (ok) {
                  ++it;
#pragma unroll
                  for (int i = 0; i < kScaleRows; ++i) {
                    sh.scale[s].s[0][u + kScaleThreads * i] = x[j][i] * w[j][0];
                    if (GATED) sh.scale[s].s[1][u + kScaleThreads * i] = x[j][i] * w[j][1];
                  }
                  afd::mbar_arrive(scale_full + 8 * s);
                }
              }
            }
          }
        }
      }
    }
  } else {
    // ----------------------------------------------------------- accumulators
    if (FP8) asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(kDrainRegs));
    const int q = warp & 3, h = (warp - 4) >> 2;  // lanes 32 q .. of TMEM; every fourth 16 columns
    Turns mine = turns;
    mine.tmem += (uint32_t)(32 * q) << 16;
    uint32_t unit = 0;
    bool ok = p.wait_cycles != 0;
    Tile tile;
    for (int turn = 0; ok && next_tile(sh, p, turn, pair, pairs, tiles, &tile); ++turn) {
      const int n0 = GATED ? tile.m * (kPairRows / 2) + (int)rank * (kCtaRows / 2) + 16 * q
                           : tile.m * kPairRows + (int)rank * kCtaRows + 32 * q;
      const Out out = lane_out<GATED>(p, tile, n0, lane);
      if (!FP8) {
        const uint32_t b = turns.buf(unit);
        ok = afd::mbar_wait(drain_full + 8 * b, turns.phase(unit), gave_up, p.wait_cycles);
        if (!ok) break;
        afd::tcgen05_fence_after();
        for (int c = 16 * h; c < tile.cols(); c += 16 * kDrainParts) {
          float v[16];
          afd::tmem_load16(mine.tmem + b * turns.cols + c, v);
          store16<GATED>(p, tile, out, c, lane, v);
        }
        afd::tcgen05_fence_before();
        __syncwarp();
        if (lane == 0) afd::mbar_arrive(drained + 8 * b);
        ++unit;
      } else {
        // this warp's 16-column steps of the tile
        const int steps = max(0, (tile.cols() - 16 * h + 16 * kDrainParts - 1) / (16 * kDrainParts));
        if (steps == 4) ok = drain_blocks<GATED, 4>(p, sh, tile, mine, out, h, lane, unit);
        else if (steps == 3) ok = drain_blocks<GATED, 3>(p, sh, tile, mine, out, h, lane, unit);
        else if (steps == 2) ok = drain_blocks<GATED, 2>(p, sh, tile, mine, out, h, lane, unit);
        else if (steps == 1) ok = drain_blocks<GATED, 1>(p, sh, tile, mine, out, h, lane, unit);
        else ok = drain_blocks<GATED, 0>(p, sh, tile, mine, out, h, lane, unit);
      }
    }
  }
  // Neither CTA leaves while the other may signal it or read its operands.
  __syncthreads();
  if (*gave_up) {
    // Whichever role gave up: the pair's copies and products in flight finish
    // before shared memory and TMEM are freed (a millisecond; they take some us).
    const long long t0 = clock64();
    while (clock64() - t0 < 2000000) {
    }
    if (threadIdx.x == 0 && p.error) *p.error = AFD_ERR_TIMEOUT;
  }
  afd::tcgen05_fence_before();
  afd::cluster_sync_all();
  afd::tcgen05_fence_after();
  if (warp == 1) afd::tmem_free_pair(tmem, kColumns);
}

// ---------------------------------------------------------------------- host
std::atomic<int64_t> g_wait_cycles{afd::kWaitCycles};

using EncodeTiled = decltype(&cuTensorMapEncodeTiled);

// The driver's encoder, looked up once (a library without a driver loads).
EncodeTiled encoder() {
  static std::atomic<EncodeTiled> cached{nullptr};
  EncodeTiled f = cached.load(std::memory_order_acquire);
  if (f) return f;
  void* p = nullptr;
  cudaDriverEntryPointQueryResult q;
  if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &p, 12000, cudaEnableDefault, &q) != cudaSuccess ||
      q != cudaDriverEntryPointSuccess) {
    cudaGetLastError();
    return nullptr;
  }
  f = reinterpret_cast<EncodeTiled>(p);
  cached.store(f, std::memory_order_release);
  return f;
}

bool encode(EncodeTiled f, CUtensorMap* map, bool fp8, uint32_t rank, const void* base, const cuuint64_t* dims,
            const cuuint64_t* strides, const cuuint32_t* box) {
  const cuuint32_t ones[4] = {1, 1, 1, 1};
  return f(map, fp8 ? CU_TENSOR_MAP_DATA_TYPE_UINT8 : CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, rank, const_cast<void*>(base),
           dims, strides, box, ones, CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B,
           CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

template <bool FP8, bool GATED>
cudaError_t launch_grouped(const Maps& maps, const ExpertParams& p, int device, int pairs, cudaStream_t stream) {
  if (FP8) {
    // the registers that the hand-over gives out must be there at launch (asked
    // until there is an answer: a failed query says nothing about the next call)
    static std::atomic<bool> enough{false};
    if (!enough.load(std::memory_order_relaxed)) {
      cudaFuncAttributes a;
      const cudaError_t e = cudaFuncGetAttributes(&a, grouped_linear_kernel<FP8, GATED>);
      if (e != cudaSuccess) return e;
      if (a.numRegs * kThreads < kFrontRegs * 128 + kDrainRegs * 32 * kDrainWarps) return cudaErrorInvalidKernelImage;
      enough.store(true, std::memory_order_relaxed);
    }
  }
  static std::atomic<uint64_t> set{0};
  const cudaError_t e = afd::allow_shared(grouped_linear_kernel<FP8, GATED>, (int)kSmem, device, set);
  if (e != cudaSuccess) return e;
  return afd::launch_dependent(grouped_linear_kernel<FP8, GATED>, 2 * pairs, kThreads, kSmem, stream, maps, p);
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

extern "C" AFD_API afd_status afd_set_product_wait_limit(int64_t cycles) {
  if (cycles < 0) return AFD_ERR_ARG;
  g_wait_cycles.store(cycles, std::memory_order_relaxed);
  return AFD_OK;
}

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
  if (num_groups > afd::kMaxExperts || num_rows > afd::kMaxRows - expert_alignment || N > afd::kMaxFeatures ||
      K > afd::kMaxFeatures)
    return AFD_ERR_UNSUPPORTED;
  if (K * elt % 16 || x_stride * elt % 16 || (fp8 && (K % 128 || N % 128))) return AFD_ERR_UNSUPPORTED;
  // the most tiles there can be, counted in 32 bits by the kernel
  const int m_tiles = ((gated ? 2 * N : N) + kPairRows - 1) / kPairRows;
  const int64_t most = ((num_groups < num_rows ? num_groups : num_rows) + num_rows / kTileRows) * m_tiles;
  if (most > (1 << 30)) return AFD_ERR_UNSUPPORTED;
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
  EncodeTiled enc = encoder();
  int sms = 0;
  if (!enc || cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess) return AFD_ERR_CUDA;

  const int W = gated ? 2 * N : N, block = kBlockBytes / elt;
  Maps maps;
  const cuuint64_t k_bytes = (cuuint64_t)K * elt;
  bool ok;
  if (gated) {
    const cuuint64_t dims[4] = {(cuuint64_t)K, 2, (cuuint64_t)N, (cuuint64_t)num_groups};
    const cuuint64_t strides[3] = {k_bytes * N, k_bytes, k_bytes * W};
    const cuuint32_t box[4] = {(cuuint32_t)block, 2, kCtaRows / 2, 1};
    ok = encode(enc, &maps.w, fp8, 4, weight, dims, strides, box);
  } else {
    const cuuint64_t dims[3] = {(cuuint64_t)K, (cuuint64_t)N, (cuuint64_t)num_groups};
    const cuuint64_t strides[2] = {k_bytes, k_bytes * N};
    const cuuint32_t box[3] = {(cuuint32_t)block, kCtaRows, 1};
    ok = encode(enc, &maps.w, fp8, 3, weight, dims, strides, box);
  }
  for (int i = 0; ok && i < kRowMaps; ++i) {
    const cuuint64_t dims[2] = {(cuuint64_t)K, (cuuint64_t)num_rows};
    const cuuint64_t strides[1] = {(cuuint64_t)x_stride * elt};
    const cuuint32_t box[2] = {(cuuint32_t)block, 16u * (i + 1)};
    ok = encode(enc, &maps.x[i], fp8, 2, x, dims, strides, box);
  }
  if (!ok) return AFD_ERR_CUDA;

  ExpertParams p = {};
  p.x_scale = x_scale, p.w_scale = weight_scale, p.ends = ends;
  p.G = num_groups, p.alpha = expert_alignment, p.R = (int32_t)num_rows, p.K = K, p.N = N;
  p.m_tiles = m_tiles;
  p.k_blocks = (K + block - 1) / block;
  p.out = static_cast<uint16_t*>(out), p.out_stride = out_stride, p.error = error;
  p.wait_cycles = g_wait_cycles.load(std::memory_order_relaxed);
  p.vec = N % 2 == 0 && out_stride % 2 == 0 && afd::aligned_to(out, 4);
  const int pairs = (int)(most < sms / 2 ? most : sms / 2);  // no more than there can be tiles
  cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
  const cudaError_t e = fp8 ? (gated ? launch_grouped<true, true>(maps, p, dev, pairs, s) : launch_grouped<true, false>(maps, p, dev, pairs, s))
                            : (gated ? launch_grouped<false, true>(maps, p, dev, pairs, s) : launch_grouped<false, false>(maps, p, dev, pairs, s));
  return e == cudaSuccess ? AFD_OK : AFD_ERR_CUDA;
}
