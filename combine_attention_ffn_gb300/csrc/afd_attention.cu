// afd_decode_attention: one new token a sequence against its paged cache.
//
// The work is one pass over the live keys and values, at about 2 G flops a byte
// for G query heads a KV head: bound by DRAM, so everything here is about keeping
// loads in flight and every SM busy whatever the lengths are.
//
// Tiles and their order: the tokens of a sequence that are seen, 16, 32 or 64 at
// a time (4 KB of keys and as much of values), once for each KV head and each 8
// or 16 of its query heads; sequences, heads and tiles in that order make one
// line. A (sequence, heads) segment counts a tile or two more on it, for its
// queries and its result. The line is cut into equal shares, one a warp, so that
// no length leaves a warp idle; a share may begin or end inside a segment. Those
// parts are joined by the block after its warps are done, and what the blocks
// leave open by a second kernel.
//
// A warp works alone: its own ring of tiles in shared memory, filled by
// asynchronous copies ahead of their use, its own running maximum and sum. The
// products are m16n8k16 on tensor cores, transposed: 16 tokens by 8 query heads
// for the scores, 16 columns by 8 heads for the result, so that no row of a
// product is empty with up to eight heads; probabilities pass from one to the
// other through registers (one 8 x 8 transposition each). The rate of mma.sync is
// more than the traffic needs. The order of columns inside a product is free as
// long as both sides agree, so a lane takes 16 neighbouring bytes of a key at a
// time, and 16 of four tokens' values, whose pairs are then interleaved.
//
// Measured (us, a copy's time of the same bytes behind it): 128 sequences of up to 8,192
// tokens (64 query and 8 KV heads of 128, BF16, 1.36 GB) 207.7 (203.4); one of 131,072
// tokens 87.9 (80.1); 64 of up to 16,384 over E4M3, 16 heads a KV head, 71.8 (53.3); 250 of
// up to 1,000 (64 columns, pages of 16) 36.4 (24.5); 96 windows of 1,024 over E4M3, 64
// columns, 25.3 (13.0). Inside the loop that is 6.4 to 7.5 TB/s, as reads alone are faster than
// a copy. What is around it, in the same order: 4.6, 3.7, 4.6, 4.5 and 4.6 to the first
// tile; from the warps' mean end to the last one's 7.9, 4.5, 3.8, 3.2 and 2.3; the
// blocks' joins 4.1, 2.8, 5.9, 2.3 and 2.0; the second launch 2.6, 3.6, 3.9, 2.5 and 2.0.

#include <cuda_runtime.h>
#include <stdint.h>

#include "afd.h"
#include "afd_cache.cuh"
#include "afd_device.cuh"
#include "afd_pointers.cuh"
#include "afd_ragged.cuh"

namespace {

constexpr unsigned kFull = 0xffffffffu;
constexpr int kMaxBlocks = 160;
// Warps of a block, each with two stages of 8 KB. Three or four stages are slower:
// 128 sequences (BF16) 218 us with three, 209 with two; twelve warps take 212, six
// with three stages 217, seven with two 209.5, nine 205.5, ten 206.6 against 205.6
// for eight; 64 sequences (E4M3, 16 heads a KV head) 75, 93 and 86 against 70.8.
constexpr int kWarps = 8;
constexpr int kSoloBlocks = 148;  // no more than SMs
constexpr float kLazy = 8.f;  // log2 of how far a score may pass the running maximum before that moves
// Tiles a warp up to which a block takes a whole segment: where the lengths say so,
// and where full tables would (then in one launch). One sequence, 8 KV heads, us, a
// block for each segment against shares: BF16, 128 columns, 500 tokens 8.7 / 10.0, 800
// 10.7 / 10.1; E4M3, 1,000 10.1 / 11.9, 1,500 12.2 / 12.0; 64 columns, 1,000 8.4 / 9.4,
// 1,500 10.1 / 9.5. By the lengths, beside a second launch: 300 8.5 / 9.9, 500 10.3 / 10.0.
constexpr int kSolo = 4, kSoloFull = 6;
constexpr int kRun = 16;    // tokens that are in one page where its size is a multiple
constexpr float kLn2 = 0.693147180559945f;

// A split (sequence, head): where its last part is (see join).
struct __align__(16) Split {
  int32_t seg;   // sequence * chunks of heads + chunk, or -1
  int32_t last;  // the last block that has a part of it
  int32_t pad[2];
};

// A segment's parts in a block: the last one of warp w0 (-1: none), the first ones
// of the warps behind it before w1.
struct Chain {
  int32_t w0, w1, rows, whole;
  int64_t out, lse;  // its first row
};

struct AttentionParams {
  const uint16_t* q;
  int64_t q_stride;
  afd::CacheParams cache;
  const int32_t* table;
  int64_t table_stride;
  int32_t max_pages;
  const int32_t* lengths;
  int32_t B, Hq, Hkv, G, chunks;  // chunks: of at most 8 or 16 query heads, all KV heads'
  int32_t page_shift;             // log2 of the page size, or -1
  int32_t solo;                   // every segment has a block of its own, whatever the lengths are
  float scale_log2;
  int32_t window;
  uint16_t* out;
  int64_t out_stride;
  float* lse;
  Split* splits;  // workspace, [blocks]
  float* parts;   // workspace, [blocks][2][rows][D + 2]: O, then the maxima and the sums
  float* kept;    // workspace, [blocks * warps][rows][D]: O of warps' first parts
};

template <int D, bool FP8>
struct Shape {
  static constexpr int kRow = FP8 ? D : 2 * D;               // bytes of a token's head
  static constexpr int kTile = 4096 / kRow;                  // tokens
  static constexpr int kBytes = kTile * kRow;                // of a tile's keys, or values
  static constexpr int kScales = 2 * kBytes;                 // a stage's scales, {key, value} a token ...
  static constexpr int kBias = kScales + (FP8 ? 8 * kTile : 0);  // ... and what a score is lowered by
  static constexpr int kStage = kBias + 4 * kTile;
  static constexpr int E = FP8 && D == 128 ? 16 : 8;         // neighbouring columns of a lane
  static constexpr int H = D / 8 / E;                        // ... and how many such groups
  // What a segment counts beside its tiles, in tiles (1 at least: a step of more than one
  // is how a cursor tells of a new segment). With 1 and 2, us: E4M3, 128 columns, 64 unlike
  // sequences 74.4, 71.8 (16 heads a KV head) and 40.1, 40.1 (8), 250 short ones 41.5, 42.0;
  // E4M3, 64 columns, 96 windows 25.3, 25.5, 250 short ones 26.7, 28.0; BF16, 128 columns,
  // 128 sequences 207.9, 208.4, 64 62.7, 62.4, 250 short ones 62.6, 63.2; BF16, 64 columns,
  // 250 short ones 36.4, 37.2.
  static constexpr int kBegin = FP8 && D == 128 ? 2 : 1;
  static_assert(kBegin >= 1, "a new segment looks like the last one's next tile otherwise");
};

// NH: query heads of a chunk, in eights.
template <int D, bool FP8, int NH>
struct Layout {
  using S = Shape<D, FP8>;
  static constexpr int kRows = 8 * NH;
  static constexpr int kRing = 2 * S::kStage;  // one tile is taken while the next one comes
  static constexpr int kShared = kWarps * kRing;
  static_assert(kRing >= kRows * D * 4, "a part goes where the ring was");
};

__device__ __forceinline__ uint32_t smem_addr(const void* p) { return (uint32_t)__cvta_generic_to_shared(p); }

// 16 bytes, or zeros where `in` is false (nothing is read then).
__device__ __forceinline__ void copy16(uint32_t dst, const void* src, bool in) {
  asm volatile("cp.async.cg.shared.global.L2::128B [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(in ? 16 : 0) : "memory");
}
__device__ __forceinline__ void copy4(uint32_t dst, const void* src, bool in) {
  asm volatile("cp.async.ca.shared.global [%0], [%1], 4, %2;" ::"r"(dst), "l"(src), "r"(in ? 4 : 0) : "memory");
}
__device__ __forceinline__ void copies_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N>
__device__ __forceinline__ void copies_wait() { asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory"); }

template <bool F16>
__device__ __forceinline__ void mma(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, const uint32_t (&b)[2]) {
  if (F16)
    asm volatile("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, {%0, %1, %2, %3};"
                 : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
                 : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b[0]), "r"(b[1]));
  else
    asm volatile("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, {%0, %1, %2, %3};"
                 : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
                 : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b[0]), "r"(b[1]));
}

// Two E4M3 values (the low half of v, or the high one) as two FP16, exactly.
template <int HALF>
__device__ __forceinline__ uint32_t half2_of(uint32_t v) {
  uint32_t r;
  if (HALF == 0)
    asm("{\n.reg .b16 l, h;\nmov.b32 {l, h}, %1;\ncvt.rn.f16x2.e4m3x2 %0, l;\n}" : "=r"(r) : "r"(v));
  else
    asm("{\n.reg .b16 l, h;\nmov.b32 {l, h}, %1;\ncvt.rn.f16x2.e4m3x2 %0, h;\n}" : "=r"(r) : "r"(v));
  return r;
}

__device__ __forceinline__ uint32_t pack_f16(float lo, float hi) {
  uint32_t r;
  asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
  return r;
}

// Powers of two and their logarithms, accurate to 2^-22 (masked scores are
// -infinity: 0).
__device__ __forceinline__ float exp2_of(float v) {
  float r;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(v));
  return r;
}
__device__ __forceinline__ float log2_of(float v) {
  float r;
  asm("lg2.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(v));
  return r;
}

// A token's values weigh p * their scale, so E4M3 caches raise the running maximum
// by the scale's logarithm, within these bounds, and all weights by 2^kRaise: the largest
// of a warp's tokens is 2^7 (2^15 where the maximum lags, kLazy), and what FP16 loses is
// below 2^-32 of it. Without the raise tokens of 2^-25 were lost, and long tails of them
// counted in the sum alone. Scales from 2^-100 to 2^-93 have less: 2^-25.
// A sum of exponentials then ends up to 2^100 (with values of zero) or down to 2^-73
// where the largest score is: the tokens that leave FP32's range below that are 2^-53 of
// it each. Above 2^80 a weight passes FP16 and the result becomes infinite or NaN, as it
// does with an infinite scale; the scores' log-sum does not.
// A second FP16 part for each weight (as BF16 caches have) changes the results by less
// than their rounding to BF16 does: 64 sequences, 16 heads a KV head, 81.3 us against 71.8.
constexpr float kLiftLeast = -93.f, kLiftMost = 80.f;
template <bool FP8>
constexpr float kRaise = FP8 ? 7.f : 0.f;

// Two maxima may be raised unlike, so what a sum is weighted by where it moves from one
// to the other, 2^(m - most), may leave FP32's range where the weighted sum does not:
// E4M3 sums take the weight's root twice. Returns the root (E4M3), or the weight.
template <bool FP8>
__device__ __forceinline__ float weight_root(float m, float most) { return exp2_of(FP8 ? 0.5f * (m - most) : m - most); }
template <bool FP8>
__device__ __forceinline__ float weight_of(float root) { return FP8 ? root * root : root; }
template <bool FP8>
__device__ __forceinline__ float add_weighted(float l, float root, float sum) {
  return FP8 ? fmaf(l * root, root, sum) : fmaf(l, root, sum);
}

// The natural logarithm of sum * 2^most; the sum's own, good to 2^-22, by lg2.
__device__ __forceinline__ float log_sum(float most, float sum) { return (most + log2_of(sum)) * kLn2; }

// Over the eight lanes that hold other tokens of the same heads.
__device__ __forceinline__ float tokens_max(float v) {
#pragma unroll
  for (int d = 4; d <= 16; d <<= 1) v = fmaxf(v, __shfl_xor_sync(kFull, v, d));
  return v;
}
__device__ __forceinline__ float tokens_sum(float v) {
#pragma unroll
  for (int d = 4; d <= 16; d <<= 1) v += __shfl_xor_sync(kFull, v, d);
  return v;
}
__device__ __forceinline__ float quad_max(float v) {
  v = fmaxf(v, __shfl_xor_sync(kFull, v, 1));
  return fmaxf(v, __shfl_xor_sync(kFull, v, 2));
}

// An 8 x 8 matrix of 16-bit values, two of a row a lane, transposed.
__device__ __forceinline__ uint32_t transposed(uint32_t v) {
  uint32_t r;
  asm("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(r) : "r"(v));
  return r;
}

// Where 16-byte chunk `chunk` of a tile's row lies: eight lanes that read the
// same chunk of rows two apart, or two chunks apart of one row and its
// neighbour, meet all banks once.
template <int ROW>
__device__ __forceinline__ int swizzled(int row, int chunk) {
  if (ROW == 256) return row * 256 + ((chunk & 8) | ((chunk ^ row) & 7)) * 16;
  if (ROW == 128) return row * 128 + ((chunk ^ row) & 7) * 16;
  return row * 64 + ((chunk ^ (row >> 1)) & 3) * 16;
}

// Quotients of numbers that mostly have 32 bits (a division of 64 takes 200 ns).
__device__ __forceinline__ int64_t quotient(int64_t a, int64_t b) {
  if (((a | b) >> 32) == 0) return (uint32_t)a / (uint32_t)b;
  return a / b;
}

// The tiles [first, end) of a sequence that hold tokens [from, len).
struct Span {
  int from, len, first, end;
};

template <int TILE>
__device__ __forceinline__ Span span_of(const AttentionParams& p, int b) {
  Span s;
  const int64_t most = (int64_t)p.max_pages * p.cache.page_size;
  s.len = (int)min((int64_t)max(p.lengths[b], 0), most);
  s.from = p.window > 0 ? max(s.len - p.window, 0) : 0;
  s.first = s.from / TILE;
  s.end = s.len > 0 ? (s.len + TILE - 1) / TILE : s.first;
  return s;
}

// A place in the line; next() returns how far it went.
template <int TILE, int BEGIN>
struct Cursor {
  Span span;
  int b, chunk, tile;
  __device__ __forceinline__ int next(const AttentionParams& p) {
    if (++tile < span.end) return 1;
    if (++chunk == p.chunks) {
      chunk = 0;
      do {
        if (++b >= p.B) return 1 + BEGIN;  // (the end of the line)
        span = span_of<TILE>(p, b);
      } while (span.first == span.end);
    }
    tile = span.first;
    return 1 + BEGIN;
  }
};

// Where tokens are, in registers across a warp's lanes. Pages of a multiple of
// kRun tokens: run `first` + lane of the sequence; else the tokens of one tile.
template <int TILE>
struct Lookup {
  static constexpr int N = TILE > 32 ? TILE / 32 : 1;
  int page[N], at[N];  // -1: not seen
  int first;
  template <typename C>
  __device__ __forceinline__ void find(const AttentionParams& p, const C& c, int i, int token) {
    const uint32_t n = p.page_shift >= 0 ? (uint32_t)token >> p.page_shift : (uint32_t)token / (uint32_t)p.cache.page_size;
    at[i] = token - (int)(n * (uint32_t)p.cache.page_size);
    page[i] = p.table[c.b * p.table_stride + n];
  }
  // `fresh`: another sequence, or the sequence's first tile again.
  template <typename C>
  __device__ __forceinline__ void update(const AttentionParams& p, const C& c, bool runs, bool fresh, int lane) {
    if (runs) {
      const int run = c.tile * (TILE / kRun);
      if (!fresh && run + TILE / kRun <= first + 32) return;
      first = run;
      const int token = (run + lane) * kRun;
      page[0] = -1, at[0] = 0;
      if (token < c.span.len) find(p, c, 0, token);
    } else {
#pragma unroll
      for (int i = 0; i < N; ++i) {
        const int token = c.tile * TILE + ((32 * i + lane) & (TILE - 1));
        page[i] = -1, at[i] = 0;
        if (token >= c.span.from && token < c.span.len) find(p, c, i, token);
      }
    }
  }
};

template <int D, bool FP8, int NH>
__global__ void __launch_bounds__(kWarps * 32, 1) decode_attention_kernel(const AttentionParams p) {
  using S = Shape<D, FP8>;
  using Y = Layout<D, FP8, NH>;
  constexpr int TILE = S::kTile, ROW = S::kRow, E = S::E, H = S::H, TB = TILE / 16, W = kWarps, ROWS = Y::kRows;
  constexpr int THREADS = W * 32, kBegin = S::kBegin;
  extern __shared__ __align__(128) uint8_t shared[];
  __shared__ int64_t before[THREADS + 1];          // the line before each thread's sequences, of one chunk
  __shared__ float part_m[W][2][ROWS], part_l[W][2][ROWS];
  __shared__ int seg_a[W], seg_b[W], done_a[W], away_a[W];
  __shared__ int64_t end_b[W];
  __shared__ Chain chains[W + 1];
  __shared__ int chain_count;
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, g = lane >> 2, c = lane & 3;

  afd::pdl_wait();
  afd::pdl_launch_dependents();

  // ---- the line, and this warp's share of it
  const int each = (p.B + THREADS - 1) / THREADS;
  bool solo = p.solo;
  // (Up to 32 sequences every warp has them in its lanes and waits for no other:
  // 0.6 us less, and 0.2 more with more of them.)
  const bool few = p.B <= 32;
  int64_t mine = 0, sum = 0;
  if (!solo) {
    int longest = 0;
    const int b0 = few ? lane : threadIdx.x * each, b1 = min(p.B, b0 + (few ? 1 : each));
    for (int b = b0; b < b1; ++b) {
      const Span s = span_of<TILE>(p, b);
      mine += s.end > s.first ? s.end - s.first + kBegin : 0;
      longest = max(longest, s.end - s.first);
    }
    sum = mine;
#pragma unroll
    for (int d = 1; d < 32; d <<= 1) {
      const int64_t o = __shfl_up_sync(kFull, sum, d);
      if (lane >= d) sum += o;
    }
    // Short sequences, and a block for each: nothing is left for the second kernel.
    const bool short_all = longest <= kSolo * W && p.B * p.chunks <= gridDim.x;
    if (few) {
      solo = __all_sync(kFull, short_all);
    } else {
      if (lane == 31) end_b[warp] = sum;
      solo = __syncthreads_and(short_all);
      for (int w = 0; w < warp; ++w) sum += end_b[w];
      before[threadIdx.x + 1] = sum;
      if (threadIdx.x == 0) before[0] = 0;
      __syncthreads();
    }
  }
  Cursor<TILE, kBegin> at;
  int64_t lo = 0, each_share = 1;  // this warp's first place on the line, and those of a warp
  int share = 0, place = 0;        // places it has; where its next tile is behind the first
  if (solo) {
    const int seg = min((int)blockIdx.x, p.B * p.chunks - 1);
    at.b = seg / p.chunks, at.chunk = seg - at.b * p.chunks;
    at.span = span_of<TILE>(p, at.b);
    const int n = (int)blockIdx.x == seg ? at.span.end - at.span.first : 0, per = (n + W - 1) / W;
    const int first = min(per * warp, n);
    at.tile = at.span.first + first;
    share = min(per, n - first);
  } else {
    // Equal shares, but of few tiles the first blocks' warps take one each.
    const int64_t total = (few ? __shfl_sync(kFull, sum, 31) : before[THREADS]) * p.chunks;
    each_share = max(quotient(total + gridDim.x * W - 1, gridDim.x * W), (int64_t)(1 + kBegin));
    lo = min(each_share * (blockIdx.x * W + warp), total);
    share = (int)min(each_share, total - lo);
    if (share > 0) {
      int64_t left;
      if (few) {
        const int i = __popc(__ballot_sync(kFull, sum * p.chunks <= lo));
        left = lo - __shfl_sync(kFull, sum - mine, i) * p.chunks;
        at.b = i;
      } else {
        int i = 0;
#pragma unroll 1
        for (int step = 256; step; step >>= 1)
          if (i + step < THREADS && before[i + step] * p.chunks <= lo) i += step;
        left = lo - before[i] * p.chunks;
        at.b = i * each;
      }
      at.span = span_of<TILE>(p, at.b);
#pragma unroll 1
      for (;;) {
        const int64_t n = at.span.end > at.span.first ? (int64_t)(at.span.end - at.span.first + kBegin) * p.chunks : 0;
        if (left < n) break;
        left -= n;
        at.span = span_of<TILE>(p, ++at.b);
      }
      const int n = at.span.end - at.span.first + kBegin;
      at.chunk = (int)quotient(left, n);
      const int in = (int)(left - (int64_t)at.chunk * n);  // on the segment
      at.tile = at.span.first + max(in - kBegin, 0);
      place = max(kBegin - in, 0);
    }
  }

  const int groups = p.chunks / p.Hkv;  // chunks of a KV head
  uint8_t* ring = shared + warp * Y::kRing;
  float* kept = p.kept + (int64_t)(blockIdx.x * W + warp) * ROWS * D;
  if (lane == 0) seg_a[warp] = seg_b[warp] = -1, done_a[warp] = away_a[warp] = 0, end_b[warp] = 0;

  if (place < share) {
    const bool runs = p.cache.page_size % kRun == 0;

    // Places in a cache are counted in 64 bytes, which 32 bits hold.
    const uint8_t *k_lane = p.cache.k + lane * 16, *v_lane = p.cache.v + lane * 16;
    const uint32_t page_scales = (uint32_t)p.Hkv * (uint32_t)p.cache.page_size;
    // A lane's place in the j-th 512 bytes of a stage's keys, or values: the rows of
    // a step begin at a multiple of their number, so their swizzle is a constant.
    const uint32_t own = swizzled<ROW>(lane / (ROW / 16), lane % (ROW / 16));
    auto step_of = [&](int j) {
      return j * 512 + (own ^ (ROW == 256 ? (j & 3) * 32 : ROW == 128 ? (j & 1) * 64 : 0));
    };
    Cursor<TILE, kBegin> ahead = at;
    int ahead_place = place;
    Lookup<TILE> next;
    next.update(p, ahead, runs, true, lane);
    bool next_whole = true;  // every token of the tile staged last is seen
    // Starts the copies of the tile looked up last, and looks the one after it up.
    auto issue = [&](int stage) {
      if (ahead_place < share) {
        constexpr int CH = ROW / 16;  // chunks of a row
        uint8_t* to = ring + stage * S::kStage;
        const uint32_t dst = smem_addr(to);
        const int base = ahead.tile * TILE;
        const uint32_t head_row = (uint32_t)(groups == 1 ? ahead.chunk : ahead.chunk / groups) * (uint32_t)p.cache.page_size;
        const int lowest = ahead.span.from - base, end = ahead.span.len - base;  // rows that are seen
        next_whole = lowest <= 0 && end >= TILE;
        if (runs) {
          constexpr int JS = kRun * CH / 32;  // 512-byte steps of a run
          const int r0 = ahead.tile * (TILE / kRun) - next.first;
          const uint8_t *k[TILE / kRun], *v[TILE / kRun];
          bool ok[TILE / kRun];
#pragma unroll
          for (int r = 0; r < TILE / kRun; ++r) {
            const int page = __shfl_sync(kFull, next.page[0], r0 + r);
            const uint32_t row = (head_row + __shfl_sync(kFull, next.at[0], r0 + r)) * (ROW / 64);
            ok[r] = (uint32_t)page < (uint32_t)p.cache.pages;
            const uint32_t pg = ok[r] ? (uint32_t)page : 0u;
            k[r] = k_lane + (uint64_t)(pg * p.cache.k_page_units + row) * 64;
            v[r] = v_lane + (uint64_t)(pg * p.cache.v_page_units + row) * 64;
            next_whole &= ok[r];
          }
          if (next_whole) {
#pragma unroll
            for (int j = 0; j < S::kBytes / 512; ++j) {
              const uint32_t d = dst + step_of(j);
              copy16(d, k[j / JS] + j % JS * 512, true);
              copy16(d + S::kBytes, v[j / JS] + j % JS * 512, true);
            }
          } else {
#pragma unroll
            for (int j = 0; j < S::kBytes / 512; ++j) {
              const int row = (j * 32 + lane) / CH;
              const bool in = ok[j / JS] && row >= lowest && row < end;
              const uint32_t d = dst + step_of(j);
              copy16(d, in ? k[j / JS] + j % JS * 512 : p.cache.k, in);
              copy16(d + S::kBytes, in ? v[j / JS] + j % JS * 512 : p.cache.v, in);
            }
          }
          if (FP8 || !next_whole) {
#pragma unroll
            for (int i = 0; i < Lookup<TILE>::N; ++i) {
              const int tok = (32 * i + lane) & (TILE - 1);
              const int page = __shfl_sync(kFull, next.page[0], r0 + tok / kRun);
              const uint32_t row = head_row + __shfl_sync(kFull, next.at[0], r0 + tok / kRun) + tok % kRun;
              const bool in = next_whole || (tok >= lowest && tok < end && (uint32_t)page < (uint32_t)p.cache.pages);
              if (FP8) {
                const uint32_t o = in ? (uint32_t)page * page_scales + row : 0;
                copy4(dst + S::kScales + tok * 8, p.cache.k_scale + o, in);
                copy4(dst + S::kScales + tok * 8 + 4, p.cache.v_scale + o, in);
              }
              if (!next_whole) reinterpret_cast<float*>(to + S::kBias)[tok] = in ? 0.f : -INFINITY;
            }
          }
        } else {
#pragma unroll
          for (int i = 0; i < Lookup<TILE>::N; ++i) {
            const int tok = (32 * i + lane) & (TILE - 1);
            const bool in = (uint32_t)next.page[i] < (uint32_t)p.cache.pages;  // (-1: not seen)
            const uint32_t mask = __ballot_sync(kFull, in);
            next_whole &= mask == kFull;
            const uint32_t row = head_row + next.at[i];
            const uint32_t pg = in ? (uint32_t)next.page[i] : 0u;
            const uint32_t k_off = pg * p.cache.k_page_units + row * (ROW / 64), v_off = pg * p.cache.v_page_units + row * (ROW / 64);
            // (As a loop: 64 sequences of up to 4,096 tokens, pages of 1 80.7 us, of 24
            // 70.2; unrolled 71.2 and 65.5, where pages of 16 take 63.1.)
#pragma unroll
            for (int j = 0; j < (TILE < 32 ? TILE : 32) * CH / 32; ++j) {
              const int r = (j * 32 + lane) / CH, ch = (j * 32 + lane) % CH;
              const uint64_t ko = (uint64_t)__shfl_sync(kFull, k_off, r) * 64, vo = (uint64_t)__shfl_sync(kFull, v_off, r) * 64;
              const bool ok = (mask >> r) & 1u;
              const uint32_t d = dst + swizzled<ROW>(32 * i + r, ch);
              copy16(d, ok ? p.cache.k + ko + ch * 16 : p.cache.k, ok);
              copy16(d + S::kBytes, ok ? p.cache.v + vo + ch * 16 : p.cache.v, ok);
            }
            if (FP8) {
              const uint32_t o = in ? pg * page_scales + row : 0;
              copy4(dst + S::kScales + tok * 8, p.cache.k_scale + o, in);
              copy4(dst + S::kScales + tok * 8 + 4, p.cache.v_scale + o, in);
            }
            reinterpret_cast<float*>(to + S::kBias)[tok] = in ? 0.f : -INFINITY;
          }
        }
        const int went = ahead.next(p);
        ahead_place += went;
        if (ahead_place < share) next.update(p, ahead, runs, went > 1, lane);
      }
      copies_commit();
    };
    issue(0);

    uint32_t qb[NH][D / 16][2];
    float row_scale[NH][2];
    float o[D / 16][NH][4];
    float m[NH][2], l[NH][2];  // of heads 2 c and 2 c + 1, l this lane's tokens' part
    bool began = at.tile == at.span.first;  // the segment's first tile is this warp's

    // Query heads of the segment, zeros beyond the KV head's.
    auto load_q = [&]() {
      const int head = at.chunk / groups, sub = at.chunk % groups;
      const int rows = min(p.G - sub * ROWS, ROWS);
      const uint16_t* q = p.q + at.b * p.q_stride + (int64_t)(head * p.G + sub * ROWS) * D;
#pragma unroll
      for (int n = 0; n < NH; ++n) {
        uint4 v[D / 32];
#pragma unroll
        for (int i = 0; i < D / 32; ++i) {
          // chunk i of this lane, as the keys' (16 bytes of theirs are 8 or 16 columns)
          const int col = FP8 ? (D == 128 ? (2 * c + i / 2) * 16 + i % 2 * 8 : c * 16 + i * 8)
                              : (D == 128 ? (2 * c + (i & 1) + 8 * (i >> 1)) * 8 : (2 * c + i) * 8);
          v[i] = g + 8 * n < rows ? *reinterpret_cast<const uint4*>(q + (g + 8 * n) * D + col) : make_uint4(0, 0, 0, 0);
        }
        row_scale[n][0] = row_scale[n][1] = p.scale_log2;
        if (FP8) {
          // FP16 queries: the row's power of two taken out, so that the largest
          // lies in [1, 2) and the others keep their digits down to 2^-24 of it.
          float most = 0.f;
#pragma unroll
          for (int i = 0; i < D / 32; ++i) {
            float f[8];
            afd::bf16x8_to_float(v[i], f);
#pragma unroll
            for (int e = 0; e < 8; ++e) most = fmaxf(most, fabsf(f[e]));
          }
          most = quad_max(most);
          const int ex = min(max((int)(__float_as_uint(most) >> 23) - 127, -120), 120);
          const float down = __uint_as_float((uint32_t)(127 - ex) << 23);
          const float up = p.scale_log2 * __uint_as_float((uint32_t)(127 + ex) << 23);
          row_scale[n][0] = __shfl_sync(kFull, up, 8 * c);  // (a lane of head 2 c)
          row_scale[n][1] = __shfl_sync(kFull, up, 8 * c + 4);
#pragma unroll
          for (int i = 0; i < D / 32; ++i) {
            float f[8];
            afd::bf16x8_to_float(v[i], f);
            v[i] = make_uint4(pack_f16(f[0] * down, f[1] * down), pack_f16(f[2] * down, f[3] * down),
                              pack_f16(f[4] * down, f[5] * down), pack_f16(f[6] * down, f[7] * down));
          }
        }
#pragma unroll
        for (int i = 0; i < D / 32; ++i) {
          qb[n][2 * i][0] = v[i].x, qb[n][2 * i][1] = v[i].y;
          qb[n][2 * i + 1][0] = v[i].z, qb[n][2 * i + 1][1] = v[i].w;
        }
#pragma unroll
        for (int d = 0; d < D / 16; ++d) o[d][n][0] = o[d][n][1] = o[d][n][2] = o[d][n][3] = 0.f;
        m[n][0] = m[n][1] = -INFINITY;
        l[n][0] = l[n][1] = 0.f;
      }
    };

    bool fresh = true;
    int stage = 0;
#pragma unroll 1
    while (place < share) {  // (a share may hold a segment's beginning alone)
      const bool all = next_whole;
      copies_wait<0>();
      __syncwarp();
      issue(stage ^ 1);  // into the stage that the last tile has left
      if (fresh) load_q();
      fresh = false;
      const uint8_t* ks = ring + stage * S::kStage;
      const uint8_t* vs = ks + S::kBytes;

      // ---- scores: token 16 t + g (and + 8), heads 8 n + 2 c (and + 1)
      float s[TB][NH][4];
#pragma unroll
      for (int t = 0; t < TB; ++t)
#pragma unroll
        for (int n = 0; n < NH; ++n) s[t][n][0] = s[t][n][1] = s[t][n][2] = s[t][n][3] = 0.f;
#pragma unroll
      for (int ii = 0; ii < ROW / 64; ++ii) {
        const int chunk = ROW == 256 ? 2 * c + (ii & 1) + 8 * (ii >> 1) : ROW == 128 ? 2 * c + ii : c;
#pragma unroll
        for (int t = 0; t < TB; ++t) {
          const uint4 x = *reinterpret_cast<const uint4*>(ks + swizzled<ROW>(16 * t + g, chunk));
          const uint4 y = *reinterpret_cast<const uint4*>(ks + swizzled<ROW>(16 * t + 8 + g, chunk));
          const uint32_t xs[4] = {x.x, x.y, x.z, x.w}, ys[4] = {y.x, y.y, y.z, y.w};
          if (FP8) {
#pragma unroll
            for (int w = 0; w < 4; ++w) {
              const uint32_t a0 = half2_of<0>(xs[w]), a1 = half2_of<0>(ys[w]), a2 = half2_of<1>(xs[w]), a3 = half2_of<1>(ys[w]);
#pragma unroll
              for (int n = 0; n < NH; ++n) mma<true>(s[t][n], a0, a1, a2, a3, qb[n][(4 * ii + w) % (D / 16)]);
            }
          } else {
#pragma unroll
            for (int w = 0; w < 2; ++w)
#pragma unroll
              for (int n = 0; n < NH; ++n)
                mma<false>(s[t][n], xs[2 * w], ys[2 * w], xs[2 * w + 1], ys[2 * w + 1], qb[n][(2 * ii + w) % (D / 16)]);
          }
        }
      }
      // ---- softmax. E4M3: the weight of a token's values is p * its scale, so
      // the running maximum is that of s + log2(scale): the FP16 weights stay in
      // range, and what they lose is small beside the largest contribution. The
      // maximum moves, and what was summed is rescaled, only where a score is
      // kLazy above it; weights are then at most 2^(kLazy + kRaise).
      float top[NH][2], vscale[TB][2];
#pragma unroll
      for (int n = 0; n < NH; ++n) top[n][0] = top[n][1] = -INFINITY;
#pragma unroll
      for (int t = 0; t < TB; ++t)
#pragma unroll
        for (int y = 0; y < 2; ++y) {
          const int tok = 16 * t + 8 * y + g;
          float kscale = 1.f, lift = 0.f;
          if (FP8) {
            const float2 two = *reinterpret_cast<const float2*>(ks + S::kScales + tok * 8);
            kscale = two.x, vscale[t][y] = two.y;
            lift = fminf(fmaxf(log2_of(two.y), kLiftLeast), kLiftMost);
          }
          // (a token that is not seen has a key of zeros)
          const float bias = all ? 0.f : reinterpret_cast<const float*>(ks + S::kBias)[tok];
#pragma unroll
          for (int n = 0; n < NH; ++n)
#pragma unroll
            for (int x = 0; x < 2; ++x) {
              float& v = s[t][n][2 * y + x];
              v = fmaf(v, FP8 ? row_scale[n][x] * kscale : row_scale[n][x], bias);
              top[n][x] = fmaxf(top[n][x], v + lift);
            }
        }
      bool over = false;
#pragma unroll
      for (int n = 0; n < NH; ++n) over |= top[n][0] > m[n][0] + kLazy || top[n][1] > m[n][1] + kLazy;
      if (__any_sync(kFull, over)) {
#pragma unroll
        for (int n = 0; n < NH; ++n)
#pragma unroll
          for (int x = 0; x < 2; ++x) {
            const float to = fmaxf(tokens_max(top[n][x]), m[n][x]);
            const float root = m[n][x] == -INFINITY ? 0.f : weight_root<FP8>(m[n][x], to), f = weight_of<FP8>(root);
            m[n][x] = to;
            l[n][x] = FP8 ? l[n][x] * root * root : l[n][x] * f;
#pragma unroll
            for (int d = 0; d < D / 16; ++d) o[d][n][x] *= f, o[d][n][2 + x] *= f;
          }
      }
#pragma unroll
      for (int n = 0; n < NH; ++n)
#pragma unroll
        for (int x = 0; x < 2; ++x) {
          const float minus = (m[n][x] == -INFINITY ? 0.f : m[n][x]) - kRaise<FP8>;
#pragma unroll
          for (int t = 0; t < TB; ++t)
#pragma unroll
            for (int y = 0; y < 2; ++y) {
              float& v = s[t][n][2 * y + x];
              v = exp2_of(v - minus);
              l[n][x] += v;
              if (FP8) v *= vscale[t][y];
            }
        }
      // ---- values: columns (8 h + g) E + e of heads 8 n + 2 c (and + 1)
#pragma unroll
      for (int t = 0; t < TB; ++t) {
        uint32_t pa[NH][2], pb[NH][2];  // probabilities, and (BF16) what their rounding left
#pragma unroll
        for (int n = 0; n < NH; ++n)
#pragma unroll
          for (int y = 0; y < 2; ++y) {
            const float a = s[t][n][2 * y], b = s[t][n][2 * y + 1];
            if (FP8) {
              pa[n][y] = transposed(pack_f16(a, b));
            } else {
              const uint32_t high = afd::pack_bf16(a, b);
              pa[n][y] = transposed(high);
              pb[n][y] = transposed(afd::pack_bf16(a - __uint_as_float(high << 16), b - __uint_as_float(high & 0xffff0000u)));
            }
          }
#pragma unroll
        for (int h = 0; h < H; ++h) {
          uint32_t v[4][4];
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            const int row = 16 * t + 2 * c + (i & 1) + 8 * (i >> 1);
            if constexpr (ROW == 64) {
              const uint2 u = *reinterpret_cast<const uint2*>(vs + swizzled<ROW>(row, g >> 1) + (g & 1) * 8);
              v[i][0] = u.x, v[i][1] = u.y;
            } else {
              const uint4 u = *reinterpret_cast<const uint4*>(vs + swizzled<ROW>(row, 8 * h + g));
              v[i][0] = u.x, v[i][1] = u.y, v[i][2] = u.z, v[i][3] = u.w;
            }
          }
          if constexpr (FP8) {
#pragma unroll
            for (int w = 0; w < E / 4; ++w) {
              const uint32_t x0 = __byte_perm(v[0][w], v[1][w], 0x5140), x1 = __byte_perm(v[2][w], v[3][w], 0x5140);
              const uint32_t y0 = __byte_perm(v[0][w], v[1][w], 0x7362), y1 = __byte_perm(v[2][w], v[3][w], 0x7362);
#pragma unroll
              for (int n = 0; n < NH; ++n) {
                mma<true>(o[2 * w][n], half2_of<0>(x0), half2_of<1>(x0), half2_of<0>(x1), half2_of<1>(x1), pa[n]);
                mma<true>(o[2 * w + 1][n], half2_of<0>(y0), half2_of<1>(y0), half2_of<0>(y1), half2_of<1>(y1), pa[n]);
              }
            }
          } else {
#pragma unroll
            for (int w = 0; w < 4; ++w) {
              const uint32_t a0 = __byte_perm(v[0][w], v[1][w], 0x5410), a1 = __byte_perm(v[0][w], v[1][w], 0x7632);
              const uint32_t a2 = __byte_perm(v[2][w], v[3][w], 0x5410), a3 = __byte_perm(v[2][w], v[3][w], 0x7632);
#pragma unroll
              for (int n = 0; n < NH; ++n) {
                mma<false>(o[4 * h + w][n], a0, a1, a2, a3, pa[n]);
                mma<false>(o[4 * h + w][n], a0, a1, a2, a3, pb[n]);
              }
            }
          }
        }
      }

      stage ^= 1;
      // ---- the end of a segment, or of the share
      const bool ends = at.tile + 1 == at.span.end;
      const bool last = place + (ends ? 1 + kBegin : 1) >= share;
      if (ends || last) {
#pragma unroll
        for (int n = 0; n < NH; ++n) l[n][0] = tokens_sum(l[n][0]), l[n][1] = tokens_sum(l[n][1]);
        const int seg = at.b * p.chunks + at.chunk;
        if (began && ends) {
          const int head = at.chunk / groups, sub = at.chunk % groups;
          const int rows = min(p.G - sub * ROWS, ROWS), q0 = head * p.G + sub * ROWS;
#pragma unroll
          for (int n = 0; n < NH; ++n)
#pragma unroll
            for (int x = 0; x < 2; ++x) {
              const int row = 8 * n + 2 * c + x;
              if (row >= rows) continue;
              const float inv = l[n][x] == 0.f ? 0.f : 1.f / l[n][x];
              uint16_t* out = p.out + at.b * p.out_stride + (int64_t)(q0 + row) * D;
#pragma unroll
              for (int h = 0; h < H; ++h)
#pragma unroll
                for (int e = 0; e < E; e += 8) {
                  float f[8];
#pragma unroll
                  for (int k = 0; k < 8; ++k) f[k] = o[(h * E + e + k) / 2][n][2 * (k & 1) + x] * inv;
                  *reinterpret_cast<uint4*>(out + (8 * h + g) * E + e) = afd::float_to_bf16x8(f);
                }
              if (p.lse && g == 0)
                p.lse[(int64_t)at.b * p.Hq + q0 + row] = l[n][x] == 0.f ? -INFINITY : log_sum(m[n][x] - kRaise<FP8>, l[n][x]);
            }
        } else {
          // Left open. What began in an earlier warp's share goes to the warp's own
          // place if more follows; the share's last goes where the ring was.
          const int which = began ? 1 : 0;
          float* to = kept;
          if (last) {
            copies_wait<0>();
            __syncwarp();
            to = reinterpret_cast<float*>(ring);
          }
#pragma unroll
          for (int n = 0; n < NH; ++n)
#pragma unroll
            for (int x = 0; x < 2; ++x) {
              const int row = 8 * n + 2 * c + x;
#pragma unroll
              for (int h = 0; h < H; ++h)
#pragma unroll
                for (int e = 0; e < E; e += 4) {
                  const int d = (h * E + e) / 2;
                  *reinterpret_cast<float4*>(to + row * D + (8 * h + g) * E + e) =
                      make_float4(o[d][n][x], o[d][n][2 + x], o[d + 1][n][x], o[d + 1][n][2 + x]);
                }
              if (g == 0) part_m[warp][which][row] = m[n][x] - kRaise<FP8>, part_l[warp][which][row] = l[n][x];
            }
          if (lane == 0) {
            if (which) seg_b[warp] = seg, end_b[warp] = lo + place + (at.span.end - at.tile);
            else seg_a[warp] = seg, done_a[warp] = ends, away_a[warp] = !last;
          }
        }
        began = true;
        fresh = true;
      }
      if (last) break;
      place += at.next(p);
    }
    copies_wait<0>();
  }
  // Sequences that see nothing.
  for (int b = blockIdx.x; b < p.B; b += gridDim.x) {
    const Span s = span_of<TILE>(p, b);
    if (s.first != s.end) continue;
    for (int i = threadIdx.x; i < p.Hq * (D / 8); i += THREADS)
      *reinterpret_cast<uint4*>(p.out + b * p.out_stride + i * 8) = make_uint4(0, 0, 0, 0);
    if (p.lse)
      for (int i = threadIdx.x; i < p.Hq; i += THREADS) p.lse[(int64_t)b * p.Hq + i] = -INFINITY;
  }
  __syncthreads();

  // ---- the block's open parts: a chain begins with the first warp's part of an
  // earlier block's segment, or with a warp's last one, and goes on through the
  // next warps' first ones. All chains' rows are joined side by side.
  if (warp == 0) {
    const int w0 = lane - 1;
    const int seg = lane > W ? -1 : w0 < 0 ? seg_a[0] : seg_b[w0];
    int w1 = w0 + 1;
    bool done = false;
    if (seg >= 0)
      while (w1 < W && seg_a[w1] == seg) done |= done_a[w1] != 0, ++w1;
    const bool open = seg >= 0 && w0 >= 0 && !done;
    const unsigned found = __ballot_sync(kFull, seg >= 0), opens = __ballot_sync(kFull, open);
    if (seg >= 0) {
      const int b = seg / p.chunks, chunk = seg - b * p.chunks, head = chunk / groups, sub = chunk - head * groups;
      Chain c;
      c.w0 = w0, c.w1 = w1, c.rows = min(p.G - sub * ROWS, ROWS), c.whole = w0 >= 0 && done;
      const int q = head * p.G + sub * ROWS;
      c.out = b * p.out_stride + (int64_t)q * D;
      c.lse = (int64_t)b * p.Hq + q;
      chains[__popc(found & ((1u << lane) - 1))] = c;
    }
    // (the one segment that goes on behind the block, if there is one)
    if (p.splits && (open || (lane == 0 && !opens)))
      p.splits[blockIdx.x] = {open ? seg : -1, open ? (int)(quotient(end_b[w0] - 1, each_share) / W) : 0, {0, 0}};
    if (lane == 0) chain_count = __popc(found);
  }
  __syncthreads();
  // Eight columns of a row a thread. (Code that runs once is fetched from L2 as it
  // runs: it is kept short.)
  constexpr int ITEMS = ROWS * (D / 8);  // of a chain
#pragma unroll 1
  for (int i = threadIdx.x; i < chain_count * ITEMS; i += THREADS) {
    const Chain& c = chains[i / ITEMS];
    const int row = i % ITEMS / (D / 8), col = i % (D / 8) * 8;
    if (row >= c.rows) continue;
    float most = -INFINITY, sum = 0.f, f[8] = {};
#pragma unroll 1
    for (int w = max(c.w0, 0); w < c.w1; ++w) most = fmaxf(most, part_m[w][w == c.w0][row]);
    const float minus = most == -INFINITY ? 0.f : most;
#pragma unroll 1
    for (int w = max(c.w0, 0); w < c.w1; ++w) {
      const int which = w == c.w0;
      const float root = weight_root<FP8>(part_m[w][which][row], minus), scale = weight_of<FP8>(root);
      const float* from = (which || !away_a[w] ? reinterpret_cast<const float*>(shared + w * Y::kRing)
                                               : p.kept + (int64_t)(blockIdx.x * W + w) * ROWS * D) + row * D + col;
      const float4 x = *reinterpret_cast<const float4*>(from), y = *reinterpret_cast<const float4*>(from + 4);
      sum = add_weighted<FP8>(part_l[w][which][row], root, sum);
      f[0] = fmaf(x.x, scale, f[0]), f[1] = fmaf(x.y, scale, f[1]), f[2] = fmaf(x.z, scale, f[2]), f[3] = fmaf(x.w, scale, f[3]);
      f[4] = fmaf(y.x, scale, f[4]), f[5] = fmaf(y.y, scale, f[5]), f[6] = fmaf(y.z, scale, f[6]), f[7] = fmaf(y.w, scale, f[7]);
    }
    if (c.whole) {
      const float inv = sum == 0.f ? 0.f : 1.f / sum;
#pragma unroll
      for (int k = 0; k < 8; ++k) f[k] *= inv;
      *reinterpret_cast<uint4*>(p.out + c.out + row * D + col) = afd::float_to_bf16x8(f);
      if (p.lse && col == 0) p.lse[c.lse + row] = sum == 0.f ? -INFINITY : log_sum(most, sum);
    } else {
      float* part = p.parts + ((int64_t)blockIdx.x * 2 + (c.w0 >= 0)) * ROWS * (D + 2);
      *reinterpret_cast<float4*>(part + row * D + col) = make_float4(f[0], f[1], f[2], f[3]);
      *reinterpret_cast<float4*>(part + row * D + col + 4) = make_float4(f[4], f[5], f[6], f[7]);
      if (col == 0) part[ROWS * D + row] = most, part[ROWS * (D + 1) + row] = sum;
    }
  }
}

// Joins what the blocks left open: a warp per row of a segment that began in
// block `from`; its parts are that block's second and the next ones' first.
template <int D, bool FP8, int NH>
__global__ void __launch_bounds__(256) decode_join_kernel(const AttentionParams p) {
  afd::pdl_wait();
  afd::pdl_launch_dependents();
  constexpr int ROWS = 8 * NH;
  const int lane = threadIdx.x & 31;
  const int item = blockIdx.x * 8 + (threadIdx.x >> 5), from = item / ROWS, row = item % ROWS;
  const Split split = p.splits[from];
  if (split.seg < 0) return;
  const int b = split.seg / p.chunks, chunk = split.seg % p.chunks, groups = p.chunks / p.Hkv;
  const int head = chunk / groups, sub = chunk % groups;
  if (row >= min(p.G - sub * ROWS, ROWS)) return;
  constexpr int64_t kPart = ROWS * (D + 2);
  auto part = [&](int i) { return p.parts + ((int64_t)i * 2 + (i == from)) * kPart; };
  // 32 parts at a time, their maxima and sums one a lane; kAhead of them in flight.
  constexpr int N = D / 32, kAhead = 8;
  float most = -INFINITY, sum = 0.f, f[N] = {};
  for (int i0 = from; i0 <= split.last; i0 += 32) {
    const int n = min(split.last + 1 - i0, 32);
    float v[kAhead][N];
    auto fetch = [&](int j) {
#pragma unroll
      for (int u = 0; u < kAhead; ++u) {
        const float* q = part(i0 + min(j + u, n - 1)) + row * D + lane * N;
        if constexpr (N == 4) {
          const float4 x = *reinterpret_cast<const float4*>(q);
          v[u][0] = x.x, v[u][1] = x.y, v[u][2] = x.z, v[u][3] = x.w;
        } else {
          const float2 x = *reinterpret_cast<const float2*>(q);
          v[u][0] = x.x, v[u][1] = x.y;
        }
      }
    };
    const float* mine = part(i0 + min(lane, n - 1));
    const float m = lane < n ? mine[ROWS * D + row] : -INFINITY, l = lane < n ? mine[ROWS * (D + 1) + row] : 0.f;
    fetch(0);
    float top = fmaxf(m, most);
#pragma unroll
    for (int d = 16; d; d >>= 1) top = fmaxf(top, __shfl_xor_sync(kFull, top, d));
    const float minus = top == -INFINITY ? 0.f : top;
    const float before_root = weight_root<FP8>(most, minus), before = weight_of<FP8>(before_root);
    const float root = weight_root<FP8>(m, minus), weight = weight_of<FP8>(root);
    most = top;
    sum = add_weighted<FP8>(sum, before_root, FP8 ? l * root * root : l * weight);  // (each lane's own parts)
#pragma unroll
    for (int k = 0; k < N; ++k) f[k] *= before;
    for (int j = 0;;) {
#pragma unroll
      for (int u = 0; u < kAhead; ++u) {
        const float w = __shfl_sync(kFull, weight, min(j + u, 31));
        if (j + u < n)
#pragma unroll
          for (int k = 0; k < N; ++k) f[k] = fmaf(v[u][k], w, f[k]);
      }
      j += kAhead;
      if (j >= n) break;
      fetch(j);
    }
  }
#pragma unroll
  for (int d = 16; d; d >>= 1) sum += __shfl_xor_sync(kFull, sum, d);
  const float inv = sum == 0.f ? 0.f : 1.f / sum;
  const int q = head * p.G + sub * ROWS + row;
  uint32_t* out = reinterpret_cast<uint32_t*>(p.out + b * p.out_stride + (int64_t)q * D + lane * N);
#pragma unroll
  for (int k = 0; k < N; k += 2) out[k / 2] = afd::pack_bf16(f[k] * inv, f[k + 1] * inv);
  if (p.lse && lane == 0) p.lse[(int64_t)b * p.Hq + q] = sum == 0.f ? -INFINITY : log_sum(most, sum);
}

int tile_tokens(int head_dim, bool fp8) { return 4096 / (head_dim * (fp8 ? 1 : 2)); }
int smallest_tile(int head_dim) { return tile_tokens(head_dim, false); }

int chunk_rows(int group) { return group > 8 ? 16 : 8; }

int64_t parts_of(int head_dim, int rows) { return kMaxBlocks * (int64_t)2 * rows * (head_dim + 2); }
int64_t workspace_of(int head_dim, int rows) {
  return kMaxBlocks * (int64_t)sizeof(Split) +
         (parts_of(head_dim, rows) + kMaxBlocks * (int64_t)kWarps * rows * head_dim) * (int64_t)sizeof(float);
}

int64_t segments(int64_t seqs, int64_t q_heads, int64_t kv_heads) {
  const int64_t group = q_heads / kv_heads, rows = chunk_rows((int)group);
  return seqs * kv_heads * ((group + rows - 1) / rows);
}

// Whether a block for each segment does even where all tables are full.
bool is_solo(int64_t segments, int64_t tokens, int tile) {
  return segments <= kSoloBlocks && tokens <= (int64_t)kSoloFull * kWarps * tile;
}

template <int D, bool FP8, int NH>
cudaError_t launch_attention(const AttentionParams& p, int64_t tiles, int device, int sms, cudaStream_t stream) {
  using Y = Layout<D, FP8, NH>;
  static std::atomic<uint64_t> done{0};
  cudaError_t e = afd::allow_shared(decode_attention_kernel<D, FP8, NH>, Y::kShared, device, done);
  if (e != cudaSuccess) return e;
  const int64_t most = sms < kMaxBlocks ? sms : kMaxBlocks, want = p.solo ? p.B * p.chunks : tiles;
  const int blocks = (int)(tiles == 0 || (want > most && !p.solo) ? most : want);
  e = afd::launch_dependent(decode_attention_kernel<D, FP8, NH>, blocks, kWarps * 32, Y::kShared, stream, p);
  if (e != cudaSuccess || p.solo) return e;
  return afd::launch_dependent(decode_join_kernel<D, FP8, NH>, blocks * NH, 256, 0, stream, p);
}

template <int D>
cudaError_t launch_of(const AttentionParams& p, bool fp8, int64_t tiles, int device, int sms, cudaStream_t stream) {
  if (p.G > 8)
    return fp8 ? launch_attention<D, true, 2>(p, tiles, device, sms, stream)
               : launch_attention<D, false, 2>(p, tiles, device, sms, stream);
  return fp8 ? launch_attention<D, true, 1>(p, tiles, device, sms, stream)
             : launch_attention<D, false, 1>(p, tiles, device, sms, stream);
}

constexpr int64_t kMaxTokens = INT32_MAX - 1024;  // of a table's row
// Places on the line that the tables allow (tiles of 16 tokens, the beginnings): a warp
// counts its own in 32 bits, and there are more than 1,024 warps.
constexpr int64_t kMaxPlaces = (int64_t)1 << 41;

}  // namespace

extern "C" {

AFD_API int64_t afd_decode_workspace_bytes(int32_t num_seqs, int32_t num_q_heads, int32_t num_kv_heads, int32_t head_dim,
                                           int32_t max_pages, int32_t page_size) {
  if (num_seqs < 0 || num_kv_heads < 1 || num_q_heads < 1 || num_q_heads % num_kv_heads || max_pages < 0 || page_size < 1 ||
      (head_dim != 64 && head_dim != 128))
    return -1;
  const int64_t tokens = (int64_t)max_pages * page_size;
  if (tokens == 0 || is_solo(segments(num_seqs, num_q_heads, num_kv_heads), tokens, smallest_tile(head_dim))) return 0;
  return workspace_of(head_dim, chunk_rows(num_q_heads / num_kv_heads));
}

AFD_API afd_status afd_decode_attention(const void* q, int64_t q_stride, const afd_cache* cache,
                                        const int32_t* page_table, int64_t table_stride, int32_t max_pages,
                                        const int32_t* lengths, int32_t num_seqs, int32_t num_q_heads, float scale,
                                        int32_t window, void* out, int64_t out_stride, float* lse,
                                        void* workspace, int64_t workspace_bytes, afd_stream stream) {
  if (num_seqs < 0 || num_q_heads < 1 || max_pages < 0 || window < 0) return AFD_ERR_ARG;
  const afd_status checked = afd::check_cache(cache);
  if (checked != AFD_OK) return checked;
  const int D = cache->head_dim, Hkv = cache->num_kv_heads;
  const int64_t width = (int64_t)num_q_heads * D;
  if (num_q_heads % Hkv || (num_seqs > 1 && (q_stride < width || out_stride < width || table_stride < max_pages))) return AFD_ERR_ARG;
  const int64_t tokens = (int64_t)max_pages * cache->page_size;
  const int rows = chunk_rows(num_q_heads / Hkv), groups = (num_q_heads / Hkv + rows - 1) / rows;
  if (num_q_heads > afd::kMaxHeads || tokens > kMaxTokens || (int64_t)num_seqs * Hkv * groups > afd::kMaxRows ||
      q_stride % 8 || out_stride % 8)
    return AFD_ERR_UNSUPPORTED;
  if (segments(num_seqs, num_q_heads, Hkv) * (tokens / 16 + 3) > kMaxPlaces) return AFD_ERR_UNSUPPORTED;
  if (num_seqs == 0) return AFD_OK;
  if (!q || !out || !lengths || (max_pages > 0 && !page_table)) return AFD_ERR_ARG;
  const int64_t need = afd_decode_workspace_bytes(num_seqs, num_q_heads, Hkv, D, max_pages, cache->page_size);
  if (need < 0 || (need > 0 && (!workspace || workspace_bytes < need))) return AFD_ERR_ARG;
  if (!afd::aligned_to(page_table, 4) || !afd::aligned_to(lengths, 4) || !afd::aligned_to(lse, 4) ||
      (need > 0 && !afd::aligned_to(workspace, 16)))
    return AFD_ERR_ARG;
  if (!afd::aligned_to(q, 16) || !afd::aligned_to(out, 16)) return AFD_ERR_UNSUPPORTED;
  AttentionParams p = {};
  if (!afd::device_view(static_cast<const uint16_t*>(q), &p.q) || !afd::view_cache(cache, &p.cache) ||
      (max_pages > 0 && !afd::device_view(page_table, &p.table)) || !afd::device_view(lengths, &p.lengths) ||
      !afd::device_view(static_cast<uint16_t*>(out), &p.out) || (lse && !afd::device_view(lse, &p.lse)) ||
      (need > 0 && !afd::device_view(static_cast<Split*>(workspace), &p.splits)))
    return AFD_ERR_ARG;
  p.q_stride = q_stride, p.table_stride = table_stride, p.max_pages = max_pages, p.out_stride = out_stride;
  p.B = num_seqs, p.Hq = num_q_heads, p.Hkv = Hkv, p.G = num_q_heads / Hkv, p.chunks = Hkv * groups;
  p.scale_log2 = scale * 1.4426950408889634f, p.window = window;
  if (need > 0) p.parts = reinterpret_cast<float*>(p.splits + kMaxBlocks), p.kept = p.parts + parts_of(D, rows);
  p.page_shift = -1;
  for (int i = 0; i < 31; ++i)
    if (cache->page_size == 1 << i) p.page_shift = i;
  int dev = -1, sms = 0;
  if (cudaGetDevice(&dev) != cudaSuccess || cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess)
    return AFD_ERR_CUDA;
  const bool fp8 = cache->dtype == AFD_FP8_E4M3;
  // (of the two types' tiles the smaller decides, as for the workspace)
  p.solo = need == 0;
  const int64_t tiles = (tokens + tile_tokens(D, fp8) - 1) / tile_tokens(D, fp8) * num_seqs * p.chunks;
  cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
  const cudaError_t e = D == 64 ? launch_of<64>(p, fp8, tiles, dev, sms, s) : launch_of<128>(p, fp8, tiles, dev, sms, s);
  return e == cudaSuccess ? AFD_OK : AFD_ERR_CUDA;
}

}  // extern "C"
