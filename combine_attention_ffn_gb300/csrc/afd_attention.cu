// afd_decode_attention: one new token a sequence against its paged cache.
//
// The work is one pass over the live keys and values, at about 2 G flops a byte
// for G query heads a KV head: bound by DRAM, so everything here is about keeping
// loads in flight and every SM busy whatever the lengths are.
//
// Tiles and their order: the tokens of a sequence that are seen, 16 or 32 at a
// time (4 KB of keys and as much of values), once for each KV head and each 16
// of its query heads; sequences, heads and tiles in that order make one line of
// tiles. The line is cut into equal shares, one a warp, so that no length leaves
// a warp idle; a share may begin or end inside a (sequence, head). Those parts
// are joined by the block after its warps are done, and what the blocks leave
// open by a second kernel.
//
// A warp works alone: its own ring of tiles in shared memory, filled by
// asynchronous copies a few tiles ahead, its own running maximum and sum. The
// products are m16n8k16 on tensor cores with the query heads as the 16 rows;
// the rate of mma.sync is far more than the traffic needs, and its register
// operands let the probabilities go from one product to the next in place. The
// order of columns inside a product is free as long as both sides agree, so a
// lane takes 16 neighbouring bytes of a key at a time, and 16 of four tokens'
// values, whose pairs are then interleaved in registers.

#include <cuda_runtime.h>
#include <stdint.h>

#include "afd.h"
#include "afd_cache.cuh"
#include "afd_device.cuh"
#include "afd_pointers.cuh"
#include "afd_ragged.cuh"

namespace {

constexpr unsigned kFull = 0xffffffffu;
constexpr int kRows = 16;       // query heads of a product
constexpr int kMaxBlocks = 256;
constexpr float kLn2 = 0.693147180559945f;

// A split (sequence, head): where its last part is (see join).
struct __align__(16) Split {
  int32_t seg;   // sequence * chunks of heads + chunk, or -1
  int32_t last;  // the last block that has a part of it
  int32_t pad[2];
};

struct AttentionParams {
  const uint16_t* q;
  int64_t q_stride;
  afd::CacheParams cache;
  const int32_t* table;
  int64_t table_stride;
  int32_t max_pages;
  const int32_t* lengths;
  int32_t B, Hq, Hkv, G, chunks;  // chunks: of at most 16 query heads, all KV heads'
  float scale_log2;
  int32_t window;
  uint16_t* out;
  int64_t out_stride;
  float* lse;
  Split* splits;  // workspace, [blocks]
  float* parts;   // workspace, [blocks][2][kRows][D + 2]: O, then the maxima and the sums
};

template <int D, bool FP8>
struct Shape {
  static constexpr int kRow = FP8 ? D : 2 * D;               // bytes of a token's head
  static constexpr int kTile = kRow == 256 ? 16 : 32;        // tokens
  static constexpr int kBytes = kTile * kRow;                // of a tile's keys, or values
  static constexpr int kStage = 2 * kBytes + (FP8 ? 2 * kTile * 4 : 0);
  static constexpr int E = FP8 && D == 128 ? 16 : 8;         // neighbouring columns of a lane
  static constexpr int H = D / 8 / E;                        // ... and how many such groups
};

// Warps of a block and stages of a warp's ring; HI: more than eight query heads.
template <int D, bool FP8, bool HI>
struct Layout {
  using S = Shape<D, FP8>;
  static constexpr int kWarps = 6;
  static constexpr int kPart = (HI ? 16 : 8) * D * 4;
  static constexpr int kStages = (216 * 1024 / kWarps - kPart) / S::kStage < 4 ? (216 * 1024 / kWarps - kPart) / S::kStage : 4;
  static constexpr int kRing = kStages * S::kStage;
  static constexpr int kShared = kWarps * (kRing + kPart);
  static_assert(kStages >= 2 && kRing >= kPart, "a part goes where the ring was");
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
__device__ __forceinline__ void mma(float (&d)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
  if (F16)
    asm volatile("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, {%0, %1, %2, %3};"
                 : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
                 : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
  else
    asm volatile("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, {%0, %1, %2, %3};"
                 : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
                 : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
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

__device__ __forceinline__ float quad_max(float v) {
  v = fmaxf(v, __shfl_xor_sync(kFull, v, 1));
  return fmaxf(v, __shfl_xor_sync(kFull, v, 2));
}
__device__ __forceinline__ float quad_sum(float v) {
  v += __shfl_xor_sync(kFull, v, 1);
  return v + __shfl_xor_sync(kFull, v, 2);
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

// A place in the line of tiles.
template <int TILE>
struct Cursor {
  Span span;
  int b, chunk, tile;
  __device__ __forceinline__ void next(const AttentionParams& p) {
    if (++tile < span.end) return;
    if (++chunk == p.chunks) {
      chunk = 0;
      do {
        if (++b >= p.B) return;  // (the end of the line)
        span = span_of<TILE>(p, b);
      } while (span.first == span.end);
    }
    tile = span.first;
  }
};

// What a lane looks up for a tile: its token's page and place there.
struct Lookup {
  int page, at, chunk;
  bool in;
};

template <int TILE>
__device__ __forceinline__ Lookup look_up(const AttentionParams& p, const Cursor<TILE>& c, int lane) {
  Lookup l;
  const int token = c.tile * TILE + lane;
  l.in = lane < TILE && token >= c.span.from && token < c.span.len;
  l.chunk = c.chunk;
  l.page = 0;
  l.at = 0;
  if (l.in) {
    const uint32_t page = (uint32_t)token / (uint32_t)p.cache.page_size;
    l.at = token - (int)(page * (uint32_t)p.cache.page_size);
    l.page = p.table[c.b * p.table_stride + page];
  }
  return l;
}

template <int D, bool FP8, bool HI>
__global__ void __launch_bounds__(Layout<D, FP8, HI>::kWarps * 32, 1) decode_attention_kernel(const AttentionParams p) {
  using S = Shape<D, FP8>;
  using Y = Layout<D, FP8, HI>;
  constexpr int TILE = S::kTile, ROW = S::kRow, E = S::E, H = S::H, NT = TILE / 8, W = Y::kWarps;
  constexpr int THREADS = W * 32, R = HI ? 2 : 1;  // R: rows of a lane (g, g + 8)
  extern __shared__ __align__(128) uint8_t shared[];
  __shared__ int64_t before[THREADS + 1];          // tiles before each thread's sequences
  __shared__ uint32_t seen[W][Y::kStages];         // a staged tile's tokens that count
  __shared__ float part_m[W][2][kRows], part_l[W][2][kRows];
  __shared__ int seg_a[W], seg_b[W], done_a[W];
  __shared__ int64_t end_b[W];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, g = lane >> 2, c = lane & 3;

  afd::pdl_wait();
  afd::pdl_launch_dependents();

  // ---- the line of tiles, and this warp's share of it
  const int each = (p.B + THREADS - 1) / THREADS;
  {
    int64_t mine = 0;
    const int b0 = threadIdx.x * each, b1 = min(p.B, b0 + each);
    for (int b = b0; b < b1; ++b) {
      const Span s = span_of<TILE>(p, b);
      mine += s.end - s.first;
    }
    int64_t sum = mine;
#pragma unroll
    for (int d = 1; d < 32; d <<= 1) {
      const int64_t o = __shfl_up_sync(kFull, sum, d);
      if (lane >= d) sum += o;
    }
    if (lane == 31) end_b[warp] = sum;
    __syncthreads();
    for (int w = 0; w < warp; ++w) sum += end_b[w];
    before[threadIdx.x + 1] = sum;
    if (threadIdx.x == 0) before[0] = 0;
  }
  __syncthreads();
  const int64_t total = before[THREADS] * p.chunks;
  // A tile a warp at least: of few tiles the first blocks' warps take one each.
  const int workers = (int)min(total, (int64_t)gridDim.x * W), worker = blockIdx.x * W + warp;
  const bool works = worker < workers;
  const int64_t lo = works ? total * worker / workers : 0, hi = works ? total * (worker + 1) / workers : 0;

  // Sequences that see nothing.
  for (int b = blockIdx.x; b < p.B; b += gridDim.x) {
    const Span s = span_of<TILE>(p, b);
    if (s.first != s.end) continue;
    for (int i = threadIdx.x; i < p.Hq * (D / 8); i += THREADS)
      *reinterpret_cast<uint4*>(p.out + b * p.out_stride + i * 8) = make_uint4(0, 0, 0, 0);
    if (p.lse)
      for (int i = threadIdx.x; i < p.Hq; i += THREADS) p.lse[(int64_t)b * p.Hq + i] = -INFINITY;
  }

  uint8_t* ring = shared + warp * Y::kRing;
  float* kept = reinterpret_cast<float*>(shared + W * Y::kRing + warp * Y::kPart);
  if (lane == 0) seg_a[warp] = seg_b[warp] = -1, done_a[warp] = 0, end_b[warp] = 0;

  if (lo < hi) {
    // ---- where the share begins
    Cursor<TILE> at;
    {
      const int64_t line = lo / p.chunks;  // tiles of whole sequences, times the chunks
      int i = 0;
#pragma unroll 1
      for (int step = 256; step; step >>= 1)
        if (i + step < THREADS && before[i + step] <= line) i += step;
      int64_t left = lo - before[i] * p.chunks;
      at.b = i * each;
      at.span = span_of<TILE>(p, at.b);
      for (;;) {
        const int64_t n = (int64_t)(at.span.end - at.span.first) * p.chunks;
        if (left < n) break;
        left -= n;
        at.span = span_of<TILE>(p, ++at.b);
      }
      const int n = at.span.end - at.span.first;
      at.chunk = (int)(left / n);
      at.tile = at.span.first + (int)(left - (int64_t)at.chunk * n);
    }
    const int tiles = (int)(hi - lo);
    const int groups = p.chunks / p.Hkv;  // chunks of a KV head

    Cursor<TILE> ahead = at;
    Lookup next = look_up(p, ahead, lane);
    ahead.next(p);
    // Starts the copies of the tile looked up last, and looks the one after it up.
    auto issue = [&](int i) {
      if (i < tiles) {
        const bool in = next.in && (uint32_t)next.page < (uint32_t)p.cache.pages;
        const int stage = i % Y::kStages;
        const uint32_t dst = smem_addr(ring + stage * S::kStage);
        const uint32_t mask = __ballot_sync(kFull, in);
        if (lane == 0) seen[warp][stage] = mask;
        const int head = next.chunk / groups;
        const int64_t row = (int64_t)head * p.cache.page_size + next.at;
        const int64_t k_off = in ? next.page * p.cache.k_page_bytes + row * ROW : 0;
        const int64_t v_off = in ? next.page * p.cache.v_page_bytes + row * ROW : 0;
        constexpr int CH = ROW / 16;  // chunks of a row
#pragma unroll
        for (int j = 0; j < S::kBytes / 512; ++j) {
          const int idx = j * 32 + lane, r = idx / CH, ch = idx % CH;
          const int64_t ko = __shfl_sync(kFull, k_off, r), vo = __shfl_sync(kFull, v_off, r);
          const bool ok = (mask >> r) & 1u;
          const uint32_t to = dst + swizzled<ROW>(r, ch);
          copy16(to, p.cache.k + ko + ch * 16, ok);
          copy16(to + S::kBytes, p.cache.v + vo + ch * 16, ok);
        }
        if (FP8) {
          const int64_t o = in ? (int64_t)next.page * p.Hkv * p.cache.page_size + row : 0;
          copy4(dst + 2 * S::kBytes + lane * 4, p.cache.k_scale + o, in);
          copy4(dst + 2 * S::kBytes + (TILE + lane) * 4, p.cache.v_scale + o, in);
        }
        if (i + 1 < tiles) {
          next = look_up(p, ahead, lane);
          ahead.next(p);
        }
      }
      copies_commit();
    };
#pragma unroll 1
    for (int i = 0; i < Y::kStages - 1; ++i) issue(i);

    uint32_t qa[D / 16][4];
    float row_scale[2];
    float o[D / 8][4];
    float m[2], l[2];
    bool began = at.tile == at.span.first;  // the segment's first tile is this warp's

    // Query heads of the segment, zeros beyond the KV head's.
    auto load_q = [&]() {
      const int head = at.chunk / groups, sub = at.chunk % groups;
      const int rows = min(p.G - sub * kRows, kRows);
      const uint16_t* q = p.q + at.b * p.q_stride + (int64_t)(head * p.G + sub * kRows) * D;
      uint4 v[R][D / 32];
#pragma unroll
      for (int r = 0; r < R; ++r)
#pragma unroll
        for (int i = 0; i < D / 32; ++i) {
          // chunk i of this lane, as the keys' (16 bytes of theirs are 8 or 16 columns)
          const int col = FP8 ? (D == 128 ? (2 * c + i / 2) * 16 + i % 2 * 8 : c * 16 + i * 8)
                              : (D == 128 ? (2 * c + (i & 1) + 8 * (i >> 1)) * 8 : (2 * c + i) * 8);
          v[r][i] = g + 8 * r < rows ? *reinterpret_cast<const uint4*>(q + (g + 8 * r) * D + col) : make_uint4(0, 0, 0, 0);
        }
#pragma unroll
      for (int r = 0; r < 2; ++r) {
        row_scale[r] = p.scale_log2;
        if (!FP8 || r >= R) continue;
        // FP16 queries: the row's power of two taken out, so that the largest
        // lies in [1, 2) and the others keep their digits down to 2^-24 of it.
        float most = 0.f;
#pragma unroll
        for (int i = 0; i < D / 32; ++i) {
          float f[8];
          afd::bf16x8_to_float(v[r % R][i], f);
#pragma unroll
          for (int e = 0; e < 8; ++e) most = fmaxf(most, fabsf(f[e]));
        }
        most = quad_max(most);
        int ex = (int)(__float_as_uint(most) >> 23) - 127;
        ex = min(max(ex, -120), 120);
        const float down = __uint_as_float((uint32_t)(127 - ex) << 23);
        row_scale[r] = p.scale_log2 * __uint_as_float((uint32_t)(127 + ex) << 23);
#pragma unroll
        for (int i = 0; i < D / 32; ++i) {
          float f[8];
          afd::bf16x8_to_float(v[r % R][i], f);
          v[r % R][i] = make_uint4(pack_f16(f[0] * down, f[1] * down), pack_f16(f[2] * down, f[3] * down),
                               pack_f16(f[4] * down, f[5] * down), pack_f16(f[6] * down, f[7] * down));
        }
      }
#pragma unroll
      for (int i = 0; i < D / 32; ++i) {
        const uint4 a = v[0][i], b = HI ? v[R - 1][i] : make_uint4(0, 0, 0, 0);
        qa[2 * i][0] = a.x, qa[2 * i][1] = b.x, qa[2 * i][2] = a.y, qa[2 * i][3] = b.y;
        qa[2 * i + 1][0] = a.z, qa[2 * i + 1][1] = b.z, qa[2 * i + 1][2] = a.w, qa[2 * i + 1][3] = b.w;
      }
#pragma unroll
      for (int n = 0; n < D / 8; ++n) o[n][0] = o[n][1] = o[n][2] = o[n][3] = 0.f;
      m[0] = m[1] = -INFINITY;
      l[0] = l[1] = 0.f;
    };

    bool fresh = true;
#pragma unroll 1
    for (int i = 0; i < tiles; ++i) {
      copies_wait<Y::kStages - 2>();
      __syncwarp();
      issue(i + Y::kStages - 1);  // into the stage that the last tile has left
      if (fresh) load_q();
      fresh = false;
      const int stage = i % Y::kStages;
      const uint8_t* ks = ring + stage * S::kStage;
      const uint8_t* vs = ks + S::kBytes;
      const uint32_t mask = seen[warp][stage];

      // ---- scores
      float s[NT][4];
#pragma unroll
      for (int j = 0; j < NT; ++j) s[j][0] = s[j][1] = s[j][2] = s[j][3] = 0.f;
#pragma unroll
      for (int ii = 0; ii < ROW / 64; ++ii) {
        const int chunk = ROW == 256 ? 2 * c + (ii & 1) + 8 * (ii >> 1) : ROW == 128 ? 2 * c + ii : c;
#pragma unroll
        for (int j = 0; j < NT; ++j) {
          const uint4 kv = *reinterpret_cast<const uint4*>(ks + swizzled<ROW>(8 * j + g, chunk));
          if (FP8) {
            mma<true>(s[j], qa[(4 * ii) % (D / 16)], half2_of<0>(kv.x), half2_of<1>(kv.x));
            mma<true>(s[j], qa[(4 * ii + 1) % (D / 16)], half2_of<0>(kv.y), half2_of<1>(kv.y));
            mma<true>(s[j], qa[(4 * ii + 2) % (D / 16)], half2_of<0>(kv.z), half2_of<1>(kv.z));
            mma<true>(s[j], qa[(4 * ii + 3) % (D / 16)], half2_of<0>(kv.w), half2_of<1>(kv.w));
          } else {
            mma<false>(s[j], qa[(2 * ii) % (D / 16)], kv.x, kv.y);
            mma<false>(s[j], qa[(2 * ii + 1) % (D / 16)], kv.z, kv.w);
          }
        }
      }
      // ---- softmax. E4M3: the weight of a token's values is p * its scale, so
      // the running maximum is that of s + log2(scale): the FP16 weights are at
      // most 1, and what they lose is small beside the largest contribution.
      float top[2] = {m[0], m[1]};
      float vscale[NT][2];
#pragma unroll
      for (int j = 0; j < NT; ++j)
#pragma unroll
        for (int x = 0; x < 2; ++x) {
          const int tok = 8 * j + 2 * c + x;
          const bool in = (mask >> tok) & 1u;
          float kscale = 1.f, lift = 0.f;
          if (FP8) {
            kscale = reinterpret_cast<const float*>(vs + S::kBytes)[tok];
            vscale[j][x] = reinterpret_cast<const float*>(vs + S::kBytes)[TILE + tok];
            lift = fmaxf(log2_of(vscale[j][x]), -120.f);
          }
#pragma unroll
          for (int r = 0; r < R; ++r) {
            float& v = s[j][2 * r + x];
            v = in ? v * row_scale[r] * kscale : -INFINITY;
            top[r] = fmaxf(top[r], v + lift);
          }
        }
      float minus[2];
      bool moved = false;
#pragma unroll
      for (int r = 0; r < R; ++r) {
        top[r] = quad_max(top[r]);
        moved |= top[r] != m[r];
        minus[r] = top[r] == -INFINITY ? 0.f : top[r];
      }
      if (__any_sync(kFull, moved)) {
#pragma unroll
        for (int r = 0; r < R; ++r) {
          const float f = m[r] == -INFINITY ? 0.f : exp2_of(m[r] - minus[r]);
          m[r] = top[r];
          l[r] *= f;
#pragma unroll
          for (int n = 0; n < D / 8; ++n) o[n][2 * r] *= f, o[n][2 * r + 1] *= f;
        }
      }
#pragma unroll
      for (int j = 0; j < NT; ++j)
#pragma unroll
        for (int r = 0; r < R; ++r)
#pragma unroll
          for (int x = 0; x < 2; ++x) {
            float& v = s[j][2 * r + x];
            v = exp2_of(v - minus[r]);
            l[r] += v;
            if (FP8) v *= vscale[j][x];
          }
      // ---- values
#pragma unroll
      for (int n = 0; n < NT / 2; ++n) {
        uint32_t pa[4], pb[4];
        const float(&s0)[4] = s[2 * n];
        const float(&s1)[4] = s[2 * n + 1];
        if (FP8) {
          pa[0] = pack_f16(s0[0], s0[1]), pa[2] = pack_f16(s1[0], s1[1]);
          pa[1] = HI ? pack_f16(s0[2], s0[3]) : 0u, pa[3] = HI ? pack_f16(s1[2], s1[3]) : 0u;
        } else {
          auto two = [](float a, float b, uint32_t& high, uint32_t& low) {
            high = afd::pack_bf16(a, b);
            low = afd::pack_bf16(a - __uint_as_float(high << 16), b - __uint_as_float(high & 0xffff0000u));
          };
          pa[1] = pa[3] = pb[1] = pb[3] = 0u;
          two(s0[0], s0[1], pa[0], pb[0]);
          two(s1[0], s1[1], pa[2], pb[2]);
          if (HI) {
            two(s0[2], s0[3], pa[1], pb[1]);
            two(s1[2], s1[3], pa[3], pb[3]);
          }
        }
        const int t0 = 16 * n + 2 * c;
        if constexpr (!FP8) {
#pragma unroll
          for (int h = 0; h < H; ++h) {
            uint32_t v[4][4];
#pragma unroll
            for (int t = 0; t < 4; ++t) {
              const uint4 u = *reinterpret_cast<const uint4*>(vs + swizzled<ROW>(t0 + (t & 1) + 8 * (t >> 1), 8 * h + g));
              v[t][0] = u.x, v[t][1] = u.y, v[t][2] = u.z, v[t][3] = u.w;
            }
#pragma unroll
            for (int e = 0; e < 8; ++e) {
              const uint32_t b0 = __byte_perm(v[0][e / 2], v[1][e / 2], e & 1 ? 0x7632 : 0x5410);
              const uint32_t b1 = __byte_perm(v[2][e / 2], v[3][e / 2], e & 1 ? 0x7632 : 0x5410);
              mma<false>(o[h * 8 + e], pa, b0, b1);
              mma<false>(o[h * 8 + e], pb, b0, b1);
            }
          }
        } else {
          uint32_t v[4][E / 4];
#pragma unroll
          for (int t = 0; t < 4; ++t) {
            const int row = t0 + (t & 1) + 8 * (t >> 1);
            if constexpr (D == 128) {
              const uint4 u = *reinterpret_cast<const uint4*>(vs + swizzled<ROW>(row, g));
              v[t][0] = u.x, v[t][1] = u.y, v[t][2] = u.z, v[t][3] = u.w;
            } else {
              const uint2 u = *reinterpret_cast<const uint2*>(vs + swizzled<ROW>(row, g >> 1) + (g & 1) * 8);
              v[t][0] = u.x, v[t][1] = u.y;
            }
          }
#pragma unroll
          for (int w = 0; w < E / 4; ++w) {
            const uint32_t x0 = __byte_perm(v[0][w], v[1][w], 0x5140), x1 = __byte_perm(v[2][w], v[3][w], 0x5140);
            const uint32_t y0 = __byte_perm(v[0][w], v[1][w], 0x7362), y1 = __byte_perm(v[2][w], v[3][w], 0x7362);
            mma<true>(o[4 * w], pa, half2_of<0>(x0), half2_of<0>(x1));
            mma<true>(o[4 * w + 1], pa, half2_of<1>(x0), half2_of<1>(x1));
            mma<true>(o[4 * w + 2], pa, half2_of<0>(y0), half2_of<0>(y1));
            mma<true>(o[4 * w + 3], pa, half2_of<1>(y0), half2_of<1>(y1));
          }
        }
      }

      // ---- the end of a segment, or of the share
      const bool ends = at.tile + 1 == at.span.end;
      if (ends || i + 1 == tiles) {
#pragma unroll
        for (int r = 0; r < R; ++r) l[r] = quad_sum(l[r]);
        const int seg = at.b * p.chunks + at.chunk;
        if (began && ends) {
          const int head = at.chunk / groups, sub = at.chunk % groups;
          const int rows = min(p.G - sub * kRows, kRows), q0 = head * p.G + sub * kRows;
#pragma unroll
          for (int r = 0; r < R; ++r) {
            const int row = g + 8 * r;
            if (row >= rows) continue;
            const float inv = l[r] == 0.f ? 0.f : 1.f / l[r];
            uint16_t* out = p.out + at.b * p.out_stride + (int64_t)(q0 + row) * D;
#pragma unroll
            for (int h = 0; h < H; ++h)
#pragma unroll
              for (int x = 0; x < 2; ++x)
#pragma unroll
                for (int e = 0; e < E; e += 8) {
                  float f[8];
#pragma unroll
                  for (int k = 0; k < 8; ++k) f[k] = o[h * 8 + e + k][2 * r + x] * inv;
                  *reinterpret_cast<uint4*>(out + (8 * h + 2 * c + x) * E + e) = afd::float_to_bf16x8(f);
                }
            if (p.lse && c == 0) p.lse[(int64_t)at.b * p.Hq + q0 + row] = l[r] == 0.f ? -INFINITY : m[r] * kLn2 + logf(l[r]);
          }
        } else {
          // Left open: in the warp's own place if it began in an earlier warp's
          // share, else (then it is the share's last) where the ring was.
          const int which = began ? 1 : 0;
          float* to = kept;
          if (which) {
            copies_wait<0>();
            __syncwarp();
            to = reinterpret_cast<float*>(ring);
          }
#pragma unroll
          for (int r = 0; r < R; ++r) {
#pragma unroll
            for (int h = 0; h < H; ++h)
#pragma unroll
              for (int x = 0; x < 2; ++x)
#pragma unroll
                for (int e = 0; e < E; e += 4)
                  *reinterpret_cast<float4*>(to + (g + 8 * r) * D + (8 * h + 2 * c + x) * E + e) =
                      make_float4(o[h * 8 + e][2 * r + x], o[h * 8 + e + 1][2 * r + x], o[h * 8 + e + 2][2 * r + x],
                                  o[h * 8 + e + 3][2 * r + x]);
            if (c == 0) part_m[warp][which][g + 8 * r] = m[r], part_l[warp][which][g + 8 * r] = l[r];
          }
          if (lane == 0) {
            if (which) seg_b[warp] = seg, end_b[warp] = lo + i + (at.span.end - at.tile);
            else seg_a[warp] = seg, done_a[warp] = ends;
          }
        }
        began = true;
        fresh = true;
      }
      if (i + 1 < tiles) at.next(p);
    }
    copies_wait<0>();
  }
  __syncthreads();

  // ---- the block's open parts: a chain begins with the first warp's part of an
  // earlier block's segment, or with a warp's last one, and goes on through the
  // next warps' first ones.
  const int valid = HI ? 16 : 8;
  int tail = -1;
  int64_t tail_end = 0;
#pragma unroll 1
  for (int w0 = -1; w0 < W; ++w0) {
    const int seg = w0 < 0 ? seg_a[0] : seg_b[w0];
    if (seg < 0) continue;
    int w1 = w0 + 1;
    bool done = false;
    while (w1 < W && seg_a[w1] == seg) done |= done_a[w1] != 0, ++w1;
    const bool whole = w0 >= 0 && done;
    if (w0 >= 0 && !done) tail = seg, tail_end = end_b[w0];
    const int b = seg / p.chunks, chunk = seg % p.chunks, groups = p.chunks / p.Hkv;
    const int head = chunk / groups, sub = chunk % groups;
    const int rows = min(min(p.G - sub * kRows, kRows), valid), q0 = head * p.G + sub * kRows;
    float* part = p.parts + ((int64_t)blockIdx.x * 2 + (w0 >= 0)) * kRows * (D + 2);
    for (int i = threadIdx.x; i < rows * (D / 8); i += THREADS) {
      const int row = i / (D / 8), col = i % (D / 8) * 8;
      float most = w0 >= 0 ? part_m[w0][1][row] : -INFINITY;
      for (int w = w0 + 1; w < w1; ++w) most = fmaxf(most, part_m[w][0][row]);
      const float minus = most == -INFINITY ? 0.f : most;
      float sum = 0.f, f[8] = {};
      for (int w = max(w0, 0); w < w1; ++w) {
        const int which = w == w0;
        const float scale = exp2_of(part_m[w][which][row] - minus);
        const float* from = which ? reinterpret_cast<const float*>(shared + w * Y::kRing)
                                  : reinterpret_cast<const float*>(shared + W * Y::kRing + w * Y::kPart);
        sum += part_l[w][which][row] * scale;
#pragma unroll
        for (int k = 0; k < 8; ++k) f[k] = fmaf(from[row * D + col + k], scale, f[k]);
      }
      if (whole) {
        const float inv = sum == 0.f ? 0.f : 1.f / sum;
#pragma unroll
        for (int k = 0; k < 8; ++k) f[k] *= inv;
        *reinterpret_cast<uint4*>(p.out + b * p.out_stride + (int64_t)(q0 + row) * D + col) = afd::float_to_bf16x8(f);
        if (p.lse && col == 0) p.lse[(int64_t)b * p.Hq + q0 + row] = sum == 0.f ? -INFINITY : most * kLn2 + logf(sum);
      } else {
        *reinterpret_cast<float4*>(part + row * D + col) = make_float4(f[0], f[1], f[2], f[3]);
        *reinterpret_cast<float4*>(part + row * D + col + 4) = make_float4(f[4], f[5], f[6], f[7]);
        if (col == 0) part[kRows * D + row] = most, part[kRows * (D + 1) + row] = sum;
      }
    }
  }
  if (p.splits && threadIdx.x == 0) {
    // the block with the segment's last tile: its first tile is at or before it
    const int last = tail < 0 ? 0 : (int)((tail_end * workers - 1) / total / W);
    p.splits[blockIdx.x] = {tail, last, {0, 0}};
  }
}

// Joins what the blocks left open: a warp per row of a segment that began in
// block `from`; its parts are that block's second and the next ones' first.
template <int D>
__global__ void __launch_bounds__(256) decode_join_kernel(const AttentionParams p) {
  afd::pdl_wait();
  afd::pdl_launch_dependents();
  const int lane = threadIdx.x & 31;
  const int item = blockIdx.x * 8 + (threadIdx.x >> 5), from = item / kRows, row = item % kRows;
  const Split split = p.splits[from];
  if (split.seg < 0) return;
  const int b = split.seg / p.chunks, chunk = split.seg % p.chunks, groups = p.chunks / p.Hkv;
  const int head = chunk / groups, sub = chunk % groups;
  if (row >= min(p.G - sub * kRows, kRows)) return;
  constexpr int64_t kPart = kRows * (D + 2);
  auto part = [&](int i) { return p.parts + ((int64_t)i * 2 + (i == from)) * kPart; };
  float most = -INFINITY;
  for (int i = from + lane; i <= split.last; i += 32) most = fmaxf(most, part(i)[kRows * D + row]);
#pragma unroll
  for (int d = 16; d; d >>= 1) most = fmaxf(most, __shfl_xor_sync(kFull, most, d));
  const float minus = most == -INFINITY ? 0.f : most;
  constexpr int N = D / 32;
  float sum = 0.f, f[N] = {};
#pragma unroll 4
  for (int i = from; i <= split.last; ++i) {
    const float* q = part(i);
    const float scale = exp2_of(q[kRows * D + row] - minus);
    sum = fmaf(q[kRows * (D + 1) + row], scale, sum);
    if constexpr (N == 4) {
      const float4 v = *reinterpret_cast<const float4*>(q + row * D + lane * 4);
      f[0] = fmaf(v.x, scale, f[0]), f[1] = fmaf(v.y, scale, f[1]);
      f[2] = fmaf(v.z, scale, f[2]), f[3] = fmaf(v.w, scale, f[3]);
    } else {
      const float2 v = *reinterpret_cast<const float2*>(q + row * D + lane * 2);
      f[0] = fmaf(v.x, scale, f[0]), f[1] = fmaf(v.y, scale, f[1]);
    }
  }
  const float inv = sum == 0.f ? 0.f : 1.f / sum;
  const int q = head * p.G + sub * kRows + row;
  uint32_t* out = reinterpret_cast<uint32_t*>(p.out + b * p.out_stride + (int64_t)q * D + lane * N);
#pragma unroll
  for (int k = 0; k < N; k += 2) out[k / 2] = afd::pack_bf16(f[k] * inv, f[k + 1] * inv);
  if (p.lse && lane == 0) p.lse[(int64_t)b * p.Hq + q] = sum == 0.f ? -INFINITY : most * kLn2 + logf(sum);
}

int tile_tokens(int head_dim, bool fp8) { return head_dim == 128 && !fp8 ? 16 : 32; }

int64_t workspace_of(int head_dim) {
  return kMaxBlocks * (int64_t)(sizeof(Split) + 2 * kRows * (head_dim + 2) * sizeof(float));
}

// The most tiles there can be: those of full tables.
int64_t most_tiles(int64_t seqs, int64_t q_heads, int64_t kv_heads, int64_t tokens, int tile) {
  const int64_t chunks = kv_heads * ((q_heads / kv_heads + kRows - 1) / kRows);
  const int64_t tiles = (tokens + tile - 1) / tile;
  return tiles == 0 ? 0 : seqs * chunks > INT64_MAX / tiles ? INT64_MAX : seqs * chunks * tiles;
}

template <int D, bool FP8, bool HI>
cudaError_t launch_attention(const AttentionParams& p, int64_t tiles, int device, int sms, cudaStream_t stream) {
  using Y = Layout<D, FP8, HI>;
  static std::atomic<uint64_t> done{0};
  cudaError_t e = afd::allow_shared(decode_attention_kernel<D, FP8, HI>, Y::kShared, device, done);
  if (e != cudaSuccess) return e;
  const int64_t want = tiles / Y::kWarps + (tiles % Y::kWarps != 0), most = sms < kMaxBlocks ? sms : kMaxBlocks;
  const int blocks = (int)(want < 1 ? 1 : want < most ? want : most);
  e = afd::launch_dependent(decode_attention_kernel<D, FP8, HI>, blocks, Y::kWarps * 32, Y::kShared, stream, p);
  if (e != cudaSuccess || blocks == 1) return e;
  return afd::launch_dependent(decode_join_kernel<D>, blocks * kRows / 8, 256, 0, stream, p);
}

template <int D>
cudaError_t launch_of(const AttentionParams& p, bool fp8, int64_t tiles, int device, int sms, cudaStream_t stream) {
  if (p.G > 8)
    return fp8 ? launch_attention<D, true, true>(p, tiles, device, sms, stream)
               : launch_attention<D, false, true>(p, tiles, device, sms, stream);
  return fp8 ? launch_attention<D, true, false>(p, tiles, device, sms, stream)
             : launch_attention<D, false, false>(p, tiles, device, sms, stream);
}

constexpr int64_t kMaxTokens = INT32_MAX - 1024;  // of a table's row

}  // namespace

extern "C" {

AFD_API int64_t afd_decode_workspace_bytes(int32_t num_seqs, int32_t num_q_heads, int32_t num_kv_heads, int32_t head_dim,
                                           int32_t max_pages, int32_t page_size) {
  if (num_seqs < 0 || num_kv_heads < 1 || num_q_heads < 1 || num_q_heads % num_kv_heads || max_pages < 0 || page_size < 1 ||
      (head_dim != 64 && head_dim != 128))
    return -1;
  // (of the two types' tiles the smaller, so the larger number of them)
  const int64_t tiles = most_tiles(num_seqs, num_q_heads, num_kv_heads, (int64_t)max_pages * page_size, 16);
  return tiles <= Layout<128, false, false>::kWarps ? 0 : workspace_of(head_dim);
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
  const int64_t row = (int64_t)num_q_heads * D;
  if (num_q_heads % Hkv || (num_seqs > 1 && (q_stride < row || out_stride < row || table_stride < max_pages))) return AFD_ERR_ARG;
  const int64_t tokens = (int64_t)max_pages * cache->page_size;
  const int groups = (num_q_heads / Hkv + kRows - 1) / kRows;
  if (num_q_heads > afd::kMaxHeads || tokens > kMaxTokens || (int64_t)num_seqs * Hkv * groups > afd::kMaxRows ||
      q_stride % 8 || out_stride % 8)
    return AFD_ERR_UNSUPPORTED;
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
  if (need > 0) p.parts = reinterpret_cast<float*>(p.splits + kMaxBlocks);
  int dev = -1, sms = 0;
  if (cudaGetDevice(&dev) != cudaSuccess || cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess)
    return AFD_ERR_CUDA;
  const bool fp8 = cache->dtype == AFD_FP8_E4M3;
  const int64_t tiles = most_tiles(num_seqs, num_q_heads, Hkv, tokens, tile_tokens(D, fp8));
  cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
  const cudaError_t e = D == 64 ? launch_of<64>(p, fp8, tiles, dev, sms, s) : launch_of<128>(p, fp8, tiles, dev, sms, s);
  return e == cudaSuccess ? AFD_OK : AFD_ERR_CUDA;
}

}  // extern "C"
