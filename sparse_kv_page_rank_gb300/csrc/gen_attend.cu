// Attention of one query token per row of the cache, where the W rows of a request share
// their first pages (beams of one prompt): the shared pages are read once for
// all of the request's rows, the rest once per row.
//
// Mathematics.  The softmax over a row's keys is that over two parts, joined by their
// maxima and sums.  For the shared part the rows of the products are (beam, query head of
// the group), up to 32 at a time; for a row's own part the group's heads.
//
// What bounds it: the bytes of the shared pages once and of the rows' own pages.
//
// Layout.  mma.sync m16n8k16 with one or two tiles of 16 rows: a CTA of four warps takes
// 64 tokens at a time from a ring that bulk and tensor copies fill.  Warp w has the logits and weights
// of tokens 16 w .. 16 w + 15; the weights go to the other warps by shared memory, and a warp has 32 columns
// of the outputs for all tokens.  So every value is loaded, and every code taken apart, once, a piece ends
// without a merge of outputs, and 172 registers suffice (168 at 4 bits, where the
// kernel of 16-token pages spills 8 bytes).  With all 128 columns of its own
// tokens in each warp (255 registers) 32 K tokens in bf16 took 34.1 us for 32.3, 16-token pages 36.3
// for 33.3, 4-bit ones 45.7 for 42; but 43.3 for 44.1 where 64 rows share 32 K tokens (one set of inputs,
// of which L2 holds a part).
// bf16 pages: ldmatrix.  4-bit pages: keys' codes are bf16 numbers (exact) and get their scale on the
// four partial sums of a logit; values are s * code rounded to half precision (2^-11), and so are the
// weights.  The queries lie in shared memory in the order of the products' registers (42 us to 39.8 on one
// set of inputs); three CTAs per SM, four of 128 registers take 43.6 us for 41.2 (the last case below).
//
// Work split.  All 64-token tiles of all problems lie in one line: request by request, KV
// head by head, first the shared pages (once per block of 32 rows), then each row's own.  Every
// CTA gets an equal part of it; a segment counts a few tiles more
// than it has, which is what its queries, its first copies and its merge cost.  A piece
// (the part of a segment that a CTA has) leaves its state in the workspace at place
// CTA + segment, which no two pieces share; a second, dependent kernel joins them.
//
// Measured, 32 query / 8 KV heads, in a graph, on inputs that change and exceed L2 (floor by bytes; every row
// by itself): eight rows that share 32 K tokens of bf16 pages and have 60 of their own 33.3 us (20.1; 82.7), 300
// 34.1 (21.2; 82.8); 131 K shared 89.1 us (79.6; 274); of 2 K 12.2 us, four rows 10.5.  Four requests of eight rows, up to
// 16 K tokens of 4-bit pages 39.4 us, 16-token ones 41.2 us (8.1; 74 and 81): 32 rows per key make the instructions
// the bound there, some 730 per warp and 64 tokens.
#include <algorithm>
#include <climits>
#include <type_traits>

#include "gen.h"
#include "kv_q4.cuh"

namespace locks {

namespace {

constexpr int kWarps = 4;
constexpr int kThreads = kWarps * 32;
constexpr int kHalfTile = 64 * 128;   // bytes of a 64-row x 64-column bf16 box
constexpr int kTile = 2 * kHalfTile;  // 64 tokens of K (or V)
constexpr int kQueryBytes = kSharedRows * kHeadDim * 2;
template <bool Q4>
constexpr int kOStride = Q4 ? 132 : 136;  // padded row of outputs (floats), against bank conflicts
template <bool Q4>
constexpr int kStageBytes = Q4 ? kQ4Slot : 2 * kTile;
// Measured for 4 bits (3, 4, 5, 6 stages): four requests of 16 K, 64-token pages 41.9, 39.5, 40.3, 40.8 us, 16-token ones
// 42.3, 41.2, 41.6, 42.1; 131 K 77.3, 77.5, 78.7, 79.5; one request of 32 K 28.8, 29.2, 29.8, 30.4.
template <bool Q4>
constexpr int kStages = Q4 ? 4 : 3;
template <bool Q4>
constexpr int kCtas = Q4 ? 3 : 2;  // per SM
// Whether the warps take turns at asking for a tile; warps that ask for one.
template <int P, bool Q4>
constexpr bool kTurns = Q4 && P == kPage;
template <int P, bool Q4>
constexpr int kAsking = kTurns<P, Q4> ? 1 : kWarps;
constexpr int kWeightBytes = kWarps * 2 * 32 * 16;  // weights of a tile
template <bool Q4>
constexpr int kSmem = kStages<Q4> * kStageBytes<Q4> + kQueryBytes + kWeightBytes + 1024;
static_assert(kSharedRows * kOStride<true> * 4 <= kStages<true> * kStageBytes<true> &&
                  kSharedRows * kOStride<false> * 4 <= kStages<false> * kStageBytes<false>,
              "the outputs fit the ring");

// ---- lengths, and what follows from them ----------------------------------------------

__device__ __forceinline__ int row_length(const GroupArgs& a, int row, bool says) {
  int len = a.seq_lens[row];  // (plain loads where the kernel before may have written)
  if (len < 0 || len > a.max_pages * a.page_size) {
    if (says) set_error(a.err, LOCKS_DEVERR_LENGTHS);
    len = len < 0 ? 0 : a.max_pages * a.page_size;
  }
  return len;
}
// Shared pages of a request whose `live` rows have at least `full` whole pages: a row
// alone shares with nobody.
__device__ __forceinline__ int shared_of(int given, int full, int live) { return live > 1 ? max(0, min(given, full)) : 0; }
__device__ __forceinline__ int tiles_of(int tokens) { return tokens > 0 ? (tokens - 1) / kPage + 1 : 0; }
__device__ __forceinline__ int line_of(int tiles) { return tiles > 0 ? tiles + kSegment : 0; }

// One thread: the places in the line of one KV head of request g.
__device__ __forceinline__ int head_line(const GroupArgs& a, int g, bool says) {
  const int given = a.shared_pages[g], base = g * a.beams;
  int full = INT_MAX, live = 0;
#pragma unroll 8
  for (int w = 0; w < a.beams; ++w) {
    const int len = row_length(a, base + w, says);
    if (len > 0) full = min(full, len / a.page_size), ++live;
  }
  const int sp = shared_of(given, full, live);
  int n = a.n_blocks * line_of(tiles_of(sp * a.page_size));
#pragma unroll 8
  for (int w = 0; w < a.beams; ++w) n += line_of(tiles_of(row_length(a, base + w, false) - sp * a.page_size));
  return n;
}

// A request, for the CTA at hand.
struct Group {
  int g, sp, first, shared_tiles, line;  // line: places of one head
  int len[LOCKSGEN_MAX_BEAMS];
  int upto[LOCKSGEN_MAX_BEAMS];          // places of the rows' own parts, up to and with row w
};
// One warp.
__device__ void load_group(const GroupArgs& a, int g, Group& s, bool says) {
  const int lane = threadIdx.x & 31, given = a.shared_pages[g];
  const int len = lane < a.beams ? row_length(a, g * a.beams + lane, says) : 0;
  const uint32_t live = __ballot_sync(0xffffffffu, len > 0);
  const int full = __reduce_min_sync(0xffffffffu, len > 0 ? len / a.page_size : INT_MAX);
  const int sp = shared_of(given, full, __popc(live));
  int upto = line_of(tiles_of(len > 0 ? len - sp * a.page_size : 0));
#pragma unroll
  for (int d = 1; d < 32; d *= 2) {
    const int other = __shfl_up_sync(0xffffffffu, upto, d);
    if (lane >= d) upto += other;
  }
  s.len[lane] = len;
  s.upto[lane] = upto;
  if (lane == 31) {
    s.g = g;
    s.sp = sp;
    s.first = live ? __ffs(live) - 1 : 0;
    s.shared_tiles = tiles_of(sp * a.page_size);
    s.line = upto + a.n_blocks * line_of(s.shared_tiles);
  }
}
static_assert(LOCKSGEN_MAX_BEAMS == 32, "a lane per row");

// The line in equal parts: the first `more` CTAs have one place more than the others.
struct Parts {
  uint32_t ctas, each, more;
  __device__ __forceinline__ Parts(uint32_t total, int n) {
    ctas = max(min((uint32_t)n, total), 1u);
    each = total / ctas;
    more = total - each * ctas;
  }
  __device__ __forceinline__ uint32_t begin(uint32_t cta) const {
    const uint32_t c = min(cta, ctas);
    return c * each + min(c, more);
  }
  // the CTA that has place y
  __device__ __forceinline__ uint32_t owner(uint32_t y) const {
    const uint32_t big = more * (each + 1);
    return y < big ? y / (each + 1) : more + (y - big) / each;
  }
};

// ---- a piece of a segment ---------------------------------------------------------------

struct Piece {
  bool shared;
  int h, w, block;     // KV head; row (own part); block of rows (shared part)
  int rows;            // of the products
  int t0, t1;          // tiles of the segment
  int page0, pages;    // first logical page, pages
  int limit;           // tokens that may be seen
  const int32_t* table;
};

constexpr int kFewGroups = 2 * kWarps;
struct Shared {
  uint64_t full[8];
  int left[8][4];  // per stage (and page of it): tokens of the tile to be seen
  float m[kWarps][kSharedRows], l[kWarps][kSharedRows];
  Group grp;
  Group few[kWarps];
  uint32_t offset, scan[kWarps], lines[kFewGroups];
  int group, abort;
};

// The query of row r of a piece.
__device__ __forceinline__ size_t query_row(const GroupArgs& a, const Piece& p, int g, int r) {
  int w = p.w, e = r;
  if (p.shared) {
    const int i = p.block * kSharedRows + r;
    w = i / a.group;
    e = i % a.group;
  }
  return ((size_t)(g * a.beams + w) * a.num_kv_heads + p.h) * a.group + e;
}

// Address of 16 bytes (chunk) of a query, for ldmatrix.
__device__ __forceinline__ uint32_t query_addr(uint32_t base, int row, int chunk) {
  return base + row * 256 + ((chunk ^ (row & 7)) << 4);
}
// For 4-bit pages queries lie as the products take them, 16 bytes a lane: of row tile i and
// dimensions 32 j + .., the first or second step.
__device__ __forceinline__ uint32_t fragment_addr(uint32_t base, int i, int j, int step, int lane) {
  return base + ((i * 4 + j) * 2 + step) * 512 + lane * 16;
}
__device__ __forceinline__ void sts32(uint32_t addr, uint32_t v) { asm volatile("st.shared.u32 [%0], %1;\n" ::"r"(addr), "r"(v) : "memory"); }
__device__ __forceinline__ uint32_t tile_addr(uint32_t base, int row, int chunk) {
  return base + (chunk >> 3) * kHalfTile + row * 128 + (((chunk & 7) ^ (row & 7)) << 4);
}
// Mask of a packed pair of tokens (t, t + 1) that keeps those before `len`.
__device__ __forceinline__ uint32_t pair_mask(int t, int len) {
  return (t < len ? 0x0000ffffu : 0u) | (t + 1 < len ? 0xffff0000u : 0u);
}

// A warp's sums for its tokens and outputs for its columns: rows 16 i + g, 16 i + g + 8.  m is the
// reference of a row's weights 2^(s - m): the largest logit when it was set, less kBelow.
// It is the same in all warps and moves only when a weight would exceed 2^kLimit, so the usual tile
// needs no maximum across lanes, only a vote.  bf16 weights: any range will do.  Half-precision ones: the
// largest lies between 2^7 and 2^15, so those below 2^-32 of it are what is lost.
template <int MT, bool Q4>
struct State {
  static constexpr float kBelow = Q4 ? 7.f : 0.f, kLimit = Q4 ? 15.f : 8.f;
  static constexpr int kBlocks = 4;  // of eight output columns
  float m[MT][2], l[MT][2];
  float o[MT][kBlocks][4];
  __device__ __forceinline__ void reset() {
#pragma unroll
    for (int i = 0; i < MT; ++i) {
      m[i][0] = m[i][1] = -INFINITY;
      l[i][0] = l[i][1] = 0.f;
#pragma unroll
      for (int n = 0; n < kBlocks; ++n) o[i][n][0] = o[i][n][1] = o[i][n][2] = o[i][n][3] = 0.f;
    }
  }
  // This lane's largest logits (s: unscaled); whether one of them moves its row's reference.
  __device__ __forceinline__ bool look(const float (&s)[MT][2][4], float scale_log2, float (&top)[MT][2]) const {
    bool moved = false;
#pragma unroll
    for (int i = 0; i < MT; ++i)
#pragma unroll
      for (int k = 0; k < 2; ++k) {
        top[i][k] = fmaxf(fmaxf(s[i][0][2 * k], s[i][0][2 * k + 1]), fmaxf(s[i][1][2 * k], s[i][1][2 * k + 1])) * scale_log2;
        moved |= top[i][k] > m[i][k] + kLimit;
      }
    return moved;
  }
  // The largest logit of a row among the lanes that hold it.
  __device__ __forceinline__ static float row_top(float t) {
    t = fmaxf(t, __shfl_xor_sync(0xffffffffu, t, 1));
    return fmaxf(t, __shfl_xor_sync(0xffffffffu, t, 2));
  }
  // The reference of a row of which logit t is the largest in sight.  It moves for the row's own
  // logits alone, so that no other row, an idle one whose query is whatever memory held least
  // of all, has a part in how this one's weights are rounded.
  __device__ __forceinline__ void move(int i, int k, float t) {
    t = t > m[i][k] + kLimit ? t - kBelow : m[i][k];
    const float al = t == m[i][k] ? 1.f : fast_exp2(m[i][k] - t);
    m[i][k] = t;
    l[i][k] *= al;
#pragma unroll
    for (int n = 0; n < kBlocks; ++n) {
      o[i][n][2 * k] *= al;
      o[i][n][2 * k + 1] *= al;
    }
  }
  // Logits to weights.
  __device__ __forceinline__ void weigh(float (&s)[MT][2][4], float scale_log2) {
#pragma unroll
    for (int i = 0; i < MT; ++i)
#pragma unroll
      for (int k = 0; k < 2; ++k) {
        const float ref = m[i][k] == -INFINITY ? 0.f : m[i][k];
#pragma unroll
        for (int n = 0; n < 2; ++n)
#pragma unroll
          for (int e = 0; e < 2; ++e) {
            float& x = s[i][n][2 * k + e];
            x = fast_exp2(fmaf(x, scale_log2, -ref));
            l[i][k] += x;
          }
      }
  }
};

// The logits of tokens 16 warp .. + 15 of a tile of bf16 pages at `base` (keys, then values), of
// which the first `left` are seen.
template <int MT>
__device__ __forceinline__ void logits_bf16(float (&s)[MT][2][4], uint32_t base, uint32_t queries, int left) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, c = lane & 3, mi = lane >> 3;
#pragma unroll
  for (int i = 0; i < MT; ++i)
#pragma unroll
    for (int e = 0; e < 4; ++e) s[i][0][e] = s[i][1][e] = 0.f;
  const int krow = 16 * warp + (mi >> 1) * 8 + (lane & 7);
#pragma unroll
  for (int kk = 0; kk < 8; ++kk) {
    uint32_t b0, b1, b2, b3;
    ldmatrix_x4(b0, b1, b2, b3, tile_addr(base, krow, 2 * kk + (mi & 1)));
#pragma unroll
    for (int i = 0; i < MT; ++i) {
      uint32_t a0, a1, a2, a3;
      ldmatrix_x4(a0, a1, a2, a3, query_addr(queries, 16 * i + (mi & 1) * 8 + (lane & 7), 2 * kk + (mi >> 1)));
      mma_16816(s[i][0], a0, a1, a2, a3, b0, b1);
      mma_16816(s[i][1], a0, a1, a2, a3, b2, b3);
    }
  }
  if (left < 16) {
#pragma unroll
    for (int i = 0; i < MT; ++i)
#pragma unroll
      for (int n = 0; n < 2; ++n)
#pragma unroll
        for (int e = 0; e < 4; ++e)
          if (8 * n + 2 * c + (e & 1) >= left) s[i][n][e] = -INFINITY;
  }
}
// The weights of 16 tokens (a fragment each lane: `weights`) times this warp's 32 columns of their values.
template <int MT, bool WHOLE>
__device__ __forceinline__ void values_bf16(State<MT, false>& st, uint32_t base, int group, uint32_t weights, int left) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, c = lane & 3, mi = lane >> 3;
  const int vrow = 16 * group + (mi & 1) * 8 + (lane & 7);
  uint4 p[MT];
#pragma unroll
  for (int i = 0; i < MT; ++i) p[i] = lds128(weights + ((group * MT + i) * 32 + lane) * 16);
#pragma unroll
  for (int n = 0; n < 2; ++n) {
    uint32_t v0, v1, v2, v3;
    ldmatrix_x4_trans(v0, v1, v2, v3, tile_addr(base + kTile, vrow, 4 * warp + 2 * n + (mi >> 1)));
    if constexpr (!WHOLE) {  // what lies past the end may be anything
      const uint32_t k0 = pair_mask(2 * c, left), k1 = pair_mask(8 + 2 * c, left);
      v0 &= k0, v1 &= k1, v2 &= k0, v3 &= k1;
    }
#pragma unroll
    for (int i = 0; i < MT; ++i) {
      mma_16816(st.o[i][2 * n], p[i].x, p[i].y, p[i].z, p[i].w, v0, v1);
      mma_16816(st.o[i][2 * n + 1], p[i].x, p[i].y, p[i].z, p[i].w, v2, v3);
    }
  }
}

// Fields i of both halves of w, each holding code + 8, as a bf16 pair of codes: the field under
// the exponent of 128 is 128 + u exactly, from which 136 is taken.
template <int I>
__device__ __forceinline__ uint32_t code_pair(uint32_t w) {
  uint32_t d = field_under<0x000f000fu, 0x43004300u>(w >> (4 * I));
  asm("sub.rn.bf16x2 %0, %0, %1;\n" : "+r"(d) : "r"(0x43084308u));
  return d;
}
// D = A B: the first of a chain of products.
__device__ __forceinline__ void mma_first(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0, uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%10,%10,%10,%10};\n"
      : "=f"(d[0]), "=f"(d[1]), "=f"(d[2]), "=f"(d[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1), "f"(0.f));
}

// 4-bit pages: the logits of tokens 16 warp .. + 15, of which the first `left` are seen.  A key
// word holds dimensions 32 j + 8 c .. + 7 of one token, field i the pair 8 c + 2 i, + 1, so fields 0
// and 1 are one step of a product, 2 and 3 the next; the queries are read in that order.
template <int P, int MT>
__device__ __forceinline__ void logits_q4(float (&s)[MT][2][4], uint32_t base, uint32_t queries, int left) {
  using At = Q4Tile<P>;
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, c = lane & 3;
  {
    // keys: tokens g and 8 + g for the products, their scales for columns 2c, 2c + 1
    const uint32_t kb = base + At::key_codes(warp), sb = base + At::key_scales(warp);
    const uint4 w0 = lds128(kb + lane * 16), w1 = lds128(kb + 512 + lane * 16);
    const uint4 z0 = lds128(sb + c * 16), z1 = lds128(sb + 64 + c * 16);
    const uint32_t kw0[4] = {w0.x, w0.y, w0.z, w0.w}, kw1[4] = {w1.x, w1.y, w1.z, w1.w};
    // halves j of tokens 2c (x, y) and 2c + 1 (z, w)
    const uint32_t za[2][2] = {{z0.x, z0.y}, {z1.x, z1.y}}, zb[2][2] = {{z0.z, z0.w}, {z1.z, z1.w}};
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const uint32_t f[2][4] = {{code_pair<0>(kw0[j]), code_pair<1>(kw0[j]), code_pair<2>(kw0[j]), code_pair<3>(kw0[j])},
                                {code_pair<0>(kw1[j]), code_pair<1>(kw1[j]), code_pair<2>(kw1[j]), code_pair<3>(kw1[j])}};
#pragma unroll
      for (int i = 0; i < MT; ++i) {
        const uint4 q0 = lds128(fragment_addr(queries, i, j, 0, lane)), q1 = lds128(fragment_addr(queries, i, j, 1, lane));
#pragma unroll
        for (int n = 0; n < 2; ++n) {
          float acc[4];
          mma_first(acc, q0.x, q0.y, q0.z, q0.w, f[n][0], f[n][1]);
          mma_16816(acc, q1.x, q1.y, q1.z, q1.w, f[n][2], f[n][3]);
          const float s0 = j & 1 ? f16_hi(za[n][j >> 1]) : f16_lo(za[n][j >> 1]);
          const float s1 = j & 1 ? f16_hi(zb[n][j >> 1]) : f16_lo(zb[n][j >> 1]);
          s[i][n][0] = j == 0 ? s0 * acc[0] : fmaf(s0, acc[0], s[i][n][0]);
          s[i][n][1] = j == 0 ? s1 * acc[1] : fmaf(s1, acc[1], s[i][n][1]);
          s[i][n][2] = j == 0 ? s0 * acc[2] : fmaf(s0, acc[2], s[i][n][2]);
          s[i][n][3] = j == 0 ? s1 * acc[3] : fmaf(s1, acc[3], s[i][n][3]);
        }
      }
    }
  }
  if (left < 16) {
#pragma unroll
    for (int i = 0; i < MT; ++i)
#pragma unroll
      for (int n = 0; n < 2; ++n)
#pragma unroll
        for (int e = 0; e < 4; ++e)
          if (8 * n + 2 * c + (e & 1) >= left) s[i][n][e] = -INFINITY;
  }
}
// The weights of 16 tokens (a fragment each lane: `weights`) times their values, of which this
// warp has a quarter of the dimensions.  A value word holds four dimensions of two tokens, field
// i dimension 32 j + 4 n + i of column n.  The warp takes two neighbouring words and two
// neighbouring fields, j0, j0 + 1 and i0, i0 + 1: output block 2 y + x, whose columns 2c and
// 2c + 1 are dimensions 32 (j0 + y) + 8 c + i0 + x and 4 more.
__device__ __forceinline__ int first_word() { return 2 * (threadIdx.x >> 5 & 1); }
__device__ __forceinline__ int first_field() { return 2 * (threadIdx.x >> 6); }
__device__ __forceinline__ uint2 lds64(uint32_t a) {
  uint2 v;
  asm volatile("ld.shared.v2.u32 {%0,%1}, [%2];\n" : "=r"(v.x), "=r"(v.y) : "r"(a));
  return v;
}
template <int P, int MT, bool WHOLE>
__device__ __forceinline__ void values_q4(State<MT, true>& st, uint32_t base, int group, uint32_t weights, int left) {
  using At = Q4Tile<P>;
  const int lane = threadIdx.x & 31, c = lane & 3;
  const uint32_t vb = base + At::value_codes(group) + 4 * first_word(), zb = base + At::value_scales(group) + 4 * first_word();
  const uint2 v0 = lds64(vb + lane * 16), v1 = lds64(vb + 512 + lane * 16);
  uint2 z0 = lds64(zb + c * 32), z1 = lds64(zb + c * 32 + 16);
  if constexpr (!WHOLE) {
    // scales past the end may be anything, a NaN too
    const uint32_t m0 = pair_mask(2 * c, left), m1 = pair_mask(8 + 2 * c, left);
    z0.x &= m0; z0.y &= m0;
    z1.x &= m1; z1.y &= m1;
  }
  const uint32_t vw0[2] = {v0.x, v0.y}, vw1[2] = {v1.x, v1.y}, zw0[2] = {z0.x, z0.y}, zw1[2] = {z1.x, z1.y};
  uint4 p[MT];
#pragma unroll
  for (int i = 0; i < MT; ++i) p[i] = lds128(weights + ((group * MT + i) * 32 + lane) * 16);
#pragma unroll
  for (int y = 0; y < 2; ++y) {
    uint32_t f[2], h[2];
    q4_codes01(vw0[y] >> (4 * first_field()), f[0], f[1]);
    q4_codes01(vw1[y] >> (4 * first_field()), h[0], h[1]);
#pragma unroll
    for (int x = 0; x < 2; ++x) {
      const uint32_t f0 = mul_f16x2(f[x], zw0[y]), f1 = mul_f16x2(h[x], zw1[y]);
#pragma unroll
      for (int i = 0; i < MT; ++i) mma_16816_f16(st.o[i][2 * y + x], p[i].x, p[i].y, p[i].z, p[i].w, f0, f1);
    }
  }
}

// False where a wait gave up.
template <int P, bool Q4, int MT>
__device__ __forceinline__ bool run_piece(const GroupArgs& a, const CUtensorMap& tk, const CUtensorMap& tv, const Piece& p, Shared& sh,
                                          uint8_t* ring, uint8_t* queries, uint32_t& seq, float* part_o, float2* part_ml) {
  // (a tile's weights follow the queries)
  constexpr int kPPT = kPage / P, S = kStages<Q4>, kBatch = 32;  // pages of a tile; page entries a warp looks up at once
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31, g = lane >> 2, c = lane & 3;
  const int nt = p.t1 - p.t0, G = sh.grp.g;
  const uint32_t rbase = smem_u32(ring), qbase = smem_u32(queries);

  // Every warp asks for its quarter of a tile: one of four 16-token pages, or one box of a 64-token one
  // (of which 4-bit ones are one copy: the warps take turns).  Its lanes hold 32 pages' entries, and the next 32.
  int cur = 0, nxt = 0, batch = -2, asked = -1;
  auto entry = [&](int k) { return k < p.pages ? p.table[p.page0 + k] : 0; };  // of page k of the piece
  auto issue = [&](int t) {  // whole warps: tile t of the piece
    if (kTurns<P, Q4> && t % kWarps != warp) return;
    const int k0 = t * kPPT, need = k0 / kBatch;
    if (need != batch) {
      cur = need == batch + 1 ? nxt : entry(need * kBatch + lane);
      nxt = entry((need + 1) * kBatch + lane);
      batch = need;
    }
    asked = t;
    const int stage = (seq + t) % S, w = P == kPage ? 0 : warp, k = k0 + w;
    const int phys = __shfl_sync(0xffffffffu, cur, k % kBatch);
    if (lane != 0) return;
    const bool there = k < p.pages, good = there && phys >= 0 && phys < a.pages_total;
    if (there && !good) set_error(a.err, LOCKS_DEVERR_BLOCK_TABLE);
    if (P != kPage || kTurns<P, Q4> || warp == 0) sh.left[stage][w] = good ? min(P, p.limit - (p.page0 + k) * P) : 0;
    if (!there) {
      mbar_arrive(&sh.full[stage]);
      return;
    }
    const size_t ph = (size_t)(good ? phys : 0) * a.num_kv_heads + p.h;  // (a page outside the pool: any, unseen)
    uint8_t* dst = ring + stage * kStageBytes<Q4>;
    mbar_arrive_expect_tx(&sh.full[stage], kStageBytes<Q4> / kAsking<P, Q4>);
    if constexpr (Q4) {
      constexpr int kBytes = LOCKS_KV_Q4_BLOCK_BYTES(P);
      bulk_load(smem_u32(dst + w * kBytes), a.blocks + ph * kBytes, kBytes, &sh.full[stage]);
    } else if constexpr (P == kPage) {
      tma_load_2d(dst + warp * kHalfTile, warp < 2 ? &tk : &tv, &sh.full[stage], 64 * (warp & 1), (int)(ph * P));
    } else {
      const int y = (int)(ph * P);
      uint8_t* d = dst + w * (P * 128);
      tma_load_2d(d, &tk, &sh.full[stage], 0, y);
      tma_load_2d(d + kHalfTile, &tk, &sh.full[stage], 64, y);
      tma_load_2d(d + kTile, &tv, &sh.full[stage], 0, y);
      tma_load_2d(d + kTile + kHalfTile, &tv, &sh.full[stage], 64, y);
    }
  };
  for (int t = 0; t < min(S, nt); ++t) issue(t);
  // the queries; rows past the last are zero
  for (int e = tid; e < MT * 16 * 16; e += kThreads) {
    const int r = e / 16, chunk = e % 16;
    uint4 v = make_uint4(0, 0, 0, 0);
    if (r < p.rows) v = *(reinterpret_cast<const uint4*>(a.q + query_row(a, p, G, r) * kHeadDim) + chunk);
    if constexpr (Q4) {
      // row g (or g + 8) of its tile, dimensions 32 j + 8 c ..: words 0 and 1 for the first step, 2 and 3 for the second
      const uint32_t at = fragment_addr(qbase, r / 16, chunk / 4, 0, r % 8 * 4 + chunk % 4) + r / 8 % 2 * 4;
      sts32(at, v.x);
      sts32(at + 8, v.y);
      sts32(at + 512, v.z);
      sts32(at + 520, v.w);
    } else {
      asm volatile("st.shared.v4.u32 [%0], {%1, %2, %3, %4};\n" ::"r"(query_addr(qbase, r, chunk)), "r"(v.x), "r"(v.y), "r"(v.z), "r"(v.w)
                   : "memory");
    }
  }
  // one head's last warp sees, while the first copies are under way, whether the rows do share
  if (p.shared && p.h == 0 && p.block == 0 && warp == kWarps - 1) {
    bool differs = false;
    for (int k = lane; k < p.pages; k += 32) {
      const int32_t* column = a.block_table + (size_t)G * a.beams * a.max_pages + p.page0 + k;
      const int phys = p.table[p.page0 + k];
#pragma unroll 8
      for (int w = 0; w < a.beams; ++w) differs |= column[(size_t)w * a.max_pages] != phys && sh.grp.len[w] > 0;
    }
    if (differs) set_error(a.err, LOCKS_DEVERR_BLOCK_TABLE);
  }
  __syncthreads();

  State<MT, Q4> st;
  st.reset();
  bool ok = true;
  const uint32_t weights = qbase + kQueryBytes;
  for (int t = 0; t < nt; ++t) {
    const int stage = (seq + t) % S;
    const uint32_t base = rbase + stage * kStageBytes<Q4>;
    if (!__all_sync(0xffffffffu, mbar_wait(&sh.full[stage], ((seq + t) / S) & 1))) {
      if (lane == 0) atomicExch(&sh.abort, 1);
      ok = false;
    }
    // tokens of 16 that are seen
    auto left_of = [&](int group) { return P == kPage ? min(16, sh.left[stage][0] - 16 * group) : sh.left[stage][P == kPage ? 0 : group]; };
    const int left = left_of(warp);
    float s[MT][2][4], top[MT][2];
    if (ok && left > 0) {
      if constexpr (Q4) logits_q4<P, MT>(s, base, qbase, left);
      else logits_bf16<MT>(s, base, qbase, left);
    } else {
#pragma unroll
      for (int i = 0; i < MT; ++i)
#pragma unroll
        for (int e = 0; e < 4; ++e) s[i][0][e] = s[i][1][e] = -INFINITY;
    }
    // the reference of a row is the same in all warps
    const bool moved = __syncthreads_or(st.look(s, a.scale_log2, top));
    ok = *reinterpret_cast<volatile int*>(&sh.abort) == 0;  // (set before the barrier, and not again before the next one)
    if (!ok) break;
    // all warps are done with the tile before this one, and its stage is free
    if (t > 0 && t - 1 + S < nt) issue(t - 1 + S);
    if (moved) {
#pragma unroll
      for (int i = 0; i < MT; ++i)
#pragma unroll
        for (int k = 0; k < 2; ++k) {
          const float x = st.row_top(top[i][k]);
          if (c == 0) sh.m[warp][16 * i + 8 * k + g] = x;
        }
      __syncthreads();
#pragma unroll
      for (int i = 0; i < MT; ++i)
#pragma unroll
        for (int k = 0; k < 2; ++k) {
          float x = -INFINITY;
#pragma unroll
          for (int w = 0; w < kWarps; ++w) x = fmaxf(x, sh.m[w][16 * i + 8 * k + g]);
          st.move(i, k, x);
        }
    }
    st.weigh(s, a.scale_log2);
    auto packed = [](float x, float y) { return Q4 ? pack_f16(x, y) : pack_bf16(x, y); };
#pragma unroll
    for (int i = 0; i < MT; ++i)
      asm volatile("st.shared.v4.u32 [%0], {%1, %2, %3, %4};\n" ::"r"(weights + ((warp * MT + i) * 32 + lane) * 16),
                   "r"(packed(s[i][0][0], s[i][0][1])), "r"(packed(s[i][0][2], s[i][0][3])),
                   "r"(packed(s[i][1][0], s[i][1][1])), "r"(packed(s[i][1][2], s[i][1][3]))
                   : "memory");
    __syncthreads();
    auto values = [&](auto all, int w, int left_w) {
      if constexpr (Q4) values_q4<P, MT, decltype(all)::value>(st, base, w, weights, left_w);
      else values_bf16<MT, decltype(all)::value>(st, base, w, weights, left_w);
    };
    bool whole = true;
#pragma unroll
    for (int w = 0; w < kPPT; ++w) whole &= sh.left[stage][w] >= P;
    if (whole) {
#pragma unroll
      for (int w = 0; w < kWarps; ++w) values(std::true_type(), w, 16);
    } else {
#pragma unroll 1
      for (int w = 0; w < kWarps; ++w)
        if (left_of(w) > 0) values(std::false_type(), w, left_of(w));
    }
  }
  if (!ok) {
    if (lane == 0) {
      atomicExch(&sh.abort, 1);
      set_error(a.err, kDevErrTimeout);
    }
    // the copies that this warp has asked for get a bounded time to land
    for (int t = asked; t >= 0 && t > asked - S; --t) (void)mbar_wait(&sh.full[(seq + t) % S], ((seq + t) / S) & 1);
  }
  seq += nt;
  // ---- the piece's state ----
#pragma unroll
  for (int i = 0; i < MT; ++i)
#pragma unroll
    for (int k = 0; k < 2; ++k) {
      st.l[i][k] += __shfl_xor_sync(0xffffffffu, st.l[i][k], 1);
      st.l[i][k] += __shfl_xor_sync(0xffffffffu, st.l[i][k], 2);
      if (c == 0) {
        if (warp == 0) sh.m[0][16 * i + 8 * k + g] = st.m[i][k];
        sh.l[warp][16 * i + 8 * k + g] = st.l[i][k];
      }
    }
  __syncthreads();  // every warp is done with the ring
  float* so = reinterpret_cast<float*>(ring);
  // of one reference, and each warp has its own columns; the sums are left
#pragma unroll
  for (int i = 0; i < MT; ++i)
#pragma unroll
    for (int k = 0; k < 2; ++k) {
      float* row = so + (16 * i + 8 * k + g) * kOStride<Q4>;
#pragma unroll
      for (int y = 0; y < 2; ++y)
#pragma unroll
        for (int e = 0; e < 2; ++e)
          if constexpr (Q4)
            *reinterpret_cast<float2*>(row + 32 * (first_word() + y) + 8 * c + 4 * e + first_field()) =
                make_float2(st.o[i][2 * y][2 * k + e], st.o[i][2 * y + 1][2 * k + e]);
          else
            *reinterpret_cast<float2*>(row + 32 * warp + 16 * y + 8 * e + 2 * c) =
                make_float2(st.o[i][2 * y + e][2 * k], st.o[i][2 * y + e][2 * k + 1]);
    }
  if (tid < p.rows) {
    float L = 0.f;
#pragma unroll
    for (int w = 0; w < kWarps; ++w) L += sh.l[w][tid];
    part_ml[tid] = make_float2(sh.m[0][tid], L);
  }
  __syncthreads();
  for (int e = tid; e < p.rows * (kHeadDim / 4); e += kThreads)
    reinterpret_cast<float4*>(part_o)[e] = *reinterpret_cast<const float4*>(so + e / (kHeadDim / 4) * kOStride<Q4> + e % (kHeadDim / 4) * 4);
  // the ring was written with ordinary stores: before the next copies into it
  fence_proxy_async();
  __syncthreads();
  return !sh.abort;
}

template <int P, bool Q4>
__global__ void __launch_bounds__(kThreads, kCtas<Q4>) group_attend_kernel(const __grid_constant__ CUtensorMap tk,
                                                                   const __grid_constant__ CUtensorMap tv,
                                                                   const GroupArgs a) {
  constexpr int kPPT = kPage / P;
  extern __shared__ uint8_t dyn_raw[];
  __shared__ Shared sh;
  uint8_t* ring = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(dyn_raw) + 1023) & ~uintptr_t(1023));
  uint8_t* queries = ring + kStages<Q4> * kStageBytes<Q4>;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, cta = blockIdx.x;
  const int groups = a.batch / a.beams;
  if (tid == 0) {
    if constexpr (!Q4) {
      prefetch_tmap(&tk);
      prefetch_tmap(&tv);
    }
    for (int s = 0; s < kStages<Q4>; ++s) mbar_init(&sh.full[s], kAsking<P, Q4>);
    fence_mbar_init();
    sh.abort = 0;
  }
  pdl_wait();
  // the join's CTAs start, and read the lengths, as this kernel's first ones finish
  pdl_launch_dependents();

  uint32_t lo, hi;
  if (groups == 1) {
    if (warp == 0) load_group(a, 0, sh.grp, cta == 0);
    if (tid == 0) sh.group = 0, sh.offset = 0;
    __syncthreads();
    const Parts parts((uint32_t)sh.grp.line * a.num_kv_heads, a.n_ctas);
    lo = parts.begin(cta);
    hi = parts.begin(cta + 1);
  } else {
    // the whole line; few requests: a warp each, else a thread each
    uint32_t total = 0;
    if (groups <= kFewGroups) {
      for (int g = warp; g < groups; g += kWarps) {
        load_group(a, g, sh.few[warp], cta == 0);
        __syncwarp();
        if (lane == 0) sh.lines[g] = (uint32_t)sh.few[warp].line * a.num_kv_heads;
        __syncwarp();
      }
      __syncthreads();
      for (int g = 0; g < groups; ++g) total += sh.lines[g];
    } else {
      uint32_t mine = 0;
      for (int g = tid; g < groups; g += kThreads) mine += (uint32_t)head_line(a, g, cta == 0) * a.num_kv_heads;
      const uint32_t sum = __reduce_add_sync(0xffffffffu, mine);
      if (lane == 0) sh.scan[warp] = sum;
      __syncthreads();
      total = sh.scan[0] + sh.scan[1] + sh.scan[2] + sh.scan[3];
    }
    const Parts parts(total, a.n_ctas);
    lo = parts.begin(cta);
    hi = parts.begin(cta + 1);
    // the request that holds place lo; CTA 0 leaves every request's first place for the join
    uint32_t before = 0;
    for (int g0 = 0; g0 < groups; g0 += kThreads) {
      const int g = g0 + tid;
      const uint32_t own = g >= groups ? 0 : groups <= kFewGroups ? sh.lines[g] : (uint32_t)head_line(a, g, false) * a.num_kv_heads;
      uint32_t upto = own;
#pragma unroll
      for (int d = 1; d < 32; d *= 2) {
        const uint32_t other = __shfl_up_sync(0xffffffffu, upto, d);
        if (lane >= d) upto += other;
      }
      if (groups > 32) {
        __syncthreads();
        if (lane == 31) sh.scan[warp] = upto;
        __syncthreads();
        for (int w = 0; w < kWarps; ++w) upto += w < warp ? sh.scan[w] : 0;
      }
      const uint32_t first = before + upto - own;
      if (lo >= first && lo < first + own) {
        sh.group = g;
        sh.offset = first;
      }
      if (cta == 0 && g < groups) a.offsets[g] = first;
      if (groups > 32) before += sh.scan[0] + sh.scan[1] + sh.scan[2] + sh.scan[3];
      if (cta != 0 && before > lo) break;
    }
    if (cta == 0 && tid == 0) a.offsets[groups] = total;
    __syncthreads();
  }
  if (lo >= hi) return;
  int g = sh.group;
  uint32_t offset = sh.offset, pos = lo, seq = 0;
  auto load = [&] {
    if (warp == 0) load_group(a, g, sh.grp, false);
    __syncthreads();
  };
  if (groups > 1) load();
  const size_t own_base = (size_t)a.n_ctas + (size_t)groups * a.num_kv_heads * a.n_blocks;  // records of shared parts
  while (pos < hi) {
    while (pos >= offset + (uint32_t)sh.grp.line * a.num_kv_heads) {
      offset += (uint32_t)sh.grp.line * a.num_kv_heads;
      ++g;
      __syncthreads();  // all have read the last request's
      load();
    }
    const Group& s = sh.grp;
    Piece p;
    const uint32_t in = pos - offset;
    p.h = (int)(in / (uint32_t)s.line);
    int x = (int)(in - (uint32_t)p.h * s.line);
    const int shared_line = line_of(s.shared_tiles), shared_all = a.n_blocks * shared_line;
    uint32_t start = offset + (uint32_t)p.h * s.line;
    int tiles, end_page;
    p.shared = x < shared_all;
    p.w = p.block = 0;
    if (p.shared) {
      p.block = x / shared_line;
      start += p.block * shared_line;
      tiles = s.shared_tiles;
      p.rows = min(kSharedRows, a.beams * a.group - p.block * kSharedRows);
      p.limit = s.sp * P;
      end_page = s.sp;
      p.table = a.block_table + (size_t)(g * a.beams + s.first) * a.max_pages;
    } else {
      x -= shared_all;
      while (x >= s.upto[p.w]) ++p.w;
      start += shared_all + (p.w ? s.upto[p.w - 1] : 0);
      p.limit = s.len[p.w];
      tiles = tiles_of(p.limit - s.sp * P);
      p.rows = a.group;
      end_page = (p.limit - 1) / P + 1;
      p.table = a.block_table + (size_t)(g * a.beams + p.w) * a.max_pages;
    }
    p.t0 = max(0, (int)(pos - start) - kSegment);
    p.t1 = min(tiles, max(0, (int)(hi - start) - kSegment));
    if (p.t1 > p.t0) {
      p.page0 = (p.shared ? 0 : s.sp) + p.t0 * kPPT;
      p.pages = min(end_page - p.page0, (p.t1 - p.t0) * kPPT);
      const size_t problem = (size_t)g * a.num_kv_heads + p.h;
      size_t row;  // of the partial results
      if (p.shared) row = (cta + problem * a.n_blocks + p.block) * kSharedRows;
      else row = own_base * kSharedRows + (cta + problem * a.beams + p.w) * a.group;
      float* part_o = a.part_o + row * kHeadDim;
      float2* part_ml = a.part_ml + row;
      const bool done = p.rows > 16 ? run_piece<P, Q4, 2>(a, tk, tv, p, sh, ring, queries, seq, part_o, part_ml)
                                    : run_piece<P, Q4, 1>(a, tk, tv, p, sh, ring, queries, seq, part_o, part_ml);
      if (!done) return;
    }
    pos = start + kSegment + tiles;
  }
}

// Joins the pieces of one (row, query head).  Grid (batch * Hkv, group).
constexpr int kJoinWarps = 8;   // at most
constexpr int kJoinFlight = 8;  // pieces that a warp loads at once

__global__ void __launch_bounds__(32 * kJoinWarps) group_join_kernel(const GroupArgs a) {
  __shared__ __align__(16) float so[kJoinWarps][kHeadDim];  // (read and written 16 bytes at a time)
  __shared__ float sl[kJoinWarps];
  __shared__ Group few[kJoinWarps];
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31, warps = blockDim.x >> 5;
  const int b = blockIdx.x / a.num_kv_heads, h = blockIdx.x % a.num_kv_heads, e = blockIdx.y;
  const int g = b / a.beams, w = b % a.beams, groups = a.batch / a.beams;
  // Where the pieces are follows from the lengths, which were complete before the other
  // kernel let this one begin; few requests' are gone through while that one still runs, and with more
  // it is read from what that one leaves.
  const bool known = groups <= min(2 * warps, kJoinWarps);
  if (known)
    for (int i = warp; i < groups; i += warps) load_group(a, i, few[i], false);
  else if (warp == 0) load_group(a, g, few[0], false);
  __syncthreads();
  const Group& s = few[known ? g : 0];
  uint32_t total = 0, first = 0;
  if (known) {
    for (int i = 0; i < groups; ++i) {
      const uint32_t line = (uint32_t)few[i].line * a.num_kv_heads;
      first += i < g ? line : 0;
      total += line;
    }
  } else {
    pdl_wait();
    total = a.offsets[groups];
    first = a.offsets[g];
  }
  const Parts parts(total, a.n_ctas);
  const int len = s.len[w];
  const size_t out_row = ((size_t)b * a.num_kv_heads + h) * a.group + e;
  // the CTAs that have pieces of the two segments
  const int i = w * a.group + e, block = i / kSharedRows;
  const int shared_line = line_of(s.shared_tiles), own_tiles = tiles_of(len - s.sp * a.page_size);
  const uint32_t head = first + (uint32_t)h * s.line;
  const size_t problem = (size_t)g * a.num_kv_heads + h;
  const size_t own_base = (size_t)a.n_ctas + (size_t)groups * a.num_kv_heads * a.n_blocks;
  constexpr uint32_t extra = kSegment;
  uint32_t c0[2] = {0, 0};
  int n[2] = {0, 0};
  auto segment = [&](int k, uint32_t start, int tiles) {
    if (tiles <= 0) return;
    c0[k] = parts.owner(start);
    n[k] = (int)(parts.owner(start + extra + tiles - 1) - c0[k]) + 1;
    // the first of them may end before the first tile
    while (parts.begin(c0[k] + 1) <= start + extra) ++c0[k], --n[k];
  };
  segment(0, head + (uint32_t)block * shared_line, s.shared_tiles);
  segment(1, head + (uint32_t)a.n_blocks * shared_line + (w ? s.upto[w - 1] : 0), own_tiles);
  const size_t slot[2] = {(c0[0] + problem * a.n_blocks + block) * kSharedRows + i % kSharedRows,
                          own_base * kSharedRows + (c0[1] + problem * a.beams + w) * a.group + e};
  const int all = n[0] + n[1];
  if (known) pdl_wait();
  pdl_launch_dependents();
  if (len == 0) {
    for (int d = tid; d < kHeadDim; d += blockDim.x) a.out[out_row * kHeadDim + d] = 0;
    if (a.lse && tid == 0) a.lse[out_row] = -INFINITY;
    return;
  }
  auto row = [&](int k) { return k < n[0] ? slot[0] + (size_t)k * kSharedRows : slot[1] + (size_t)(k - n[0]) * a.group; };
  // a warp takes every so manieth piece, the first of them under way while the reference is found
  float4 v[kJoinFlight];
  float2 ml[kJoinFlight];
  auto fetch = [&](int k0) {
#pragma unroll
    for (int k = 0; k < kJoinFlight; ++k) {
      const int at = k0 + warps * k;
      v[k] = make_float4(0.f, 0.f, 0.f, 0.f);
      ml[k] = make_float2(-INFINITY, 0.f);
      if (at >= all) continue;
      v[k] = __ldcg(reinterpret_cast<const float4*>(a.part_o + row(at) * kHeadDim) + lane);
      ml[k] = __ldcg(a.part_ml + row(at));
    }
  };
  fetch(warp);
  float M = -INFINITY, L = 0.f;
  for (int k = lane; k < all; k += 32) M = fmaxf(M, __ldcg(a.part_ml + row(k)).x);
  M = warp_max(M);
  const float ref = M == -INFINITY ? 0.f : M;
  float4 O = make_float4(0.f, 0.f, 0.f, 0.f);
  for (int k0 = warp; k0 < all; k0 += warps * kJoinFlight) {
    if (k0 != warp) fetch(k0);
#pragma unroll
    for (int k = 0; k < kJoinFlight; ++k) {
      const bool none = ml[k].x == -INFINITY;  // a piece of which the row has seen nothing (or a NaN: its sum)
      const float f = none ? 1.f : fast_exp2(ml[k].x - ref);
      L = fmaf(ml[k].y, f, L);
      O.x = fmaf(v[k].x, f, O.x);
      O.y = fmaf(v[k].y, f, O.y);
      O.z = fmaf(v[k].z, f, O.z);
      O.w = fmaf(v[k].w, f, O.w);
    }
  }
  *reinterpret_cast<float4*>(&so[warp][4 * lane]) = O;
  if (lane == 0) sl[warp] = L;
  __syncthreads();
  float Ls = 0.f;
  for (int k = 0; k < warps; ++k) Ls += sl[k];
  for (int d = tid; d < kHeadDim; d += blockDim.x) {
    float Os = 0.f;
    for (int k = 0; k < warps; ++k) Os += so[k][d];
    const float val = Ls == 0.f ? 0.f : Os / Ls;  // a NaN stays one
    a.out[out_row * kHeadDim + d] = __bfloat16_as_ushort(__float2bfloat16_rn(val));
  }
  if (a.lse && tid == 0) a.lse[out_row] = Ls == 0.f ? -INFINITY : (M + log2f(Ls)) * kLn2;
}

template <int P, bool Q4>
cudaError_t launch(const GroupArgs& a, const CUtensorMap& tk, const CUtensorMap& tv, cudaStream_t s) {
  auto kern = group_attend_kernel<P, Q4>;
  const cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, kSmem<Q4>);
  if (e != cudaSuccess) return e;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(a.n_ctas, 1, 1);
  cfg.blockDim = dim3(kThreads, 1, 1);
  cfg.dynamicSmemBytes = kSmem<Q4>;
  cfg.stream = s;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, kern, tk, tv, a);
}

}  // namespace

int group_attend_ctas_per_sm(bool q4) { return q4 ? kCtas<true> : kCtas<false>; }

// Warps per result: few results take their pieces side by side, many need few warps each.
// Measured, the whole call in us (8, 4, 2, 1 warps): 256 results of 2 K 12.2, 11.9, 13.1, 14.1, of 32 K
// in 4 bits 29.3, 30.4, 32.6, 36.9; 512 of 32 K 50.5, 47.2, 48.4, 50.0; 1024 of 16 K, 4-bit, 49.2, 43.6, 41.2,
// 44.5; 2048 of 3 K 62.9, 51.0, 47.6, 44.8.
static int join_warps(const GroupArgs& a) {
  const long long results = (long long)a.batch * a.num_kv_heads * a.group, n = a.n_ctas;
  return results <= n ? kJoinWarps : results <= 2 * n ? 4 : results <= 4 * n ? 2 : 1;
}

cudaError_t launch_group_attend(const GroupArgs& a, const CUtensorMap& tk, const CUtensorMap& tv, cudaStream_t s) {
  const cudaError_t e = a.q4 ? (a.page_size == 16 ? launch<16, true>(a, tk, tv, s) : launch<64, true>(a, tk, tv, s))
                             : (a.page_size == 16 ? launch<16, false>(a, tk, tv, s) : launch<64, false>(a, tk, tv, s));
  if (e != cudaSuccess) return e;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(a.batch * a.num_kv_heads, a.group, 1);
  cfg.blockDim = dim3(32 * join_warps(a), 1, 1);
  cfg.stream = s;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, group_join_kernel, a);
}

}  // namespace locks
