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
// 64 tokens at a time from a ring that bulk and tensor copies fill, warp w tokens 16 w ..
// 16 w + 15, with the softmax and the outputs of its tokens in registers; the warps' states
// meet in shared memory at the end of a piece.  The queries stay in shared memory (their
// fragments would take 64 more registers than there are).  bf16 pages: ldmatrix.
// 4-bit pages: keys' codes are bf16 numbers (exact) and get their scale on the four partial
// sums of a logit; values are s * code rounded to half precision (2^-11), and so are the weights.
//
// Work split.  All 64-token tiles of all problems lie in one line: request by request, KV
// head by head, first the shared pages (once per block of 32 rows), then each row's own.  Every
// CTA gets an equal part of it, two CTAs per SM; a segment counts a few tiles more
// than it has, which is what its queries, its first copies and its merge cost.  A piece
// (the part of a segment that a CTA has) leaves its state in the workspace at place
// CTA + segment, which no two pieces share; a second, dependent kernel joins them.
//
// Measured, 32 query / 8 KV heads (floor by bytes): eight rows that share 32 K tokens of bf16
// pages and have 300 of their own 33.9 us (21.2; every row by itself 83); 131 K shared 89 us (79.6; 274);
// four rows of 2 K 11 us.  Four requests of eight rows, up to 16 K tokens of 4-bit pages 41 us, 16-token
// ones 45 us (8.1; 72 and 79): 32 rows per key make the instructions the bound there (35% of the issue
// slots with two warps per scheduler, which is what 255 registers leave).
#include <algorithm>
#include <climits>

#include "gen.h"
#include "kv_q4.cuh"

namespace locks {

namespace {

constexpr int kWarps = 4;
constexpr int kThreads = kWarps * 32;
// Places that a segment has beyond its tiles.  Measured (2, 3, 4): bf16 pages, 131,000 shared
// tokens 99, 91, 93 us, 32 K 34.4, 33.6, 33.6; 4-bit, four requests of 16 K 51.5, 52.9, 54.1.
constexpr int kSegmentBf16 = 3, kSegmentQ4 = 2;
constexpr int kHalfTile = 64 * 128;   // bytes of a 64-row x 64-column bf16 box
constexpr int kTile = 2 * kHalfTile;  // 64 tokens of K (or V)
constexpr int kQueryBytes = kSharedRows * kHeadDim * 2;
template <bool Q4>
constexpr int kOStride = Q4 ? 132 : 136;  // padded row of a warp's outputs (floats): no two lanes' stores meet in a bank
template <bool Q4>
constexpr int kStageBytes = Q4 ? kQ4Slot : 2 * kTile;
template <bool Q4>
constexpr int kStages = Q4 ? 8 : 3;
template <bool Q4>
constexpr int kSmem = kStages<Q4> * kStageBytes<Q4> + kQueryBytes + 1024;
static_assert(kWarps * kSharedRows * kOStride<true> * 4 <= kStages<true> * kStageBytes<true> &&
                  kWarps * kSharedRows * kOStride<false> * 4 <= kStages<false> * kStageBytes<false>,
              "the merge fits the ring");

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
__device__ __forceinline__ int segment_of(const GroupArgs& a) { return a.q4 ? kSegmentQ4 : kSegmentBf16; }
__device__ __forceinline__ int line_of(const GroupArgs& a, int tiles) { return tiles > 0 ? tiles + segment_of(a) : 0; }

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
  int n = a.n_blocks * line_of(a, tiles_of(sp * a.page_size));
#pragma unroll 8
  for (int w = 0; w < a.beams; ++w) n += line_of(a, tiles_of(row_length(a, base + w, false) - sp * a.page_size));
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
  int upto = line_of(a, tiles_of(len > 0 ? len - sp * a.page_size : 0));
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
    s.line = upto + a.n_blocks * line_of(a, s.shared_tiles);
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
  uint64_t full[8], empty[8];
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

// Address of 16 bytes (chunk) of a query: bf16 pages read them by ldmatrix, 8 rows of one
// chunk together; 4-bit pages as 16 bytes per lane, two rows of four chunks.
template <bool Q4>
__device__ __forceinline__ uint32_t query_addr(uint32_t base, int row, int chunk) {
  return base + row * 256 + ((chunk ^ (Q4 ? (row & 1) * 4 : row & 7)) << 4);
}
__device__ __forceinline__ uint32_t tile_addr(uint32_t base, int row, int chunk) {
  return base + (chunk >> 3) * kHalfTile + row * 128 + (((chunk & 7) ^ (row & 7)) << 4);
}
// Mask of a packed pair of tokens (t, t + 1) that keeps those before `len`.
__device__ __forceinline__ uint32_t pair_mask(int t, int len) {
  return (t < len ? 0x0000ffffu : 0u) | (t + 1 < len ? 0xffff0000u : 0u);
}

// A warp's softmax state and outputs for its tokens: rows 16 i + g, 16 i + g + 8.  m is the
// reference of a row's weights 2^(s - m): the largest logit when it was set, less kBelow.
// It moves only when a weight would exceed 2^kLimit, so the usual tile needs no maximum
// across lanes, only a vote.  bf16 weights: any range will do.  Half-precision ones: the
// largest lies between 2^7 and 2^15, so those below 2^-32 of it are what is lost.
template <int MT, bool Q4>
struct State {
  static constexpr float kBelow = Q4 ? 7.f : 0.f, kLimit = Q4 ? 15.f : 8.f;
  float m[MT][2], l[MT][2];
  float o[MT][16][4];
  __device__ __forceinline__ void reset() {
#pragma unroll
    for (int i = 0; i < MT; ++i) {
      m[i][0] = m[i][1] = -INFINITY;
      l[i][0] = l[i][1] = 0.f;
#pragma unroll
      for (int n = 0; n < 16; ++n) o[i][n][0] = o[i][n][1] = o[i][n][2] = o[i][n][3] = 0.f;
    }
  }
  // Logits (unscaled) to weights.
  __device__ __forceinline__ void weigh(float (&s)[MT][2][4], float scale_log2) {
    bool moved = false;
    float top[MT][2];
#pragma unroll
    for (int i = 0; i < MT; ++i)
#pragma unroll
      for (int k = 0; k < 2; ++k) {
        top[i][k] = fmaxf(fmaxf(s[i][0][2 * k], s[i][0][2 * k + 1]), fmaxf(s[i][1][2 * k], s[i][1][2 * k + 1])) * scale_log2;
        moved |= top[i][k] > m[i][k] + kLimit;
      }
    if (__any_sync(0xffffffffu, moved)) {
#pragma unroll
      for (int i = 0; i < MT; ++i)
#pragma unroll
        for (int k = 0; k < 2; ++k) {
          float t = fmaxf(top[i][k], __shfl_xor_sync(0xffffffffu, top[i][k], 1));
          t = fmaxf(t, __shfl_xor_sync(0xffffffffu, t, 2));
          t = fmaxf(t - kBelow, m[i][k]);
          const float al = t == -INFINITY ? 1.f : fast_exp2(m[i][k] - t);
          m[i][k] = t;
          l[i][k] *= al;
#pragma unroll
          for (int n = 0; n < 16; ++n) {
            o[i][n][2 * k] *= al;
            o[i][n][2 * k + 1] *= al;
          }
        }
    }
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

// Tokens 16 warp .. + 15 of a tile of bf16 pages at `base` (keys, then values), of which the
// first `left` are seen.
template <int MT, bool WHOLE>
__device__ __forceinline__ void tile_bf16(State<MT, false>& st, uint32_t base, uint32_t queries, int left, float scale_log2) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, c = lane & 3, mi = lane >> 3;
  float s[MT][2][4];
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
      ldmatrix_x4(a0, a1, a2, a3, query_addr<false>(queries, 16 * i + (mi & 1) * 8 + (lane & 7), 2 * kk + (mi >> 1)));
      mma_16816(s[i][0], a0, a1, a2, a3, b0, b1);
      mma_16816(s[i][1], a0, a1, a2, a3, b2, b3);
    }
  }
  if constexpr (!WHOLE) {
#pragma unroll
    for (int i = 0; i < MT; ++i)
#pragma unroll
      for (int n = 0; n < 2; ++n)
#pragma unroll
        for (int e = 0; e < 4; ++e)
          if (8 * n + 2 * c + (e & 1) >= left) s[i][n][e] = -INFINITY;
  }
  st.weigh(s, scale_log2);
  uint32_t p[MT][4];
#pragma unroll
  for (int i = 0; i < MT; ++i) {
    p[i][0] = pack_bf16(s[i][0][0], s[i][0][1]);
    p[i][1] = pack_bf16(s[i][0][2], s[i][0][3]);
    p[i][2] = pack_bf16(s[i][1][0], s[i][1][1]);
    p[i][3] = pack_bf16(s[i][1][2], s[i][1][3]);
  }
  const int vrow = 16 * warp + (mi & 1) * 8 + (lane & 7);
  const uint32_t k0 = WHOLE ? ~0u : pair_mask(2 * c, left), k1 = WHOLE ? ~0u : pair_mask(8 + 2 * c, left);
#pragma unroll
  for (int dn = 0; dn < 8; ++dn) {
    uint32_t v0, v1, v2, v3;
    ldmatrix_x4_trans(v0, v1, v2, v3, tile_addr(base + kTile, vrow, 2 * dn + (mi >> 1)));
    if constexpr (!WHOLE) v0 &= k0, v1 &= k1, v2 &= k0, v3 &= k1;  // what lies past the end may be anything
#pragma unroll
    for (int i = 0; i < MT; ++i) {
      mma_16816(st.o[i][2 * dn], p[i][0], p[i][1], p[i][2], p[i][3], v0, v1);
      mma_16816(st.o[i][2 * dn + 1], p[i][0], p[i][1], p[i][2], p[i][3], v2, v3);
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

// The same of 4-bit pages.  A key word holds dimensions 32 j + 8 c .. + 7 of one token, field
// i the pair 8 c + 2 i, + 1, so fields 0 and 1 are one step of a product, 2 and 3 the next; the
// queries are read in that order.  A value word holds four dimensions of two tokens, field
// i dimension 32 j + 4 n + i of column n: output block 4 j + i, whose columns 2c and 2c + 1 are
// dimensions 32 j + 8 c + i and 32 j + 8 c + 4 + i.
template <int P, int MT, bool WHOLE>
__device__ __forceinline__ void tile_q4(State<MT, true>& st, uint32_t base, uint32_t queries, int left, float scale_log2) {
  using At = Q4Tile<P>;
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, g = lane >> 2, c = lane & 3;
  float s[MT][2][4];
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
        const uint4 qa = lds128(query_addr<true>(queries, 16 * i + g, 4 * j + c));
        const uint4 qb = lds128(query_addr<true>(queries, 16 * i + g + 8, 4 * j + c));
#pragma unroll
        for (int n = 0; n < 2; ++n) {
          float acc[4];
          mma_first(acc, qa.x, qb.x, qa.y, qb.y, f[n][0], f[n][1]);
          mma_16816(acc, qa.z, qb.z, qa.w, qb.w, f[n][2], f[n][3]);
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
  if constexpr (!WHOLE) {
#pragma unroll
    for (int i = 0; i < MT; ++i)
#pragma unroll
      for (int n = 0; n < 2; ++n)
#pragma unroll
        for (int e = 0; e < 4; ++e)
          if (8 * n + 2 * c + (e & 1) >= left) s[i][n][e] = -INFINITY;
  }
  st.weigh(s, scale_log2);
  const uint32_t vb = base + At::value_codes(warp), zb = base + At::value_scales(warp);
  const uint4 v0 = lds128(vb + lane * 16), v1 = lds128(vb + 512 + lane * 16);
  uint4 z0 = lds128(zb + c * 32), z1 = lds128(zb + c * 32 + 16);
  if constexpr (!WHOLE) {
    // scales past the end may be anything, a NaN too
    const uint32_t m0 = pair_mask(2 * c, left), m1 = pair_mask(8 + 2 * c, left);
    z0.x &= m0; z0.y &= m0; z0.z &= m0; z0.w &= m0;
    z1.x &= m1; z1.y &= m1; z1.z &= m1; z1.w &= m1;
  }
  const uint32_t vw0[4] = {v0.x, v0.y, v0.z, v0.w}, vw1[4] = {v1.x, v1.y, v1.z, v1.w};
  const uint32_t zw0[4] = {z0.x, z0.y, z0.z, z0.w}, zw1[4] = {z1.x, z1.y, z1.z, z1.w};
  uint32_t p[MT][4];
#pragma unroll
  for (int i = 0; i < MT; ++i) {
    p[i][0] = pack_f16(s[i][0][0], s[i][0][1]);
    p[i][1] = pack_f16(s[i][0][2], s[i][0][3]);
    p[i][2] = pack_f16(s[i][1][0], s[i][1][1]);
    p[i][3] = pack_f16(s[i][1][2], s[i][1][3]);
  }
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    uint32_t f[4], h[4];
    q4_codes01(vw0[j], f[0], f[1]);
    q4_codes01(vw0[j] >> 8, f[2], f[3]);
    q4_codes01(vw1[j], h[0], h[1]);
    q4_codes01(vw1[j] >> 8, h[2], h[3]);
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      const uint32_t f0 = mul_f16x2(f[k], zw0[j]), f1 = mul_f16x2(h[k], zw1[j]);
#pragma unroll
      for (int i = 0; i < MT; ++i) mma_16816_f16(st.o[i][4 * j + k], p[i][0], p[i][1], p[i][2], p[i][3], f0, f1);
    }
  }
}

// False where a wait gave up.
template <int P, bool Q4, int MT>
__device__ __forceinline__ bool run_piece(const GroupArgs& a, const CUtensorMap& tk, const CUtensorMap& tv, const Piece& p, Shared& sh,
                                          uint8_t* ring, uint8_t* queries, uint32_t& seq, float* part_o, float2* part_ml) {
  constexpr int kPPT = kPage / P, S = kStages<Q4>, kBatch = 32;  // pages of a tile; page entries a warp looks up at once
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31, g = lane >> 2, c = lane & 3;
  const int nt = p.t1 - p.t0, G = sh.grp.g;
  const uint32_t rbase = smem_u32(ring), qbase = smem_u32(queries);

  // The warps take turns at asking for the copies, tile t warp t % kWarps; their lanes hold
  // 32 pages' entries, and the next 32.
  int cur = 0, nxt = 0, batch = -2, asked = -1;
  auto entry = [&](int k) { return k < p.pages ? p.table[p.page0 + k] : 0; };  // of page k of the piece
  auto issue = [&](int t) {  // whole warps: tile t of the piece
    const int k0 = t * kPPT, need = k0 / kBatch;
    if (need != batch) {
      cur = need == batch + 1 ? nxt : entry(need * kBatch + lane);
      nxt = entry((need + 1) * kBatch + lane);
      batch = need;
    }
    asked = t;
    const int stage = (seq + t) % S;
    const int np = min(kPPT, p.pages - k0);
    uint8_t* dst = ring + stage * kStageBytes<Q4>;
    int mine = __shfl_sync(0xffffffffu, cur, (k0 + lane % kPPT) % kBatch);  // lane w: page w of the tile
    if (mine < 0 || mine >= a.pages_total) {
      if (lane < np) set_error(a.err, LOCKS_DEVERR_BLOCK_TABLE);
      mine = -1;
    }
    if (lane < kPPT) sh.left[stage][lane] = lane < np && mine >= 0 ? min(P, p.limit - (p.page0 + k0 + lane) * P) : 0;
    __syncwarp();  // before the arrival, which releases it
    if (lane == 0) mbar_arrive_expect_tx(&sh.full[stage], (uint32_t)np * (Q4 ? LOCKS_KV_Q4_BLOCK_BYTES(P) : 2 * P * kHeadDim * 2));
#pragma unroll
    for (int w = 0; w < kPPT; ++w) {
      const int phys = __shfl_sync(0xffffffffu, mine, w);
      if (lane == 0 && w < np) {
        const size_t ph = (size_t)max(phys, 0) * a.num_kv_heads + p.h;  // (a page outside the pool: any, unseen)
        if constexpr (Q4) {
          bulk_load(smem_u32(dst + w * LOCKS_KV_Q4_BLOCK_BYTES(P)), a.blocks + ph * LOCKS_KV_Q4_BLOCK_BYTES(P),
                    LOCKS_KV_Q4_BLOCK_BYTES(P), &sh.full[stage]);
        } else {
          const int y = (int)(ph * P);
          uint8_t* d = dst + w * (P * 128);
          tma_load_2d(d, &tk, &sh.full[stage], 0, y);
          tma_load_2d(d + kHalfTile, &tk, &sh.full[stage], 64, y);
          tma_load_2d(d + kTile, &tv, &sh.full[stage], 0, y);
          tma_load_2d(d + kTile + kHalfTile, &tv, &sh.full[stage], 64, y);
        }
      }
    }
  };
  for (int t = warp; t < min(S, nt); t += kWarps) issue(t);
  // the queries; rows past the last are zero
  for (int e = tid; e < MT * 16 * 16; e += kThreads) {
    const int r = e / 16, chunk = e % 16;
    uint4 v = make_uint4(0, 0, 0, 0);
    if (r < p.rows) v = *(reinterpret_cast<const uint4*>(a.q + query_row(a, p, G, r) * kHeadDim) + chunk);
    const uint32_t at = query_addr<Q4>(qbase, r, chunk);
    asm volatile("st.shared.v4.u32 [%0], {%1, %2, %3, %4};\n" ::"r"(at), "r"(v.x), "r"(v.y), "r"(v.z), "r"(v.w) : "memory");
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
  for (int t = 0; t < nt; ++t) {
    const int ahead = t - 1 + S;
    if (t > 0 && ahead < nt && ahead % kWarps == warp) {
      // into the stage of the tile before this one, when all warps are done with it
      ok = mbar_wait(&sh.empty[(seq + t - 1) % S], ((seq + t - 1) / S) & 1);
      if (!ok) break;
      issue(ahead);
    }
    const int stage = (seq + t) % S;
    ok = mbar_wait(&sh.full[stage], ((seq + t) / S) & 1);
    if (!ok) break;
    const int left = P == kPage ? min(16, sh.left[stage][0] - 16 * warp) : sh.left[stage][P == kPage ? 0 : warp];
    const uint32_t base = rbase + stage * kStageBytes<Q4>;
    if constexpr (Q4) {
      if (left >= 16) tile_q4<P, MT, true>(st, base, qbase, 16, a.scale_log2);
      else if (left > 0) tile_q4<P, MT, false>(st, base, qbase, left, a.scale_log2);
    } else {
      if (left >= 16) tile_bf16<MT, true>(st, base, qbase, 16, a.scale_log2);
      else if (left > 0) tile_bf16<MT, false>(st, base, qbase, left, a.scale_log2);
    }
    __syncwarp();
    if (lane == 0) mbar_arrive(&sh.empty[stage]);
  }
  if (!ok) {
    if (lane == 0) {
      atomicExch(&sh.abort, 1);
      set_error(a.err, kDevErrTimeout);
    }
    // the copies that this warp has asked for get a bounded time to land
    for (int t = asked; t >= 0 && t > asked - S; t -= kWarps) (void)mbar_wait(&sh.full[(seq + t) % S], ((seq + t) / S) & 1);
  }
  seq += nt;
  // ---- the warps' states, merged ----
#pragma unroll
  for (int i = 0; i < MT; ++i)
#pragma unroll
    for (int k = 0; k < 2; ++k) {
      st.l[i][k] += __shfl_xor_sync(0xffffffffu, st.l[i][k], 1);
      st.l[i][k] += __shfl_xor_sync(0xffffffffu, st.l[i][k], 2);
      if (c == 0) {
        sh.m[warp][16 * i + 8 * k + g] = st.m[i][k];
        sh.l[warp][16 * i + 8 * k + g] = st.l[i][k];
      }
    }
  __syncthreads();  // every warp is done with the ring
  float* so = reinterpret_cast<float*>(ring);
#pragma unroll
  for (int i = 0; i < MT; ++i)
#pragma unroll
    for (int k = 0; k < 2; ++k) {
      const int r = 16 * i + 8 * k + g;
      float M = -INFINITY;
#pragma unroll
      for (int w = 0; w < kWarps; ++w) M = fmaxf(M, sh.m[w][r]);
      const float f = M == -INFINITY ? 1.f : fast_exp2(st.m[i][k] - M);
      float* row = so + (warp * kSharedRows + r) * kOStride<Q4>;
      if constexpr (Q4) {
#pragma unroll
        for (int j = 0; j < 4; ++j)
#pragma unroll
          for (int e = 0; e < 2; ++e)
            *reinterpret_cast<float4*>(row + 32 * j + 8 * c + 4 * e) =
                make_float4(f * st.o[i][4 * j][2 * k + e], f * st.o[i][4 * j + 1][2 * k + e],
                            f * st.o[i][4 * j + 2][2 * k + e], f * st.o[i][4 * j + 3][2 * k + e]);
      } else {
#pragma unroll
        for (int n = 0; n < 16; ++n)
          *reinterpret_cast<float2*>(row + 8 * n + 2 * c) = make_float2(f * st.o[i][n][2 * k], f * st.o[i][n][2 * k + 1]);
      }
    }
  if (tid < p.rows) {
    float M = -INFINITY, L = 0.f;
#pragma unroll
    for (int w = 0; w < kWarps; ++w) M = fmaxf(M, sh.m[w][tid]);
#pragma unroll
    for (int w = 0; w < kWarps; ++w) L = fmaf(sh.l[w][tid], M == -INFINITY ? 1.f : fast_exp2(sh.m[w][tid] - M), L);
    part_ml[tid] = make_float2(M, L);
  }
  __syncthreads();
  for (int e = tid; e < p.rows * (kHeadDim / 4); e += kThreads) {
    const float* at = so + e / (kHeadDim / 4) * kOStride<Q4> + e % (kHeadDim / 4) * 4;
    float4 O = *reinterpret_cast<const float4*>(at);
#pragma unroll
    for (int w = 1; w < kWarps; ++w) {
      const float4 v = *reinterpret_cast<const float4*>(at + w * kSharedRows * kOStride<Q4>);
      O = make_float4(O.x + v.x, O.y + v.y, O.z + v.z, O.w + v.w);
    }
    reinterpret_cast<float4*>(part_o)[e] = O;
  }
  // the ring was written with ordinary stores: before the next copies into it
  fence_proxy_async();
  __syncthreads();
  return !sh.abort;
}

template <int P, bool Q4>
__global__ void __launch_bounds__(kThreads, 2) group_attend_kernel(const __grid_constant__ CUtensorMap tk,
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
    for (int s = 0; s < kStages<Q4>; ++s) {
      mbar_init(&sh.full[s], 1);
      mbar_init(&sh.empty[s], kWarps);
    }
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
  constexpr int kSegment = Q4 ? kSegmentQ4 : kSegmentBf16;
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
    const int shared_line = line_of(a, s.shared_tiles), shared_all = a.n_blocks * shared_line;
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
  const int shared_line = line_of(a, s.shared_tiles), own_tiles = tiles_of(len - s.sp * a.page_size);
  const uint32_t head = first + (uint32_t)h * s.line;
  const size_t problem = (size_t)g * a.num_kv_heads + h;
  const size_t own_base = (size_t)a.n_ctas + (size_t)groups * a.num_kv_heads * a.n_blocks;
  const uint32_t extra = segment_of(a);
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

int group_attend_ctas_per_sm() { return 2; }

// Warps per result: few results take their pieces side by side, many need few warps each.
// Measured, the whole call in us (8, 4, 2, 1 warps): 128 results of 2 K 11.9, 12.1, 13.2, 14.5; 512
// of 32 K 46.0, 43.4, 44.6, 45.8; 1024 of 16 K, 4-bit, 54.6, 48.6, 46.0, 47.0; 2048 of 3 K 62.4,
// 50.3, 47.2, 44.1.
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
