// Causal attention of the newest tokens of every sequence over the paged cache
// (a prompt, the next chunk of one, or a few draft tokens), bf16 or 4-bit pages.
//
// Mathematics.  Rows are (token, query head of the group): the G heads of a KV head
// share its keys, so a tile of 128 rows holds 128 / G tokens and its products are
// S = Q K^T and O += P V with the online softmax between them; row r of token i at
// position p sees the keys t <= p.
//
// What bounds it: 4 * 128 operations per visible (row, key) at the tensor cores'
// rate; for few rows over a long cache, the cache's bytes.
//
// Layout.  Tensor memory (512 columns): two S buffers of 128 columns, whose first 64
// columns P overwrites (16-bit pairs, the A operand of the second product), and one or
// two O of 128 columns.  Keys and values come as 32 KiB operands (128 tokens in the
// instructions' 128-byte swizzle) through a ring of five or six, so that copies run one
// to two blocks ahead.  Warps: 0 issues the matrix instructions, 1 the copies, 4 and up
// are the softmax of a tile, one thread per row, so neither maximum nor sum needs a
// shuffle.  Matrix instructions of one CTA execute in the order of issue, so S of the
// next block may be issued right behind the product that reads P from the same
// columns.  O is rescaled in place by the softmax warps, and only when a row's
// maximum has grown by more than 2^8 since its last reference.
//
// Three sources of the operands:
//  - bf16 pages: TMA copies of the pages (64-column boxes).  A CTA takes two tiles
//    (256 rows), so that one tile's softmax runs while the other's products do.  Pages of
//    16 tokens make 64 copies of 2 KiB per block, which at some 37 ns each take twice as
//    long as its products: with many rows one kernel first gathers keys and values into
//    planes, of which a block is eight copies.  Up to 128 rows: a CTA takes one tile and
//    both S buffers, so that S of the next block is made while the softmax of this one
//    runs; its queries are in tensor memory.
//  - 4-bit pages, many rows: each key is needed by many CTAs, so one kernel first
//    writes the sequence's keys and values as fp16 planes into the workspace, and
//    TMA copies fetch those; else as above.
//  - 4-bit pages, few rows: eight warps turn the pages' codes into operands in shared
//    memory, for one tile per CTA in the same way.
// Precision.  S, O, maxima and sums are fp32.  bf16 pages: both operands of a matrix
// instruction have one type, so with bf16 values the softmax weights are rounded to bf16
// too (2^-8 of each; the sum that divides them is of the unrounded ones): 2048 new tokens
// over 30,011 keys are off by 0.0023 of the result where fp32 weights are by 0.0017, the
// outputs' own rounding included in both.
// fp16 operands (4-bit pages): q is scaled by a power of two.  A key s * code has up to 14
// significant bits: it is held as the nearest half and the remainder, both exact, and
// S is the sum of the products with both (one half alone would put 2^-11 of
// sum |q||k| into every logit).  Values are s * code rounded once (2^-11), weights are
// scaled by 2^6, so that those 2^-30 of the largest still count.
//
// Values that a row does not see must not reach it, not even as 0 * NaN: in the
// blocks that straddle a tile's diagonal or the end of the sequence, value rows past
// the end are zeroed in shared memory, and the infinities and NaN of tokens that not
// every row sees are zeroed there too and added, as they are, to the rows that do see
// the token at the end.
//
// Few row tiles, or some left over after whole waves of CTAs: the keys of a tile are cut
// among several CTAs, whose partial (reference, sum, O) go to the workspace; a second,
// dependent kernel joins them, a warp per row.  (The last CTA to finish did it before, alone: 64 tokens over 131,000, 8 KV
// heads, 260 us, now 154.)
//
// Measured, 32 heads over 8 KV heads, on changing inputs: 2048 new tokens of two sequences
// over caches of up to 30,011, bf16, 1136 us, 1290 TFLOP/s (0.68 of the library product's
// burst rate); a prompt of 8191 tokens, 4-bit pages, 644 us, 853 TFLOP/s counted, 1280 with
// the keys' second halves.  What is left is the chain of a tile, softmax (1400 clocks of some
// 3000 per block), notice, products, notice, which the other tile's products fill only in
// part; a third tile has no room in tensor memory.
#include "common.cuh"
#include "kernels.h"
#include "kv_q4.cuh"
#include "tcgen05.cuh"

namespace locks {

namespace {

constexpr int kRows = 128;                   // rows of a tile
constexpr int kBlock = 128;                  // keys of a block
constexpr int kHalf = kBlock * 128;          // bytes of 64 columns of 128 16-bit rows
constexpr int kOperand = 2 * kHalf;          // one tile of Q, K or V: 32 KiB
constexpr int kRawSlots = 3;                 // 4-bit pages: 64-token slots of codes
constexpr int kSkipRing = 8;                 // the copies run at most five operands ahead of the products
constexpr int kMaxBad = 2 * kRows;           // tokens near a diagonal: no more than a CTA has
constexpr float kLazy = 8.f;                 // growth of a maximum (base 2) that O's reference tolerates
constexpr uint32_t kTmemCols = 512;
constexpr uint32_t kTmemO = 256;             // S: columns 0 and 128; O: 256 and 384
constexpr uint32_t kTmemQ = 384;             // one tile: the queries, in place of a second O

// Where the operands come from.
enum Source { kBf16Pages, kBf16Few, kBf16Planes, kPlanes, kCodes };
template <Source S>
constexpr bool kIsBf16 = S == kBf16Pages || S == kBf16Few || S == kBf16Planes;  // else fp16
template <Source S>
constexpr int kTiles = S == kCodes || S == kBf16Few ? 1 : 2;  // tiles of a CTA
template <Source S>
constexpr int kQueryTiles = kTiles<S> == 1 ? 0 : 2;  // of those, in shared memory (else in tensor memory)
template <Source S>
constexpr int kUnits = kIsBf16<S> ? 2 : 3;  // operands of a block: keys (two halves), values
// With three operands of a block the ring of five is short of one: the second half of the
// next keys lands in the place of this block's values.  It is asked for as soon as those
// are used, and waited for only when it is needed.
template <Source S>
constexpr bool kLateKeys = kTiles<S> == 2 && kUnits<S> == 3;
// Operands in the ring of keys and values.
template <Source S>
constexpr int kSlots = kTiles<S> == 1 ? 6 : 5;
constexpr int kMaxSlots = 6;
template <Source S>
constexpr int kThreadsOf = S == kCodes ? 512 : S == kBf16Few ? 256 : 384;

struct PromptShared {
  uint64_t q_full, full[kMaxSlots];
  // done[n % 4]: the products with the values of block n and the keys of block n + 1
  // are complete (the ring holds fewer than four blocks, so no waiter can be a whole turn
  // behind)
  uint64_t s_full[2], p_ready[2], o_full[2], done[4], drain;
  uint64_t v_free[2];  // kLateKeys: the products with the values of block n are complete
  uint64_t raw_full[kRawSlots], raw_empty[kRawSlots];
  uint32_t tmem;
  int skip[2][kSkipRing];   // per half of a block: 16-token groups whose page is outside the pool (bits)
  int raw_skip[kRawSlots];  // the same of a slot of codes
  int abort;                // a bounded wait gave up
  int n_bad, bad[kMaxBad];
};

// Waits for phase `parity`; gives up after the iteration limit, or once another
// role has given up.
__device__ __forceinline__ bool wait_bar(uint64_t* bar, uint32_t parity, PromptShared& sh) {
  const uint32_t addr = smem_u32(bar);
  for (uint32_t it = 0; it < kMbarSpinLimit; ++it) {
    uint32_t done;
    asm volatile(
        "{\n .reg .pred p;\n mbarrier.try_wait.parity.shared::cta.b64 p, [%1], %2;\n selp.u32 %0, 1, 0, p;\n}\n"
        : "=r"(done)
        : "r"(addr), "r"(parity)
        : "memory");
    if (done) return true;
    if (*reinterpret_cast<volatile int*>(&sh.abort)) return false;
  }
  *reinterpret_cast<volatile int*>(&sh.abort) = 1;
  return false;
}

// The same for a phase that is due soon: by testing, without being put to sleep.
__device__ __forceinline__ bool spin_bar(uint64_t* bar, uint32_t parity, PromptShared& sh) {
  for (uint32_t it = 0; it < kMbarSpinLimit; ++it) {
    if (mbar_test(bar, parity)) return true;
    if ((it & 63) == 63 && *reinterpret_cast<volatile int*>(&sh.abort)) return false;
  }
  *reinterpret_cast<volatile int*>(&sh.abort) = 1;
  return false;
}
// wait_bar by a whole warp, which goes on or gives up as one.
__device__ __forceinline__ bool wait_warp(uint64_t* bar, uint32_t parity, PromptShared& sh) {
  return __all_sync(0xffffffffu, wait_bar(bar, parity, sh));
}

__device__ __forceinline__ bool block_done(int n, PromptShared& sh) {
  return wait_warp(&sh.done[n & 3], (n >> 2) & 1, sh);
}

// Byte offset of 16-byte chunk `cc` (0..7) of row `row` in a 64-column half-tile
// (128-byte swizzle).
__device__ __forceinline__ uint32_t swz(int row, int cc) { return row * 128 + ((cc ^ (row & 7)) << 4); }

__device__ __forceinline__ void sts128(uint32_t addr, uint32_t x, uint32_t y, uint32_t z, uint32_t w) {
  asm volatile("st.shared.v4.u32 [%0], {%1, %2, %3, %4};\n" ::"r"(addr), "r"(x), "r"(y), "r"(z), "r"(w) : "memory");
}
__device__ __forceinline__ void sts64(uint32_t addr, uint32_t x, uint32_t y) {
  asm volatile("st.shared.v2.u32 [%0], {%1, %2};\n" ::"r"(addr), "r"(x), "r"(y) : "memory");
}

// The four fields of both halves of w as fp16 pairs of codes.
__device__ __forceinline__ void q4_codes(uint32_t w, uint32_t (&f)[4]) {
  q4_codes01(w, f[0], f[1]);
  q4_codes01(w >> 8, f[2], f[3]);
}

// What one CTA works on.
struct PromptPlace {
  int b, hkv, tile, split, n_splits;
  int row0;          // first token row of the sequence in the token arrays
  int len;           // tokens in the cache
  int start;         // position of the sequence's first new token
  int tok0, n_tok;   // new tokens of this CTA
  int n_tiles;
  int kv_end;        // keys that its last token sees
  int j0, j1;        // its blocks of keys
};

// A row tile's place (all but split, j0, j1); false where there is nothing to do.
template <int TILES>
__device__ __forceinline__ bool find_place(const PromptArgs& a, PromptPlace& w, int tile, bool says) {
  const int problems = a.batch * a.num_kv_heads, x = tile % problems;
  w.hkv = x % a.num_kv_heads;
  w.b = x / a.num_kv_heads;
  const int qt = a.n_qtiles - 1 - tile / problems;
  says = says && tile < problems;
  const int cap = a.max_pages * a.page_size;
  int len = a.seq_lens[w.b];
  if (len < 0 || len > cap) {
    if (says) set_error(a.err, LOCKS_DEVERR_LENGTHS);
    len = len < 0 ? 0 : cap;
  }
  int c0 = w.b, c1 = w.b + (len > 0 ? 1 : 0);
  if (a.cu_tokens) {
    c0 = a.cu_tokens[w.b];
    c1 = a.cu_tokens[w.b + 1];
  }
  int n = c1 - c0;
  if (c0 < 0 || n < 0 || c1 > a.total) {
    if (says) set_error(a.err, LOCKS_DEVERR_LENGTHS);
    n = 0;
  }
  if (says && (n > len || n > a.max_tokens)) set_error(a.err, LOCKS_DEVERR_LENGTHS);
  const int mine = min(n, a.max_tokens), per_tile = kRows / a.group, per_cta = TILES * per_tile;
  w.row0 = c0;
  w.len = len;
  w.start = len - n;
  w.tok0 = qt * per_cta;
  if (w.tok0 >= mine) return false;
  w.n_tok = min(per_cta, mine - w.tok0);
  w.n_tiles = w.n_tok > per_tile ? 2 : 1;
  w.kv_end = max(0, min(len, w.start + w.tok0 + w.n_tok));
  return true;
}

// Row tiles are numbered tile by tile, those with the most keys first, sequence by
// sequence and head by head within; from a.n_whole on the keys of each are cut in
// a.n_splits parts, whose partial results (of 256 rows each) are numbered likewise.
__device__ __forceinline__ size_t part_of(const PromptArgs& a, int tile, int split) {
  return (size_t)(tile - a.n_whole) * a.n_splits + split;
}

// One value of the cache (bf16 pages: any; 4-bit pages: with its scale).
template <bool Q4, int P>
__device__ float value_at(const PromptArgs& a, const PromptPlace& w, int t, int d) {
  const int phys = __ldg(a.block_table + (size_t)w.b * a.max_pages + t / P);
  const size_t ph = (size_t)phys * a.num_kv_heads + w.hkv;
  const int slot = t % P;
  if (!Q4) {
    const uint16_t x = __ldg(static_cast<const uint16_t*>(a.v_pool) + (ph * P + slot) * kHeadDim + d);
    return __uint_as_float((uint32_t)x << 16);
  }
  const int u = slot & 15, j = d / 32;
  const uint8_t* p = static_cast<const uint8_t*>(a.k_pool) + ph * (size_t)LOCKS_KV_Q4_BLOCK_BYTES(P);
  const uint16_t c = *reinterpret_cast<const uint16_t*>(p + 72 * P + 1024 * (slot / 16) + 512 * (u / 8) +
                                                        64 * ((d % 32) / 4) + 16 * ((u % 8) / 2) + 4 * j + 2 * (u % 2));
  const __half s = *reinterpret_cast<const __half*>(p + 136 * P + 128 * (slot / 16) + 32 * ((u % 8) / 2) +
                                                    16 * (u / 8) + 4 * j + 2 * (u % 2));
  return __half2float(s) * (float)(((c >> (4 * (d % 4))) & 15) - 8);
}

// ---- warp 1: the copies ---------------------------------------------------------
template <Source S, int P>
__device__ void load_role(const PromptArgs& a, const PromptPlace& w, const CUtensorMap* tk, const CUtensorMap* tv,
                          PromptShared& sh, uint8_t* ring, uint8_t* raw) {
  constexpr int kPPB = kBlock / P;  // pages of a block
  constexpr int kAtOnce = 32 / kPPB;
  const int lane = threadIdx.x & 31;
  const int n_pages = (w.len + P - 1) / P;
  int asked = 0;  // operands (slots of codes) asked for
  int seen = 0;   // blocks known to be done
  int seen_v = 0; // blocks whose values are known to be free
  bool ok = true;
  for (int jb = w.j0; jb < w.j1 && ok; jb += kAtOnce) {
    // the pages of several blocks at a time, one per lane
    const int lp = jb * kPPB + lane;
    int phys = -1;
    if (lp < n_pages && lp < w.j1 * kPPB) {
      phys = __ldg(a.block_table + (size_t)w.b * a.max_pages + lp);
      if (phys < 0 || phys >= a.pages_total) {
        set_error(a.err, LOCKS_DEVERR_BLOCK_TABLE);
        phys = -1;
      }
    }
    for (int j = jb; j < min(jb + kAtOnce, w.j1) && ok; ++j) {
      const int n = j - w.j0;
      int pg[kPPB], skip = 0;
#pragma unroll
      for (int i = 0; i < kPPB; ++i) {
        pg[i] = __shfl_sync(0xffffffffu, phys, (j - jb) * kPPB + i);
        if (pg[i] < 0) skip |= ((1 << (P / 16)) - 1) << (i * (P / 16));
      }
      if constexpr (S != kCodes) {
        const int copies = kPPB - __popc(skip) / (P / 16);
#pragma unroll
        for (int u = 0; u < kUnits<S>; ++u, ++asked) {  // keys, then values
          const int slot = asked % kSlots<S>;
          // the operand that was in the slot: values of block m are free after block m,
          // keys after block m - 1 (the first block's after block 0, like the second's)
          if (asked >= kSlots<S>) {
            const int old = asked - kSlots<S>, m = old / kUnits<S>;
            const bool values = old % kUnits<S> == kUnits<S> - 1;
            if (kLateKeys<S> && values) {
              for (; ok && seen_v <= m; ++seen_v) ok = wait_warp(&sh.v_free[seen_v & 1], (seen_v >> 1) & 1, sh);
            } else {
              const int need = values ? m : max(0, m - 1);
              for (; ok && seen <= need; ++seen) ok = block_done(seen, sh);
            }
            if (!ok) break;
          }
          if (lane == 0) {
            uint64_t* full = &sh.full[slot];
            uint8_t* dst = ring + slot * kOperand;
            if (u == 0) {
              sh.skip[0][n % kSkipRing] = skip & 15;
              sh.skip[1][n % kSkipRing] = skip >> 4;
            }
            if constexpr (S == kPlanes || S == kBf16Planes) {
              // plane u of this sequence and head
              const int y = (int)(((long long)u * a.batch + w.b) * a.num_kv_heads + w.hkv) * a.plane_rows + j * kBlock;
              mbar_arrive_expect_tx(full, kOperand);
              tma_load_2d(dst, tk, full, 0, y);
              tma_load_2d(dst + kHalf, tk, full, 64, y);
            } else {
              mbar_arrive_expect_tx(full, (uint32_t)copies * P * 256);
#pragma unroll
              for (int i = 0; i < kPPB; ++i) {
                if (pg[i] < 0) continue;
                const int y = (pg[i] * a.num_kv_heads + w.hkv) * P;
                tma_load_2d(dst + i * P * 128, u ? tv : tk, full, 0, y);
                tma_load_2d(dst + kHalf + i * P * 128, u ? tv : tk, full, 64, y);
              }
            }
          }
          __syncwarp();
        }
      } else {
        // two 64-token slots of codes; the converters hand `skip` on with the block
#pragma unroll
        for (int hh = 0; hh < 2; ++hh, ++asked) {
          const int rs = asked % kRawSlots;
          if (asked >= kRawSlots && !wait_warp(&sh.raw_empty[rs], (asked / kRawSlots - 1) & 1, sh)) {
            ok = false;
            break;
          }
          const int part = (skip >> (4 * hh)) & 15;
          if (lane == 0) {
            sh.raw_skip[rs] = part;
            mbar_arrive_expect_tx(&sh.raw_full[rs],
                                  (uint32_t)(kPPB / 2 - __popc(part) / (P / 16)) * LOCKS_KV_Q4_BLOCK_BYTES(P));
#pragma unroll
            for (int i = 0; i < kPPB / 2; ++i) {
              const int ph = pg[hh * (kPPB / 2) + i];
              if (ph < 0) continue;
              bulk_load(smem_u32(raw) + rs * kQ4Slot + i * LOCKS_KV_Q4_BLOCK_BYTES(P),
                        static_cast<const uint8_t*>(a.k_pool) +
                            ((size_t)ph * a.num_kv_heads + w.hkv) * (size_t)LOCKS_KV_Q4_BLOCK_BYTES(P),
                        LOCKS_KV_Q4_BLOCK_BYTES(P), &sh.raw_full[rs]);
            }
          }
          __syncwarp();
        }
      }
    }
  }
  if (!ok && lane == 0) {
    // let the copies in flight land before the memory is given back
    constexpr int kRing = S == kCodes ? kRawSlots : kSlots<S>;
    for (int i = max(0, asked - kRing); i < asked; ++i)
      (void)mbar_wait(S == kCodes ? &sh.raw_full[i % kRing] : &sh.full[i % kRing], (i / kRing) & 1);
  }
}

// ---- codes to fp16 --------------------------------------------------------------
// The keys of a 16-byte piece c of one token's codes (its 8-byte scales z): for each
// scale group j the eight dimensions 32 j + 8 c .. + 7 as the nearest halves and the
// remainders; out(j, hi, lo).
template <typename Out>
__device__ __forceinline__ void convert_keys(uint4 x, uint2 z, Out out) {
  const uint32_t words[4] = {x.x, x.y, x.z, x.w};
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    const uint32_t zz = __byte_perm(j < 2 ? z.x : z.y, 0, j & 1 ? 0x3232 : 0x1010);
    uint32_t f[4], hi[4], lo[4];
    q4_codes(words[j], f);
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      hi[e] = mul_f16x2(f[e], zz);
      lo[e] = fma_f16x2(f[e], zz, hi[e] ^ 0x80008000u);  // s * code - hi, exact
    }
    out(j, hi, lo);
  }
}
// The values of a lane's 16 bytes: for each j the dimensions 32 j + 4 g .. + 3 of two
// tokens, whose scales are the halves of z's words; out(j, token 0's, token 1's).
template <typename Out>
__device__ __forceinline__ void convert_values(uint4 x, uint4 z, Out out) {
  const uint32_t words[4] = {x.x, x.y, x.z, x.w}, zw[4] = {z.x, z.y, z.z, z.w};
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    uint32_t f[4];
    q4_codes(words[j], f);
#pragma unroll
    for (int i = 0; i < 4; ++i) f[i] = mul_f16x2(f[i], zw[j]);
    out(j, make_uint2(__byte_perm(f[0], f[1], 0x5410), __byte_perm(f[2], f[3], 0x5410)),
        make_uint2(__byte_perm(f[0], f[1], 0x7632), __byte_perm(f[2], f[3], 0x7632)));
  }
}

// Warps 8-15 (kCodes): four warps for each half of a block.
template <int P>
__device__ void convert_role(const PromptPlace& w, PromptShared& sh, uint32_t ring, uint32_t raw) {
  using At = Q4Tile<P>;
  const int hh = (threadIdx.x >> 7) & 1, warp = (threadIdx.x >> 5) & 3, lane = threadIdx.x & 31;
  int seen = 0;  // blocks known to be done: each is waited for once, in order
  auto done_until = [&](int m) {
    for (; seen <= m; ++seen)
      if (!block_done(seen, sh)) return false;
    return true;
  };
  for (int n = 0; n < w.j1 - w.j0; ++n) {
    const int s = 2 * n + hh, rs = s % kRawSlots, i = 3 * n;
    const uint32_t src = raw + rs * kQ4Slot;
    // both halves' codes: every warp sees every phase of every slot, in order, so that
    // none can take an earlier phase for the one it waits for; and the other half's slot is
    // filled anew only when this warp has seen it full, so that no phase passes it by
    for (int y = 2 * n; y < 2 * n + 2; ++y)
      if (!wait_warp(&sh.raw_full[y % kRawSlots], (y / kRawSlots) & 1, sh)) return;
    if (lane == 0) mbar_arrive(&sh.raw_empty[(2 * n + 1 - hh) % kRawSlots]);
    // the ring holds two blocks: that of n - 2 makes room, its keys when block n - 3 is
    // done (the first block's with the second's), its values when it is
    if (n >= 2 && !done_until(max(0, n - 3))) return;
    if (warp == 0 && lane == 0) sh.skip[hh][n % kSkipRing] = sh.raw_skip[rs];
    {
      // a warp takes a 16-token tile, 8 tokens at a time; lane: 16 bytes of codes
      // (piece c) of one token, the eight lanes of a store phase on rows r and r + 4
      const uint32_t kh = ring + i % kSlots<kCodes> * kOperand, kl = ring + (i + 1) % kSlots<kCodes> * kOperand;
      const int c = lane & 3;
#pragma unroll
      for (int k = 0; k < 2; ++k) {
        const int r = 8 * k + ((lane >> 2) & 1) * 4 + (lane >> 3), row = 64 * hh + 16 * warp + r;
        convert_keys(lds128(src + At::key_codes(warp) + 64 * r + 16 * c), lds64(src + At::key_scales(warp) + 8 * r),
                     [&](int j, const uint32_t (&hi)[4], const uint32_t (&lo)[4]) {
                       const uint32_t at = (j >> 1) * kHalf + swz(row, (j & 1) * 4 + c);
                       sts128(kh + at, hi[0], hi[1], hi[2], hi[3]);
                       sts128(kl + at, lo[0], lo[1], lo[2], lo[3]);
                     });
      }
    }
    fence_proxy_async();
    __syncwarp();
    if (lane == 0) {
      mbar_arrive(&sh.full[i % kSlots<kCodes>]);
      mbar_arrive(&sh.full[(i + 1) % kSlots<kCodes>]);
    }
    if (n >= 2 && !done_until(n - 2)) return;
    {
      // lane (g, c): dimensions 32 j + 4 g .. + 3 of tokens 2c, 2c + 1 (+ 8)
      const uint32_t vd = ring + (i + 2) % kSlots<kCodes> * kOperand;
      const int g = lane >> 2, c = lane & 3;
#pragma unroll
      for (int hi = 0; hi < 2; ++hi) {
        const int row = 64 * hh + 16 * warp + 8 * hi + 2 * c;
        convert_values(lds128(src + At::value_codes(warp) + 512 * hi + 16 * lane),
                       lds128(src + At::value_scales(warp) + 32 * c + 16 * hi), [&](int j, uint2 t0, uint2 t1) {
                         const uint32_t base = vd + (j >> 1) * kHalf + (g & 1) * 8;
                         const int cc = (j & 1) * 4 + (g >> 1);
                         sts64(base + swz(row, cc), t0.x, t0.y);
                         sts64(base + swz(row + 1, cc), t1.x, t1.y);
                       });
      }
    }
    fence_proxy_async();
    __syncwarp();
    if (lane == 0) {
      mbar_arrive(&sh.raw_empty[rs]);
      mbar_arrive(&sh.full[(i + 2) % kSlots<kCodes>]);
    }
  }
}

// The fp16 planes of every sequence and head: plane 0 the keys' nearest halves, 1 the
// remainders, 2 the values, [3][batch][Hkv][plane_rows][128].  A CTA converts 64
// tokens, a warp 16; pages outside the pool leave their rows as they are (the
// attention leaves those tokens out).
template <int P>
__global__ void __launch_bounds__(128) planes_kernel(const PromptArgs a) {
  using At = Q4Tile<P>;
  pdl_wait();
  const int hkv = blockIdx.y % a.num_kv_heads, b = blockIdx.y / a.num_kv_heads;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int len = min(max(a.seq_lens[b], 0), a.max_pages * P), t0 = blockIdx.x * 64 + 16 * warp;
  pdl_launch_dependents();
  if (t0 >= len) return;
  const int phys = a.block_table[(size_t)b * a.max_pages + t0 / P];
  if (phys < 0 || phys >= a.pages_total) return;  // reported by the attention
  const uint8_t* block = static_cast<const uint8_t*>(a.k_pool) +
                         ((size_t)phys * a.num_kv_heads + hkv) * (size_t)LOCKS_KV_Q4_BLOCK_BYTES(P);
  const int tile = P == 64 ? warp : 0;
  const size_t plane = (size_t)a.batch * a.num_kv_heads * a.plane_rows * kHeadDim;
  uint16_t* dst = a.planes + ((size_t)blockIdx.y * a.plane_rows + t0) * kHeadDim;
  {
    const int c = lane & 3;
#pragma unroll
    for (int k = 0; k < 2; ++k) {
      const int r = 8 * k + (lane >> 2);
      convert_keys(__ldg(reinterpret_cast<const uint4*>(block + At::key_codes(tile) + 64 * r + 16 * c)),
                   __ldg(reinterpret_cast<const uint2*>(block + At::key_scales(tile) + 8 * r)),
                   [&](int j, const uint32_t (&hi)[4], const uint32_t (&lo)[4]) {
                     uint16_t* at = dst + r * kHeadDim + 32 * j + 8 * c;
                     *reinterpret_cast<uint4*>(at) = make_uint4(hi[0], hi[1], hi[2], hi[3]);
                     *reinterpret_cast<uint4*>(at + plane) = make_uint4(lo[0], lo[1], lo[2], lo[3]);
                   });
    }
  }
  const int g = lane >> 2, c = lane & 3;
#pragma unroll
  for (int hi = 0; hi < 2; ++hi) {
    uint16_t* row = dst + 2 * plane + (8 * hi + 2 * c) * kHeadDim + 4 * g;
    convert_values(__ldg(reinterpret_cast<const uint4*>(block + At::value_codes(tile) + 512 * hi + 16 * lane)),
                   __ldg(reinterpret_cast<const uint4*>(block + At::value_scales(tile) + 32 * c + 16 * hi)),
                   [&](int j, uint2 x0, uint2 x1) {
                     *reinterpret_cast<uint2*>(row + 32 * j) = x0;
                     *reinterpret_cast<uint2*>(row + kHeadDim + 32 * j) = x1;
                   });
  }
}

// The same of bf16 pages of 16 tokens: keys and values, [2][batch][Hkv][plane_rows][128].
__global__ void __launch_bounds__(128) bf16_planes_kernel(const PromptArgs a) {
  constexpr int P = 16;
  pdl_wait();
  const int hkv = blockIdx.y % a.num_kv_heads, b = blockIdx.y / a.num_kv_heads, lane = threadIdx.x & 31;
  const int len = min(max(a.seq_lens[b], 0), a.max_pages * P), t0 = blockIdx.x * 64 + P * (threadIdx.x >> 5);
  pdl_launch_dependents();
  if (t0 >= len) return;
  const int phys = a.block_table[(size_t)b * a.max_pages + t0 / P];
  if (phys < 0 || phys >= a.pages_total) return;  // reported by the attention
  const size_t from = ((size_t)phys * a.num_kv_heads + hkv) * P * kHeadDim;
  const size_t plane = (size_t)a.batch * a.num_kv_heads * a.plane_rows * kHeadDim;
  uint4* dst = reinterpret_cast<uint4*>(a.planes + ((size_t)blockIdx.y * a.plane_rows + t0) * kHeadDim) + lane;
  const uint4* k = reinterpret_cast<const uint4*>(static_cast<const uint16_t*>(a.k_pool) + from) + lane;
  const uint4* v = reinterpret_cast<const uint4*>(static_cast<const uint16_t*>(a.v_pool) + from) + lane;
  constexpr int kSteps = P * kHeadDim / 8 / 32;
  uint4 x[2 * kSteps];
#pragma unroll
  for (int i = 0; i < kSteps; ++i) {
    x[i] = __ldg(k + 32 * i);
    x[kSteps + i] = __ldg(v + 32 * i);
  }
#pragma unroll
  for (int i = 0; i < kSteps; ++i) {
    dst[32 * i] = x[i];
    dst[plane / 8 + 32 * i] = x[kSteps + i];
  }
}

// ---- warp 0, one thread: the matrix instructions ------------------------------------
// The thread's own steps (a test, a commit) cost some hundred clocks beside the busy
// softmax warps, and the tensor core stands still meanwhile; so there are few of them:
// with two tiles one test and one or two commits per tile and block.
template <Source S>
__device__ void mma_role(const PromptPlace& w, PromptShared& sh, uint32_t q, uint32_t ring, uint32_t tmem) {
  constexpr bool kBf16 = kIsBf16<S>, kOne = kTiles<S> == 1;
  constexpr uint32_t kIdS = umma_idesc(kRows, kBlock, kBf16, false), kIdO = umma_idesc(kRows, kHeadDim, kBf16, true);
  constexpr int kKeys = kUnits<S> - 1, kN = kSlots<S>;
  const int n_blocks = w.j1 - w.j0;
  // the next operand of the ring; they come in order, a block's keys before its values
  int slot = 0, phase = 0;
  auto next = [&](int& got, bool wait) {
    got = slot;
    const bool there = !wait || spin_bar(&sh.full[slot], phase, sh);
    if (++slot == kN) slot = 0, phase ^= 1;
    return there;
  };
  const uint32_t q_lo = umma_desc_lo(q, 16), k_lo = umma_desc_lo(ring, 16), v_lo = umma_desc_lo(ring, kHalf);
  int key[kKeys], value = 0, late_phase = 0;
  auto next_keys = [&](bool wait) {
    bool there = true;
#pragma unroll
    for (int part = 0; part < kKeys; ++part) {
      late_phase = phase;
      there = next(key[part], wait && there) && there;
    }
    return there;
  };
  auto scores = [&](int t, int buf) {  // S = Q_t K^T (fp16: both halves of K)
    const uint32_t d = tmem + buf * kBlock, qd = q_lo + t * (kOperand / 16);
#pragma unroll
    for (int part = 0; part < kKeys; ++part) {
      const uint32_t kd = k_lo + key[part] * (kOperand / 16);
      if (kLateKeys<S> && part == 1 && t == 0) {
        if (!spin_bar(&sh.full[key[1]], late_phase, sh)) return false;
        tc_fence_after();
      }
#pragma unroll
      for (int s = 0; s < kHeadDim / 16; ++s) {
        const uint32_t off = ((s / 4) * kHalf + (s % 4) * 32) / 16;
        if (kOne) umma_ts(d, tmem + kTmemQ + s * 8, kd + off, kIdS, part + s > 0);
        else umma_ss(d, qd + off, kd + off, kIdS, part + s > 0);
      }
    }
    umma_commit(&sh.s_full[buf]);
    return true;
  };
  auto values = [&](int t, int buf, bool more) {  // O_t (+)= P V
    const uint32_t p = tmem + buf * kBlock, vd = v_lo + value * (kOperand / 16), o = tmem + kTmemO + t * kHeadDim;
    umma_ts(o, p, vd, kIdO, more);
#pragma unroll
    for (int s = 1; s < kBlock / 16; ++s) umma_ts(o, p + s * 8, vd + s * 16 * 128 / 16, kIdO, true);
  };
  bool ok = wait_bar(&sh.q_full, 0, sh) && next_keys(true);
  if (ok) {
    tc_fence_after();
    for (int t = 0; ok && t < w.n_tiles; ++t) ok = scores(t, kOne ? 0 : t);
  }
  for (int n = 0; ok && n < n_blocks; ++n) {
    const bool last = n + 1 == n_blocks;
    if constexpr (kOne) {
      // S of the next block while the softmax of this one runs
      if (!(ok = next(value, true))) break;
      if (!last) {
        if (!(ok = next_keys(true))) break;
        tc_fence_after();
        (void)scores(0, (n + 1) & 1);
      }
      if (!(ok = spin_bar(&sh.p_ready[n & 1], (n >> 1) & 1, sh))) break;
      tc_fence_after();
      values(0, n & 1, n > 0);
    } else {
      // each tile's O, then its S of the next block, while the other's softmax runs;
      // tile 0's weights come with the news that the operands are there
      (void)next(value, false);
      if (!last) (void)next_keys(false);
      for (int t = 0; t < w.n_tiles; ++t) {
        if (!(ok = spin_bar(&sh.p_ready[t], n & 1, sh))) break;
        tc_fence_after();
        values(t, t, n > 0);
        if (kLateKeys<S> && !last && t + 1 == w.n_tiles) umma_commit(&sh.v_free[n & 1]);
        if (!last) ok = scores(t, t);
        else if (t + 1 < w.n_tiles) umma_commit(&sh.o_full[t]);
        if (!ok) break;
      }
    }
    if (ok) umma_commit(last ? &sh.o_full[w.n_tiles - 1] : &sh.done[n & 3]);
  }
  if (!ok) {
    // what was issued must end before its memory is given back
    umma_commit(&sh.drain);
    (void)mbar_wait(&sh.drain, 0);
  }
}

// ---- warp 2 (two tiles): tells the issuing thread, with tile 0's weights of a block,
// that the block's values and the next one's keys have landed ---------------------------
template <Source S>
__device__ void landed_role(const PromptPlace& w, PromptShared& sh) {
  constexpr int kU = kUnits<S>;
  const int n_blocks = w.j1 - w.j0;
  for (int n = 0; n < n_blocks; ++n) {
    // operands kU n + kU - 1 (values) and kU (n + 1) (keys; their second half: see kLateKeys)
    for (int i = kU * n + kU - 1; i <= (n + 1 < n_blocks ? kU * (n + 1) : kU * n + kU - 1); ++i)
      if (!wait_warp(&sh.full[i % kSlots<S>], (i / kSlots<S>) & 1, sh)) return;
    if ((threadIdx.x & 31) == 0) mbar_arrive(&sh.p_ready[0]);
    // one arrival per phase
    if (!wait_warp(&sh.p_ready[0], n & 1, sh)) return;
  }
}

// ---- warps 4 and up: one softmax row per thread -------------------------------------------
template <Source S, int P>
__device__ void softmax_role(const PromptArgs& a, const PromptPlace& w, PromptShared& sh, uint8_t* smem, uint32_t tmem_base) {
  constexpr bool Q4 = !kIsBf16<S>;
  constexpr bool kOne = kTiles<S> == 1;      // one tile, two S buffers
  constexpr float kOffset = Q4 ? 6.f : 0.f;  // weights are scaled by 2^kOffset
  const int warp = threadIdx.x >> 5, t = (warp - 4) / 4;
  if (t >= w.n_tiles) return;
  const int row = threadIdx.x & 127, lane = threadIdx.x & 31;
  const int G = a.group, tpt = kRows / G, Hq = a.num_kv_heads * G;
  const int ti = row / G, h = row - ti * G;
  const int i = t * tpt + ti;  // token of this CTA
  const bool valid = ti < tpt && i < w.n_tok;
  const int tok = w.tok0 + i;
  const int pos = w.start + tok;
  const int limit = valid ? max(0, pos + 1) : w.kv_end;  // keys that this row sees
  const size_t qrow = (size_t)w.row0 + tok;
  const uint32_t tmem = tmem_base + ((uint32_t)(warp & 3) << 21);
  float factor = a.scale_log2;

  // the row's query into the operand's order
  {
    const uint16_t* src = a.q + qrow * a.q_stride + (size_t)(w.hkv * G + h) * kHeadDim;
    const uint32_t dst = smem_u32(smem) + t * kOperand;
    uint4 x[16];
    uint32_t qt[2][32];  // one tile: the row in tensor memory
#pragma unroll
    for (int k = 0; k < 16; ++k) x[k] = valid ? __ldg(reinterpret_cast<const uint4*>(src) + k) : make_uint4(0, 0, 0, 0);
    float down = 1.f;
    if (Q4) {
      uint32_t m = 0;  // largest magnitude, as bf16 bits
#pragma unroll
      for (int k = 0; k < 16; ++k) {
        const uint32_t v[4] = {x[k].x, x[k].y, x[k].z, x[k].w};
#pragma unroll
        for (int e = 0; e < 4; ++e) m = max(m, max(v[e] & 0x7fffu, (v[e] >> 16) & 0x7fffu));
      }
      int e = (int)(m >> 7) - 127;
      e = m == 0 || e > 127 ? 0 : min(max(e, -100), 126);
      down = __uint_as_float((uint32_t)(127 - e) << 23);
      factor *= __uint_as_float((uint32_t)(127 + e) << 23);
    }
#pragma unroll
    for (int k = 0; k < 16; ++k) {
      uint32_t v[4] = {x[k].x, x[k].y, x[k].z, x[k].w};
      if (Q4) {
#pragma unroll
        for (int e = 0; e < 4; ++e)
          v[e] = pack_f16(__uint_as_float(v[e] << 16) * down, __uint_as_float(v[e] & 0xffff0000u) * down);
      }
      if (kOne) {
#pragma unroll
        for (int e = 0; e < 4; ++e) qt[k >> 3][(k & 7) * 4 + e] = v[e];
      } else {
        sts128(dst + (k >> 3) * kHalf + swz(row, k & 7), v[0], v[1], v[2], v[3]);
      }
    }
    if (kOne) {
      tmem_st32(tmem + kTmemQ, qt[0]);
      tmem_st32(tmem + kTmemQ + 32, qt[1]);
      tmem_wait_st();
      tc_fence_before();
    } else {
      fence_proxy_async();
    }
    __syncwarp();
    if (lane == 0) mbar_arrive(&sh.q_full);
  }

  float m = -INFINITY, l0 = 0.f, l1 = 0.f;  // reference (base 2), sum of the weights (two halves)
  const int first_limit = max(0, w.start + w.tok0 + 1);  // keys that every row of the CTA sees
  const int n_blocks = w.j1 - w.j0;
  for (int n = 0; n < n_blocks; ++n) {
    const int kv0 = (w.j0 + n) * kBlock;
    const int buf = kOne ? n & 1 : t;
    const uint32_t phase = kOne ? (n >> 1) & 1 : n & 1;
    if (!wait_warp(&sh.s_full[buf], phase, sh)) return;
    tc_fence_after();
    const int skip = *reinterpret_cast<volatile int*>(&sh.skip[0][n % kSkipRing]) |
                     *reinterpret_cast<volatile int*>(&sh.skip[1][n % kSkipRing]) << 4;
    // values that some row must not see are cleared by tile 0's threads, one token
    // each, before its weights are handed over: the products of both tiles come later
    const bool clear = kv0 + kBlock > first_limit || kv0 + kBlock > w.len || skip;
    const int i = kUnits<S> * n + kUnits<S> - 1, slot = i % kSlots<S>;
    if (t == 0 && clear) {
      if (!wait_warp(&sh.full[slot], (i / kSlots<S>) & 1, sh)) return;
      uint8_t* v = smem + kQueryTiles<S> * kOperand + slot * kOperand + row * 128;
      const int at = kv0 + row;
      if (at >= w.kv_end || at >= w.len || ((skip >> (row / 16)) & 1)) {
#pragma unroll
        for (int k = 0; k < 16; ++k) *reinterpret_cast<uint4*>(v + (k >> 3) * kHalf + (k & 7) * 16) = make_uint4(0, 0, 0, 0);
      } else if (at >= first_limit) {
        // infinities and NaN: cleared here, and added at the end to the rows that see them
        constexpr uint32_t e = Q4 ? 0x7c007c00u : 0x7f807f80u;  // an exponent of all ones
        auto hit = [&](uint32_t y) { return __vcmpeq2(y & e, e); };
        uint32_t bad = 0;
#pragma unroll
        for (int k = 0; k < 16; ++k) {
          const uint4 x = *reinterpret_cast<const uint4*>(v + (k >> 3) * kHalf + (k & 7) * 16);
          bad |= hit(x.x) | hit(x.y) | hit(x.z) | hit(x.w);
        }
        if (bad) {
#pragma unroll 1
          for (int k = 0; k < 64; ++k) {
            uint32_t* x = reinterpret_cast<uint32_t*>(v + (k >> 5) * kHalf) + (k & 31);
            *x &= ~hit(*x);
          }
          const int k = atomicAdd(&sh.n_bad, 1);
          if (k < kMaxBad) sh.bad[k] = at;
        }
      }
      fence_proxy_async();
    }

    const int lim = limit - kv0;
    const bool masked = __any_sync(0xffffffffu, lim < kBlock) || skip;
    auto hide = [&](uint32_t (&s)[32], int c0) {
#pragma unroll
      for (int k = 0; k < 32; ++k)
        if (c0 + k >= lim || ((skip >> ((c0 + k) / 16)) & 1)) s[k] = 0xff800000u;  // -infinity
    };
    // two S buffers: the products of the block before are done (every block waits for
    // that once, so that no phase is missed)
    bool settled = !kOne || n == 0;
    auto o_settled = [&] {
      if (!settled && !block_done(n - 1, sh)) return false;
      settled = true;
      tc_fence_after();
      return true;
    };
    const uint32_t ts = tmem + buf * kBlock, to = tmem + kTmemO + t * kHeadDim;
    // the row's logits, all of them in registers, and their maximum: that of the first
    // half while the second is loaded
    uint32_t s[4][32];
    float m4[4];
    tmem_ld32(s[0], ts);
    tmem_ld32(s[1], ts + 32);
    tmem_wait_ld32(s[0]);
    tmem_wait_ld32(s[1]);
    tmem_ld32(s[2], ts + 64);
    tmem_ld32(s[3], ts + 96);
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      if (k >= 2) tmem_wait_ld32(s[k]);
      if (masked) hide(s[k], 32 * k);
      m4[k] = __uint_as_float(s[k][0]);
#pragma unroll
      for (int e = 1; e < 31; e += 2) m4[k] = max3(m4[k], __uint_as_float(s[k][e]), __uint_as_float(s[k][e + 1]));
      m4[k] = fmaxf(m4[k], __uint_as_float(s[k][31]));
    }
    const float mx = fmaxf(fmaxf(m4[0], m4[1]), fmaxf(m4[2], m4[3])) * factor;  // the factor is positive
    if (__any_sync(0xffffffffu, mx > m + kLazy || (m == -INFINITY && mx > m))) {
      const float mn = fmaxf(m, mx);
      const float al = mn == -INFINITY ? 1.f : fast_exp2(m - mn);
      m = mn;
      l0 *= al;
      l1 *= al;
      if (n > 0) {
        // O holds every block before this one: S of this block came behind them, or,
        // with two S buffers, once they are done
        if (kOne && !o_settled()) return;
#pragma unroll 1
        for (int c0 = 0; c0 < kHeadDim; c0 += 32) {
          uint32_t o[32];
          tmem_ld32(o, to + c0);
          tmem_wait_ld32(o);
#pragma unroll
          for (int k = 0; k < 32; ++k) o[k] = __float_as_uint(__uint_as_float(o[k]) * al);
          tmem_st32(to + c0, o);
        }
      }
    }
    const float ref = m == -INFINITY ? 0.f : m - kOffset;
    const uint64_t f2 = f32x2(factor, factor), r2 = f32x2(-ref, -ref);
    uint64_t sum = f32x2(l0, l1);
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      uint32_t p[16];
#pragma unroll
      for (int e = 0; e < 16; ++e) {
        float x, y;
        unpack_f32x2(fma_f32x2(f32x2(__uint_as_float(s[k][2 * e]), __uint_as_float(s[k][2 * e + 1])), f2, r2), x, y);
        x = fast_exp2(x);
        y = fast_exp2(y);
        sum = add_f32x2(sum, f32x2(x, y));
        p[e] = Q4 ? pack_f16(x, y) : pack_bf16(x, y);
      }
      tmem_st16(ts + 16 * k, p);
    }
    if (kOne && !o_settled()) return;
    tmem_wait_st();
    tc_fence_before();
    __syncwarp();
    if (lane == 0) mbar_arrive(&sh.p_ready[buf]);
    unpack_f32x2(sum, l0, l1);
  }
  const float l = l0 + l1;

  // ---- the rows' results ----
  if (n_blocks > 0) {
    if (!wait_warp(&sh.o_full[t], 0, sh)) return;
    tc_fence_after();
  }
  const int n_bad = min(*reinterpret_cast<volatile int*>(&sh.n_bad), kMaxBad);
  const float lse2 = (m == -INFINITY ? 0.f : m - kOffset) + fast_log2(l);
  const size_t oi = qrow * Hq + (size_t)w.hkv * G + h;
  const size_t pi = w.n_splits > 1 ? part_of(a, w.tile, w.split) * (2 * kRows) + t * kRows + row : 0;
  const float inv = l == 0.f ? 0.f : 1.f / l;
#pragma unroll
  for (int c0 = 0; c0 < kHeadDim; c0 += 32) {
    uint32_t o[32];
    if (n_blocks > 0) {
      tmem_ld32(o, tmem + kTmemO + t * kHeadDim + c0);
      tmem_wait_ld32(o);
    } else {
#pragma unroll
      for (int k = 0; k < 32; ++k) o[k] = 0u;
    }
    for (int x = 0; x < n_bad; ++x) {
      const int at = sh.bad[x];
      if (!valid || at >= limit) continue;
#pragma unroll
      for (int k = 0; k < 32; ++k) {
        const float v = value_at<Q4, P>(a, w, at, c0 + k);
        if (!isfinite(v)) o[k] = __float_as_uint(__uint_as_float(o[k]) + v);
      }
    }
    if (!valid) continue;
    if (w.n_splits > 1) {
#pragma unroll
      for (int k = 0; k < 32; k += 4)
        *reinterpret_cast<uint4*>(a.part_o + pi * kHeadDim + c0 + k) = make_uint4(o[k], o[k + 1], o[k + 2], o[k + 3]);
    } else {
#pragma unroll
      for (int k = 0; k < 32; k += 8) {
        uint32_t y[4];
#pragma unroll
        for (int e = 0; e < 4; ++e)
          y[e] = pack_bf16(__uint_as_float(o[k + 2 * e]) * inv, __uint_as_float(o[k + 2 * e + 1]) * inv);
        *reinterpret_cast<uint4*>(a.out + oi * kHeadDim + c0 + k) = make_uint4(y[0], y[1], y[2], y[3]);
      }
    }
  }
  if (valid) {
    if (w.n_splits > 1) a.part_ml[pi] = make_float2(l == 0.f ? -INFINITY : (m == -INFINITY ? 0.f : m - kOffset), l);
    else if (a.lse) a.lse[oi] = l == 0.f ? -INFINITY : lse2 * kLn2;
  }
}

template <Source S, int P>
__global__ void __launch_bounds__(kThreadsOf<S>, 1)
    prompt_kernel(const __grid_constant__ CUtensorMap tk, const __grid_constant__ CUtensorMap tv, const PromptArgs a) {
  extern __shared__ uint8_t dyn_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(dyn_raw) + 1023) & ~uintptr_t(1023));
  __shared__ PromptShared sh;
  uint8_t* ring = smem + kQueryTiles<S> * kOperand;
  uint8_t* raw = ring + kSlots<S> * kOperand;
  const int tid = threadIdx.x, warp = tid >> 5;

  pdl_wait();
  PromptPlace w;
  {
    const int cut = (int)blockIdx.x - a.n_whole;  // CTAs of whole tiles first
    w.tile = cut < 0 ? blockIdx.x : a.n_whole + cut / a.n_splits;
    w.split = cut < 0 ? 0 : cut % a.n_splits;
    w.n_splits = cut < 0 ? 1 : a.n_splits;
    if (!find_place<kTiles<S>>(a, w, w.tile, tid == 0 && w.split == 0)) return;  // the whole CTA
    const long long nb = (w.kv_end + kBlock - 1) / kBlock;
    w.j0 = (int)(nb * w.split / w.n_splits);
    w.j1 = (int)(nb * (w.split + 1) / w.n_splits);
  }
  if (tid == 0) {
    mbar_init(&sh.q_full, kRows / 32 * w.n_tiles);
    for (int s = 0; s < kSlots<S>; ++s) mbar_init(&sh.full[s], S == kCodes ? 8 : 1);
    for (int t = 0; t < 2; ++t) {
      mbar_init(&sh.s_full[t], 1);
      mbar_init(&sh.p_ready[t], kRows / 32 + (kTiles<S> == 2 && t == 0 ? 1 : 0));
      mbar_init(&sh.o_full[t], 1);
      mbar_init(&sh.done[t], 1);
      mbar_init(&sh.done[2 + t], 1);
      mbar_init(&sh.v_free[t], 1);
    }
    mbar_init(&sh.drain, 1);
    for (int s = 0; s < kRawSlots; ++s) {
      mbar_init(&sh.raw_full[s], 1);
      mbar_init(&sh.raw_empty[s], 8);
    }
    fence_mbar_init();
    sh.abort = 0;
    sh.n_bad = 0;
  }
  if (warp == 0) tmem_alloc(&sh.tmem, kTmemCols);
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  // All 512 columns, so they begin at address 0: a constant, which saves the address
  // arithmetic of every tensor memory access (662 us, not 673, for 8K tokens of 4-bit pages).
  constexpr uint32_t tmem = 0;

  // registers per warpgroup: the launch's 504 (512) between them; 256 threads have
  // enough each
  if (warp < 4) {
    if constexpr (S != kBf16Few) set_registers_down<S == kCodes ? 72 : 88>();
    if (warp == 0) {
      if ((tid & 31) == 0 && w.j1 > w.j0) mma_role<S>(w, sh, smem_u32(smem), smem_u32(ring), tmem);
      __syncwarp();
    } else if (warp == 1) {
      load_role<S, P>(a, w, &tk, &tv, sh, ring, raw);
    } else if (warp == 2 && kTiles<S> == 2) {
      landed_role<S>(w, sh);
    }
  } else if (warp < 4 + 4 * kTiles<S>) {
    if constexpr (S != kBf16Few) set_registers_up<208>();
    softmax_role<S, P>(a, w, sh, smem, tmem);
  } else if constexpr (S == kCodes) {
    set_registers_down<112>();
    convert_role<P>(w, sh, smem_u32(ring), smem_u32(raw));
  }
  __syncwarp();
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  if (warp == 0) tmem_dealloc(tmem, kTmemCols);
  pdl_launch_dependents();
  if (tid == 0 && sh.abort) set_error(a.err, kDevErrTimeout);
}

// ---- joins the partial results: grid (tiles that were cut, blocks of eight rows) ------------
constexpr int kJoinWarps = 8;
constexpr int kJoinFlight = 8;  // partials that a warp loads at once

template <int TILES>
__global__ void __launch_bounds__(kJoinWarps * 32) prompt_join_kernel(const PromptArgs a) {
  const int lane = threadIdx.x & 31, r = blockIdx.y * kJoinWarps + (threadIdx.x >> 5), tile = a.n_whole + blockIdx.x;
  PromptPlace w;
  // the other kernel's inputs were complete before it let this one begin
  const bool some = find_place<TILES>(a, w, tile, false);
  const int G = a.group, tpt = kRows / G, n = a.n_splits;
  const int ti = (r % kRows) / G, h = (r % kRows) % G, i = (r / kRows) * tpt + ti;
  // also where there is nothing to join: whatever follows may rely on this kernel's end
  pdl_wait();
  pdl_launch_dependents();
  if (!some || ti >= tpt || i >= w.n_tok) return;
  const size_t p0 = part_of(a, tile, 0) * (2 * kRows) + r;
  auto part = [&](int s) { return p0 + (size_t)s * (2 * kRows); };
  float M = -INFINITY, L = 0.f;
  for (int s = lane; s < n; s += 32) M = fmaxf(M, __ldcg(a.part_ml + part(s)).x);
  M = warp_max(M);
  float4 O = make_float4(0.f, 0.f, 0.f, 0.f);
  for (int s0 = 0; s0 < n; s0 += kJoinFlight) {
    float4 v[kJoinFlight];
    float2 ml[kJoinFlight];
#pragma unroll
    for (int k = 0; k < kJoinFlight; ++k) {
      ml[k] = make_float2(0.f, 0.f);
      if (s0 + k >= n) continue;
      v[k] = __ldcg(reinterpret_cast<const float4*>(a.part_o + part(s0 + k) * kHeadDim) + lane);
      ml[k] = __ldcg(a.part_ml + part(s0 + k));
    }
#pragma unroll
    for (int k = 0; k < kJoinFlight; ++k) {
      if (ml[k].y == 0.f) continue;  // saw no key
      const float f = fast_exp2(ml[k].x - M);
      L = fmaf(ml[k].y, f, L);
      O.x = fmaf(v[k].x, f, O.x);
      O.y = fmaf(v[k].y, f, O.y);
      O.z = fmaf(v[k].z, f, O.z);
      O.w = fmaf(v[k].w, f, O.w);
    }
  }
  const float inv = L == 0.f ? 0.f : 1.f / L;
  const size_t oi = ((size_t)w.row0 + w.tok0 + i) * ((size_t)a.num_kv_heads * G) + (size_t)w.hkv * G + h;
  *reinterpret_cast<uint2*>(a.out + oi * kHeadDim + 4 * lane) =
      make_uint2(pack_bf16(O.x * inv, O.y * inv), pack_bf16(O.z * inv, O.w * inv));
  if (a.lse && lane == 0) a.lse[oi] = L == 0.f ? -INFINITY : (M + fast_log2(L)) * kLn2;
}

template <Source S, int P>
cudaError_t launch(const PromptArgs& a, const CUtensorMap& tk, const CUtensorMap& tv, cudaStream_t s) {
  auto kern = prompt_kernel<S, P>;
  const size_t smem = 1024 + (size_t)(kQueryTiles<S> + kSlots<S>) * kOperand + (S == kCodes ? kRawSlots * kQ4Slot : 0);
  cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem);
  if (e != cudaSuccess) return e;
  cudaLaunchConfig_t cfg = {};
  cfg.stream = s;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  if constexpr (S == kPlanes || S == kBf16Planes) {
    cfg.gridDim = dim3((a.max_pages * P + 63) / 64, a.batch * a.num_kv_heads, 1);
    cfg.blockDim = dim3(128, 1, 1);
    if ((e = cudaLaunchKernelEx(&cfg, S == kPlanes ? planes_kernel<P> : bf16_planes_kernel, a)) != cudaSuccess) return e;
  }
  const int tiles = a.batch * a.num_kv_heads * a.n_qtiles, cut = tiles - a.n_whole;
  cfg.gridDim = dim3(a.n_whole + cut * a.n_splits, 1, 1);
  cfg.blockDim = dim3(kThreadsOf<S>, 1, 1);
  cfg.dynamicSmemBytes = smem;
  if ((e = cudaLaunchKernelEx(&cfg, kern, tk, tv, a)) != cudaSuccess || cut == 0) return e;
  cfg.gridDim = dim3(cut, kTiles<S> * kRows / kJoinWarps, 1);
  cfg.blockDim = dim3(kJoinWarps * 32, 1, 1);
  cfg.dynamicSmemBytes = 0;
  return cudaLaunchKernelEx(&cfg, prompt_join_kernel<kTiles<S>>, a);
}

template <int P>
cudaError_t launch_page(const PromptArgs& a, const CUtensorMap& tk, const CUtensorMap& tv, cudaStream_t s) {
  if constexpr (P == 16)
    if (!a.q4 && a.planes) return launch<kBf16Planes, P>(a, tk, tv, s);
  if (!a.q4) return a.one_tile ? launch<kBf16Few, P>(a, tk, tv, s) : launch<kBf16Pages, P>(a, tk, tv, s);
  return a.planes ? launch<kPlanes, P>(a, tk, tv, s) : launch<kCodes, P>(a, tk, tv, s);
}

}  // namespace

cudaError_t launch_prompt(const PromptArgs& a, const CUtensorMap& tk, const CUtensorMap& tv, cudaStream_t s) {
  return a.page_size == 16 ? launch_page<16>(a, tk, tv, s) : launch_page<kPage>(a, tk, tv, s);
}

}  // namespace locks
