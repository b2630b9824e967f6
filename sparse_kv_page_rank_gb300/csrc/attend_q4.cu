// Attention of one query token per sequence over a cache held in 4 bits
// (LOCKS_KV_Q4): over a page list and the open tail, over every page, or the exact
// per-page log-sum-exp; the three uses that attend.cu has for bf16 pages.
//
// Mathematics.  A key is k_d = s_j c_d with integer codes c and one scale per 32
// dimensions j, so  q.k = sum_j s_j (sum_{d in j} q_d c_d): the codes go through
// the matrix instructions as exact small integers and the scales multiply the four
// fp32 partial sums.  A value is v_d = z_j c_d, so  sum_t p_t v_td =
// sum_t (p_t z_tj) c_td: the weight of a token is multiplied by its scale of the
// 32 dimensions at hand, in fp16 pairs, before the product with the exact codes.
//
// What bounds it: 288 bytes per token and KV head at the memory's rate.  A 16-token
// tile (2304 bytes) arrives every ~98 clocks per SM at the measured copy rate, in
// which its four schedulers issue ~390 warp instructions; a tile costs a warp
// about 220, so the codes have to be taken apart cheaply:
//  - Codes are stored as u = code + 8.  A 4-bit field under a fixed fp16 exponent is
//    1024 + u (or, four bits up, 64 + u) exactly: one logical operation for two.
//  - Keys: the matrix instruction runs on 64 + u = code + 72 and its accumulator
//    starts at -72 sum_d q_d (per head and scale group), which takes the offset out.
//    Values, whose sums run over all tokens, are freed of it by a packed subtraction
//    (an offset carried through thousands of accumulations would cost digits).
//    e4m3 operands would need fewer operations (0000uuuu is the number u 2^-9), but
//    this instruction has no 8-bit form of its own here: 128K took 46 us, not 42.
//  - The products have M = tokens (or dimensions) and N = 8 query heads, so that
//    the group's few heads sit on the instruction's short side, and the pages store
//    the codes in the order in which a lane needs them: 16 bytes per lane, 512
//    contiguous bytes per warp, no conflicts and no shuffles.  The weights move
//    from the first product's layout to the second's by one 8x8 transpose per
//    eight tokens.
//
// Precision.  q is scaled by a power of two to fit fp16 (bf16's 8 bits are exact
// there); logits, maxima, sums and outputs are fp32.  Weights are rounded to fp16
// twice (2^-11 each, before and after their scale).  Two things keep both in fp16's
// range.  The reference R of the softmax lets a warp's largest weight lie between 2^11
// and 2^15.  And value scales are multiplied by the power of two that brings the largest
// that the warp has seen to between 1/2 and 1 (or between 1/4 and 1 as it is), which its
// outputs give back in fp32 at the end; so weight * scale stays below 2^15, and how small
// a cache's values are takes no bits from the weights.  Below 2^-14 fp16 is no finer than
// 2^-24: each rounding is off by 2^-25 at most, 2^-36 of the largest weight for the first
// and, for the second, 2^-34 of the largest weight times the largest scale.  R and the
// power of two move only when a token outgrows them, so the usual unit needs no maximum
// across lanes, only a vote.  (32 sequences of 9K take 64.8 us, and 1.8 us more where the
// scales are multiplied.)
//
// Buffers.  Every warp copies for itself: its lane 0 issues bulk copies of whole pages
// into the warp's own two 64-token buffers (9216 or 4 x 2304 contiguous bytes; with
// few pages per CTA eight 16-token buffers, so that a page occupies four warps).  A
// warp waits for its own copies in order and refills a buffer only when it is done
// with it, so no warp waits for another.  With 9 to 16 heads a warp works on half a
// buffer at a time, which is what its registers hold; copies of half pages, in four
// pieces each, took 95 us for 1M tokens, whole ones 88.  Two CTAs of six warps per SM hold 221 KB of
// buffers, half of them in flight at any time.
//
// Work split.  Over every page: the 64-token slots of all sequences and heads in one
// line, cut into equal parts, one per CTA (two CTAs per SM), so that ragged lengths and
// any number of problems fill every SM.  A CTA whose part ends inside a problem writes
// its partial (R, sum, O) to the workspace, and a second, dependent kernel joins them.
// Over a page list, a few pages of each problem: one thread-block cluster per problem,
// whose CTAs push their partial states to each other through distributed shared memory.
//
// Measured (floor by bytes): 131,001 tokens of 8 KV heads, 4 heads each, 32.7 us (22.3),
// streaming at 7.08 TB/s; 32 sequences of up to 9216 tokens in 16-token pages 64.8 us
// (40.0); 1M tokens of 2 KV heads, 16 heads each, 87.7 us (44.5); 4096 tokens of one
// head 6.7 us; a list of 32 pages of 8 KV heads 8.0 us.  Five rows over eight sequences
// of up to 16,411 tokens 60 us (14.2).
#include <algorithm>
#include <type_traits>

#include "common.cuh"
#include "kernels.h"
#include "kv_q4.cuh"

namespace locks {

namespace {

constexpr int kW = 6;                                    // warps
constexpr int kThreads = kW * 32;
constexpr int kTileBytes = LOCKS_KV_Q4_BLOCK_BYTES(16);  // 16 tokens
constexpr int kWarpTiles = 8;                            // tiles of buffers per warp
constexpr int kRing = kW * kWarpTiles * kTileBytes;      // 110,592 bytes: two CTAs per SM
constexpr int kOStride = 132;                            // padded row of a warp's outputs (floats)
constexpr int kRecvMl = 16 * 16 * 8;                     // (R, sum) received from the cluster, [rank][head]
constexpr int kSmem = kRing + 128;

struct Q4Shared {
  uint64_t full[kW][kWarpTiles], recv;
  int len[kW][kWarpTiles][4], lp[kW][kWarpTiles];
  float m[kW][16], l[kW][16], f[kW][16];
  float cta_m[16], cta_l[16];
};

__device__ __forceinline__ uint32_t transpose8x8(uint32_t x) {
  uint32_t d;
  asm volatile("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;\n" : "=r"(d) : "r"(x));
  return d;
}
// The four fields of both halves of w as fp16 pairs 64 + u (exact).
__device__ __forceinline__ void fields64(uint32_t w, uint32_t (&f)[4]) {
  const uint32_t v = w >> 8;
  f[0] = sub_f16x2(field_under<0x000f000fu, 0x64006400u>(w), 0x63806380u);  // 1024 + u, less 960
  f[1] = field_under<0x00f000f0u, 0x54005400u>(w);
  f[2] = sub_f16x2(field_under<0x000f000fu, 0x64006400u>(v), 0x63806380u);
  f[3] = field_under<0x00f000f0u, 0x54005400u>(v);
}
// The lowest power of two above the finite half with bits `h`, as half bits: 0x7c00
// stands for 2^16, which is where it lies in order.
__device__ __forceinline__ uint32_t half_limit(uint32_t h) {
  return h < 0x400u ? 1u << (32 - __clz(h)) : (h >> 10) + 1 << 10;
}
// Its number, and half bits of its inverse; below 2^-14 of 2^-9 times the inverse, which a half can hold.
__device__ __forceinline__ float limit_value(uint32_t lim) {
  return __uint_as_float((lim < 0x400u ? 134 - __clz(lim) : (lim >> 10) + 112) << 23);
}
__device__ __forceinline__ uint32_t limit_inverse(uint32_t lim) {
  if (lim < 0x400u) return (__clz(lim) - 1) << 10;
  const int e = lim >> 10;
  return e < 30 ? (30 - e) << 10 : 0x400u >> (e - 29);
}
// D = A B + C with an accumulator that is not overwritten.
__device__ __forceinline__ void mma_from(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0,
                                         uint32_t b1, const float (&c)[4]) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%10,%11,%12,%13};\n"
      : "=f"(d[0]), "=f"(d[1]), "=f"(d[2]), "=f"(d[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1), "f"(c[0]), "f"(c[1]), "f"(c[2]), "f"(c[3]));
}

// Mask of a packed pair of tokens (t, t + 1) that keeps those inside `len`.
__device__ __forceinline__ uint32_t pair_mask(int t, int len) {
  return (t < len ? 0x0000ffffu : 0u) | (t + 1 < len ? 0xffff0000u : 0u);
}

// One warp's share of a problem.  TPU: 16-token tiles per turn (one buffer); NT:
// blocks of 8 columns.  A column is a query head of the group; with ROWS that of one of
// several query tokens, which do not all see the last keys.
template <int P, int TPU, int NT, bool LSE, bool ROWS = false>
struct Q4Warp {
  static constexpr int TP = P / 16;                        // tiles of a page
  static constexpr int kPages = TP >= TPU ? 1 : TPU / TP;  // pages a unit touches
  static constexpr int kUPP = TP >= TPU ? TP / TPU : 1;    // units of a page
  static constexpr int kBufs = kWarpTiles / TPU;
  // tiles worked on together: with two blocks of columns the registers hold two tiles' logits
  static constexpr int kTiles = NT == 2 && !LSE && TPU == 4 ? 2 : TPU;
  static_assert(kTiles == TPU || 2 * kTiles == TPU, "one or two turns");
  static constexpr int kBufBytes = TPU * kTileBytes;
  // one block of heads has the registers to start its products at the codes' offset
  static constexpr bool kBiased = NT == 1;
  static_assert(!LSE || (kPages == 1 && kUPP == 1), "a unit of the page LSE is one page");
  static constexpr uint32_t kOne = 0x3c003c00u;  // two halves 1
  using At = Q4Tile<P, TPU>;

  Q4Shared& sh;
  const int warp, lane, g, c;
  int group;             // columns in use
  const uint32_t wbase;  // this warp's buffers
  // q of head 8 nt + g, dimensions 32 j + 8 c .. + 7, scaled into fp16
  uint32_t qf[NT][4][4];
  float init[NT][4][4];  // -72 sum of q over the scale group's 32 dimensions, heads 2c, 2c + 1 (twice)
  float fac[NT][2];      // logit factor of heads 2c, 2c + 1
  float R[NT][2], l[NT][2];  // their softmax reference (base 2) and sum
  float o[4][2][NT][4];  // their outputs: dimensions 32 j + 4 g + 2 half, + 1 (rows)
  uint32_t zlim, zup;    // the power of two above every value scale so far, and its inverse (twice), as halves
  int seq;               // units consumed so far: buffer seq % kBufs, phase seq / kBufs
  // ROWS: keys at the end that heads 2c, 2c + 1 and head g, and the first column, do not see
  int back[NT][2], back_g[NT], back_max;
  float* page_lse;       // LSE only
  size_t lse_stride;

  __device__ __forceinline__ Q4Warp(Q4Shared& s, uint32_t ring, int grp)
      : sh(s), warp(threadIdx.x >> 5), lane(threadIdx.x & 31), g((threadIdx.x & 31) >> 2), c(threadIdx.x & 3),
        group(grp), wbase(ring + (threadIdx.x >> 5) * kWarpTiles * kTileBytes), seq(0), back_max(0), page_lse(nullptr),
        lse_stride(0) {}

  __device__ __forceinline__ void set_limit(uint32_t lim) {
    zlim = lim == 0x3800u ? 0x3c00u : lim;  // 1/2 counts as 1, which costs no multiplication
    zup = limit_inverse(zlim) * 0x10001u;
  }
  // Two scales times the power of two under which the largest so far is below 1.
  __device__ __forceinline__ uint32_t scaled_up(uint32_t z) const {
    if (zlim < 0x400u) z = mul_f16x2(z, 0x60006000u);  // 2^9
    return mul_f16x2(z, zup);
  }

  __device__ __forceinline__ void reset() {
    set_limit(2);  // 2^-23: only zeros and the smallest half lie below
#pragma unroll
    for (int nt = 0; nt < NT; ++nt) {
      R[nt][0] = R[nt][1] = -INFINITY;
      l[nt][0] = l[nt][1] = 0.f;
#pragma unroll
      for (int j = 0; j < 4; ++j)
#pragma unroll
        for (int hf = 0; hf < 2; ++hf)
#pragma unroll
          for (int e = 0; e < 4; ++e) o[j][hf][nt][e] = 0.f;
    }
  }

  // The columns' queries (bf16), that of column h at row(h).
  template <typename Row>
  __device__ __forceinline__ void load_q(Row row, float scale_log2) {
    const int G = group;
#pragma unroll
    for (int nt = 0; nt < NT; ++nt) {
      const int h = 8 * nt + g;
      uint4 raw[4];
      uint32_t mx = 0;  // largest magnitude, as bf16 bits
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        raw[j] = make_uint4(0, 0, 0, 0);
        if (h < G)
          raw[j] = __ldg(reinterpret_cast<const uint4*>(row(h) + 32 * j + 8 * c));
        const uint32_t w[4] = {raw[j].x, raw[j].y, raw[j].z, raw[j].w};
#pragma unroll
        for (int k = 0; k < 4; ++k) mx = max(mx, max(w[k] & 0x7fffu, (w[k] >> 16) & 0x7fffu));
      }
      mx = max(mx, __shfl_xor_sync(0xffffffffu, mx, 1));
      mx = max(mx, __shfl_xor_sync(0xffffffffu, mx, 2));
      // 2^-e with e the exponent of the largest element (0 for a zero or
      // non-finite row), kept away from the ends of fp32's range
      int e = (int)(mx >> 7) - 127;
      e = mx == 0 || e > 127 ? 0 : min(max(e, -100), 126);
      const float down = __uint_as_float((uint32_t)(127 - e) << 23);
      float sum[4];
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const uint32_t w[4] = {raw[j].x, raw[j].y, raw[j].z, raw[j].w};
        sum[j] = 0.f;
#pragma unroll
        for (int k = 0; k < 4; ++k) {
          qf[nt][j][k] = pack_f16(__uint_as_float(w[k] << 16) * down, __uint_as_float(w[k] & 0xffff0000u) * down);
          sum[j] += f16_lo(qf[nt][j][k]) + f16_hi(qf[nt][j][k]);
        }
        sum[j] += __shfl_xor_sync(0xffffffffu, sum[j], 1);
        sum[j] += __shfl_xor_sync(0xffffffffu, sum[j], 2);
        if constexpr (kBiased)
#pragma unroll
          for (int k = 0; k < 2; ++k)
            init[nt][j][k] = init[nt][j][2 + k] = -72.f * __shfl_sync(0xffffffffu, sum[j], 8 * c + 4 * k);
      }
      const float up = scale_log2 * __uint_as_float((uint32_t)(127 + e) << 23);
#pragma unroll
      for (int k = 0; k < 2; ++k) fac[nt][k] = __shfl_sync(0xffffffffu, up, 8 * c + 4 * k);
    }
  }

  // behind(h): keys at the end that column h does not see (the first column the most).
  template <typename Behind>
  __device__ __forceinline__ void set_back(Behind behind) {
#pragma unroll
    for (int nt = 0; nt < NT; ++nt) {
#pragma unroll
      for (int k = 0; k < 2; ++k) back[nt][k] = behind(8 * nt + 2 * c + k);
      back_g[nt] = behind(8 * nt + g);
    }
    back_max = behind(0);
  }

  // One unit in buffer `buf`; WHOLE: every column sees all its tokens, else
  // left[t] counts those of tile t (two copies of the code, so that whole units
  // carry no masks).  Tiles t0 .. t0 + kTiles - 1 of the buffer.
  template <bool WHOLE>
  __device__ __forceinline__ void unit(uint32_t base, int buf, int t0, const int (&left)[kTiles]) {
    float sc[kTiles][NT][4];
    float mx[NT][2];
#pragma unroll
    for (int nt = 0; nt < NT; ++nt) mx[nt][0] = mx[nt][1] = -INFINITY;
    // ---- logits of the unit's tokens (rows g, g + 8 of each tile) ----
#pragma unroll
    for (int t = 0; t < kTiles; ++t) {
      const uint4 k0 = lds128(base + At::key_codes(t0 + t) + lane * 16), k1 = lds128(base + At::key_codes(t0 + t) + 512 + lane * 16);
      const uint2 s0 = lds64(base + At::key_scales(t0 + t) + g * 8), s1 = lds64(base + At::key_scales(t0 + t) + 64 + g * 8);
      const uint32_t kw0[4] = {k0.x, k0.y, k0.z, k0.w}, kw1[4] = {k1.x, k1.y, k1.z, k1.w};
      const float z0[4] = {f16_lo(s0.x), f16_hi(s0.x), f16_lo(s0.y), f16_hi(s0.y)};
      const float z1[4] = {f16_lo(s1.x), f16_hi(s1.x), f16_lo(s1.y), f16_hi(s1.y)};
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        uint32_t f0[4], f1[4];
        if constexpr (kBiased) {
          fields64(kw0[j], f0);
          fields64(kw1[j], f1);
        } else {
          q4_codes01(kw0[j], f0[0], f0[1]);
          q4_codes01(kw0[j] >> 8, f0[2], f0[3]);
          q4_codes01(kw1[j], f1[0], f1[1]);
          q4_codes01(kw1[j] >> 8, f1[2], f1[3]);
        }
#pragma unroll
        for (int nt = 0; nt < NT; ++nt) {
          float acc[4];
          if constexpr (kBiased) {
            mma_from(acc, f0[0], f1[0], f0[1], f1[1], qf[nt][j][0], qf[nt][j][1], init[nt][j]);
          } else {
            acc[0] = acc[1] = acc[2] = acc[3] = 0.f;
            mma_16816_f16(acc, f0[0], f1[0], f0[1], f1[1], qf[nt][j][0], qf[nt][j][1]);
          }
          mma_16816_f16(acc, f0[2], f1[2], f0[3], f1[3], qf[nt][j][2], qf[nt][j][3]);
          if (j == 0) {
            sc[t][nt][0] = z0[0] * acc[0];
            sc[t][nt][1] = z0[0] * acc[1];
            sc[t][nt][2] = z1[0] * acc[2];
            sc[t][nt][3] = z1[0] * acc[3];
          } else {
            sc[t][nt][0] = fmaf(z0[j], acc[0], sc[t][nt][0]);
            sc[t][nt][1] = fmaf(z0[j], acc[1], sc[t][nt][1]);
            sc[t][nt][2] = fmaf(z1[j], acc[2], sc[t][nt][2]);
            sc[t][nt][3] = fmaf(z1[j], acc[3], sc[t][nt][3]);
          }
        }
      }
      if constexpr (!WHOLE) {
#pragma unroll
        for (int nt = 0; nt < NT; ++nt)
#pragma unroll
          for (int k = 0; k < 2; ++k) {
            const int n = ROWS ? left[t] - back[nt][k] : left[t];
            if (g >= n) sc[t][nt][k] = -INFINITY;
            if (g + 8 >= n) sc[t][nt][2 + k] = -INFINITY;
          }
      }
#pragma unroll
      for (int nt = 0; nt < NT; ++nt)
#pragma unroll
        for (int k = 0; k < 2; ++k) mx[nt][k] = fmaxf(mx[nt][k], fmaxf(sc[t][nt][k], sc[t][nt][2 + k]));
    }
    // the unit's maximum per head, base 2 (the lanes of a column hold different tokens)
    auto whole_max = [&] {
#pragma unroll
      for (int nt = 0; nt < NT; ++nt)
#pragma unroll
        for (int k = 0; k < 2; ++k) {
          mx[nt][k] = fmaxf(mx[nt][k], __shfl_xor_sync(0xffffffffu, mx[nt][k], 4));
          mx[nt][k] = fmaxf(mx[nt][k], __shfl_xor_sync(0xffffffffu, mx[nt][k], 8));
          mx[nt][k] = fmaxf(mx[nt][k], __shfl_xor_sync(0xffffffffu, mx[nt][k], 16));
          mx[nt][k] *= fac[nt][k];  // the factor is positive
        }
    };
    if constexpr (LSE) {
      // a unit is one page (a slot of P = 64, a tile of P = 16)
      whole_max();
#pragma unroll
      for (int nt = 0; nt < NT; ++nt)
#pragma unroll
        for (int k = 0; k < 2; ++k) {
          float ps = 0.f;
#pragma unroll
          for (int t = 0; t < kTiles; ++t)
            ps += fast_exp2(fmaf(sc[t][nt][k], fac[nt][k], -mx[nt][k])) +
                  fast_exp2(fmaf(sc[t][nt][2 + k], fac[nt][k], -mx[nt][k]));
          ps += __shfl_xor_sync(0xffffffffu, ps, 4);
          ps += __shfl_xor_sync(0xffffffffu, ps, 8);
          ps += __shfl_xor_sync(0xffffffffu, ps, 16);
          const int h = 8 * nt + 2 * c + k;
          if (g == 0 && h < group) {
            page_lse[(size_t)h * lse_stride + sh.lp[warp][buf]] = (mx[nt][k] + fast_log2(ps)) * kLn2;
          }
        }
    } else {
      // The weights 2^(s - R) have to stay below 2^15, and the value scales below the
      // limit.  R or the limit is moved only when a token or a scale of the unit breaks
      // that; then the largest weight becomes 2^11.
      uint32_t top = 0;  // largest scale of this lane's 16 bytes, as half bits
      if (lane < 8 * kTiles) {
        const int t = t0 + (lane >> 3);
        uint4 w = lds128(base + At::value_scales(t) + (lane & 7) * 16);
        if constexpr (!WHOLE) {
          // each word: tokens 8 (lane%2) + (lane%8)/2 2, + 1 of tile t
          const int ln = P == 64 ? sh.len[warp][buf][0] - 16 * t : sh.len[warp][buf][t];
          const uint32_t msk = pair_mask(8 * (lane & 1) + 2 * ((lane & 7) >> 1), ln);
          w.x &= msk; w.y &= msk; w.z &= msk; w.w &= msk;
        }
        const uint32_t v = __vmaxu2(__vmaxu2(w.x, w.y), __vmaxu2(w.z, w.w));
        top = max(v & 0xffffu, v >> 16);
      }
      bool moved = top >= zlim;
#pragma unroll
      for (int nt = 0; nt < NT; ++nt)
#pragma unroll
        for (int k = 0; k < 2; ++k) moved |= fmaf(mx[nt][k], fac[nt][k], -R[nt][k]) > 15.f;
      if (__any_sync(0xffffffffu, moved)) {
        whole_max();
        float down = 1.f;
        uint32_t largest = __reduce_max_sync(0xffffffffu, top);
        if (largest >= 0x7c00u) {
          // a NaN stays one under any power of two, and must not take the others' bits
          top = 0;
          const int t = lane >> 3, u = 8 * (lane & 1) + 2 * ((lane & 7) >> 1);  // tile, first of two tokens
          const int ln = lane >= 8 * kTiles ? 0 : P == 64 ? sh.len[warp][buf][0] - 16 * (t0 + t) : sh.len[warp][buf][t0 + t];
#pragma unroll 1
          for (int e = 0; e < 8; ++e) {
            if (u + (e & 1) >= ln) continue;
            const uint32_t h = lds16(base + At::value_scales(t0 + t) + (lane & 7) * 16 + 2 * e);
            if (h < 0x7c00u) top = max(top, h);
          }
          largest = __reduce_max_sync(0xffffffffu, top);
        }
        if (largest >= zlim) {
          const float was = limit_value(zlim);
          set_limit(half_limit(largest));
          down = was * __uint_as_float((254u << 23) - __float_as_uint(limit_value(zlim)));  // powers of two
        }
#pragma unroll
        for (int nt = 0; nt < NT; ++nt)
#pragma unroll
          for (int k = 0; k < 2; ++k) {
            const float Rn = fmaxf(R[nt][k], mx[nt][k] - 11.f);
            float al = Rn == -INFINITY ? 1.f : fast_exp2(R[nt][k] - Rn);
            R[nt][k] = Rn;
            l[nt][k] *= al;
            al *= down;
#pragma unroll
            for (int j = 0; j < 4; ++j)
#pragma unroll
              for (int hf = 0; hf < 2; ++hf) {
                o[j][hf][nt][k] *= al;
                o[j][hf][nt][2 + k] *= al;
              }
          }
      }
      // ---- weights and the values they weight ---- (two copies of the code: a branch per
      // tile would keep the tiles' loads apart, 65.1 us for 63.9 on 32 sequences of 9K)
      auto weigh = [&](auto scaled) {
#pragma unroll
        for (int t = 0; t < kTiles; ++t) {
          uint32_t pb[NT][2];
#pragma unroll
          for (int nt = 0; nt < NT; ++nt) {
            float p[4];
#pragma unroll
            for (int k = 0; k < 4; ++k) {
              // a column that has seen no key yet has the reference -infinity
              const float ref = ROWS && !WHOLE && R[nt][k & 1] == -INFINITY ? 0.f : R[nt][k & 1];
              p[k] = fast_exp2(fmaf(sc[t][nt][k], fac[nt][k & 1], -ref));
              l[nt][k & 1] += p[k];
            }
            pb[nt][0] = transpose8x8(pack_f16(p[0], p[1]));  // tokens 2c, 2c + 1 of head g
            pb[nt][1] = transpose8x8(pack_f16(p[2], p[3]));  // tokens 8 + 2c, + 1
          }
          const uint4 v0 = lds128(base + At::value_codes(t0 + t) + lane * 16), v1 = lds128(base + At::value_codes(t0 + t) + 512 + lane * 16);
          uint4 z0 = lds128(base + At::value_scales(t0 + t) + c * 32), z1 = lds128(base + At::value_scales(t0 + t) + c * 32 + 16);
          if constexpr (!WHOLE) {
            // scales past the end may be anything, a NaN too
            const uint32_t m0 = pair_mask(2 * c, left[t]), m1 = pair_mask(8 + 2 * c, left[t]);
            z0.x &= m0; z0.y &= m0; z0.z &= m0; z0.w &= m0;
            z1.x &= m1; z1.y &= m1; z1.z &= m1; z1.w &= m1;
          }
          if constexpr (scaled) {
            z0 = make_uint4(scaled_up(z0.x), scaled_up(z0.y), scaled_up(z0.z), scaled_up(z0.w));
            z1 = make_uint4(scaled_up(z1.x), scaled_up(z1.y), scaled_up(z1.z), scaled_up(z1.w));
          }
          const uint32_t vw0[4] = {v0.x, v0.y, v0.z, v0.w}, vw1[4] = {v1.x, v1.y, v1.z, v1.w};
          const uint32_t zw0[4] = {z0.x, z0.y, z0.z, z0.w}, zw1[4] = {z1.x, z1.y, z1.z, z1.w};
#pragma unroll
          for (int j = 0; j < 4; ++j) {
            uint32_t a0, a1, a2, a3, b0, b1, b2, b3;
            q4_codes01(vw0[j], a0, a1);
            q4_codes01(vw1[j], a2, a3);
            q4_codes01(vw0[j] >> 8, b0, b1);
            q4_codes01(vw1[j] >> 8, b2, b3);
#pragma unroll
            for (int nt = 0; nt < NT; ++nt) {
              uint32_t p0 = mul_f16x2(pb[nt][0], zw0[j]), p1 = mul_f16x2(pb[nt][1], zw1[j]);
              if constexpr (ROWS && !WHOLE) {
                // 0 * NaN: a token that the column does not see
                p0 &= pair_mask(2 * c, left[t] - back_g[nt]);
                p1 &= pair_mask(8 + 2 * c, left[t] - back_g[nt]);
              }
              mma_16816_f16(o[j][0][nt], a0, a1, a2, a3, p0, p1);
              mma_16816_f16(o[j][1][nt], b0, b1, b2, b3, p0, p1);
            }
          }
        }
      };
      if (zup == kOne) weigh(std::false_type{});
      else weigh(std::true_type{});
    }
  }

  // n_pages pages, dealt out to the CTA's warps: page_of(i, lp, phys, len) gives page i
  // (len 0: left out); meanwhile() runs while the first copies are under way.  Called by
  // whole warps.
  template <typename PageOf, typename Meanwhile>
  __device__ __forceinline__ void run(const uint8_t* blocks, size_t head_stride, int hkv, int n_pages, int* err,
                                      PageOf page_of, Meanwhile meanwhile) {
    const int n_units = (n_pages + kPages - 1) / kPages * kUPP;
    const int n_mine = (n_units - warp + kW - 1) / kW;  // units warp, warp + 6, ...
    // the pages of units m0 .. m0 + 31 of this warp, one unit per lane
    int phys[kPages], len[kPages], lp0 = -1;
    auto resolve = [&](int m0) {
      const int u = warp + kW * (m0 + lane);
#pragma unroll
      for (int w = 0; w < kPages; ++w) {
        const int i = u / kUPP * kPages + w;
        phys[w] = 0;
        len[w] = 0;
        if (u < n_units && i < n_pages) {
          int lp = -1, ph = 0, ln = 0;
          page_of(i, lp, ph, ln);
          if (w == 0) lp0 = lp;
          phys[w] = ph;
          len[w] = max(0, ln - u % kUPP * TPU * 16);  // tokens from the unit's first tile on
        }
      }
    };
    // unit m into its buffer (all lanes; the copies are lane 0's)
    auto issue = [&](int m) {
      const int src = m & 31, buf = (seq + m) % kBufs;
      int ph[kPages], ln[kPages];
#pragma unroll
      for (int w = 0; w < kPages; ++w) {
        ph[w] = __shfl_sync(0xffffffffu, phys[w], src);
        ln[w] = __shfl_sync(0xffffffffu, len[w], src);
      }
      const int lp = LSE ? __shfl_sync(0xffffffffu, lp0, src) : 0;
      if (lane == 0) {
        constexpr uint32_t kBytes = (kUPP > 1 ? kBufBytes : LOCKS_KV_Q4_BLOCK_BYTES(P)) / (LSE ? 2 : 1);
        uint64_t* bar = &sh.full[warp][buf];
        uint32_t bytes = 0;
#pragma unroll
        for (int w = 0; w < kPages; ++w) {
          sh.len[warp][buf][w] = ln[w];
          bytes += ln[w] > 0 ? kBytes : 0u;
        }
        if (LSE) sh.lp[warp][buf] = lp;
        mbar_arrive_expect_tx(bar, bytes);
        const uint32_t dst = wbase + buf * kBufBytes;
#pragma unroll
        for (int w = 0; w < kPages; ++w) {
          if (ln[w] <= 0) continue;
          const uint8_t* block = blocks + (size_t)ph[w] * head_stride + (size_t)hkv * LOCKS_KV_Q4_BLOCK_BYTES(P);
          if constexpr (kUPP == 1) {
            bulk_load(dst + w * LOCKS_KV_Q4_BLOCK_BYTES(P), block, kBytes, bar);
          } else {
            // the unit's tiles of the page's four parts
            const int t = (warp + kW * m) % kUPP * TPU;
            bulk_load(dst, block + 1024 * t, 1024 * TPU, bar);
            bulk_load(dst + 1024 * TPU, block + 64 * P + 128 * t, 128 * TPU, bar);
            bulk_load(dst + 1152 * TPU, block + 72 * P + 1024 * t, 1024 * TPU, bar);
            bulk_load(dst + 2176 * TPU, block + 136 * P + 128 * t, 128 * TPU, bar);
          }
        }
      }
    };
    int issued = 0, done = 0;
    if (n_mine > 0) resolve(0);
    for (; issued < min(kBufs, n_mine); ++issued) issue(issued);
    meanwhile();
    for (; done < n_mine; ++done) {
      const int s = seq + done, buf = s % kBufs;
      if (!__all_sync(0xffffffffu, mbar_wait(&sh.full[warp][buf], (s / kBufs) & 1))) {
        if (lane == 0) set_error(err, kDevErrTimeout);
        break;
      }
      const uint32_t base = wbase + buf * kBufBytes;
#pragma unroll 1
      for (int t0 = 0; t0 < TPU; t0 += kTiles) {
        // tokens from each tile's first on (one page's, or a page per tile)
        int left[kTiles];
        bool whole = true, any = false;
#pragma unroll
        for (int t = 0; t < kTiles; ++t) {
          left[t] = P == 64 ? sh.len[warp][buf][0] - 16 * (t0 + t) : sh.len[warp][buf][t0 + t];
          whole &= left[t] >= (ROWS ? 16 + back_max : 16);
          any |= left[t] > 0;
        }
        if (whole) unit<true>(base, buf, t0, left);
        else if (any) unit<false>(base, buf, t0, left);
      }
      __syncwarp();  // every lane is done with the buffer
      if (issued < n_mine) {
        if ((issued & 31) == 0) resolve(issued);
        issue(issued);
        ++issued;
      }
    }
    // after a failed wait: let the copies in flight land before the memory is reused
    if (done < n_mine && lane == 0)
      for (int m = done; m < issued; ++m) (void)mbar_wait(&sh.full[warp][(seq + m) % kBufs], ((seq + m) / kBufs) & 1);
    __syncwarp();
    seq += issued;
  }

  // The six warps' states to the CTA's: (R, sum) in sh.cta_m, sh.cta_l and O [16][128]
  // in octa (shared memory over the buffers; whole CTA, ends with a barrier).
  __device__ __forceinline__ float* merge(uint8_t* ring) {
    float* so = reinterpret_cast<float*>(ring);  // [kW][8 NT][kOStride]
    float* octa = so + kW * 8 * NT * kOStride;   // [16][128]
    const int tid = threadIdx.x, G = group;
    const float back = limit_value(zlim);  // the power of two that the scales were held under
    __syncthreads();  // the buffers are no longer read, nor written by copies
#pragma unroll
    for (int nt = 0; nt < NT; ++nt)
#pragma unroll
      for (int k = 0; k < 2; ++k) {
        float s = l[nt][k];
        s += __shfl_xor_sync(0xffffffffu, s, 4);
        s += __shfl_xor_sync(0xffffffffu, s, 8);
        s += __shfl_xor_sync(0xffffffffu, s, 16);
        const int h = 8 * nt + 2 * c + k;
        if (g == 0) {
          sh.m[warp][h] = R[nt][k];
          sh.l[warp][h] = s;
        }
        if (h < G)
#pragma unroll
          for (int j = 0; j < 4; ++j)
            *reinterpret_cast<float4*>(so + (warp * 8 * NT + h) * kOStride + 32 * j + 4 * g) =
                make_float4(o[j][0][nt][k] * back, o[j][0][nt][2 + k] * back, o[j][1][nt][k] * back,
                            o[j][1][nt][2 + k] * back);
      }
    __syncthreads();
    if (tid < G) {
      float M = -INFINITY;
#pragma unroll
      for (int w = 0; w < kW; ++w) M = fmaxf(M, sh.m[w][tid]);
      float Ls = 0.f;
#pragma unroll
      for (int w = 0; w < kW; ++w) {
        const float f = M == -INFINITY ? 1.f : fast_exp2(sh.m[w][tid] - M);
        sh.f[w][tid] = f;
        Ls = fmaf(sh.l[w][tid], f, Ls);
      }
      sh.cta_m[tid] = M;
      sh.cta_l[tid] = Ls;
    }
    __syncthreads();
    for (int e = tid; e < G * (kHeadDim / 4); e += kThreads) {
      const int h = e / (kHeadDim / 4), d4 = 4 * (e % (kHeadDim / 4));
      float4 O = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
      for (int w = 0; w < kW; ++w) {
        const float f = sh.f[w][h];
        const float4 v = *reinterpret_cast<const float4*>(so + (w * 8 * NT + h) * kOStride + d4);
        O.x = fmaf(v.x, f, O.x);
        O.y = fmaf(v.y, f, O.y);
        O.z = fmaf(v.z, f, O.z);
        O.w = fmaf(v.w, f, O.w);
      }
      *reinterpret_cast<float4*>(octa + h * kHeadDim + d4) = O;
    }
    __syncthreads();
    return octa;
  }
};

__device__ __forceinline__ uint8_t* align_ring(uint8_t* raw) {
  return reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(raw) + 127) & ~uintptr_t(127));
}
__device__ __forceinline__ int checked_length(const AttendArgs& a, int b, int P, bool says) {
  const int L = a.seq_lens[b];
  if (L >= 0 && L <= a.max_pages * P) return L;
  if (says) set_error(a.err, LOCKS_DEVERR_LENGTHS);
  return L < 0 ? 0 : a.max_pages * P;
}
// Physical page of logical page lp of sequence b, -1 (reported) when there is none.
__device__ __forceinline__ int physical_page(const AttendArgs& a, int b, int lp) {
  const int ph = a.block_table[(size_t)b * a.max_pages + lp];
  if (ph >= 0 && ph < a.pages_total) return ph;
  set_error(a.err, LOCKS_DEVERR_BLOCK_TABLE);
  return -1;
}
__device__ __forceinline__ void store_result(const AttendArgs& a, size_t row, int col, float O, float M, float Ls) {
  a.out[row * kHeadDim + col] = __bfloat16_as_ushort(__float2bfloat16_rn(Ls == 0.f ? 0.f : O / Ls));
  if (a.lse && col == 0) a.lse[row] = Ls == 0.f ? -INFINITY : (M + fast_log2(Ls)) * kLn2;
}

// ---- every page ------------------------------------------------------------------
// A problem is a KV head of a sequence with, for the newest tokens of a sequence (ROWS),
// up to 8 NT of their (token, head) rows as columns; its blocks of rows follow each other
// in the line, so that they read the pages at about the same time.
// Partial results a.part_ml, a.part_o: two per CTA (its first problem, which another
// CTA began, and the one it begins itself), [2 CTA + begins][G or 8 NT].  A second kernel
// joins those of a problem, each column on its own.  (The last CTA of a problem to finish
// did it before, alone, in two levels: 17 of 110 us for 16 heads and 152 CTAs per
// problem, which took 95 then; one head over 4096 tokens 10.3 us, 6.4 with the join.)
struct Q4Seq {
  int keys;             // that its newest token sees
  int row0, n, start;   // its query tokens: first row, number, position of the first
};
template <int P, bool ROWS>
__device__ __forceinline__ Q4Seq sequence(const AttendArgs& a, int b, bool says) {
  Q4Seq s;
  const int len = checked_length(a, b, P, says);
  s.keys = len;
  s.row0 = b;
  s.n = 1;
  s.start = len - 1;
  if constexpr (ROWS) {
    int n = len > 0 ? 1 : 0;
    if (a.cu_tokens) {
      s.row0 = a.cu_tokens[b];
      const int end = a.cu_tokens[b + 1];
      n = end - s.row0;
      if (s.row0 < 0 || n < 0 || end > a.total) {
        if (says) set_error(a.err, LOCKS_DEVERR_LENGTHS);
        n = 0;
      }
    }
    if (says && (n > len || n > a.max_tokens)) set_error(a.err, LOCKS_DEVERR_LENGTHS);
    s.n = min(n, a.max_tokens);
    s.start = len - n;
    s.keys = s.n > 0 ? max(0, min(len, s.start + s.n)) : 0;
  }
  return s;
}

// The line of all slots: sequence by sequence, head by head, block of COLS rows by block.
template <int P, bool ROWS, int COLS>
struct Q4Line {
  const AttendArgs& a;
  long long total = 0, C = 1;  // slots, and the CTAs that have a part of them
  // the sequence at hand: its first slot, slots per problem, problems per head
  int b = 0, nb = 0, n_blocks = 1;
  long long first = 0;
  Q4Seq q = {};

  __device__ __forceinline__ explicit Q4Line(const AttendArgs& args) : a(args) {}
  __device__ __forceinline__ int blocks_of(const Q4Seq& s) const { return ROWS ? (s.n * a.group + COLS - 1) / COLS : 1; }
  __device__ __forceinline__ int slots_of(int i, bool says) const {  // per head
    const Q4Seq s = sequence<P, ROWS>(a, i, says);
    return (s.keys + kPage - 1) / kPage * blocks_of(s);
  }
  // Whole warps: all slots, and those before sequence `until`.
  __device__ __forceinline__ long long measure(int ctas, int until, bool says) {
    long long before = 0;
#pragma unroll 4
    for (int i = threadIdx.x & 31; i < a.batch; i += 32) {
      const int n = slots_of(i, says);
      total += n;
      before += i < until ? n : 0;
    }
#pragma unroll
    for (int d = 16; d; d >>= 1) {
      total += __shfl_xor_sync(0xffffffffu, total, d);
      before += __shfl_xor_sync(0xffffffffu, before, d);
    }
    total *= a.num_kv_heads;
    // with fewer slots than CTAs the last CTAs get none, so that no part is empty
    C = min((long long)ctas, max(total, 1LL));
    return before * a.num_kv_heads;
  }
  __device__ __forceinline__ long long begin(long long cta) const { return cta < C ? total * cta / C : total; }
  // the CTA whose part holds slot y
  __device__ __forceinline__ long long owner(long long y) const { return ((y + 1) * C - 1) / total; }
  __device__ __forceinline__ void load() {
    q = sequence<P, ROWS>(a, b, false);
    n_blocks = blocks_of(q);
    nb = (q.keys + kPage - 1) / kPage;
  }
  // Whole warps: to the sequence that holds slot y, 32 at a time.
  __device__ __forceinline__ void skip(long long y) {
    const int lane = threadIdx.x & 31;
    while (b < a.batch) {
      // slots of this lane's sequence and those of the 32 before it
      long long upto = b + lane < a.batch ? (long long)slots_of(b + lane, false) * a.num_kv_heads : 0;
      const long long own = upto;
#pragma unroll
      for (int d = 1; d < 32; d *= 2) {
        const long long other = __shfl_up_sync(0xffffffffu, upto, d);
        if (lane >= d) upto += other;
      }
      const uint32_t past = __ballot_sync(0xffffffffu, y < first + upto);
      if (past) {
        const int at = __ffs(past) - 1;
        b += at;
        first += __shfl_sync(0xffffffffu, upto - own, at);
        return;
      }
      first += __shfl_sync(0xffffffffu, upto, 31);
      b += 32;
    }
  }
  // The sequence that holds slot y (from the current one on).
  __device__ __forceinline__ void seek(long long y) {
    while (b < a.batch) {
      load();
      const long long n = (long long)nb * n_blocks * a.num_kv_heads;
      if (y < first + n) return;
      first += n;
      ++b;
    }
  }
  // Problem `prob` of the sequence at hand: its head, first row of the head's, columns.
  __device__ __forceinline__ int head(int prob) const { return prob / n_blocks; }
  __device__ __forceinline__ int row0(int prob) const { return ROWS ? prob % n_blocks * COLS : 0; }
  __device__ __forceinline__ int columns(int prob) const {
    return ROWS ? min(COLS, q.n * a.group - row0(prob)) : a.group;
  }
  // Column x of it: the row in the outputs.
  __device__ __forceinline__ size_t out_row(int prob, int x) const {
    const int r = row0(prob) + x, i = ROWS ? r / a.group : 0, e = ROWS ? r % a.group : x;
    return ((size_t)(q.row0 + i) * a.num_kv_heads + head(prob)) * a.group + e;
  }
};

template <int P, int TPU, int NT, bool ROWS>
__global__ void __launch_bounds__(kThreads, 2) attend_q4_dense_kernel(const AttendArgs a) {
  extern __shared__ __align__(128) uint8_t ring_raw[];
  __shared__ Q4Shared sh;
  uint8_t* ring = align_ring(ring_raw);
  constexpr int kPPS = kPage / P;  // pages of a slot
  const int tid = threadIdx.x, lane = tid & 31;
  const int G = a.group, hkv_n = a.num_kv_heads;
  constexpr int kCols = 8 * NT;
  static_assert(!ROWS || kCols == kQ4RowColumns, "the columns of a partial result");
  const int pitch = ROWS ? kCols : G;  // columns of a partial result
  Q4Warp<P, TPU, NT, false, ROWS> w(sh, smem_u32(ring), G);
  if (lane == 0) {
    for (int s = 0; s < kWarpTiles; ++s) mbar_init(&sh.full[w.warp][s], 1);
    fence_mbar_init();
  }
  __syncthreads();
  pdl_wait();

  Q4Line<P, ROWS, kCols> line(a);
  const long long cta = blockIdx.x;
  line.measure(gridDim.x, 0, cta == 0 && tid < 32);
  long long at = line.begin(cta);
  const long long end = line.begin(cta + 1);
  // sequences without a token have no slots and get their rows here
  for (int b0 = 32 * blockIdx.x; b0 < a.batch; b0 += 32 * gridDim.x) {
    Q4Seq s = {};
    if (b0 + lane < a.batch) s = sequence<P, ROWS>(a, b0 + lane, false);
    for (uint32_t none = __ballot_sync(0xffffffffu, s.keys == 0 && s.n > 0); none; none &= none - 1) {
      const int src = __ffs(none) - 1;
      const int row0 = __shfl_sync(0xffffffffu, s.row0, src), n = __shfl_sync(0xffffffffu, s.n, src);
      for (int e = tid; e < n * hkv_n * G * kHeadDim; e += kThreads)
        store_result(a, (size_t)row0 * hkv_n * G + e / kHeadDim, e % kHeadDim, 0.f, 0.f, 0.f);
    }
  }
  line.skip(at);
  while (at < end) {
    line.seek(at);
    const int nb = line.nb, prob = (int)((at - line.first) / nb), h = line.head(prob);
    const long long p0 = line.first + (long long)prob * nb, p1 = p0 + nb;  // its slots in the line
    const int s0 = (int)(at - p0), s1 = (int)(min(end, p1) - p0);          // this CTA's of them
    const int L = line.q.keys, pg0 = s0 * kPPS, pg1 = min(s1 * kPPS, (L + P - 1) / P);
    const int cols = line.columns(prob), r0 = line.row0(prob);
    auto query = [&](int x) {
      if constexpr (!ROWS) return a.q + line.out_row(prob, x) * kHeadDim;
      return a.q + (size_t)(line.q.row0 + (r0 + x) / G) * a.q_stride + (size_t)(h * G + (r0 + x) % G) * kHeadDim;
    };
    w.group = cols;
    if constexpr (ROWS) w.set_back([&](int x) { return x < cols ? L - max(0, line.q.start + (r0 + x) / G + 1) : 0; });
    w.run(reinterpret_cast<const uint8_t*>(a.k_pool16), (size_t)hkv_n * LOCKS_KV_Q4_BLOCK_BYTES(P), h, pg1 - pg0, a.err,
          [&](int i, int& lp, int& phys, int& len) {
            lp = pg0 + i;
            phys = physical_page(a, line.b, lp);
            // with rows all that follow, against which a column's own end is counted
            len = phys < 0 ? 0 : ROWS ? L - lp * P : min(P, L - lp * P);
          },
          [&] {
            w.reset();
            w.load_q(query, a.scale_log2);
          });
    if (p0 + s1 >= end) pdl_launch_dependents();
    const float* octa = w.merge(ring);
    if (s0 == 0 && s1 == nb) {
      for (int e = tid; e < cols * kHeadDim; e += kThreads)
        store_result(a, line.out_row(prob, e / kHeadDim), e % kHeadDim, octa[e], sh.cta_m[e / kHeadDim],
                     sh.cta_l[e / kHeadDim]);
    } else {
      const size_t mine = (2 * (size_t)cta + (s0 == 0 ? 1 : 0)) * pitch;
      for (int e = tid; e < cols * (kHeadDim / 4); e += kThreads)
        reinterpret_cast<float4*>(a.part_o + mine * kHeadDim)[e] = reinterpret_cast<const float4*>(octa)[e];
      if (tid < cols) a.part_ml[mine + tid] = make_float2(sh.cta_m[tid], sh.cta_l[tid]);
    }
    at = p0 + s1;
    // the buffers were written with ordinary stores: before the next copies into them
    fence_proxy_async();
    __syncthreads();
  }
}

// Joins the partial results of the problems that were cut.  Grid (a.n_joins, columns):
// problem by problem where there are fewer than CTAs of the other kernel (a.join_blocks
// blocks of rows per head at most), else the problem that CTA blockIdx.x begins and
// does not finish.
constexpr int kJoinThreads = 256;
constexpr int kJoinWarps = kJoinThreads / 32;
constexpr int kJoinFlight = 8;  // partials that a warp loads at once

template <int P, bool ROWS, int COLS>
__global__ void __launch_bounds__(kJoinThreads) join_kernel(const AttendArgs a) {
  __shared__ float so[kJoinWarps][kHeadDim];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, h = blockIdx.y;
  // the other kernel's inputs were complete before it let this one begin
  Q4Line<P, ROWS, COLS> line(a);
  int prob = 0;
  long long p0 = 0;
  bool cut = false;
  if (a.join_blocks > 0) {
    const int per_seq = a.num_kv_heads * a.join_blocks;
    line.b = blockIdx.x / per_seq;
    prob = blockIdx.x % per_seq;
    line.first = line.measure(a.n_splits, line.b, false);
    line.load();
    if (line.nb > 0 && prob < line.n_blocks * a.num_kv_heads) {
      p0 = line.first + (long long)prob * line.nb;
      cut = line.owner(p0) != line.owner(p0 + line.nb - 1);
    }
  } else {
    line.measure(a.n_splits, 0, false);
    const long long at = line.begin(blockIdx.x), end = line.begin((long long)blockIdx.x + 1);
    if (at < end) {
      line.skip(end - 1);
      line.seek(end - 1);
      prob = (int)((end - 1 - line.first) / line.nb);
      p0 = line.first + (long long)prob * line.nb;
      cut = p0 >= at && p0 + line.nb > end;
    }
  }
  cut = cut && h < line.columns(prob);
  // also where there is nothing to join: whatever follows may rely on this kernel's end
  pdl_wait();
  pdl_launch_dependents();
  if (!cut) return;
  const int pitch = ROWS ? COLS : a.group;
  const int c0 = (int)line.owner(p0), n = (int)line.owner(p0 + line.nb - 1) - c0 + 1;
  auto slot = [&](int i) { return (size_t)(2 * (c0 + i) + (i == 0 ? 1 : 0)) * pitch + h; };
  // a warp takes partials warp, warp + 8, ...; each warp finds the reference of all
  float M = -INFINITY, L = 0.f;
  for (int i = lane; i < n; i += 32) M = fmaxf(M, __ldcg(a.part_ml + slot(i)).x);
  M = warp_max(M);
  float4 O = make_float4(0.f, 0.f, 0.f, 0.f);
  for (int i0 = warp; i0 < n; i0 += kJoinWarps * kJoinFlight) {
    float4 v[kJoinFlight];
    float2 ml[kJoinFlight];
#pragma unroll
    for (int k = 0; k < kJoinFlight; ++k) {
      const int i = i0 + kJoinWarps * k;
      v[k] = make_float4(0.f, 0.f, 0.f, 0.f);
      ml[k] = make_float2(M, 0.f);
      if (i >= n) continue;
      v[k] = __ldcg(reinterpret_cast<const float4*>(a.part_o + slot(i) * kHeadDim) + lane);
      ml[k] = __ldcg(a.part_ml + slot(i));
    }
#pragma unroll
    for (int k = 0; k < kJoinFlight; ++k) {
      const float f = M == -INFINITY ? 1.f : fast_exp2(ml[k].x - M);
      L = fmaf(ml[k].y, f, L);
      O.x = fmaf(v[k].x, f, O.x);
      O.y = fmaf(v[k].y, f, O.y);
      O.z = fmaf(v[k].z, f, O.z);
      O.w = fmaf(v[k].w, f, O.w);
    }
  }
  __shared__ float sl[kJoinWarps];
  *reinterpret_cast<float4*>(&so[warp][4 * lane]) = O;
  if (lane == 0) sl[warp] = L;
  __syncthreads();
  if (threadIdx.x >= kHeadDim) return;
  float Os = 0.f, Ls = 0.f;
#pragma unroll
  for (int k = 0; k < kJoinWarps; ++k) {
    Os += so[k][threadIdx.x];
    Ls += sl[k];
  }
  store_result(a, line.out_row(prob, h), threadIdx.x, Os, M, Ls);
}

// ---- a page list, or the exact page log-sum-exp ------------------------------------
// Grid (CTAs of the cluster, B * Hkv); for the page LSE (splits, B * Hkv), no clusters.
template <int MODE, int P, int TPU, int NT>
__global__ void __launch_bounds__(kThreads, 2) attend_q4_kernel(const AttendArgs a) {
  constexpr bool LSE = MODE == kAttendPageLse;
  extern __shared__ __align__(128) uint8_t ring_raw[];
  __shared__ Q4Shared sh;
  uint8_t* ring = align_ring(ring_raw);
  const int tid = threadIdx.x, lane = tid & 31;
  const int split = blockIdx.x, bh = blockIdx.y;
  const int b = bh / a.num_kv_heads, hkv = bh % a.num_kv_heads;
  const int G = a.group;
  Q4Warp<P, TPU, NT, LSE> w(sh, smem_u32(ring), G);
  constexpr int kPages = Q4Warp<P, TPU, NT, LSE>::kPages;
  if (lane == 0) {
    for (int s = 0; s < kWarpTiles; ++s) mbar_init(&sh.full[w.warp][s], 1);
    if (w.warp == 0) mbar_init(&sh.recv, a.cluster);
    fence_mbar_init();
  }
  __syncthreads();
  if (!LSE) cluster_arrive();  // matched by the wait before the first remote access
  pdl_wait();

  const int L = checked_length(a, b, P, tid == 0 && split == 0);
  const int n_pages = (L + P - 1) / P;
  int ns = 0, cnt = 0, n_items = n_pages;
  if (!LSE) {
    const int cap = min(L / P, a.max_pages);
    ns = min(max(a.n_summarized[b], 0), cap);
    const int kcap = min(a.k_max, ns);
    cnt = a.sel_count[bh];
    if (cnt < 0 || cnt > kcap) {
      if (tid == 0) set_error(a.err, LOCKS_DEVERR_SEL_PAGE);
      cnt = cnt < 0 ? 0 : kcap;
    }
    n_items = cnt + (n_pages - ns);
  }
  // this CTA's pages (whole units)
  const int ipc = ((n_items + a.n_splits - 1) / a.n_splits + kPages - 1) / kPages * kPages;
  const int i0 = min(n_items, split * ipc), i1 = min(n_items, i0 + ipc);
  const size_t row = (size_t)b * a.num_kv_heads * G + (size_t)hkv * G;
  if (LSE) {
    w.page_lse = a.page_lse + row * a.max_pages;
    w.lse_stride = a.max_pages;
  }
  w.run(reinterpret_cast<const uint8_t*>(a.k_pool16), (size_t)a.num_kv_heads * LOCKS_KV_Q4_BLOCK_BYTES(P), hkv, i1 - i0,
        a.err, [&](int k, int& lp, int& phys, int& len) {
          const int i = i0 + k;
          if (!LSE && i < cnt) {
            lp = a.sel_pages[(size_t)bh * a.k_max + i];
            // inside the decode step the top-k also wrote the physical pages
            phys = a.sel_phys ? a.sel_phys[(size_t)bh * a.k_max + i] : 0;
            if (lp < 0 || lp >= ns) {
              set_error(a.err, LOCKS_DEVERR_SEL_PAGE);
              return;
            }
            if (!a.sel_phys) {
              phys = physical_page(a, b, lp);
            } else if (phys < 0 || phys >= a.pages_total) {
              set_error(a.err, LOCKS_DEVERR_BLOCK_TABLE);
              phys = -1;
            }
          } else {
            lp = LSE ? i : ns + (i - cnt);
            phys = physical_page(a, b, lp);
          }
          len = phys >= 0 ? min(P, L - lp * P) : 0;
        },
        [&] {
          w.reset();
          w.load_q([&](int h) { return a.q + (row + h) * kHeadDim; }, a.scale_log2);
        });
  pdl_launch_dependents();
  if constexpr (!LSE) {
    const float* octa = w.merge(ring);
    float* recv_o = reinterpret_cast<float*>(ring) + kW * 8 * NT * kOStride + 16 * kHeadDim;
    float2* recv_ml = reinterpret_cast<float2*>(recv_o + 16 * kHeadDim);
    static_assert((kW * 8 * NT * kOStride + 32 * kHeadDim) * 4 + kRecvMl <= kRing, "the merge fits the buffers");
    const int CS = a.cluster;
    const uint32_t rank = cluster_ctarank();
    const int cols = kHeadDim / CS;
    cluster_wait();  // every CTA of the cluster has set up its receive barrier
    cluster_sync();  // and is done with its buffers, which the others now write
    const uint32_t ro = smem_u32(recv_o), rml = smem_u32(recv_ml);
    for (int e = tid; e < G * (kHeadDim / 4); e += kThreads) {
      const int h = e / (kHeadDim / 4), c4 = 4 * (e % (kHeadDim / 4));
      const float4 v = *reinterpret_cast<const float4*>(octa + h * kHeadDim + c4);
      st_dsmem_f4(dsmem_addr(ro + 4 * (((int)rank * G + h) * cols + c4 % cols), c4 / cols), v);
    }
    for (int e = tid; e < CS * G; e += kThreads) {
      const int dst = e / G, h = e % G;
      st_dsmem_f2(dsmem_addr(rml + 8 * ((int)rank * 16 + h), dst), make_float2(sh.cta_m[h], sh.cta_l[h]));
    }
    __syncthreads();  // the whole CTA's stores precede the release arrivals
    if (tid < CS) mbar_arrive_remote(dsmem_addr(smem_u32(&sh.recv), tid));
    if (!mbar_wait_cluster(&sh.recv, 0) && tid == 0) set_error(a.err, kDevErrTimeout);
    for (int e = tid; e < G * cols; e += kThreads) {
      const int h = e / cols, cc = e % cols;
      float M = -INFINITY;
      for (int rr = 0; rr < CS; ++rr) M = fmaxf(M, recv_ml[rr * 16 + h].x);
      float Ls = 0.f, O = 0.f;
      for (int rr = 0; rr < CS; ++rr) {
        const float2 ml = recv_ml[rr * 16 + h];
        const float f = M == -INFINITY ? 1.f : fast_exp2(ml.x - M);
        Ls = fmaf(ml.y, f, Ls);
        O = fmaf(recv_o[(rr * G + h) * cols + cc], f, O);
      }
      store_result(a, row + h, (int)rank * cols + cc, O, M, Ls);
    }
  }
}

using Kern = void (*)(const AttendArgs);

template <int MODE, int P>
Kern pick(int group, int tiles) {
  if constexpr (MODE == kAttendPageLse) {
    // a unit is one page: four tiles, or one
    return group <= 8 ? attend_q4_kernel<MODE, P, P / 16, 1> : attend_q4_kernel<MODE, P, P / 16, 2>;
  } else if constexpr (MODE == kAttendSparse) {
    if (group <= 8) return tiles == 4 ? attend_q4_kernel<MODE, P, 4, 1> : attend_q4_kernel<MODE, P, 1, 1>;
    return tiles == 4 ? attend_q4_kernel<MODE, P, 4, 2> : attend_q4_kernel<MODE, P, 1, 2>;
  } else {
    if (group <= 8) return tiles == 4 ? attend_q4_dense_kernel<P, 4, 1, false> : attend_q4_dense_kernel<P, 1, 1, false>;
    return tiles == 4 ? attend_q4_dense_kernel<P, 4, 2, false> : attend_q4_dense_kernel<P, 1, 2, false>;
  }
}

Kern kernel_of(int mode, int group, int page_size, int tiles) {
  const bool p16 = page_size == 16;
  if (mode == kAttendSparse) return p16 ? pick<kAttendSparse, 16>(group, tiles) : pick<kAttendSparse, 64>(group, tiles);
  if (mode == kAttendDense) return p16 ? pick<kAttendDense, 16>(group, tiles) : pick<kAttendDense, 64>(group, tiles);
  return p16 ? pick<kAttendPageLse, 16>(group, tiles) : pick<kAttendPageLse, 64>(group, tiles);
}

bool prepare(Kern k, int cluster) {
  if (cudaFuncSetAttribute(k, cudaFuncAttributeMaxDynamicSharedMemorySize, kSmem) != cudaSuccess) return false;
  return cluster <= 8 || cudaFuncSetAttribute(k, cudaFuncAttributeNonPortableClusterSizeAllowed, 1) == cudaSuccess;
}

int active_clusters(Kern k, int cs) {
  if (!prepare(k, cs)) return 0;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(cs, 1, 1);
  cfg.blockDim = dim3(kThreads, 1, 1);
  cfg.dynamicSmemBytes = kSmem;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim.x = cs;
  attr[0].val.clusterDim.y = 1;
  attr[0].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  int n = 0;
  if (cudaOccupancyMaxActiveClusters(&n, k, &cfg) != cudaSuccess) {
    (void)cudaGetLastError();
    return 0;
  }
  return n;
}

}  // namespace

int attend_q4_active_clusters(int group, int page_size, int tiles, int cs) {
  // one entry per kernel variant, cluster size and device; the answer depends on nothing else
  static int cache[2][2][2][5][64] = {};
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= 64 || cs < 1 || cs > 16) return 1;
  int& slot = cache[group > 8][page_size == 16][tiles == 4][31 - __builtin_clz((unsigned)cs)][dev];
  if (slot == 0) {
    const int n = active_clusters(kernel_of(kAttendSparse, group, page_size, tiles), cs);
    slot = n > 0 ? n : -1;
  }
  return slot > 0 ? slot : 0;
}

static cudaError_t launch_kernel(Kern k, const AttendArgs& a, int mode, cudaStream_t s) {
  if (!prepare(k, a.cluster)) return cudaErrorInvalidConfiguration;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(a.n_splits, mode == kAttendDense ? 1 : a.batch * a.num_kv_heads, 1);
  cfg.blockDim = dim3(kThreads, 1, 1);
  cfg.dynamicSmemBytes = kSmem;
  cfg.stream = s;
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim.x = a.cluster;
  attr[0].val.clusterDim.y = 1;
  attr[0].val.clusterDim.z = 1;
  attr[1].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[1].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 2;
  return cudaLaunchKernelEx(&cfg, k, a);
}

// After the kernel over every page: `columns` of a problem, `blocks` of rows per head.
template <bool ROWS, int COLS>
static cudaError_t launch_join(AttendArgs a, int columns, int blocks, cudaStream_t s) {
  const long long problems = (long long)a.batch * a.num_kv_heads * blocks;
  a.join_blocks = problems <= a.n_splits ? blocks : 0;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)(a.join_blocks ? problems : a.n_splits), columns, 1);
  cfg.blockDim = dim3(kJoinThreads, 1, 1);
  cfg.stream = s;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return a.page_size == 16 ? cudaLaunchKernelEx(&cfg, join_kernel<16, ROWS, COLS>, a)
                           : cudaLaunchKernelEx(&cfg, join_kernel<64, ROWS, COLS>, a);
}

cudaError_t launch_attend_q4(const AttendArgs& a, int mode, int tiles, cudaStream_t s) {
  const cudaError_t e = launch_kernel(kernel_of(mode, a.group, a.page_size, tiles), a, mode, s);
  if (e != cudaSuccess || mode != kAttendDense || a.n_splits == 1) return e;
  return launch_join<false, 8>(a, a.group, 1, s);
}

template <int P>
static Kern rows_kernel(int tiles) {
  return tiles == 4 ? attend_q4_dense_kernel<P, 4, 1, true> : attend_q4_dense_kernel<P, 1, 1, true>;
}

cudaError_t launch_attend_q4_rows(const AttendArgs& a, int tiles, cudaStream_t s) {
  const cudaError_t e =
      launch_kernel(a.page_size == 16 ? rows_kernel<16>(tiles) : rows_kernel<64>(tiles), a, kAttendDense, s);
  if (e != cudaSuccess || a.n_splits == 1) return e;
  const int rows = a.max_tokens * a.group;
  return launch_join<true, kQ4RowColumns>(a, std::min(rows, kQ4RowColumns), (rows + kQ4RowColumns - 1) / kQ4RowColumns, s);
}

}  // namespace locks
