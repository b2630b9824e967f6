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
//  - Codes are stored as u = code + 8.  A pair of 4-bit fields under a fixed fp16
//    exponent is the pair (64 + u) or (1024 + u) exactly: one logical operation.
//  - Keys: the matrix instruction runs on (64 + u) = code + 72 and its accumulator
//    starts at -72 sum_d q_d (per head and scale group), so nothing is subtracted
//    from the codes.  Values, whose sums run over all tokens, are freed of the
//    offset by one packed subtraction (an offset carried through thousands of
//    accumulations would cost digits).
//  - The products have M = tokens (or dimensions) and N = 8 query heads, so that
//    the group's few heads sit on the instruction's short side, and the pages store
//    the codes in the order in which a lane needs them: 16 bytes per lane, 512
//    contiguous bytes per warp, no conflicts and no shuffles.  The weights move
//    from the first product's layout to the second's by one 8x8 transpose per
//    eight tokens.
//
// Precision.  q is scaled by a power of two to fit fp16 (bf16's 8 bits are exact
// there); logits, maxima, sums and outputs are fp32.  Weights are rounded to fp16
// twice (2^-11 each, before and after their scale).  They are kept in fp16's range
// by the reference of the softmax: R = (running maximum) - x with x chosen from the
// largest value scale seen, so that weight * scale stays below 2^16 and weights
// 2^-30 below the largest still count.
//
// Work split: grid (CS * NC, B * Hkv), clusters of CS CTAs, as attend.cu: each CTA
// takes a contiguous range of the problem's pages.  Eight warps: one issues the
// bulk copies of whole page-heads (9216 or 2304 contiguous bytes) into a ring of
// 64-token slots, seven consume.  With many pages per CTA a warp takes a whole slot
// (one maximum and at most one rescale per 64 tokens); with few, 16 tokens, so that
// all warps work on two slots.  Partial states meet in shared memory, then
// across the cluster, then (several clusters per problem) in the workspace, where
// the last cluster to finish joins them.
#include "common.cuh"
#include "kernels.h"
#include "kv_q4.cuh"

namespace locks {

namespace {

constexpr int kW = 7;                           // consumer warps
constexpr int kThreads = (kW + 1) * 32;         // and the producer
constexpr int kStages = 11;                     // 101,376 bytes: two CTAs per SM
constexpr int kOStride = 132;                   // padded row of a warp's outputs (floats)
constexpr int kRing = kStages * kQ4Slot;
constexpr int kRecvMl = 16 * 16 * 8;            // their (R, sum), [rank][head]
constexpr int kSmem = kRing + 128;

struct Q4Shared {
  uint64_t full[kStages], empty[kStages], recv;
  int len[kStages][4], lp[kStages];
  float m[kW][16], l[kW][16], f[kW][16];
  float cta_m[16], cta_l[16];
  int failed, last;
};

__device__ __forceinline__ uint32_t transpose8x8(uint32_t x) {
  uint32_t d;
  asm volatile("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;\n" : "=r"(d) : "r"(x));
  return d;
}
// Field i (0..3) of both halves of w as the fp16 pair 64 + u (exact).
template <int I>
__device__ __forceinline__ uint32_t field64(uint32_t w) {
  const uint32_t x = I == 0 ? w << 4 : (I == 1 ? w : (I == 2 ? w >> 4 : w >> 8));
  return (x & 0x00f000f0u) | 0x54005400u;
}
// Mask of a packed pair of tokens (t, t + 1) that keeps those inside `len`.
__device__ __forceinline__ uint32_t pair_mask(int t, int len) {
  return (t < len ? 0x0000ffffu : 0u) | (t + 1 < len ? 0xffff0000u : 0u);
}

// TPU: 16-token tiles per warp and turn (4: a whole slot, 1: a quarter).
// NT: blocks of 8 query heads.
template <int MODE, int P, int TPU, int NT>
__global__ void __launch_bounds__(kThreads, NT == 1 ? 2 : 1) attend_q4_kernel(const AttendArgs a) {
  constexpr bool LSE = MODE == kAttendPageLse;
  constexpr int kPPS = kPage / P;  // pages per slot
  constexpr uint32_t kPageBytes = LSE ? 72 * P : 144 * P;
  using At = Q4Tile<P>;
  extern __shared__ __align__(128) uint8_t ring_raw[];
  __shared__ Q4Shared sh;
  uint8_t* ring = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(ring_raw) + 127) & ~uintptr_t(127));
  const uint32_t rbase = smem_u32(ring);

  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int g = lane >> 2, c = lane & 3;
  const int split = blockIdx.x, bh = blockIdx.y;
  const int b = bh / a.num_kv_heads, hkv = bh % a.num_kv_heads;
  const int G = a.group, Hq = a.num_kv_heads * G;

  if (tid == 0) {
    for (int s = 0; s < kStages; ++s) {
      mbar_init(&sh.full[s], 1);
      mbar_init(&sh.empty[s], TPU == 4 ? 1 : 4);
    }
    mbar_init(&sh.recv, a.cluster);
    fence_mbar_init();
    sh.failed = 0;
  }
  __syncthreads();
  if (!LSE) cluster_arrive();  // matched by the wait before the first remote access
  pdl_wait();

  int L = a.seq_lens[b];
  if (L < 0 || L > a.max_pages * P) {
    if (tid == 0 && split == 0) set_error(a.err, LOCKS_DEVERR_LENGTHS);
    L = L < 0 ? 0 : a.max_pages * P;
  }
  const int n_pages = (L + P - 1) / P;
  int ns = 0, cnt = 0, n_items = n_pages;
  if (MODE == kAttendSparse) {
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
  // this CTA's pages: a whole number of slots
  const int ipc = ((n_items + a.n_splits - 1) / a.n_splits + kPPS - 1) / kPPS * kPPS;
  const int i0 = min(n_items, split * ipc), i1 = min(n_items, i0 + ipc);
  const int n_slots = (i1 - i0 + kPPS - 1) / kPPS;

  float R[NT][2], l[NT][2];   // softmax reference (base 2) and sum of heads 8 nt + 2c, + 1
  float o[4][2][NT][4];       // outputs: dimensions 32 j + 4 g + 2 half, + 1 (rows) of those heads
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

  if (warp == kW) {
    // ---- producer: resolve 32 pages at a time, then copy them slot by slot ----
    bool ok = true;
    int issued = 0;
    for (int base = 0; base < i1 - i0 && ok; base += 32) {
      const int i = i0 + base + lane;
      int phys = -1, len = 0, lp = -1;
      if (i < i1) {
        if (MODE == kAttendSparse && i < cnt) {
          lp = a.sel_pages[(size_t)bh * a.k_max + i];
          if (a.sel_phys) phys = a.sel_phys[(size_t)bh * a.k_max + i];
          if (lp < 0 || lp >= ns) {
            set_error(a.err, LOCKS_DEVERR_SEL_PAGE);
            lp = -1;
          } else if (!a.sel_phys) {
            phys = a.block_table[(size_t)b * a.max_pages + lp];
          }
        } else {
          lp = MODE == kAttendSparse ? ns + (i - cnt) : i;
          phys = a.block_table[(size_t)b * a.max_pages + lp];
        }
        if (lp >= 0 && (phys < 0 || phys >= a.pages_total)) {
          set_error(a.err, LOCKS_DEVERR_BLOCK_TABLE);
          lp = -1;
        }
        if (lp >= 0) len = min(P, L - lp * P);
      }
      const int here = min(32, i1 - i0 - base);
      for (int k = 0; k < here; k += kPPS) {
        const int s = (base + k) / kPPS, st = s % kStages;
        if (s >= kStages && !mbar_wait(&sh.empty[st], (s / kStages - 1) & 1)) {
          ok = false;
          break;
        }
        uint32_t bytes = 0;
#pragma unroll
        for (int w = 0; w < kPPS; ++w) {
          const int ln = __shfl_sync(0xffffffffu, len, (k + w) & 31);
          if (lane == 0) sh.len[st][w] = k + w < here ? ln : 0;
          if (k + w < here && ln > 0) bytes += kPageBytes;
        }
        const int lp0 = __shfl_sync(0xffffffffu, lp, k);
        if (lane == 0) {
          if (kPPS == 1) sh.lp[st] = lp0;
          mbar_arrive_expect_tx(&sh.full[st], bytes);
        }
        if (LSE && kPPS > 1) {
          // the pages of the slot in the order of the list; page numbers follow from the first item
          if (lane == 0) sh.lp[st] = i0 + base + k;
        }
        __syncwarp();
#pragma unroll
        for (int w = 0; w < kPPS; ++w) {
          const int ln = __shfl_sync(0xffffffffu, len, (k + w) & 31);
          const int ph = __shfl_sync(0xffffffffu, phys, (k + w) & 31);
          if (lane == 0 && k + w < here && ln > 0)
            bulk_load(rbase + st * kQ4Slot + w * LOCKS_KV_Q4_BLOCK_BYTES(P),
                      reinterpret_cast<const uint8_t*>(a.k_pool16) +
                          ((size_t)ph * a.num_kv_heads + hkv) * (size_t)LOCKS_KV_Q4_BLOCK_BYTES(P),
                      kPageBytes, &sh.full[st]);
        }
        issued = s + 1;
      }
    }
    if (!ok) {
      // consumers gave up: let the copies in flight land before the ring is reused
      if (lane == 0) {
        set_error(a.err, kDevErrTimeout);
        sh.failed = 1;
        for (int s = max(0, issued - kStages); s < issued; ++s) (void)mbar_wait(&sh.full[s % kStages], (s / kStages) & 1);
      }
    }
  } else {
    // ---- consumers ----
    // q of head 8 nt + g, dimensions 32 j + 8 c .. + 7, scaled into fp16
    uint32_t qf[NT][4][4];
    float init[NT][4][2];   // -72 sum of q over the group's 32 dimensions, heads 2c, 2c + 1
    float fac[NT][2];       // logit factor of heads 2c, 2c + 1
#pragma unroll
    for (int nt = 0; nt < NT; ++nt) {
      const int h = 8 * nt + g;
      uint4 raw[4];
      float mx = 0.f;
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        raw[j] = make_uint4(0, 0, 0, 0);
        if (h < G)
          raw[j] = __ldg(reinterpret_cast<const uint4*>(a.q + ((size_t)b * Hq + (size_t)hkv * G + h) * kHeadDim +
                                                        32 * j + 8 * c));
        const uint32_t w[4] = {raw[j].x, raw[j].y, raw[j].z, raw[j].w};
#pragma unroll
        for (int k = 0; k < 4; ++k)
          mx = fmaxf(mx, fmaxf(fabsf(__uint_as_float(w[k] << 16)), fabsf(__uint_as_float(w[k] & 0xffff0000u))));
      }
      mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 1));
      mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 2));
      // 2^-e with e the exponent of the largest element (0 for a zero or
      // non-finite row), kept away from the ends of fp32's range
      int e = (int)(__float_as_uint(mx) >> 23) - 127;
      e = mx == 0.f || e > 127 ? 0 : min(max(e, -100), 126);
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
#pragma unroll
        for (int k = 0; k < 2; ++k) init[nt][j][k] = -72.f * __shfl_sync(0xffffffffu, sum[j], 8 * c + 4 * k);
      }
      const float up = a.scale_log2 * __uint_as_float((uint32_t)(127 + e) << 23);
#pragma unroll
      for (int k = 0; k < 2; ++k) fac[nt][k] = __shfl_sync(0xffffffffu, up, 8 * c + 4 * k);
    }

    float m[NT][2];
#pragma unroll
    for (int nt = 0; nt < NT; ++nt) m[nt][0] = m[nt][1] = -INFINITY;
    int x = 15;  // exponent offset of the weights, lowered by large value scales

    const int n_units = TPU == 4 ? n_slots : 4 * n_slots;
    for (int u = warp; u < n_units; u += kW) {
      const int s = TPU == 4 ? u : u >> 2, st = s % kStages, t0 = TPU == 4 ? 0 : u & 3;
      if (!mbar_wait(&sh.full[st], (s / kStages) & 1)) {
        if (lane == 0) {
          set_error(a.err, kDevErrTimeout);
          sh.failed = 1;
        }
        break;
      }
      const uint32_t base = rbase + st * kQ4Slot;
      // tokens of the tile, or of the slot at P = 64 (from its first token)
      int len[TPU];
      bool whole = true, any = false;
#pragma unroll
      for (int t = 0; t < TPU; ++t) {
        const int ln = P == 64 ? sh.len[st][0] - 16 * (t0 + t) : sh.len[st][t0 + t];
        len[t] = ln;
        whole &= ln >= 16;
        any |= ln > 0;
      }
      if (any) {
        float sc[TPU][NT][4];
        float mx[NT][2];
#pragma unroll
        for (int nt = 0; nt < NT; ++nt) mx[nt][0] = mx[nt][1] = -INFINITY;
        // ---- logits of the unit's tokens (rows g, g + 8 of each tile) ----
#pragma unroll
        for (int t = 0; t < TPU; ++t) {
          const uint4 k0 = lds128(base + At::key_codes(t0 + t) + lane * 16), k1 = lds128(base + At::key_codes(t0 + t) + 512 + lane * 16);
          const uint2 s0 = lds64(base + At::key_scales(t0 + t) + g * 8), s1 = lds64(base + At::key_scales(t0 + t) + 64 + g * 8);
          const uint32_t kw0[4] = {k0.x, k0.y, k0.z, k0.w}, kw1[4] = {k1.x, k1.y, k1.z, k1.w};
          const float z0[4] = {f16_lo(s0.x), f16_hi(s0.x), f16_lo(s0.y), f16_hi(s0.y)};
          const float z1[4] = {f16_lo(s1.x), f16_hi(s1.x), f16_lo(s1.y), f16_hi(s1.y)};
#pragma unroll
          for (int j = 0; j < 4; ++j) {
            const uint32_t a00 = field64<0>(kw0[j]), a01 = field64<1>(kw0[j]), a02 = field64<2>(kw0[j]), a03 = field64<3>(kw0[j]);
            const uint32_t a10 = field64<0>(kw1[j]), a11 = field64<1>(kw1[j]), a12 = field64<2>(kw1[j]), a13 = field64<3>(kw1[j]);
#pragma unroll
            for (int nt = 0; nt < NT; ++nt) {
              float acc[4] = {init[nt][j][0], init[nt][j][1], init[nt][j][0], init[nt][j][1]};
              mma_16816_f16(acc, a00, a10, a01, a11, qf[nt][j][0], qf[nt][j][1]);
              mma_16816_f16(acc, a02, a12, a03, a13, qf[nt][j][2], qf[nt][j][3]);
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
          if (!whole) {
#pragma unroll
            for (int nt = 0; nt < NT; ++nt) {
              if (g >= len[t]) sc[t][nt][0] = sc[t][nt][1] = -INFINITY;
              if (g + 8 >= len[t]) sc[t][nt][2] = sc[t][nt][3] = -INFINITY;
            }
          }
#pragma unroll
          for (int nt = 0; nt < NT; ++nt)
#pragma unroll
            for (int k = 0; k < 2; ++k) mx[nt][k] = fmaxf(mx[nt][k], fmaxf(sc[t][nt][k], sc[t][nt][2 + k]));
        }
#pragma unroll
        for (int nt = 0; nt < NT; ++nt)
#pragma unroll
          for (int k = 0; k < 2; ++k) {
            mx[nt][k] = fmaxf(mx[nt][k], __shfl_xor_sync(0xffffffffu, mx[nt][k], 4));
            mx[nt][k] = fmaxf(mx[nt][k], __shfl_xor_sync(0xffffffffu, mx[nt][k], 8));
            mx[nt][k] = fmaxf(mx[nt][k], __shfl_xor_sync(0xffffffffu, mx[nt][k], 16));
            mx[nt][k] *= fac[nt][k];  // the factor is positive
          }
        if constexpr (LSE) {
          // a unit is one page (a slot of P = 64, a tile of P = 16)
#pragma unroll
          for (int nt = 0; nt < NT; ++nt)
#pragma unroll
            for (int k = 0; k < 2; ++k) {
              float ps = 0.f;
#pragma unroll
              for (int t = 0; t < TPU; ++t)
                ps += fast_exp2(fmaf(sc[t][nt][k], fac[nt][k], -mx[nt][k])) +
                      fast_exp2(fmaf(sc[t][nt][2 + k], fac[nt][k], -mx[nt][k]));
              ps += __shfl_xor_sync(0xffffffffu, ps, 4);
              ps += __shfl_xor_sync(0xffffffffu, ps, 8);
              ps += __shfl_xor_sync(0xffffffffu, ps, 16);
              const int h = 8 * nt + 2 * c + k;
              if (g == 0 && h < G) {
                const int lp = sh.lp[st] + (kPPS > 1 ? t0 : 0);
                a.page_lse[((size_t)b * Hq + (size_t)hkv * G + h) * a.max_pages + lp] = (mx[nt][k] + fast_log2(ps)) * kLn2;
              }
            }
        } else {
          // ---- the weights' exponent offset: the largest value scale, below 2^(e+1),
          // times weights of up to 2^x stays below 2^15 ----
          {
            uint32_t top = 0;
            if (TPU == 4 || lane < 8) {
              const int t = TPU == 4 ? lane >> 3 : 0;  // this lane's 16 bytes of scales
              uint4 w = lds128(base + At::value_scales(t0 + t) + (lane & 7) * 16);
              if (!whole) {
                // each word: tokens 8 (lane%2) + (lane%8)/2 2, + 1 of tile t
                const int ln = P == 64 ? sh.len[st][0] - 16 * (t0 + t) : sh.len[st][t0 + t];
                const uint32_t msk = pair_mask(8 * (lane & 1) + 2 * ((lane & 7) >> 1), ln);
                w.x &= msk; w.y &= msk; w.z &= msk; w.w &= msk;
              }
              const uint32_t v0 = __vmaxu2(w.x, w.y), v1 = __vmaxu2(w.z, w.w);
              const uint32_t v = __vmaxu2(v0, v1);
              top = max(v & 0xffffu, v >> 16);
            }
            top = __reduce_max_sync(0xffffffffu, top);
            // half bits -> exponent; a NaN scale (its product is NaN anyway) counts as the largest
            const int e = min((int)(top >> 10), 29) - 15;
            x = min(x, min(15, 14 - e));
          }
          bool moved = false;
          float Rn[NT][2];
#pragma unroll
          for (int nt = 0; nt < NT; ++nt)
#pragma unroll
            for (int k = 0; k < 2; ++k) {
              m[nt][k] = fmaxf(m[nt][k], mx[nt][k]);
              Rn[nt][k] = m[nt][k] - (float)x;
              moved |= Rn[nt][k] != R[nt][k];
            }
          if (__any_sync(0xffffffffu, moved)) {
#pragma unroll
            for (int nt = 0; nt < NT; ++nt)
#pragma unroll
              for (int k = 0; k < 2; ++k) {
                const float al = Rn[nt][k] == -INFINITY ? 1.f : fast_exp2(R[nt][k] - Rn[nt][k]);
                R[nt][k] = Rn[nt][k];
                l[nt][k] *= al;
#pragma unroll
                for (int j = 0; j < 4; ++j)
#pragma unroll
                  for (int hf = 0; hf < 2; ++hf) {
                    o[j][hf][nt][k] *= al;
                    o[j][hf][nt][2 + k] *= al;
                  }
              }
          }
          // ---- weights and the values they weight ----
#pragma unroll
          for (int t = 0; t < TPU; ++t) {
            uint32_t pb[NT][2];
#pragma unroll
            for (int nt = 0; nt < NT; ++nt) {
              float p[4];
#pragma unroll
              for (int k = 0; k < 4; ++k) {
                p[k] = fast_exp2(fmaf(sc[t][nt][k], fac[nt][k & 1], -R[nt][k & 1]));
                l[nt][k & 1] += p[k];
              }
              pb[nt][0] = transpose8x8(pack_f16(p[0], p[1]));  // tokens 2c, 2c + 1 of head g
              pb[nt][1] = transpose8x8(pack_f16(p[2], p[3]));  // tokens 8 + 2c, + 1
            }
            const uint4 v0 = lds128(base + At::value_codes(t0 + t) + lane * 16), v1 = lds128(base + At::value_codes(t0 + t) + 512 + lane * 16);
            uint4 z0 = lds128(base + At::value_scales(t0 + t) + c * 32), z1 = lds128(base + At::value_scales(t0 + t) + c * 32 + 16);
            if (!whole) {
              // scales past the end may be anything, a NaN too
              const uint32_t m0 = pair_mask(2 * c, len[t]), m1 = pair_mask(8 + 2 * c, len[t]);
              z0.x &= m0; z0.y &= m0; z0.z &= m0; z0.w &= m0;
              z1.x &= m1; z1.y &= m1; z1.z &= m1; z1.w &= m1;
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
                const uint32_t p0 = mul_f16x2(pb[nt][0], zw0[j]), p1 = mul_f16x2(pb[nt][1], zw1[j]);
                mma_16816_f16(o[j][0][nt], a0, a1, a2, a3, p0, p1);
                mma_16816_f16(o[j][1][nt], b0, b1, b2, b3, p0, p1);
              }
            }
          }
        }
      }
      __syncwarp();
      if (lane == 0) mbar_arrive(&sh.empty[st]);
    }
  }
  if (LSE) {
    pdl_launch_dependents();
    return;
  }
  __syncthreads();  // the ring is no longer read or written by copies
  pdl_launch_dependents();

  // ---- merge the warps of this CTA ----
  float* so = reinterpret_cast<float*>(ring);  // [kW][8 NT][kOStride]
  float* octa = so + kW * 8 * NT * kOStride;   // [16][128]
  float* recv_o = octa + 16 * kHeadDim;
  float2* recv_ml = reinterpret_cast<float2*>(recv_o + 16 * kHeadDim);
  static_assert((kW * 8 * NT * kOStride + 32 * kHeadDim) * 4 + kRecvMl <= kRing, "the merge fits the ring");
  if (warp < kW) {
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
#pragma unroll
        for (int j = 0; j < 4; ++j)
          *reinterpret_cast<float4*>(so + (warp * 8 * NT + h) * kOStride + 32 * j + 4 * g) =
              make_float4(o[j][0][nt][k], o[j][0][nt][2 + k], o[j][1][nt][k], o[j][1][nt][2 + k]);
      }
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
      Ls += sh.l[w][tid] * f;
    }
    sh.cta_m[tid] = M;
    sh.cta_l[tid] = Ls;
  }
  __syncthreads();
  const int CS = a.cluster, NC = a.n_splits / a.cluster;
  const uint32_t rank = cluster_ctarank();
  const int cols = kHeadDim / CS;
  cluster_wait();  // every CTA of the cluster has set up its receive barrier
  // Before anybody's ring may be written from outside, its owner must be done with
  // it: the second cluster barrier.
  cluster_arrive();
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
  cluster_wait();
  // ---- push this CTA's state to the owners of its columns ----
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
  const int q = split / CS;
  for (int e = tid; e < G * cols; e += kThreads) {
    const int h = e / cols, cc = e % cols, col = (int)rank * cols + cc;
    float M = -INFINITY;
    for (int rr = 0; rr < CS; ++rr) M = fmaxf(M, recv_ml[rr * 16 + h].x);
    float Ls = 0.f, O = 0.f;
    for (int rr = 0; rr < CS; ++rr) {
      const float2 ml = recv_ml[rr * 16 + h];
      const float f = M == -INFINITY ? 1.f : fast_exp2(ml.x - M);
      Ls = fmaf(ml.y, f, Ls);
      O = fmaf(recv_o[(rr * G + h) * cols + cc], f, O);
    }
    const size_t oi = (size_t)b * Hq + (size_t)hkv * G + h;
    if (NC == 1) {
      a.out[oi * kHeadDim + col] = __bfloat16_as_ushort(__float2bfloat16_rn(Ls == 0.f ? 0.f : O / Ls));
      if (a.lse && col == 0) a.lse[oi] = Ls == 0.f ? -INFINITY : (M + fast_log2(Ls)) * kLn2;
    } else {
      const size_t pi = ((size_t)bh * NC + q) * G + h;
      a.part_o[pi * kHeadDim + col] = O;
      if (col == 0) a.part_ml[pi] = make_float2(M, Ls);
    }
  }
  if (NC == 1) return;

  // ---- several clusters per problem: the last one to finish joins them ----
  __threadfence();
  cluster_sync();
  if (rank == 0 && tid == 0) {
    const int last = atomicAdd(a.counters + bh, 1u) == (unsigned)(NC - 1);
    for (int rr = 0; rr < CS; ++rr) st_dsmem(dsmem_addr(smem_u32(&sh.last), rr), last);
  }
  cluster_sync();
  if (!sh.last) return;
  __threadfence();
  for (int e = tid; e < G * cols; e += kThreads) {
    const int h = e / cols, col = (int)rank * cols + e % cols;
    const size_t p0 = (size_t)bh * NC * G + h;
    float M = -INFINITY;
    for (int qq = 0; qq < NC; ++qq) M = fmaxf(M, __ldcg(a.part_ml + p0 + (size_t)qq * G).x);
    float Ls = 0.f, O = 0.f;
    for (int qq = 0; qq < NC; ++qq) {
      const float2 ml = __ldcg(a.part_ml + p0 + (size_t)qq * G);
      const float f = M == -INFINITY ? 1.f : fast_exp2(ml.x - M);
      Ls = fmaf(ml.y, f, Ls);
      O = fmaf(__ldcg(a.part_o + (p0 + (size_t)qq * G) * kHeadDim + col), f, O);
    }
    const size_t oi = (size_t)b * Hq + (size_t)hkv * G + h;
    a.out[oi * kHeadDim + col] = __bfloat16_as_ushort(__float2bfloat16_rn(Ls == 0.f ? 0.f : O / Ls));
    if (a.lse && col == 0) a.lse[oi] = Ls == 0.f ? -INFINITY : (M + fast_log2(Ls)) * kLn2;
  }
  if (rank == 0 && tid == 0) a.counters[bh] = 0;  // ready for the next call
}

using Kern = void (*)(const AttendArgs);

template <int MODE, int P>
Kern pick(int group, int tiles) {
  if (group <= 8) return tiles == 4 ? attend_q4_kernel<MODE, P, 4, 1> : attend_q4_kernel<MODE, P, 1, 1>;
  return tiles == 4 ? attend_q4_kernel<MODE, P, 4, 2> : attend_q4_kernel<MODE, P, 1, 2>;
}

Kern kernel_of(int mode, int group, int page_size, int tiles) {
  if (mode == kAttendPageLse) {
    // a unit is one page: a slot, or a tile of it
    if (page_size == 16)
      return group <= 8 ? attend_q4_kernel<kAttendPageLse, 16, 1, 1> : attend_q4_kernel<kAttendPageLse, 16, 1, 2>;
    return group <= 8 ? attend_q4_kernel<kAttendPageLse, 64, 4, 1> : attend_q4_kernel<kAttendPageLse, 64, 4, 2>;
  }
  if (page_size == 16) return mode == kAttendSparse ? pick<kAttendSparse, 16>(group, tiles) : pick<kAttendDense, 16>(group, tiles);
  return mode == kAttendSparse ? pick<kAttendSparse, 64>(group, tiles) : pick<kAttendDense, 64>(group, tiles);
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

int attend_q4_ctas_per_sm(int group) { return group <= 8 ? 2 : 1; }

int attend_q4_active_clusters(int mode, int group, int page_size, int tiles, int cs) {
  // one entry per kernel variant, cluster size and device; the answer depends on nothing else
  static int cache[2][2][2][2][5][64] = {};
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= 64 || cs < 1 || cs > 16) return 1;
  int& slot = cache[mode == kAttendSparse][group > 8][page_size == 16][tiles == 4][31 - __builtin_clz((unsigned)cs)][dev];
  if (slot == 0) {
    const int n = active_clusters(kernel_of(mode, group, page_size, tiles), cs);
    slot = n > 0 ? n : -1;
  }
  return slot > 0 ? slot : 0;
}

int attend_q4_max_cluster(int mode, int group, int page_size, int tiles) {
  for (int cs = 16; cs > 1; cs /= 2)
    if (attend_q4_active_clusters(mode, group, page_size, tiles, cs) > 0) return cs;
  return 1;
}

cudaError_t launch_attend_q4(const AttendArgs& a, int mode, int tiles, cudaStream_t s) {
  const Kern k = kernel_of(mode, a.group, a.page_size, tiles);
  if (!prepare(k, a.cluster)) return cudaErrorInvalidConfiguration;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(a.n_splits, a.batch * a.num_kv_heads, 1);
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

}  // namespace locks
