// Writing tokens into the paged cache, and reading them back.
//
// One pass over a token's rows: queries and keys get their position rotation
//   a' = a c - b s,  b' = b c + a s
// (each product and the sum rounded once in fp32, so that a 4-bit code never
// depends on how a compiler contracts the sum; the result is rounded to bf16,
// the precision of the queries and of a bf16 page), values pass unchanged, and
// keys and values go to their page's slot.  A 4-bit page holds, for each 32
// dimensions of those bf16 numbers, s = half(max|x| / 7) and rint(x / s), exactly.
//
// What bounds it: bytes (a token is read once and written once) for prompts, and
// one round trip of dependent loads (lengths, block table, table row, data) plus
// the launch for a decode step.
//
// Split: 16 threads take a row of 128 elements, 8 (16 bytes) each, so a thread's
// dimensions, and with them its cosines and sines, are the same for every row of a
// token.  The partner of a (d, d + rot/2) pair is another thread's of the row.  A
// 32-dimension group is 4 neighbouring threads, whose maximum takes two shuffles.  A
// prompt's token is one warp's, which has four pairs of rows in flight while it finds
// the token's place; a decode step's few tokens are a CTA's each, whose eight warps
// load all rows at once.
//
// Measured: 13,000 prompt tokens of 32 + 8 heads into bf16 pages 52.7 us, 6.2 TB/s
// (0.91 of a copy's rate); 27,000 tokens of 32 + 2 heads into 4-bit pages and back 94 us
// (76 us of bytes); one step of 8 sequences 2.6 us on the device, of 32 into 4-bit pages
// and back 5.4 us.
#include <cuda_fp16.h>

#include "common.cuh"
#include "kernels.h"

namespace locks {

namespace {

constexpr int kAppendThreads = 256;
constexpr int kAppendWarps = kAppendThreads / 32;
constexpr int kRowThreads = kHeadDim / 8;  // threads of one row: two rows per warp and step
constexpr int kInFlight = 4;               // steps whose rows are loaded together

// The sequence of token row t and its place: position, physical page, slot.
struct TokenPlace {
  int b, pos, phys, slot;
  bool ok;
};

// Whole warps; every lane gets the same answer.
__device__ __forceinline__ TokenPlace token_place(const KvTokenArgs& a, int t, bool report) {
  TokenPlace r;
  r.ok = false;
  r.pos = r.phys = r.slot = 0;
  r.b = t;
  int n_b = 1, i = 0;
  if (a.cu_tokens) {
    // the last b with cu_tokens[b] <= t: 32 sequences at a time
    const int lane = threadIdx.x & 31;
    r.b = 0;
    for (int b0 = 1; b0 <= a.batch; b0 += 32) {
      const int n = __popc(__ballot_sync(0xffffffffu, b0 + lane <= a.batch && __ldg(a.cu_tokens + b0 + lane) <= t));
      r.b += n;
      if (n < 32) break;
    }
    if (r.b >= a.batch) return r;  // a row behind the last sequence
    const int c0 = __ldg(a.cu_tokens + r.b), c1 = __ldg(a.cu_tokens + r.b + 1);
    n_b = c1 - c0;
    i = t - c0;
    if (i < 0 || i >= n_b || i >= a.max_tokens) {
      if (report) set_error(a.err, LOCKS_DEVERR_LENGTHS);
      return r;
    }
  }
  const int len = __ldg(a.seq_lens + r.b);
  if (!a.cu_tokens && len == 0) return r;  // an idle slot of a padded batch
  const long long pos = (long long)len - n_b + i;
  if (pos < 0 || pos >= (long long)a.max_pages * a.page_size) {
    if (report) set_error(a.err, LOCKS_DEVERR_LENGTHS);
    return r;
  }
  r.pos = (int)pos;
  const int lp = r.pos / a.page_size;
  r.slot = r.pos - lp * a.page_size;
  r.phys = __ldg(a.block_table + (size_t)r.b * a.max_pages + lp);
  if (r.phys < 0 || r.phys >= a.pages_total) {
    if (report) set_error(a.err, LOCKS_DEVERR_BLOCK_TABLE);
    return r;
  }
  r.ok = true;
  return r;
}

__device__ __forceinline__ float bf16_lo(uint32_t w) { return __uint_as_float(w << 16); }
__device__ __forceinline__ float bf16_hi(uint32_t w) { return __uint_as_float(w & 0xffff0000u); }

// This thread's cosines and sines, for two dimensions at a time; the sines carry the
// sign of their product: y = x c + mate s.
struct Turn {
  uint64_t c[4], s[4];
};

// 8 elements of a row, rotated.  PAIRS_NEXT: pairs are neighbours, else `mate` holds
// the partners.
template <bool PAIRS_NEXT>
__device__ __forceinline__ uint4 rotate8(uint4 x, uint4 mate, const Turn& tr) {
  const uint32_t in[4] = {x.x, x.y, x.z, x.w}, mt[4] = {mate.x, mate.y, mate.z, mate.w};
  uint32_t out[4];
#pragma unroll
  for (int k = 0; k < 4; ++k) {
    const float v0 = bf16_lo(in[k]), v1 = bf16_hi(in[k]);
    const uint64_t m = PAIRS_NEXT ? f32x2(v1, v0) : f32x2(bf16_lo(mt[k]), bf16_hi(mt[k]));
    // the sums one by one: of packed products and a packed sum the compiler makes one
    // operation with one rounding less
    float a0, a1, b0, b1;
    unpack_f32x2(mul_f32x2(f32x2(v0, v1), tr.c[k]), a0, a1);
    unpack_f32x2(mul_f32x2(m, tr.s[k]), b0, b1);
    out[k] = pack_bf16(__fadd_rn(a0, b0), __fadd_rn(a1, b1));
  }
  return make_uint4(out[0], out[1], out[2], out[3]);
}

// The 4-bit form of 8 elements of a row: code + 8 of each, and the group's scale
// (the same in the 4 threads of a 32-dimension group).
//
// rint(x / s) without a division per element: 200 + x fl(1/s), rounded once to a
// multiple of 2^-16, is off by less than 2^-16.  A bf16 x and a half s have x / s either
// exactly at a tie k + 1/2 or at least 2^-12 away from it (2x - (2k+1) s is a multiple of
// the lowest bit of s, and s has 11), so this neither crosses a tie nor leaves one, and
// 200 is even: rounding the sum to an integer, ties to even, gives 200 + rint(x / s).
__device__ __forceinline__ __half quantise8(uint4 x, uint32_t (&u)[8]) {
  uint32_t in[4] = {x.x, x.y, x.z, x.w};
  uint32_t m = 0;  // max |x| as bf16 bits, whose order is the numbers'
#pragma unroll
  for (int k = 0; k < 4; ++k) m = max(m, max(in[k] & 0x7fffu, (in[k] >> 16) & 0x7fffu));
  m = max(m, __shfl_xor_sync(0xffffffffu, m, 1));
  m = max(m, __shfl_xor_sync(0xffffffffu, m, 2));
  const bool finite = m < 0x7f80u;
  const __half s = finite ? __float2half_rn(fminf(__fdiv_rn(__uint_as_float(m << 16), 7.f), (float)LOCKS_KV_Q4_MAX_SCALE))
                          : __ushort_as_half((unsigned short)0x7fff);
  const float sf = __half2float(s);
  const float r = finite && sf > 0.f ? __fdiv_rn(1.f, sf) : 0.f;
#pragma unroll
  for (int k = 0; k < 8; ++k) {
    const float v = finite ? (k & 1 ? bf16_hi(in[k / 2]) : bf16_lo(in[k / 2])) : 0.f;
    const float y = fminf(fmaxf(__fmaf_rn(v, r, 200.f), 193.f), 207.f);
    u[k] = __float_as_uint(__fadd_rn(y, 12582912.f)) & 15u;  // 1.5 2^23: the low bits are the integer
  }
  return s;
}

// Stores of dimensions 8 ch .. 8 ch + 7 of a token in its 4-bit block (u: code + 8).
__device__ __forceinline__ void put_k_q4(uint8_t* block, int P, int slot, int ch, const uint32_t (&u)[8], __half s) {
  uint32_t w = 0;
#pragma unroll
  for (int e = 0; e < 8; ++e) w |= u[e] << (4 * (e / 2) + 16 * (e % 2));
  const int j = ch >> 2, c = ch & 3;
  *reinterpret_cast<uint32_t*>(block + 64 * slot + 16 * c + 4 * j) = w;
  if (c == 0) *reinterpret_cast<__half*>(block + 64 * P + 8 * slot + 2 * j) = s;
}
__device__ __forceinline__ void put_v_q4(uint8_t* block, int P, int slot, int ch, const uint32_t (&u)[8], __half s) {
  const int j = ch >> 2, tile = slot >> 4, t = slot & 15;
  uint8_t* base = block + 72 * P + 1024 * tile + 512 * (t >> 3) + 16 * ((t & 7) >> 1) + 4 * j + 2 * (t & 1);
#pragma unroll
  for (int h = 0; h < 2; ++h)
    *reinterpret_cast<uint16_t*>(base + 64 * (2 * (ch & 3) + h)) =
        (uint16_t)(u[4 * h] | u[4 * h + 1] << 4 | u[4 * h + 2] << 8 | u[4 * h + 3] << 12);
  if ((ch & 3) == 0)
    *reinterpret_cast<__half*>(block + 136 * P + 128 * tile + 32 * ((t & 7) >> 1) + 16 * (t >> 3) + 4 * j +
                               2 * (t & 1)) = s;
}

// WPT: warps of a token (1 or 8).  A step is two rows, either of keys and values (an
// even number together) or of queries.
template <bool Q4, int WPT, bool PAIRS_NEXT>
__global__ void __launch_bounds__(kAppendThreads, 4) append_kernel(const KvAppendArgs a) {
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int t = blockIdx.x * (kAppendWarps / WPT) + warp / WPT;
  const int ch = lane % kRowThreads, sub = lane / kRowThreads;
  pdl_wait();
  pdl_launch_dependents();
  if (t >= a.tok.total) return;
  const int hkv = a.tok.num_kv_heads, P = a.tok.page_size;
  const int half = a.rotary_dim / 2, d0 = 8 * ch;
  const bool turns = d0 < a.rotary_dim;
  const bool upper = !PAIRS_NEXT && d0 >= half;
  // rows of the token: keys, values, then queries
  const int rows = 2 * hkv + (a.q ? a.num_q_heads : 0), steps = (rows + 1) / 2;
  const uint16_t* kr = a.k + (size_t)t * a.k_stride + d0;
  const uint16_t* vr = a.v + (size_t)t * a.v_stride + d0 - hkv * kHeadDim;
  const uint16_t* qr = a.q + (size_t)t * a.q_stride + d0 - 2 * hkv * kHeadDim;
  // the lane with the partners of this one's elements (rotary_dim / 2 is a multiple of 8)
  const int mate_lane = !turns ? lane : upper ? lane - half / 8 : lane + half / 8;
  uint4 x[kInFlight];
  auto load = [&](int i) {
#pragma unroll
    for (int k = 0; k < kInFlight; ++k, i += WPT) {
      const int r = 2 * i + sub;
      x[k] = make_uint4(0, 0, 0, 0);
      if (r < rows) x[k] = *reinterpret_cast<const uint4*>((i >= hkv ? qr : r < hkv ? kr : vr) + r * kHeadDim);
    }
  };
  const int i0 = warp % WPT;
  load(i0);  // under way while the token's place is looked up
  const bool says = lane == 0 && warp % WPT == 0;
  const TokenPlace tp = token_place(a.tok, t, says);
  if (!tp.ok) return;
  Turn tr;
  if (a.rotary_dim) {
    const int row = a.positions ? __ldg(a.positions + t) : tp.pos;
    if (row < 0 || row >= a.rope_rows) {
      if (says) set_error(a.tok.err, LOCKS_DEVERR_POSITION);
      return;
    }
    if (turns) {
      const float* cs = a.rope + (size_t)row * a.rotary_dim + (PAIRS_NEXT ? d0 / 2 : (upper ? d0 - half : d0));
#pragma unroll
      for (int k = 0; k < (PAIRS_NEXT ? 1 : 2); ++k) {
        const float4 c = __ldg(reinterpret_cast<const float4*>(cs) + k);
        const float4 s = __ldg(reinterpret_cast<const float4*>(cs + half) + k);
        if constexpr (PAIRS_NEXT) {
          const float cc[4] = {c.x, c.y, c.z, c.w}, ss[4] = {s.x, s.y, s.z, s.w};
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            tr.c[e] = f32x2(cc[e], cc[e]);
            tr.s[e] = f32x2(-ss[e], ss[e]);
          }
        } else {
          const float sign = upper ? 1.f : -1.f;
          tr.c[2 * k] = f32x2(c.x, c.y);
          tr.c[2 * k + 1] = f32x2(c.z, c.w);
          tr.s[2 * k] = f32x2(sign * s.x, sign * s.y);
          tr.s[2 * k + 1] = f32x2(sign * s.z, sign * s.w);
        }
      }
    }
  }
  const size_t page = (size_t)tp.phys * hkv;
  uint16_t* q_out = a.q_out + (size_t)t * a.q_out_stride + d0 - 2 * hkv * kHeadDim;
  for (int ib = i0; ib < steps; ib += WPT * kInFlight) {
    if (ib != i0) load(ib);
#pragma unroll
    for (int k = 0; k < kInFlight; ++k) {
      const int i = ib + WPT * k;  // the same for the whole warp
      if (i >= steps) break;
      const int r = 2 * i + sub;
      const bool is_v = i < hkv && r >= hkv;
      uint4 y = x[k], mate = make_uint4(0, 0, 0, 0);
      if (a.rotary_dim) {
        if constexpr (!PAIRS_NEXT) {
          mate.x = __shfl_sync(0xffffffffu, y.x, mate_lane);
          mate.y = __shfl_sync(0xffffffffu, y.y, mate_lane);
          mate.z = __shfl_sync(0xffffffffu, y.z, mate_lane);
          mate.w = __shfl_sync(0xffffffffu, y.w, mate_lane);
        }
        if (turns && !is_v) y = rotate8<PAIRS_NEXT>(y, mate, tr);
      }
      if (i >= hkv) {
        if (r < rows) *reinterpret_cast<uint4*>(q_out + (size_t)r * kHeadDim) = y;
        continue;
      }
      const size_t ph = page + (is_v ? r - hkv : r);
      if (Q4) {
        uint8_t* block = reinterpret_cast<uint8_t*>(a.k_pool) + ph * (size_t)LOCKS_KV_Q4_BLOCK_BYTES(P);
        uint32_t u[8];
        const __half s = quantise8(y, u);
        if (is_v) put_v_q4(block, P, tp.slot, ch, u, s);
        else put_k_q4(block, P, tp.slot, ch, u, s);
      } else {
        uint16_t* pool = reinterpret_cast<uint16_t*>(is_v ? a.v_pool : a.k_pool);
        *reinterpret_cast<uint4*>(pool + (ph * P + tp.slot) * kHeadDim + d0) = y;
      }
    }
  }
}

template <bool Q4, int WPT>
__global__ void __launch_bounds__(kAppendThreads) read_kernel(const KvReadArgs a) {
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int t = blockIdx.x * (kAppendWarps / WPT) + warp / WPT;
  const int ch = lane % kRowThreads, r0 = warp % WPT * 2 + lane / kRowThreads;
  pdl_wait();
  pdl_launch_dependents();
  if (t >= a.tok.total) return;
  const TokenPlace tp = token_place(a.tok, t, lane == 0 && warp % WPT == 0);
  if (!tp.ok) return;
  const int hkv = a.tok.num_kv_heads, P = a.tok.page_size, slot = tp.slot;
#pragma unroll 4
  for (int r = r0; r < 2 * hkv; r += 2 * WPT) {
    const bool is_k = r < hkv;
    const int h = is_k ? r : r - hkv;
    uint16_t* out = is_k ? a.k_out : a.v_out;
    if (!out) continue;
    const size_t ph = (size_t)tp.phys * hkv + h;
    uint4 x;
    if (Q4) {
      const uint8_t* block = reinterpret_cast<const uint8_t*>(a.k_pool) + ph * (size_t)LOCKS_KV_Q4_BLOCK_BYTES(P);
      const int j = ch >> 2, tile = slot >> 4, u = slot & 15;
      int c[8];
      __half s;
      if (is_k) {
        const uint32_t w = *reinterpret_cast<const uint32_t*>(block + 64 * slot + 16 * (ch & 3) + 4 * j);
#pragma unroll
        for (int e = 0; e < 8; ++e) c[e] = (int)((w >> (4 * (e / 2) + 16 * (e % 2))) & 15u) - 8;
        s = *reinterpret_cast<const __half*>(block + 64 * P + 8 * slot + 2 * j);
      } else {
        const uint8_t* base = block + 72 * P + 1024 * tile + 512 * (u >> 3) + 16 * ((u & 7) >> 1) + 4 * j + 2 * (u & 1);
#pragma unroll
        for (int half = 0; half < 2; ++half) {
          const uint32_t w = *reinterpret_cast<const uint16_t*>(base + 64 * (2 * (ch & 3) + half));
#pragma unroll
          for (int i = 0; i < 4; ++i) c[4 * half + i] = (int)((w >> (4 * i)) & 15u) - 8;
        }
        s = *reinterpret_cast<const __half*>(block + 136 * P + 128 * tile + 32 * ((u & 7) >> 1) + 16 * (u >> 3) +
                                             4 * j + 2 * (u & 1));
      }
      const float sf = __half2float(s);
      x = make_uint4(pack_bf16(sf * c[0], sf * c[1]), pack_bf16(sf * c[2], sf * c[3]),
                     pack_bf16(sf * c[4], sf * c[5]), pack_bf16(sf * c[6], sf * c[7]));
    } else {
      const uint16_t* pool = reinterpret_cast<const uint16_t*>(is_k ? a.k_pool : a.v_pool);
      x = *reinterpret_cast<const uint4*>(pool + (ph * P + slot) * kHeadDim + 8 * ch);
    }
    *reinterpret_cast<uint4*>(out + ((size_t)t * hkv + h) * kHeadDim + 8 * ch) = x;
  }
}

// A CTA per token for so few that they take one or two rounds of resident CTAs (four
// per SM), so that a decode step takes one round of loads; beyond that a warp per token,
// which has one wait for its place per token and not eight.  32 + 8 heads, bf16, in us
// (CTA, warp): 8 tokens 2.7, 7.2; 608 tokens 4.0, 7.4; 1216 tokens 6.8, 7.5; 2432 tokens
// 12.1, 9.1.
constexpr int kWideTokens = 8 * 152;

template <typename K, typename A>
cudaError_t launch_tokens(K wide, K narrow, const A& a, cudaStream_t s) {
  const bool w = a.tok.total <= kWideTokens;
  const K kern = w ? wide : narrow;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(w ? a.tok.total : (a.tok.total + kAppendWarps - 1) / kAppendWarps, 1, 1);
  cfg.blockDim = dim3(kAppendThreads, 1, 1);
  cfg.stream = s;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, kern, a);
}

}  // namespace

cudaError_t launch_append(const KvAppendArgs& a, cudaStream_t s) {
  if (a.interleaved)
    return a.tok.q4 ? launch_tokens(append_kernel<true, 8, true>, append_kernel<true, 1, true>, a, s)
                    : launch_tokens(append_kernel<false, 8, true>, append_kernel<false, 1, true>, a, s);
  return a.tok.q4 ? launch_tokens(append_kernel<true, 8, false>, append_kernel<true, 1, false>, a, s)
                  : launch_tokens(append_kernel<false, 8, false>, append_kernel<false, 1, false>, a, s);
}

cudaError_t launch_read(const KvReadArgs& a, cudaStream_t s) {
  return a.tok.q4 ? launch_tokens(read_kernel<true, 8>, read_kernel<true, 1>, a, s)
                  : launch_tokens(read_kernel<false, 8>, read_kernel<false, 1>, a, s);
}

}  // namespace locks
