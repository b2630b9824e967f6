// Writing tokens into the paged cache, and reading them back.
//
// One pass over a token's rows: queries and keys get their position rotation
//   a' = a c - b s,  b' = b c + a s
// (each product and the sum rounded once in fp32, so that a 4-bit code never
// depends on how a compiler contracts the sum; the result is rounded to bf16,
// the precision of the queries and of a bf16 page), values pass unchanged, and
// keys and values go to their page's slot.  A 4-bit page holds, for each 32
// dimensions of those bf16 numbers, s = half(max|x| / 7) and rint(x / s): the
// quotients are IEEE divisions of a bf16 by a half, whose distance from a tie is
// either zero or far above their rounding, so the codes are the exact ones.
//
// What bounds it: bytes (a token is read once and written once) for prompts, and
// one round trip of dependent loads (lengths, block table, table row, data) plus
// the launch for a decode step.
//
// Split: 16 threads take a row of 128 elements, 8 (16 bytes) each, so a thread's
// dimensions, and with them its cosines and sines, are the same for every row of a
// token.  The partner of a (d, d + rot/2) pair is read a second time, from L1.  A
// 32-dimension group is 4 neighbouring threads, whose maximum takes two shuffles.  A
// prompt's token is one warp's, which has four pairs of rows in flight while it finds
// the token's place; a decode step's few tokens are a CTA's each, whose eight warps
// load all rows at once.
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

// This thread's 8 cosines and sines (dimensions 8 ch .. 8 ch + 7).
struct Turn {
  float c[8], s[8];
};

// 8 elements of a row, rotated.  half pairs: `mate` holds the partners and
// `upper` says that these are the second ones (b' = b c + a s).
__device__ __forceinline__ uint4 rotate8(uint4 x, uint4 mate, const Turn& tr, bool interleaved, bool upper) {
  uint32_t in[4] = {x.x, x.y, x.z, x.w}, mt[4] = {mate.x, mate.y, mate.z, mate.w}, out[4];
#pragma unroll
  for (int k = 0; k < 4; ++k) {
    const float v0 = bf16_lo(in[k]), v1 = bf16_hi(in[k]);
    float y0, y1;
    if (interleaved) {
      y0 = __fsub_rn(__fmul_rn(v0, tr.c[k]), __fmul_rn(v1, tr.s[k]));
      y1 = __fadd_rn(__fmul_rn(v1, tr.c[k]), __fmul_rn(v0, tr.s[k]));
    } else {
      const float m0 = bf16_lo(mt[k]), m1 = bf16_hi(mt[k]);
      const float p0 = __fmul_rn(v0, tr.c[2 * k]), r0 = __fmul_rn(m0, tr.s[2 * k]);
      const float p1 = __fmul_rn(v1, tr.c[2 * k + 1]), r1 = __fmul_rn(m1, tr.s[2 * k + 1]);
      y0 = upper ? __fadd_rn(p0, r0) : __fsub_rn(p0, r0);
      y1 = upper ? __fadd_rn(p1, r1) : __fsub_rn(p1, r1);
    }
    out[k] = pack_bf16(y0, y1);
  }
  return make_uint4(out[0], out[1], out[2], out[3]);
}

// The 4-bit form of 8 elements of a row: code + 8 of each, and the group's scale
// (the same in the 4 threads of a 32-dimension group).
__device__ __forceinline__ __half quantise8(uint4 x, int (&u)[8]) {
  const uint32_t in[4] = {x.x, x.y, x.z, x.w};
  uint32_t m = 0;  // max |x| as bf16 bits, whose order is the numbers'
#pragma unroll
  for (int k = 0; k < 4; ++k) m = max(m, max(in[k] & 0x7fffu, (in[k] >> 16) & 0x7fffu));
  m = max(m, __shfl_xor_sync(0xffffffffu, m, 1));
  m = max(m, __shfl_xor_sync(0xffffffffu, m, 2));
  const bool finite = m < 0x7f80u;
  // 9352 = the largest half whose 7-fold is finite in half precision, where
  // attention over prompts holds s * code
  const __half s = finite ? __float2half_rn(fminf(__fdiv_rn(__uint_as_float(m << 16), 7.f), 9352.f))
                          : __ushort_as_half((unsigned short)0x7fff);
  const float sf = __half2float(s);
#pragma unroll
  for (int k = 0; k < 8; ++k) {
    const float v = k & 1 ? bf16_hi(in[k / 2]) : bf16_lo(in[k / 2]);
    int c = 0;
    if (finite && sf > 0.f) c = (int)rintf(fminf(fmaxf(__fdiv_rn(v, sf), -7.f), 7.f));
    u[k] = c + 8;
  }
  return s;
}

// Stores of dimensions 8 ch .. 8 ch + 7 of a token in its 4-bit block (u: code + 8).
__device__ __forceinline__ void put_k_q4(uint8_t* block, int P, int slot, int ch, const int (&u)[8], __half s) {
  uint32_t w = 0;
#pragma unroll
  for (int e = 0; e < 8; ++e) w |= (uint32_t)u[e] << (4 * (e / 2) + 16 * (e % 2));
  const int j = ch >> 2, c = ch & 3;
  *reinterpret_cast<uint32_t*>(block + 64 * slot + 16 * c + 4 * j) = w;
  if (c == 0) *reinterpret_cast<__half*>(block + 64 * P + 8 * slot + 2 * j) = s;
}
__device__ __forceinline__ void put_v_q4(uint8_t* block, int P, int slot, int ch, const int (&u)[8], __half s) {
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

// WPT: warps of a token (1 or 8).
template <bool Q4, int WPT>
__global__ void __launch_bounds__(kAppendThreads) append_kernel(const KvAppendArgs a) {
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int t = blockIdx.x * (kAppendWarps / WPT) + warp / WPT;
  const int ch = lane % kRowThreads, r0 = warp % WPT * 2 + lane / kRowThreads;
  pdl_wait();
  pdl_launch_dependents();
  if (t >= a.tok.total) return;
  const int hkv = a.tok.num_kv_heads, P = a.tok.page_size;
  const int half = a.rotary_dim / 2, d0 = 8 * ch;
  const bool turns = d0 < a.rotary_dim;
  const bool upper = !a.interleaved && d0 >= half;
  // rows of the token: keys, values, then queries
  const int rows = 2 * hkv + (a.q ? a.num_q_heads : 0);
  const uint16_t* kr = a.k + (size_t)t * a.k_stride + d0;
  const uint16_t* vr = a.v + (size_t)t * a.v_stride + d0 - hkv * kHeadDim;
  const uint16_t* qr = a.q + (size_t)t * a.q_stride + d0 - 2 * hkv * kHeadDim;
  const int to_mate = upper ? -half : half;
  uint4 x[kInFlight], mate[kInFlight];
  auto load = [&](int r) {
#pragma unroll
    for (int k = 0; k < kInFlight; ++k, r += 2 * WPT) {
      if (r >= rows) continue;
      const uint16_t* src = (r < hkv ? kr : (r < 2 * hkv ? vr : qr)) + r * kHeadDim;
      x[k] = *reinterpret_cast<const uint4*>(src);
      if (turns && !a.interleaved && (r < hkv || r >= 2 * hkv)) mate[k] = *reinterpret_cast<const uint4*>(src + to_mate);
    }
  };
  load(r0);  // under way while the token's place is looked up
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
      const float* cs = a.rope + (size_t)row * a.rotary_dim + (a.interleaved ? d0 / 2 : (upper ? d0 - half : d0));
#pragma unroll
      for (int k = 0; k < 8; k += 4) {
        if (k == 0 || !a.interleaved) {
          const float4 c = __ldg(reinterpret_cast<const float4*>(cs + k));
          const float4 s = __ldg(reinterpret_cast<const float4*>(cs + half + k));
          tr.c[k] = c.x, tr.c[k + 1] = c.y, tr.c[k + 2] = c.z, tr.c[k + 3] = c.w;
          tr.s[k] = s.x, tr.s[k + 1] = s.y, tr.s[k + 2] = s.z, tr.s[k + 3] = s.w;
        }
      }
    }
  }
  const size_t page = (size_t)tp.phys * hkv;
  uint16_t* q_out = a.q_out + (size_t)t * a.q_out_stride + d0 - 2 * hkv * kHeadDim;
  // both rows of a warp's step exist or end together but for the last one
  for (int rb = r0; rb - lane / kRowThreads < rows; rb += 2 * WPT * kInFlight) {
    if (rb != r0) load(rb);
    // queries may be rotated in place: a row's partners are read before either is written
    __syncwarp();
#pragma unroll
    for (int k = 0; k < kInFlight; ++k) {
      const int r = rb + 2 * WPT * k;
      const bool in = r < rows, is_kv = r < 2 * hkv, is_v = is_kv && r >= hkv;
      uint4 y = in ? x[k] : make_uint4(0, 0, 0, 0);
      if (in && turns && !is_v) y = rotate8(y, mate[k], tr, a.interleaved, upper);
      const size_t ph = page + (is_v ? r - hkv : r);
      if (Q4) {
        // the shuffles of the quantiser are a whole warp's, whose two rows may be of
        // different kinds
        if (__any_sync(0xffffffffu, in && is_kv)) {
          uint8_t* block = reinterpret_cast<uint8_t*>(a.k_pool) + ph * (size_t)LOCKS_KV_Q4_BLOCK_BYTES(P);
          int u[8];
          const __half s = quantise8(y, u);
          if (in && is_kv && !is_v) put_k_q4(block, P, tp.slot, ch, u, s);
          if (in && is_v) put_v_q4(block, P, tp.slot, ch, u, s);
        }
      } else if (in && is_kv) {
        uint16_t* pool = reinterpret_cast<uint16_t*>(is_v ? a.v_pool : a.k_pool);
        *reinterpret_cast<uint4*>(pool + (ph * P + tp.slot) * kHeadDim + d0) = y;
      }
      if (in && !is_kv) *reinterpret_cast<uint4*>(q_out + (size_t)r * kHeadDim) = y;
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

// A CTA per token while that many CTAs are resident at once (eight per SM), so that a
// decode step takes one round of loads; beyond that a warp per token.
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
  return a.tok.q4 ? launch_tokens(append_kernel<true, 8>, append_kernel<true, 1>, a, s)
                  : launch_tokens(append_kernel<false, 8>, append_kernel<false, 1>, a, s);
}

cudaError_t launch_read(const KvReadArgs& a, cudaStream_t s) {
  return a.tok.q4 ? launch_tokens(read_kernel<true, 8>, read_kernel<true, 1>, a, s)
                  : launch_tokens(read_kernel<false, 8>, read_kernel<false, 1>, a, s);
}

}  // namespace locks
