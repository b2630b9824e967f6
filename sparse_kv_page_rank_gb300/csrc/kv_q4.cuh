// The 4-bit page format (LOCKS_KV_Q4 in locks.h) as the kernels that compute on it
// see it, and the fp16-pair arithmetic that takes its codes apart.
#pragma once

#include <cuda_fp16.h>

#include "common.cuh"

namespace locks {

constexpr int kQ4Slot = LOCKS_KV_Q4_BLOCK_BYTES(64);  // 64 tokens: one page, or four 16-token pages

// Byte offset of 16-token tile t's part in a buffer of N tiles: of a 64-token page
// (or N tiles of one) each of the four parts of all tokens together, of 16-token
// pages one page per tile.
template <int P, int N = 4>
struct Q4Tile {
  __device__ static uint32_t key_codes(int t) { return P == 64 ? 1024 * t : 2304 * t; }
  __device__ static uint32_t key_scales(int t) { return P == 64 ? 1024 * N + 128 * t : 2304 * t + 1024; }
  __device__ static uint32_t value_codes(int t) { return P == 64 ? 1152 * N + 1024 * t : 2304 * t + 1152; }
  __device__ static uint32_t value_scales(int t) { return P == 64 ? 2176 * N + 128 * t : 2304 * t + 2176; }
};

__device__ __forceinline__ uint32_t pack_f16(float lo, float hi) {
  const __half2 v = __floats2half2_rn(lo, hi);
  return *reinterpret_cast<const uint32_t*>(&v);
}
__device__ __forceinline__ float f16_lo(uint32_t w) { return __low2float(*reinterpret_cast<__half2*>(&w)); }
__device__ __forceinline__ float f16_hi(uint32_t w) { return __high2float(*reinterpret_cast<__half2*>(&w)); }
__device__ __forceinline__ uint32_t mul_f16x2(uint32_t a, uint32_t b) {
  uint32_t d;
  asm("mul.rn.f16x2 %0, %1, %2;\n" : "=r"(d) : "r"(a), "r"(b));
  return d;
}
__device__ __forceinline__ uint32_t sub_f16x2(uint32_t a, uint32_t b) {
  uint32_t d;
  asm("sub.rn.f16x2 %0, %1, %2;\n" : "=r"(d) : "r"(a), "r"(b));
  return d;
}
__device__ __forceinline__ uint32_t fma_f16x2(uint32_t a, uint32_t b, uint32_t c) {
  uint32_t d;
  asm("fma.rn.f16x2 %0, %1, %2, %3;\n" : "=r"(d) : "r"(a), "r"(b), "r"(c));
  return d;
}
// (w & MASK) | MAGIC in one operation (written out: the compiler makes two of the
// expression, which cost the decode kernel 64 of 313 instructions per 16 tokens).
template <uint32_t MASK, uint32_t MAGIC>
__device__ __forceinline__ uint32_t field_under(uint32_t w) {
  uint32_t d;
  asm("lop3.b32 %0, %1, %2, %3, 0xea;\n" : "=r"(d) : "r"(w), "n"(MASK), "n"(MAGIC));
  return d;
}
// Fields 0 and 1 (bits 0-3, 4-7) of both halves of w, each holding code + 8, as
// fp16 pairs of codes: a field under the exponent of 1024 (or, four bits up, of
// 64) is the number 1024 + u (64 + u) exactly, from which 1032 (72) is taken.
__device__ __forceinline__ void q4_codes01(uint32_t w, uint32_t& f0, uint32_t& f1) {
  f0 = sub_f16x2(field_under<0x000f000fu, 0x64006400u>(w), 0x64086408u);
  f1 = sub_f16x2(field_under<0x00f000f0u, 0x54005400u>(w), 0x54805480u);
}

}  // namespace locks
