// Host-side checks and small helpers shared by the files that implement the C ABI.
#pragma once

#include <cudaTypedefs.h>

#include <cmath>
#include <mutex>

#include "../../include/locks.h"
#include "../../include/lockskv.h"
#include "common.cuh"
#include "kernels.h"

namespace locks {

constexpr size_t kAlign = 256;
inline size_t align_up(size_t x) { return (x + kAlign - 1) / kAlign * kAlign; }

inline int device_sm_count() {
  static int cache[64] = {0};
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess || dev < 0) return 152;
  if (dev < 64 && cache[dev] > 0) return cache[dev];
  int n = 0;
  if (cudaDeviceGetAttribute(&n, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess || n <= 0) n = 152;
  if (dev < 64) cache[dev] = n;
  return n;
}

inline bool is_q4(const locks_cache_t* c) { return c->kv_format == LOCKS_KV_Q4; }

inline locks_status_t check_cache(const locks_cache_t* c, bool need_kv) {
  if (!c) return LOCKS_ERR_INVALID_ARG;
  if (c->batch <= 0 || c->num_kv_heads <= 0 || c->pages_total <= 0 || c->max_pages <= 0)
    return LOCKS_ERR_INVALID_ARG;
  if (c->head_dim != kHeadDim || (c->page_size != kPage && c->page_size != 16)) return LOCKS_ERR_UNSUPPORTED;
  if (c->kv_format != LOCKS_KV_BF16 && c->kv_format != LOCKS_KV_Q4) return LOCKS_ERR_INVALID_ARG;
  if (need_kv) {
    const void* v_pool = is_q4(c) ? c->k_pool : c->v_pool;  // a 4-bit block holds both
    if (!c->k_pool || !v_pool || !c->block_table || !c->seq_lens) return LOCKS_ERR_INVALID_ARG;
    if ((reinterpret_cast<uintptr_t>(c->k_pool) | reinterpret_cast<uintptr_t>(v_pool)) & 15)
      return LOCKS_ERR_INVALID_ARG;
  }
  // TMA row coordinate and 32-bit page-head offsets
  // (key rows >= basis rows, since r <= 16 <= P)
  if ((long long)c->pages_total * c->num_kv_heads * c->page_size > 0x7fffffffLL) return LOCKS_ERR_UNSUPPORTED;
  if ((long long)c->max_pages * c->page_size > 0x7fffffffLL) return LOCKS_ERR_UNSUPPORTED;
  return LOCKS_OK;
}

inline locks_status_t check_params(const locks_cache_t* c, const locks_params_t* p) {
  if (!p) return LOCKS_ERR_INVALID_ARG;
  if (p->num_q_heads <= 0 || p->num_q_heads % c->num_kv_heads) return LOCKS_ERR_INVALID_ARG;
  const int G = p->num_q_heads / c->num_kv_heads;
  if (G > 16) return LOCKS_ERR_UNSUPPORTED;
  if (p->budget_tokens < 0 || (p->flags & ~(LOCKS_FLAG_UNFUSED | LOCKS_FLAG_FUSED)) != 0) return LOCKS_ERR_INVALID_ARG;
  if ((p->flags & LOCKS_FLAG_UNFUSED) && (p->flags & LOCKS_FLAG_FUSED)) return LOCKS_ERR_INVALID_ARG;
  if (!(p->scale >= 0.f) || !std::isfinite(p->scale)) return LOCKS_ERR_INVALID_ARG;
  return LOCKS_OK;
}

inline float scale_of(const locks_params_t* p) {
  return p->scale > 0.f ? p->scale : 1.0f / std::sqrt((float)kHeadDim);
}

template <typename T>
inline T* at(void* ws, size_t off) {
  return reinterpret_cast<T*>(static_cast<uint8_t*>(ws) + off);
}

inline PFN_cuTensorMapEncodeTiled_v12000 encode_fn() {
  static PFN_cuTensorMapEncodeTiled_v12000 fn = nullptr;
  static std::once_flag once;
  std::call_once(once, [] {
    void* p = nullptr;
    cudaDriverEntryPointQueryResult q = cudaDriverEntryPointSymbolNotFound;
    if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &p, 12000, cudaEnableDefault, &q) ==
            cudaSuccess &&
        q == cudaDriverEntryPointSuccess)
      fn = reinterpret_cast<PFN_cuTensorMapEncodeTiled_v12000>(p);
  });
  return fn;
}

// 2-D view of 128-column 16-bit rows; 64-column boxes of box_rows rows with
// 128-byte swizzle.  (Copies move bits, so the type only says their size.)
inline bool encode_matrix(CUtensorMap* m, const void* pool, size_t rows, int box_rows) {
  auto fn = encode_fn();
  if (!fn) return false;
  cuuint64_t dims[2] = {(cuuint64_t)kHeadDim, (cuuint64_t)rows};
  cuuint64_t strides[1] = {(cuuint64_t)kHeadDim * 2};
  cuuint32_t box[2] = {64, (cuuint32_t)box_rows};
  cuuint32_t estr[2] = {1, 1};
  CUresult r = fn(m, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 2, const_cast<void*>(pool), dims, strides, box, estr,
                  CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                  CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
  return r == CUDA_SUCCESS;
}

// A pool of bf16 pages (rows = pages_total * Hkv * rows_per_page).
inline bool encode_rows(CUtensorMap* m, const void* pool, const locks_cache_t* c, int rows_per_page, int box_rows) {
  return encode_matrix(m, pool, (size_t)c->pages_total * c->num_kv_heads * rows_per_page, box_rows);
}

// K or V pool: boxes of one page-head's rows x 64 columns (one page-head is
// two boxes).
inline bool encode_pool(CUtensorMap* m, const void* pool, const locks_cache_t* c) {
  return encode_rows(m, pool, c, c->page_size, c->page_size);
}

inline locks_status_t cuda_status(cudaError_t e) { return e == cudaSuccess ? LOCKS_OK : LOCKS_ERR_CUDA; }

inline locks_status_t check_tokens(const locks_cache_t* c, const lockskv_tokens_t* t) {
  if (!t || t->total < 0 || t->max_tokens < 0) return LOCKS_ERR_INVALID_ARG;
  if (!t->cu_tokens && (t->total != c->batch || t->max_tokens > 1)) return LOCKS_ERR_INVALID_ARG;
  return LOCKS_OK;
}

// bf16 token rows: 16-byte aligned, `stride` elements apart, `row` elements long.
inline locks_status_t check_rows(const void* p, int64_t stride, int64_t row) {
  if ((reinterpret_cast<uintptr_t>(p) & 15) || stride < row || (stride & 7)) return LOCKS_ERR_INVALID_ARG;
  return LOCKS_OK;
}

// A workspace that only holds the error word (or none).
inline locks_status_t check_err_ws(void* ws, size_t bytes) {
  if (ws && (bytes < sizeof(int) || (reinterpret_cast<uintptr_t>(ws) & (kAlign - 1)))) return LOCKS_ERR_WORKSPACE;
  return LOCKS_OK;
}

}  // namespace locks
