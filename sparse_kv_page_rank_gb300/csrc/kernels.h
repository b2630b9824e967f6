// Internal launch interface between the C-ABI layer (api.cu) and the kernels.
#pragma once

#include <cuda.h>
#include <cuda_runtime.h>
#include <stdint.h>

namespace locks {

// Summary scan: page-mass estimates s_hat for every summarised page and head.
struct ScanArgs {
  const uint16_t* basis_t;     // bf16 [pages_total][Hkv][r][d]
  const uint16_t* coeffs;      // bf16 [pages_total][Hkv][P][r]
  const uint16_t* q;           // bf16 [B][Hq][d]
  const int32_t* block_table;  // [B][max_pages]
  const int32_t* seq_lens;     // [B]
  const int32_t* n_summarized; // [B]
  float* shat;                 // ws: [B*Hkv][max_pages][G] natural log
  float2* part;                // ws: [B*Hkv][n_chunks][G] (max, sum) of base-2 LSE
  float* page_lse;             // optional [B][Hq][max_pages]
  int* err;
  int batch, num_kv_heads, group, rank, max_pages, pages_total;
  int chunk_pages, n_chunks;
  float scale_log2;            // scale * log2(e)
  int q4;                      // 1: basis_t holds LOCKS_DTYPE_Q4 blocks (coeffs unused)
  int packed;                  // 1: basis_t holds LOCKS_DTYPE_BF16_PACKED blocks (coeffs unused)
  int page_size;               // P: 64 or 16
  int heads_per_block;         // HG: KV heads one CTA scans together (a power of two dividing Hkv, <= 4)
  // set by the launcher: ring of `slots` slots, one page of the head block each
  int slots, slot_bytes, basis_bytes, coef_bytes;
};

// GSA scores + top-k (chunk-local candidates, merged by the last CTA).
struct TopkArgs {
  const float* shat;
  const float2* part;
  int n_scan_chunks;
  const int32_t* seq_lens;
  const int32_t* n_summarized;
  uint32_t* cand_key;   // ws: [B*Hkv][n_chunks][k_max]
  int32_t* cand_idx;    // ws: same
  unsigned* counters;   // ws: [B*Hkv]
  int32_t* sel_pages;   // [B*Hkv][k_max]
  int32_t* sel_count;   // [B*Hkv]
  const int32_t* block_table;  // read before the grid dependency wait when sel_phys is set
  int32_t* sel_phys;    // ws: [B*Hkv][k_max] physical page of each selected page (one-chunk problems), or null
  int* err;
  int batch, num_kv_heads, group, max_pages, k_max;
  int chunk_pages, n_chunks;
  size_t smem_keys;     // capacity (entries) of the dynamic key buffer
  int page_size;
};

// Paged flash-decode over a page list (sparse), every page (dense), or the
// exact per-page LSE of every page (page_lse mode).
struct AttendArgs {
  const uint16_t* q;
  const int32_t* block_table;
  const int32_t* seq_lens;
  const int32_t* n_summarized;
  const int32_t* sel_pages;   // sparse mode only
  const int32_t* sel_count;   // sparse mode only
  const int32_t* sel_phys;    // sparse mode inside the decode step: physical pages of sel_pages, or null
  uint16_t* out;              // bf16 [B][Hq][d]
  float* lse;                 // optional [B][Hq]
  float* page_lse;            // page_lse mode: [B][Hq][max_pages]
  float* part_o;              // ws: [B*Hkv][n_splits][G][d]
  float2* part_ml;            // ws: [B*Hkv][n_splits][G]
  unsigned* counters;         // ws: [B*Hkv]
  int* err;
  int batch, num_kv_heads, group, max_pages, pages_total, k_max;
  int n_splits;               // CTAs per problem = cluster * clusters per problem
  int cluster;                // CTAs per thread-block cluster (1 in page-LSE mode)
  int inputs_early;           // 1: the step's inputs may be read before the grid dependency wait
  float scale_log2;
  int page_size;              // P: 64 (one page per 64-token tile) or 16 (four pages per tile)
  // fused mode only: the scan's page-mass estimates and per-CTA partials,
  // from which the cluster selects the pages itself
  const float* shat;          // ws: [B*Hkv][max_pages][G] natural log
  const float2* part;         // ws: [B*Hkv][n_scan_chunks][G] (max, sum) of base-2 LSE
  int n_scan_chunks;
  const uint16_t* k_pool16;   // fused mode: pool bases for L2 prefetches of likely pages; LOCKS_KV_Q4: the blocks
  const uint16_t* v_pool16;
  int32_t* sel_pages_out;     // fused mode: the page list it selected, [B*Hkv][k_max] (as locks_select)
  int32_t* sel_count_out;     // fused mode: [B*Hkv]
  // newest tokens of LOCKS_KV_Q4 pages only (launch_attend_q4_rows)
  const int32_t* cu_tokens;   // [B+1], or null: one token each
  int64_t q_stride;
  int total, max_tokens;
  int join_blocks;            // set by the launch
  unsigned long long* trace_cta;  // tracing builds only: per-CTA timestamps [B*Hkv][n_splits][16], or null
};

// kAttendFused: the sparse mode with the group-shared top-k computed inside
// the thread-block cluster from the scan's outputs (64-token pages, k_max <=
// kFusedMaxK, at most kAttendThreads summarised pages per CTA of the cluster).
enum AttendMode { kAttendSparse = 0, kAttendDense = 1, kAttendPageLse = 2, kAttendFused = 3 };
constexpr int kFusedMaxK = 32;
constexpr int kFusedPrefetch = 4;  // each CTA's best pages whose K/V are prefetched into L2 before the merge

// Summary builder.
struct BuildArgs {
  const uint16_t* k_pool;  // bf16 pages, or LOCKS_KV_Q4 blocks
  void* basis_t;
  void* coeffs;
  const int32_t* page_ids;
  int n, num_kv_heads, rank, pages_total;
  int format;  // LOCKS_DTYPE_BF16 / _F32 (basis_t + coeffs) or _Q4 (packed blocks in basis_t)
  int* err;
  int page_size;
  int kv_q4;  // 1: the pages are LOCKS_KV_Q4 blocks
};

// The newest tokens of a batch (lockskv.h), as the cache-writing kernels see them.
struct KvTokenArgs {
  const int32_t* cu_tokens;  // [batch + 1], or null: one token per sequence
  const int32_t* block_table;
  const int32_t* seq_lens;
  int* err;
  int batch, num_kv_heads, max_pages, pages_total, page_size;
  int total, max_tokens;
  int q4;  // 1: k_pool holds LOCKS_KV_Q4 blocks (v_pool unused)
};
struct KvAppendArgs {
  KvTokenArgs tok;
  void* k_pool;
  void* v_pool;
  const uint16_t* k;
  const uint16_t* v;
  const uint16_t* q;  // or null
  uint16_t* q_out;
  const float* rope;
  const int32_t* positions;  // or null: the position in the sequence
  long long k_stride, v_stride, q_stride, q_out_stride;  // elements
  int num_q_heads, rope_rows, rotary_dim, interleaved;
  // positions of several axes (num_axes > 0): positions is [num_axes][axis_stride], and
  // pair i is of axis pair_axes[i / 16] >> 2 (i % 16) & 3
  int num_axes;
  long long axis_stride;
  uint32_t pair_axes[4];
};
struct KvReadArgs {
  KvTokenArgs tok;
  const void* k_pool;
  const void* v_pool;
  uint16_t* k_out;  // or null
  uint16_t* v_out;  // or null
};

// Causal attention of the newest tokens (prompt.cu).
struct PromptArgs {
  const uint16_t* q;         // bf16 [total][Hq][d], rows q_stride elements apart
  long long q_stride;
  const void* k_pool;        // LOCKS_KV_Q4: the blocks
  const void* v_pool;
  const int32_t* cu_tokens;  // or null
  const int32_t* block_table;
  const int32_t* seq_lens;
  uint16_t* out;
  float* lse;                // or null
  float* part_o;             // ws: [tiles that are cut][n_splits][256][d]
  float2* part_ml;           // ws: the same without d: (reference, sum), base 2
  int* err;
  int batch, num_kv_heads, group, max_pages, pages_total, page_size;
  int total, max_tokens;
  int n_qtiles;              // CTAs along a sequence's new tokens (256 rows each; 128 for 4-bit codes)
  int one_tile;              // bf16 pages: a sequence's new rows fit one tile of 128
  int n_whole, n_splits;     // row tiles of one CTA each; CTAs along the keys of each of the others
  float scale_log2;
  int q4;
  uint16_t* planes;          // many rows: ws [3 (4-bit pages, fp16) or 2 (bf16)][B][Hkv][plane_rows][d]; else null
  int plane_rows;            // tokens of a plane, whole blocks of 128
};

// tk, tv: the pools; with planes tk is their tensor map (boxes of 128 rows x 64 columns).
cudaError_t launch_prompt(const PromptArgs& a, const CUtensorMap& tk, const CUtensorMap& tv, cudaStream_t s);
cudaError_t launch_append(const KvAppendArgs& a, cudaStream_t s);
cudaError_t launch_read(const KvReadArgs& a, cudaStream_t s);
// Attention over a LOCKS_KV_Q4 cache, one query token per sequence.  `tiles`:
// 4 for many 16-token tiles per warp and turn, 1 where a CTA has few pages.
// Page list: a.cluster = a.n_splits CTAs per problem.  Every page: a.n_splits CTAs in
// all, a.part_* hold two partials per CTA, which a second kernel joins.
cudaError_t launch_attend_q4(const AttendArgs& a, int mode, int tiles, cudaStream_t s);
// The newest tokens of each sequence over every page, for few of them: blocks of
// kQ4RowColumns (token, head) rows; partials of that many columns.
cudaError_t launch_attend_q4_rows(const AttendArgs& a, int tiles, cudaStream_t s);
constexpr int kQ4RowColumns = 8;
// Clusters of cs CTAs of the page-list kernel that the device holds at once.
int attend_q4_active_clusters(int group, int page_size, int tiles, int cs);
constexpr int kQ4CtasPerSm = 2;

cudaError_t launch_scan(const ScanArgs& a, cudaStream_t s, bool pdl);
cudaError_t launch_topk(const TopkArgs& a, cudaStream_t s, bool pdl);
cudaError_t launch_attend(const AttendArgs& a, const CUtensorMap& tk, const CUtensorMap& tv,
                          int mode, cudaStream_t s, bool pdl);
cudaError_t launch_build(const BuildArgs& a, cudaStream_t s);

size_t topk_smem_bytes(size_t keys);
int topk_pages_per_cta(int group);  // pages one top-k CTA scores
int attend_max_cluster(int mode, int page_size);  // largest placeable cluster (<= 16) for that mode
                                                  // (kAttendFused: page_size 64 only)
int attend_active_clusters(int mode, int cs, int page_size);  // clusters of cs CTAs resident at once
// Scan CTA (one per SM): 16 consumer warps + 1 producer warp.
constexpr int kScanWarps = 16;
// KV heads one scan CTA covers: the largest power of two <= 4 dividing Hkv
// (measured on GB300: 4 beats 8 at 128K context and ties elsewhere).
inline int scan_heads_per_block(int num_kv_heads) {
  int hg = 4;
  while (num_kv_heads % hg) hg /= 2;
  return hg;
}
constexpr int kScanThreads = (kScanWarps + 1) * 32;
constexpr int kTopkThreads = 512;
constexpr int kAttendThreads = 128;

}  // namespace locks
