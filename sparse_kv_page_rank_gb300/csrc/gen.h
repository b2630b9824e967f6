// Internal launch interface between the C ABI of locksgen.h (gen_api.cu) and its kernels.
#pragma once

#include <cuda.h>
#include <cuda_runtime.h>
#include <stdint.h>

#include "../../include/locksgen.h"

namespace locks {

// Choice of continuations (gen_select.cu).
constexpr int kSelectChunk = 4096, kSelectSmall = 2048;  // logits that a CTA takes into its registers
constexpr int kSelectCtas = 4;  // of them per SM
struct SelectArgs {
  const void* logits;
  const float* scores;
  const int32_t* ended;  // or null
  float* out_scores;
  int32_t* out_parents;
  int32_t* out_tokens;
  int32_t* out_ended;  // or null
  float4* parts;       // ws: [rows][n_parts] (maximum, sum of exponentials, entries of the list as bits, -)
  uint2* lists;        // ws: [rows][n_parts][keep] (ordered logit, token), best first
  int* err;
  long long row_stride;
  int batch, beams, vocab, keep, end_token;
  int n_parts, chunks;  // parts of a row, chunks of a part
  int small;            // 1: chunks of kSelectSmall
};
cudaError_t launch_select(const SelectArgs& a, bool f32, cudaStream_t s);

// Rows that follow their parents (gen_reorder.cu).
constexpr int kReorderLayers = 64;  // caches of one launch
struct ReorderRow {
  int parent, owner;  // rows whose table entries this one takes before, and from, column `split`
  int split;
  int tokens;         // of the open page, in whole groups of 16, to be copied; 0 for none
  int src, dst;       // its physical pages
};
struct ReorderArgs {
  const int32_t* parents;
  int32_t* block_table;
  int32_t* seq_lens;
  int32_t* n_summarized;  // or null
  ReorderRow* rows;       // ws: [batch]
  int* err;
  int batch, beams, num_kv_heads, max_pages, pages_total, page_size, q4;
  int n_layers;
  void* k_pool[kReorderLayers];
  void* v_pool[kReorderLayers];
};
bool reorder_fits(const ReorderArgs& a, int layers);  // the launch of so many layers
cudaError_t launch_reorder_plan(const ReorderArgs& a, cudaStream_t s);
cudaError_t launch_reorder_move(const ReorderArgs& a, bool tables, int sms, cudaStream_t s);

// Attention of rows that share pages (gen_attend.cu).
constexpr int kSharedRows = 32;  // (row, head) pairs that a pass over the shared pages serves
// Places that a segment has beyond its tiles.  Measured (1, 2, 3, 4): bf16 pages, 131,000 shared
// tokens 98.6, 92.7, 89.0, 90.6 us, 64 rows of 32 K 54.7, 48.0, 47.2, 46.9; 4-bit, four requests of 16 K, 64-token pages
// 44.0, 40.1, 39.5, 40.9, 16-token ones 45.3, 41.3, 41.2, 42.5.
constexpr int kSegment = 3;
struct GroupArgs {
  const uint16_t* q;  // bf16 [batch][Hq][d]
  const uint8_t* blocks;  // LOCKS_KV_Q4 blocks
  const int32_t* block_table;
  const int32_t* seq_lens;
  const int32_t* shared_pages;  // [batch / beams]
  uint16_t* out;
  float* lse;         // or null
  uint32_t* offsets;  // ws: [requests + 1] first place of each in the line, and their number
  // ws, partial results: [ctas + problems * blocks][kSharedRows] of the shared parts, then
  // [ctas + batch * Hkv][group] of the rows' own
  float* part_o;
  float2* part_ml;
  int* err;
  int batch, beams, num_kv_heads, group, max_pages, pages_total, page_size;
  int n_blocks;       // blocks of kSharedRows rows of a request's head
  int n_ctas;
  float scale_log2;
  int q4;
};
int group_attend_ctas_per_sm(bool q4);
cudaError_t launch_group_attend(const GroupArgs& a, const CUtensorMap& tk, const CUtensorMap& tv, cudaStream_t s);

}  // namespace locks
