// Rows of a cache that follow their parents: block tables, lengths and open pages.
//
// A request's rows are W <= 32 lanes of one warp.  Of the W rows, D are somebody's parent;
// their open pages stay with their lowest children.  The other W - D rows of the result,
// further children and idle ones, take the pages of the W - D rows that are nobody's
// parent: as many as are needed, so no page is allocated, and a copy reads pages that stay
// and writes pages that were given up, so the copies of one call do not wait for each
// other.  Columns before the open page are references and change no page.
//
// The first kernel writes this plan, the lengths and the counts; the second permutes the
// tables, column by column (a thread reads all rows of its column before it writes any), and
// copies the open pages of all layers.
//
// What bounds it: the copied pages' bytes, for few the latency of the two launches.
// Measured (floor by bytes), in a graph: 16 requests of 8 beams, four layers of bf16 pages 13.1 us
// (6.4); 32 of 8, 16 layers 69.6 us (53.1); one request of 4 beams, a table of 2048 columns 3.5 us.
#include <algorithm>

#include "common.cuh"
#include "gen.h"

namespace locks {

namespace {

constexpr int kThreads = 256;
constexpr int kColumnThreads = 64;            // columns of a CTA that permutes tables
// A CTA copies a head of a 64-token page (of one pool), or four of 16-token ones, at a time: what
// a thread then has in flight, 16 bytes each.
constexpr int kFlight = 4;
static_assert(64 * kHeadDim * 2 <= kFlight * kThreads * 16 && LOCKS_KV_Q4_BLOCK_BYTES(64) <= kFlight * kThreads * 16 &&
                  16 * kHeadDim * 2 <= kThreads * 16 && LOCKS_KV_Q4_BLOCK_BYTES(16) <= kThreads * 16,
              "a thread's share of a head");
constexpr int kCopyCtas = 8;                  // per SM

// The n-th set bit (from 0) of m.
__device__ __forceinline__ int nth_bit(uint32_t m, int n) {
  for (; n > 0; --n) m &= m - 1;
  return __ffs(m) - 1;
}

// One warp per request.
__global__ void plan_kernel(const ReorderArgs a) {
  const int lane = threadIdx.x, W = a.beams, base = blockIdx.x * W, P = a.page_size;
  pdl_wait();
  pdl_launch_dependents();
  const bool in = lane < W;
  int p = in ? a.parents[base + lane] : -1;
  if (p < -1 || p >= W) {
    set_error(a.err, LOCKSGEN_DEVERR_PARENT);
    p = -1;
  }
  int len = in ? a.seq_lens[base + lane] : 0;
  const int nsum = in && a.n_summarized ? a.n_summarized[base + lane] : 0;
  const bool fits = len >= 0 && (long long)len <= (long long)a.max_pages * P;
  // a row that no table can hold has no copies; it may still give up its pages, none of
  // which is known to be its own but those from its last column on
  const int open = !fits ? a.max_pages : len / P;
  const uint32_t ok_rows = __ballot_sync(0xffffffffu, in && fits);
  if (p >= 0 && !(ok_rows >> p & 1)) {
    set_error(a.err, LOCKS_DEVERR_LENGTHS);
    p = -1;
  }
  const uint32_t same = __match_any_sync(0xffffffffu, p);
  const bool first = p >= 0 && __ffs(same) - 1 == lane;
  const uint32_t used = __reduce_or_sync(0xffffffffu, p >= 0 ? 1u << p : 0u);
  const uint32_t all = W == 32 ? 0xffffffffu : (1u << W) - 1u;
  const uint32_t unused = all & ~used;
  const uint32_t further = __ballot_sync(0xffffffffu, in && p >= 0 && !first);
  const uint32_t idle = __ballot_sync(0xffffffffu, in && p < 0);
  const uint32_t below = (1u << lane) - 1u;
  int owner = p;
  if (in && !first) {
    const int n = p >= 0 ? __popc(further & below) : __popc(further) + __popc(idle & below);
    owner = nth_bit(unused, n);
  }
  const int src_row = p >= 0 ? p : 0;
  const int p_len = __shfl_sync(0xffffffffu, len, src_row), p_nsum = __shfl_sync(0xffffffffu, nsum, src_row);
  const int o_open = __shfl_sync(0xffffffffu, open, owner < 0 ? 0 : owner);
  if (!in) return;
  ReorderRow r = {};
  int new_len = 0, new_nsum = 0;
  if (p >= 0 && !first && o_open > p_len / P) {
    // its pages up to o_open may be others' too
    set_error(a.err, LOCKS_DEVERR_LENGTHS);
    p = -1;
  }
  r.parent = base + (p >= 0 ? p : owner);
  r.owner = base + owner;
  if (p >= 0) {
    new_len = p_len;
    new_nsum = p_nsum;
    r.split = p_len / P;
    const int n = p_len - r.split * P;
    if (!first && n > 0) {
      r.src = a.block_table[(size_t)r.parent * a.max_pages + r.split];
      r.dst = a.block_table[(size_t)r.owner * a.max_pages + r.split];
      if (r.src < 0 || r.src >= a.pages_total || r.dst < 0 || r.dst >= a.pages_total || r.src == r.dst)
        set_error(a.err, LOCKS_DEVERR_BLOCK_TABLE);
      else
        r.tokens = (n + 15) / 16 * 16;
    }
  }
  a.rows[base + lane] = r;
  a.seq_lens[base + lane] = new_len;
  if (a.n_summarized) a.n_summarized[base + lane] = new_nsum;
}

// The first n_tables CTAs permute tables, `chunks` of columns per request; the others copy:
// every one finds the rows that have a page to copy, 256 rows at a time, and takes its share
// of their pages' pieces in all layers.
__global__ void __launch_bounds__(kThreads) move_kernel(const __grid_constant__ ReorderArgs a, int chunks, int n_tables,
                                                        int pieces) {
  const int tid = threadIdx.x, W = a.beams;
  pdl_wait();
  pdl_launch_dependents();
  if ((int)blockIdx.x < n_tables) {
    __shared__ int col[LOCKSGEN_MAX_BEAMS][kColumnThreads];
    __shared__ ReorderRow plan[LOCKSGEN_MAX_BEAMS];
    const int g = blockIdx.x / chunks, c0 = blockIdx.x % chunks * kColumnThreads;
    const int base = g * W;
    if (tid < W) plan[tid] = a.rows[base + tid];
    // each of the CTA's columns by kThreads / kColumnThreads threads, rows dealt among them
    const int c = c0 + tid % kColumnThreads, sub = tid / kColumnThreads;
    constexpr int kSub = kThreads / kColumnThreads;
    int32_t* table = a.block_table + (size_t)base * a.max_pages;
    if (c < a.max_pages)
#pragma unroll 4
      for (int w = sub; w < W; w += kSub) col[w][tid % kColumnThreads] = table[(size_t)w * a.max_pages + c];
    __syncthreads();
    if (c < a.max_pages)
#pragma unroll 4
      for (int w = sub; w < W; w += kSub) {
        const int from = (c < plan[w].split ? plan[w].parent : plan[w].owner) - base;
        if (from != w) table[(size_t)w * a.max_pages + c] = col[from][tid % kColumnThreads];
      }
    return;
  }
  __shared__ ReorderRow todo[kThreads];
  __shared__ int found[kThreads / 32];
  const int lane = tid & 31, warp = tid >> 5, n_ctas = gridDim.x - n_tables;
  const int hkv = a.num_kv_heads, P = a.page_size;
  const size_t page_bytes = a.q4 ? (size_t)hkv * LOCKS_KV_Q4_BLOCK_BYTES(P) : (size_t)hkv * P * kHeadDim * 2;
  for (int row0 = 0; row0 < a.batch; row0 += kThreads) {
    ReorderRow mine = {};
    if (row0 + tid < a.batch) mine = a.rows[row0 + tid];
    const uint32_t copies = __ballot_sync(0xffffffffu, mine.tokens > 0);
    __syncthreads();  // the last rows are done with
    if (lane == 0) found[warp] = __popc(copies);
    __syncthreads();
    int at = __popc(copies & ((1u << lane) - 1u)), n = 0;
    for (int w = 0; w < kThreads / 32; ++w) {
      at += w < warp ? found[w] : 0;
      n += found[w];
    }
    if (mine.tokens > 0) todo[at] = mine;
    __syncthreads();
    // heads of a page, page by page, layer by layer
    const int items = n * pieces * a.n_layers, heads = hkv * (a.q4 ? 1 : 2);
    const bool small = P == 16;
    for (int i = blockIdx.x - n_tables; i < items; i += n_ctas) {
      const int rest = i / pieces, layer = rest / n;
      const ReorderRow r = todo[rest - layer * n];
      const int h0 = (i - rest * pieces) * (small ? kFlight : 1), groups = r.tokens / 16;
      const int units = groups * (a.q4 ? 144 : 256);  // of 16 bytes, of a head
      uint8_t *k_pool = static_cast<uint8_t*>(a.k_pool[layer]), *v_pool = static_cast<uint8_t*>(a.v_pool[layer]);
      const size_t src = r.src * page_bytes, dst = r.dst * page_bytes;
      uint4 v[kFlight];
      uint8_t* out[kFlight];
#pragma unroll
      for (int k = 0; k < kFlight; ++k) {
        int h = h0 + (small ? k : 0);
        const int x = tid + (small ? 0 : k * kThreads);
        out[k] = nullptr;
        if (h >= heads || x >= units) continue;
        uint8_t* pool = k_pool;
        size_t off;
        if (a.q4) {
          // four parts of a block, each with those of the first 16 tokens first
          off = (size_t)h * LOCKS_KV_Q4_BLOCK_BYTES(P) + 16 * x;
          if (x >= 136 * groups) off += 136 * P - 16 * 136 * groups;
          else if (x >= 72 * groups) off += 72 * P - 16 * 72 * groups;
          else if (x >= 64 * groups) off += 64 * P - 16 * 64 * groups;
        } else {
          if (h >= hkv) h -= hkv, pool = v_pool;
          off = (size_t)h * P * kHeadDim * 2 + 16 * x;
        }
        v[k] = *reinterpret_cast<const uint4*>(pool + src + off);
        out[k] = pool + dst + off;
      }
#pragma unroll
      for (int k = 0; k < kFlight; ++k)
        if (out[k]) *reinterpret_cast<uint4*>(out[k]) = v[k];
    }
  }
}

cudaLaunchConfig_t config(unsigned grid, unsigned block, cudaLaunchAttribute* attr, cudaStream_t s) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(grid, 1, 1);
  cfg.blockDim = dim3(block, 1, 1);
  cfg.stream = s;
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cfg;
}

}  // namespace

cudaError_t launch_reorder_plan(const ReorderArgs& a, cudaStream_t s) {
  cudaLaunchAttribute attr[1];
  const cudaLaunchConfig_t cfg = config(a.batch / a.beams, 32, attr, s);
  return cudaLaunchKernelEx(&cfg, plan_kernel, a);
}

static int table_chunks(const ReorderArgs& a) { return (a.max_pages + kColumnThreads - 1) / kColumnThreads; }
static int page_pieces(const ReorderArgs& a) {
  const int heads = a.num_kv_heads * (a.q4 ? 1 : 2);
  return a.page_size == 16 ? (heads + kFlight - 1) / kFlight : heads;
}

bool reorder_fits(const ReorderArgs& a, int layers) {
  return (long long)table_chunks(a) * (a.batch / a.beams) + (long long)page_pieces(a) * a.batch * layers <= 0x7fffffffLL;
}

cudaError_t launch_reorder_move(const ReorderArgs& a, bool tables, int sms, cudaStream_t s) {
  const int chunks = table_chunks(a), pieces = page_pieces(a);
  const int n_tables = tables ? chunks * (a.batch / a.beams) : 0;
  // at most all rows of a request but one are copies
  const long long items = (long long)pieces * (a.batch / a.beams) * (a.beams - 1) * a.n_layers;
  const int copies = (int)std::min<long long>(items, (long long)kCopyCtas * sms);
  if (n_tables + copies == 0) return cudaSuccess;
  cudaLaunchAttribute attr[1];
  const cudaLaunchConfig_t cfg = config((unsigned)(n_tables + copies), kThreads, attr, s);
  return cudaLaunchKernelEx(&cfg, move_kernel, a, chunks, n_tables, pieces);
}

}  // namespace locks
