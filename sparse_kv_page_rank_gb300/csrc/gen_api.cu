// C ABI of locksgen.h, but for locksgen_append_axes (which is lockskv_append's, api.cu):
// host-side validation, launch planning, workspace layout.
#include <algorithm>
#include <cstring>

#include "gen.h"
#include "host.h"

namespace {

using namespace locks;

locks_status_t check_ws(void* ws, size_t bytes, size_t need) {
  if (!ws || (reinterpret_cast<uintptr_t>(ws) & (kAlign - 1)) || bytes < need) return LOCKS_ERR_WORKSPACE;
  return LOCKS_OK;
}

// Parts of the rows of a choice: small chunks while chunks are few, and as many parts as take
// least, in chunks' times: waves of CTAs, each of its chunks and some two more.
constexpr double kPartChunks = 2.0;
struct SelectPlan {
  int n_parts = 0, chunks = 1, small = 0;
  size_t off_parts = 0, off_lists = 0, total = 0;
};

constexpr long long kMaxLists = 16384;  // of a request: a CTA of the merge keeps two bytes of each

locks_status_t plan_select(const locksgen_choice_t* c, SelectPlan* pl) {
  if (!c || c->batch <= 0 || c->beams <= 0 || c->vocab <= 0 || c->keep <= 0) return LOCKS_ERR_INVALID_ARG;
  if (c->dtype != LOCKS_DTYPE_BF16 && c->dtype != LOCKS_DTYPE_F32) return LOCKS_ERR_INVALID_ARG;
  if (c->beams > LOCKSGEN_MAX_BEAMS || c->keep > LOCKSGEN_MAX_KEEP || c->vocab > LOCKSGEN_MAX_VOCAB) return LOCKS_ERR_UNSUPPORTED;
  const long long rows = (long long)c->batch * c->beams;
  if (rows > LOCKSGEN_MAX_ROWS) return LOCKS_ERR_UNSUPPORTED;  // the launch's second dimension
  // a row may begin inside its first 16 bytes
  const int vec = c->dtype == LOCKS_DTYPE_BF16 ? 8 : 4;
  const long long span = c->vocab + vec - 1, sms = device_sm_count();
  auto count = [&](int size) { return (span + size - 1) / size; };
  pl->small = rows * count(kSelectChunk) <= sms / 2 ? 1 : 0;
  const long long chunks = count(pl->small ? kSelectSmall : kSelectChunk);
  const long long slots = kSelectCtas * sms;
  double best = 1e30;
  for (long long n = 1; n <= chunks && n * c->beams <= kMaxLists; ++n) {
    const long long each = (chunks + n - 1) / n, waves = (rows * n + slots - 1) / slots;
    const double time = (double)waves * ((double)each + kPartChunks);
    if (time >= best) continue;
    best = time;
    pl->n_parts = (int)((chunks + each - 1) / each);
    pl->chunks = (int)each;
  }
  size_t off = kAlign;  // the error word
  pl->off_parts = off;
  off = align_up(off + sizeof(float4) * rows * pl->n_parts);
  pl->off_lists = off;
  pl->total = align_up(off + sizeof(uint2) * rows * pl->n_parts * c->keep);
  return LOCKS_OK;
}

locks_status_t check_beams(const locks_cache_t* c, int32_t beams) {
  if (beams <= 0 || c->batch % beams) return LOCKS_ERR_INVALID_ARG;
  return beams > LOCKSGEN_MAX_BEAMS ? LOCKS_ERR_UNSUPPORTED : LOCKS_OK;
}

size_t reorder_bytes(const locks_cache_t* c) { return align_up(kAlign + sizeof(ReorderRow) * c->batch); }

struct GroupPlan {
  int n_ctas = 0, n_blocks = 0;
  size_t off_line = 0, off_ml = 0, off_o = 0, total = 0;
};

locks_status_t plan_group(const locks_cache_t* c, const locks_params_t* p, int beams, GroupPlan* pl) {
  const int G = p->num_q_heads / c->num_kv_heads;
  const long long groups = c->batch / beams, hkv = c->num_kv_heads, rows = c->batch * hkv;
  if (rows > 0x7fffffffLL) return LOCKS_ERR_UNSUPPORTED;
  pl->n_blocks = (beams * G + kSharedRows - 1) / kSharedRows;
  const long long segments = groups * hkv * pl->n_blocks + rows;
  const long long tiles = ((long long)c->max_pages * c->page_size + kPage - 1) / kPage;
  if (segments * (tiles + kSegment) > 0x7fffffffLL) return LOCKS_ERR_UNSUPPORTED;  // places of the line are 32-bit numbers
  pl->n_ctas = (int)std::min<long long>((long long)group_attend_ctas_per_sm(is_q4(c)) * device_sm_count(), segments * tiles);
  const size_t parts = (size_t)(pl->n_ctas + groups * hkv * pl->n_blocks) * kSharedRows + (size_t)(pl->n_ctas + rows) * G;
  size_t off = kAlign;  // the error word
  pl->off_line = off;
  off = align_up(off + sizeof(uint32_t) * (groups + 1));
  pl->off_ml = off;
  off = align_up(off + sizeof(float2) * parts);
  pl->off_o = off;
  pl->total = align_up(off + sizeof(float) * parts * kHeadDim);
  return LOCKS_OK;
}

}  // namespace

extern "C" {

locks_status_t locksgen_select_workspace_size(const locksgen_choice_t* choice, size_t* bytes) {
  if (!bytes) return LOCKS_ERR_INVALID_ARG;
  SelectPlan pl;
  const locks_status_t st = plan_select(choice, &pl);
  if (st != LOCKS_OK) return st;
  *bytes = pl.total;
  return LOCKS_OK;
}

locks_status_t locksgen_select(const locksgen_choice_t* c, void* ws, size_t ws_bytes, void* stream) {
  SelectPlan pl;
  locks_status_t st = plan_select(c, &pl);
  if (st != LOCKS_OK) return st;
  if (!c->logits || !c->scores || !c->out_scores || !c->out_parents || !c->out_tokens) return LOCKS_ERR_INVALID_ARG;
  const size_t element = c->dtype == LOCKS_DTYPE_BF16 ? 2 : 4;
  if (c->row_stride < c->vocab || (reinterpret_cast<uintptr_t>(c->logits) & (element - 1))) return LOCKS_ERR_INVALID_ARG;
  if (c->end_token < -1 || c->end_token >= c->vocab || (c->ended && c->end_token < 0)) return LOCKS_ERR_INVALID_ARG;
  // (a request's rows are read before its continuations are written, but not before another's are)
  if (c->keep != c->beams && c->batch > 1 && (c->out_scores == c->scores || (c->ended && c->out_ended == c->ended))) return LOCKS_ERR_INVALID_ARG;
  if ((st = check_ws(ws, ws_bytes, pl.total)) != LOCKS_OK) return st;
  SelectArgs a;
  a.logits = c->logits;
  a.scores = c->scores;
  a.ended = c->ended;
  a.out_scores = c->out_scores;
  a.out_parents = c->out_parents;
  a.out_tokens = c->out_tokens;
  a.out_ended = c->out_ended;
  a.parts = at<float4>(ws, pl.off_parts);
  a.lists = at<uint2>(ws, pl.off_lists);
  a.err = at<int>(ws, 0);
  a.row_stride = c->row_stride;
  a.batch = c->batch;
  a.beams = c->beams;
  a.vocab = c->vocab;
  a.keep = c->keep;
  a.end_token = c->end_token;
  a.n_parts = pl.n_parts;
  a.chunks = pl.chunks;
  a.small = pl.small;
  return cuda_status(launch_select(a, c->dtype == LOCKS_DTYPE_F32, static_cast<cudaStream_t>(stream)));
}

locks_status_t locksgen_reorder_workspace_size(const locks_cache_t* cache, int32_t beams, size_t* bytes) {
  if (!bytes) return LOCKS_ERR_INVALID_ARG;
  locks_status_t st = check_cache(cache, false);
  if (st != LOCKS_OK) return st;
  if ((st = check_beams(cache, beams)) != LOCKS_OK) return st;
  *bytes = reorder_bytes(cache);
  return LOCKS_OK;
}

locks_status_t locksgen_reorder(const locks_cache_t* caches, int32_t num_caches, int32_t beams, const int32_t* parents,
                                void* ws, size_t ws_bytes, void* stream) {
  if (!caches || num_caches <= 0 || !parents) return LOCKS_ERR_INVALID_ARG;
  const locks_cache_t& c = caches[0];
  locks_status_t st;
  for (int i = 0; i < num_caches; ++i) {
    const locks_cache_t& x = caches[i];
    if ((st = check_cache(&x, true)) != LOCKS_OK) return st;
    if (x.block_table != c.block_table || x.seq_lens != c.seq_lens || x.n_summarized != c.n_summarized ||
        x.batch != c.batch || x.num_kv_heads != c.num_kv_heads || x.page_size != c.page_size ||
        x.pages_total != c.pages_total || x.max_pages != c.max_pages || x.kv_format != c.kv_format)
      return LOCKS_ERR_INVALID_ARG;
  }
  if ((st = check_beams(&c, beams)) != LOCKS_OK) return st;
  if ((st = check_ws(ws, ws_bytes, reorder_bytes(&c))) != LOCKS_OK) return st;
  const cudaStream_t s = static_cast<cudaStream_t>(stream);
  ReorderArgs a = {};
  a.parents = parents;
  a.block_table = const_cast<int32_t*>(c.block_table);
  a.seq_lens = const_cast<int32_t*>(c.seq_lens);
  a.n_summarized = const_cast<int32_t*>(c.n_summarized);
  a.rows = at<ReorderRow>(ws, kAlign);
  a.err = at<int>(ws, 0);
  a.batch = c.batch;
  a.beams = beams;
  a.num_kv_heads = c.num_kv_heads;
  a.max_pages = c.max_pages;
  a.pages_total = c.pages_total;
  a.page_size = c.page_size;
  a.q4 = is_q4(&c) ? 1 : 0;
  if (!reorder_fits(a, std::min(num_caches, kReorderLayers))) return LOCKS_ERR_UNSUPPORTED;
  if (launch_reorder_plan(a, s) != cudaSuccess) return LOCKS_ERR_CUDA;
  for (int first = 0; first < num_caches; first += kReorderLayers) {
    a.n_layers = std::min(kReorderLayers, num_caches - first);
    for (int i = 0; i < a.n_layers; ++i) {
      a.k_pool[i] = const_cast<void*>(caches[first + i].k_pool);
      a.v_pool[i] = const_cast<void*>(caches[first + i].v_pool);
    }
    if (launch_reorder_move(a, first == 0, device_sm_count(), s) != cudaSuccess) return LOCKS_ERR_CUDA;
  }
  return LOCKS_OK;
}

locks_status_t locksgen_attend_workspace_size(const locks_cache_t* cache, const locks_params_t* params, int32_t beams,
                                              size_t* bytes) {
  if (!bytes) return LOCKS_ERR_INVALID_ARG;
  locks_status_t st = check_cache(cache, false);
  if (st != LOCKS_OK) return st;
  if ((st = check_params(cache, params)) != LOCKS_OK) return st;
  if ((st = check_beams(cache, beams)) != LOCKS_OK) return st;
  GroupPlan pl;
  if ((st = plan_group(cache, params, beams, &pl)) != LOCKS_OK) return st;
  *bytes = pl.total;
  return LOCKS_OK;
}

locks_status_t locksgen_attend(const locks_cache_t* cache, const locks_params_t* params, int32_t beams,
                               const int32_t* shared_pages, const void* q, void* out, float* lse, void* ws,
                               size_t ws_bytes, void* stream) {
  locks_status_t st = check_cache(cache, true);
  if (st != LOCKS_OK) return st;
  if ((st = check_params(cache, params)) != LOCKS_OK) return st;
  if ((st = check_beams(cache, beams)) != LOCKS_OK) return st;
  if (!shared_pages || !q || !out || (reinterpret_cast<uintptr_t>(q) & 15)) return LOCKS_ERR_INVALID_ARG;
  GroupPlan pl;
  if ((st = plan_group(cache, params, beams, &pl)) != LOCKS_OK) return st;
  if ((st = check_ws(ws, ws_bytes, pl.total)) != LOCKS_OK) return st;
  GroupArgs a;
  a.q = static_cast<const uint16_t*>(q);
  a.blocks = static_cast<const uint8_t*>(cache->k_pool);
  a.block_table = cache->block_table;
  a.seq_lens = cache->seq_lens;
  a.shared_pages = shared_pages;
  a.out = static_cast<uint16_t*>(out);
  a.lse = lse;
  a.offsets = at<uint32_t>(ws, pl.off_line);
  a.part_o = at<float>(ws, pl.off_o);
  a.part_ml = at<float2>(ws, pl.off_ml);
  a.err = at<int>(ws, 0);
  a.batch = cache->batch;
  a.beams = beams;
  a.num_kv_heads = cache->num_kv_heads;
  a.group = params->num_q_heads / cache->num_kv_heads;
  a.max_pages = cache->max_pages;
  a.pages_total = cache->pages_total;
  a.page_size = cache->page_size;
  a.n_blocks = pl.n_blocks;
  a.n_ctas = pl.n_ctas;
  a.scale_log2 = scale_of(params) * kLog2e;
  a.q4 = is_q4(cache) ? 1 : 0;
  CUtensorMap tk, tv;
  std::memset(&tk, 0, sizeof(tk));
  std::memset(&tv, 0, sizeof(tv));
  if (!is_q4(cache) && (!encode_pool(&tk, cache->k_pool, cache) || !encode_pool(&tv, cache->v_pool, cache)))
    return LOCKS_ERR_CUDA;
  return cuda_status(launch_group_attend(a, tk, tv, static_cast<cudaStream_t>(stream)));
}

}  // extern "C"
