// Choosing the beams' continuations: of beams x vocabulary candidates
//   score[w] + x_v - ln sum_u exp(x_u)
// the `keep` largest of each request.
//
// One pass over the logits.  The best of a request are among the best `keep` of each
// row, whose order is that of the logits alone; so a CTA takes a part of a row into
// registers, sums its exponentials against the part's own maximum and writes its best
// `keep`, in order.  A second kernel, one CTA per request, adds up the sums, and merges
// the sorted lists of all parts of all beams.
//
// A part's best: candidates are compared as (logit, lower token) in one 64-bit number, so
// that no two are equal.  The threads form kGroups groups; the keep-th largest of the
// groups' largest is a lower bound T of the keep-th largest of all, and those at least T
// lie in `keep` groups, so that their list has a bound whatever the logits; its members
// are ranked against each other.
//
// What bounds it: the logits' bytes, for few rows the latency of the two launches.
#include "common.cuh"
#include "gen.h"

namespace locks {

namespace {

constexpr int kThreads = 256;
// Members at least T, at most: `keep` groups of LANES threads with 32 logits each; up to 16
// kept the groups are of four threads, which makes T four times cheaper to find.
constexpr int kFewKept = 16;
constexpr int kPartList = kFewKept * 4 * kSelectPart / kThreads;
static_assert(kPartList >= LOCKSGEN_MAX_KEEP * kSelectPart / kThreads, "the list holds both");
static_assert(kThreads >= LOCKSGEN_MAX_KEEP, "a group per continuation");

__device__ __forceinline__ bool is_live(float score, int ended) { return score > -INFINITY && score < INFINITY && !ended; }

// (logit, lower token), larger is better; zero below every candidate.
__device__ __forceinline__ unsigned long long part_key(float x, int token) {
  return ((unsigned long long)orderable_key(x) << 32) | (0xffffffffu - (uint32_t)token);
}

__device__ __forceinline__ unsigned long long shfl_max(unsigned long long v, int lanes) {
  for (int o = lanes / 2; o; o >>= 1) {
    const unsigned long long w = __shfl_xor_sync(0xffffffffu, v, o);
    v = w > v ? w : v;
  }
  return v;
}

// exp(d): log2(e) in two parts, so that the exponent is rounded once.
__device__ __forceinline__ float exp_of(float d) { return fast_exp2(fmaf(d, 1.44269502f, d * 1.92596303e-8f)); }

template <typename T>
__device__ __forceinline__ float logit_of(const T* row, int i);
template <>
__device__ __forceinline__ float logit_of<uint16_t>(const uint16_t* row, int i) {
  return __uint_as_float((uint32_t)__ldg(row + i) << 16);
}
template <>
__device__ __forceinline__ float logit_of<float>(const float* row, int i) {
  return __ldg(row + i);
}

// Grid (parts, rows).
template <typename T, int LANES>
__global__ void __launch_bounds__(kThreads) part_kernel(const SelectArgs a) {
  constexpr int kGroups = kThreads / LANES;
  constexpr int kVec = 16 / sizeof(T);                    // elements of a 16-byte load
  constexpr int kLoads = kSelectPart / kThreads / kVec;   // of a thread
  constexpr int kMine = kLoads * kVec;
  __shared__ unsigned long long top[kGroups], list[kPartList], thresh;
  __shared__ float sm_m[kThreads / 32], sm_l[kThreads / 32];
  __shared__ int n_list;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int part = blockIdx.x, row = blockIdx.y;
  pdl_wait();
  if (!is_live(__ldg(a.scores + row), a.ended ? __ldg(a.ended + row) : 0)) {
    pdl_launch_dependents();
    return;
  }
  if (tid == 0) n_list = 0;
  // 16-byte loads of the aligned pieces that cover the row; the pieces at its ends
  // element by element
  const T* base = reinterpret_cast<const T*>(a.logits) + (size_t)row * a.row_stride;
  const int before = (int)((reinterpret_cast<uintptr_t>(base) & 15) / sizeof(T));
  const int first = part * kSelectPart - before;
  float x[kMine];
#pragma unroll
  for (int k = 0; k < kLoads; ++k) {
    const int i = first + (k * kThreads + tid) * kVec;
    if (i >= 0 && i + kVec <= a.vocab) {
      const uint4 v = __ldg(reinterpret_cast<const uint4*>(base + i));
      const uint32_t w[4] = {v.x, v.y, v.z, v.w};
      if constexpr (sizeof(T) == 2) {
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          x[k * kVec + 2 * e] = __uint_as_float(w[e] << 16);
          x[k * kVec + 2 * e + 1] = __uint_as_float(w[e] & 0xffff0000u);
        }
      } else {
#pragma unroll
        for (int e = 0; e < 4; ++e) x[k * kVec + e] = __uint_as_float(w[e]);
      }
    } else {
#pragma unroll
      for (int e = 0; e < kVec; ++e) x[k * kVec + e] = i + e >= 0 && i + e < a.vocab ? logit_of(base, i + e) : -INFINITY;
    }
  }
  pdl_launch_dependents();
  // maximum (a NaN shows in the sum), and this thread's best
  float m = -INFINITY;
#pragma unroll
  for (int j = 0; j < kMine; ++j) m = fmaxf(m, x[j]);
  float mine = m;
  m = warp_max(m);
  if (lane == 0) sm_m[warp] = m;
  unsigned long long best = 0;
  if (mine > -INFINITY) {
    int at = 0;
#pragma unroll
    for (int j = kMine - 1; j >= 0; --j)
      if (x[j] == mine) at = j;
    best = part_key(mine, first + ((at / kVec) * kThreads + tid) * kVec + at % kVec);
  }
  best = shfl_max(best, LANES);
  if (tid % LANES == 0) top[tid / LANES] = best;
  __syncthreads();
  m = sm_m[0];
#pragma unroll
  for (int w = 1; w < kThreads / 32; ++w) m = fmaxf(m, sm_m[w]);
  float l = 0.f;
  // (-infinity less itself is no number; all others are)
  const float ref = m == -INFINITY ? 0.f : m;
#pragma unroll
  for (int j = 0; j < kMine; ++j) l += exp_of(x[j] - ref);
  l = warp_sum(l);
  if (lane == 0) sm_l[warp] = l;
  // the keep-th largest of the groups' best
  for (int i = tid; i < kGroups; i += kThreads) {
    const unsigned long long v = top[i];
    int rank = 0;
#pragma unroll 8
    for (int j = 0; j < kGroups; ++j) rank += top[j] > v || (top[j] == v && j < i);  // empty groups are equal
    if (rank == a.keep - 1) thresh = v;
  }
  __syncthreads();
  const unsigned long long t = thresh;
  if (mine > -INFINITY && (uint32_t)(t >> 32) <= orderable_key(mine)) {
#pragma unroll
    for (int j = 0; j < kMine; ++j) {
      const unsigned long long key = part_key(x[j], first + ((j / kVec) * kThreads + tid) * kVec + j % kVec);
      if (x[j] > -INFINITY && key >= t) list[atomicAdd(&n_list, 1)] = key;
    }
  }
  __syncthreads();
  const int n = n_list;
  const size_t slot = (size_t)row * a.n_parts + part;
  uint2* out = a.lists + slot * a.keep;
  for (int i = tid; i < n; i += kThreads) {
    const unsigned long long v = list[i];
    int rank = 0;
#pragma unroll 4
    for (int j = 0; j < n; ++j) rank += list[j] > v;
    if (rank < a.keep) out[rank] = make_uint2((uint32_t)(v >> 32), 0xffffffffu - (uint32_t)v);
  }
  if (tid == 0) {
    float sum = 0.f;
#pragma unroll
    for (int w = 0; w < kThreads / 32; ++w) sum += sm_l[w];
    a.parts[slot] = make_float4(m, sum, __int_as_float(min(n, a.keep)), 0.f);
  }
}

// The logit of a part_key's upper half.
__device__ __forceinline__ float key_logit(uint32_t k) {
  return __uint_as_float(k & 0x80000000u ? k ^ 0x80000000u : ~k);
}
// Monotone map double -> uint64; -0 maps like +0.
__device__ __forceinline__ unsigned long long orderable(double d) {
  const long long b = __double_as_longlong(d + 0.0);
  return b < 0 ? ~(unsigned long long)b : (unsigned long long)b | 0x8000000000000000ull;
}

// One CTA per request.  Lists: (beam, part), list i is thread i % kThreads'.  In each of `keep`
// rounds the threads' best heads are compared and the winner's list moves on.
struct Head {
  unsigned long long score;  // orderable, 0 for none
  unsigned long long flat;   // beam * vocab + token
};
__device__ __forceinline__ bool better(const Head& x, const Head& y) {
  return x.score > y.score || (x.score == y.score && x.flat < y.flat);
}

__global__ void __launch_bounds__(kThreads) merge_kernel(const SelectArgs a) {
  extern __shared__ uint8_t taken[];  // entries used of each list
  __shared__ double lse[LOCKSGEN_MAX_BEAMS];
  __shared__ float score[LOCKSGEN_MAX_BEAMS];
  __shared__ int state[LOCKSGEN_MAX_BEAMS];  // 0: no continuation, 1: live, 2: ended
  __shared__ Head heads[2][kThreads / 32];
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, W = a.beams, b = blockIdx.x;
  const int lists = W * a.n_parts;
  for (int i = tid; i < lists; i += kThreads) taken[i] = 0;
  pdl_wait();
  pdl_launch_dependents();
  for (int w = warp; w < W; w += kThreads / 32) {
    const size_t row = (size_t)b * W + w;
    const float s = a.scores[row];  // (these two may be written in place further down)
    const int over = a.ended ? a.ended[row] : 0;
    int st = !(s > -INFINITY) || !(s < INFINITY) ? 0 : over ? 2 : 1;
    bool bad = !(s < INFINITY);  // a NaN too
    if (st == 1) {
      float m = -INFINITY;
      for (int i = lane; i < a.n_parts; i += 32) m = fmaxf(m, a.parts[row * a.n_parts + i].x);
      m = warp_max(m);
      double sum = 0.0;
      for (int i = lane; i < a.n_parts; i += 32) {
        const float4 p = a.parts[row * a.n_parts + i];
        sum += p.x == -INFINITY ? (double)p.y : (double)p.y * exp_of(p.x - m);
      }
#pragma unroll
      for (int o = 16; o; o >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
      if (!(sum < INFINITY) || m == INFINITY) bad = true;
      if (m == -INFINITY || bad) st = 0;
      if (lane == 0) lse[w] = st ? (double)m + log(sum) : 0.0;
    }
    if (lane == 0) {
      if (bad) set_error(a.err, LOCKSGEN_DEVERR_LOGITS);
      score[w] = s;
      state[w] = st;
    }
  }
  __syncthreads();
  auto head_of = [&](int i) {
    Head h = {0, ~0ull};
    const int w = i / a.n_parts, part = i % a.n_parts, at = taken[i];
    if (state[w] == 2) {
      if (part == 0 && at == 0) h = {orderable((double)score[w]), (unsigned long long)w * a.vocab + a.end_token};
    } else if (state[w] == 1) {
      const size_t slot = ((size_t)b * W + w) * a.n_parts + part;
      if (at < __float_as_int(a.parts[slot].z)) {
        const uint2 e = a.lists[slot * a.keep + at];
        const double d = (double)score[w] + ((double)key_logit(e.x) - lse[w]);
        if (d > -INFINITY) h = {orderable(d), (unsigned long long)w * a.vocab + e.y};
      }
    }
    return h;
  };
  Head mine = {0, ~0ull};
  int my_list = -1;
  auto refresh = [&] {
    mine = {0, ~0ull};
    for (int i = tid; i < lists; i += kThreads) {
      const Head h = head_of(i);
      if (better(h, mine)) mine = h, my_list = i;
    }
  };
  refresh();
  for (int k = 0; k < a.keep; ++k) {
    Head h = mine;
#pragma unroll
    for (int o = 16; o; o >>= 1) {
      Head y;
      y.score = __shfl_xor_sync(0xffffffffu, h.score, o);
      y.flat = __shfl_xor_sync(0xffffffffu, h.flat, o);
      if (better(y, h)) h = y;
    }
    if (lane == 0) heads[k & 1][warp] = h;
    __syncthreads();
    h = heads[k & 1][0];
#pragma unroll
    for (int w = 1; w < kThreads / 32; ++w)
      if (better(heads[k & 1][w], h)) h = heads[k & 1][w];
    const size_t at = (size_t)b * a.keep + k;
    if (h.score == 0) {  // nothing is left
      if (tid == 0) {
        a.out_scores[at] = -INFINITY;
        a.out_parents[at] = a.out_tokens[at] = -1;
        if (a.out_ended) a.out_ended[at] = 0;
      }
      continue;
    }
    if (mine.score == h.score && mine.flat == h.flat) {
      const int w = (int)(h.flat / a.vocab), token = (int)(h.flat % a.vocab);
      const unsigned long long bits = h.score >> 63 ? h.score & 0x7fffffffffffffffull : ~h.score;
      a.out_scores[at] = (float)__longlong_as_double((long long)bits);
      a.out_parents[at] = w;
      a.out_tokens[at] = token;
      if (a.out_ended) a.out_ended[at] = state[w] == 2 || token == a.end_token;
      ++taken[my_list];
      refresh();
    }
  }
}

template <typename T>
cudaError_t launch_parts(const SelectArgs& a, cudaStream_t s) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(a.n_parts, a.batch * a.beams, 1);
  cfg.blockDim = dim3(kThreads, 1, 1);
  cfg.stream = s;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, a.keep <= kFewKept ? part_kernel<T, 4> : part_kernel<T, 1>, a);
}

}  // namespace

cudaError_t launch_select(const SelectArgs& a, bool f32, cudaStream_t s) {
  const cudaError_t e = f32 ? launch_parts<float>(a, s) : launch_parts<uint16_t>(a, s);
  if (e != cudaSuccess) return e;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(a.batch, 1, 1);
  cfg.blockDim = dim3(kThreads, 1, 1);
  cfg.dynamicSmemBytes = (size_t)a.beams * a.n_parts;
  cfg.stream = s;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, merge_kernel, a);
}

}  // namespace locks
