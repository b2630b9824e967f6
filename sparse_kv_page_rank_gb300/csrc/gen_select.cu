// Choosing the beams' continuations: of beams x vocabulary candidates
//   score[w] + x_v - ln sum_u exp(x_u)
// the `keep` largest of each request.
//
// One pass over the logits.  The best of a request are among the best `keep` of each
// row, whose order is that of the logits alone.  A CTA goes through a part of a row,
// a chunk in registers while the next one is under way; every thread sums exponentials
// against its own maximum so far, and the CTA keeps a short list of what may be among the
// part's best.  A second kernel, one CTA per request, adds up the sums and chooses among
// the lists of all parts of all beams.
//
// Both choose in the same way: of the groups' (or threads') best the keep-th largest is a lower
// bound T of the keep-th largest of all, and the few that reach T are ranked
// against each other.  In a part T comes from the first chunk, later ones add what
// exceeds it, and no chunk waits for another thread.  Equal or rising numbers can make the members many,
// however; where their place does not suffice, the part is gone through again, comparing (logit,
// lower token) as one 64-bit number, no two of which are equal, against thread by thread bests,
// which bounds them for any logits; and the merge takes the best of the heads of its
// sorted lists, `keep` times.
//
// What bounds it: the logits' bytes and one exponential each; for few rows the latency of
// the two launches.  Measured (floor by bytes), in a graph, on inputs that change and
// exceed L2: 32 requests of 4 beams, 128,256 bf16 logits, some ended, 16.5 us (4.3); 24 of 8, 100,003
// float32 logits, 16 kept, 24.4 us (11.3); one request of 4 beams, 32,000 logits 7.1 us.  One kernel, whose
// last CTA of a request merges, took 17.9, 26.2 and 8.7 where two took 16.5, 25.1 and 7.2.
#include "common.cuh"
#include "gen.h"

namespace locks {

namespace {

constexpr int kThreads = 256;
// T of a part's first chunk: from 32 groups of eight threads, a lane each, or from all threads.
constexpr int kFewKept = 16;
constexpr int kGroupLanes = 8;
static_assert(kThreads / kGroupLanes == 32, "a lane per group");
static_assert(kThreads >= LOCKSGEN_MAX_KEEP, "a thread per continuation");
// The list of a part: members that chunks may add to, and beside them those of the slow
// way, `keep` threads with all their logits.
constexpr int kShort = 256;
constexpr int kTidy = 8;  // so many more than `keep` are cut back after chunks 1, 3, 7, ..., which raises T

__device__ __forceinline__ bool is_live(float score, int ended) { return score > -INFINITY && score < INFINITY && !ended; }

// (logit, lower token), larger is better; zero below every candidate.
__device__ __forceinline__ unsigned long long part_key(float x, int token) {
  return ((unsigned long long)orderable_key(x) << 32) | (0xffffffffu - (uint32_t)token);
}

// The logit of a part_key's upper half.
__device__ __forceinline__ float key_logit(uint32_t k) {
  return __uint_as_float(k & 0x80000000u ? k ^ 0x80000000u : ~k);
}
// The key of the next larger number.
__device__ __forceinline__ uint32_t above(uint32_t k) { return k + 1 == 0x7fffffffu ? 0x80000000u : k + 1; }

__device__ __forceinline__ float exp_of(float d) { return fast_exp2(d * kLog2e); }

template <typename T, int LOADS>
struct Chunk {
  static constexpr int kVec = 16 / sizeof(T);  // elements of a 16-byte load
  static constexpr int kMine = LOADS * kVec;   // of a thread
  static constexpr int kSize = kThreads * kMine;
  uint4 raw[LOADS];
  // 16-byte loads of the aligned pieces that cover the row, which begins at element
  // -first of the chunk; the pieces at its ends element by element
  __device__ __forceinline__ void load(const T* base, int first, int vocab) {
    if (first >= 0 && first + kSize <= vocab) {
      const uint4* at = reinterpret_cast<const uint4*>(base + first) + threadIdx.x;
#pragma unroll
      for (int k = 0; k < LOADS; ++k) raw[k] = at[k * kThreads];
      return;
    }
#pragma unroll
    for (int k = 0; k < LOADS; ++k) {
      const int i = first + (k * kThreads + threadIdx.x) * kVec;
      if (i >= 0 && i + kVec <= vocab) {
        raw[k] = *reinterpret_cast<const uint4*>(base + i);
      } else {
        uint32_t w[4];
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          if constexpr (sizeof(T) == 2) {
            const int j = i + 2 * e;
            const uint32_t lo = j >= 0 && j < vocab ? reinterpret_cast<const uint16_t*>(base)[j] : 0xff80u;
            const uint32_t hi = j + 1 >= 0 && j + 1 < vocab ? reinterpret_cast<const uint16_t*>(base)[j + 1] : 0xff80u;
            w[e] = lo | hi << 16;
          } else {
            w[e] = i + e >= 0 && i + e < vocab ? reinterpret_cast<const uint32_t*>(base)[i + e] : 0xff800000u;
          }
        }
        raw[k] = make_uint4(w[0], w[1], w[2], w[3]);
      }
    }
  }
  __device__ __forceinline__ void unpack(float (&x)[kMine]) const {
#pragma unroll
    for (int k = 0; k < LOADS; ++k) {
      const uint32_t w[4] = {raw[k].x, raw[k].y, raw[k].z, raw[k].w};
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        if constexpr (sizeof(T) == 2) {
          x[k * kVec + 2 * e] = __uint_as_float(w[e] << 16);
          x[k * kVec + 2 * e + 1] = __uint_as_float(w[e] & 0xffff0000u);
        } else {
          x[k * kVec + e] = __uint_as_float(w[e]);
        }
      }
    }
  }
  __device__ __forceinline__ static float logit(const T* base, int i) {
    if constexpr (sizeof(T) == 2) return __uint_as_float((uint32_t)reinterpret_cast<const uint16_t*>(base)[i] << 16);
    else return reinterpret_cast<const float*>(base)[i];
  }
  __device__ __forceinline__ static int token(int first, int j) {
    return first + ((j / kVec) * kThreads + threadIdx.x) * kVec + j % kVec;
  }
};

// The largest number below that of key k (-infinity below itself, too).
__device__ __forceinline__ float below(uint32_t k) {
  if (k <= 0x007fffffu) return -INFINITY;
  --k;
  if (k == 0x7fffffffu) --k;  // no number has this key
  return key_logit(k);
}

// Grid (parts, rows).
template <typename T, int LOADS>
__global__ void __launch_bounds__(kThreads, kSelectCtas) part_kernel(const SelectArgs a) {
  using C = Chunk<T, LOADS>;
  constexpr int kMine = C::kMine;
  static_assert(kMine <= 32, "a bit per logit");
  __shared__ unsigned long long list[kShort + LOCKSGEN_MAX_KEEP * kMine], best_of[kThreads], tidy[LOCKSGEN_MAX_KEEP], thresh;
  __shared__ float sm_m[kThreads / 32], sm_l[kThreads / 32], first_t;
  __shared__ uint32_t top[kThreads];
  __shared__ int n_list;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int part = blockIdx.x, row = blockIdx.y;
  pdl_wait();
  const T* base = reinterpret_cast<const T*>(a.logits) + (size_t)row * a.row_stride;
  const int before = (int)((reinterpret_cast<uintptr_t>(base) & 15) / sizeof(T));
  const int begin = part * a.chunks * C::kSize - before;
  C next;
  next.load(base, begin, a.vocab);  // under way while the row's state is looked up
  if (!is_live(a.scores[row], a.ended ? a.ended[row] : 0)) {  // (plain loads: the choice before may have written them)
    pdl_launch_dependents();
    return;
  }
  if (tid == 0) n_list = 0;
  float m = -INFINITY, l = 0.f;  // this thread's maximum and sum
  float t = -INFINITY;           // what exceeds it joins the list
  // the best `keep` of the list's n members, in order; the list's size
  auto cut = [&](int n) {
    for (int i = tid; i < n; i += kThreads) {
      const unsigned long long v = list[i];
      int rank = 0;
#pragma unroll 4
      for (int j = 0; j < n; ++j) rank += list[j] > v;
      if (rank < a.keep) tidy[rank] = v;
    }
    __syncthreads();
    n = min(n, a.keep);
    if (tid < n) list[tid] = tidy[tid];
    if (tid == 0) n_list = n;
    __syncthreads();
    return n;
  };
  for (int c = 0; c < a.chunks; ++c) {
    float x[kMine];
    next.unpack(x);
    const int here = begin + c * C::kSize;
    const bool last = c + 1 == a.chunks;
    if (!last) next.load(base, here + C::kSize, a.vocab);  // (past the row's end: -infinity, nothing is read)
    else pdl_launch_dependents();
    float mine = -INFINITY;  // (a NaN shows in the sum)
#pragma unroll
    for (int j = 0; j < kMine; ++j) mine = fmaxf(mine, x[j]);
    if (c == 0) {
      if (a.keep <= kFewKept) {
        float g = mine;
#pragma unroll
        for (int o = 1; o < kGroupLanes; o *= 2) g = fmaxf(g, __shfl_xor_sync(0xffffffffu, g, o));
        if (lane % kGroupLanes == 0) top[tid / kGroupLanes] = orderable_key(g);
        __syncthreads();
        if (warp == 0) {
          const uint32_t v = top[lane];
          int rank = 0;
#pragma unroll
          for (int j = 0; j < 32; ++j) {
            const uint32_t w = __shfl_sync(0xffffffffu, v, j);
            rank += w > v || (w == v && j < lane);
          }
          if (rank == a.keep - 1) first_t = below(v);
        }
      } else {
        top[tid] = orderable_key(mine);
        __syncthreads();
        if (warp == 0) {
          // halving until about `keep` threads reach T
          uint32_t v[kThreads / 32];
#pragma unroll
          for (int i = 0; i < kThreads / 32; ++i) v[i] = top[32 * i + lane];
          uint32_t lo = 0, hi = 0xffffffffu;  // at least `keep` reach lo
          while (lo < hi) {
            const uint32_t mid = lo + (hi - lo) / 2 + 1;
            int count = 0;
#pragma unroll
            for (int i = 0; i < kThreads / 32; ++i) count += __popc(__ballot_sync(0xffffffffu, v[i] >= mid));
            if (count >= a.keep) lo = mid;
            else hi = mid - 1;
            if (count >= a.keep && count <= a.keep + 4) break;
          }
          if (lane == 0) first_t = below(lo);
        }
      }
    }
    {  // (the first chunk's while one warp looks for T)
      const float was = m;
      m = fmaxf(m, mine);
      const float ref = m == -INFINITY ? 0.f : m;  // (-infinity less itself is no number)
      const uint64_t less = f32x2(-ref, -ref), factor = f32x2(kLog2e, kLog2e);
      uint64_t sum = f32x2(0.f, 0.f);
#pragma unroll
      for (int j = 0; j < kMine; j += 2) {
        float e0, e1;
        unpack_f32x2(mul_f32x2(add_f32x2(f32x2(x[j], x[j + 1]), less), factor), e0, e1);
        sum = add_f32x2(sum, f32x2(fast_exp2(e0), fast_exp2(e1)));
      }
      float s0, s1;
      unpack_f32x2(sum, s0, s1);
      l = c == 0 ? s0 + s1 : fmaf(l, exp_of(was - ref), s0 + s1);
    }
    if (c == 0) {
      __syncthreads();
      t = first_t;
    }
    if (mine > t) {
      uint32_t mask = 0;
#pragma unroll
      for (int j = 0; j < kMine; ++j)
        if (x[j] > t) mask |= 1u << j;
      for (; mask; mask &= mask - 1) {
        const int i = C::token(here, __ffs(mask) - 1);
        const int at = atomicAdd(&n_list, 1);
        if (at < kShort) list[at] = part_key(C::logit(base, i), i);
      }
    }
    if (c == 0) {
      // `keep` members reach T (unless T is -infinity), and what is equal to it in later chunks
      // comes after them: from here on T itself must be exceeded.
      if (t > -INFINITY) t = key_logit(above(orderable_key(t)));
    } else if ((c & (c + 1)) == 0 && !last) {
      __syncthreads();
      const int n = n_list;
      __syncthreads();
      if (n > a.keep + kTidy && n <= kShort && cut(n) == a.keep) t = key_logit((uint32_t)(tidy[a.keep - 1] >> 32));
    }
  }
  __syncthreads();
  int n = n_list;
  if (n > kShort) {
    // again, chunk by chunk, the exact best of each and of those before
    __syncthreads();
    n = 0;
    for (int c = 0; c < a.chunks; ++c) {
      const int here = begin + c * C::kSize;
      next.load(base, here, a.vocab);
      float x[kMine];
      next.unpack(x);
      unsigned long long best = 0;
#pragma unroll
      for (int j = 0; j < kMine; ++j) {
        const unsigned long long key = x[j] > -INFINITY ? part_key(x[j], C::token(here, j)) : 0;
        best = key > best ? key : best;
      }
      best_of[tid] = best;
      if (tid == 0) n_list = n;
      __syncthreads();
      int rank = 0;
#pragma unroll 8
      for (int j = 0; j < kThreads; ++j) rank += best_of[j] > best || (best_of[j] == best && j < tid);  // those without one are equal
      if (rank == a.keep - 1) thresh = best;
      __syncthreads();
      const unsigned long long bound = thresh;
      if (best > 0 && best >= bound) {
#pragma unroll
        for (int j = 0; j < kMine; ++j) {
          const unsigned long long key = x[j] > -INFINITY ? part_key(x[j], C::token(here, j)) : 0;
          if (key > 0 && key >= bound) list[atomicAdd(&n_list, 1)] = key;
        }
      }
      __syncthreads();
      n = n_list;
      n = cut(n);
    }
  }
  const size_t slot = (size_t)row * a.n_parts + part;
  uint2* out = a.lists + slot * a.keep;
  for (int i = tid; i < n; i += kThreads) {
    const unsigned long long v = list[i];
    int rank = 0;
#pragma unroll 4
    for (int j = 0; j < n; ++j) rank += list[j] > v;
    if (rank < a.keep) out[rank] = make_uint2((uint32_t)(v >> 32), 0xffffffffu - (uint32_t)v);
  }
  // the part's maximum and sum
  const float wm = warp_max(m);
  l = warp_sum(m == -INFINITY ? l : l * exp_of(m - wm));
  if (lane == 0) {
    sm_m[warp] = wm;
    sm_l[warp] = l;
  }
  __syncthreads();
  if (tid == 0) {
    float all = -INFINITY, sum = 0.f;
#pragma unroll
    for (int w = 0; w < kThreads / 32; ++w) all = fmaxf(all, sm_m[w]);
#pragma unroll
    for (int w = 0; w < kThreads / 32; ++w) sum += sm_m[w] == -INFINITY ? sm_l[w] : sm_l[w] * exp_of(sm_m[w] - all);
    a.parts[slot] = make_float4(all, sum, __int_as_float(min(n, a.keep)), 0.f);
  }
}

// Monotone map double -> uint64; -0 maps like +0.
__device__ __forceinline__ unsigned long long orderable(double d) {
  const long long b = __double_as_longlong(d + 0.0);
  return b < 0 ? ~(unsigned long long)b : (unsigned long long)b | 0x8000000000000000ull;
}

// The order among equal scores is that of the places, lower is better: the beam, then the logit's
// key turned round, then the token.  Logits that differ may score the same in 64 bits, and a
// part's list has been cut by logit and token, so the merge goes by them too.
struct Head {
  unsigned long long score;  // orderable, 0 for none
  unsigned long long place;
};
constexpr int kTokenBits = 22;
static_assert(LOCKSGEN_MAX_VOCAB <= 1 << kTokenBits && LOCKSGEN_MAX_BEAMS <= 1 << (64 - 32 - kTokenBits), "a place is 64 bits");
__device__ __forceinline__ unsigned long long place_of(int beam, uint32_t key, uint32_t token) {
  return ((unsigned long long)beam << (32 + kTokenBits)) | ((unsigned long long)~key << kTokenBits) | token;
}
__device__ __forceinline__ int beam_of(unsigned long long place) { return (int)(place >> (32 + kTokenBits)); }
__device__ __forceinline__ int token_of(unsigned long long place) { return (int)(place & ((1u << kTokenBits) - 1)); }
constexpr uint32_t kEndedKey = 0xffffffffu;  // an ended beam has one continuation
__device__ __forceinline__ bool better(const Head& x, const Head& y) {
  return x.score > y.score || (x.score == y.score && x.place < y.place);
}
// ln of a sum >= 1 in 64 bits: its exponent's exactly, its fraction's in float32, where it is
// below 0.35 and so off by 2^-25.
__device__ __forceinline__ double ln_of(float sum) {
  int e = (int)(__float_as_uint(sum) >> 23) - 127;
  float f = __uint_as_float((__float_as_uint(sum) & 0x007fffffu) | 0x3f800000u);
  if (f > 1.41421356f) f *= 0.5f, ++e;
  return (double)e * 0.693147180559945309 + (double)logf(f);
}

// One CTA per request.  Its entries, list after list, are dealt to the threads so that a
// thread's lie at different places of their lists.
constexpr int kMergeGroups = 64;  // of four threads: at least as many as are kept
static_assert(kMergeGroups >= LOCKSGEN_MAX_KEEP, "a group per continuation");
constexpr int kMergeList = 512;
constexpr int kEager = 8;  // entries that a thread loads before it knows the sums

__global__ void __launch_bounds__(kThreads) merge_kernel(const SelectArgs a) {
  extern __shared__ uint8_t counts[];  // entries of each list; then the slow way's: entries used
  __shared__ double lse[LOCKSGEN_MAX_BEAMS];
  __shared__ float score[LOCKSGEN_MAX_BEAMS], base[LOCKSGEN_MAX_BEAMS];  // base: score - lse in float32
  __shared__ int state[LOCKSGEN_MAX_BEAMS];  // 0: no continuation, 1: live, 2: ended
  __shared__ __align__(16) uint32_t top[kMergeGroups];
  __shared__ uint32_t thresh;
  __shared__ Head list[kMergeList], heads[2][kThreads / 32];
  __shared__ int n_list;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, W = a.beams, b = blockIdx.x;
  const int lists = W * a.n_parts, entries = lists * a.keep;
  uint8_t* taken = counts + lists;
  if (tid == 0) n_list = 0;
  pdl_wait();
  pdl_launch_dependents();
  // the first entries, under way while the sums are added up (those of lists that hold
  // fewer, or that no part has written, are left aside below)
  const uint2* all = a.lists + (size_t)b * entries;
  const float4* parts = a.parts + (size_t)b * lists;
  auto place = [&](int k) { return k * kThreads + ((tid + 20 * k) & (kThreads - 1)); };
  static_assert((kThreads & (kThreads - 1)) == 0, "a power of two");
  uint2 eager[kEager];
#pragma unroll
  for (int k = 0; k < kEager; ++k) eager[k] = place(k) < entries ? __ldcg(all + place(k)) : make_uint2(0, 0);
  for (int w = warp; w < W; w += kThreads / 32) {
    const size_t row = (size_t)b * W + w;
    const float s = a.scores[row];  // (these two may be written in place further down)
    const int over = a.ended ? a.ended[row] : 0;
    float m = -INFINITY, sum = 0.f;
    for (int i = lane; i < a.n_parts; i += 32) {
      const float4 p = __ldcg(parts + w * a.n_parts + i);
      counts[w * a.n_parts + i] = (uint8_t)__float_as_int(p.z);
      const float was = m;
      m = fmaxf(m, p.x);
      sum = (m == was ? sum : sum * exp_of(was - m)) + (p.x == m || p.x == -INFINITY ? p.y : p.y * exp_of(p.x - m));
    }
    const float top_m = warp_max(m);
    sum = warp_sum(m == top_m || m == -INFINITY ? sum : sum * exp_of(m - top_m));
    if (lane == 0) {
      int st = !(s > -INFINITY) || !(s < INFINITY) ? 0 : over ? 2 : 1;
      bool bad = !(s < INFINITY);  // a NaN too
      if (st == 1) {
        if (!(sum < INFINITY) || top_m == INFINITY) bad = true;
        if (top_m == -INFINITY || bad) st = 0;
        lse[w] = st ? (double)top_m + ln_of(sum) : 0.0;
        base[w] = (float)((double)s - lse[w]);
      }
      if (bad) set_error(a.err, LOCKSGEN_DEVERR_LOGITS);
      score[w] = s;
      state[w] = st;
    }
  }
  __syncthreads();
  // entry e of a live beam's list in float32, and how far it may be off: two roundings,
  // 2^-24 each of the numbers below, taken as 2^-22
  struct Rough {
    float value, error;
  };
  auto rough = [&](int e, const uint2& v) {
    const int l = e / a.keep, w = l / a.n_parts;
    Rough r = {-INFINITY, -1.f};  // no entry
    if (e < entries && state[w] == 1 && e - l * a.keep < counts[l]) {
      r.value = base[w] + key_logit(v.x);
      r.error = 2.4e-7f * (fabsf(base[w]) + fabsf(r.value));
    }
    return r;
  };
  // each thread's best lower bound
  float best = -INFINITY;
  if (tid < W && state[tid] == 2) best = score[tid];
  auto bound = [&](const Rough& r) {
    if (r.error >= 0.f) best = fmaxf(best, r.value - r.error);
  };
  Rough first[kEager];
#pragma unroll
  for (int k = 0; k < kEager; ++k) bound(first[k] = rough(place(k), eager[k]));
  for (int k = kEager; k * kThreads < entries; ++k)
    if (place(k) < entries) bound(rough(place(k), __ldcg(all + place(k))));
  best = fmaxf(best, __shfl_xor_sync(0xffffffffu, best, 1));
  best = fmaxf(best, __shfl_xor_sync(0xffffffffu, best, 2));
  if (tid % 4 == 0) top[tid / 4] = orderable_key(best);
  __syncthreads();
  if (tid < kMergeGroups) {
    const uint32_t v = top[tid];
    int rank = 0;
#pragma unroll
    for (int j = 0; j < kMergeGroups / 4; ++j) {
      const uint4 u = reinterpret_cast<const uint4*>(top)[j];
      const uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
      for (int i = 0; i < 4; ++i) rank += w[i] > v || (w[i] == v && 4 * j + i < tid);
    }
    if (rank == a.keep - 1) thresh = v;
  }
  __syncthreads();
  const float t = key_logit(thresh);  // `keep` continuations are at least this
  auto add = [&](double d, unsigned long long where) {
    const int at = atomicAdd(&n_list, 1);
    if (at < kMergeList) list[at] = {orderable(d), where};
  };
  auto consider = [&](int e, const Rough& r, const uint2& v) {
    if (r.error < 0.f || r.value + r.error < t) return;
    const int w = e / a.keep / a.n_parts;
    const double d = (double)score[w] + ((double)key_logit(v.x) - lse[w]);
    if (d > -INFINITY) add(d, place_of(w, v.x, v.y));
  };
  if (tid < W && state[tid] == 2) add((double)score[tid], place_of(tid, kEndedKey, (uint32_t)a.end_token));
#pragma unroll
  for (int k = 0; k < kEager; ++k) consider(place(k), first[k], eager[k]);
  for (int k = kEager; k * kThreads < entries; ++k)
    if (place(k) < entries) {
      const uint2 v = __ldcg(all + place(k));
      consider(place(k), rough(place(k), v), v);
    }
  __syncthreads();
  const int n = n_list;
  auto put = [&](int k, const Head& h) {
    const size_t at = (size_t)b * a.keep + k;
    const int w = beam_of(h.place), token = token_of(h.place);
    const unsigned long long bits = h.score >> 63 ? h.score & 0x7fffffffffffffffull : ~h.score;
    a.out_scores[at] = (float)__longlong_as_double((long long)bits);
    a.out_parents[at] = w;
    a.out_tokens[at] = token;
    if (a.out_ended) a.out_ended[at] = state[w] == 2 || token == a.end_token;
  };
  auto put_none = [&](int k) {
    const size_t at = (size_t)b * a.keep + k;
    a.out_scores[at] = -INFINITY;
    a.out_parents[at] = a.out_tokens[at] = -1;
    if (a.out_ended) a.out_ended[at] = 0;
  };
  if (n <= kMergeList) {
    for (int i = tid; i < n; i += kThreads) {
      const Head h = list[i];
      int rank = 0;
      for (int j = 0; j < n; ++j) rank += better(list[j], h);
      if (rank < a.keep) put(rank, h);
    }
    for (int k = n + tid; k < a.keep; k += kThreads) put_none(k);
    return;
  }
  // many that are nearly equal: the best of the lists' heads, `keep` times
  for (int i = tid; i < lists; i += kThreads) taken[i] = 0;
  auto head_of = [&](int i) {
    Head h = {0, ~0ull};
    const int w = i / a.n_parts, at = taken[i];
    if (state[w] == 2) {
      if (i % a.n_parts == 0 && at == 0) h = {orderable((double)score[w]), place_of(w, kEndedKey, (uint32_t)a.end_token)};
    } else if (state[w] == 1 && at < counts[i]) {
      const uint2 e = __ldcg(all + (size_t)i * a.keep + at);
      const double d = (double)score[w] + ((double)key_logit(e.x) - lse[w]);
      if (d > -INFINITY) h = {orderable(d), place_of(w, e.x, e.y)};
    }
    return h;
  };
  Head mine = {0, ~0ull};
  int my_list = -1;
  auto refresh = [&] {  // a thread's own lists only
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
      y.place = __shfl_xor_sync(0xffffffffu, h.place, o);
      if (better(y, h)) h = y;
    }
    if (lane == 0) heads[k & 1][warp] = h;
    __syncthreads();
    h = heads[k & 1][0];
#pragma unroll
    for (int w = 1; w < kThreads / 32; ++w)
      if (better(heads[k & 1][w], h)) h = heads[k & 1][w];
    if (h.score == 0) {  // nothing is left
      if (tid == 0) put_none(k);
    } else if (mine.score == h.score && mine.place == h.place) {
      put(k, h);
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
  constexpr int kWide = kSelectChunk / kThreads * sizeof(T) / 16, kNarrow = kSelectSmall / kThreads * sizeof(T) / 16;
  static_assert(Chunk<T, kWide>::kSize == kSelectChunk && Chunk<T, kNarrow>::kSize == kSelectSmall, "the planned sizes");
  return cudaLaunchKernelEx(&cfg, a.small ? part_kernel<T, kNarrow> : part_kernel<T, kWide>, a);
}

}  // namespace

cudaError_t launch_select(const SelectArgs& a, bool f32, cudaStream_t s) {
  const cudaError_t e = f32 ? launch_parts<float>(a, s) : launch_parts<uint16_t>(a, s);
  if (e != cudaSuccess) return e;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(a.batch, 1, 1);
  cfg.blockDim = dim3(kThreads, 1, 1);
  cfg.dynamicSmemBytes = 2 * (size_t)a.beams * a.n_parts;
  cfg.stream = s;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, merge_kernel, a);
}

}  // namespace locks
