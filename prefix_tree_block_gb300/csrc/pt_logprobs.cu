// pt_logprobs.cu -- log probabilities of given tokens under rows of logits,
// with the rows' entropy and most likely tokens, and their gradient.
//
// "cp=1 shared-prefix prefix-tree attention for rollouts" (PR description): a
// group's prompt is encoded once, so its last row of logits is scored against
// the first token of every completion.  A row therefore has any number of
// tokens (row_ptr, index; pt_fold_successors gives both for a tree).
//
// With z = scale * x: LSE = m + ln sum exp(z - m), logp = z[target] - LSE,
// H = -sum p ln p = ln S - sum (z - m) exp(z - m) / S, S = sum exp(z - m); and
// d logits = scale (sum_n g_n 1[target_n] - p (sum_n g_n + dH (ln p + H))).
#include <cooperative_groups.h>
#include <cuda_bf16.h>

#include <algorithm>
#include <atomic>
#include <cfloat>
#include <climits>
#include <cmath>
#include <type_traits>

#include "pt.h"
#include "pt_device.cuh"
#include "pt_internal.h"

namespace pt {
int take_status_logprobs(cudaStream_t s) { return take_status_here(s); }
}  // namespace pt

using namespace pt;
namespace cg = cooperative_groups;

namespace {

constexpr int kMaxTop = 64;
constexpr int kMaxParts = 8;   // CTAs of a row: a cluster
constexpr int kCandidates = 1024;
constexpr int kGroups = 16;      // of a thread's slots

// Entries of the rows: row r has entries [row_ptr[r], row_ptr[r + 1]), or entry
// r; entry n is token index[n], or n.
struct Entries {
  const long long* targets;
  const int* row_ptr;
  const int* index;
  int R, N;
  __device__ __forceinline__ void range(int r, int& e0, int& e1) const {
    e0 = row_ptr ? row_ptr[r] : r;
    e1 = row_ptr ? row_ptr[r + 1] : r + 1;
    if (e0 < 0 || e1 < e0 || e1 > N) {
      record_status(PT_STATUS_INVALID);
      e0 = e1 = 0;
    }
  }
  // The token of an entry, or -1.
  __device__ __forceinline__ int token(int n) const {
    const int t = index ? index[n] : n;
    if ((unsigned)t >= (unsigned)N) {
      record_status(PT_STATUS_INVALID);
      return -1;
    }
    return t;
  }
  // A token's target, or -1.
  __device__ __forceinline__ int target(int t, int V) const {
    const long long x = t < 0 ? -1 : targets[t];
    if (x >= V) {
      record_status(PT_STATUS_INVALID);
      return -1;
    }
    return x < 0 ? -1 : (int)x;
  }
};

template <class E>
struct Type;
template <>
struct Type<float> {
  static constexpr int V = 4;  // of 16 bytes
  static __device__ __forceinline__ float f(float x) { return x; }
};
template <>
struct Type<__nv_bfloat16> {
  static constexpr int V = 8;
  static __device__ __forceinline__ float f(__nv_bfloat16 x) { return __bfloat162float(x); }
};

// The elements of 16 bytes as floats.
__device__ __forceinline__ void unpack(const uint4& v, float (&x)[8]) {
  const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    x[2 * i] = __uint_as_float(w[i] << 16);
    x[2 * i + 1] = __uint_as_float(w[i] & 0xffff0000u);
  }
}
__device__ __forceinline__ void unpack(const uint4& v, float (&x)[4]) {
  x[0] = __uint_as_float(v.x), x[1] = __uint_as_float(v.y), x[2] = __uint_as_float(v.z), x[3] = __uint_as_float(v.w);
}

// A row's elements in slots of 16 aligned bytes: element v sits in slot
// (v + lead) / V; the first and the last slot may hold fewer than V.
template <class E>
struct Row {
  static constexpr int V = Type<E>::V;
  const E* x;
  int n, lead;  // elements; those that slot 0 lacks in front
  __device__ __forceinline__ Row(const E* x_, int n_) : x(x_), n(n_) {
    lead = (int)((reinterpret_cast<uintptr_t>(x_) & 15u) / sizeof(E));
  }
  __device__ __forceinline__ int slots() const { return (n + lead + V - 1) / V; }
  __device__ __forceinline__ bool whole(int s) const { return s * V >= lead && s * V + V <= n + lead; }
  __device__ __forceinline__ uint4 load(int s) const {  // of a whole slot
    return __ldg(reinterpret_cast<const uint4*>(x + ((long long)s * V - lead)));
  }
  __device__ __forceinline__ uint4 pack(int s) const {  // any slot; -inf where there is no element
    if (whole(s)) return load(s);
    uint32_t w[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      if constexpr (sizeof(E) == 4) {
        const int v = s * V - lead + i;
        w[i] = v >= 0 && v < n ? __float_as_uint(x[v]) : 0xff800000u;
      } else {
        const int v = s * V - lead + 2 * i;
        const uint32_t lo = v >= 0 && v < n ? __bfloat16_as_ushort(x[v]) : 0xff80u;
        const uint32_t hi = v + 1 >= 0 && v + 1 < n ? __bfloat16_as_ushort(x[v + 1]) : 0xff80u;
        w[i] = lo | hi << 16;
      }
    }
    return make_uint4(w[0], w[1], w[2], w[3]);
  }
  __device__ __forceinline__ void get(int s, float (&f)[V]) const {
    unpack(pack(s), f);
  }
};

// Order of the alternatives: a larger value first, then the lower index.  NaN
// counts as -inf.  0: nothing.
__device__ __forceinline__ unsigned ordered(float x) {
  const unsigned b = x != x ? 0xff800000u : x == 0.f ? 0u : __float_as_uint(x);  // (-0 equals 0)
  return b >> 31 ? ~b : b | 0x80000000u;
}
__device__ __forceinline__ unsigned long long key_of(float x, int v) {
  return (unsigned long long)ordered(x) << 32 | (0xffffffffu - (unsigned)v);
}
__device__ __forceinline__ float value_of(unsigned long long key) {
  const unsigned o = (unsigned)(key >> 32);
  return __uint_as_float(o >> 31 ? o & 0x7fffffffu : ~o);
}
__device__ __forceinline__ int index_of(unsigned long long key) { return (int)(0xffffffffu - (unsigned)key); }

// Statistics of a softmax in base 2, c1 = scale log2(e): a logit m near the
// largest, and the sums of 2^((x - m) c1) and of (x - m) c1 2^((x - m) c1).
struct Stat {
  float m, s, t;
};
// The sums when every exponent grows by d.  (A sum without weight has no share,
// however far below it was.)
__device__ __forceinline__ void rebase(float& s, float& t, float d) {
  const float f = ex2(d);
  t = f > 0.f ? f * fmaf(d, s, t) : t != t ? t : 0.f;
  s *= f;
}
// Of the warp's lanes below 2 * HALF, in all of them: on the largest m, then summed.
template <int HALF>
__device__ __forceinline__ Stat join_lanes(Stat a, float c1) {
  float m = a.m;
#pragma unroll
  for (int o = HALF; o; o >>= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, o));
  rebase(a.s, a.t, (a.m - (m == -INFINITY ? 0.f : m)) * c1);
#pragma unroll
  for (int o = HALF; o; o >>= 1) {
    a.s += __shfl_xor_sync(0xffffffffu, a.s, o);
    a.t += __shfl_xor_sync(0xffffffffu, a.t, o);
  }
  return Stat{m, a.s, a.t};
}

// Largest of packed pairs of bf16 (NaN gives way), and the same with NaN kept.
__device__ __forceinline__ uint32_t max_bf2(uint32_t a, uint32_t b) {
  uint32_t r;
  asm("max.bf16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
  return r;
}
__device__ __forceinline__ uint32_t max_nan_bf2(uint32_t a, uint32_t b) {
  uint32_t r;
  asm("max.NaN.bf16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
  return r;
}

// The sums of one slot's terms, by differences from m.
template <class E>
__device__ __noinline__ float2 far_terms(uint4 v, float m, float c1) {
  float x[Type<E>::V], s = 0.f, t = 0.f;
  unpack(v, x);
#pragma unroll
  for (int k = 0; k < Type<E>::V; ++k) {
    const float d = (x[k] - m) * c1, e = ex2(d);
    s += e;
    t = fmaf(fmaxf(d, -3.402823466e38f), e, t);
  }
  return make_float2(s, t);
}

struct ScoreArgs {
  const void* x;
  long long stride;  // elements between rows
  int V, lparts, k;  // 2^lparts CTAs a row
  float scale, c1;
  Entries e;
  float* logp;
  float* lse;
  float* H;
  float* top;
  long long* ids;
};

// A warp takes from n listed keys those that reach no less than the k-th largest
// value, by halving, to the list's front; returns their number.  (14000 x 150 with 20
// 65 us, all of the row ranked 126.)
__device__ __noinline__ int prune(unsigned long long* list, int n, int k, unsigned lo) {
  const int lane = threadIdx.x & 31;
  unsigned top = 0;
  for (int i = lane; i < n; i += 32) top = max(top, (unsigned)(list[i] >> 32));
  unsigned hi = __reduce_max_sync(0xffffffffu, top) + 1;
  int c = n;
#pragma unroll 1
  while (hi - lo > 1 && c > k + 8) {
    const unsigned mid = lo + ((hi - lo) >> 1);
    int m = 0;
    for (int i = lane; i < n; i += 32) m += (unsigned)(list[i] >> 32) >= mid;
    m = __reduce_add_sync(0xffffffffu, m);
    if (m >= k)
      lo = mid, c = m;
    else
      hi = mid;
  }
  c = 0;
#pragma unroll 1
  for (int i = lane; i - lane < n; i += 32) {  // (in place: none moves up)
    const unsigned long long key = i < n ? list[i] : 0ull;
    const bool keep = i < n && (unsigned)(key >> 32) >= lo;
    const unsigned kept = __ballot_sync(0xffffffffu, keep);
    if (keep) list[c + __popc(kept & ((1u << lane) - 1u))] = key;
    c += __popc(kept);
    __syncwarp();
  }
  return c;
}

// The alternatives' second look at slots [s0, s1) of a row, where many logits tie and
// the first one listed too many: a thread keeps its largest key (of equal logits
// the first), the bound is the k-th largest of them by halving, and the elements
// that reach it are listed; returns their number, which is above `cap` where few
// threads hold many large ones.  Two passes from L2, where a search for each
// alternative takes k.
template <class E, int ALL>
__device__ __noinline__ int list_again(Row<E> row, int s0, int s1, int k, unsigned long long* list, int cap, int* count) {
  constexpr int V = Type<E>::V;
  const int tid = threadIdx.x;
  auto look = [&](auto use) {  // use(slot, its elements, their largest)
#pragma unroll 1
    for (int s = s0 + tid; s < s1; s += ALL) {
      float y[V];
      row.get(s, y);
      float m = y[0];
#pragma unroll
      for (int i = 1; i < V; ++i) m = fmaxf(m, y[i]);
      use(s, y, m);
    }
  };
  float top = -INFINITY;
  int at = -1;
  look([&](int s, const float (&y)[V], float m) {
    if (at >= 0 && !(m > top)) return;
#pragma unroll
    for (int i = V - 1; i >= 0; --i) {
      const int v = s * V - row.lead + i;
      if (v >= 0 && v < row.n && ordered(y[i]) == ordered(m)) at = v;
    }
    top = fmaxf(top, m);
  });
  const unsigned long long best = at < 0 ? 0ull : key_of(top, at);
  if (tid == 0) *count = 0;
  unsigned long long lo = 0, hi = ~0ull;
#pragma unroll 1
  while (hi - lo > 1) {
    const unsigned long long mid = lo + ((hi - lo) >> 1);
    if (__syncthreads_count(best >= mid) >= k)
      lo = mid;
    else
      hi = mid;
  }
  const float least = value_of(lo);  // (of 0: NaN, which nothing is below)
  look([&](int s, const float (&y)[V], float m) {
    if (m < least) return;
#pragma unroll
    for (int i = 0; i < V; ++i) {
      const int v = s * V - row.lead + i;
      const unsigned long long key = key_of(y[i], v);
      if (v >= 0 && v < row.n && key >= lo) {
        const int x = atomicAdd(count, 1);
        if (x < cap) list[x] = key;
      }
    }
  });
  __syncthreads();
  return *count;
}

// ---------------------------------------------------------------------------
// Scores: one pass over the logits.  A row is one CTA's, or a cluster's that
// shares it where rows are few; a thread takes every NT-th 16 bytes, U of them
// in flight, and keeps its own running maximum and sums, which are joined at
// the end (through shared memory, then the cluster's).  A CTA takes rows one
// after the other, the next one's first loads issued before the joining.
//   RING: long rows, and many of them.  One warp brings the rows by bulk copies
//     into a ring of stages, running ahead across the rows' ends, so that no
//     thread waits for memory and the joining costs no time in which nothing is
//     loaded; one warp looks up the row's tokens (row_ptr, index, target, logit:
//     a chain of latencies); eight compute.  Three such CTAs on an SM.
//   CLERK alone: few rows, shared by clusters; loads into registers.
//   NT = 32, 128: many rows, or short ones; those at once hide their latencies.
//
// The alternatives take one more look at very little.  If every warp has q threads
// whose maxima reach a bound, and all warps together at least k, the bound is no
// higher than the k-th largest element; so it is the least of the warps' q-th
// largest maxima.  A thread also keeps the maxima of groups of U slots (16 bits of
// their order, 16 groups): only the groups that reach the bound are read again
// (from L2), their elements at or above it listed, and the list ranked.  Where
// many more threads reach the bound it is raised by halving, and equal maxima are
// told apart by their first index, so that a row of equal logits lists few of
// them.  CTAs of one warp or four have too few threads to tell that from; a list
// that overflows there is made again with such a bound (1300 x 4096 equal logits
// with 24 51 us, by searches 283, random ones 16; 700 x 30001 with 64 99, 1932, 24).  One that
// overflows all the same (many large elements in few threads) is replaced by k
// searches through the part.
//
// Bound by memory and, in bf16, nearly by issue: per element half an instruction
// each for the maximum, the clamp, the exponent and the two sums, one each to
// unpack and for ex2.  14k x 65536 in bf16 (1.83 GB) 272 us, the copy's rate; with
// loads into registers instead of rings 357, with separate differences, one join of
// all warps' statistics in each of them and no packed arithmetic 474.  One row of
// 131072 5.3 us, 64 rows 7.7, 12 with 20 alternatives.
// ---------------------------------------------------------------------------
constexpr int kStages = 3;  // (four: the same; two: 2% more without alternatives)
// Shared memory of the ring: stages of four slots a thread.
constexpr int ring_bytes(int nt) { return kStages * nt * 4 * 16; }

template <class E, int NT, bool TOP, bool CLERK, bool RING>
__global__ void __launch_bounds__(NT + 32 * (CLERK + RING), RING ? 3 : NT == 32 && TOP ? 24 : 1024 / (NT + 32 * CLERK)) k_score(const ScoreArgs a) {
  constexpr int V = Type<E>::V, U = 4, ALL = NT + 32 * CLERK;  // ALL: without the warp that loads
  constexpr int CAND = NT == 32 ? kCandidates / 2 : kCandidates;  // (a warp's: more CTAs on an SM)
  __shared__ Stat sm_stat[NT / 32];
  __shared__ Stat sm_part;
  __shared__ unsigned sm_most[NT / 32], sm_least[NT / 32];
  __shared__ unsigned long long sm_key[TOP ? kMaxTop : 1], sm_cand[TOP ? CAND : 1], sm_best[TOP ? kMaxTop : 1];
  __shared__ int sm_who[TOP ? CAND : 1];  // groups: thread, and 2^16 times the group
  __shared__ unsigned short sm_group[TOP ? kGroups : 1][TOP ? NT : 1];
  __shared__ int sm_n, sm_w, sm_e0, sm_e1;
  __shared__ uint64_t sm_full[RING ? kStages : 1], sm_empty[RING ? kStages : 1];
  __shared__ volatile int abort_flag;
  extern __shared__ __align__(128) uint8_t sm_ring[];
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const bool reads = tid < NT;
  const auto sync = [&]() {
    if constexpr (RING)
      named_bar_sync(1, ALL);
    else
      __syncthreads();
  };
  static_assert(!(RING && TOP), "the alternatives' barriers are the whole CTA's");
  const auto count = [](bool p) { return __syncthreads_count(p); };
  if constexpr (RING) {
    if (tid == 0) {
      for (int i = 0; i < kStages; ++i) mbar_init(sm_full + i, 1), mbar_init(sm_empty + i, NT / 32);
      abort_flag = 0;
      fence_mbar_init();
    }
    __syncthreads();
  }
  pdl_wait();
  const int part = blockIdx.x & ((1 << a.lparts) - 1), step = gridDim.x >> a.lparts;
  // a row: its slots that are this part's, and of those the whole ones
  struct Span {
    int slots, s0, s1, w0, w1;
  };
  auto row_of = [&](int r) { return Row<E>(static_cast<const E*>(a.x) + (long long)r * a.stride, a.V); };
  auto span_of = [&](const Row<E>& row) {
    Span p;
    p.slots = row.slots();
    p.s0 = (int)((unsigned)p.slots * part >> a.lparts), p.s1 = (int)((unsigned)p.slots * (part + 1) >> a.lparts);  // (up to 2^28 slots)
    p.w0 = max(p.s0, row.whole(0) ? 0 : 1), p.w1 = min(p.s1, row.whole(p.slots - 1) ? p.slots : p.slots - 1);
    return p;
  };
  if constexpr (RING) {
    if (warp == ALL / 32) {
      if (lane == 0) {
        uint32_t n = 0;  // stages filled
        bool ok = true;
#pragma unroll 1
        for (int r = blockIdx.x; ok && r < a.e.R; r += step) {
          const Row<E> row = row_of(r);
          const Span p = span_of(row);
#pragma unroll 1
          for (int s = p.w0; s < p.w1; s += NT * U, ++n) {
            const uint32_t st = n % kStages;
            if (n >= kStages) ok = mbar_wait(sm_empty + st, (n / kStages - 1) & 1, &abort_flag);
            if (!ok) break;
            const uint32_t bytes = min(p.w1 - s, NT * U) * 16;
            mbar_expect_tx(sm_full + st, bytes);
            bulk_load(sm_ring + st * (NT * U * 16), row.x + ((long long)s * V - row.lead), bytes, sm_full + st);
          }
        }
        if (!ok)  // a wait ran out: let the copies in flight land
          for (uint32_t i = 0; i < kStages && i < n; ++i)
            mbar_wait_drain(sm_full + (n - 1 - i) % kStages, ((n - 1 - i) / kStages) & 1, 20000000);
      }
      return;
    }
  }
  uint32_t used = 0;  // RING: stages read
  uint4 v[U];
  auto fetch = [&](const Row<E>& row, int s, int w1) {
    if constexpr (RING) {
      // (a wait that runs out is recorded; the barriers are kept, so that the CTA ends)
      const uint32_t st = used % kStages;
      mbar_wait(sm_full + st, (used / kStages) & 1, &abort_flag);
      const uint4* from = reinterpret_cast<const uint4*>(sm_ring + st * (NT * U * 16)) + tid;
#pragma unroll
      for (int u = 0; u < U; ++u)
        if (s + u * NT < w1) v[u] = from[u * NT];
      ++used;
      __syncwarp();
      if (lane == 0) mbar_arrive(sm_empty + st);
      return;
    }
#pragma unroll
    for (int u = 0; u < U; ++u)
      if (reads && s + u * NT < w1) v[u] = row.load(s + u * NT);
  };
  int r = blockIdx.x >> a.lparts;
  if constexpr (!RING) {
    const Row<E> row = row_of(r);
    const Span p = span_of(row);
    fetch(row, p.w0 + tid, p.w1);
  }
#pragma unroll 1
  for (; r < a.e.R; r += step) {
    const Row<E> row = row_of(r);
    const Span span = span_of(row);
    const int slots = span.slots, s0 = span.s0, s1 = span.s1, w0 = span.w0, w1 = span.w1;
    // the first entries' logits, while the row is read
    int my_tok = -1, my_target = -1;
    float my_x = 0.f;
    const int me = CLERK ? tid - NT : tid;  // the entry (of the first 32, or as many as threads) that is this thread's
    if (part == 0 && (!CLERK || me >= 0)) {
      int e0, e1;
      a.e.range(r, e0, e1);
      if (me < e1 - e0) {
        my_tok = a.e.token(e0 + me);
        my_target = a.e.target(my_tok, a.V);
        if (my_target >= 0) my_x = Type<E>::f(row.x[my_target]);
      }
      if (me == 0) sm_e0 = e0, sm_e1 = e1;
    }
    // A term's exponent is one fused product and difference, x c1 - ref with ref the
    // rounded m c1; what the rounding took is made up for at the end.
    // ref follows the largest logit in steps of 2^8 of the terms' size.
    Stat st = {-INFINITY, 0.f, 0.f};
    float ref = 0.f, next = -INFINITY, own_max = -INFINITY;
    bool plain = true;  // (ref is small enough for that (what it lost is below 1 / 16); else the sums are m's own)
    int first = -1;     // TOP: the slots (from this one on, U of them) that the largest was first seen in
    // Terms that are 0 in any case are raised to `low`, where their exponent is
    // finite: 0 times it stays 0.  It lies so far below m, by 2^13 in the exponent
    // and by several steps of bf16, that no term with a weight is touched.
    float low = -1e4f / a.c1;
    uint32_t low2 = pack_bf16(low, low);
    auto take = [&](const uint4* v, auto count, int at) {  // so many slots from `at` on; their largest
      constexpr int n = decltype(count)::value;
      const uint32_t* w = reinterpret_cast<const uint32_t*>(v);
      float bm;
      if constexpr (sizeof(E) == 2) {
        uint32_t b[4] = {w[0], w[1], w[2], w[3]};
#pragma unroll
        for (int i = 4; i < 4 * n; ++i) b[i & 3] = max_bf2(b[i & 3], w[i]);
        const uint32_t c = max_bf2(max_bf2(b[0], b[1]), max_bf2(b[2], b[3]));
        bm = fmaxf(__uint_as_float(c << 16), __uint_as_float(c & 0xffff0000u));
      } else {
        bm = fmaxf(fmaxf(__uint_as_float(w[0]), __uint_as_float(w[1])), fmaxf(__uint_as_float(w[2]), __uint_as_float(w[3])));
#pragma unroll
        for (int i = 4; i < 4 * n; i += 2) bm = fmax3(bm, __uint_as_float(w[i]), __uint_as_float(w[i + 1]));
      }
      if constexpr (TOP) {
        if (first < 0 || bm > own_max) first = at;
        own_max = fmaxf(own_max, bm);
      }
      if (bm > next) {
        const float old = st.m, old_ref = ref;
        const bool was = plain;
        st.m = bm;
        next = bm + 8.f / a.c1;
        const float base = st.m == -INFINITY ? 0.f : st.m;
        ref = base * a.c1;
        plain = fabsf(ref) < 1048576.f && fabsf(base) < 1e37f;
        if (old != -INFINITY)
          rebase(st.s, st.t, was && plain ? old_ref - ref
                                          : (old - base) * a.c1 - (was ? fmaf(old, a.c1, -old_ref) : 0.f) + (plain ? fmaf(base, a.c1, -ref) : 0.f));
        low = base - fmaxf(1e4f / a.c1, fabsf(base) * 0.03125f);
        low2 = pack_bf16(low, low);
      }
      if (plain) {
        const unsigned long long c2 = f2_splat(a.c1), r2 = f2_splat(-ref);
        unsigned long long s2[2] = {0ull, 0ull}, t2[2] = {0ull, 0ull};
#pragma unroll
        for (int i = 0; i < 4 * n; ++i) {
          unsigned long long x2;
          if constexpr (sizeof(E) == 2) {
            const uint32_t y = max_nan_bf2(w[i], low2);
            x2 = f2_pack(__uint_as_float(y << 16), __uint_as_float(y & 0xffff0000u));
          } else {
            if (i & 1) continue;
            const float x = __uint_as_float(w[i]), y = __uint_as_float(w[i + 1]);
            x2 = f2_pack(x < low ? low : x, y < low ? low : y);
          }
          const unsigned long long d2 = f2_fma(x2, c2, r2);
          float d0, d1;
          f2_unpack(d2, d0, d1);
          const unsigned long long e2 = f2_pack(ex2(d0), ex2(d1));
          s2[(i >> 1) & 1] = f2_add(s2[(i >> 1) & 1], e2);
          t2[(i >> 1) & 1] = f2_fma(d2, e2, t2[(i >> 1) & 1]);
        }
        float x0, x1, y0, y1;
        f2_unpack(f2_add(s2[0], s2[1]), x0, x1);
        f2_unpack(f2_add(t2[0], t2[1]), y0, y1);
        st.s += x0 + x1;
        st.t += y0 + y1;
      } else {  // logits (times scale) of a million and more, infinities: differences first
#pragma unroll
        for (int i = 0; i < n; ++i) {
          const float2 d = far_terms<E>(v[i], st.m == -INFINITY ? 0.f : st.m, a.c1);
          st.s += d.x, st.t += d.y;
        }
      }
      return bm;
    };
    using One = std::integral_constant<int, 1>;
    using All = std::integral_constant<int, U>;
    // whole slots, then the ones at the row's ends
    int chunks = 0;  // rounds of U slots
#pragma unroll 1
    for (int s = w0 + tid; reads && (RING ? s - tid : s) < w1; s += NT * U, ++chunks) {  // (RING: whole warps, for the stages)
      if (RING || s != w0 + tid) fetch(row, s, w1);
      float largest = -INFINITY;
      if (s + (U - 1) * NT < w1) {
        largest = take(v, All{}, s);
      } else {
#pragma unroll
        for (int u = 0; u < U; ++u)
          if (s + u * NT < w1) largest = fmaxf(largest, take(v + u, One{}, s + u * NT));
      }
      if constexpr (TOP) {
        const unsigned short o = (unsigned short)(ordered(largest) >> 16);
        unsigned short& g = sm_group[chunks & (kGroups - 1)][tid];
        g = chunks < kGroups ? o : max(g, o);
      }
    }
    int edge = -1;  // a slot at the row's end that is this thread's
    if (tid == 0 && s0 == 0 && s1 > 0 && !row.whole(0)) edge = 0;
    if (tid == NT - 1 && s1 == slots && s1 > s0 && slots > 1 && !row.whole(slots - 1)) edge = slots - 1;
    if (edge >= 0) {
      const uint4 y = row.pack(edge);
      take(&y, One{}, edge);
    }
    if (!RING && r + step < a.e.R) {
      const Row<E> next_row = row_of(r + step);
      const Span p = span_of(next_row);
      fetch(next_row, p.w0 + tid, p.w1);
    }
    if (plain) rebase(st.s, st.t, -fmaf(st.m == -INFINITY ? 0.f : st.m, a.c1, -ref));
    // the CTA's statistics
    st = join_lanes<16>(st, a.c1);
    if (lane == 0 && reads) sm_stat[warp] = st;
    unsigned mine = 0;  // TOP: this thread's largest logit
    if constexpr (TOP) {
      mine = first >= 0 ? ordered(own_max) : 0u;
      // the warp's largest maximum and its q-th largest
      unsigned rest = mine, most = 0, least = 0;
      const int q = (a.k + NT / 32 - 1) / (NT / 32);
#pragma unroll 1
      for (int i = 0; i < q; ++i) {
        least = __reduce_max_sync(0xffffffffu, rest);
        if (i == 0) most = least;
        if (lane == __ffs(__ballot_sync(0xffffffffu, rest == least)) - 1) rest = 0;
      }
      if (lane == 0 && reads) sm_most[warp] = most, sm_least[warp] = least;
      if (tid == 0) sm_n = sm_w = 0;
      for (int i = tid; i < a.k; i += ALL) sm_best[i] = 0;
    }
    sync();
    if (warp == 0) {
      if constexpr (NT > 32) st = join_lanes<NT <= 128 ? 2 : 8>(lane < NT / 32 ? sm_stat[lane] : Stat{-INFINITY, 0.f, 0.f}, a.c1);
      if (lane == 0) sm_part = st;
    }
    if constexpr (TOP) {
      const int k = a.k;
      unsigned lo = 0xffffffffu, hi = 0;
#pragma unroll
      for (int w = 0; w < NT / 32; ++w) lo = min(lo, sm_least[w]), hi = max(hi, sm_most[w]);
      ++hi;  // (a value's order is below 2^32 - 1)
      int reach = count(mine >= lo);  // threads that reach lo: k at least (with lo = 0 all)
      // (0: a warp without q threads that hold any; fewer than k in all: everything is listed)
      const bool far = lo ? reach > 2 * k + 32 : count(mine > 0) >= k;
#pragma unroll 1
      while (far && hi - lo > 1 && reach > k + 8) {
        const unsigned mid = lo + ((hi - lo) >> 1);
        const int n = count(mine >= mid);
        if (n >= k)
          lo = mid, reach = n;
        else
          hi = mid;
      }
      unsigned long long bound = (unsigned long long)lo << 32;
      unsigned long long best_key = (unsigned long long)mine << 32 | 0xffffffffu;  // (no less than the thread's best)
      if (far && hi - lo == 1 && lo && reach > k + 8) {
        // equal maxima: by the first index that holds it
        unsigned inv = 0;  // ~index: larger for lower ones
        if (mine == lo) {
          int at = INT_MAX;
          if (first == edge) {
            float y[V];
            row.get(edge, y);
#pragma unroll
            for (int i = V - 1; i >= 0; --i) {
              const int v = edge * V - row.lead + i;
              if (v >= 0 && v < a.V && ordered(y[i]) == mine) at = v;
            }
          } else {
#pragma unroll 1
            for (int s = first; s < w1 && s < first + NT * U; s += NT) {
              float y[V];
              row.get(s, y);
#pragma unroll
              for (int i = V - 1; i >= 0; --i)
                if (ordered(y[i]) == mine) at = min(at, s * V - row.lead + i);
            }
          }
          inv = 0xffffffffu - (unsigned)at;
          best_key = (unsigned long long)mine << 32 | inv;
        }
        const int above = count(mine > lo);
        unsigned l = 0, h = 0xffffffffu;
#pragma unroll 1
        while (h - l > 1) {
          const unsigned mid = l + ((h - l) >> 1);
          if (above + count(mine == lo && inv >= mid) >= k)
            l = mid;
          else
            h = mid;
        }
        bound |= l;
      }
      // the groups that hold candidates, and their elements
      if (reads && mine && best_key >= bound) {
        const unsigned reach16 = (unsigned)(bound >> 48);
#pragma unroll 1
        for (int c = 0; c < min(chunks, kGroups); ++c)
          if (sm_group[c][tid] >= reach16) {
            const int at = atomicAdd(&sm_w, 1);
            if (at < CAND) sm_who[at] = tid | c << 16;
          }
      }
      sync();
      const float least = value_of(bound);
      auto put = [&](int s, const uint4& w) {
        float y[V];
        unpack(w, y);
        float top = y[0];
#pragma unroll
        for (int i = 1; i < V; ++i) top = fmaxf(top, y[i]);
        if (top < least || *(volatile int*)&sm_n > CAND) return;  // most slots (a NaN passes on); a list that overflows is no use
#pragma unroll
        for (int i = 0; i < V; ++i) {
          if (y[i] < least) continue;
          const int v = s * V - row.lead + i;
          const unsigned long long key = key_of(y[i], v);
          if (key >= bound && v >= 0 && v < a.V) {
            const int at = atomicAdd(&sm_n, 1);
            if (at < CAND) sm_cand[at] = key;
          }
        }
      };
      // (a group: U slots of every kGroups-th round)
      const int rounds = (w1 - w0 + NT * U - 1) / (NT * U), reps = (rounds + kGroups - 1) / kGroups, listed = sm_w;
      const int all = listed > CAND ? 0 : listed * U * reps;
#pragma unroll 1
      for (int x = tid; x < all; x += ALL) {
        const int y = x / U, i = reps == 1 ? y : y / reps, g = sm_who[i];
        const int s = w0 + (g & 0xffff) + ((g >> 16) + (y - i * reps) * kGroups) * (NT * U) + (x % U) * NT;
        if (s < w1) put(s, row.load(s));
      }
      if (edge >= 0) put(edge, row.pack(edge));
      sync();
      int n = listed <= CAND ? sm_n : CAND + 1;
      if (n > CAND && !far) {
        sync();  // (all have read sm_n)
        n = list_again<E, ALL>(row, s0, s1, k, sm_cand, CAND, &sm_n);
      }
      if (n <= CAND) {
        if constexpr (NT == 32)  // (a row of fewer slots than k, mostly: fewer of them, for the ranking's n^2)
          if (n > 2 * k && n > 45) n = prune(sm_cand, n, k, (unsigned)(bound >> 32));  // (the bound of the first look will do)
#pragma unroll 1
        for (int i = tid; i < n; i += ALL) {
          const unsigned long long key = sm_cand[i];
          int above = 0;
#pragma unroll 4
          for (int j = 0; j < n; ++j) above += sm_cand[j] > key;
          if (above < k) sm_best[above] = key;
        }
      } else {  // k searches
        unsigned long long below = ~0ull;
#pragma unroll 1
        for (int i = 0; i < k; ++i) {
          unsigned long long best = 0;
#pragma unroll 1
          for (int s = s0 + tid; s < s1; s += ALL) {
            float y[V];
            row.get(s, y);
#pragma unroll
            for (int j = 0; j < V; ++j) {
              const int v = s * V - row.lead + j;
              const unsigned long long key = key_of(y[j], v);
              if (v >= 0 && v < a.V && key < below && key > best) best = key;
            }
          }
#pragma unroll
          for (int o = 16; o; o >>= 1) best = max(best, __shfl_xor_sync(0xffffffffu, best, o));
          sync();
          if (lane == 0) sm_cand[warp] = best;
          sync();
          below = 0;
          for (int w = 0; w < ALL / 32; ++w) below = max(below, sm_cand[w]);
          if (tid == 0) sm_best[i] = below;
          if (below == 0) below = 1;  // (no more of them)
        }
      }
      sync();
    }
    if (a.lparts > 0) {  // the cluster's
      cg::cluster_group cluster = cg::this_cluster();
      cluster.sync();
      if (part == 0) {
        if (warp == 0) st = join_lanes<kMaxParts / 2>(lane < 1 << a.lparts ? *cluster.map_shared_rank(&sm_part, lane) : Stat{-INFINITY, 0.f, 0.f}, a.c1);
        if constexpr (TOP) {
          const int n = a.k << a.lparts;  // (at most kMaxParts * kMaxTop)
          for (int i = tid; i < n; i += ALL) sm_cand[i] = cluster.map_shared_rank(&sm_best[0], i / a.k)[i % a.k];
          sync();
          for (int i = tid; i < n; i += ALL) {
            const unsigned long long key = sm_cand[i];
            int above = 0;
#pragma unroll 4
            for (int j = 0; j < n; ++j) above += sm_cand[j] > key;
            if (above < a.k && key) sm_key[above] = key;
          }
        }
      }
      cluster.sync();  // (the others' shared memory has been read)
      if (part) return;
      if (tid == 0) sm_part = st;
    }
    const int e0 = sm_e0, e1 = sm_e1;  // (before the barrier: behind it the next row's may come)
    sync();
    st = sm_part;
    // the row's results
    // (a row without weight is one whose largest logit is -inf; that z is beyond fp32 says nothing about its weights)
    const bool none = st.m == -INFINITY && st.s == st.s;
    const float ln_s = st.m == -INFINITY ? 0.f : logf(st.s);  // (S is at least 1)
    if (tid == 0) {
      const float lse = fminf(fmaxf(st.m * a.scale + ln_s, -FLT_MAX), FLT_MAX);
      a.lse[r] = st.s != st.s ? st.s : none ? -INFINITY : lse;
      if (a.H) a.H[r] = none ? 0.f : ln_s - 0.69314718055994531f * (st.t / st.s);
    }
    // (from m, not from LSE: large logits then lose nothing)
    auto log_p = [&](float x) { return none ? -INFINITY : (x - st.m) * a.scale - ln_s; };
    if constexpr (TOP) {
      const unsigned long long* best = a.lparts > 0 ? sm_key : sm_best;
      for (int i = tid; i < a.k; i += ALL) {
        const unsigned long long key = best[i];
        a.top[(long long)r * a.k + i] = log_p(value_of(key));
        a.ids[(long long)r * a.k + i] = index_of(key);
      }
    }
    auto put_logp = [&](int tok, int target, float x) {
      if (tok >= 0) a.logp[tok] = target < 0 ? 0.f : log_p(x);
    };
    if (me >= 0) put_logp(my_tok, my_target, my_x);
#pragma unroll 1
    for (int n = e0 + (CLERK ? 32 : NT) + tid; n < e1; n += ALL) {
      const int tok = a.e.token(n), target = a.e.target(tok, a.V);
      put_logp(tok, target, target >= 0 ? Type<E>::f(row.x[target]) : 0.f);
    }
    if (r == a.e.R - 1 && a.e.row_ptr) {  // entries of no row
      const int first_e = min(max(a.e.row_ptr[0], 0), a.e.N), end = min(max(a.e.row_ptr[a.e.R], first_e), a.e.N);
      for (int n = tid; n < a.e.N; n += ALL) {
        if (n >= first_e && n < end) n += (end - n + ALL - 1) / ALL * ALL;
        if (n >= a.e.N) break;
        const int tok = a.e.token(n);
        if (tok >= 0) a.logp[tok] = 0.f;
      }
    }
  }
}

struct GradArgs {
  const void* x;
  void* d;
  long long stride, d_stride;
  int V, lparts;
  float scale;
  Entries e;
  const float* g;
  const float* lse;
  const float* H;
  const float* dH;
};

// ---------------------------------------------------------------------------
// Gradient: one pass that reads the logits and writes their gradient, a
// product, an exponential and a product an element; `parts` CTAs a row.  The
// scored tokens get theirs in that pass: a bit for each (hashed) slot says
// whether it holds one, and a slot that does adds the entries' gradients in
// their order before it rounds, so equal targets and any order of the calls
// give the same bits.  A thread holds what it read until it writes, so the
// gradient may take the logits' place.  Its first loads are issued before the
// tokens are looked up.  Bound by memory: 14k x 65536 in bf16 with the entropy's
// part (3.7 GB) 549 us, the copy's rate; 1000 x 50001 in fp32 64 us, 92%.  A gradient
// that starts elsewhere modulo 16 bytes than its logits (VEC false) is stored by
// elements, with one load in flight: 109 us for the latter, 2400 for the former.
// ---------------------------------------------------------------------------
constexpr int kSlotBits = 4096;
// From this |LSE| on, z - LSE has lost too much to LSE's rounding (2^-17 of p there,
// 2^-24 |LSE| in general; all of ln S in a row masked with -1e9), and the row's
// maximum and sum are computed again.  Logits whose LSE is that large come from
// masks and broken scales, so the second look costs ordinary rows nothing.
constexpr float kFarLse = 256.f;

// Adds a slot's scored tokens' gradients, in the entries' order.
template <class E>
__device__ __forceinline__ void add_entries(const GradArgs& a, const Row<E>& row, const unsigned* bits, int e0, int e1,
                                            int s, float (&y)[Type<E>::V]) {
  constexpr int V = Type<E>::V;
  if (!(bits[(s & (kSlotBits - 1)) >> 5] >> (s & 31) & 1u)) return;
#pragma unroll 1
  for (int n = e0; n < e1; ++n) {
    const int tok = a.e.token(n), target = a.e.target(tok, a.V);
    if (target < 0) continue;
    const int i = target + row.lead - s * V;
    if (i < 0 || i >= V) continue;
    const float g = a.g[tok] * a.scale;
#pragma unroll
    for (int k = 0; k < V; ++k)
      if (k == i) y[k] += g;
  }
}

// Stores a slot of the gradient at out, the row's start: whole where its 16 bytes are
// the row's own and aligned, else by elements.
template <class E>
__device__ __forceinline__ void store_slot(E* out, const Row<E>& row, int s, bool whole, const float (&y)[Type<E>::V]) {
  constexpr int V = Type<E>::V;
  if (whole) {
    uint4 w;
    if constexpr (sizeof(E) == 2)
      w = make_uint4(pack_bf16(y[0], y[1]), pack_bf16(y[2], y[3]), pack_bf16(y[4], y[5]), pack_bf16(y[6], y[7]));
    else
      w = make_uint4(__float_as_uint(y[0]), __float_as_uint(y[1]), __float_as_uint(y[2]), __float_as_uint(y[3]));
    *reinterpret_cast<uint4*>(out + ((long long)s * V - row.lead)) = w;
    return;
  }
#pragma unroll
  for (int i = 0; i < V; ++i) {
    const int v = s * V - row.lead + i;
    if (v >= 0 && v < row.n) {
      if constexpr (sizeof(E) == 2)
        out[v] = __float2bfloat16_rn(y[i]);
      else
        out[v] = y[i];
    }
  }
}

// A whole row of k_grad by one CTA, ln p = (x - m) scale - ln S with m and S from the
// row itself (three looks at it).  The other CTAs of the row leave it alone, since
// the gradient may take the logits' place.  Bound by latency: one row of 131072 in bf16
// 90 us (2.5 by all of its CTAs on the near path), 4000 x 65536 379 us (157).
template <class E, int NT, bool ENT, bool VEC>
__device__ __noinline__ void far_row(const GradArgs& a, int r, const unsigned* bits, float* sm, int e0, int e1, float ca,
                                     float cb) {
  constexpr int V = Type<E>::V;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const Row<E> row(static_cast<const E*>(a.x) + (long long)r * a.stride, a.V);
  E* out = static_cast<E*>(a.d) + (long long)r * a.d_stride;
  const int slots = row.slots();
  auto get = [&](int at, float (&y)[V]) {  // (not as read-only memory: the gradient may be written there)
    if (row.whole(at))
      unpack(*reinterpret_cast<const uint4*>(row.x + ((long long)at * V - row.lead)), y);
    else
      row.get(at, y);
  };
  const float c1 = a.scale * 1.4426950408889634f;
  float m = -INFINITY, s = 0.f;
#pragma unroll 1
  for (int at = tid; at < slots; at += NT) {
    float y[V];
    get(at, y);
#pragma unroll
    for (int i = 0; i < V; ++i) m = fmaxf(m, y[i]);
  }
#pragma unroll
  for (int o = 16; o; o >>= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, o));
  __syncthreads();  // (sm has been read)
  if (lane == 0) sm[warp] = m;
  __syncthreads();
#pragma unroll
  for (int w = 0; w < NT / 32; ++w) m = fmaxf(m, sm[w]);
#pragma unroll 1
  for (int at = tid; at < slots; at += NT) {
    float y[V];
    get(at, y);
#pragma unroll
    for (int i = 0; i < V; ++i) s += ex2((y[i] - m) * c1);
  }
#pragma unroll
  for (int o = 16; o; o >>= 1) s += __shfl_xor_sync(0xffffffffu, s, o);
  __syncthreads();
  if (lane == 0) sm[warp] = s;
  __syncthreads();
  s = 0.f;
#pragma unroll
  for (int w = 0; w < NT / 32; ++w) s += sm[w];
  const float ln_s = logf(s);
#pragma unroll 1
  for (int at = tid; at < slots; at += NT) {
    float y[V];
    get(at, y);
#pragma unroll
    for (int i = 0; i < V; ++i) {
      const float l = fmaxf(fmaf(y[i] - m, a.scale, -ln_s), -1000.f);
      y[i] = ex2(l * 1.4426950408889634f) * (ENT ? fmaf(cb, l, ca) : ca);
    }
    add_entries<E>(a, row, bits, e0, e1, at, y);
    store_slot<E>(out, row, at, VEC && row.whole(at), y);
  }
}

template <class E, int NT, bool ENT, bool VEC>
__global__ void __launch_bounds__(NT, 1024 / NT) k_grad(const __grid_constant__ GradArgs a) {
  constexpr int V = Type<E>::V, U = VEC ? 4 : 1;
  __shared__ unsigned bits[kSlotBits / 32];
  __shared__ float sm_g[NT / 32];
  pdl_wait();
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int part = blockIdx.x & ((1 << a.lparts) - 1), r = blockIdx.x >> a.lparts;
  const Row<E> row(static_cast<const E*>(a.x) + (long long)r * a.stride, a.V);
  E* out = static_cast<E*>(a.d) + (long long)r * a.d_stride;
  const int slots = row.slots();
  const int s0 = (int)((long long)slots * part >> a.lparts), s1 = (int)((long long)slots * (part + 1) >> a.lparts);
  uint4 v[U];
  auto fetch = [&](int s) {
#pragma unroll
    for (int u = 0; u < U; ++u)
      if (s + u * NT < s1 && row.whole(s + u * NT)) v[u] = *reinterpret_cast<const uint4*>(row.x + ((long long)(s + u * NT) * V - row.lead));
  };
  fetch(s0 + tid);
  int e0, e1;
  a.e.range(r, e0, e1);
  float lse = a.lse[r];
  const bool far = fabsf(lse) >= kFarLse && lse != -INFINITY;
  const float dh = ENT ? a.dH[r] * a.scale : 0.f, H = ENT ? a.H[r] : 0.f;
  if (lse == -INFINITY) lse = INFINITY;  // a row without a weight: every p is 0
  for (int i = tid; i < kSlotBits / 32; i += NT) bits[i] = 0;
  __syncthreads();
  float sum = 0.f;
#pragma unroll 1
  for (int n = e0 + tid; n < e1; n += NT) {
    const int tok = a.e.token(n), target = a.e.target(tok, a.V);
    if (target < 0) continue;
    sum += a.g[tok];
    const int s = (target + row.lead) / V & (kSlotBits - 1);
    atomicOr(&bits[s >> 5], 1u << (s & 31));
  }
#pragma unroll
  for (int o = 16; o; o >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
  if (lane == 0) sm_g[warp] = sum;
  __syncthreads();
  sum = 0.f;
#pragma unroll
  for (int w = 0; w < NT / 32; ++w) sum += sm_g[w];
  // d = p (ca + cb ln p) + scale * g of the entries
  const float ca = lse != lse ? lse : -(sum * a.scale + dh * H), cb = -dh;
  if (far) {
    if (part == 0) far_row<E, NT, ENT, VEC>(a, r, bits, sm_g, e0, e1, ca, cb);
    return;
  }
  auto one = [&](float x) {
    const float l = fmaxf(fmaf(x, a.scale, -lse), -1000.f);  // ln p (p is 0 from -104 on: its product with ln p too)
    const float p = ex2(l * 1.4426950408889634f);
    return p * (ENT ? fmaf(cb, l, ca) : ca);
  };
  auto entries = [&](int s, float (&y)[V]) { add_entries<E>(a, row, bits, e0, e1, s, y); };
#pragma unroll 1
  for (int s = s0 + tid; s < s1; s += NT * U) {
    if (s != s0 + tid) fetch(s);
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const int at = s + u * NT;
      if (at >= s1) break;
      const bool whole = row.whole(at);
      float y[V];
      if (whole) {
        unpack(v[u], y);
      } else {
#pragma unroll
        for (int i = 0; i < V; ++i) {
          const int e = at * V - row.lead + i;
          y[i] = e >= 0 && e < a.V ? Type<E>::f(row.x[e]) : 0.f;
        }
      }
#pragma unroll
      for (int i = 0; i < V; ++i) y[i] = one(y[i]);
      entries(at, y);
      store_slot<E>(out, row, at, VEC && whole, y);
    }
  }
}

int launch_status(const char* who, cudaError_t e) {
  if (e == cudaSuccess) e = cudaGetLastError();
  if (e != cudaSuccess) {
    set_error("%s: launch failed: %s", who, cudaGetErrorString(e));
    return PT_ERR_CUDA;
  }
  return PT_OK;
}

// Lets a kernel use `bytes` of shared memory, once per device (a bit each).
template <class K>
cudaError_t opt_in_smem(K kernel, size_t bytes, int dev, std::atomic<uint64_t>& opted) {
  if (dev < 64 && (opted.load(std::memory_order_relaxed) >> dev & 1)) return cudaSuccess;
  const cudaError_t e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)bytes);
  if (e == cudaSuccess && dev < 64) opted.fetch_or(1ull << dev, std::memory_order_relaxed);
  return e;
}

// As launch_pdl, with `parts` CTAs a cluster.
template <class K, class A>
cudaError_t launch_cluster(K kernel, unsigned grid, int threads, size_t smem, int parts, cudaStream_t s, const A& a) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(grid);
  cfg.blockDim = dim3(threads);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = s;
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  attr[1].id = cudaLaunchAttributeClusterDimension;
  attr[1].val.clusterDim.x = parts, attr[1].val.clusterDim.y = 1, attr[1].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = parts > 1 ? 2 : 1;
  return cudaLaunchKernelEx(&cfg, kernel, a);
}

// Shared checks of both calls; es: bytes of an element.
pt_status check(const char* who, pt_dtype dtype, int R, int V, int N, int64_t stride, const int32_t* row_ptr, float scale) {
  if (dtype != PT_BF16 && dtype != PT_F32) {
    set_error("%s: unknown dtype %d", who, (int)dtype);
    return PT_ERR_INVALID_ARG;
  }
  if (R < 0 || V < 1 || N < 0) {
    set_error("%s: %d rows of %d logits or %d tokens out of range", who, R, V, N);
    return PT_ERR_INVALID_ARG;
  }
  if (V > 1 << 30 || N > 1 << 30 || R > INT_MAX / kMaxParts) {
    set_error("%s: %d rows of %d logits or %d tokens are more than supported", who, R, V, N);
    return PT_ERR_UNSUPPORTED;
  }
  if (stride < V) {
    set_error("%s: rows %lld elements apart, %d logits", who, (long long)stride, V);
    return PT_ERR_INVALID_ARG;
  }
  if (!row_ptr && N != R) {
    set_error("%s: %d tokens for %d rows without row_ptr", who, N, R);
    return PT_ERR_INVALID_ARG;
  }
  if (!(scale >= 1e-30f && scale <= 1e30f)) {
    set_error("%s: scale = %g, 1e-30 to 1e30 wanted", who, (double)scale);
    return PT_ERR_INVALID_ARG;
  }
  return PT_OK;
}

}  // namespace

extern "C" pt_status pt_token_logprobs(const void* logits, int64_t row_stride, pt_dtype dtype, int32_t R, int32_t V,
                                       const int64_t* targets, const int32_t* row_ptr, const int32_t* index, int32_t N,
                                       float scale, int32_t top_k, float* logp, float* LSE, float* entropy,
                                       float* top_logp, int64_t* top_ids, cudaStream_t stream) {
  static const char* who = "pt_token_logprobs";
  if (pt_status rc = check(who, dtype, R, V, N, row_stride, row_ptr, scale)) return rc;
  if (top_k < 0 || top_k > V) {
    set_error("%s: top_k = %d of %d logits", who, top_k, V);
    return PT_ERR_INVALID_ARG;
  }
  if (top_k > kMaxTop) {
    set_error("%s: top_k = %d, at most %d", who, top_k, kMaxTop);
    return PT_ERR_UNSUPPORTED;
  }
  if (R == 0) {
    if (N > 0) {
      set_error("%s: %d tokens and no rows", who, N);
      return PT_ERR_INVALID_ARG;
    }
    return PT_OK;
  }
  if (!logits || !LSE || (N > 0 && (!targets || !logp)) || (top_k > 0 && (!top_logp || !top_ids))) {
    set_error("%s: a pointer is NULL", who);
    return PT_ERR_INVALID_ARG;
  }
  const int es = dtype == PT_BF16 ? 2 : 4;
  if (reinterpret_cast<uintptr_t>(logits) & (uintptr_t)(es - 1)) {
    set_error("%s: logits are not aligned to their elements", who);
    return PT_ERR_INVALID_ARG;
  }
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess) {
    set_error("%s: no CUDA device", who);
    return PT_ERR_CUDA;
  }
  ScoreArgs a;
  a.x = logits, a.stride = row_stride, a.V = V, a.k = top_k;
  a.scale = scale, a.c1 = scale * 1.4426950408889634f;
  a.e = Entries{reinterpret_cast<const long long*>(targets), row_ptr, index, R, N};
  a.logp = logp, a.lse = LSE, a.H = entropy, a.top = top_logp;
  a.ids = reinterpret_cast<long long*>(top_ids);
  // Which kernel (slots: 16 bytes of a row; us, bf16).
  // Without alternatives: a warp a row where rows are short, or many and not long
  // (30000 x 2048 30 and with rings 140, 15000 x 16384 87 and 113, 4864 x 32768 54
  // and 60; but 1500 x 50001 48 and 31, 4864 x 65536 99 and 100); else a ring, or a
  // cluster a row where rows are few.  With them: CTAs of four warps from four rows
  // an SM on (4864 x 65536 137, with rings 167, 1000 x 16384 15 and 24), else again
  // clusters.  A cluster's CTAs: the least of the slots that the busiest SM reads
  // and about 5000 more for the latencies of each round of CTAs.
  const int slots = (V + 16 / es - 1) / (16 / es), sms = num_sms(dev);
  const bool rows = slots <= 512 || (top_k ? R >= 4 * sms : slots <= 4096 && R >= 20 * sms);
  // Few alternatives of many short rows, or rows that a warp's list holds whole: a
  // warp a row (1300 x 1000 with 5 7.5 us and with 20 12.3, four warps 11.4 and 14.1;
  // 14000 x 1000 28 and 48, four warps 71 and 86; 14000 x 300 with 50 96 and 338; but
  // 14000 x 4000 with 32 133 and 119, 800 x 1000 with 20 11.3 and 8.9: eight CTAs of
  // four warps stay on an SM).
  const bool warps = rows && (top_k <= 24 || V <= kCandidates / 2) && slots <= 512 && R >= 8 * sms;
  const int per_sm = top_k ? 2 : 3;  // of the undivided rows' CTAs
  int parts = 1;
  if (!rows) {
    long long least = LLONG_MAX;
    for (int p = 1; p <= kMaxParts && slots / p >= 480; p *= 2) {
      const long long all = (long long)R * p, at_once = sms * (p == 1 ? per_sm : 2);
      const long long cost = (all + sms - 1) / sms * (slots / p) + (all + at_once - 1) / at_once * 5000;
      if (cost < least) least = cost, parts = p;
    }
  }
  a.lparts = __builtin_ctz((unsigned)parts);
  cudaError_t e;
  {
    ProfScope ps(stream, "token_logprobs");
    // CTAs take rows in turn (a cluster one row)
    auto go = [&](auto kernel, int threads, int per_sm) {
      const long long grid = parts > 1 ? (long long)R * parts : std::min<long long>(R, (long long)sms * per_sm);
      const size_t smem = threads == 320 ? ring_bytes(256) : 0;
      if (smem) {
        static std::atomic<uint64_t> opted[2];
        if (cudaError_t o = opt_in_smem(kernel, smem, dev, opted[dtype == PT_BF16 ? 0 : 1])) return o;
      }
      return launch_cluster(kernel, (unsigned)grid, threads, smem, parts, stream, a);
    };
    auto pick = [&](auto type) {
      using E = decltype(type);
      if (top_k && warps) return go(k_score<E, 32, true, false, false>, 32, 24);
      if (top_k) return rows ? go(k_score<E, 128, true, false, false>, 128, 8) : go(k_score<E, 480, true, true, false>, 512, 2);
      if (rows) return go(k_score<E, 32, false, false, false>, 32, 32);
      return parts == 1 ? go(k_score<E, 256, false, true, true>, 320, 3) : go(k_score<E, 480, false, true, false>, 512, 2);
    };
    e = dtype == PT_BF16 ? pick(__nv_bfloat16()) : pick(float());
    count_launch();
  }
  return (pt_status)launch_status(who, e);
}

extern "C" pt_status pt_token_logprobs_bwd(const float* dlogp, const float* dentropy, const void* logits,
                                           int64_t row_stride, pt_dtype dtype, int32_t R, int32_t V,
                                           const int64_t* targets, const int32_t* row_ptr, const int32_t* index,
                                           int32_t N, float scale, const float* LSE, const float* entropy,
                                           void* dlogits, int64_t d_stride, cudaStream_t stream) {
  static const char* who = "pt_token_logprobs_bwd";
  if (pt_status rc = check(who, dtype, R, V, N, row_stride, row_ptr, scale)) return rc;
  if (d_stride < V) {
    set_error("%s: rows of the gradient %lld elements apart, %d logits", who, (long long)d_stride, V);
    return PT_ERR_INVALID_ARG;
  }
  if (R == 0) return PT_OK;
  if (!logits || !LSE || !dlogits || (N > 0 && (!targets || !dlogp)) || (dentropy && !entropy)) {
    set_error("%s: a pointer is NULL", who);
    return PT_ERR_INVALID_ARG;
  }
  const int es = dtype == PT_BF16 ? 2 : 4, vec = 16 / es;
  const uintptr_t x = reinterpret_cast<uintptr_t>(logits), y = reinterpret_cast<uintptr_t>(dlogits);
  if ((x | y) & (uintptr_t)(es - 1)) {
    set_error("%s: logits or their gradient are not aligned to their elements", who);
    return PT_ERR_INVALID_ARG;
  }
  const uintptr_t nx = ((uintptr_t)(R - 1) * row_stride + V) * es, ny = ((uintptr_t)(R - 1) * d_stride + V) * es;
  if (!(x == y && row_stride == d_stride) && x < y + ny && y < x + nx) {
    // (columns of one buffer that do not meet: equal strides, the rows side by side)
    const uintptr_t gap = (x > y ? x - y : y - x) % ((uintptr_t)row_stride * es), row = (uintptr_t)V * es;
    if (row_stride != d_stride || gap < row || (uintptr_t)row_stride * es - gap < row) {
      set_error("%s: the gradient overlaps the logits without taking their place", who);
      return PT_ERR_INVALID_ARG;
    }
  }
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess) {
    set_error("%s: no CUDA device", who);
    return PT_ERR_CUDA;
  }
  GradArgs a;
  a.x = logits, a.d = dlogits, a.stride = row_stride, a.d_stride = d_stride, a.V = V;
  a.scale = scale;
  a.e = Entries{reinterpret_cast<const long long*>(targets), row_ptr, index, R, N};
  a.g = dlogp, a.lse = LSE, a.H = entropy, a.dH = dentropy;
  // 16-byte stores where every row of the gradient starts as its logits do
  const bool whole = ((x ^ y) & 15u) == 0 && (row_stride - d_stride) % vec == 0;
  // Threads of a CTA: a warp for short rows (30000 x 4096 77 us, four warps 97, eight
  // 149), eight for many long ones (3000 x 50001 97, four 102), else four (15000 x
  // 16384 147, eight 161, one 160; 256 x 131072 24 and 27).
  const int slots = (V + vec - 1) / vec;
  const int nt = slots <= 768 ? 32 : slots <= 4096 || R < 16 * num_sms(dev) ? 128 : 256;
  // CTAs of a row: each thread keeps at least one round of loads
  int parts = 1;
  while (parts < 64 && slots / (parts * 2) >= nt * 4 && (long long)R * parts < 16ll * num_sms(dev)) parts *= 2;
  while (parts > 1 && (long long)R * parts > INT_MAX) parts /= 2;
  a.lparts = __builtin_ctz((unsigned)parts);
  cudaError_t e;
  {
    ProfScope ps(stream, "token_logprobs_bwd");
    auto go = [&](auto kernel) { return launch_pdl(kernel, dim3((unsigned)R * (unsigned)parts), dim3(nt), 0, stream, a); };
    auto pick = [&](auto type, auto threads) {
      using E = decltype(type);
      constexpr int NT = decltype(threads)::value;
      if (dentropy) return whole ? go(k_grad<E, NT, true, true>) : go(k_grad<E, NT, true, false>);
      return whole ? go(k_grad<E, NT, false, true>) : go(k_grad<E, NT, false, false>);
    };
    auto by_threads = [&](auto type) {
      if (nt == 32) return pick(type, std::integral_constant<int, 32>{});
      return nt == 128 ? pick(type, std::integral_constant<int, 128>{}) : pick(type, std::integral_constant<int, 256>{});
    };
    e = dtype == PT_BF16 ? by_threads(__nv_bfloat16()) : by_threads(float());
    count_launch();
  }
  return (pt_status)launch_status(who, e);
}
