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
  int V, parts, k;
  float scale, c1;
  Entries e;
  float* logp;
  float* lse;
  float* H;
  float* top;
  long long* ids;
};

// ---------------------------------------------------------------------------
// Scores: one pass over the logits.  A row is one CTA's, or a cluster's that
// shares it where rows are few; a thread takes every NT-th 16 bytes, U of them
// in flight, and keeps its own running maximum and sums, which are joined at
// the end (through shared memory, then the cluster's).
//
// The alternatives take one more look at very little: the k-th largest of the
// threads' maxima bounds the k-th largest element from below, so only the
// threads whose maximum is at least that have candidates, k of them unless
// values are equal; their elements are read again (from L2), those at or above
// the bound listed, and the list ranked.  Equal maxima are told apart by their
// first index before, so that a row of equal logits lists few of them.  A list
// that overflows all the same (many large elements in few threads) is replaced
// by k searches through the part.
// ---------------------------------------------------------------------------
template <class E, int NT, bool TOP>
__global__ void __launch_bounds__(NT, 1024 / NT) k_score(const ScoreArgs a) {
  constexpr int V = Type<E>::V, U = 4;
  __shared__ Stat sm_stat[NT / 32];
  __shared__ Stat sm_part;
  __shared__ unsigned sm_most[NT / 32];
  __shared__ unsigned long long sm_key[TOP ? NT : 1], sm_cand[TOP ? kCandidates : 1], sm_best[TOP ? kMaxTop : 1];
  __shared__ int sm_who[TOP ? NT : 1];
  __shared__ int sm_n, sm_w;
  pdl_wait();
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int part = blockIdx.x % a.parts, r = blockIdx.x / a.parts;
  const Row<E> row(static_cast<const E*>(a.x) + (long long)r * a.stride, a.V);
  const int slots = row.slots();
  const int s0 = (int)((long long)slots * part / a.parts), s1 = (int)((long long)slots * (part + 1) / a.parts);
  // the first entries' logits, while the row is read
  int e0 = 0, e1 = 0, my_tok = -1, my_target = -1;
  float my_x = 0.f;
  if (part == 0) {
    a.e.range(r, e0, e1);
    if (tid < e1 - e0) {
      my_tok = a.e.token(e0 + tid);
      my_target = a.e.target(my_tok, a.V);
      if (my_target >= 0) my_x = Type<E>::f(row.x[my_target]);
    }
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
  auto take = [&](const uint4* v, auto count, int at) {  // so many slots from `at` on
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
  };
  using One = std::integral_constant<int, 1>;
  using All = std::integral_constant<int, U>;
  // whole slots, then the ones at the row's ends
  const int w0 = max(s0, row.whole(0) ? 0 : 1), w1 = min(s1, row.whole(slots - 1) ? slots : slots - 1);
#pragma unroll 1
  for (int s = w0 + tid; s < w1; s += NT * U) {
    uint4 v[U];
#pragma unroll
    for (int u = 0; u < U; ++u)
      if (s + u * NT < w1) v[u] = row.load(s + u * NT);
    if (s + (U - 1) * NT < w1) {
      take(v, All{}, s);
    } else {
#pragma unroll
      for (int u = 0; u < U; ++u)
        if (s + u * NT < w1) take(v + u, One{}, s + u * NT);
    }
  }
  int edge = -1;  // a slot at the row's end that is this thread's
  if (tid == 0 && s0 == 0 && s1 > 0 && !row.whole(0)) edge = 0;
  if (tid == NT - 1 && s1 == slots && s1 > s0 && slots > 1 && !row.whole(slots - 1)) edge = slots - 1;
  if (edge >= 0) {
    const uint4 y = row.pack(edge);
    take(&y, One{}, edge);
  }
  if (plain) rebase(st.s, st.t, -fmaf(st.m == -INFINITY ? 0.f : st.m, a.c1, -ref));
  // the CTA's statistics
  st = join_lanes<16>(st, a.c1);
  if (lane == 0) sm_stat[warp] = st;
  unsigned mine = 0;  // TOP: this thread's largest logit
  if constexpr (TOP) {
    mine = first >= 0 ? ordered(own_max) : 0u;
    const unsigned most = __reduce_max_sync(0xffffffffu, mine);
    if (lane == 0) sm_most[warp] = most;
    if (tid == 0) sm_n = sm_w = 0;
  }
  __syncthreads();
  if (warp == 0) {
    st = join_lanes<NT / 64>(lane < NT / 32 ? sm_stat[lane] : Stat{-INFINITY, 0.f, 0.f}, a.c1);
    if (lane == 0) sm_part = st;
  }
  if constexpr (TOP) {
    // The bound: at least k threads' maxima reach it, by halving; not many more
    // unless they are equal.
    const int k = a.k;
    unsigned lo = 0, hi = 0;
#pragma unroll 1
    for (int w = 0; w < NT / 32; ++w) hi = max(hi, sm_most[w]);
    ++hi;  // (a value's order is below 2^32 - 1)
    int reach = NT;                           // threads that reach lo
#pragma unroll 1
    while (hi - lo > 1 && reach > k + 8) {
      const unsigned mid = lo + ((hi - lo) >> 1);
      const int n = __syncthreads_count(mine >= mid);
      if (n >= k)
        lo = mid, reach = n;
      else
        hi = mid;
    }
    unsigned long long bound = (unsigned long long)lo << 32;
    unsigned long long best_key = (unsigned long long)mine << 32 | 0xffffffffu;  // (no less than the thread's best)
    if (hi - lo == 1 && lo && reach > k + 8) {
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
      const int above = __syncthreads_count(mine > lo);
      unsigned l = 0, h = 0xffffffffu;
#pragma unroll 1
      while (h - l > 1) {
        const unsigned mid = l + ((h - l) >> 1);
        if (above + __syncthreads_count(mine == lo && inv >= mid) >= k)
          l = mid;
        else
          h = mid;
      }
      bound |= l;
    }
    // the threads that hold candidates, and their elements
    if (mine && best_key >= bound) sm_who[atomicAdd(&sm_w, 1)] = tid;
    __syncthreads();
    auto put = [&](int s) {
      float y[V];
      row.get(s, y);
#pragma unroll
      for (int i = 0; i < V; ++i) {
        const int v = s * V - row.lead + i;
        const unsigned long long key = key_of(y[i], v);
        if (key >= bound && v >= 0 && v < a.V) {
          const int at = atomicAdd(&sm_n, 1);
          if (at < kCandidates) sm_cand[at] = key;
        }
      }
    };
    const int each = w1 > w0 ? (w1 - w0 + NT - 1) / NT : 0, who = sm_w;
#pragma unroll 1
    for (int x = tid; x < who * each; x += NT) {
      const int s = w0 + sm_who[x / each] + (x % each) * NT;
      if (s < w1) put(s);
    }
    if (edge >= 0) put(edge);
    __syncthreads();
    const int n = sm_n;
    if (n <= kCandidates) {
      for (int i = tid; i < k; i += NT) sm_best[i] = 0;
      __syncthreads();
#pragma unroll 1
      for (int i = tid; i < n; i += NT) {
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
        for (int s = s0 + tid; s < s1; s += NT) {
          float y[V];
          row.get(s, y);
#pragma unroll
          for (int j = 0; j < V; ++j) {
            const int v = s * V - row.lead + j;
            const unsigned long long key = key_of(y[j], v);
            if (v >= 0 && v < a.V && key < below && key > best) best = key;
          }
        }
        __syncthreads();
        sm_key[tid] = best;
        __syncthreads();
        for (int o = NT / 2; o; o >>= 1) {
          if (tid < o) sm_key[tid] = max(sm_key[tid], sm_key[tid + o]);
          __syncthreads();
        }
        below = sm_key[0];
        if (tid == 0) sm_best[i] = below;
        __syncthreads();
        if (below == 0) below = 1;  // (no more of them)
      }
    }
    __syncthreads();
  }
  if (a.parts > 1) {  // the cluster's
    cg::cluster_group cluster = cg::this_cluster();
    cluster.sync();
    if (part == 0) {
      if (warp == 0) st = join_lanes<kMaxParts / 2>(lane < a.parts ? *cluster.map_shared_rank(&sm_part, lane) : Stat{-INFINITY, 0.f, 0.f}, a.c1);
      if constexpr (TOP) {
        const int n = a.parts * a.k;  // (at most kMaxParts * kMaxTop)
        for (int i = tid; i < n; i += NT) sm_cand[i] = cluster.map_shared_rank(&sm_best[0], i / a.k)[i % a.k];
        __syncthreads();
        for (int i = tid; i < n; i += NT) {
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
  __syncthreads();
  st = sm_part;
  // the row's results
  const float z = st.m * a.scale;  // (S is at least 1)
  const float ln_s = st.m == -INFINITY ? 0.f : logf(st.s);
  const float lse = st.s != st.s ? st.s : st.m == -INFINITY ? -INFINITY : z + ln_s;
  if (tid == 0) {
    a.lse[r] = lse;
    if (a.H) a.H[r] = st.m == -INFINITY && st.s == st.s ? 0.f : ln_s - 0.69314718055994531f * (st.t / st.s);
  }
  // (from m, not from LSE: large logits then lose nothing)
  auto log_p = [&](float x) { return lse == -INFINITY ? -INFINITY : (x - st.m) * a.scale - ln_s; };
  if constexpr (TOP) {
    const unsigned long long* best = a.parts > 1 ? sm_key : sm_best;
    for (int i = tid; i < a.k; i += NT) {
      const unsigned long long key = best[i];
      a.top[(long long)r * a.k + i] = log_p(value_of(key));
      a.ids[(long long)r * a.k + i] = index_of(key);
    }
  }
  auto put_logp = [&](int tok, int target, float x) {
    if (tok >= 0) a.logp[tok] = target < 0 ? 0.f : log_p(x);
  };
  if (tid < e1 - e0) put_logp(my_tok, my_target, my_x);
#pragma unroll 1
  for (int n = e0 + NT + tid; n < e1; n += NT) {
    const int tok = a.e.token(n), target = a.e.target(tok, a.V);
    put_logp(tok, target, target >= 0 ? Type<E>::f(row.x[target]) : 0.f);
  }
  if (r == a.e.R - 1 && a.e.row_ptr) {  // entries of no row
    const int end = min(max(a.e.row_ptr[a.e.R], 0), a.e.N);
    for (int n = end + tid; n < a.e.N; n += NT) {
      const int tok = a.e.token(n);
      if (tok >= 0) a.logp[tok] = 0.f;
    }
  }
}

struct GradArgs {
  const void* x;
  void* d;
  long long stride, d_stride;
  int V, parts;
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
// gradient may take the logits' place.
// ---------------------------------------------------------------------------
constexpr int kSlotBits = 4096;

template <class E, int NT, bool ENT, bool VEC>
__global__ void __launch_bounds__(NT, 1024 / NT) k_grad(const GradArgs a) {
  constexpr int V = Type<E>::V, U = VEC ? 4 : 1;
  __shared__ unsigned bits[kSlotBits / 32];
  __shared__ float sm_g[NT / 32];
  pdl_wait();
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int part = blockIdx.x % a.parts, r = blockIdx.x / a.parts;
  const Row<E> row(static_cast<const E*>(a.x) + (long long)r * a.stride, a.V);
  E* out = static_cast<E*>(a.d) + (long long)r * a.d_stride;
  const int slots = row.slots();
  const int s0 = (int)((long long)slots * part / a.parts), s1 = (int)((long long)slots * (part + 1) / a.parts);
  int e0, e1;
  a.e.range(r, e0, e1);
  float lse = a.lse[r];
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
  auto one = [&](float x) {
    const float l = fmaxf(fmaf(x, a.scale, -lse), -1000.f);  // ln p (p is 0 from -104 on: its product with ln p too)
    const float p = ex2(l * 1.4426950408889634f);
    return p * (ENT ? fmaf(cb, l, ca) : ca);
  };
  auto entries = [&](int s, float (&y)[V]) {
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
  };
  auto store_some = [&](int s, const float (&y)[V]) {
#pragma unroll
    for (int i = 0; i < V; ++i) {
      const int v = s * V - row.lead + i;
      if (v >= 0 && v < a.V) {
        if constexpr (sizeof(E) == 2)
          out[v] = __float2bfloat16_rn(y[i]);
        else
          out[v] = y[i];
      }
    }
  };
#pragma unroll 1
  for (int s = s0 + tid; s < s1; s += NT * U) {
    uint4 v[U];
#pragma unroll
    for (int u = 0; u < U; ++u)
      if (s + u * NT < s1 && row.whole(s + u * NT)) v[u] = *reinterpret_cast<const uint4*>(row.x + ((long long)(s + u * NT) * V - row.lead));
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
      if (VEC && whole) {
        uint4 w;
        if constexpr (sizeof(E) == 2)
          w = make_uint4(pack_bf16(y[0], y[1]), pack_bf16(y[2], y[3]), pack_bf16(y[4], y[5]), pack_bf16(y[6], y[7]));
        else
          w = make_uint4(__float_as_uint(y[0]), __float_as_uint(y[1]), __float_as_uint(y[2]), __float_as_uint(y[3]));
        *reinterpret_cast<uint4*>(out + ((long long)at * V - row.lead)) = w;
      } else {
        store_some(at, y);
      }
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

// As launch_pdl, with `parts` CTAs a cluster.
template <class K, class A>
cudaError_t launch_cluster(K kernel, unsigned grid, int threads, int parts, cudaStream_t s, const A& a) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(grid);
  cfg.blockDim = dim3(threads);
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
  if (V > 1 << 30 || R > INT_MAX / kMaxParts) {
    set_error("%s: %d rows of %d logits are out of range", who, R, V);
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
  const int slots = (V + 16 / es - 1) / (16 / es), nt = slots >= 1024 ? 512 : 128;
  // Few rows: a cluster each, until the SMs have three CTAs or a thread less than four loads.
  int parts = 1;
  while (parts < kMaxParts && (long long)R * parts * 2 <= 3ll * num_sms(dev) && slots / (parts * 2) >= nt * 4) parts *= 2;
  a.parts = parts;
  cudaError_t e;
  {
    ProfScope ps(stream, "token_logprobs");
    auto go = [&](auto kernel) { return launch_cluster(kernel, (unsigned)R * (unsigned)parts, nt, parts, stream, a); };
    if (dtype == PT_BF16) {
      if (top_k)
        e = nt == 512 ? go(k_score<__nv_bfloat16, 512, true>) : go(k_score<__nv_bfloat16, 128, true>);
      else
        e = nt == 512 ? go(k_score<__nv_bfloat16, 512, false>) : go(k_score<__nv_bfloat16, 128, false>);
    } else {
      if (top_k)
        e = nt == 512 ? go(k_score<float, 512, true>) : go(k_score<float, 128, true>);
      else
        e = nt == 512 ? go(k_score<float, 512, false>) : go(k_score<float, 128, false>);
    }
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
    set_error("%s: the gradient overlaps the logits without taking their place", who);
    return PT_ERR_INVALID_ARG;
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
  const int slots = (V + vec - 1) / vec;
  constexpr int NT = 256;
  // about two rounds of loads a CTA where rows are few
  int parts = 1;
  while (parts < 64 && slots / (parts * 2) >= NT * 4 && (long long)R * parts < 16ll * num_sms(dev)) parts *= 2;
  while (parts > 1 && (long long)R * parts > INT_MAX) parts /= 2;
  a.parts = parts;
  cudaError_t e;
  {
    ProfScope ps(stream, "token_logprobs_bwd");
    auto go = [&](auto kernel) { return launch_pdl(kernel, dim3((unsigned)R * (unsigned)parts), dim3(NT), 0, stream, a); };
    if (dtype == PT_BF16) {
      if (dentropy)
        e = whole ? go(k_grad<__nv_bfloat16, NT, true, true>) : go(k_grad<__nv_bfloat16, NT, true, false>);
      else
        e = whole ? go(k_grad<__nv_bfloat16, NT, false, true>) : go(k_grad<__nv_bfloat16, NT, false, false>);
    } else {
      if (dentropy)
        e = whole ? go(k_grad<float, NT, true, true>) : go(k_grad<float, NT, true, false>);
      else
        e = whole ? go(k_grad<float, NT, false, true>) : go(k_grad<float, NT, false, false>);
    }
    count_launch();
  }
  return (pt_status)launch_status(who, e);
}
