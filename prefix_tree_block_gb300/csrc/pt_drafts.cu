// pt_drafts.cu -- trees of drafted tokens behind the samples of a cached
// prefix tree: what each draft sees and where it stands (pt_draft_tree), and
// the accepted drafts' keys and values moved together (pt_cache_keep).  The
// attention between the two is pt_attn_decode_drafts.
#include <cuda_bf16.h>

#include <algorithm>
#include <climits>

#include "pt.h"
#include "pt_decode.cuh"
#include "pt_device.cuh"
#include "pt_internal.h"

namespace pt {
int take_status_drafts(cudaStream_t s) { return take_status_here(s); }
}  // namespace pt

using namespace pt;

namespace {

constexpr int kMaxDrafts = 256;  // of a sample: 8 words of a mask

// A sample's last node.
__device__ __forceinline__ int leaf_of(const int* path_ptr, const int2* path_ent, int s) {
  return path_ent[path_ptr[s + 1] - 1].x;
}

// ---------------------------------------------------------------------------
// Ancestors by doubling: after round k a draft's bits hold the 2^k drafts
// nearest above it (itself among them), and its pointer names the next one;
// log2(q_len) rounds, each over all drafts at once.  Integer work of a few
// hundred bytes a sample: bound by latency (a launch, a chain of loads, the
// rounds in shared memory).  `per` samples a CTA, so that short trees fill it.
// 4096 samples of 64 drafts 13.4 us so, 3.2 in k_draft_tree64.
// ---------------------------------------------------------------------------
struct TreeArgs {
  const int* parents;
  const int* lens;
  const int* q_count;
  const int* start;
  const int* path_ptr;
  const int2* path_ent;
  int S, q, w, per;
  int* mask;
  long long* positions;
};

// Up to 64 drafts: a warp per sample and a lane for two drafts, all in registers.
// 64 samples 1.8 us (a launch and its chain of loads).
__global__ void __launch_bounds__(128) k_draft_tree64(const TreeArgs a) {
  pdl_wait();
  const int s = blockIdx.x * 4 + (threadIdx.x >> 5), lane = threadIdx.x & 31;
  if (s >= a.S) return;
  int c = a.q_count ? a.q_count[s] : a.q;
  const long long row0 = (long long)s * a.q;
  int up[2];
  unsigned m[2][2];  // [draft lane, draft lane + 32][word]
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    const int j = lane + 32 * i;
    up[i] = j < a.q ? a.parents[row0 + j] : -1;
  }
  long long first = 0;
  if (a.positions) {
    const int leaf = leaf_of(a.path_ptr, a.path_ent, s);
    first = (long long)a.lens[leaf] + (a.start ? a.start[leaf] : 0);
  }
  bool bad = c < 0 || c > a.q;
  c = min(max(c, 0), a.q);
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    const int j = lane + 32 * i;
    bad |= j < c && (up[i] < -1 || up[i] >= j);
    if (j >= c || up[i] < 0 || up[i] >= j) up[i] = -1;
    m[i][0] = i == 0 ? 1u << lane : 0u;
    m[i][1] = i == 1 ? 1u << lane : 0u;
  }
  if (bad) record_status(PT_STATUS_INVALID);
#pragma unroll 1
  for (int span = 1; span < a.q; span <<= 1) {
    unsigned n[2][2];
    int nu[2];
#pragma unroll
    for (int i = 0; i < 2; ++i) {  // (draft up[i] is lane up[i] & 31's, its first or second)
      const int from = up[i] & 31;
      const bool hi = up[i] >= 32;
#pragma unroll
      for (int w = 0; w < 2; ++w) {
        const unsigned x = __shfl_sync(0xffffffffu, m[0][w], from), y = __shfl_sync(0xffffffffu, m[1][w], from);
        n[i][w] = m[i][w] | (up[i] < 0 ? 0u : hi ? y : x);
      }
      const int x = __shfl_sync(0xffffffffu, up[0], from), y = __shfl_sync(0xffffffffu, up[1], from);
      nu[i] = up[i] < 0 ? -1 : hi ? y : x;
    }
#pragma unroll
    for (int i = 0; i < 2; ++i) m[i][0] = n[i][0], m[i][1] = n[i][1], up[i] = nu[i];
  }
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    const int j = lane + 32 * i;
    if (j >= a.q) continue;
    const bool real = j < c;
    if (a.w == 1)
      a.mask[row0 + j] = real ? (int)m[i][0] : 0;
    else
      reinterpret_cast<int2*>(a.mask)[row0 + j] = real ? make_int2((int)m[i][0], (int)m[i][1]) : make_int2(0, 0);
    if (a.positions) a.positions[row0 + j] = real ? first - c + __popc(m[i][0]) + __popc(m[i][1]) - 1 : 0;
  }
}

__global__ void __launch_bounds__(128) k_draft_tree(const TreeArgs a) {
  extern __shared__ int sm[];
  pdl_wait();
  const int rows = a.per * a.q, s0 = blockIdx.x * a.per;
  const int n = min(a.per, a.S - s0) * a.q;  // rows there are
  int *up0 = sm, *up1 = sm + rows;
  unsigned *m0 = reinterpret_cast<unsigned*>(sm + 2 * rows), *m1 = m0 + rows * a.w;
  int* cnt = sm + 2 * rows + 2 * rows * a.w;  // [per]
  for (int i = threadIdx.x; i < a.per && s0 + i < a.S; i += 128) {
    const int c = a.q_count ? a.q_count[s0 + i] : a.q;
    if (c < 0 || c > a.q) record_status(PT_STATUS_INVALID);
    cnt[i] = min(max(c, 0), a.q);
  }
  for (int r = threadIdx.x; r < n; r += 128) {
    const int j = r % a.q;
    int p = a.parents[(long long)s0 * a.q + r];
    // (parents behind the count are not looked at: their rows end as zeros)
    up0[r] = p;
    for (int w = 0; w < a.w; ++w) m0[r * a.w + w] = w == (j >> 5) ? 1u << (j & 31) : 0u;
  }
  __syncthreads();
  for (int r = threadIdx.x; r < n; r += 128) {
    const int j = r % a.q, p = up0[r];
    const bool real = j < cnt[r / a.q];
    if (real && (p < -1 || p >= j)) record_status(PT_STATUS_INVALID);
    up0[r] = real && p >= 0 && p < j ? p : -1;
  }
  __syncthreads();
#pragma unroll 1
  for (int span = 1; span < a.q; span <<= 1) {
    for (int x = threadIdx.x; x < n * a.w; x += 128) {
      const int r = x / a.w, p = up0[r];
      const int above = (r - r % a.q + p) * a.w + (x - r * a.w);
      m1[x] = m0[x] | (p >= 0 ? m0[above] : 0u);
    }
    for (int r = threadIdx.x; r < n; r += 128) {
      const int p = up0[r];
      up1[r] = p >= 0 ? up0[r - r % a.q + p] : -1;
    }
    __syncthreads();
    int* t = up0;
    up0 = up1, up1 = t;
    unsigned* u = m0;
    m0 = m1, m1 = u;
  }
  for (int r = threadIdx.x; r < n; r += 128) {
    const int i = r / a.q, s = s0 + i, c = cnt[i], j = r - i * a.q;
    const bool real = j < c;
    int depth = -1;
    for (int w = 0; w < a.w; ++w) {
      const unsigned bits = real ? m0[r * a.w + w] : 0u;
      depth += __popc(bits);
      a.mask[((long long)s0 * a.q + r) * a.w + w] = (int)bits;
    }
    if (a.positions) {
      const int leaf = leaf_of(a.path_ptr, a.path_ent, s);
      const long long first = (long long)a.lens[leaf] - c + (a.start ? a.start[leaf] : 0);
      a.positions[(long long)s0 * a.q + r] = real ? first + depth : 0;
    }
  }
}

// ---------------------------------------------------------------------------
// The i-th accepted draft is at its place or behind it (they come in
// ascending order), so a thread that moves its 16 bytes of every token in
// that order, some tokens' loads before their stores, never overwrites what
// it has still to read; and no other thread touches those bytes.  A CTA per
// sample and part of a token's row; K and V in one launch.  Bound by memory,
// or by a chain of latencies where samples are few: the counts, the accepted
// drafts, their pages, the rows.  64 samples of 8 drafts 2.7 us; 1024 of 16, 8 kv
// heads of 128 in bf16 (15 MB moved) 4.8 us.
// ---------------------------------------------------------------------------
struct KeepArgs {
  const int* kept;
  const int* lens;
  const int* q_count;
  const int* tables;
  const int* path_ptr;
  const int2* path_ent;
  char* Kc;
  char* Vc;
  int q, ps, max_pages, n_pages;
  int nv, hv;  // vectors of a token's row, and of one head's part
};

template <class Vec>
__global__ void __launch_bounds__(256) k_cache_keep(const KeepArgs a) {
  pdl_wait();
  const int s = blockIdx.x;
  __shared__ long long from[kMaxDrafts], to[kMaxDrafts];  // vectors: the token's row in head 0
  __shared__ int order_ok, total;
  const int leaf = leaf_of(a.path_ptr, a.path_ent, s);
  const long long cap = (long long)a.max_pages * a.ps;
  const int len = a.lens[leaf];
  int c = a.q_count ? a.q_count[s] : a.q;
  bool bad = c < 0 || c > a.q || len < 0 || len > cap;
  c = min(max(c, 0), a.q);
  const int base = len - c;
  bad |= base < 0;
  if (threadIdx.x == 0) order_ok = 1, total = a.q;
  __syncthreads();
  // the accepted drafts, up to the first that is negative
  for (int i = threadIdx.x; i < a.q; i += blockDim.x)
    if (a.kept[(long long)s * a.q + i] < 0) atomicMin(&total, i);
  __syncthreads();
  const int n = total;
  if (n == 0 || bad) {
    if (bad && threadIdx.x == 0 && blockIdx.y == 0) record_status(PT_STATUS_INVALID);
    return;
  }
  for (int i = threadIdx.x; i < n; i += blockDim.x) {
    const int j = a.kept[(long long)s * a.q + i], before = i ? a.kept[(long long)s * a.q + i - 1] : -1;
    bool fine = j < c && j > before;
    long long at[2] = {0, 0};
    if (fine && i != j) {
#pragma unroll
      for (int k = 0; k < 2; ++k) {
        const int tok = base + (k ? i : j), pi = tok / a.ps;
        const int page = a.tables[(long long)leaf * a.max_pages + pi];
        if ((unsigned)page >= (unsigned)a.n_pages) fine = false;
        at[k] = (long long)page * a.nv * a.ps + (long long)(tok - pi * a.ps) * a.hv;
      }
    }
    if (!fine) order_ok = 0;
    from[i] = i == j ? -1 : at[0];
    to[i] = at[1];
  }
  __syncthreads();
  if (!order_ok) {  // the sample stays as it is
    if (threadIdx.x == 0 && blockIdx.y == 0) record_status(PT_STATUS_INVALID);
    return;
  }
  constexpr int U = 4;
#pragma unroll 1
  for (int v = blockIdx.y * blockDim.x + threadIdx.x; v < 2 * a.nv; v += gridDim.y * blockDim.x) {
    const int x = v >= a.nv ? v - a.nv : v, h = x / a.hv;
    Vec* cache = reinterpret_cast<Vec*>(v >= a.nv ? a.Vc : a.Kc) + (long long)h * a.ps * a.hv + (x - h * a.hv);
#pragma unroll 1
    for (int i0 = 0; i0 < n; i0 += U) {
      Vec r[U];
#pragma unroll
      for (int u = 0; u < U; ++u)
        if (i0 + u < n && from[i0 + u] >= 0) r[u] = cache[from[i0 + u]];
#pragma unroll
      for (int u = 0; u < U; ++u)
        if (i0 + u < n && from[i0 + u] >= 0) cache[to[i0 + u]] = r[u];
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

int check_plan(const char* who, const pt_decodeplan* plan) {
  if (!plan) {
    set_error("%s: plan is NULL", who);
    return PT_ERR_INVALID_ARG;
  }
  if (plan->q_len > kMaxDrafts) {
    set_error("%s: q_len = %d, at most %d drafts a sample", who, plan->q_len, kMaxDrafts);
    return PT_ERR_UNSUPPORTED;
  }
  int dev = -1;
  if (cudaGetDevice(&dev) != cudaSuccess || dev != plan->device) {
    set_error("%s: the plan lives on device %d, the current device is %d", who, plan->device, dev);
    return PT_ERR_INVALID_ARG;
  }
  return PT_OK;
}

}  // namespace

extern "C" pt_status pt_draft_tree(const int32_t* parents, const int32_t* lens, const int32_t* q_count,
                                   const int32_t* start, const pt_decodeplan* plan, int32_t* mask, int64_t* positions,
                                   cudaStream_t stream) {
  static const char* who = "pt_draft_tree";
  if (int rc = check_plan(who, plan)) return (pt_status)rc;
  if (plan->S == 0) return PT_OK;
  if (!parents || !lens || !mask) {
    set_error("%s: a pointer is NULL", who);
    return PT_ERR_INVALID_ARG;
  }
  TreeArgs a;
  a.parents = parents, a.lens = lens, a.q_count = q_count, a.start = start;
  a.path_ptr = plan->path_ptr, a.path_ent = plan->path_ent;
  a.S = plan->S, a.q = plan->q_len, a.w = (a.q + 31) / 32;
  a.per = std::max(1, 128 / a.q);
  a.mask = mask;
  a.positions = reinterpret_cast<long long*>(positions);
  const size_t smem = 4 * ((size_t)a.per * a.q * (2 + 2 * a.w) + a.per);
  const bool warps = a.q <= 64 && (reinterpret_cast<uintptr_t>(mask) & 7) == 0;
  cudaError_t e;
  {
    ProfScope ps(stream, "draft_tree");
    e = warps ? launch_pdl(k_draft_tree64, dim3((unsigned)((a.S + 3) / 4)), dim3(128), 0, stream, a)
              : launch_pdl(k_draft_tree, dim3((unsigned)((a.S + a.per - 1) / a.per)), dim3(128), smem, stream, a);
    count_launch();
  }
  return (pt_status)launch_status(who, e);
}

extern "C" pt_status pt_cache_keep(const int32_t* kept, const int32_t* q_count, const int32_t* lens,
                                   const int32_t* tables, int32_t max_pages, pt_dtype dtype, int32_t D, void* Kc,
                                   void* Vc, int32_t n_pages, int32_t page_size, const pt_decodeplan* plan,
                                   cudaStream_t stream) {
  static const char* who = "pt_cache_keep";
  if (dtype != PT_BF16 && dtype != PT_F32) {
    set_error("%s: unknown dtype %d", who, (int)dtype);
    return PT_ERR_INVALID_ARG;
  }
  if (int rc = check_plan(who, plan)) return (pt_status)rc;
  const int es = dtype == PT_BF16 ? 2 : 4;
  if (D < 1 || n_pages < 0 || page_size < 1 || max_pages < 0 || (long long)max_pages * page_size > INT_MAX / 2 ||
      (long long)plan->Hkv * D > INT_MAX / 8) {
    set_error("%s: D = %d, n_pages = %d, page_size = %d or max_pages = %d out of range", who, D, n_pages, page_size,
              max_pages);
    return PT_ERR_INVALID_ARG;
  }
  if (!plan->own_leaves) {
    set_error("%s: two samples of the plan end at one node", who);
    return PT_ERR_INVALID_ARG;
  }
  if (plan->S == 0) return PT_OK;
  if (!kept || !lens || (!tables && max_pages > 0) || ((!Kc || !Vc) && n_pages > 0)) {
    set_error("%s: a pointer is NULL", who);
    return PT_ERR_INVALID_ARG;
  }
  const uintptr_t all = reinterpret_cast<uintptr_t>(Kc) | reinterpret_cast<uintptr_t>(Vc) | (uintptr_t)(D * es);
  if (all & (uintptr_t)(es - 1)) {
    set_error("%s: a pointer is not aligned to its elements", who);
    return PT_ERR_INVALID_ARG;
  }
  const uintptr_t kc = reinterpret_cast<uintptr_t>(Kc), vc = reinterpret_cast<uintptr_t>(Vc);
  const uintptr_t bytes = (uintptr_t)n_pages * plan->Hkv * page_size * D * es;
  if (kc < vc + bytes && vc < kc + bytes) {  // (each of the two would move the other's)
    set_error("%s: Kc and Vc overlap", who);
    return PT_ERR_INVALID_ARG;
  }
  int unit = 16;
  while (unit > es && (all & (uintptr_t)(unit - 1))) unit >>= 1;
  KeepArgs a;
  a.kept = kept, a.lens = lens, a.q_count = q_count, a.tables = tables;
  a.path_ptr = plan->path_ptr, a.path_ent = plan->path_ent;
  a.Kc = static_cast<char*>(Kc), a.Vc = static_cast<char*>(Vc);
  a.q = plan->q_len, a.ps = page_size, a.max_pages = max_pages, a.n_pages = n_pages;
  a.hv = D * es / unit;
  a.nv = plan->Hkv * a.hv;
  const int threads = std::min(256, std::max(32, (2 * a.nv + 31) / 32 * 32));
  const int parts = std::min((2 * a.nv + threads - 1) / threads, 64);
  cudaError_t e;
  {
    ProfScope ps(stream, "cache_keep");
    auto go = [&](auto kernel) {
      return launch_pdl(kernel, dim3((unsigned)plan->S, (unsigned)parts), dim3(threads), 0, stream, a);
    };
    e = unit == 16  ? go(k_cache_keep<uint4>)
        : unit == 8 ? go(k_cache_keep<uint2>)
        : unit == 4 ? go(k_cache_keep<uint32_t>)
                    : go(k_cache_keep<unsigned short>);
    count_launch();
  }
  return (pt_status)launch_status(who, e);
}
