// pt_cache.cu -- the paged key/value cache of rollout decoding: page tables,
// slots and position ids of one step from the rows' lengths, and the store of
// the step's keys and values into their slots.
//
// "cp=1 shared-prefix prefix-tree attention for rollouts" (PR description)
// stores a prompt once for all its completions; the cache does the same while
// they are generated.  A cache row is a tree node (a prompt, one sample's own
// continuation), its tokens sit in pages of page_size tokens, and a page is
// [Hkv][page_size][D], so one head's keys of a page are one contiguous run.
#include <cuda_bf16.h>

#include <algorithm>
#include <climits>

#include "pt.h"
#include "pt_device.cuh"
#include "pt_internal.h"

namespace pt {
int take_status_drafts(cudaStream_t s);  // pt_drafts.cu
int take_status_cache(cudaStream_t s) {
  const int a = take_status_here(s), b = take_status_drafts(s);
  return a < 0 || b < 0 ? -1 : a | b;
}
}  // namespace pt

using namespace pt;

namespace {

constexpr int kTabWarps = 32;
constexpr int kTabMaxRows = 1 << 18;  // 12 bytes of shared memory per 32 rows
constexpr int kTabMaxNew = 1 << 30;
// Ids of a ring: a place in it plus a count of pages below its size fits in 32
// bits, and no page of it lies behind the sums' clamp.
constexpr int kTabMaxRing = 1 << 30;

// What a row does in this step, from its lengths.
struct RowMove {
  int held, grow;  // tokens before, tokens appended (0 when it shrinks)
  int p0, take, back;  // pages before; pages it takes or gives back
  int p1, len;     // pages and tokens after
  bool bad;
};

__device__ __forceinline__ RowMove row_move(int held, int added, int ps, long long most) {
  RowMove m;
  const long long after = (long long)held + added;
  m.bad = held < 0 || held > most || after < 0 || after > most;
  if (m.bad) {  // left as it is
    held = (int)min((long long)max(held, 0), most);
    added = 0;
  }
  m.held = held;
  m.len = held + added;
  m.grow = max(added, 0);
  m.p0 = (held + ps - 1) / ps;
  m.p1 = (m.len + ps - 1) / ps;
  m.take = max(m.p1 - m.p0, 0);
  m.back = max(m.p0 - m.p1, 0);
  return m;
}

__device__ __forceinline__ int warp_incl_scan(int v, int lane) {
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int u = __shfl_up_sync(0xffffffffu, v, o);
    if (lane >= o) v += u;
  }
  return v;
}

// Tokens before each of a chunk's rows, `before` those of the chunks before it;
// none above kTabMaxNew + 1, where 32 rows may hold more than 2^31.
__device__ __forceinline__ int tokens_before(int before, int grow, int lane) {
  constexpr unsigned top = (unsigned)kTabMaxNew + 1;
  unsigned s = min((unsigned)grow, top);
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const unsigned u = __shfl_up_sync(0xffffffffu, s, o);
    if (lane >= o) s = min(s + u, top);
  }
  const unsigned excl = __shfl_up_sync(0xffffffffu, s, 1);
  return (int)min((unsigned)before + (lane ? excl : 0u), top);
}

// The lane whose half-open run [start of lane, start of lane + 1) holds x:
// the last lane with excl <= x (runs of length zero are passed over).
__device__ __forceinline__ int lane_of(int excl, int x) {
  int at = 0;
#pragma unroll
  for (int o = 16; o; o >>= 1) {
    const int e = __shfl_sync(0xffffffffu, excl, at + o);
    if (e <= x) at += o;
  }
  return at;
}

// (a call each: 64-bit divisions are long, and their instructions come from memory)
__device__ __noinline__ long long mod_call(long long a, long long b) { return a % b; }

struct TabArgs {
  const int* held;
  const int* added;
  const int* start;
  const long long* counters;
  int* tables;
  int* ring;
  int* lens;
  int* row_ptr;
  long long* slots;
  long long* positions;
  long long* counters_out;
  int n, ps, cap, max_pages, max_new;
};

// Walks a line of units that belong to chunks of rows (cum: exclusive sums over
// chunks, cum[nc] all of them), cut into runs of kRun for the warps: f(chunk,
// x0, x1) for each chunk's part of a run.  A chunk counts kPad units more than
// it has, what looking at its rows costs: without that, a run over rows of one
// token each would visit dozens of chunks one after another.
constexpr int kRun = 256, kPad = 64;
template <class F>
__device__ __forceinline__ void for_line(const int* cum, int nc, int upto, int first, int warps, F f) {
  const int line = upto + kPad * nc;
#pragma unroll 1
  for (int r = first; (long long)r * kRun < line; r += warps) {
    int pos = r * kRun;
    const int end = min(pos + kRun, line);
    int c = 0;
#pragma unroll 1
    for (int span = 1 << (31 - __clz(nc)); span; span >>= 1)
      if (c + span < nc && cum[c + span] + kPad * (c + span) <= pos) c += span;
#pragma unroll 1
    for (; pos < end && c < nc; ++c) {
      const int lo = cum[c], hi = min(cum[c + 1], upto), shift = lo + kPad * c;
      const int x0 = lo + pos - shift, x1 = min(lo + end - shift, hi);
      if (x0 < x1) f(c, x0, x1);
      pos = max(pos, cum[c + 1] + kPad * (c + 1));
    }
  }
}

// One launch.  Every CTA sums the rows' tokens and pages itself, 32 rows (a
// chunk) per warp step, and scans the chunk sums in shared memory (three sums
// per chunk), so no CTA waits for another.  Then the pages taken, the pages
// given back and the tokens' slots are three lines of units, each cut evenly
// over all warps whatever the rows' lengths.  A slot's page comes from the
// row's table when the row held that page before, else straight from the ring,
// so nothing written here is read here.  Bound by the latency of these steps:
// 72 rows, 64 tokens 7 us; 4096 rows with 0.8 million new tokens (13.5 MB)
// 13.3 us, of which the bytes are 2.
__global__ void __launch_bounds__(kTabWarps * 32) k_cache_tables(const TabArgs a) {
  pdl_wait();
  extern __shared__ int sm[];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int nc = (a.n + 31) >> 5;
  int* c_new = sm;                // [nc + 1] exclusive sums over chunks
  int* c_take = sm + (nc + 1);
  int* c_back = sm + 2 * (nc + 1);
  const long long most = (long long)a.max_pages * a.ps;
  int h = 0, ad = 0;  // of this lane's row, loaded a chunk ahead
  if (warp * 32 + lane < a.n) h = a.held[warp * 32 + lane], ad = a.added[warp * 32 + lane];
#pragma unroll 1
  for (int c = warp; c < nc; c += kTabWarps) {
    const RowMove m = row_move(h, ad, a.ps, most);
    const int i = (c + kTabWarps) * 32 + lane;
    h = i < a.n ? a.held[i] : 0, ad = i < a.n ? a.added[i] : 0;
    if (m.bad && blockIdx.x == 0) record_status(PT_STATUS_INVALID);
    // tokens in two halves: 32 rows can hold more than 2^31 of them
    const long long g = ((long long)__reduce_add_sync(0xffffffffu, m.grow >> 16) << 16) +
                        __reduce_add_sync(0xffffffffu, m.grow & 0xffff);
    const int t = __reduce_add_sync(0xffffffffu, m.take), b = __reduce_add_sync(0xffffffffu, m.back);
    if (lane == 0) c_new[c] = (int)min(g, (long long)kTabMaxNew + 1), c_take[c] = t, c_back[c] = b;
  }
  __syncthreads();
  if (warp < 3) {  // exclusive scan of one of the three sums (tokens stop at kTabMaxNew + 1, over any max_new)
    int* v = warp == 0 ? c_new : warp == 1 ? c_take : c_back;
    long long carry = 0;
#pragma unroll 1
    for (int c0 = 0; c0 < nc; c0 += 32) {
      const long long x = c0 + lane < nc ? v[c0 + lane] : 0;
      long long s = x;
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const long long u = __shfl_up_sync(0xffffffffu, s, o);
        if (lane >= o) s += u;
      }
      if (c0 + lane < nc) v[c0 + lane] = (int)min(carry + s - x, (long long)kTabMaxNew + 1);
      carry += __shfl_sync(0xffffffffu, s, 31);
    }
    if (lane == 0) v[nc] = (int)min(carry, (long long)kTabMaxNew + 1);
  }
  __syncthreads();
  const long long head = a.counters[0], tail = a.counters[1];
  long long avail_l = tail - head;
  const bool ring_bad = head < 0 || avail_l < 0 || avail_l > a.cap;
  if (ring_bad) avail_l = 0;
  const int avail = (int)avail_l;
  const int h0 = ring_bad ? 0 : (int)mod_call(head, a.cap), t0 = ring_bad ? 0 : (int)mod_call(tail, a.cap);
  const int n_new = c_new[nc], n_take = c_take[nc], n_back = c_back[nc];
  // pages given back beyond the ring's room are dropped (the caller's page
  // count is then wrong, which is recorded)
  const int room = a.cap - avail;
  if (blockIdx.x == 0 && threadIdx.x == 0) {
    if (ring_bad || n_new > a.max_new || n_back > room) record_status(PT_STATUS_INVALID);
    if (n_take > avail) record_status(PT_STATUS_NOMEM);
    a.counters_out[0] = head + min(n_take, avail);
    a.counters_out[1] = tail + (ring_bad ? 0 : min(n_back, room));
    a.row_ptr[a.n] = n_new;
  }
  // the rows' own outputs
#pragma unroll 1
  for (int c = blockIdx.x + gridDim.x * warp; c < nc; c += gridDim.x * kTabWarps) {
    const int i = c * 32 + lane;
    const RowMove m = row_move(i < a.n ? a.held[i] : 0, i < a.n ? a.added[i] : 0, a.ps, most);
    const int e_new = tokens_before(c_new[c], m.grow, lane);
    const int e_take = warp_incl_scan(m.take, lane) - m.take;
    if (i < a.n) {
      a.row_ptr[i] = e_new;
      // a row that got fewer pages than it needs holds what fits in them
      const int got = min(m.take, max(avail - (c_take[c] + e_take), 0));
      a.lens[i] = got < m.take ? (int)min((long long)m.len, (long long)(m.p0 + got) * a.ps) : m.len;
    }
  }
  const int warps = gridDim.x * kTabWarps, me = blockIdx.x + gridDim.x * warp;
  constexpr int U = 4;  // loads in flight per lane
  if (n_take)
    for_line(c_take, nc, min(n_take, avail), me, warps, [&](int c, int x0, int x1) {
      const int i = c * 32 + lane;
      const RowMove m = row_move(i < a.n ? a.held[i] : 0, i < a.n ? a.added[i] : 0, a.ps, most);
      const int excl = c_take[c] + warp_incl_scan(m.take, lane) - m.take;
#pragma unroll 1
      for (int x = x0; x < x1; x += 32 * U) {
        int id[U];
        size_t at[U];
#pragma unroll
        for (int u = 0; u < U; ++u) {
          const int y = min(x + u * 32 + lane, x1 - 1), l = lane_of(excl, y);
          at[u] = (size_t)(c * 32 + l) * a.max_pages + __shfl_sync(0xffffffffu, m.p0, l) + y - __shfl_sync(0xffffffffu, excl, l);
          const int r = h0 + y;
          id[u] = a.ring[r >= a.cap ? r - a.cap : r];
        }
#pragma unroll
        for (int u = 0; u < U; ++u)
          if (x + u * 32 + lane < x1) a.tables[at[u]] = id[u];
      }
    });
  if (n_back && !ring_bad)
    for_line(c_back, nc, min(n_back, room), warps - 1 - me, warps, [&](int c, int x0, int x1) {
      const int i = c * 32 + lane;
      const RowMove m = row_move(i < a.n ? a.held[i] : 0, i < a.n ? a.added[i] : 0, a.ps, most);
      const int excl = c_back[c] + warp_incl_scan(m.back, lane) - m.back;
#pragma unroll 1
      for (int x = x0; x < x1; x += 32 * U) {
        int id[U];
#pragma unroll
        for (int u = 0; u < U; ++u) {
          const int y = min(x + u * 32 + lane, x1 - 1), l = lane_of(excl, y);
          id[u] = a.tables[(size_t)(c * 32 + l) * a.max_pages + __shfl_sync(0xffffffffu, m.p1, l) + y -
                           __shfl_sync(0xffffffffu, excl, l)];
        }
#pragma unroll
        for (int u = 0; u < U; ++u)
          if (x + u * 32 + lane < x1) {
            const int r = t0 + x + u * 32 + lane;
            if (id[u] < 0) record_status(PT_STATUS_INVALID);
            a.ring[r >= a.cap ? r - a.cap : r] = id[u];
          }
      }
    });
  const int n_real = min(n_new, a.max_new);
  if (n_real)
    for_line(c_new, nc, n_real, (me + warps / 2) % warps, warps, [&](int c, int x0, int x1) {
      const int i = c * 32 + lane;
      const RowMove m = row_move(i < a.n ? a.held[i] : 0, i < a.n ? a.added[i] : 0, a.ps, most);
      const int st = a.start && i < a.n ? a.start[i] : 0;
      const int e_new = tokens_before(c_new[c], m.grow, lane);
      const int e_take = c_take[c] + warp_incl_scan(m.take, lane) - m.take;
#pragma unroll 1
      for (int x = x0; x < x1; x += 32 * U) {
        int page[U], tok[U], pos[U], rest[U];
#pragma unroll
        for (int u = 0; u < U; ++u) {
          const int y = min(x + u * 32 + lane, x1 - 1), l = lane_of(e_new, y);
          tok[u] = __shfl_sync(0xffffffffu, m.held, l) + y - __shfl_sync(0xffffffffu, e_new, l);
          pos[u] = __shfl_sync(0xffffffffu, st, l);
          const int p0 = __shfl_sync(0xffffffffu, m.p0, l), et = __shfl_sync(0xffffffffu, e_take, l);
          const int pi = tok[u] / a.ps;
          rest[u] = tok[u] - pi * a.ps;
          page[u] = -1;
          if (pi < p0) {
            page[u] = a.tables[(size_t)(c * 32 + l) * a.max_pages + pi];
          } else if (et + pi - p0 < avail) {
            const int r = h0 + et + pi - p0;
            page[u] = a.ring[r >= a.cap ? r - a.cap : r];
          }
        }
#pragma unroll
        for (int u = 0; u < U; ++u) {
          const int y = x + u * 32 + lane;
          if (y < x1) {
            a.slots[y] = page[u] >= 0 ? (long long)page[u] * a.ps + rest[u] : -1;
            if (a.positions) a.positions[y] = (long long)pos[u] + tok[u];
          }
        }
      }
    });
  // behind the last token
#pragma unroll 1
  for (int y = n_real + blockIdx.x * blockDim.x + threadIdx.x; y < a.max_new; y += gridDim.x * blockDim.x) {
    a.slots[y] = -1;
    if (a.positions) a.positions[y] = 0;
  }
}

// ---------------------------------------------------------------------------
__device__ __noinline__ long long div_call(long long a, long long b) { return a / b; }

struct WriteArgs {
  const char* K;
  const char* V;
  const long long* slots;
  char* Kc;
  char* Vc;
  long long k_stride, v_stride;  // bytes between tokens
  long long n_slots;
  int T, ps, shift;  // shift: log2(ps), or -1
  int nv, tx;        // vectors per token row; threads per token
  int hv;            // vectors per head row
};

// Copies token t's rows of K and V (Hkv x D each) to slot t's page: head h's
// row to [page][h][offset].  tx threads share a token, each takes every tx-th
// vector; four tokens' loads are issued before their stores.  Bound by memory:
// 213 MB of bf16 rows 34.6 us (91% of the copy's bandwidth), 142 MB of fp32
// 24.2 us (87%).
template <class Vec>
__global__ void __launch_bounds__(256) k_cache_write(const WriteArgs a) {
  pdl_wait();
  const int per = 256 / a.tx, v0 = threadIdx.x % a.tx, tg = threadIdx.x / a.tx;
  if (tg >= per) return;
  constexpr int U = 4;
#pragma unroll 1
  for (long long tb = (long long)blockIdx.x * per * U; tb < a.T; tb += (long long)gridDim.x * per * U) {
    long long off[U];  // first vector of the slot's row in head 0, or -1
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const long long t = tb + u * per + tg;
      const long long s = t < a.T ? a.slots[t] : -1;
      off[u] = -1;
      if (s >= a.n_slots) {
        if (v0 == 0) record_status(PT_STATUS_INVALID);
      } else if (s >= 0) {
        const long long page = a.shift >= 0 ? s >> a.shift : div_call(s, a.ps);
        const int row = (int)(s - page * a.ps);
        off[u] = page * ((long long)a.nv * a.ps) + (long long)row * a.hv;
      }
    }
#pragma unroll 1
    for (int v = v0; v < a.nv; v += a.tx) {
      const int h = v / a.hv;
      const long long in_page = (long long)h * a.ps * a.hv + (v - h * a.hv);
      Vec k[U], w[U];
#pragma unroll
      for (int u = 0; u < U; ++u)
        if (off[u] >= 0) {
          const long long t = tb + u * per + tg;
          k[u] = reinterpret_cast<const Vec*>(a.K + t * a.k_stride)[v];
          w[u] = reinterpret_cast<const Vec*>(a.V + t * a.v_stride)[v];
        }
#pragma unroll
      for (int u = 0; u < U; ++u)
        if (off[u] >= 0) {
          reinterpret_cast<Vec*>(a.Kc)[off[u] + in_page] = k[u];
          reinterpret_cast<Vec*>(a.Vc)[off[u] + in_page] = w[u];
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

bool overlap(const void* a, size_t na, const void* b, size_t nb) {
  const uintptr_t x = reinterpret_cast<uintptr_t>(a), y = reinterpret_cast<uintptr_t>(b);
  return na && nb && x < y + nb && y < x + na;
}

}  // namespace

extern "C" pt_status pt_cache_tables(const int32_t* held, const int32_t* added, const int32_t* start, int32_t n_rows,
                                     int32_t page_size, int32_t* tables, int32_t max_pages, int32_t* ring,
                                     int32_t ring_cap, const int64_t* counters, int32_t* lens, int32_t* row_ptr,
                                     int64_t* slots, int64_t* positions, int32_t max_new, int64_t* counters_out,
                                     cudaStream_t stream) {
  static const char* who = "pt_cache_tables";
  if (n_rows < 0 || max_pages < 0 || max_new < 0 || ring_cap < 1 || ring_cap > kTabMaxRing || page_size < 1) {
    set_error("%s: n_rows = %d, max_pages = %d, max_new = %d, ring_cap = %d or page_size = %d out of range", who,
              n_rows, max_pages, max_new, ring_cap, page_size);
    return PT_ERR_INVALID_ARG;
  }
  if ((long long)max_pages * page_size > INT_MAX / 2 || (long long)max_pages * n_rows > INT_MAX || max_new > kTabMaxNew) {
    set_error("%s: %d rows of %d pages of %d tokens, or %d new tokens, are out of range", who, n_rows, max_pages,
              page_size, max_new);
    return PT_ERR_INVALID_ARG;
  }
  if (n_rows > kTabMaxRows) {
    set_error("%s: %d rows, more than %d", who, n_rows, kTabMaxRows);
    return PT_ERR_UNSUPPORTED;
  }
  if (!ring || !counters || !counters_out || !row_ptr || (max_new > 0 && !slots) ||
      (n_rows > 0 && (!held || !added || !lens || (max_pages > 0 && !tables)))) {
    set_error("%s: a pointer is NULL", who);
    return PT_ERR_INVALID_ARG;
  }
  // every CTA reads the inputs while others write the outputs, and different warps write different outputs
  const size_t nb = (size_t)n_rows * 4;
  const struct {
    const void* p;
    size_t n;
  } in[] = {{held, nb}, {added, nb}, {start, start ? nb : 0}, {counters, 16}},
    out[] = {{lens, nb}, {row_ptr, nb + 4}, {slots, (size_t)max_new * 8}, {positions, positions ? (size_t)max_new * 8 : 0},
             {counters_out, 16}, {tables, nb * (size_t)max_pages}, {ring, (size_t)ring_cap * 4}};
  for (const auto& i : in)
    for (const auto& o : out)
      if (overlap(i.p, i.n, o.p, o.n)) {
        set_error("%s: an output overlaps an input", who);
        return PT_ERR_INVALID_ARG;
      }
  for (const auto& x : out)
    for (const auto& y : out)
      if (&x < &y && overlap(x.p, x.n, y.p, y.n)) {
        set_error("%s: two outputs overlap", who);
        return PT_ERR_INVALID_ARG;
      }
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess) {
    set_error("%s: no CUDA device", who);
    return PT_ERR_CUDA;
  }
  TabArgs a;
  a.held = held, a.added = added, a.start = start;
  a.counters = reinterpret_cast<const long long*>(counters);
  a.tables = tables, a.ring = ring, a.lens = lens, a.row_ptr = row_ptr;
  a.slots = reinterpret_cast<long long*>(slots);
  a.positions = reinterpret_cast<long long*>(positions);
  a.counters_out = reinterpret_cast<long long*>(counters_out);
  a.n = n_rows, a.ps = page_size, a.cap = ring_cap, a.max_pages = max_pages, a.max_new = max_new;
  const size_t smem = 12 * (((size_t)n_rows + 31) / 32 + 1);
  if (smem > 48 * 1024 && cudaFuncSetAttribute(k_cache_tables, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem) !=
                              cudaSuccess) {
    set_error("%s: no shared memory for %d rows", who, n_rows);
    return PT_ERR_CUDA;
  }
  // one CTA up to 4096 tokens and 512 rows; then enough for a run or two per warp
  const long long by_new = ((long long)max_new + 4095) / 4096, by_rows = ((long long)n_rows + 511) / 512;
  const int grid = (int)std::max(1LL, std::min<long long>(std::max(by_new, by_rows), num_sms(dev)));
  cudaError_t e;
  {
    ProfScope ps(stream, "cache_tables");
    e = launch_pdl(k_cache_tables, dim3(grid), dim3(kTabWarps * 32), smem, stream, a);
    count_launch();
  }
  return (pt_status)launch_status(who, e);
}

extern "C" pt_status pt_cache_write(const void* K, const void* V, int64_t k_stride, int64_t v_stride, pt_dtype dtype,
                                    int32_t T, int32_t Hkv, int32_t D, const int64_t* slots, void* Kc, void* Vc,
                                    int32_t n_pages, int32_t page_size, cudaStream_t stream) {
  static const char* who = "pt_cache_write";
  if (dtype != PT_BF16 && dtype != PT_F32) {
    set_error("%s: unknown dtype %d", who, (int)dtype);
    return PT_ERR_INVALID_ARG;
  }
  const int es = dtype == PT_BF16 ? 2 : 4;
  if (T < 0 || Hkv < 1 || D < 1 || n_pages < 0 || page_size < 1 || (long long)Hkv * D > INT_MAX / 4) {
    set_error("%s: T = %d, Hkv = %d, D = %d, n_pages = %d or page_size = %d out of range", who, T, Hkv, D, n_pages,
              page_size);
    return PT_ERR_INVALID_ARG;
  }
  if (k_stride < (int64_t)Hkv * D || v_stride < (int64_t)Hkv * D) {
    set_error("%s: tokens %lld and %lld elements apart, rows of %lld", who, (long long)k_stride, (long long)v_stride,
              (long long)Hkv * D);
    return PT_ERR_INVALID_ARG;
  }
  if (T == 0) return PT_OK;
  if (!K || !V || !slots || ((!Kc || !Vc) && n_pages > 0)) {
    set_error("%s: a pointer is NULL", who);
    return PT_ERR_INVALID_ARG;
  }
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess) {
    set_error("%s: no CUDA device", who);
    return PT_ERR_CUDA;
  }
  // the widest vector that the rows, the strides and the addresses allow
  int unit = 16;
  const uintptr_t all = reinterpret_cast<uintptr_t>(K) | reinterpret_cast<uintptr_t>(V) | reinterpret_cast<uintptr_t>(Kc) |
                        reinterpret_cast<uintptr_t>(Vc) | (uintptr_t)(D * es) | (uintptr_t)(k_stride * es) |
                        (uintptr_t)(v_stride * es);
  while (unit > es && (all & (unit - 1))) unit >>= 1;
  if (all & (es - 1)) {
    set_error("%s: a pointer is not aligned to its elements", who);
    return PT_ERR_INVALID_ARG;
  }
  WriteArgs a;
  a.K = static_cast<const char*>(K), a.V = static_cast<const char*>(V);
  a.slots = reinterpret_cast<const long long*>(slots);
  a.Kc = static_cast<char*>(Kc), a.Vc = static_cast<char*>(Vc);
  a.k_stride = k_stride * es, a.v_stride = v_stride * es;
  a.n_slots = (long long)n_pages * page_size;
  a.T = T, a.ps = page_size;
  a.shift = (page_size & (page_size - 1)) ? -1 : __builtin_ctz((unsigned)page_size);
  a.nv = (int)((long long)Hkv * D * es / unit);
  a.hv = D * es / unit;
  a.tx = 1;
  while (a.tx < 256 && a.tx < a.nv) a.tx <<= 1;
  const long long per = 256 / a.tx * 4;
  const int grid = (int)std::max(1LL, std::min<long long>((T + per - 1) / per, (long long)num_sms(dev) * 8));
  cudaError_t e;
  {
    ProfScope ps(stream, "cache_write");
    auto go = [&](auto kernel) { return launch_pdl(kernel, dim3(grid), dim3(256), 0, stream, a); };
    e = unit == 16  ? go(k_cache_write<uint4>)
        : unit == 8 ? go(k_cache_write<uint2>)
        : unit == 4 ? go(k_cache_write<uint32_t>)
                    : go(k_cache_write<unsigned short>);
    count_launch();
  }
  return (pt_status)launch_status(who, e);
}
