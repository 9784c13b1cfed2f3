// pt_decode.cuh -- what the decoding attention's kernels share: the segments
// of the tree, their split over workers, and the partial results.
//
// A segment is a run of one node's cached tokens with the query rows that read
// it: every q head of every query token of every sample below the node, per kv
// head (rows = members * q_len * Hq / Hkv).  An item is (segment, row tile, kv
// head); its units are its token tiles, and a few more for what beginning and
// ending it costs.  All items' units laid end to end (segments in order, in a
// segment the row tiles, in a row tile the kv heads) are cut into equal runs,
// one per worker, wherever the cuts fall: no worker has more than one unit
// above another, whatever the nodes' lengths, and a prompt that many samples
// share is read once per row tile.  What a worker computes of an item is a
// piece.  Worker w and item i have at most one piece in common and both grow
// along the line, so w + i numbers the pieces without a list: that is the slot
// of its partial result (each row's normalised output in fp32 and its base-2
// log-sum-exp), and a row's pieces are found again from its path's segments
// alone.  The lengths are read on the device, so a captured graph follows them.
#pragma once

#include <cuda_bf16.h>

#include <climits>

#include "pt_device.cuh"

namespace pt {

constexpr int kDecMaxNodes = 1 << 16;  // 4 or 8 bytes of shared memory per 32 nodes

// Row and token tiles of a class: 2^r rows, 2^t tokens; and the units that an
// item counts beside its tiles', what beginning and ending it costs.
struct DecTiling {
  int r, t, k;
};

// The plan's classes: a call uses kDecSimt, or kDecRows, or kDecRowsFew with
// kDecTile.
enum : int {
  kDecSimt = 0,     // CUDA cores: every node
  kDecRows = 1,     // mma: every node
  kDecRowsFew = 2,  // mma: nodes that few rows read, and the tails of the others
  kDecTile = 3,     // tcgen05: the rest
  kDecClasses = 4
};
constexpr DecTiling kSimt = {2, 4, 1};  // a warp per worker
constexpr DecTiling kRows = {4, 4, 2};  // a warp per worker
constexpr DecTiling kTile = {8, 7, 4};  // a CTA per worker; an item of up to 128 rows has two partial results
constexpr int kSimtR = 1 << kSimt.r, kSimtBT = 1 << kSimt.t;
constexpr int kRowsR = 1 << kRows.r, kRowsBT = 1 << kRows.t;
constexpr int kTileR = 1 << kTile.r, kTileBT = 1 << kTile.t;
// Which nodes the tile kernel takes, and when a call uses it: nodes that more
// than 32 rows read (three row tiles of the other kernel, which reads a node
// once for each), up to this head_dim, and only where that saves enough, since
// both kernels then start later than the one alone.  128 tokens of an item take
// an SM about 0.9 us for each tile of 16 rows, or 1.1 us for 128 rows and 2.2
// for 256; kTileMinGain is in such us, over the tokens of a full table row.
// 32 q heads over 8, head_dim 128, us on rows alone and with tiles: two prompts
// of 1024 tokens, 64 samples (gain 1560) 35 and 39; of 4096 tokens, 16 samples
// (1280) 35 and 38; four of 4096, 16 samples (2560) 46 and 39; two of 2048, 64
// samples (3120) 49 and 40; two of 32768, 64 samples 631 and 168.
// The host does not know the lengths, so a table that is much wider than its
// nodes are long counts as if they were: see pt_attn_decode.
constexpr int kTileMinRows = 33, kTileMaxD = 128;
constexpr float kTileMinGain = 2000.f;
// Element (row, column) of a tile-class partial result: groups of 8 columns, in
// each the rows one after another (D is a multiple of 8 there).
__host__ __device__ inline long long tile_at(int D, long long slot, int row, int col) {
  return ((slot * (D >> 3) + (col >> 3)) * kTileR + row) * 8 + (col & 7);
}
inline int dec_r(int cls) { return cls == kDecSimt ? kSimtR : cls == kDecTile ? kTileR : kRowsR; }

// Which of a node's tokens a class's segment covers.  A class has at most one
// segment per node, so a segment's number is its node's and its length is read
// beside its entry, not after it.
enum : int {
  kSegFull = 0,  // all of them
  kSegBody = 1,  // a sample's own continuation up to its first query token, in whole groups of 16
  kSegTail = 2,  // the rest of it: the tokens that some of the queries must not see
};

// One node of a class.
struct alignas(16) DecSeg {
  int rows_kind;  // rows | kind << 29; no rows: the class passes the node over
  int item0;      // items of the class before the node's
  int member0;    // the node's samples in DecArgs::member
  int solo;       // the node's only sample, else -1
  __host__ __device__ int rows() const { return rows_kind & ((1 << 29) - 1); }
  __host__ __device__ int kind() const { return (int)((unsigned)rows_kind >> 29); }
};

// One class of segments (one kernel's share of the tree).
struct DecClass {
  const DecSeg* seg;  // [n_nodes]
  int nseg, nitems;
  // the class's part of the workspace
  int* pref;        // [nseg + 1] units before each segment; units per worker
  float* lse;       // [slot][R]
  float* opart;     // [slot][R][D]; the tile class: see tile_at
};

struct DecArgs {
  const int* member;   // samples of each node, ascending; bit 31: the node is the sample's last
  const int* lens;     // [n_nodes]
  const int* tables;   // [n_nodes][max_pages]
  const int* q_count;  // [n_samples] or NULL
  const void* Q;
  const void* Kc;
  const void* Vc;
  long long q_stride;  // elements between query tokens
  int q_len, Hq, Hkv, g, D;
  int ps, max_pages, n_pages;
  int cap;             // max_pages * ps: tokens of a full table row
  int sms;
  int workers, min_units;  // CUDA cores
  int q_vec;           // Q's rows start on 16-byte boundaries
  float scale_log2;
};

__device__ __forceinline__ DecSeg load_seg(const DecSeg* p) {
  const int4 v = *reinterpret_cast<const int4*>(p);
  return DecSeg{v.x, v.y, v.z, v.w};
}

// A node's length, or the nearest that its table can hold.
__device__ __forceinline__ int dec_clamp(const DecArgs& a, int len) { return min(max(len, 0), a.cap); }

// Tokens [b, e) of a node of len tokens.
__device__ __forceinline__ void dec_range(const DecArgs& a, int kind, int len, int& b, int& e) {
  const int body = max(len - a.q_len + 1, 0) & ~15;
  b = kind == kSegTail ? body : 0;
  e = kind == kSegBody ? body : len;
}

__device__ __forceinline__ int dec_count(const DecArgs& a, int s) {
  return a.q_count ? min(max(a.q_count[s], 0), a.q_len) : a.q_len;
}

// Query row r of a segment: its query token, q head, and the first token of
// the node that it must not see.
struct DecRow {
  int tok, head, lim;
};
__device__ __forceinline__ DecRow dec_row(const DecArgs& a, int member0, int hk, int r, int len) {
  DecRow d;
  const int x = (int)((unsigned)r / (unsigned)a.g), h = r - x * a.g;
  int m = x, j = 0;
  if (a.q_len > 1) m = (int)((unsigned)x / (unsigned)a.q_len), j = x - m * a.q_len;
  const int mb = a.member[member0 + m], s = mb & INT_MAX;
  d.head = hk * a.g + h;
  d.tok = s * a.q_len + j;
  const int cnt = dec_count(a, s);
  d.lim = j >= cnt ? 0 : mb < 0 ? len - cnt + j + 1 : len;
  return d;
}

// Page that holds the node's tokens from pi * page_size (an entry out of range
// is recorded and page 0 read in its place).
__device__ __forceinline__ int dec_page(const DecArgs& a, int node, int pi) {
  const int p = a.tables[(size_t)node * a.max_pages + pi];
  if ((unsigned)p >= (unsigned)a.n_pages) {
    record_status(PT_STATUS_INVALID);
    return 0;
  }
  return p;
}

// Code that runs once per launch is kept short here: its instructions come from
// memory at about 2 GB/s per SM, 60 ns for every 128 bytes, and that is most of
// these kernels' fixed cost.  So loops that are not hot stay rolled, a kernel
// has one copy of the walk along the units, and units are counted in 32 bits
// (the host refuses trees whose items, times the tiles of a full table row,
// pass 2^31).
__device__ __forceinline__ int warp_incl_scan(int v, int lane) {
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int u = __shfl_up_sync(0xffffffffu, v, o);
    if (lane >= o) v += u;
  }
  return v;
}

// A tile of an item counts 2^wide units: in the tile class twice when the
// segment has more than half a row tile, which costs twice the time.
__device__ __forceinline__ int dec_wide(DecTiling g, int rows) { return g.r == kTile.r && rows > kTileR / 2; }

// Units of an item of so many tiles.
__device__ __forceinline__ int dec_line(DecTiling g, int rows, int tiles) {
  return tiles > 0 ? (tiles << dec_wide(g, rows)) + g.k : 0;
}

// Units of segment i, and what it takes to know them: its entry, its length
// and the tiles of one of its items (0 when its only sample has no queries).
__device__ __forceinline__ int dec_units(const DecArgs& a, const DecClass& c, DecTiling g, int i, DecSeg& sg, int& raw,
                                         int& tiles) {
  sg = DecSeg{0, 0, 0, -1};
  raw = 0;
  if (i < c.nseg) {
    raw = a.lens[i];
    sg = load_seg(c.seg + i);
  }
  int b, e;
  dec_range(a, sg.kind(), dec_clamp(a, raw), b, e);
  tiles = (e - b + (1 << g.t) - 1) >> g.t;
  if (a.q_count && sg.solo >= 0 && a.q_count[sg.solo] <= 0) tiles = 0;
  return ((sg.rows() + (1 << g.r) - 1) >> g.r) * a.Hkv * dec_line(g, sg.rows(), tiles);
}

// Exclusive sums of the units over chunks of 32 segments, in shared memory
// (chunk[nc] = all of them); every thread of the block calls it.  With cost, of
// two classes, the tile class first; cost[i], zero before, then receives class
// i's units.
__device__ __forceinline__ void dec_scan(const DecArgs& a, const DecClass& c0, const DecClass& c1, DecTiling g0,
                                         DecTiling g1, int* chunk0, int* chunk1, unsigned long long* cost) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, nw = blockDim.x >> 5;
  const int nc = (c0.nseg + 31) >> 5;
#pragma unroll 1
  for (int k = warp; k < nc; k += nw) {
#pragma unroll 1
    for (int i = 0; i < (cost ? 2 : 1); ++i) {
      DecSeg sg;
      int raw, tiles;
      const DecTiling g = {i ? g1.r : g0.r, i ? g1.t : g0.t, i ? g1.k : g0.k};
      const int u = dec_units(a, i ? c1 : c0, g, k * 32 + lane, sg, raw, tiles);
      if (blockIdx.x == 0 && (raw < 0 || raw > a.cap)) record_status(PT_STATUS_INVALID);
      const int sum = __reduce_add_sync(0xffffffffu, u);
      if (lane == 0) (i ? chunk1 : chunk0)[k] = sum;
      if (cost) {
        const unsigned x = u;
        const unsigned hi = __reduce_add_sync(0xffffffffu, x >> 16), lo = __reduce_add_sync(0xffffffffu, x & 0xffffu);
        if (lane == 0) atomicAdd(cost + i, ((unsigned long long)hi << 16) + lo);
      }
    }
  }
  __syncthreads();
  if (warp < (cost ? 2 : 1)) {
    int* chunk = warp ? chunk1 : chunk0;
    int carry = 0;
#pragma unroll 1
    for (int k0 = 0; k0 < nc; k0 += 32) {
      const int x = k0 + lane < nc ? chunk[k0 + lane] : 0;
      const int s = warp_incl_scan(x, lane);
      if (k0 + lane < nc) chunk[k0 + lane] = carry + s - x;
      carry += __shfl_sync(0xffffffffu, s, 31);
    }
    if (lane == 0) chunk[nc] = carry;
  }
  __syncthreads();
}

// Units per worker.
__device__ __forceinline__ int dec_share(int total, int workers, int min_units) {
  return max((int)(((unsigned)total + workers - 1) / (unsigned)workers), min_units);
}

// What the merge needs of a class: the units before each segment, and a
// worker's share.  One block of the grid calls it.
__device__ __forceinline__ void dec_publish(const DecArgs& a, const DecClass& c, DecTiling g, const int* chunk, int per) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, nw = blockDim.x >> 5;
#pragma unroll 1
  for (int k = warp; k < (c.nseg + 31) >> 5; k += nw) {
    DecSeg sg;
    int raw, tiles;
    const int i = k * 32 + lane, u = dec_units(a, c, g, i, sg, raw, tiles);
    const int x = warp_incl_scan(u, lane) - u;
    if (i < c.nseg) c.pref[i] = chunk[k] + x;
  }
  if (threadIdx.x == 0) c.pref[c.nseg] = per;
}

// A piece: tiles [t0, t1) of one item of segment `node`.
struct DecPiece {
  int node, len, kind, rows, member0;
  int rt, hk;  // row tile and kv head
  int t0, t1;
  int slot;
};

// A worker's way along the line of units; every lane of a warp walks alike.
struct DecWalk {
  const DecArgs& a;
  const DecClass& c;
  const DecTiling g;
  const int* chunk;
  int pos, end, w;
  int k, nc;
  // the chunk's segments, one per lane
  DecSeg sg;
  int raw, tiles, excl;

  __device__ __forceinline__ DecWalk(const DecArgs& a_, const DecClass& c_, DecTiling g_, const int* ch, int worker,
                                     int per)
      : a(a_), c(c_), g(g_), chunk(ch), w(worker) {
    nc = (c.nseg + 31) >> 5;
    const int total = chunk[nc];
    pos = (int)min((long long)worker * per, (long long)total);
    end = (int)min((long long)pos + per, (long long)total);
    k = 0;
    if (pos < end) {
#pragma unroll 1
      for (int span = 1 << (31 - __clz(nc)); span; span >>= 1)
        if (k + span < nc && chunk[k + span] <= pos) k += span;
    }
    --k;  // loaded by the first next()
  }
  __device__ __forceinline__ bool next(DecPiece& p) {
    if (pos >= end) return false;
    if (k < 0 || pos >= chunk[k + 1]) {
#pragma unroll 1
      do ++k;
      while (pos >= chunk[k + 1]);
      const int lane = threadIdx.x & 31, u = dec_units(a, c, g, k * 32 + lane, sg, raw, tiles);
      excl = chunk[k] + warp_incl_scan(u, lane) - u;
    }
    // the segment that holds pos: the last that starts at or before it
    const int l = 31 - __clz(__ballot_sync(0xffffffffu, excl <= pos));
    const int rk = __shfl_sync(0xffffffffu, sg.rows_kind, l);
    p.node = k * 32 + l;
    p.len = dec_clamp(a, __shfl_sync(0xffffffffu, raw, l));
    p.rows = rk & ((1 << 29) - 1);
    p.kind = (int)((unsigned)rk >> 29);
    p.member0 = __shfl_sync(0xffffffffu, sg.member0, l);
    const int item0 = __shfl_sync(0xffffffffu, sg.item0, l);
    const int wide = dec_wide(g, p.rows), nu = dec_line(g, p.rows, __shfl_sync(0xffffffffu, tiles, l));
    const int rel = pos - __shfl_sync(0xffffffffu, excl, l);
    const int it = (int)((unsigned)rel / (unsigned)nu), u0 = rel - it * nu, u1 = min(nu, u0 + (end - pos));
    // (a cut inside a tile leaves it to the piece before, one inside the item's own units gives that an empty piece)
    p.t0 = (max(u0 - g.k, 0) + wide) >> wide;
    p.t1 = (max(u1 - g.k, 0) + wide) >> wide;
    p.rt = (int)((unsigned)it / (unsigned)a.Hkv);
    p.hk = it - p.rt * a.Hkv;
    p.slot = w + item0 + it;
    pos += u1 - u0;
    return true;
  }
};

}  // namespace pt

// The decoding plan of one tree and head layout.
struct pt_decodeplan {
  int device, sms;
  cudaStream_t stream;  // the build stream; memory goes back to the pool in its order
  void* mem;            // one pool allocation for every array below
  int32_t N, S, Hq, Hkv, q_len;
  float tile_gain;      // what the tile kernel saves per 128 tokens of every node that it takes
  int32_t* member;
  struct Class {
    pt::DecSeg* seg;
    int32_t nitems;
  } cls[pt::kDecClasses];
  int32_t* path_ptr;  // [S + 1]
  int2* path_ent;     // {node, the sample's place among the node's}
};

namespace pt {
// Tensor-core kernels (pt_decode_tc.cu).  Returns a PT_* status code.
bool decode_tc_supported(int D, int ps);
int decode_tc(const pt_decodeplan* p, DecArgs a, const DecClass& rows, const DecClass& tile, cudaStream_t s);
int take_status_decode_tc(cudaStream_t s);
constexpr int kRowsWarps = 12;  // workers of the rows kernel per SM, at most
inline int dec_workers(const pt_decodeplan* p, int cls) {
  return cls == kDecSimt ? p->sms * 16 : cls == kDecTile ? p->sms : p->sms * kRowsWarps;
}
}  // namespace pt
