// pt_decode.cuh -- what the decoding attention's kernels share: the segments
// of the tree, their split over workers, and the partial results.
//
// A segment is a run of one node's cached tokens with the query rows that read
// it: every q head of every query token of every sample below the node, per kv
// head (rows = members * q_len * Hq / Hkv).  An item is (segment, tile of R
// rows, kv head); its units are tiles of BT tokens.  All items' units laid end
// to end (segments in order, in a segment the row tiles, in a row tile the kv
// heads) are cut into equal runs, one per worker, wherever the cuts fall: no
// worker has more than one unit above another, whatever the nodes' lengths,
// and a prompt that many samples share is read once per row tile.  What a
// worker computes of an item is a piece.  Worker w and item i have at most one
// piece in common and both grow along the line, so w + i numbers the pieces
// without a list: that is the slot of its partial result (each row's
// normalised output in fp32 and its base-2 log-sum-exp), and a row's pieces
// are found again from its path's segments alone.  The lengths are read on the
// device, so a captured graph follows them.
#pragma once

#include <cuda_bf16.h>

#include "pt_device.cuh"

namespace pt {

constexpr int kDecMaxSegs = 1 << 16;  // 8 bytes of shared memory per 32 segments

// Which of a node's tokens a segment covers.
enum : int {
  kSegFull = 0,  // all of them
  kSegBody = 1,  // a sample's own continuation up to its first query token, in whole groups of 16
  kSegTail = 2,  // the rest of it: the tokens that some of the queries must not see
};

// One class of segments (one kernel's share of the tree).
struct DecClass {
  const int4* seg;  // {node, kind, rows, first item}
  int nseg, nitems;
  // the class's part of the workspace
  long long* pref;  // [nseg + 1] units before each segment; units per worker
  float* lse;       // [slot][R]
  float* opart;     // [slot][R][D]
};

struct DecArgs {
  const int* node_ptr;   // [n_nodes + 1] CSR: samples through the node
  const int* node_samp;
  const int* leaf;       // [n_samples] last node of the sample's path
  const int* lens;       // [n_nodes]
  const int* tables;     // [n_nodes][max_pages]
  const int* q_count;    // [n_samples] or NULL
  const void* Q;
  const void* Kc;
  const void* Vc;
  long long q_stride;    // elements between query tokens
  int q_len, Hq, Hkv, g, D;
  int ps, max_pages, n_pages;
  int workers, min_units;
  float scale_log2;
};

__device__ __forceinline__ int dec_len(const DecArgs& a, int node, bool record) {
  const int len = a.lens[node];
  const long long cap = (long long)a.max_pages * a.ps;
  if (len < 0 || len > cap) {
    if (record) record_status(PT_STATUS_INVALID);
    return len < 0 ? 0 : (int)cap;
  }
  return len;
}

// Tokens [b, e) of a node of len tokens.
__device__ __forceinline__ void dec_range(const DecArgs& a, int kind, int len, int& b, int& e) {
  const int body = max(len - a.q_len + 1, 0) & ~15;
  b = kind == kSegTail ? body : 0;
  e = kind == kSegBody ? body : len;
}

__device__ __forceinline__ int dec_count(const DecArgs& a, int s) {
  return a.q_count ? min(max(a.q_count[s], 0), a.q_len) : a.q_len;
}

// Tiles of an item of the segment; 0 when its only sample has no queries.
template <int BT>
__device__ __forceinline__ int dec_tiles(const DecArgs& a, int4 sg, bool record) {
  int b, e;
  dec_range(a, sg.y, dec_len(a, sg.x, record), b, e);
  if (a.q_count) {
    const int p = a.node_ptr[sg.x];
    if (a.node_ptr[sg.x + 1] == p + 1 && dec_count(a, a.node_samp[p]) == 0) return 0;
  }
  return (e - b + BT - 1) / BT;
}

// Query row r of a segment: its sample, its query token's index and q head,
// and the first node token that it must not see.
struct DecRow {
  int s, j, head, lim;
};
__device__ __forceinline__ DecRow dec_row(const DecArgs& a, int node, int hk, int r, int len) {
  DecRow d;
  const int per = a.q_len * a.g, m = r / per, rest = r - m * per;
  d.j = rest / a.g;
  d.head = hk * a.g + rest - d.j * a.g;
  d.s = a.node_samp[a.node_ptr[node] + m];
  const int cnt = dec_count(a, d.s);
  d.lim = d.j >= cnt ? 0 : a.leaf[d.s] == node ? len - cnt + d.j + 1 : len;
  return d;
}

// Page that holds token t of the node (an entry out of range is recorded and
// page 0 read in its place).
__device__ __forceinline__ int dec_page(const DecArgs& a, int node, int pi) {
  const int p = a.tables[(size_t)node * a.max_pages + pi];
  if ((unsigned)p >= (unsigned)a.n_pages) {
    record_status(PT_STATUS_INVALID);
    return 0;
  }
  return p;
}

__device__ __forceinline__ long long warp_incl_scan64(long long v, int lane) {
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const long long u = __shfl_up_sync(0xffffffffu, v, o);
    if (lane >= o) v += u;
  }
  return v;
}

// Exclusive sums of the class's units over chunks of 32 segments, in shared
// memory (chunk[nc] = all of them); every thread of the block calls it.  Block
// 0 also leaves each segment's sum and the units per worker for the merge.
template <int R, int BT>
__device__ __forceinline__ long long dec_scan(const DecArgs& a, const DecClass& c, long long* chunk) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, nw = blockDim.x >> 5;
  const int nc = (c.nseg + 31) >> 5;
  for (int k = warp; k < nc; k += nw) {
    const int i = k * 32 + lane;
    long long u = 0;
    if (i < c.nseg) {
      const int4 sg = c.seg[i];
      u = (long long)((sg.z + R - 1) / R) * a.Hkv * dec_tiles<BT>(a, sg, blockIdx.x == 0);
    }
    u = warp_incl_scan64(u, lane);
    if (lane == 31) chunk[k] = u;
  }
  __syncthreads();
  if (warp == 0) {
    long long carry = 0;
    for (int k0 = 0; k0 < nc; k0 += 32) {
      const long long x = k0 + lane < nc ? chunk[k0 + lane] : 0;
      const long long s = warp_incl_scan64(x, lane);
      if (k0 + lane < nc) chunk[k0 + lane] = carry + s - x;
      carry += __shfl_sync(0xffffffffu, s, 31);
    }
    if (lane == 0) chunk[nc] = carry;
  }
  __syncthreads();
  const long long total = chunk[nc];
  const long long per = max((total + a.workers - 1) / a.workers, (long long)a.min_units);
  if (blockIdx.x == 0) {
    for (int k = warp; k < nc; k += nw) {
      const int i = k * 32 + lane;
      long long u = 0;
      if (i < c.nseg) {
        const int4 sg = c.seg[i];
        u = (long long)((sg.z + R - 1) / R) * a.Hkv * dec_tiles<BT>(a, sg, false);
      }
      const long long x = warp_incl_scan64(u, lane) - u;
      if (i < c.nseg) c.pref[i] = chunk[k] + x;
    }
    if (threadIdx.x == 0) c.pref[c.nseg] = per;
  }
  return per;
}

// A piece: units [t0, t1) of item `item` of segment `seg`.
struct DecPiece {
  int node, kind, rows, seg_item;  // the segment; the item's index in it
  int rt, hk;                      // row tile and kv head
  int t0, t1;
  long long slot;
};

// A worker's way along the line of units; every lane of a warp walks alike.
template <int R, int BT>
struct DecWalk {
  const DecArgs& a;
  const DecClass& c;
  const long long* chunk;
  long long pos, end, w;
  int k, nc;
  // the chunk's segments, one per lane
  int4 sg;
  int tiles;
  long long excl;

  __device__ __forceinline__ DecWalk(const DecArgs& a_, const DecClass& c_, const long long* ch, long long worker,
                                     long long per)
      : a(a_), c(c_), chunk(ch), w(worker) {
    nc = (c.nseg + 31) >> 5;
    const long long total = chunk[nc];
    pos = min(worker * per, total);
    end = min(pos + per, total);
    k = 0;
    if (pos < end) {
      for (int span = 1 << (31 - __clz(nc)); span; span >>= 1)
        if (k + span < nc && chunk[k + span] <= pos) k += span;
      load();
    }
  }
  __device__ __forceinline__ void load() {
    const int lane = threadIdx.x & 31, i = k * 32 + lane;
    sg = i < c.nseg ? c.seg[i] : make_int4(0, 0, 0, 0);
    tiles = i < c.nseg ? dec_tiles<BT>(a, sg, false) : 0;
    const long long u = (long long)((sg.z + R - 1) / R) * a.Hkv * tiles;
    excl = chunk[k] + warp_incl_scan64(u, lane) - u;
  }
  __device__ __forceinline__ bool next(DecPiece& p) {
    if (pos >= end) return false;
    while (pos >= chunk[k + 1]) {
      ++k;
      load();
    }
    int l = 0;
#pragma unroll
    for (int o = 16; o; o >>= 1) {
      const long long x = __shfl_sync(0xffffffffu, excl, l + o);
      if (x <= pos) l += o;
    }
    p.node = __shfl_sync(0xffffffffu, sg.x, l);
    p.kind = __shfl_sync(0xffffffffu, sg.y, l);
    p.rows = __shfl_sync(0xffffffffu, sg.z, l);
    const int item0 = __shfl_sync(0xffffffffu, sg.w, l);
    const int nt = __shfl_sync(0xffffffffu, tiles, l);
    const long long rel = pos - __shfl_sync(0xffffffffu, excl, l);
    p.seg_item = (int)(rel / nt);
    p.t0 = (int)(rel - (long long)p.seg_item * nt);
    p.t1 = (int)min((long long)nt, p.t0 + (end - pos));
    p.rt = p.seg_item / a.Hkv;
    p.hk = p.seg_item - p.rt * a.Hkv;
    p.slot = w + item0 + p.seg_item;
    pos += p.t1 - p.t0;
    return true;
  }
};

// The plan's classes.
enum : int { kDecSimt = 0, kDecRows = 1, kDecTile = 2, kDecClasses = 3 };
constexpr int kSimtR = 4, kSimtBT = 16;      // CUDA cores: rows and tokens of a tile, a warp per worker
constexpr int kRowsR = 16, kRowsBT = 16;     // mma, a warp per worker
constexpr int kTileR = 128, kTileBT = 128;   // tcgen05, a CTA per worker

}  // namespace pt

// The decoding plan of one tree and head layout.
struct pt_decodeplan {
  int device, sms;
  cudaStream_t stream;  // the build stream; memory goes back to the pool in its order
  void* mem;            // one pool allocation for every array below
  int32_t N, S, Hq, Hkv, q_len;
  int32_t* node_ptr;
  int32_t* node_samp;
  int32_t* leaf;
  struct Class {
    int4* seg;
    int32_t nseg, nitems;
  } cls[pt::kDecClasses];
  // a sample's segments, in path order: {class << 28 | segment, member}
  int32_t* path_ptr[2];  // [0] all segments of kDecSimt, [1] of the tensor-core classes
  int2* path_ent[2];
};

namespace pt {
// Tensor-core kernels (pt_decode_tc.cu).  Returns a PT_* status code.
bool decode_tc_supported(int D, int ps);
int decode_tc(const pt_decodeplan* p, DecArgs a, DecClass rows, DecClass tile, cudaStream_t s);
int take_status_decode_tc(cudaStream_t s);
constexpr int kRowsWarps = 8;
inline int dec_workers(const pt_decodeplan* p, int cls) {
  return cls == kDecSimt ? p->sms * 16 : cls == kDecRows ? p->sms * kRowsWarps : p->sms;
}
}  // namespace pt
