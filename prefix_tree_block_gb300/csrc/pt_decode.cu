// pt_decode.cu -- attention of every sample's newest tokens over its path
// through a cached prefix tree: the plan, the CUDA-core kernel (fp32, and the
// bf16 shapes that the tensor-core kernels do not take), the merge of the
// partial results, and the entry points.  pt_decode.cuh says how the work is
// cut.
//
// The rule is the forward's ("cp=1 shared-prefix prefix-tree attention for
// rollouts", PR description: full to the shared prompt, causal to itself): a
// query keeps every token of its path's earlier nodes and, of its own node,
// the tokens up to itself.
#include <cuda_bf16.h>

#include <algorithm>
#include <climits>
#include <cmath>
#include <cstring>
#include <type_traits>
#include <vector>

#include "pt.h"
#include "pt_decode.cuh"
#include "pt_internal.h"

namespace pt {
int take_status_decode(cudaStream_t s) {
  const int a = take_status_here(s), b = take_status_decode_tc(s);
  return a < 0 || b < 0 ? -1 : a | b;
}
}  // namespace pt

using namespace pt;

namespace {

__device__ __forceinline__ float to_f(float x) { return x; }
__device__ __forceinline__ float to_f(__nv_bfloat16 x) { return __bfloat162float(x); }

template <class E, int V>
struct alignas(sizeof(E) * V) VecOf {
  E e[V];
};

// ---------------------------------------------------------------------------
// CUDA cores: a warp per worker, kSimtR = 4 query rows, 8 tokens a step (4 at
// head dims over 128).
//
// Lanes hold the columns (DL each, VEC of them contiguous), so a token's key
// is one coalesced load, and four keys against four rows leave 16 partial dot
// products per lane.  These are summed over the lanes by halves: each exchange
// adds one half of the values to the partner's and keeps the other, 16
// shuffles for 16 sums where a butterfly for each would take 80, and lane l
// ends with row l/8, token (l/2) mod 4 of the group.  The softmax then runs on
// eight lanes a row.  About 28 instructions a token at head_dim 64 for 512
// bytes of fp32 keys and values.  Documents: 542 MB at head_dim 128, groups of
// two heads, 114 us (70% of the copy's bandwidth); 136 MB at 64, groups of
// three, 47 us (43%: latency and issue); bf16 in pages of 24 tokens, 69 MB at
// 128, groups of four, 40 us (25%: issue).  Every four rows read a node again:
// seven prompts of 7909 tokens, each under 62 samples (8 q heads over 4, head_dim
// 128: 227 MB, 124 rows a kv head), take 1155 us, 6 TB/s out of L2.  Head dims 65
// to 256 spill 40 to 60 bytes a thread, those from 65 to 127 that 4 does not
// divide 256: 128 registers, for two CTAs on an SM, are a little short.
// ---------------------------------------------------------------------------
template <class E, int DL, int VEC, bool TREE>
__global__ void __launch_bounds__(256, DL >= 16 ? 1 : 2) k_decode_simt(const DecArgs a, const DecClass c) {
  pdl_wait();
  extern __shared__ int chunk[];
  dec_scan(a, TREE, c, c, kSimt, kSimt, chunk, nullptr, nullptr);
  const int per = dec_share(chunk[(c.nseg + 31) >> 5], a.workers, a.min_units);
  if (blockIdx.x == gridDim.x - 1) dec_publish(a, TREE, c, kSimt, chunk, per);
  const int lane = threadIdx.x & 31;
  constexpr int R = kSimtR, NV = DL / VEC;
  constexpr int STEP = DL <= 4 ? 8 : 4;  // tokens, as registers allow
  constexpr bool EARLY = DL <= 4;        // and whether for their values beside their keys
  using V = VecOf<E, VEC>;
  const E* Qp = static_cast<const E*>(a.Q);
  DecWalk walk(a, TREE, c, kSimt, chunk, (int)blockIdx.x * 8 + (threadIdx.x >> 5), per);
  DecPiece p;
  const int my_r = lane >> 3;  // the row whose scores this lane holds
#pragma unroll 1
  while (walk.next(p)) {
    int b, e;
    dec_range(a, TREE, p.kind, p.len, b, e);
    float q[R][DL], acc[R][DL];
    int lim_max = 0, lim_min = INT_MAX, my_lim = 0;  // (the least of the rows there are)
    int lim[R];
    int my_lo = 0, my_mask = -1, my_self = 0;  // TREE: what the row sees in any case, its mask's row, its own draft
#pragma unroll
    for (int r = 0; r < R; ++r) {
      const int row = p.rt * R + r;
      lim[r] = 0;
      const E* src = nullptr;
      if (row < p.rows) {
        DecRow d;
        if constexpr (TREE) {
          const DecTreeRow tr = dec_tree_row(a, p.member0, p.hk, row, p.len);
          d = tr.d;
          lim_min = min(lim_min, tr.lo);
          if (r == my_r) my_lo = tr.lo, my_mask = tr.mask_row, my_self = tr.mask_row % a.q_len;
        } else {
          d = dec_row(a, p.member0, p.hk, row, p.len);
          lim_min = min(lim_min, d.lim);
        }
        lim[r] = d.lim;
        src = Qp + (long long)d.tok * a.q_stride + (long long)d.head * a.D;
      }
      lim_max = max(lim_max, lim[r]);
      if (r == my_r) my_lim = lim[r];
#pragma unroll
      for (int i = 0; i < DL; ++i) {
        const int col = (i / VEC * 32 + lane) * VEC + i % VEC;
        q[r][i] = src && col < a.D ? to_f(src[col]) * a.scale_log2 : 0.f;
        acc[r][i] = 0.f;
      }
    }
    float m = -INFINITY, l = 0.f;  // of row my_r, the same on its eight lanes
    const int end = min(min(b + p.t1 * kSimtBT, e), lim_max);
    // lane i's row of the cache: token kv0 + i (past the last token: the last again, so that every load may be issued)
    auto row_of = [&](int kv0) -> long long {
      const int kv = min(kv0 + (lane & (STEP - 1)), end - 1), pi = kv / a.ps;
      return (((long long)dec_page(a, p.node, pi) * a.Hkv + p.hk) * a.ps + (kv - pi * a.ps)) * a.D;
    };
    long long next = b + p.t0 * kSimtBT < end ? row_of(b + p.t0 * kSimtBT) : 0;
#pragma unroll 1
    for (int kv0 = b + p.t0 * kSimtBT; kv0 < end; kv0 += STEP) {
      // this step's values are loaded with its keys, and the next step's pages are looked up now
      const long long off = next;
      unsigned sees = 0xffffu;  // TREE: the step's tokens that row my_r sees
      if (TREE && kv0 + STEP > lim_min) sees = dec_sees(a, my_lo, my_lim, my_mask, my_self, kv0);
      V kk[STEP][NV], vv[EARLY ? STEP : 1][NV];
#pragma unroll
      for (int u = 0; u < STEP; ++u) {
        const long long o = __shfl_sync(0xffffffffu, off, u);
        const E* kp = static_cast<const E*>(a.Kc) + o;
        const E* vp = static_cast<const E*>(a.Vc) + o;
#pragma unroll
        for (int v = 0; v < NV; ++v) {
          const int col = (v * 32 + lane) * VEC;
          kk[u][v] = col < a.D ? *reinterpret_cast<const V*>(kp + col) : V{};
          if constexpr (EARLY) vv[u][v] = col < a.D ? *reinterpret_cast<const V*>(vp + col) : V{};
        }
      }
      if (kv0 + STEP < end) next = row_of(kv0 + STEP);
      float s[2] = {-INFINITY, -INFINITY};
      int hidden = 0;  // TREE: which of the two the row does not see
#pragma unroll
      for (int gq = 0; gq < STEP / 4; ++gq) {
        float d[16];
#pragma unroll
        for (int i = 0; i < 16; ++i) d[i] = 0.f;
#pragma unroll
        for (int u = 0; u < 4; ++u)
#pragma unroll
          for (int v = 0; v < NV; ++v)
#pragma unroll
            for (int x = 0; x < VEC; ++x)
#pragma unroll
              for (int r = 0; r < R; ++r)
                d[r * 4 + u] = fmaf(q[r][v * VEC + x], to_f(kk[gq * 4 + u][v].e[x]), d[r * 4 + u]);
        // 16 sums over 32 lanes: lane l keeps value l >> 1
#pragma unroll
        for (int h = 8, o = 16; h; h >>= 1, o >>= 1) {
          const bool hi = lane & o;
#pragma unroll
          for (int i = 0; i < h; ++i) {
            const float give = hi ? d[i] : d[i + h], keep = hi ? d[i + h] : d[i];
            d[i] = keep + __shfl_xor_sync(0xffffffffu, give, o);
          }
        }
        d[0] += __shfl_xor_sync(0xffffffffu, d[0], 1);
        const int kv = kv0 + gq * 4 + ((lane >> 1) & 3);
        const bool in = kv < end && (TREE ? sees >> (kv - kv0) & 1u : kv < my_lim);
        s[gq] = in ? d[0] : -INFINITY;
        if (TREE && !in) hidden |= 1 << gq;
      }
      float mt = fmaxf(s[0], s[1]);
      mt = fmaxf(mt, __shfl_xor_sync(0xffffffffu, mt, 2));
      mt = fmaxf(mt, __shfl_xor_sync(0xffffffffu, mt, 4));
      const float mn = fmaxf(m, mt), ref = mn == -INFINITY ? 0.f : mn;
      const float al = mn == m ? 1.f : ex2(m - ref);
      m = mn;
      s[0] = ex2(s[0] - ref), s[1] = ex2(s[1] - ref);
      float sum = s[0] + s[1];
      sum += __shfl_xor_sync(0xffffffffu, sum, 2);
      sum += __shfl_xor_sync(0xffffffffu, sum, 4);
      l = fmaf(l, al, sum);
      if (__any_sync(0xffffffffu, al != 1.f)) {
#pragma unroll
        for (int r = 0; r < R; ++r) {
          const float ar = __shfl_sync(0xffffffffu, al, r * 8);
#pragma unroll
          for (int i = 0; i < DL; ++i) acc[r][i] *= ar;
        }
      }
      if constexpr (TREE) {  // (weights are not negative: below 0 says that the token is not seen)
        if (hidden & 1) s[0] = -1.f;
        if (hidden & 2) s[1] = -1.f;
      }
      auto add_values = [&](auto masked) {
#pragma unroll
        for (int i = 0; i < STEP; ++i) {
          float pr[R];
#pragma unroll
          for (int r = 0; r < R; ++r) pr[r] = __shfl_sync(0xffffffffu, s[i >> 2], r * 8 + (i & 3) * 2);
          const E* vp = static_cast<const E*>(a.Vc) + (EARLY ? 0 : __shfl_sync(0xffffffffu, off, i));
#pragma unroll
          for (int v = 0; v < NV; ++v) {
            const int col = (v * 32 + lane) * VEC;
            const V w = EARLY ? vv[EARLY ? i : 0][v] : col < a.D ? *reinterpret_cast<const V*>(vp + col) : V{};
#pragma unroll
            for (int x = 0; x < VEC; ++x)
#pragma unroll
              for (int r = 0; r < R; ++r) {  // a value that the row must not see does not reach it, whatever it is
                const float y = fmaf(pr[r], to_f(w.e[x]), acc[r][v * VEC + x]);
                const bool in = !masked || (TREE ? !(pr[r] < 0.f) : kv0 + i < lim[r]);
                acc[r][v * VEC + x] = in ? y : acc[r][v * VEC + x];
              }
          }
        }
      };
      if (kv0 + STEP <= lim_min)  // every row sees all of them: half the instructions
        add_values(std::false_type{});
      else
        add_values(std::true_type{});
    }
    // the piece's partial result
#pragma unroll
    for (int r = 0; r < R; ++r) {
      if (p.rt * R + r >= p.rows) break;
      const float lr = __shfl_sync(0xffffffffu, l, r * 8), mr = __shfl_sync(0xffffffffu, m, r * 8);
      const float inv = lr == 0.f ? 0.f : 1.f / lr;
      const long long row = (long long)p.slot * R + r;
      if (lane == 0) c.lse[row] = lr == 0.f ? -INFINITY : mr + log2f(lr);
#pragma unroll
      for (int i = 0; i < DL; ++i) {
        const int col = (i / VEC * 32 + lane) * VEC + i % VEC;
        if (col < a.D) c.opart[row * a.D + col] = acc[r][i] * inv;
      }
    }
  }
}

// ---------------------------------------------------------------------------
// Merge: O = sum_p 2^(lse_p - LSE) O_p over a row's pieces, in path order and
// along each segment, so the sum's order is fixed.  A unit is one query token's
// GH q heads of one kv head: their rows lie side by side in every piece (GH
// divides the group and a row tile), so the pieces are looked up once for all
// of them, the path's entries side by side, one per lane.  W warps share a
// unit, each takes every W-th piece, lanes the columns; several pieces are
// loaded at a time.  With few rows a unit gets four warps and one head (latency);
// with many, one warp and, with the most, four heads: the lookup's
// instructions bound it then.
// ---------------------------------------------------------------------------
struct MergeArgs {
  DecArgs d;
  DecClass c0, c1;  // c1: the tile class, or none
  DecTiling g0;       // c0's
  const int* path_ptr;
  const int2* path_ent;
  int n_samples, units;
  void* O;
  float* LSE;
};

template <int VEC, int NV, int GH>
struct MergeAcc {
  float mx[GH], sum[GH], acc[GH][NV * VEC];
  int turn;  // pieces so far, modulo the warps
};

// The pieces of as many path entries as the lanes hold, one per lane: node, its
// segment and length, the sample's place among the node's.  With TWO classes the
// upper half of the lanes holds the same entries in the tile class (both in one
// pass: 16-token drafts 56.1 -> 54.0 us, 32768-token prompts 165.6 -> 163.4).
template <int VEC, int NV, int GH, int W, bool TWO>
__device__ __forceinline__ void merge_pieces(const MergeArgs& m, int node, const DecSeg& sg, int raw, int mem,
                                            int j, int hk, int h0, int warp, int lane, MergeAcc<VEC, NV, GH>& s) {
  using V = VecOf<float, VEC>;
  const DecArgs& a = m.d;
  const bool mine = TWO && lane >= 16;  // this lane's entry is of the tile class
  const int* pref = mine ? m.c1.pref : m.c0.pref;
  int count = 0, two = 0;
  int row0 = 0;  // the row in the first piece, over all slots
  if (sg.rows_kind) {
    const int rl = mine ? kTile.r : m.g0.r, bl = mine ? kTile.t : m.g0.t;
    const int before = pref[node], per = pref[m.c0.nseg];
    int b, e;
    dec_range(a, a.mask, sg.kind(), dec_clamp(a, raw), b, e);
    const int tiles = (e - b + (1 << bl) - 1) >> bl;
    if (tiles > 0) {
      const int row = (mem * a.q_len + j) * a.g + h0, rt = row >> rl, it = rt * a.Hkv + hk;
      two = mine && sg.rows() - (rt << rl) <= kTileR / 2;
      const int nu = dec_line(DecTiling{rl, bl, mine ? dec_tile(a.mask).k : m.g0.k}, sg.rows(), tiles);
      const unsigned u0 = before + it * nu, w0 = u0 / (unsigned)per, w1 = (u0 + nu - 1) / (unsigned)per;
      row0 = (((int)w0 + sg.item0 + it) << rl) + row - (rt << rl);
      count = (int)(w1 - w0 + 1) << two;
    }
  }
  int incl = count;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int u = __shfl_up_sync(0xffffffffu, incl, o);
    if (lane >= o) incl += u;
  }
  const int excl = incl - count, total = __shfl_sync(0xffffffffu, incl, 31);
  constexpr int U = GH * NV * VEC > 8 ? 2 : 4;  // pieces in flight
#pragma unroll 1
  for (int x0 = W == 1 ? 0 : (warp - s.turn) & (W - 1); x0 < total; x0 += W * U) {
    float ls[U][GH];
    V o[U][GH][NV];
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const int x = min(x0 + W * u, total - 1);
      const int l = 31 - __clz(__ballot_sync(0xffffffffu, excl <= x));
      const int y = x - __shfl_sync(0xffffffffu, excl, l), tw = __shfl_sync(0xffffffffu, two, l);
      const bool tile = TWO && l >= 16;
      const int rl = tile ? kTile.r : m.g0.r;
      // a row's columns: groups of 8, far apart in the tile class and side by side in the others
      const int row_step = tile ? 8 : a.D, col_step = tile ? kTileR * 8 : 8;
      const int at = __shfl_sync(0xffffffffu, row0, l) + ((y >> tw) << rl) + (y & tw) * (kTileR / 2);
      const bool in = x0 + W * u < total;
      const float* src = (tile ? m.c1.opart : m.c0.opart) + (long long)(at >> rl) * (a.D << rl) + (at & ((1 << rl) - 1)) * row_step;
#pragma unroll
      for (int i = 0; i < NV; ++i) {
        const int col = (i * 32 + lane) * VEC;
        const float* from = src + (col >> 3) * col_step + (col & 7);
#pragma unroll
        for (int h = 0; h < GH; ++h) o[u][h][i] = in && col < a.D ? *reinterpret_cast<const V*>(from + h * row_step) : V{};
      }
#pragma unroll
      for (int h = 0; h < GH; ++h) ls[u][h] = in ? (tile ? m.c1.lse : m.c0.lse)[at + h] : -INFINITY;
    }
#pragma unroll
    for (int u = 0; u < U; ++u)
#pragma unroll
      for (int h = 0; h < GH; ++h) {
        // (a piece that kept nothing weighs nothing, whatever the slot held)
        const float mn = fmaxf(s.mx[h], ls[u][h]), ref = mn == -INFINITY ? 0.f : mn;
        const float al = ex2(s.mx[h] - ref), f = ex2(ls[u][h] - ref);
        s.mx[h] = mn;
        s.sum[h] = fmaf(s.sum[h], al, f);
#pragma unroll
        for (int i = 0; i < NV; ++i)
#pragma unroll
          for (int x = 0; x < VEC; ++x) s.acc[h][i * VEC + x] = fmaf(s.acc[h][i * VEC + x], al, ls[u][h] == -INFINITY ? 0.f : f * o[u][h][i].e[x]);
      }
  }
  s.turn = (s.turn + total) & (W - 1);
}

// CTAs per SM: said so that the loads of a round get registers of their own
// (without it the compiler saves some and one round becomes several: documents
// at head_dim 256 17.5 -> 16.6 us, GRPO batch 12.3 -> 11.6).
constexpr int merge_ctas(int floats) { return floats <= 4 ? 7 : floats <= 8 ? 4 : 1; }

template <class E, int VEC, int NV, int GH, int W, bool TWO>
__global__ void __launch_bounds__(128, merge_ctas(GH* NV* VEC)) k_decode_merge(const MergeArgs m) {
  __shared__ float sm_m[W][GH], sm_l[W][GH];
  static_assert(W == 1 || W == 4, "a CTA is four warps");
  __shared__ VecOf<float, VEC> sm_o[W == 1 ? 1 : W][W == 1 ? 1 : GH][W == 1 ? 1 : NV * 32];
  const DecArgs& a = m.d;
  const int lane = threadIdx.x & 31, warp = W == 1 ? 0 : threadIdx.x >> 5;
  const int unit = W == 1 ? blockIdx.x * 4 + (threadIdx.x >> 5) : blockIdx.x;
  if (unit >= m.units) {
    pdl_wait();  // (so that the grid does not end before the one before it)
    return;
  }
  const int groups = a.Hq / GH, tok = unit / groups, head = (unit - tok * groups) * GH;
  const int s = a.q_len > 1 ? tok / a.q_len : tok, j = tok - s * a.q_len, hk = head / a.g, h0 = head - hk * a.g;
  // What the kernels before do not write is read while they end: they were
  // launched after all that came before them had ended.
  const int k0 = m.path_ptr[s], k1 = m.path_ptr[s + 1];
  int2 en = make_int2(0, 0);
  DecSeg sg = DecSeg{0, 0, 0, -1};
  int raw = 0;
  constexpr int AT_ONCE = TWO ? 16 : 32;  // path entries
  const DecSeg* segs = TWO && lane >= 16 ? m.c1.seg : m.c0.seg;
  const bool any = !TWO || (lane >= 16 ? m.c1.nitems : m.c0.nitems) > 0;
  auto look = [&](int k) {
    sg.rows_kind = 0;
    const int at = k + (TWO ? lane & 15 : lane);
    if (at < k1) {
      en = m.path_ent[at];
      raw = a.lens[en.x];
      if (any) sg = load_seg(segs + en.x);
    }
  };
  look(k0);
  bool idle = false;
  if (a.q_count) {
    const int n = a.q_count[s];
    if ((n < 0 || n > a.q_len) && lane == 0) record_status(PT_STATUS_INVALID);
    idle = j >= dec_count(a, s);  // the row stays as it was
  }
  pdl_wait();
  if (idle) return;
  MergeAcc<VEC, NV, GH> r;
  r.turn = 0;
#pragma unroll
  for (int h = 0; h < GH; ++h) {
    r.mx[h] = -INFINITY, r.sum[h] = 0.f;
#pragma unroll
    for (int i = 0; i < NV * VEC; ++i) r.acc[h][i] = 0.f;
  }
#pragma unroll 1
  for (int k = k0;;) {
    merge_pieces<VEC, NV, GH, W, TWO>(m, en.x, sg, raw, en.y, j, hk, h0, warp, lane, r);
    k += AT_ONCE;
    if (k >= k1) break;
    look(k);
  }
  using V = VecOf<float, VEC>;
  using VE = VecOf<E, VEC>;
  auto put = [&](int h, int i, const V& v, float inv) {
    const int col = (i * 32 + lane) * VEC;
    if (col < a.D) {
      VE w;
#pragma unroll
      for (int x = 0; x < VEC; ++x) {
        if constexpr (sizeof(E) == 2)
          w.e[x] = __float2bfloat16_rn(v.e[x] * inv);
        else
          w.e[x] = v.e[x] * inv;
      }
      *reinterpret_cast<VE*>(static_cast<E*>(m.O) + ((long long)tok * a.Hq + head + h) * a.D + col) = w;
    }
  };
  auto put_lse = [&](int h, float top, float all) {
    m.LSE[(long long)(head + h) * m.n_samples * a.q_len + tok] =
        all == 0.f ? -INFINITY : (top + log2f(all)) * 0.69314718055994531f;
  };
  if constexpr (W == 1) {
#pragma unroll
    for (int h = 0; h < GH; ++h) {
      const float inv = r.sum[h] == 0.f ? 0.f : 1.f / r.sum[h];
#pragma unroll
      for (int i = 0; i < NV; ++i) {
        V v;
#pragma unroll
        for (int x = 0; x < VEC; ++x) v.e[x] = r.acc[h][i * VEC + x];
        put(h, i, v, inv);
      }
      if (lane == 0) put_lse(h, r.mx[h], r.sum[h]);
    }
  } else {
#pragma unroll
    for (int h = 0; h < GH; ++h) {
      if (lane == 0) sm_m[warp][h] = r.mx[h], sm_l[warp][h] = r.sum[h];
#pragma unroll
      for (int i = 0; i < NV; ++i) {
        V v;
#pragma unroll
        for (int x = 0; x < VEC; ++x) v.e[x] = r.acc[h][i * VEC + x];
        sm_o[warp][h][i * 32 + lane] = v;
      }
    }
    __syncthreads();
    // warp w joins every W-th (head, column group)
#pragma unroll 1
    for (int y = warp; y < GH * NV; y += W) {
      const int h = y / NV, i = y - h * NV;
      float top = -INFINITY, all = 0.f, f[W];
#pragma unroll
      for (int w = 0; w < W; ++w) top = fmaxf(top, sm_m[w][h]);
#pragma unroll
      for (int w = 0; w < W; ++w) {
        f[w] = sm_m[w][h] == -INFINITY ? 0.f : ex2(sm_m[w][h] - top);
        all = fmaf(f[w], sm_l[w][h], all);
      }
      V v = {};
#pragma unroll
      for (int w = 0; w < W; ++w) {
        const V o = sm_o[w][h][i * 32 + lane];
#pragma unroll
        for (int x = 0; x < VEC; ++x) v.e[x] = fmaf(f[w], o.e[x], v.e[x]);
      }
      put(h, i, v, all == 0.f ? 0.f : 1.f / all);
      if (i == 0 && lane == 0) put_lse(h, top, all);
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

size_t pad256(size_t b) { return (b + 255) & ~size_t(255); }

// Bytes of a class's part of the workspace.
size_t class_bytes(const pt_decodeplan* p, int cls, int D) {
  const pt_decodeplan::Class& c = p->cls[cls];
  if (!c.nitems) return 0;
  const size_t R = dec_r(cls), slots = (size_t)c.nitems + dec_workers(p, cls);
  return pad256(4 * ((size_t)p->N + 1)) + pad256(4 * slots * R) + pad256(4 * slots * R * D);
}

DecClass class_args(const pt_decodeplan* p, int cls, int D, char*& ws) {
  const pt_decodeplan::Class& c = p->cls[cls];
  DecClass d = {};
  d.seg = c.seg;
  d.nseg = p->N;
  d.nitems = c.nitems;
  if (!c.nitems) return d;
  const size_t R = dec_r(cls), slots = (size_t)c.nitems + dec_workers(p, cls);
  d.pref = reinterpret_cast<int*>(ws), ws += pad256(4 * ((size_t)p->N + 1));
  d.lse = reinterpret_cast<float*>(ws), ws += pad256(4 * slots * R);
  d.opart = reinterpret_cast<float*>(ws), ws += pad256(4 * slots * R * D);
  return d;
}

// Whether a tensor-core call splits the nodes between the two kernels: never at
// this head_dim, or by the tokens of a full table row.
bool may_tile(const pt_decodeplan* p, int D) { return D <= kTileMaxD && p->cls[kDecTile].nitems > 0; }
bool use_tiles(const pt_decodeplan* p, int D, int cap) {
  return may_tile(p, D) && p->tile_gain * (float)cap / 128.f >= kTileMinGain;
}

size_t ws_bytes(const pt_decodeplan* p, int D) {
  size_t n = std::max(class_bytes(p, kDecSimt, D), (size_t)256);
  if (may_tile(p, D)) n = std::max(n, class_bytes(p, kDecRowsFew, D) + class_bytes(p, kDecTile, D));
  n = std::max(n, class_bytes(p, kDecRows, D));
  return n;
}

template <class E, bool TREE>
cudaError_t launch_simt(const DecArgs& a, const DecClass& c, int grid, size_t smem, cudaStream_t s) {
  const int D = a.D;
  auto go = [&](auto kernel) { return launch_pdl(kernel, dim3(grid), dim3(256), smem, s, a, c); };
  if (D <= 32) return go(k_decode_simt<E, 1, 1, TREE>);
  if constexpr (sizeof(E) == 4) {  // (bf16 head dims are multiples of 8)
    if (D % (D <= 64 ? 2 : 4)) {
      if (D <= 64) return go(k_decode_simt<E, 2, 1, TREE>);
      if (D <= 128) return go(k_decode_simt<E, 4, 1, TREE>);
      return D <= 256 ? go(k_decode_simt<E, 8, 1, TREE>) : go(k_decode_simt<E, 16, 1, TREE>);
    }
  }
  if (D <= 64) return go(k_decode_simt<E, 2, 2, TREE>);
  if (D <= 128) return go(k_decode_simt<E, 4, 4, TREE>);
  return D <= 256 ? go(k_decode_simt<E, 8, 4, TREE>) : go(k_decode_simt<E, 16, 4, TREE>);
}

// Rows of a call: below the first number a merge unit is one head on four warps
// (1024 rows of the 2 x 4096-token batch: the whole call 34.6 us, 38.4 with a
// warp each), from it on one head on one warp (2048 rows of four such prompts:
// 39.1 us, 40.1 with four warps; 4096 rows: 86 us, 89 with four heads a warp),
// and from the second on four heads on one warp where they divide the group
// (8192 rows: 53.5 us, 55.9 with two heads).
constexpr int kMergeManyRows = 2048, kMergeMostRows = 8192;

template <class E, int GH, int W, bool TWO>
cudaError_t launch_merge(MergeArgs m, cudaStream_t s) {
  m.units = m.n_samples * m.d.q_len * (m.d.Hq / GH);
  const int grid = W == 1 ? (m.units + 3) / 4 : m.units, D = m.d.D;
  auto go = [&](auto kernel) { return launch_pdl(kernel, dim3(grid), dim3(128), 0, s, m); };
  if (D <= 32) return go(k_decode_merge<E, 1, 1, GH, W, TWO>);
  if constexpr (sizeof(E) == 4) {  // (bf16 head dims are multiples of 8)
    if (D % (D <= 64 ? 2 : 4)) {
      if (D <= 64) return go(k_decode_merge<E, 1, 2, GH, W, TWO>);
      if (D <= 128) return go(k_decode_merge<E, 1, 4, GH, W, TWO>);
      if constexpr (GH == 1)
        if (D > 256) return go(k_decode_merge<E, 1, 16, GH, W, TWO>);
      return go(k_decode_merge<E, 1, 8, GH, W, TWO>);
    }
  }
  if (D <= 64) return go(k_decode_merge<E, 2, 1, GH, W, TWO>);
  if constexpr (!TWO) {  // (tiles: up to kTileMaxD; several heads to a warp: up to 256)
    if constexpr (GH == 1)
      if (D > 256) return go(k_decode_merge<E, 4, 4, GH, W, TWO>);
    if (D > 128) return go(k_decode_merge<E, 4, 2, GH, W, TWO>);
  }
  return go(k_decode_merge<E, 4, 1, GH, W, TWO>);
}

template <class E, bool TWO>
cudaError_t launch_merge(const MergeArgs& m, cudaStream_t s) {
  const long long rows = (long long)m.n_samples * m.d.q_len * m.d.Hq;
  const bool heads = m.d.g % 4 == 0 && m.d.D <= 256 && rows >= kMergeMostRows;
  if (heads) return launch_merge<E, 4, 1, TWO>(m, s);
  return rows < kMergeManyRows ? launch_merge<E, 1, 4, TWO>(m, s) : launch_merge<E, 1, 1, TWO>(m, s);
}

}  // namespace

extern "C" pt_status pt_decode_plan(int32_t n_nodes, const int32_t* path_ptr, const int32_t* path_nodes,
                                    int32_t n_samples, int32_t Hq, int32_t Hkv, int32_t q_len, cudaStream_t stream,
                                    pt_decodeplan** out) {
  static const char* who = "pt_decode_plan";
  if (!out) {
    set_error("%s: out is NULL", who);
    return PT_ERR_INVALID_ARG;
  }
  *out = nullptr;
  if (n_nodes < 0 || n_samples < 0 || !path_ptr || (n_samples > 0 && !path_nodes)) {
    set_error("%s: null array or negative count", who);
    return PT_ERR_INVALID_ARG;
  }
  if (Hq <= 0 || Hkv <= 0 || Hq % Hkv != 0) {
    set_error("%s: Hq = %d must be a positive multiple of Hkv = %d", who, Hq, Hkv);
    return PT_ERR_INVALID_ARG;
  }
  if (q_len < 1) {
    set_error("%s: q_len = %d, at least 1 wanted", who, q_len);
    return PT_ERR_INVALID_ARG;
  }
  const int N = n_nodes, S = n_samples, g = Hq / Hkv;
  if ((long long)S * q_len * Hq >= 1 << 29) {
    set_error("%s: %d samples of %d tokens and %d heads are out of range", who, S, q_len, Hq);
    return PT_ERR_INVALID_ARG;
  }
  if (N > kDecMaxNodes) {
    set_error("%s: %d nodes, more than %d", who, N, kDecMaxNodes);
    return PT_ERR_UNSUPPORTED;
  }
  if (path_ptr[0] != 0) {
    set_error("%s: path_ptr[0] must be 0", who);
    return PT_ERR_INVALID_ARG;
  }
  // (all of path_ptr before any node: path_nodes holds path_ptr[S] of them, so a later entry may be the smaller)
  for (int s = 0; s < S; ++s)
    if (path_ptr[s + 1] <= path_ptr[s]) {
      set_error("%s: sample path %d is empty", who, s);
      return PT_ERR_INVALID_ARG;
    }
  std::vector<int32_t> np(N + 1, 0), leaf(std::max(S, 1), 0), seen(std::max(N, 1), -1);
  std::vector<uint8_t> is_leaf(std::max(N, 1), 0);
  bool own_leaves = true;
  for (int s = 0; s < S; ++s) {
    for (int k = path_ptr[s]; k < path_ptr[s + 1]; ++k) {
      const int n = path_nodes[k];
      if (n < 0 || n >= N) {
        set_error("%s: path %d names node %d, out of range", who, s, n);
        return PT_ERR_INVALID_ARG;
      }
      if (seen[n] == s) {
        set_error("%s: path %d names node %d twice", who, s, n);
        return PT_ERR_INVALID_ARG;
      }
      seen[n] = s;
      ++np[n + 1];
    }
    leaf[s] = path_nodes[path_ptr[s + 1] - 1];
    own_leaves &= !is_leaf[leaf[s]];
    is_leaf[leaf[s]] = 1;
  }
  for (int i = 0; i < N; ++i) np[i + 1] += np[i];
  const int E = S ? path_ptr[S] : 0;
  // samples of each node, ascending; a path entry's place among them
  std::vector<int32_t> samp(std::max(E, 1)), member(std::max(E, 1));
  {
    std::vector<int32_t> fill(np.begin(), np.end() - 1);
    for (int s = 0; s < S; ++s)
      for (int k = path_ptr[s]; k < path_ptr[s + 1]; ++k) {
        const int n = path_nodes[k];
        member[k] = fill[n] - np[n];
        samp[fill[n]++] = s;
      }
  }
  for (int s = 0; s < S; ++s)  // the member entry of the sample's own node
    samp[np[leaf[s]] + member[path_ptr[s + 1] - 1]] |= INT_MIN;
  // each class's share of the nodes
  std::vector<DecSeg> seg[kDecClasses];
  long long items[kDecClasses] = {0, 0, 0, 0};
  double tile_gain = 0.0;
  bool few = false;
  for (int i = 0; i < N; ++i) {
    const int n = np[i + 1] - np[i];
    const long long rows = (long long)n * q_len * g;
    int kind[kDecClasses] = {kSegFull, kSegFull, kSegFull, -1};
    if (rows >= kTileMinRows) {
      const bool mixed = is_leaf[i] && q_len > 1;
      kind[kDecTile] = mixed ? kSegBody : kSegFull;
      kind[kDecRowsFew] = mixed ? kSegTail : -1;
      tile_gain += Hkv * (0.9 * (double)((rows + 15) / 16) - 1.1 * (double)((rows + 127) / 128));
    }
    for (int c = 0; c < kDecClasses; ++c) {
      const int rk = n && kind[c] >= 0 ? (int)rows | kind[c] << 29 : 0;
      seg[c].push_back(DecSeg{rk, (int)std::min<long long>(items[c], INT_MAX), np[i], n == 1 ? samp[np[i]] & INT_MAX : -1});
      if (rk) items[c] += (rows + dec_r(c) - 1) / dec_r(c) * Hkv;
      if (rk && c == kDecRowsFew && kind[c] != kSegTail) few = true;
    }
  }
  for (int c = 0; c < kDecClasses; ++c)
    if (items[c] > INT_MAX / 512) {
      set_error("%s: %lld work items are out of range", who, items[c]);
      return PT_ERR_INVALID_ARG;
    }
  std::vector<int2> ent(std::max(E, 1));
  for (int k = 0; k < E; ++k) ent[k] = make_int2(path_nodes[k], member[k]);
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess) {
    set_error("%s: no CUDA device", who);
    return PT_ERR_CUDA;
  }
  // one packed upload
  std::vector<char> host;
  auto put = [&](const void* src, size_t bytes) {
    const size_t at = host.size();
    host.resize(at + pad256(std::max<size_t>(bytes, 1)), 0);
    if (bytes) std::memcpy(host.data() + at, src, bytes);
    return at;
  };
  const size_t o_mem = put(samp.data(), 4 * (size_t)E), o_pp = put(path_ptr, 4 * (size_t)(S + 1)),
               o_pe = put(ent.data(), sizeof(int2) * (size_t)E);
  size_t o_seg[kDecClasses];
  for (int c = 0; c < kDecClasses; ++c) o_seg[c] = put(seg[c].data(), sizeof(DecSeg) * seg[c].size());
  pt_decodeplan* p = new pt_decodeplan();
  p->device = dev;
  p->sms = num_sms(dev);
  p->stream = stream;
  p->N = N, p->S = S, p->Hq = Hq, p->Hkv = Hkv, p->q_len = q_len, p->own_leaves = own_leaves, p->few = few, p->tile_gain = (float)tile_gain;
  int rc = pool_alloc(&p->mem, host.size(), dev, stream);
  if (rc) {
    delete p;
    return (pt_status)rc;
  }
  char* base = static_cast<char*>(p->mem);
  p->member = reinterpret_cast<int32_t*>(base + o_mem);
  p->path_ptr = reinterpret_cast<int32_t*>(base + o_pp);
  p->path_ent = reinterpret_cast<int2*>(base + o_pe);
  for (int c = 0; c < kDecClasses; ++c) {
    p->cls[c].seg = reinterpret_cast<DecSeg*>(base + o_seg[c]);
    p->cls[c].nitems = (int32_t)items[c];
  }
  rc = upload(p->mem, host.data(), host.size(), dev, stream);
  if (rc) {
    set_error("%s: upload of the plan tables failed", who);
    pool_free(p->mem, stream);
    delete p;
    return PT_ERR_CUDA;
  }
  *out = p;
  return PT_OK;
}

extern "C" void pt_decodeplan_free(pt_decodeplan* p) {
  if (!p) return;
  pool_free(p->mem, p->stream);
  delete p;
}

extern "C" size_t pt_decode_workspace_bytes(const pt_decodeplan* p, int32_t D) {
  if (!p || D <= 0 || D > 512) return 256;
  return ws_bytes(p, D);
}

namespace {

pt_status attn_decode(const char* who, const void* Q, int64_t q_stride, const void* Kc, const void* Vc, pt_dtype dtype,
                      int32_t D, int32_t n_pages, int32_t page_size, const int32_t* tables, int32_t max_pages,
                      const int32_t* lens, const int32_t* q_count, const int32_t* mask, float scale,
                      const pt_decodeplan* plan, void* O, float* LSE, void* workspace, size_t workspace_bytes,
                      cudaStream_t stream) {
  if (!plan) {
    set_error("%s: plan is NULL", who);
    return PT_ERR_INVALID_ARG;
  }
  if (D <= 0 || D > 512) {
    set_error("%s: head_dim %d outside 1..512", who, D);
    return D <= 0 ? PT_ERR_INVALID_ARG : PT_ERR_UNSUPPORTED;
  }
  if (dtype != PT_BF16 && dtype != PT_F32) {
    set_error("%s: unknown dtype %d", who, (int)dtype);
    return PT_ERR_INVALID_ARG;
  }
  if (dtype == PT_BF16 && D % 8 != 0) {
    set_error("%s: bf16 needs head_dim %% 8 == 0 (got %d)", who, D);
    return PT_ERR_UNSUPPORTED;
  }
  if (n_pages < 1 || page_size < 1 || max_pages < 0 || (long long)max_pages * page_size > INT_MAX / 2) {
    set_error("%s: n_pages = %d, page_size = %d or max_pages = %d out of range", who, n_pages, page_size, max_pages);
    return PT_ERR_INVALID_ARG;
  }
  if (q_stride < (int64_t)plan->Hq * D) {
    set_error("%s: query tokens %lld elements apart, rows of %d", who, (long long)q_stride, plan->Hq * D);
    return PT_ERR_INVALID_ARG;
  }
  int dev = -1;
  if (cudaGetDevice(&dev) != cudaSuccess || dev != plan->device) {
    set_error("%s: the plan lives on device %d, the current device is %d", who, plan->device, dev);
    return PT_ERR_INVALID_ARG;
  }
  if (plan->S == 0) return PT_OK;
  if (!Q || !Kc || !Vc || (!tables && max_pages > 0) || !lens || !O || !LSE) {
    set_error("%s: a pointer is NULL", who);
    return PT_ERR_INVALID_ARG;
  }
  const uintptr_t al = reinterpret_cast<uintptr_t>(Kc) | reinterpret_cast<uintptr_t>(Vc) | reinterpret_cast<uintptr_t>(O);
  if ((al & 15u) || (reinterpret_cast<uintptr_t>(Q) & 3u) || (dtype == PT_BF16 && (q_stride & 1))) {
    set_error("%s: Kc, Vc and O must be 16-byte aligned, Q and its rows 4-byte aligned", who);
    return PT_ERR_INVALID_ARG;
  }
  const size_t need = ws_bytes(plan, D);
  if (!workspace || workspace_bytes < need || (reinterpret_cast<uintptr_t>(workspace) & 255u)) {
    set_error("%s: workspace must be 256-byte aligned and hold at least %zu bytes (got %zu)", who, need, workspace_bytes);
    return PT_ERR_INVALID_ARG;
  }
  if (!(scale > 0.0f)) scale = 1.0f / sqrtf((float)D);
  DecArgs a = {};
  a.member = plan->member;
  a.lens = lens, a.tables = tables, a.q_count = q_count;
  a.Q = Q, a.Kc = Kc, a.Vc = Vc, a.q_stride = q_stride;
  a.q_len = plan->q_len, a.Hq = plan->Hq, a.Hkv = plan->Hkv, a.g = plan->Hq / plan->Hkv, a.D = D;
  a.ps = page_size, a.max_pages = max_pages, a.n_pages = n_pages, a.cap = max_pages * page_size;
  a.scale_log2 = scale * 1.4426950408889634f;
  a.mask = plan->q_len > 1 ? reinterpret_cast<const unsigned*>(mask) : nullptr;  // (one query sees itself in any case)
  a.mask_w = (plan->q_len + 31) / 32;
  const bool tc = dtype == PT_BF16 && decode_tc_supported(D, page_size);
  const bool tiles = tc && use_tiles(plan, D, max_pages * page_size);
  for (int c = 0; c < kDecClasses; ++c) {
    const bool used = c == kDecSimt ? !tc : c == kDecRows ? tc && !tiles : tiles;
    const int bt = c == kDecSimt ? kSimtBT : c == kDecTile ? kTileBT : kRowsBT;
    const long long line = 2ll * ((a.cap + bt - 1) / bt) + (a.mask ? 16 : 8);  // more than an item's units
    if (used && plan->cls[c].nitems * line > INT_MAX) {
      set_error("%s: %d work items over tables of %d tokens are out of range", who, plan->cls[c].nitems, a.cap);
      return PT_ERR_UNSUPPORTED;
    }
  }
  char* ws = static_cast<char*>(workspace);
  MergeArgs m = {};
  m.n_samples = plan->S;
  m.O = O;
  m.LSE = LSE;
  cudaError_t e = cudaSuccess;
  if (tc) {
    m.c0 = class_args(plan, tiles ? kDecRowsFew : kDecRows, D, ws);
    if (tiles) m.c1 = class_args(plan, kDecTile, D, ws);
    if (tiles && a.mask && !plan->few) m.c0.nitems = 0;  // (masks leave no tails)
    m.g0 = kRows;
    a.q_vec = (reinterpret_cast<uintptr_t>(Q) & 15u) == 0 && q_stride % 8 == 0;
    const int rc = decode_tc(who, plan, a, m.c0, m.c1, stream);
    if (rc) return (pt_status)rc;
  } else {
    m.c0 = class_args(plan, kDecSimt, D, ws);
    m.g0 = kSimt;
    a.workers = dec_workers(plan, kDecSimt);
    a.min_units = 2;
    const size_t smem = 4 * (((size_t)m.c0.nseg + 31) / 32 + 1);
    ProfScope ps(stream, "decode_simt");
    const int grid = a.workers / 8;
    if (a.mask)
      e = dtype == PT_BF16 ? launch_simt<__nv_bfloat16, true>(a, m.c0, grid, smem, stream)
                           : launch_simt<float, true>(a, m.c0, grid, smem, stream);
    else
      e = dtype == PT_BF16 ? launch_simt<__nv_bfloat16, false>(a, m.c0, grid, smem, stream)
                           : launch_simt<float, false>(a, m.c0, grid, smem, stream);
    count_launch();
    if (int rc = launch_status(who, e)) return (pt_status)rc;
  }
  m.d = a;
  m.path_ptr = plan->path_ptr;
  m.path_ent = plan->path_ent;
  {
    ProfScope ps(stream, "decode_merge");
    e = dtype == PT_F32   ? launch_merge<float, false>(m, stream)
        : m.c1.nitems ? launch_merge<__nv_bfloat16, true>(m, stream)
                      : launch_merge<__nv_bfloat16, false>(m, stream);
    count_launch();
  }
  return (pt_status)launch_status(who, e);
}

}  // namespace

extern "C" pt_status pt_attn_decode(const void* Q, int64_t q_stride, const void* Kc, const void* Vc, pt_dtype dtype,
                                    int32_t D, int32_t n_pages, int32_t page_size, const int32_t* tables,
                                    int32_t max_pages, const int32_t* lens, const int32_t* q_count, float scale,
                                    const pt_decodeplan* plan, void* O, float* LSE, void* workspace,
                                    size_t workspace_bytes, cudaStream_t stream) {
  return attn_decode("pt_attn_decode", Q, q_stride, Kc, Vc, dtype, D, n_pages, page_size, tables, max_pages, lens,
                     q_count, nullptr, scale, plan, O, LSE, workspace, workspace_bytes, stream);
}

extern "C" pt_status pt_attn_decode_drafts(const void* Q, int64_t q_stride, const void* Kc, const void* Vc,
                                           pt_dtype dtype, int32_t D, int32_t n_pages, int32_t page_size,
                                           const int32_t* tables, int32_t max_pages, const int32_t* lens,
                                           const int32_t* q_count, const int32_t* draft_mask, float scale,
                                           const pt_decodeplan* plan, void* O, float* LSE, void* workspace,
                                           size_t workspace_bytes, cudaStream_t stream) {
  static const char* who = "pt_attn_decode_drafts";
  if (!draft_mask) {
    set_error("%s: draft_mask is NULL", who);
    return PT_ERR_INVALID_ARG;
  }
  return attn_decode(who, Q, q_stride, Kc, Vc, dtype, D, n_pages, page_size, tables, max_pages, lens, q_count,
                     draft_mask, scale, plan, O, LSE, workspace, workspace_bytes, stream);
}
