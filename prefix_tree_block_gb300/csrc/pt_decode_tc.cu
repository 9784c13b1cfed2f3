// pt_decode_tc.cu -- tensor-core kernels of the decoding attention (bf16,
// head dims up to 512, pages of a multiple of 16 tokens).
#include <cuda_bf16.h>

#include <algorithm>
#include <atomic>
#include <climits>

#include "pt.h"
#include "pt_decode.cuh"
#include "pt_internal.h"

namespace pt {

int take_status_decode_tc(cudaStream_t s) { return take_status_here(s); }

namespace {

__device__ __forceinline__ void ldsm4(uint32_t (&r)[4], uint32_t addr) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0,%1,%2,%3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
               : "r"(addr)
               : "memory");
}
__device__ __forceinline__ void ldsm4t(uint32_t (&r)[4], uint32_t addr) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0,%1,%2,%3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
               : "r"(addr)
               : "memory");
}
// 16 bytes global -> shared, asynchronous; the rest of 16 past `bytes` (0 or 16) is zero
__device__ __forceinline__ void cp_async16(void* dst, const void* src, int bytes) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(smem_u32(dst)), "l"(src), "r"(bytes) : "memory");
}
// 8 floats times f, one 32-byte store
__device__ __forceinline__ void st_8(float* p, const uint32_t* v, float f) {
  asm volatile("st.global.v8.f32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8};" ::"l"(p), "f"(__uint_as_float(v[0]) * f),
               "f"(__uint_as_float(v[1]) * f), "f"(__uint_as_float(v[2]) * f), "f"(__uint_as_float(v[3]) * f),
               "f"(__uint_as_float(v[4]) * f), "f"(__uint_as_float(v[5]) * f), "f"(__uint_as_float(v[6]) * f),
               "f"(__uint_as_float(v[7]) * f)
               : "memory");
}
// d += a b, 16 x 8 x 16
__device__ __forceinline__ void mma16816(float (&d)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
      : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
      : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}

// ---------------------------------------------------------------------------
// Segments of up to a few rows per kv head: 16 query rows and 16 tokens a step,
// a warp per worker; at head dims over 128, SPLIT = 2 or 4 warps, 128 columns
// each.
//
// A step's work is 32 NP mma for 16 x 256 NP bytes of keys and values: the
// kernel is bound by memory, and what matters is that every SM keeps enough
// bytes in flight (three stages a warp instead of two, which leaves fewer
// workers, cost 1% to 12% at head_dim 128) and that no warp waits for another.
// So each warp has its own ring of stages (16 tokens of K and V, 64-column
// panels, 128-byte swizzle), fills it by TMA itself (a box is 16 tokens of one
// page) and computes on what has arrived; nothing but the walk's sums is
// shared.  The loads run up to a ring ahead of the arithmetic, across the ends
// of pieces.
// With a piece's first load its query rows are gathered too, so that they are
// there when the piece begins.
//   S = Q K^T: both operands' fragments come by ldmatrix.
//   O += P V: P is the bf16 of S's own registers (the accumulator's layout is
//   the A operand's), V's fragments come by ldmatrix.trans.
// P's rounding to bf16 (up to 2^-8 of each weight, as in the forward) is what
// the tensor cores' operands cost; sums, maxima, O and the partial results are fp32.
// The warps of a SPLIT worker add up their parts of S through shared memory,
// each in the same order, and then hold the same P; O's columns stay apart.
// The running maximum is followed in steps of 2^8, as in the forward.
// Documents read once: 1.07 GB at head_dim 128 173 us (91% of the copy's
// bandwidth), 268 MB at 256 51 us (78%; 60 us with one warp for all columns,
// which has to spill), 134 MB at 64 in pages of 16 tokens 32 us (62%).
// ---------------------------------------------------------------------------
template <int NP, int SPLIT, bool TREE = false>
struct RowsCfg {
  static constexpr int WARPS = SPLIT == 1 && NP == 2 ? 3 : 4, GROUPS = WARPS / SPLIT;  // GROUPS workers a CTA
  static constexpr int CTAS = SPLIT == 1 ? 3 : 2;                                      // per SM
  static constexpr int STAGES = 2;
  static constexpr int PANEL = 16 * 128;            // bytes: 16 tokens (or rows) x 64 columns
  static constexpr int STAGE = 2 * NP * PANEL;      // K panels, V panels
  static constexpr int QBUF = NP * PANEL;           // a piece's query rows
  static constexpr int RING = STAGES * STAGE + 2 * QBUF;  // a warp's stages, and its rows of two pieces
  static constexpr int OFF_X = WARPS * RING;        // parts of S: two of 1 KB a warp
  static constexpr int OFF_BAR = OFF_X + (SPLIT > 1 ? WARPS * 2048 : 0);
  static constexpr int NBAR = WARPS * STAGES + (SPLIT > 1 ? GROUPS : 0);
  static constexpr int LIMS = 2 * kRowsR * (TREE ? 3 : 1);  // [piece & 1][row] limits; with trees, then what all see, then mask rows
  static constexpr int OFF_LIM = OFF_BAR + NBAR * 8;       // [warp]
  static constexpr int OFF_PIECE = OFF_LIM + WARPS * LIMS * 4;  // [warp][piece & 1]
  static constexpr int OFF_CHUNK = OFF_PIECE + WARPS * 2 * (int)sizeof(DecPiece);
  static constexpr size_t smem(int nseg) { return OFF_CHUNK + 8 * ((size_t)(nseg + 31) / 32 + 1) + 1024; }
};

// One warp of a worker (the sw-th of SPLIT): its ring (1024-byte aligned), its
// barriers (initialised for one arrival), room for two pieces and their rows'
// limits, and of the worker the room for S's parts and its barrier (SPLIT
// arrivals).
template <int NP, int SPLIT, bool TREE>
__device__ __forceinline__ void rows_worker(const CUtensorMap& mK, const CUtensorMap& mV, const DecArgs& a,
                                            const DecClass& c, const int* chunk, int per, int worker, int sw,
                                            uint8_t* ring, uint64_t* full, DecPiece* pieces, int* lims, float4* xbuf,
                                            uint64_t* xbar, volatile int* abort_flag) {
  using C = RowsCfg<NP, SPLIT, TREE>;
  const int lane = threadIdx.x & 31;
  const int col0 = SPLIT == 1 ? 0 : sw * 128;  // this warp's first column
  const uint32_t ring_u = smem_u32(ring);
  DecWalk walk(a, TREE, c, kRows, chunk, worker, per);
  // loads: the piece they are at, its last page, pages l_page0 + lane, and the next tile's page and row in it
  DecPiece lp;
  lp.t0 = lp.t1 = 0;
  int l_last = 0, l_page0 = 0, l_page = 0, l_row = 0, my_page = 0;
  uint32_t issued = 0, used = 0, found = 0, at = 0;  // tiles; pieces
  // the current piece
  int t = 0, t1 = 0, kv_base = 0, rows_left = 0, lim_min = 0, lim_max = 0;
  int lim[2] = {0, 0};
  int lo[2] = {0, 0}, mask_row[2] = {-1, -1}, self[2] = {0, 0};  // TREE
  int slot = 0;
  uint8_t* qbuf = ring + C::STAGES * C::STAGE;
  float o[NP * 8][4], m[2], l[2];
  const int r_lo = lane >> 2, c2 = (lane & 3) * 2;  // this lane's rows r_lo, r_lo + 8; its column pair
  // ldmatrix rows: K (matrices: tokens 0-7 / 8-15 by lane bit 4, columns by bit 3), V transposed (tokens by bit 3,
  // columns by bit 4); 16-byte pieces XOR the row's low three bits
  const int k_row = (lane & 7) + ((lane >> 4) << 3), k_cb = (lane >> 3) & 1;
  const int v_row = (lane & 7) + (((lane >> 3) & 1) << 3), v_cb = lane >> 4;
  bool ok = true;
#pragma unroll 1
  while (true) {
    // --- loads, up to a ring ahead of the arithmetic
#pragma unroll 1
    while (issued - used < C::STAGES) {
      if (lp.t0 >= lp.t1) {
        if (found > at || !walk.next(lp)) break;  // (one piece beside the current: two have room)
        if (lp.t0 == lp.t1) {  // an empty piece: nothing for its rows
          if (lane < kRowsR && sw == 0) c.lse[(long long)lp.slot * kRowsR + lane] = -INFINITY;
          continue;
        }
        int b, e;
        dec_range(a, TREE, lp.kind, lp.len, b, e);
        const int kv0 = b + lp.t0 * kRowsBT;
        l_last = (min(e, b + lp.t1 * kRowsBT) - 1) / a.ps;
        l_page0 = kv0 / a.ps - 32, l_page = 32;  // (looked up below)
        l_row = kv0 % a.ps;
        if (lane == 0) pieces[found & 1] = lp;
        // the piece's query rows, asynchronously into the buffer that the current piece does not use; lane r looks row r up
        long long src = -1;
        if (lane < min(lp.rows - lp.rt * kRowsR, kRowsR)) {
          DecRow d;
          if constexpr (TREE) {
            const DecTreeRow tr = dec_tree_row(a, lp.member0, lp.hk, lp.rt * kRowsR + lane, lp.len);
            lims[(2 + (found & 1)) * kRowsR + lane] = tr.lo;
            lims[(4 + (found & 1)) * kRowsR + lane] = tr.mask_row;
            d = tr.d;
          } else {
            d = dec_row(a, lp.member0, lp.hk, lp.rt * kRowsR + lane, lp.len);
          }
          lims[(found & 1) * kRowsR + lane] = d.lim;
          src = (long long)d.tok * a.q_stride + (long long)d.head * a.D + col0;
        }
        constexpr int CPR = NP * 8, RPI = 32 / CPR;  // 16-byte pieces of a row; rows per warp instruction
        const int ck = lane % CPR, cr = lane / CPR;
        uint8_t* qb = qbuf + (found & 1) * C::QBUF + (ck >> 3) * C::PANEL;
#pragma unroll 2
        for (int i = 0; i < kRowsR; i += RPI) {
          const long long from = __shfl_sync(0xffffffffu, src, i + cr);
          const bool in = from >= 0 && col0 + ck * 8 < a.D;
          const __nv_bfloat16* g = static_cast<const __nv_bfloat16*>(a.Q) + (in ? from + ck * 8 : 0);
          uint8_t* dst = qb + (i + cr) * 128 + (((ck & 7) ^ ((i + cr) & 7)) << 4);
          if (a.q_vec) {
            cp_async16(dst, g, in ? 16 : 0);
          } else {
            uint4 v = make_uint4(0, 0, 0, 0);
            if (in) {
              const uint32_t* w = reinterpret_cast<const uint32_t*>(g);
              v = make_uint4(w[0], w[1], w[2], w[3]);
            }
            *reinterpret_cast<uint4*>(dst) = v;
          }
        }
        ++found;
      }
      if (l_page >= 32) {
        l_page0 += l_page;
        l_page = 0;
        my_page = l_page0 + lane <= l_last ? dec_page(a, lp.node, l_page0 + lane) : 0;
      }
      const int page = __shfl_sync(0xffffffffu, my_page, l_page);
      const uint32_t s = issued % C::STAGES;
      if (lane == 0) {
        mbar_expect_tx(full + s, C::STAGE);
        const int ph = page * a.Hkv + lp.hk;
        uint8_t* dst = ring + s * C::STAGE;
        if (NP == 1) {
          tma_load_3d(dst, &mK, full + s, 0, l_row, ph);
          tma_load_3d(dst + C::PANEL, &mV, full + s, 0, l_row, ph);
        } else if (a.D % 64 == 0) {  // both panels in one box (behind the last column: zeros)
          tma_load_4d(dst, &mK, full + s, 0, l_row, col0 >> 6, ph);
          tma_load_4d(dst + NP * C::PANEL, &mV, full + s, 0, l_row, col0 >> 6, ph);
        } else {
#pragma unroll 1
          for (int pn = 0; pn < NP; ++pn) {
            tma_load_3d(dst + pn * C::PANEL, &mK, full + s, col0 + pn * 64, l_row, ph);
            tma_load_3d(dst + (NP + pn) * C::PANEL, &mV, full + s, col0 + pn * 64, l_row, ph);
          }
        }
      }
      l_row += kRowsBT;
      if (l_row == a.ps) l_row = 0, ++l_page;
      ++lp.t0;
      ++issued;
    }
    if (used == issued) break;
    // --- a new piece: its rows
    if (t >= t1) {
      asm volatile("cp.async.wait_all;" ::: "memory");
      __syncwarp();
      const DecPiece& p = pieces[at & 1];
      int e;
      dec_range(a, TREE, p.kind, p.len, kv_base, e);
      t = p.t0, t1 = p.t1, slot = p.slot;
      rows_left = p.rows - p.rt * kRowsR;
      int own_lo = INT_MAX;
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        const bool row = r_lo + i * 8 < rows_left;
        lim[i] = row ? lims[(at & 1) * kRowsR + r_lo + i * 8] : 0;
        if constexpr (TREE) {
          lo[i] = row ? lims[(2 + (at & 1)) * kRowsR + r_lo + i * 8] : 0;
          mask_row[i] = row ? lims[(4 + (at & 1)) * kRowsR + r_lo + i * 8] : -1;
          self[i] = mask_row[i] % a.q_len;
        }
        if (row) own_lo = min(own_lo, TREE ? lo[i] : lim[i]);
        m[i] = -INFINITY, l[i] = 0.f;
      }
      ++at;
      // what all of the rows see, and what any of them does
      lim_min = __reduce_min_sync(0xffffffffu, own_lo);
      lim_max = min(__reduce_max_sync(0xffffffffu, max(lim[0], lim[1])), e);
#pragma unroll
      for (int i = 0; i < NP * 8; ++i) o[i][0] = o[i][1] = o[i][2] = o[i][3] = 0.f;
    }
    // --- a tile of 16 tokens
    const uint32_t s = used % C::STAGES;
    const int kv0 = kv_base + t * kRowsBT;
    unsigned sees[2] = {0, 0};  // TREE: the tile's tokens that this lane's rows keep, looked up while the tile is on its way
    if (TREE && kv0 + kRowsBT > lim_min) {
#pragma unroll
      for (int i = 0; i < 2; ++i) sees[i] = dec_sees(a, lo[i], lim[i], mask_row[i], self[i], kv0);
    }
    ok = mbar_wait(full + s, (used / C::STAGES) & 1, abort_flag);
    ok = __all_sync(0xffffffffu, ok);
    if (!ok) break;
    const uint32_t kb = ring_u + s * C::STAGE, vb = kb + NP * C::PANEL;
    const uint32_t qa = ring_u + C::STAGES * C::STAGE + ((at - 1) & 1) * C::QBUF;
    // S, in two chains of accumulation a column tile
    float sc[2][2][4];
#pragma unroll
    for (int i = 0; i < 16; ++i) sc[i >> 3][(i >> 2) & 1][i & 3] = 0.f;
#pragma unroll
    for (int k = 0; k < NP * 4; ++k) {
      uint32_t f[4], q[4];  // (Q's matrices: rows by lane bit 3, columns by bit 4, as V's)
      ldsm4(q, qa + (k >> 2) * C::PANEL + v_row * 128 + ((((k & 3) * 2 + v_cb) ^ (v_row & 7)) << 4));
      ldsm4(f, kb + (k >> 2) * C::PANEL + k_row * 128 + ((((k & 3) * 2 + k_cb) ^ (k_row & 7)) << 4));
      mma16816(sc[k & 1][0], q, f[0], f[1]);
      mma16816(sc[k & 1][1], q, f[2], f[3]);
    }
    float x[2][4];  // [column tile of 8][(row lo: 2 columns), (row hi: 2 columns)]
#pragma unroll
    for (int n = 0; n < 2; ++n)
#pragma unroll
      for (int i = 0; i < 4; ++i) x[n][i] = sc[0][n][i] + sc[1][n][i];
    if constexpr (SPLIT > 1) {
      // (two buffers in turn: a warp that arrives here for a tile has read the parts of the one before)
      float4* xb = xbuf + (used & 1) * (SPLIT * 64) + lane;
      xb[sw * 64] = make_float4(x[0][0], x[0][1], x[0][2], x[0][3]);
      xb[sw * 64 + 32] = make_float4(x[1][0], x[1][1], x[1][2], x[1][3]);
      __syncwarp();
      if (lane == 0) mbar_arrive(xbar);
      ok = mbar_wait(xbar, used & 1, abort_flag);
      ok = __all_sync(0xffffffffu, ok);
      if (!ok) break;
#pragma unroll
      for (int n = 0; n < 2; ++n) {
        float4 sum = xb[n * 32];
#pragma unroll
        for (int w = 1; w < SPLIT; ++w) {
          const float4 y = xb[w * 64 + n * 32];
          sum.x += y.x, sum.y += y.y, sum.z += y.z, sum.w += y.w;
        }
        x[n][0] = sum.x, x[n][1] = sum.y, x[n][2] = sum.z, x[n][3] = sum.w;
      }
    }
    int n_mul = kRowsBT, n_any = kRowsBT;  // tokens whose values the product takes; tokens that any row keeps
    if (kv0 + kRowsBT > lim_min) {
#pragma unroll
      for (int n = 0; n < 2; ++n)
#pragma unroll
        for (int i = 0; i < 4; ++i)
          if (TREE ? !(sees[i >> 1] >> (n * 8 + c2 + (i & 1)) & 1u) : kv0 + n * 8 + c2 + (i & 1) >= lim[i >> 1])
            x[n][i] = -INFINITY;
      // Values that no row keeps are cleared: a probability of 0 times what
      // lies behind the node's tokens must stay 0.  Tokens that some rows keep
      // and others do not go through the product too unless one is not finite:
      // then they are cleared as well and added row by row.
      n_any = min(max(lim_max - kv0, 0), kRowsBT);
      n_mul = n_any;
      const int n_all = min(max(lim_min - kv0, 0), kRowsBT);
      uint8_t* vs = ring + s * C::STAGE + NP * C::PANEL;
      if (n_all < n_any) {
        bool odd = false;
        if constexpr (TREE) {  // (all drafts are in question here: 0 times each value, several loads at a time; not 0: not finite)
          const __nv_bfloat162 none = __float2bfloat162_rn(0.f);
          __nv_bfloat162 sum[2] = {none, none};
#pragma unroll 4
          for (int i = n_all * (NP * 8) + lane; i < n_any * (NP * 8); i += 32) {
            const uint4 v = *reinterpret_cast<const uint4*>(vs + ((i % (NP * 8)) >> 3) * C::PANEL + (i / (NP * 8)) * 128 + (i & 7) * 16);
            const __nv_bfloat162* w = reinterpret_cast<const __nv_bfloat162*>(&v);
            sum[0] = __hfma2(w[0], none, sum[0]), sum[1] = __hfma2(w[1], none, sum[1]);
            sum[0] = __hfma2(w[2], none, sum[0]), sum[1] = __hfma2(w[3], none, sum[1]);
          }
          const float2 f = __bfloat1622float2(__hadd2(sum[0], sum[1]));
          odd = !(f.x == 0.f && f.y == 0.f);
        } else {
#pragma unroll 1
          for (int i = n_all * (NP * 8) + lane; i < n_any * (NP * 8); i += 32) {
            const uint4 v = *reinterpret_cast<const uint4*>(vs + ((i % (NP * 8)) >> 3) * C::PANEL + (i / (NP * 8)) * 128 +
                                                            (i & 7) * 16);
            const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
            for (int j = 0; j < 4; ++j) odd |= (w[j] & 0x7f80u) == 0x7f80u || (w[j] & 0x7f800000u) == 0x7f800000u;
          }
        }
        if (__any_sync(0xffffffffu, odd)) n_mul = n_all;
      }
      if (n_mul < n_any) {
        n_mul = -1 - n_mul;  // (once the probabilities are known)
      } else if (n_any < kRowsBT) {
#pragma unroll 1
        for (int i = n_any * (NP * 8) + lane; i < kRowsBT * (NP * 8); i += 32)
          *reinterpret_cast<uint4*>(vs + ((i % (NP * 8)) >> 3) * C::PANEL + (i / (NP * 8)) * 128 + (i & 7) * 16) =
              make_uint4(0, 0, 0, 0);
        fence_proxy_async_smem();  // before the stage is loaded again
        __syncwarp();
      }
    }
    bool grow = false;
    float ref[2], al[2];
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      float mx = fmaxf(fmaxf(x[0][2 * i], x[0][2 * i + 1]), fmaxf(x[1][2 * i], x[1][2 * i + 1]));
      mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 1));
      mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 2)) * a.scale_log2;
      const bool up = mx > m[i] + 8.f;
      const float mn = up ? mx : m[i];
      ref[i] = mn == -INFINITY ? 0.f : mn;
      al[i] = up ? ex2(m[i] - ref[i]) : 1.f;
      grow |= up;
      m[i] = mn;
    }
    uint32_t pa[4];
#pragma unroll
    for (int n = 0; n < 2; ++n)
#pragma unroll
      for (int i = 0; i < 4; ++i) x[n][i] = ex2(fmaf(x[n][i], a.scale_log2, -ref[i >> 1]));
    if (__any_sync(0xffffffffu, grow)) {
#pragma unroll
      for (int i = 0; i < NP * 8; ++i) {
        o[i][0] *= al[0], o[i][1] *= al[0];
        o[i][2] *= al[1], o[i][3] *= al[1];
      }
      l[0] *= al[0];
      l[1] *= al[1];
    }
    l[0] += (x[0][0] + x[0][1]) + (x[1][0] + x[1][1]);
    l[1] += (x[0][2] + x[0][3]) + (x[1][2] + x[1][3]);
    pa[0] = pack_bf16(x[0][0], x[0][1]);
    pa[1] = pack_bf16(x[0][2], x[0][3]);
    pa[2] = pack_bf16(x[1][0], x[1][1]);
    pa[3] = pack_bf16(x[1][2], x[1][3]);
    if (n_mul < 0) {  // a value that is not finite, kept by some rows only: those tokens row by row, then cleared
      n_mul = -1 - n_mul;
#pragma unroll 1
      for (int n = n_mul; n < n_any; ++n) {
        float pr[2];
#pragma unroll
        for (int i = 0; i < 2; ++i) {
          const float even = n & 8 ? x[1][2 * i] : x[0][2 * i], oddc = n & 8 ? x[1][2 * i + 1] : x[0][2 * i + 1];
          pr[i] = __shfl_sync(0xffffffffu, n & 1 ? oddc : even, (lane & ~3) | ((n & 7) >> 1));
        }
#pragma unroll
        for (int k = 0; k < NP * 8; ++k) {
          const uint32_t w = *reinterpret_cast<const uint32_t*>(ring + s * C::STAGE + (NP + (k >> 3)) * C::PANEL + n * 128 +
                                                                (((k & 7) ^ (n & 7)) << 4) + (lane & 3) * 4);
          const float v0 = __uint_as_float(w << 16), v1 = __uint_as_float(w & 0xffff0000u);
#pragma unroll
          for (int i = 0; i < 2; ++i)
            if (TREE ? sees[i] >> n & 1u : kv0 + n < lim[i]) {
              o[k][2 * i] = fmaf(pr[i], v0, o[k][2 * i]);
              o[k][2 * i + 1] = fmaf(pr[i], v1, o[k][2 * i + 1]);
            }
        }
      }
      __syncwarp();
#pragma unroll 1
      for (int i = n_mul * (NP * 8) + lane; i < kRowsBT * (NP * 8); i += 32)
        *reinterpret_cast<uint4*>(ring + s * C::STAGE + (NP + ((i % (NP * 8)) >> 3)) * C::PANEL + (i / (NP * 8)) * 128 +
                                  (i & 7) * 16) = make_uint4(0, 0, 0, 0);
      fence_proxy_async_smem();
      __syncwarp();
    }
#pragma unroll
    for (int k = 0; k < NP * 4; ++k) {
      uint32_t f[4];
      ldsm4t(f, vb + (k >> 2) * C::PANEL + v_row * 128 + ((((k & 3) * 2 + v_cb) ^ (v_row & 7)) << 4));
      mma16816(o[2 * k], pa, f[0], f[1]);
      mma16816(o[2 * k + 1], pa, f[2], f[3]);
    }
    ++used;
    ++t;
    __syncwarp();  // every lane has read the stage
    if (t < t1) continue;
    // --- the piece's partial result
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      l[i] += __shfl_xor_sync(0xffffffffu, l[i], 1);
      l[i] += __shfl_xor_sync(0xffffffffu, l[i], 2);
      if (r_lo + i * 8 >= rows_left) continue;
      const float inv = l[i] == 0.f ? 0.f : 1.f / l[i];
      const long long row = (long long)slot * kRowsR + r_lo + i * 8;
      if (c2 == 0 && sw == 0) c.lse[row] = l[i] == 0.f ? -INFINITY : m[i] + log2f(l[i]);
      float* dst = c.opart + row * a.D + col0 + c2;
#pragma unroll
      for (int k = 0; k < NP * 8; ++k)
        if (col0 + k * 8 < a.D) *reinterpret_cast<float2*>(dst + k * 8) = make_float2(o[k][2 * i] * inv, o[k][2 * i + 1] * inv);
    }
  }
  if (!ok) {  // a wait ran out: let the copies in flight land before the block ends
    *abort_flag = 1;
    for (; used < issued; ++used) mbar_wait_drain(full + used % C::STAGES, (used / C::STAGES) & 1, 20000000);
  }
}

// The fewest tile units worth a partial result of their own.
constexpr int kTileMinUnits = 4;

// How the SMs are divided when a call has both kinds of segments (below): every
// CTA of both kernels scans both classes and finds the same numbers.
struct DecSplit {
  int n_tile;         // SMs of the tile kernel; the rows kernel has the others
  int per_t, per_r;   // units per worker
};
template <int NP, bool TREE>
__device__ __forceinline__ DecSplit dec_split(const DecArgs& a, const DecClass& ct, const DecClass& cr, int* chunk_t,
                                              int* chunk_r, unsigned long long* cost, int sms, int rows_per_sm) {
  const bool both = ct.nitems && cr.nitems;
  if (both)
    dec_scan(a, TREE, ct, cr, dec_tile(TREE), kRows, chunk_t, chunk_r, cost);
  else
    dec_scan(a, TREE, ct.nitems ? ct : cr, cr, DecTiling{ct.nitems ? kTile.r : kRows.r, ct.nitems ? kTile.t : kRows.t, ct.nitems ? dec_tile(TREE).k : kRows.k}, kRows,
             ct.nitems ? chunk_t : chunk_r, chunk_r, nullptr);
  const int nc = (max(ct.nseg, cr.nseg) + 31) >> 5;
  const int units_t = ct.nitems ? chunk_t[nc] : 0, units_r = cr.nitems ? chunk_r[nc] : 0;
  DecSplit s;
  s.n_tile = units_t > 0 ? sms : 0;
  if (units_t > 0 && units_r > 0) {
    // (a tile unit of 128 rows costs an SM about as much as 10 units of 16 rows and tokens, 14 at head_dim 64)
    const float x = (float)cost[0] * (NP == 1 ? 14.f : 10.f);
    s.n_tile = min(max((int)(sms * (x / (x + (float)cost[1]))), 1), sms - 1);
  }
  s.per_t = dec_share(units_t, max(s.n_tile, 1), kTileMinUnits);
  s.per_r = dec_share(units_r, max(sms - s.n_tile, 1) * rows_per_sm, 1);
  return s;
}

template <int NP, int SPLIT, bool TREE>
__global__ void __launch_bounds__(RowsCfg<NP, SPLIT>::WARPS * 32, RowsCfg<NP, SPLIT>::CTAS)
    k_decode_rows(const __grid_constant__ CUtensorMap mK, const __grid_constant__ CUtensorMap mV, const DecArgs a,
                  const DecClass c, const DecClass ct) {
  using C = RowsCfg<NP, SPLIT, TREE>;
  // Beside a tile kernel this one starts when that one has begun (it has then
  // waited for what came before both), runs on the SMs that it leaves, and
  // ends after it, so that waiting for this kernel is waiting for both.
  const bool beside = ct.nitems > 0;
  if (!beside) pdl_wait();
  pdl_launch();
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  const int warp = threadIdx.x >> 5;
  uint64_t* bars = reinterpret_cast<uint64_t*>(smem + C::OFF_BAR);
  int* chunk = reinterpret_cast<int*>(smem + C::OFF_CHUNK);
  volatile __shared__ int abort_flag;
  __shared__ unsigned long long cost[2];
  if (threadIdx.x < C::NBAR) {
    mbar_init(bars + threadIdx.x, threadIdx.x < C::WARPS * C::STAGES ? 1 : SPLIT);
    fence_mbar_init();
  }
  if (threadIdx.x == 0) {
    abort_flag = 0;
    cost[0] = cost[1] = 0;
    prefetch_tmap(&mK);
    prefetch_tmap(&mV);
  }
  if (beside) __syncthreads();  // (the costs; the scan's barriers publish the rest)
  const DecSplit sp = dec_split<NP, TREE>(a, ct, c, chunk + ((c.nseg + 31) >> 5) + 1, chunk, cost, a.sms, C::CTAS * C::GROUPS);
  if ((int)blockIdx.x == 0) dec_publish(a, TREE, c, kRows, chunk, sp.per_r);
  if ((int)blockIdx.x < (a.sms - sp.n_tile) * C::CTAS)
    rows_worker<NP, SPLIT, TREE>(mK, mV, a, c, chunk, sp.per_r, (int)blockIdx.x * C::GROUPS + warp / SPLIT, warp % SPLIT,
                           smem + warp * C::RING, bars + warp * C::STAGES,
                           reinterpret_cast<DecPiece*>(smem + C::OFF_PIECE) + warp * 2,
                           reinterpret_cast<int*>(smem + C::OFF_LIM) + warp * C::LIMS,
                           reinterpret_cast<float4*>(smem + C::OFF_X) + (warp / SPLIT) * (SPLIT * 128),
                           bars + C::WARPS * C::STAGES + warp / SPLIT, &abort_flag);
  if (beside) pdl_wait();
}

// ---------------------------------------------------------------------------
// Trees in which many rows read a segment (a prompt under many completions):
// such segments run on tcgen05, a CTA per worker, up to 256 query rows an item,
// 128 tokens a step; the others as above, in the kernel launched behind this
// one.  The first kind is bound by its softmax and tensor work, the second by
// memory, so the SMs are divided between the two by what their units cost and
// they overlap: the CTAs of this kernel that have no share end at once, and the
// other's take their SMs.
//
// The forward's structure with the mask gone: a producer warp brings K and V
// tiles by TMA (boxes of whole pages, or of the power of two that divides
// them), an MMA warp issues S = Q K^T (M = 128 rows, N = 128 tokens) and
// O += P V with P read from TMEM, and two softmax warpgroups, a row per thread,
// turn S into P in place.  Two warpgroups are what keeps the tensor pipe busy;
// an item of more than 128 rows gives each half of the rows and both read every
// tile; a smaller one gives them alternate tiles of the same rows, and each
// ends with a partial result of its own, so the same code runs either way:
// step u belongs to warpgroup u & 1 and tile u >> pair.  S of step u is issued
// after PV of step u - 2 of the same warpgroup, so the commit of S(u) also says
// that O may be rescaled.  Warps without rows only keep the barriers moving.
// 943 MB of prompts and continuations, two prompts of 32768 tokens under 64
// samples of 512 to 2048 more, 32 q heads over 8: 165 us for the call (84% of
// the copy's bandwidth), 629 on rows alone; drafts of 16 tokens behind 32
// continuations of prompts of 4096, 16 q heads over 4, where 64 rows read every
// token of a continuation and 1024 a prompt: 54 us, 130 on rows alone.
// A step of 256 x 128 takes 2.1 us, 60% of the tensor pipe's rate: one thread
// issues its 32 products at 50 ns each.  P is rounded to bf16 as above.
// Tokens behind the segment's last are zero-filled by TMA where a whole box
// lies behind it; inside a box the threads clear V's rows, so that nothing
// stored there reaches O.
// TREE: drafts that are a tree.  In the tiles that hold some, a row's thread masks
// S by its mask's words, and values that are not finite are kept out of the
// product and added to the rows that see them afterwards.  Trees of 32 drafts
// behind 32 continuations of prompts of 4096, 32 q heads over 8 (2048 rows a kv
// head and prompt): 123 us for the call, 194 with the drafts left to
// the row kernel as tails, 142 with the SMs divided by what those cost there; a run
// of 32 drafts without masks 155.
// ---------------------------------------------------------------------------
template <int NP>
struct TileCfg {
  static constexpr int D = NP * 64;
  static constexpr int PANEL = 128 * 128;  // bytes: 128 rows x 64 columns
  static constexpr int TILE = NP * PANEL;
  static constexpr int KS = NP == 1 ? 4 : 2, VS = KS;
  static constexpr int OFF_Q = 0;  // two tiles of 128 rows
  static constexpr int OFF_K = OFF_Q + 2 * TILE;
  static constexpr int OFF_V = OFF_K + KS * TILE;
  static constexpr int OFF_BAR = OFF_V + VS * TILE;
  // q_full q_empty k_full[KS] k_empty[KS] v_full[VS] v_empty[VS] s_full[2] p_full[2] o_full[2] o_free[2] done
  static constexpr int NBAR = 2 + 2 * KS + 2 * VS + 9;
  static constexpr int OFF_PIECE_BAR = OFF_BAR + NBAR * 8;  // full[PIECES] empty[PIECES]
  static constexpr int PIECES = 4;
  static constexpr int OFF_PIECE = OFF_PIECE_BAR + 2 * PIECES * 8;
  static constexpr int OFF_MISC = OFF_PIECE + PIECES * (int)sizeof(DecPiece);
  static constexpr int OFF_CHUNK = OFF_MISC + 16;  // the classes' chunk sums: tile, rows
  static constexpr size_t smem(int nseg) { return OFF_CHUNK + 8 * ((size_t)(nseg + 31) / 32 + 1) + 1024; }
  static constexpr int TM_S = 0, TM_O = 256;  // S(h) at h * 128, O(h) at 256 + h * D
  static constexpr int THREADS = 384;         // two softmax warpgroups; producer, MMA and two query warps
  static constexpr int REG_SOFTMAX = 216, REG_CTRL = 72, REG_LAUNCH = 168;
  static_assert(256 * REG_SOFTMAX + 128 * REG_CTRL == THREADS * REG_LAUNCH, "register split");
  static_assert(OFF_CHUNK + 8 * (kDecMaxNodes / 32 + 1) + 1024 <= 232448, "shared memory budget");
  static_assert(TM_O + 2 * D <= 512, "TMEM budget");
};

// Whether a token's values (D of them, D a multiple of 8) are not all finite.
__device__ __forceinline__ bool odd_values(const uint4* v, int n) {
  const __nv_bfloat162 none = __float2bfloat162_rn(0.f);
  __nv_bfloat162 sum = none;  // 0 times each
  for (int i = 0; i < n; ++i) {
    const uint4 x = v[i];
    const __nv_bfloat162* w = reinterpret_cast<const __nv_bfloat162*>(&x);
#pragma unroll
    for (int k = 0; k < 4; ++k) sum = __hfma2(w[k], none, sum);
  }
  const float2 f = __bfloat1622float2(sum);
  return !(f.x == 0.f && f.y == 0.f);
}

// Trees of drafts, tile kernel: a draft's values that are not finite were kept out
// of the products, which would have carried them (0 times them) into every row.
// They are added here to the rows that see the draft, O in TMEM (columns from ob
// on), once a piece's products are done.  Tokens [t, end) in question; a whole
// warp, a row per lane (row < 0: none).  m: the reference of the row's weights.
__device__ __noinline__ void add_odd_values(const DecArgs& a, int node, int hk, int member0, int len, int row, int t,
                                            int end, int skip, float m, uint32_t ob) {
  DecTreeRow d = {};
  d.mask_row = -1;
  if (row >= 0) d = dec_tree_row(a, member0, hk, row, len);
  const __nv_bfloat16* q = static_cast<const __nv_bfloat16*>(a.Q) + (long long)d.d.tok * a.q_stride + (long long)d.d.head * a.D;
#pragma unroll 1
  for (; t < end; ++t) {
    if (skip >= 0 && ((t >> kTile.t) & 1) == skip) continue;  // (the other warpgroup's tile)
    const int pi = t / a.ps;
    const long long at = (((long long)dec_page(a, node, pi) * a.Hkv + hk) * a.ps + (t - pi * a.ps)) * a.D;
    const __nv_bfloat16* k = static_cast<const __nv_bfloat16*>(a.Kc) + at;
    const __nv_bfloat16* v = static_cast<const __nv_bfloat16*>(a.Vc) + at;
    if (!odd_values(reinterpret_cast<const uint4*>(v), a.D / 8)) continue;
    const bool sees = row >= 0 && (dec_sees(a, d.lo, d.d.lim, d.mask_row, d.mask_row >= 0 ? d.mask_row % a.q_len : 0, t) & 1u);
    float s = 0.f;
    if (sees)
      for (int i = 0; i < a.D; ++i) s = fmaf(__bfloat162float(q[i]), __bfloat162float(k[i]), s);
    const float w = ex2(fmaf(s, a.scale_log2, m == -INFINITY ? 0.f : -m));
#pragma unroll 1
    for (int c = 0; c < a.D; c += 32) {
      uint32_t o[32];
      tmem_ld32(ob + c, o);
      tmem_ld_wait();
#pragma unroll
      for (int i = 0; i < 32; ++i)
        if (sees && c + i < a.D) o[i] = __float_as_uint(fmaf(w, __bfloat162float(v[c + i]), __uint_as_float(o[i])));
      tmem_st32(ob + c, o);
      tmem_st_wait();
    }
  }
}

template <int NP, bool TREE>
__global__ void __launch_bounds__(TileCfg<NP>::THREADS, 1)
    k_decode_tile(const __grid_constant__ CUtensorMap mK, const __grid_constant__ CUtensorMap mV, const DecArgs a,
                  const DecClass c, const DecClass cr, const int rows_per_sm, const int box_rows, const int oob_head) {
  using C = TileCfg<NP>;
  constexpr int D = C::D;
  pdl_wait();
  pdl_launch();
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  uint64_t* q_full = reinterpret_cast<uint64_t*>(smem + C::OFF_BAR);
  uint64_t* q_empty = q_full + 1;
  uint64_t* k_full = q_empty + 1;
  uint64_t* k_empty = k_full + C::KS;
  uint64_t* v_full = k_empty + C::KS;
  uint64_t* v_empty = v_full + C::VS;
  uint64_t* s_full = v_empty + C::VS;
  uint64_t* p_full = s_full + 2;
  uint64_t* o_full = p_full + 2;
  uint64_t* o_free = o_full + 2;
  uint64_t* done = o_free + 2;
  uint64_t* piece_full = reinterpret_cast<uint64_t*>(smem + C::OFF_PIECE_BAR);
  uint64_t* piece_empty = piece_full + C::PIECES;
  DecPiece* pieces = reinterpret_cast<DecPiece*>(smem + C::OFF_PIECE);
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(smem + C::OFF_MISC);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(smem + C::OFF_MISC + 4);
  int* chunk = reinterpret_cast<int*>(smem + C::OFF_CHUNK);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  __shared__ unsigned long long cost[2];
  __shared__ volatile int odd_piece[8];  // TREE: the piece (by its number modulo 8) in which a value was not finite
  __shared__ volatile int odd_row[TREE ? 2 : 1][TREE ? kTileBT : 1];  // TREE: the tile (its number + 1, by that modulo 2) whose row's values are being cleared
  if constexpr (TREE) {
    if (threadIdx.x < 8) odd_piece[threadIdx.x] = 0;
    if (threadIdx.x < 2 * kTileBT) odd_row[threadIdx.x / kTileBT][threadIdx.x % kTileBT] = 0;
  }
  if (threadIdx.x == 0) {
    mbar_init(q_full, 8);
    mbar_init(q_empty, 1);
    for (int i = 0; i < C::KS; ++i) mbar_init(k_full + i, 1), mbar_init(k_empty + i, 1);
    for (int i = 0; i < C::VS; ++i) mbar_init(v_full + i, 1), mbar_init(v_empty + i, 1);
    for (int h = 0; h < 2; ++h) {
      mbar_init(s_full + h, 1);
      mbar_init(p_full + h, 128);
      mbar_init(o_full + h, 1);
      mbar_init(o_free + h, 128);
    }
    mbar_init(done, 1);
#pragma unroll 1
    for (int i = 0; i < C::PIECES; ++i) mbar_init(piece_full + i, 1), mbar_init(piece_empty + i, 11);
    *abort_flag = 0;
    cost[0] = cost[1] = 0;
    fence_mbar_init();
    prefetch_tmap(&mK);
    prefetch_tmap(&mV);
  }
  __syncthreads();
  const DecSplit sp = dec_split<NP, TREE>(a, c, cr, chunk, chunk + ((c.nseg + 31) >> 5) + 1, cost, gridDim.x, rows_per_sm);
  if (blockIdx.x == 0) dec_publish(a, TREE, c, dec_tile(TREE), chunk, sp.per_t);
  if ((int)blockIdx.x >= sp.n_tile) return;
  const int worker = blockIdx.x, per = sp.per_t;
  if (warp == 9) {
    tmem_alloc(tmem_slot, 512);
    tmem_relinquish();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tbase = *tmem_slot;

  // The producer walks along the CTA's units and hands each piece to the other
  // warps through a ring; one without rows ends it.
  const auto get_piece = [&](DecPiece& p, uint32_t i) {  // the i-th; all lanes of a warp
    const uint32_t s = i % C::PIECES;
    bool ok = mbar_wait(piece_full + s, (i / C::PIECES) & 1, abort_flag);
    if (!(ok = __all_sync(0xffffffffu, ok))) return false;
    p = pieces[s];
    __syncwarp();
    if (lane == 0) mbar_arrive(piece_empty + s);
    return p.rows > 0;
  };

  const auto producer_role = [&]() {
    DecWalk walk(a, TREE, c, dec_tile(TREE), chunk, worker, per);
    DecPiece p;
    uint32_t n = 0, np = 0;  // tiles issued; pieces
    bool ok = true;
    const int boxes = kTileBT / box_rows;  // 1..8, a power of two
#pragma unroll 1
    while (true) {
      const bool more = walk.next(p);
      if (more && p.t0 == p.t1) {  // an empty piece: nothing for its rows
#pragma unroll 1
        for (int r = lane; r < kTileR; r += 32) c.lse[(long long)p.slot * kTileR + r] = -INFINITY;
        continue;
      }
      if (!more) p.rows = 0;
      if (np >= C::PIECES) ok = mbar_wait(piece_empty + np % C::PIECES, (np / C::PIECES - 1) & 1, abort_flag);
      if (!(ok = __all_sync(0xffffffffu, ok))) break;
      if (lane == 0) {
        pieces[np % C::PIECES] = p;
        mbar_arrive(piece_full + np % C::PIECES);
      }
      ++np;
      if (!more) break;
      int b, e;
      dec_range(a, TREE, p.kind, p.len, b, e);
      const int bt = lane & (boxes - 1);  // this lane's box of the tile; its page, looked up a tile ahead
      auto page_of = [&](int t) {
        const int kv = t * kTileBT + bt * box_rows;
        return t < p.t1 && kv < e ? dec_page(a, p.node, kv / a.ps) : -1;
      };
      int page = page_of(p.t0);
#pragma unroll 1
      for (int t = p.t0; t < p.t1; ++t, ++n) {
        const int ahead = page_of(t + 1);
        const int kv = t * kTileBT + bt * box_rows;
        const int row = kv % a.ps, head = page >= 0 ? page * a.Hkv + p.hk : oob_head;
        const uint32_t ks = n % C::KS, vs = n % C::VS;
        if (n >= C::KS) ok = mbar_wait(k_empty + ks, (n / C::KS - 1) & 1, abort_flag);
        if (!(ok = __all_sync(0xffffffffu, ok))) break;
        if (lane == 0) mbar_expect_tx(k_full + ks, C::TILE);
        __syncwarp();
        if (lane < boxes) {
#pragma unroll
          for (int pn = 0; pn < NP; ++pn)
            tma_load_3d(smem + C::OFF_K + ks * C::TILE + pn * C::PANEL + bt * box_rows * 128, &mK, k_full + ks, pn * 64, row,
                        head);
        }
        if (n >= C::VS) ok = mbar_wait(v_empty + vs, (n / C::VS - 1) & 1, abort_flag);
        if (!(ok = __all_sync(0xffffffffu, ok))) {
          if (lane == 0) mbar_wait_drain(k_full + ks, (n / C::KS) & 1, 20000000);
          break;
        }
        if (lane == 0) mbar_expect_tx(v_full + vs, C::TILE);
        __syncwarp();
        if (lane < boxes) {
#pragma unroll
          for (int pn = 0; pn < NP; ++pn)
            tma_load_3d(smem + C::OFF_V + vs * C::TILE + pn * C::PANEL + bt * box_rows * 128, &mV, v_full + vs, pn * 64, row,
                        head);
        }
        page = ahead;
      }
      if (!ok) break;
    }
    if (!ok && lane == 0) {  // let the copies in flight land
      for (uint32_t i = 0; i < C::KS && i < n; ++i) mbar_wait_drain(k_full + (n - 1 - i) % C::KS, ((n - 1 - i) / C::KS) & 1, 20000000);
      for (uint32_t i = 0; i < C::VS && i < n; ++i) mbar_wait_drain(v_full + (n - 1 - i) % C::VS, ((n - 1 - i) / C::VS) & 1, 20000000);
    }
    __syncwarp();
  };

  const auto mma_role = [&]() {  // lane 0
    constexpr uint32_t IDESC_S = idesc_bf16(128, 128, false, false);
    constexpr uint32_t IDESC_PV = idesc_bf16(128, D, false, true);
    // (each product's descriptors by an addition: built anew, what issues them would take longer than they do)
    const uint64_t dQ = sdesc_sw128(smem_u32(smem + C::OFF_Q), 16, 1024);
    const uint64_t dK = sdesc_sw128(smem_u32(smem + C::OFF_K), 16, 1024);
    const uint64_t dV = sdesc_sw128(smem_u32(smem + C::OFF_V), C::PANEL, 1024);
    uint32_t n = 0, it = 0;   // tiles before this piece; pieces
    uint32_t pc[2] = {0, 0};  // PV steps per warpgroup
    uint32_t oc[2] = {0, 0};  // pieces in which the warpgroup had steps
    bool ok = true;
#pragma unroll 1
    while (ok) {
      const uint32_t pi = it % C::PIECES;
      if (!mbar_wait(piece_full + pi, (it / C::PIECES) & 1, abort_flag)) break;
      const int left = pieces[pi].rows - pieces[pi].rt * kTileR, tiles = pieces[pi].t1 - pieces[pi].t0;
      const bool end = pieces[pi].rows <= 0;
      mbar_arrive(piece_empty + pi);
      if (end) break;
      const int pair = left > kTileR / 2 ? 1 : 0, steps = tiles << pair;
      ok = mbar_wait(q_full, it & 1, abort_flag);
      tc_fence_after();
#pragma unroll 1
      for (int u0 = 0; u0 < steps + 2 && ok; u0 += 2) {
#pragma unroll
        for (int h = 0; h < 2; ++h) {  // (constant, so that the counters stay in registers)
          const int u = u0 + h;
          if (u >= 2 && u < steps + 2) {  // PV of step u - 2
            const uint32_t x = n + ((u - 2) >> pair), vs = x % C::VS;
            const uint64_t dv = sdesc_add(dV, vs * C::TILE);
            ok = mbar_wait(p_full + h, pc[h] & 1, abort_flag) && mbar_wait(v_full + vs, (x / C::VS) & 1, abort_flag);
            if (u < 4 && oc[h] > 0) ok = ok && mbar_wait(o_free + h, (oc[h] - 1) & 1, abort_flag);
            if (!ok) break;
            tc_fence_after();
#pragma unroll
            for (int kk = 0; kk < 8; ++kk)
              mma_ts(tbase + C::TM_O + h * D, tbase + C::TM_S + h * 128 + kk * 8, sdesc_add(dv, kk * 2048), IDESC_PV,
                     u >= 4 || kk > 0);
            if (!pair || h == 1) mma_commit(v_empty + vs);
            if (u >= steps) mma_commit(o_full + h);  // the warpgroup's last
            ++pc[h];
          }
          if (u < steps) {
            const uint32_t x = n + (u >> pair), ks = x % C::KS;
            const uint64_t dq = sdesc_add(dQ, pair ? h * C::TILE : 0), dk = sdesc_add(dK, ks * C::TILE);
            ok = mbar_wait(k_full + ks, (x / C::KS) & 1, abort_flag);
            if (!ok) break;
            tc_fence_after();
#pragma unroll
            for (int kk = 0; kk < D / 16; ++kk) {
              const uint32_t off = (kk >> 2) * C::PANEL + (kk & 3) * 32;
              mma_ss(tbase + C::TM_S + h * 128, sdesc_add(dq, off), sdesc_add(dk, off), IDESC_S, kk > 0);
            }
            mma_commit(s_full + h);
            if (!pair || h == 1) mma_commit(k_empty + ks);
            if (u == steps - 1) mma_commit(q_empty);
          }
        }
      }
      n += tiles;
      ++it;
      if (steps > 0) ++oc[0];
      if (steps > 1) ++oc[1];
    }
    mma_commit(done);
    mbar_wait_drain(done, 0, 200000000);
  };

  // Gathers an item's query rows into the Q tiles, warp w of every `nw`: 16-byte
  // asynchronous copies, a row's lanes side by side.
  const auto gather_rows = [&](const DecPiece& p, int w, int nw) {
    constexpr int CPR = NP * 8, RPI = 32 / CPR;  // 16-byte pieces of a row; rows per warp instruction
    const int k = lane % CPR, ir = lane / CPR;
    const int left = p.rows - p.rt * kTileR, rows = left > kTileR / 2 ? kTileR : kTileR / 2;
#pragma unroll 1
    for (int r0 = w * 32; r0 < rows; r0 += nw * 32) {
      long long src = -1;  // element offset of this lane's row, or -1
      if (r0 + lane < left) {
        const DecRow d = dec_row(a, p.member0, p.hk, p.rt * kTileR + r0 + lane, p.len);
        src = (long long)d.tok * a.q_stride + (long long)d.head * a.D;
      }
#pragma unroll 4
      for (int i = 0; i < 32; i += RPI) {
        const int x = r0 + i + ir;
        const long long at = __shfl_sync(0xffffffffu, src, i + ir);
        const bool in = at >= 0 && k * 8 < a.D;
        const __nv_bfloat16* g = static_cast<const __nv_bfloat16*>(a.Q) + (in ? at + k * 8 : 0);
        uint8_t* dst = smem + C::OFF_Q + (x >> 7) * C::TILE + (k >> 3) * C::PANEL + (x & 127) * 128 + (((k & 7) ^ (x & 7)) << 4);
        if (a.q_vec) {
          cp_async16(dst, g, in ? 16 : 0);
        } else {
          uint4 v = make_uint4(0, 0, 0, 0);
          if (in) {
            const uint32_t* y = reinterpret_cast<const uint32_t*>(g);
            v = make_uint4(y[0], y[1], y[2], y[3]);
          }
          *reinterpret_cast<uint4*>(dst) = v;
        }
      }
    }
    asm volatile("cp.async.wait_all;" ::: "memory");
    fence_proxy_async_smem();
    __syncwarp();
    if (lane == 0) mbar_arrive_cnt(q_full, 8 / nw);
  };

  // The first piece's rows come by the softmax warps, which have nothing else
  // to do then; the others' by two warps of their own, as soon as the last S of
  // the piece before is done, so the loads run under that piece's last steps
  // and its output.
  const auto query_role = [&]() {
    DecPiece p;
#pragma unroll 1
    for (uint32_t it = 0; get_piece(p, it); ++it) {
      if (it == 0) continue;
      bool ok = mbar_wait(q_empty, (it - 1) & 1, abort_flag);
      if (!(ok = __all_sync(0xffffffffu, ok))) break;
      gather_rows(p, warp - 10, 2);
    }
    __syncwarp();
  };

  const auto softmax_role = [&]() {
    const int h = warp >> 2, r = threadIdx.x & 127;  // warpgroup; row in its tile, TMEM lane
    const uint32_t tl = tbase + ((uint32_t)((warp & 3) * 32) << 16);
    const uint32_t sb = tl + C::TM_S + h * 128, ob = tl + C::TM_O + h * D;
    uint32_t n = 0, sc = 0, oc = 0, it = 0;
    bool ok = true;
#pragma unroll 1
    while (ok) {
      // of the piece: row tiles in it, its steps, this warpgroup's rows, tokens from its first tile on, partial result
      int pair, steps, n_rows, tok, slot;
      // TREE: the piece; its first token that a row may not see, from its first tile on; what this thread's row sees
      DecPiece tp;
      int mixed = INT_MAX, lo = 0, lim = 0, mask_row = -1, self = 0;
      {
        DecPiece p;
        if (!get_piece(p, it)) break;
        if (it++ == 0) gather_rows(p, warp, 8);
        int b;
        dec_range(a, TREE, p.kind, p.len, b, tok);
        tok -= p.t0 * kTileBT;
        const int left = p.rows - p.rt * kTileR;
        pair = left > kTileR / 2 ? 1 : 0;
        steps = (p.t1 - p.t0) << pair;
        n_rows = min(pair ? left - h * 128 : left, 128);
        slot = p.slot;
        if constexpr (TREE) {
          tp = p;
          if (p.kind == kSegBody && p.t1 * kTileBT > p.len - a.q_len) {
            mixed = max(p.len - a.q_len, 0) - p.t0 * kTileBT;
            if (r < n_rows) {
              const DecTreeRow d = dec_tree_row(a, p.member0, p.hk, p.rt * kTileR + (pair ? h * 128 : 0) + r, p.len);
              lo = d.lo, lim = d.d.lim, mask_row = d.mask_row;
              self = mask_row >= 0 ? mask_row % a.q_len : 0;
            }
          }
        }
      }
      const bool live = (warp & 3) * 32 < n_rows;  // this warp has some
      float m_use = -INFINITY, l = 0.f;
#pragma unroll 1
      for (int u = h; u < steps; u += 2, ++sc) {
        const int n_tok = min(tok - (u >> pair) * kTileBT, kTileBT);
        ok = mbar_wait(s_full + h, sc & 1, abort_flag);
        if (!(ok = __all_sync(0xffffffffu, ok))) break;
        tc_fence_after();
        const int from = (u >> pair) * kTileBT;  // the tile's first token, from the piece's first tile on
        const bool masked = TREE && from + kTileBT > mixed;
        if (masked) {
          // Values that are not finite, of tokens that some rows do not see, are cleared (see add_odd_values).  Both
          // warpgroups of a pair do so, each before its own product.  One may read a row while the other clears it, and
          // find what was not finite gone but the rest still there, which its product would add a second time: so
          // which row and that there are some is said first, and asked after the reading.  (The two are never two
          // tiles apart: S of a tile comes after both products of the last but one.)
          const uint32_t x = n + (u >> pair), vs = x % C::VS;
          ok = mbar_wait(v_full + vs, (x / C::VS) & 1, abort_flag);
          if (!(ok = __all_sync(0xffffffffu, ok))) break;
          if (from + r >= mixed && r < n_tok) {
            bool odd = false;
#pragma unroll
            for (int pn = 0; pn < NP; ++pn)
              odd |= odd_values(reinterpret_cast<const uint4*>(smem + C::OFF_V + vs * C::TILE + pn * C::PANEL + r * 128), 8);
            __threadfence_block();
            if (odd || odd_row[x & 1][r] == (int)x + 1) {
              odd_row[x & 1][r] = (int)x + 1;
              odd_piece[it & 7] = (int)it;
              __threadfence_block();
#pragma unroll
              for (int k = 0; k < NP * 8; ++k)
                *reinterpret_cast<uint4*>(smem + C::OFF_V + vs * C::TILE + (k >> 3) * C::PANEL + r * 128 + (k & 7) * 16) =
                    make_uint4(0, 0, 0, 0);
            }
          }
          __threadfence_block();
          fence_proxy_async_smem();
        }
        if (n_tok < kTileBT) {
          // Clear V's rows behind the last token (both warpgroups of a pair: the same zeros).  Only now: S of this
          // step being done, the product with the tile that was in this stage before is done too, so the parity
          // below means this tile.
          const uint32_t x = n + (u >> pair), vs = x % C::VS;
          ok = mbar_wait(v_full + vs, (x / C::VS) & 1, abort_flag);
          if (!(ok = __all_sync(0xffffffffu, ok))) break;
          if (r >= n_tok) {
#pragma unroll
            for (int k = 0; k < NP * 8; ++k)
              *reinterpret_cast<uint4*>(smem + C::OFF_V + vs * C::TILE + (k >> 3) * C::PANEL + r * 128 + (k & 7) * 16) =
                  make_uint4(0, 0, 0, 0);
          }
          fence_proxy_async_smem();
        }
        if (live) {
          uint32_t sr[128];
          tmem_ld32(sb + 0, sr + 0);
          tmem_ld32(sb + 32, sr + 32);
          tmem_ld32(sb + 64, sr + 64);
          tmem_ld32(sb + 96, sr + 96);
          tmem_ld_wait();
          if (masked) {
#pragma unroll
            for (int k = 0; k < 128; k += 32) {
              const unsigned sees = dec_sees(a, lo, lim, mask_row, self, tp.t0 * kTileBT + from + k);
#pragma unroll
              for (int i = 0; i < 32; ++i)
                if (!(sees >> i & 1u)) sr[k + i] = 0xff800000u;  // -inf
            }
          } else if (n_tok < kTileBT) {
#pragma unroll
            for (int k = 0; k < 128; ++k)
              if (k >= n_tok) sr[k] = 0xff800000u;  // -inf
          }
          float m8[8];
#pragma unroll
          for (int k = 0; k < 8; ++k) m8[k] = -INFINITY;
#pragma unroll
          for (int k = 0; k < 128; k += 2)
            m8[(k >> 1) & 7] = fmax3(m8[(k >> 1) & 7], __uint_as_float(sr[k]), __uint_as_float(sr[k + 1]));
          const float mx = fmaxf(fmaxf(fmaxf(m8[0], m8[1]), fmaxf(m8[2], m8[3])),
                                 fmaxf(fmaxf(m8[4], m8[5]), fmaxf(m8[6], m8[7])));
          const float m_blk = mx * a.scale_log2;
          const bool grow = m_blk > m_use + 8.f;
          const float m_new = grow ? m_blk : m_use, ref = m_new == -INFINITY ? 0.f : m_new;
          const unsigned long long sc2 = f2_splat(a.scale_log2), nref2 = f2_splat(-ref);
          unsigned long long r4[4] = {0ull, 0ull, 0ull, 0ull};
#pragma unroll
          for (int k = 0; k < 128; k += 2) {
            float x0, x1;
            f2_unpack(f2_fma(f2_pack(__uint_as_float(sr[k]), __uint_as_float(sr[k + 1])), sc2, nref2), x0, x1);
            const float p0 = ex2(x0), p1 = ex2(x1);
            r4[(k >> 1) & 3] = f2_add(r4[(k >> 1) & 3], f2_pack(p0, p1));
            sr[k >> 1] = pack_bf16(p0, p1);
          }
          float r8[8];
#pragma unroll
          for (int k = 0; k < 4; ++k) f2_unpack(r4[k], r8[2 * k], r8[2 * k + 1]);
          const float l_blk = ((r8[0] + r8[1]) + (r8[2] + r8[3])) + ((r8[4] + r8[5]) + (r8[6] + r8[7]));
          if (__any_sync(0xffffffffu, grow && l > 0.f)) {
            const float alpha = (grow && l > 0.f) ? ex2(m_use - m_new) : 1.f;
#pragma unroll 1
            for (int k = 0; k < D / 32; ++k) {
              uint32_t orr[32];
              tmem_ld32(ob + k * 32, orr);
              tmem_ld_wait();
#pragma unroll
              for (int i = 0; i < 32; ++i) orr[i] = __float_as_uint(__uint_as_float(orr[i]) * alpha);
              tmem_st32(ob + k * 32, orr);
            }
            l *= alpha;
          }
          m_use = m_new;
          l += l_blk;
          tmem_st32(sb + 0, sr + 0);
          tmem_st32(sb + 32, sr + 32);
          tmem_st_wait();
        }
        tc_fence_before();
        mbar_arrive(p_full + h);
      }
      if (!ok) break;
      n += steps >> pair;
      // the warpgroup's partial result
      const long long at = (long long)slot * kTileR + h * 128 + r;
      if (h < steps) {
        ok = mbar_wait(o_full + h, oc & 1, abort_flag);
        if (!(ok = __all_sync(0xffffffffu, ok))) break;
        ++oc;
        tc_fence_after();
        if (TREE && live && odd_piece[it & 7] == (int)it)
          add_odd_values(a, tp.node, tp.hk, tp.member0, tp.len,
                         r < n_rows ? tp.rt * kTileR + (pair ? h * 128 : 0) + r : -1, max(mixed, 0) + tp.t0 * kTileBT,
                         min(tp.t1 * kTileBT, tp.len), pair ? -1 : (tp.t0 + h + 1) & 1, m_use, ob);
        if (live) {
          const float inv = l == 0.f ? 0.f : 1.f / l;
          if (r < n_rows) c.lse[at] = l == 0.f ? -INFINITY : m_use + log2f(l);
          // 8 columns of all rows side by side (tile_at): a warp's store covers 1 KB in one piece, where rows of
          // their own would scatter it over 32 lines
          float* dst = c.opart + tile_at(a.D, slot, h * 128 + r, 0);
#pragma unroll 1
          for (int k = 0; k < D / 32; ++k) {
            uint32_t orr[32];
            tmem_ld32(ob + k * 32, orr);
            tmem_ld_wait();
            if (r < n_rows) {
#pragma unroll
              for (int i = 0; i < 32; i += 8)
                if (k * 32 + i < a.D) st_8(dst + (k * 4 + (i >> 3)) * (kTileR * 8), orr + i, inv);
            }
          }
        }
        tc_fence_before();
        mbar_arrive(o_free + h);
      } else if (r < n_rows) {
        c.lse[at] = -INFINITY;  // no tile of a one-tile piece was this warpgroup's
      }
    }
    if (!ok) *abort_flag = 1;
  };

  if (warp >= 8) {
    regs_dec<C::REG_CTRL>();
    if (warp == 8)
      producer_role();
    else if (warp == 9) {
      if (lane == 0) mma_role();
      __syncwarp();
    } else
      query_role();
  } else {
    regs_inc<C::REG_SOFTMAX>();
    softmax_role();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  if (warp == 9) tmem_dealloc(tbase, 512);
}

// Kc or Vc as a 3-D map (D, page_size, n_pages * Hkv) with boxes of 64 columns x
// `rows` tokens, or with `two` and D a multiple of 64 as a 4-D one (64,
// page_size, D / 64, n_pages * Hkv) with boxes of 128 columns; 128-byte swizzle.
bool make_tmap_pages(CUtensorMap* map, const void* base, int D, int ps, long long heads, int rows, bool two) {
  encode_tiled_fn enc = get_encode_tiled();
  if (!enc) {
    set_error("cuTensorMapEncodeTiled is unavailable from the driver");
    return false;
  }
  const bool all = two && D % 64 == 0;
  const int panels = D / 64;
  cuuint64_t dims[4] = {(cuuint64_t)(all ? 64 : D), (cuuint64_t)ps, (cuuint64_t)(all ? panels : heads), (cuuint64_t)heads};
  cuuint64_t strides[3] = {(cuuint64_t)D * 2, (cuuint64_t)(all ? 128 : (size_t)ps * D * 2), (cuuint64_t)ps * D * 2};
  cuuint32_t box[4] = {64, (cuuint32_t)rows, (cuuint32_t)(all ? 2 : 1), 1};
  cuuint32_t estr[4] = {1, 1, 1, 1};
  CUresult r = enc(map, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, all ? 4 : 3, const_cast<void*>(base), dims, strides, box, estr,
                   CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                   CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
  if (r != CUDA_SUCCESS) {
    set_error("cuTensorMapEncodeTiled failed (%d) for pages of %d x %d, %lld of them", (int)r, ps, D, heads);
    return false;
  }
  return true;
}

// Lets a kernel use up to `bytes` of shared memory, once per device (a bit each).
template <class K>
cudaError_t opt_in_smem(K kernel, size_t bytes, std::atomic<uint64_t>& opted) {
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess || (dev < 64 && (opted.load(std::memory_order_relaxed) >> dev & 1))) return e;
  e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)bytes);
  if (e == cudaSuccess && dev < 64) opted.fetch_or(1ull << dev, std::memory_order_relaxed);
  return e;
}

template <int NP, int SPLIT, bool TREE>
cudaError_t launch_rows(const CUtensorMap& mK, const CUtensorMap& mV, const DecArgs& a, const DecClass& c,
                        const DecClass& ct, cudaStream_t s) {
  using C = RowsCfg<NP, SPLIT, TREE>;
  static_assert(C::CTAS * C::GROUPS <= kRowsWarps, "the workspace's slots");
  const size_t smem = C::smem(c.nseg);
  auto kernel = k_decode_rows<NP, SPLIT, TREE>;
  static std::atomic<uint64_t> opted{0};
  if (cudaError_t e = opt_in_smem(kernel, C::smem(kDecMaxNodes), opted)) return e;
  count_launch();
  return launch_pdl(kernel, dim3(a.sms * C::CTAS), dim3(C::WARPS * 32), smem, s, mK, mV, a, c, ct);
}

template <bool TREE>
cudaError_t launch_rows(const CUtensorMap& mK, const CUtensorMap& mV, const DecArgs& a, const DecClass& c,
                        const DecClass& ct, cudaStream_t s) {
  if (a.D <= 64) return launch_rows<1, 1, TREE>(mK, mV, a, c, ct, s);
  if (a.D <= 128) return launch_rows<2, 1, TREE>(mK, mV, a, c, ct, s);
  return a.D <= 256 ? launch_rows<2, 2, TREE>(mK, mV, a, c, ct, s) : launch_rows<2, 4, TREE>(mK, mV, a, c, ct, s);
}

template <int NP, bool TREE>
cudaError_t launch_tile(const CUtensorMap& mK, const CUtensorMap& mV, const DecArgs& a, const DecClass& c,
                        const DecClass& cr, int box_rows, int heads, cudaStream_t s) {
  using C = TileCfg<NP>;
  const size_t smem = C::smem(c.nseg);
  static std::atomic<uint64_t> opted{0};
  if (cudaError_t e = opt_in_smem(k_decode_tile<NP, TREE>, C::smem(kDecMaxNodes), opted)) return e;
  count_launch();
  return launch_pdl(k_decode_tile<NP, TREE>, dim3(a.sms), dim3(C::THREADS), smem, s, mK, mV, a, c, cr,
                    RowsCfg<NP, 1>::CTAS * RowsCfg<NP, 1>::GROUPS, box_rows, heads);
}

}  // namespace

bool decode_tc_supported(int D, int ps) { return D % 8 == 0 && D <= 512 && ps % 16 == 0; }

int decode_tc(const char* who, const pt_decodeplan* p, DecArgs a, const DecClass& rows, const DecClass& tile,
              cudaStream_t s) {
  const long long heads = (long long)a.n_pages * a.Hkv;
  if (heads > INT_MAX - 1) {
    set_error("%s: %d pages of %d heads are out of range", who, a.n_pages, a.Hkv);
    return PT_ERR_INVALID_ARG;
  }
  CUtensorMap mK, mV, mKt, mVt;
  cudaError_t e = cudaSuccess;
  const int np = (a.D + 63) / 64;
  if (!make_tmap_pages(&mK, a.Kc, a.D, a.ps, heads, 16, np > 1) || !make_tmap_pages(&mV, a.Vc, a.D, a.ps, heads, 16, np > 1))
    return PT_ERR_CUDA;
  a.sms = p->sms;
  ProfScope ps(s, tile.nitems ? "decode_tile" : "decode_rows");  // (two kernels that overlap have one scope)
  if (tile.nitems) {
    const int box = std::min(a.ps & -a.ps, kTileBT);  // the largest power of two that divides a page
    if (!make_tmap_pages(&mKt, a.Kc, a.D, a.ps, heads, box, false) || !make_tmap_pages(&mVt, a.Vc, a.D, a.ps, heads, box, false))
      return PT_ERR_CUDA;
    auto go = [&](auto launch) { return launch(mKt, mVt, a, tile, rows, box, (int)heads, s); };
    if (a.mask)
      e = np == 1 ? go(launch_tile<1, true>) : go(launch_tile<2, true>);
    else
      e = np == 1 ? go(launch_tile<1, false>) : go(launch_tile<2, false>);
  }
  if (e == cudaSuccess && rows.nitems)
    e = a.mask ? launch_rows<true>(mK, mV, a, rows, tile, s) : launch_rows<false>(mK, mV, a, rows, tile, s);
  if (e == cudaSuccess) e = cudaGetLastError();
  if (e != cudaSuccess) {
    set_error("%s: launch failed: %s", who, cudaGetErrorString(e));
    return PT_ERR_CUDA;
  }
  return PT_OK;
}

}  // namespace pt
