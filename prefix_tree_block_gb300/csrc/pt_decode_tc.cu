// pt_decode_tc.cu -- tensor-core kernels of the decoding attention (bf16,
// head dims up to 256, pages of a multiple of 16 tokens).
#include <cuda_bf16.h>

#include <algorithm>
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
// d += a b, 16 x 8 x 16
__device__ __forceinline__ void mma16816(float (&d)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
      : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
      : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}

// ---------------------------------------------------------------------------
// Segments of up to a few rows per kv head: a warp per worker, 16 query rows,
// 16 tokens a step.
//
// A step's work is 32 NP mma for 16 x 128 NP bytes of keys and values: the
// kernel is bound by memory, and what matters is that every SM keeps enough
// bytes in flight and that no warp waits for another.  So each warp has its
// own ring of stages (16 tokens of K and V, 64-column panels, 128-byte
// swizzle), fills it by TMA itself (a box is 16 tokens of one page and one
// panel) and computes on what has arrived; nothing is shared between warps.
// The loads run up to a ring ahead of the arithmetic, across the ends of
// pieces: a second walk along the worker's units issues them.
//   S = Q K^T: Q's fragments stay in registers, K's come by ldmatrix.
//   O += P V: P is the bf16 of S's own registers (the accumulator's layout is
//   the A operand's), V's fragments come by ldmatrix.trans.
// The running maximum is followed in steps of 2^8, as in the forward.
// ---------------------------------------------------------------------------
template <int NP>
struct RowsCfg {
  static constexpr int WARPS = 4;
  static constexpr int CTAS = NP == 4 ? 1 : 2;  // per SM
  static constexpr int STAGES = NP == 1 ? 6 : NP == 2 ? 3 : NP == 3 ? 2 : 3;
  static constexpr int PANEL = 16 * 128;            // bytes: 16 tokens x 64 columns
  static constexpr int STAGE = 2 * NP * PANEL;      // K panels, V panels
  static constexpr int OFF_BAR = WARPS * STAGES * STAGE;
  static constexpr int OFF_CHUNK = OFF_BAR + WARPS * STAGES * 8;
  static constexpr size_t smem(int nseg) { return OFF_CHUNK + 8 * ((size_t)(nseg + 31) / 32 + 1) + 1024; }
};

template <int NP>
__global__ void __launch_bounds__(RowsCfg<NP>::WARPS * 32, RowsCfg<NP>::CTAS)
    k_decode_rows(const __grid_constant__ CUtensorMap mK, const __grid_constant__ CUtensorMap mV, const DecArgs a,
                  const DecClass c) {
  using C = RowsCfg<NP>;
  pdl_wait();
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  uint64_t* full = reinterpret_cast<uint64_t*>(smem + C::OFF_BAR) + warp * C::STAGES;
  long long* chunk = reinterpret_cast<long long*>(smem + C::OFF_CHUNK);
  volatile __shared__ int abort_flag;
  if (threadIdx.x == 0) {
    abort_flag = 0;
    for (int i = 0; i < C::WARPS * C::STAGES; ++i) mbar_init(reinterpret_cast<uint64_t*>(smem + C::OFF_BAR) + i, 1);
    fence_mbar_init();
    prefetch_tmap(&mK);
    prefetch_tmap(&mV);
  }
  const long long per = dec_scan<kRowsR, kRowsBT>(a, c, chunk);  // (also publishes the barriers)
  uint8_t* ring = smem + warp * (C::STAGES * C::STAGE);
  const uint32_t ring_u = smem_u32(ring);
  const long long worker = (long long)blockIdx.x * C::WARPS + warp;

  // --- loads: one tile a call, in the order of the arithmetic below
  DecWalk<kRowsR, kRowsBT> ahead(a, c, chunk, worker, per);
  DecPiece lp;
  lp.t0 = lp.t1 = 0;
  int l_base = 0, l_page0 = 0, my_page = 0;  // first token of the segment; pages l_page0 + lane
  uint32_t issued = 0;
  auto issue = [&]() {
    if (lp.t0 >= lp.t1) {
      if (!ahead.next(lp)) return;
      int e;
      dec_range(a, lp.kind, lp.len, l_base, e);
      l_page0 = INT_MIN;
    }
    const int kv0 = l_base + lp.t0 * kRowsBT, pi = kv0 / a.ps;
    if (l_page0 == INT_MIN || pi >= l_page0 + 32) {
      l_page0 = pi;
      int b, e;
      dec_range(a, lp.kind, lp.len, b, e);
      const int last = (min(e, b + lp.t1 * kRowsBT) - 1) / a.ps;  // last page of the piece
      my_page = pi + lane <= last ? dec_page(a, lp.node, pi + lane) : 0;
    }
    const int page = __shfl_sync(0xffffffffu, my_page, pi - l_page0);
    const uint32_t s = issued % C::STAGES;
    if (lane == 0) {
      mbar_expect_tx(full + s, C::STAGE);
      const int row = kv0 - pi * a.ps, ph = page * a.Hkv + lp.hk;
#pragma unroll
      for (int pn = 0; pn < NP; ++pn) {
        tma_load_3d(ring + s * C::STAGE + pn * C::PANEL, &mK, full + s, pn * 64, row, ph);
        tma_load_3d(ring + s * C::STAGE + (NP + pn) * C::PANEL, &mV, full + s, pn * 64, row, ph);
      }
    }
    ++lp.t0;
    ++issued;
  };
#pragma unroll 1
  for (int i = 0; i < C::STAGES; ++i) issue();

  // --- arithmetic
  DecWalk<kRowsR, kRowsBT> walk(a, c, chunk, worker, per);
  DecPiece p;
  uint32_t used = 0;
  const int r_lo = lane >> 2, c2 = (lane & 3) * 2;  // this lane's rows r_lo, r_lo + 8; its column pair
  // ldmatrix rows: K (matrices: tokens 0-7 / 8-15 by lane bit 4, columns by bit 3), V transposed (tokens by bit 3,
  // columns by bit 4); 16-byte pieces XOR the row's low three bits
  const int k_row = (lane & 7) + ((lane >> 4) << 3), k_cb = (lane >> 3) & 1;
  const int v_row = (lane & 7) + (((lane >> 3) & 1) << 3), v_cb = lane >> 4;
  bool ok = true;
  while (ok && walk.next(p)) {
    int b, e;
    dec_range(a, p.kind, p.len, b, e);
    uint32_t q[NP * 4][4];
    int lim[2];
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      const int row = p.rt * kRowsR + r_lo + i * 8;
      const __nv_bfloat16* src = nullptr;
      lim[i] = 0;
      if (row < p.rows) {
        const DecRow d = dec_row(a, p.member0, p.hk, row, p.len);
        lim[i] = d.lim;
        src = static_cast<const __nv_bfloat16*>(a.Q) + (long long)d.tok * a.q_stride + (long long)d.head * a.D;
      }
#pragma unroll
      for (int k = 0; k < NP * 4; ++k) {
        const int col = k * 16 + c2;
        q[k][i] = src && col < a.D ? *reinterpret_cast<const uint32_t*>(src + col) : 0u;
        q[k][i + 2] = src && col + 8 < a.D ? *reinterpret_cast<const uint32_t*>(src + col + 8) : 0u;
      }
    }
    // bounds of the piece's rows (rows that are none count as seeing nothing only for the upper one)
    const int own_lo = min(p.rt * kRowsR + r_lo < p.rows ? lim[0] : INT_MAX, p.rt * kRowsR + r_lo + 8 < p.rows ? lim[1] : INT_MAX);
    const int lim_min = __reduce_min_sync(0xffffffffu, own_lo);
    const int lim_max = min(__reduce_max_sync(0xffffffffu, max(lim[0], lim[1])), e);
    float o[NP * 8][4];
#pragma unroll
    for (int i = 0; i < NP * 8; ++i) o[i][0] = o[i][1] = o[i][2] = o[i][3] = 0.f;
    float m[2] = {-INFINITY, -INFINITY}, l[2] = {0.f, 0.f};
#pragma unroll 1
    for (int t = p.t0; t < p.t1; ++t) {
      const uint32_t s = used % C::STAGES;
      ok = mbar_wait(full + s, (used / C::STAGES) & 1, &abort_flag);
      ok = __all_sync(0xffffffffu, ok);
      if (!ok) break;
      const uint32_t kb = ring_u + s * C::STAGE, vb = kb + NP * C::PANEL;
      const int kv0 = b + t * kRowsBT;
      // S, in two chains of accumulation a column tile
      float sc[2][2][4];
#pragma unroll
      for (int i = 0; i < 16; ++i) sc[i >> 3][(i >> 2) & 1][i & 3] = 0.f;
#pragma unroll
      for (int k = 0; k < NP * 4; ++k) {
        uint32_t f[4];
        ldsm4(f, kb + (k >> 2) * C::PANEL + k_row * 128 + ((((k & 3) * 2 + k_cb) ^ (k_row & 7)) << 4));
        mma16816(sc[k & 1][0], q[k], f[0], f[1]);
        mma16816(sc[k & 1][1], q[k], f[2], f[3]);
      }
      float x[2][4];  // [column tile of 8][(row lo: 2 columns), (row hi: 2 columns)]
#pragma unroll
      for (int n = 0; n < 2; ++n)
#pragma unroll
        for (int i = 0; i < 4; ++i) x[n][i] = (sc[0][n][i] + sc[1][n][i]) * a.scale_log2;
      const bool cut = kv0 + kRowsBT > lim_min;
      if (cut) {
#pragma unroll
        for (int n = 0; n < 2; ++n)
#pragma unroll
          for (int i = 0; i < 4; ++i)
            if (kv0 + n * 8 + c2 + (i & 1) >= lim[i >> 1]) x[n][i] = -INFINITY;
      }
      bool grow = false;
      float ref[2], al[2];
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        float mx = fmaxf(fmaxf(x[0][2 * i], x[0][2 * i + 1]), fmaxf(x[1][2 * i], x[1][2 * i + 1]));
        mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 1));
        mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 2));
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
        for (int i = 0; i < 4; ++i) x[n][i] = ex2(x[n][i] - ref[i >> 1]);
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
      if (!cut) {
#pragma unroll
        for (int k = 0; k < NP * 4; ++k) {
          uint32_t f[4];
          ldsm4t(f, vb + (k >> 2) * C::PANEL + v_row * 128 + ((((k & 3) * 2 + v_cb) ^ (v_row & 7)) << 4));
          mma16816(o[2 * k], pa, f[0], f[1]);
          mma16816(o[2 * k + 1], pa, f[2], f[3]);
        }
      } else {
        // Values that no row keeps are cleared: a probability of 0 times what
        // lies behind the node's tokens must stay 0.  Tokens that some rows
        // keep and others do not go through the product too unless one is not
        // finite: then they are left out of it and added row by row.
        const int n_all = min(max(lim_min - kv0, 0), kRowsBT), n_any = min(max(lim_max - kv0, 0), kRowsBT);
        bool odd = false;
        for (int i = n_all * (NP * 8) + lane; i < n_any * (NP * 8); i += 32) {
          const uint4 v = *reinterpret_cast<const uint4*>(ring + s * C::STAGE + (NP + ((i % (NP * 8)) >> 3)) * C::PANEL +
                                                          (i / (NP * 8)) * 128 + (i & 7) * 16);
          const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
          for (int j = 0; j < 4; ++j) odd |= (w[j] & 0x7f80u) == 0x7f80u || (w[j] & 0x7f800000u) == 0x7f800000u;
        }
        odd = __any_sync(0xffffffffu, odd);
        const int n_mul = odd ? n_all : n_any;
        // this lane's V elements of a fragment: tokens c2, c2 + 1 (f[0], f[2]) and c2 + 8, c2 + 9 (f[1], f[3])
        const uint32_t k0 = (c2 < n_mul ? 0xffffu : 0u) | (c2 + 1 < n_mul ? 0xffff0000u : 0u);
        const uint32_t k1 = (c2 + 8 < n_mul ? 0xffffu : 0u) | (c2 + 9 < n_mul ? 0xffff0000u : 0u);
#pragma unroll
        for (int k = 0; k < NP * 4; ++k) {
          uint32_t f[4];
          ldsm4t(f, vb + (k >> 2) * C::PANEL + v_row * 128 + ((((k & 3) * 2 + v_cb) ^ (v_row & 7)) << 4));
          mma16816(o[2 * k], pa, f[0] & k0, f[1] & k1);
          mma16816(o[2 * k + 1], pa, f[2] & k0, f[3] & k1);
        }
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
              if (kv0 + n < lim[i]) {
                o[k][2 * i] = fmaf(pr[i], v0, o[k][2 * i]);
                o[k][2 * i + 1] = fmaf(pr[i], v1, o[k][2 * i + 1]);
              }
          }
        }
      }
      ++used;
      __syncwarp();  // every lane has read the stage
      issue();
    }
    if (!ok) break;
    // the piece's partial result
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      l[i] += __shfl_xor_sync(0xffffffffu, l[i], 1);
      l[i] += __shfl_xor_sync(0xffffffffu, l[i], 2);
      if (p.rt * kRowsR + r_lo + i * 8 >= p.rows) continue;
      const float inv = l[i] == 0.f ? 0.f : 1.f / l[i];
      const long long row = p.slot * kRowsR + r_lo + i * 8;
      if (c2 == 0) c.lse[row] = l[i] == 0.f ? -INFINITY : m[i] + log2f(l[i]);
      float* dst = c.opart + row * a.D + c2;
#pragma unroll
      for (int k = 0; k < NP * 8; ++k)
        if (k * 8 < a.D) *reinterpret_cast<float2*>(dst + k * 8) = make_float2(o[k][2 * i] * inv, o[k][2 * i + 1] * inv);
    }
  }
  if (!ok) {  // a wait ran out: let the copies in flight land before the block ends
    for (; used < issued; ++used) mbar_wait_drain(full + used % C::STAGES, (used / C::STAGES) & 1, 20000000);
  }
}

// ---------------------------------------------------------------------------
// Segments that many rows read (a prompt under many completions): tcgen05, a
// CTA per worker, up to 256 query rows an item, 128 tokens a step.
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
// Tokens behind the segment's last are zero-filled by TMA where a whole box
// lies behind it; inside a box the threads clear V's rows, so that nothing
// stored there reaches O.
// ---------------------------------------------------------------------------
template <int NP>
struct TileCfg {
  static constexpr int D = NP * 64;
  static constexpr int PANEL = 128 * 128;  // bytes: 128 rows x 64 columns
  static constexpr int TILE = NP * PANEL;
  static constexpr int KS = NP == 1 ? 4 : 2, VS = NP == 1 ? 4 : 2;
  static constexpr int OFF_Q = 0;  // two tiles of 128 rows
  static constexpr int OFF_K = OFF_Q + 2 * TILE;
  static constexpr int OFF_V = OFF_K + KS * TILE;
  static constexpr int OFF_BAR = OFF_V + VS * TILE;
  // q_full q_empty k_full[KS] k_empty[KS] v_full[VS] v_empty[VS] s_full[2] p_full[2] o_full[2] o_free[2] done
  static constexpr int NBAR = 2 + 2 * KS + 2 * VS + 9;
  static constexpr int OFF_MISC = OFF_BAR + NBAR * 8;
  static constexpr int OFF_CHUNK = OFF_MISC + 16;
  static constexpr size_t smem(int nseg) { return OFF_CHUNK + 8 * ((size_t)(nseg + 31) / 32 + 1) + 1024; }
  static constexpr int TM_S = 0, TM_O = 256;  // S(h) at h * 128, O(h) at 256 + h * D
  static constexpr int THREADS = 384;         // two softmax warpgroups; producer, MMA and two query warps
  static constexpr int REG_SOFTMAX = 216, REG_CTRL = 72, REG_LAUNCH = 168;
  static_assert(256 * REG_SOFTMAX + 128 * REG_CTRL == THREADS * REG_LAUNCH, "register split");
  static_assert(OFF_CHUNK + 8 * (kDecMaxNodes / 32 + 1) + 1024 <= 232448, "shared memory budget");
  static_assert(TM_O + 2 * D <= 512, "TMEM budget");
};

template <int NP>
__global__ void __launch_bounds__(TileCfg<NP>::THREADS, 1)
    k_decode_tile(const __grid_constant__ CUtensorMap mK, const __grid_constant__ CUtensorMap mV, const DecArgs a,
                  const DecClass c, const int box_rows, const int oob_head) {
  using C = TileCfg<NP>;
  constexpr int D = C::D;
  pdl_wait();
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
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(smem + C::OFF_MISC);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(smem + C::OFF_MISC + 4);
  long long* chunk = reinterpret_cast<long long*>(smem + C::OFF_CHUNK);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  if (threadIdx.x == 0) {
    mbar_init(q_full, 64);
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
    *abort_flag = 0;
    fence_mbar_init();
    prefetch_tmap(&mK);
    prefetch_tmap(&mV);
  }
  if (warp == 9) {
    tmem_alloc(tmem_slot, 512);
    tmem_relinquish();
  }
  tc_fence_before();
  const long long per = dec_scan<kTileR, kTileBT>(a, c, chunk);  // (its barriers publish the above)
  tc_fence_after();
  const uint32_t tbase = *tmem_slot;
  const long long worker = blockIdx.x;

  const auto producer_role = [&]() {
    DecWalk<kTileR, kTileBT> walk(a, c, chunk, worker, per);
    DecPiece p;
    uint32_t n = 0;  // tiles issued
    bool ok = true;
    const int boxes = kTileBT / box_rows;  // 1..8, a power of two
    while (ok && walk.next(p)) {
      int b, e;
      dec_range(a, p.kind, p.len, b, e);
      const int bt = lane & (boxes - 1);  // this lane's box of the tile; its page, looked up a tile ahead
      auto page_of = [&](int t) {
        const int kv = t * kTileBT + bt * box_rows;
        return t < p.t1 && kv < e ? dec_page(a, p.node, kv / a.ps) : -1;
      };
      int page = page_of(p.t0);
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
    }
    if (!ok && lane == 0) {  // let the copies in flight land
      for (uint32_t i = 0; i < C::KS && i < n; ++i) mbar_wait_drain(k_full + (n - 1 - i) % C::KS, ((n - 1 - i) / C::KS) & 1, 20000000);
      for (uint32_t i = 0; i < C::VS && i < n; ++i) mbar_wait_drain(v_full + (n - 1 - i) % C::VS, ((n - 1 - i) / C::VS) & 1, 20000000);
    }
    __syncwarp();
  };

  const auto mma_role = [&]() {
    constexpr uint32_t IDESC_S = idesc_bf16(128, 128, false, false);
    constexpr uint32_t IDESC_PV = idesc_bf16(128, D, false, true);
    const uint32_t sQ = smem_u32(smem + C::OFF_Q), sK = smem_u32(smem + C::OFF_K), sV = smem_u32(smem + C::OFF_V);
    DecWalk<kTileR, kTileBT> walk(a, c, chunk, worker, per);
    DecPiece p;
    uint32_t n = 0, it = 0;       // tiles before this piece; pieces
    uint32_t pc[2] = {0, 0};      // PV steps per warpgroup
    uint32_t oc[2] = {0, 0};      // pieces in which the warpgroup had steps
    bool ok = true;
    while (ok && walk.next(p)) {
      const int pair = p.rows - p.rt * kTileR > kTileR / 2 ? 1 : 0;
      const int tiles = p.t1 - p.t0, steps = tiles << pair;
      ok = __all_sync(0xffffffffu, mbar_wait(q_full, it & 1, abort_flag));
      for (int u = 0; u < steps + 2 && ok; ++u) {
        const int h = u & 1;
        if (u >= 2) {  // PV of step u - 2
          const uint32_t x = n + ((u - 2) >> pair), vs = x % C::VS;
          ok = mbar_wait(p_full + h, pc[h] & 1, abort_flag) && mbar_wait(v_full + vs, (x / C::VS) & 1, abort_flag);
          if (u < 4 && oc[h] > 0) ok = ok && mbar_wait(o_free + h, (oc[h] - 1) & 1, abort_flag);
          if (!(ok = __all_sync(0xffffffffu, ok))) break;
          tc_fence_after();
          if (lane == 0) {
#pragma unroll
            for (int kk = 0; kk < 8; ++kk)
              mma_ts(tbase + C::TM_O + h * D, tbase + C::TM_S + h * 128 + kk * 8,
                     sdesc_sw128(sV + vs * C::TILE + kk * 2048, C::PANEL, 1024), IDESC_PV, u >= 4 || kk > 0);
            if (!pair || h == 1) mma_commit(v_empty + vs);
            if (u >= steps) mma_commit(o_full + h);  // the warpgroup's last
          }
          ++pc[h];
        }
        if (u < steps) {
          const uint32_t x = n + (u >> pair), ks = x % C::KS;
          ok = mbar_wait(k_full + ks, (x / C::KS) & 1, abort_flag);
          if (!(ok = __all_sync(0xffffffffu, ok))) break;
          tc_fence_after();
          if (lane == 0) {
            const uint32_t qa = sQ + (pair ? h * C::TILE : 0);
#pragma unroll
            for (int kk = 0; kk < D / 16; ++kk) {
              const uint32_t off = (kk >> 2) * C::PANEL + (kk & 3) * 32;
              mma_ss(tbase + C::TM_S + h * 128, sdesc_sw128(qa + off, 16, 1024), sdesc_sw128(sK + ks * C::TILE + off, 16, 1024),
                     IDESC_S, kk > 0);
            }
            mma_commit(s_full + h);
            if (!pair || h == 1) mma_commit(k_empty + ks);
            if (u == steps - 1) mma_commit(q_empty);
          }
        }
        __syncwarp();
      }
      n += tiles;
      ++it;
      if (steps > 0) ++oc[0];
      if (steps > 1) ++oc[1];
    }
    if (lane == 0) {
      mma_commit(done);
      mbar_wait_drain(done, 0, 200000000);
    }
    __syncwarp();
  };

  // Two warps gather the item's query rows (16-byte asynchronous copies, a row's
  // lanes side by side) as soon as the last S of the piece before is done, so
  // the loads run under that piece's last steps and its output.
  const auto query_role = [&]() {
    DecWalk<kTileR, kTileBT> walk(a, c, chunk, worker, per);
    DecPiece p;
    uint32_t it = 0;
    bool ok = true;
    constexpr int CPR = NP * 8, RPI = 32 / CPR;  // 16-byte pieces of a row; rows per warp instruction
    while (walk.next(p)) {
      const int left = p.rows - p.rt * kTileR, rows = left > kTileR / 2 ? kTileR : kTileR / 2;
      if (it > 0) ok = mbar_wait(q_empty, (it - 1) & 1, abort_flag);
      if (!(ok = __all_sync(0xffffffffu, ok))) break;
      for (int r0 = (warp - 10) * 32; r0 < rows; r0 += 64) {
        long long src = -1;  // this lane's row
        if (r0 + lane < left) {
          const DecRow d = dec_row(a, p.member0, p.hk, p.rt * kTileR + r0 + lane, p.len);
          src = (long long)d.tok * a.q_stride + (long long)d.head * a.D;
        }
#pragma unroll
        for (int i = 0; i < CPR; ++i) {
          const int x = r0 + i * RPI + lane / CPR, k = lane % CPR;
          const long long at = __shfl_sync(0xffffffffu, src, i * RPI + lane / CPR);
          const bool in = at >= 0 && k * 8 < a.D;
          const __nv_bfloat16* g = static_cast<const __nv_bfloat16*>(a.Q) + (in ? at + k * 8 : 0);
          uint8_t* dst = smem + C::OFF_Q + (x >> 7) * C::TILE + (k >> 3) * C::PANEL + (x & 127) * 128 + (((k & 7) ^ (x & 7)) << 4);
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
      }
      asm volatile("cp.async.wait_all;" ::: "memory");
      fence_proxy_async_smem();
      mbar_arrive(q_full);
      ++it;
    }
    __syncwarp();
  };

  const auto softmax_role = [&]() {
    const int h = warp >> 2, r = threadIdx.x & 127;  // warpgroup; row in its tile, TMEM lane
    const uint32_t tl = tbase + ((uint32_t)((warp & 3) * 32) << 16);
    const uint32_t sb = tl + C::TM_S + h * 128, ob = tl + C::TM_O + h * D;
    DecWalk<kTileR, kTileBT> walk(a, c, chunk, worker, per);
    DecPiece p;
    uint32_t n = 0, sc = 0, oc = 0;
    bool ok = true;
    while (ok && walk.next(p)) {
      int b, e;
      dec_range(a, p.kind, p.len, b, e);
      const int left = p.rows - p.rt * kTileR;
      const int pair = left > kTileR / 2 ? 1 : 0;
      const int tiles = p.t1 - p.t0, steps = tiles << pair;
      const int n_rows = min(pair ? left - h * 128 : left, 128);  // this warpgroup's rows
      const bool live = (warp & 3) * 32 < n_rows;                 // this warp has some
      float m_use = -INFINITY, l = 0.f;
      bool any = false;
      for (int u = h; u < steps; u += 2, ++sc) {
        any = true;
        const int t = p.t0 + (u >> pair), n_tok = min(e - t * kTileBT, kTileBT);
        if (n_tok < kTileBT) {  // clear V's rows behind the last token (both warpgroups of a pair: the same zeros)
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
        ok = mbar_wait(s_full + h, sc & 1, abort_flag);
        if (!(ok = __all_sync(0xffffffffu, ok))) break;
        tc_fence_after();
        if (live) {
          uint32_t sr[128];
          tmem_ld32(sb + 0, sr + 0);
          tmem_ld32(sb + 32, sr + 32);
          tmem_ld32(sb + 64, sr + 64);
          tmem_ld32(sb + 96, sr + 96);
          tmem_ld_wait();
          if (n_tok < kTileBT) {
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
      n += tiles;
      // the warpgroup's partial result
      const long long at = p.slot * kTileR + h * 128 + r;
      if (any) {
        ok = mbar_wait(o_full + h, oc & 1, abort_flag);
        if (!(ok = __all_sync(0xffffffffu, ok))) break;
        ++oc;
        tc_fence_after();
        if (live) {
          const float inv = l == 0.f ? 0.f : 1.f / l;
          if (r < n_rows) c.lse[at] = l == 0.f ? -INFINITY : m_use + log2f(l);
          // 8 columns of all rows side by side (tile_at): a warp's store covers 1 KB in one piece, where rows of
          // their own would scatter it over 32 lines
          float* dst = c.opart + tile_at(a.D, p.slot, h * 128 + r, 0);
#pragma unroll 1
          for (int k = 0; k < D / 32; ++k) {
            uint32_t orr[32];
            tmem_ld32(ob + k * 32, orr);
            tmem_ld_wait();
            if (r < n_rows) {
#pragma unroll
              for (int i = 0; i < 32; i += 4)
                if (k * 32 + i < a.D)
                  *reinterpret_cast<float4*>(dst + (k * 4 + (i >> 3)) * (kTileR * 8) + (i & 4)) =
                      make_float4(__uint_as_float(orr[i]) * inv, __uint_as_float(orr[i + 1]) * inv,
                                  __uint_as_float(orr[i + 2]) * inv, __uint_as_float(orr[i + 3]) * inv);
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
    else if (warp == 9)
      mma_role();
    else
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

// Kc or Vc as a 3-D map (D, page_size, n_pages * Hkv), boxes of 64 columns x `rows` tokens, 128-byte swizzle.
bool make_tmap_pages(CUtensorMap* map, const void* base, int D, int ps, long long heads, int rows) {
  encode_tiled_fn enc = get_encode_tiled();
  if (!enc) {
    set_error("cuTensorMapEncodeTiled is unavailable from the driver");
    return false;
  }
  cuuint64_t dims[3] = {(cuuint64_t)D, (cuuint64_t)ps, (cuuint64_t)heads};
  cuuint64_t strides[2] = {(cuuint64_t)D * 2, (cuuint64_t)ps * D * 2};
  cuuint32_t box[3] = {64, (cuuint32_t)rows, 1};
  cuuint32_t estr[3] = {1, 1, 1};
  CUresult r = enc(map, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 3, const_cast<void*>(base), dims, strides, box, estr,
                   CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                   CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
  if (r != CUDA_SUCCESS) {
    set_error("cuTensorMapEncodeTiled failed (%d) for pages of %d x %d, %lld of them", (int)r, ps, D, heads);
    return false;
  }
  return true;
}

template <int NP>
cudaError_t launch_rows(const CUtensorMap& mK, const CUtensorMap& mV, DecArgs a, const DecClass& c, int sms,
                        cudaStream_t s) {
  using C = RowsCfg<NP>;
  const size_t smem = C::smem(c.nseg);
  cudaError_t e = cudaFuncSetAttribute(k_decode_rows<NP>, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem);
  if (e != cudaSuccess) return e;
  a.workers = sms * C::CTAS * C::WARPS;
  a.min_units = 1;
  count_launch();
  return launch_pdl(k_decode_rows<NP>, dim3(sms * C::CTAS), dim3(C::WARPS * 32), smem, s, mK, mV, a, c);
}

template <int NP>
cudaError_t launch_tile(const CUtensorMap& mK, const CUtensorMap& mV, DecArgs a, const DecClass& c, int sms, int box_rows,
                        int heads, cudaStream_t s) {
  using C = TileCfg<NP>;
  const size_t smem = C::smem(c.nseg);
  cudaError_t e = cudaFuncSetAttribute(k_decode_tile<NP>, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem);
  if (e != cudaSuccess) return e;
  a.workers = sms;
  a.min_units = 1;
  count_launch();
  return launch_pdl(k_decode_tile<NP>, dim3(sms), dim3(C::THREADS), smem, s, mK, mV, a, c, box_rows, heads);
}

}  // namespace

bool decode_tc_supported(int D, int ps) { return D % 8 == 0 && D <= 256 && ps % 16 == 0; }

int decode_tc(const pt_decodeplan* p, DecArgs a, const DecClass& rows, const DecClass& tile, cudaStream_t s) {
  const long long heads = (long long)a.n_pages * a.Hkv;
  if (heads > INT_MAX - 1) {
    set_error("pt_attn_decode: %d pages of %d heads are out of range", a.n_pages, a.Hkv);
    return PT_ERR_INVALID_ARG;
  }
  CUtensorMap mK, mV;
  cudaError_t e = cudaSuccess;
  const int np = (a.D + 63) / 64;
  if (tile.nitems) {
    const int box = std::min(a.ps & -a.ps, kTileBT);  // the largest power of two that divides a page
    if (!make_tmap_pages(&mK, a.Kc, a.D, a.ps, heads, box) || !make_tmap_pages(&mV, a.Vc, a.D, a.ps, heads, box))
      return PT_ERR_CUDA;
    ProfScope ps(s, "decode_tile");
    e = np == 1 ? launch_tile<1>(mK, mV, a, tile, p->sms, box, (int)heads, s)
                : launch_tile<2>(mK, mV, a, tile, p->sms, box, (int)heads, s);
  }
  if (e == cudaSuccess && rows.nitems) {
    if (!make_tmap_pages(&mK, a.Kc, a.D, a.ps, heads, 16) || !make_tmap_pages(&mV, a.Vc, a.D, a.ps, heads, 16))
      return PT_ERR_CUDA;
    ProfScope ps(s, "decode_rows");
    e = np == 1   ? launch_rows<1>(mK, mV, a, rows, p->sms, s)
        : np == 2 ? launch_rows<2>(mK, mV, a, rows, p->sms, s)
        : np == 3 ? launch_rows<3>(mK, mV, a, rows, p->sms, s)
                  : launch_rows<4>(mK, mV, a, rows, p->sms, s);
  }
  if (e == cudaSuccess) e = cudaGetLastError();
  if (e != cudaSuccess) {
    set_error("pt_attn_decode: launch failed: %s", cudaGetErrorString(e));
    return PT_ERR_CUDA;
  }
  return PT_OK;
}

}  // namespace pt
