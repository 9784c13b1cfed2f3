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

// Kc or Vc as a 3-D map (D, page_size, n_pages * Hkv), boxes of 64 columns x 16 tokens, 128-byte swizzle.
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

}  // namespace

bool decode_tc_supported(int D, int ps) { return D % 8 == 0 && D <= 256 && ps % 16 == 0; }

int decode_tc(const pt_decodeplan* p, DecArgs a, const DecClass& rows, const DecClass& tile, cudaStream_t s) {
  CUtensorMap mK, mV;
  const long long heads = (long long)a.n_pages * a.Hkv;
  if (heads > INT_MAX) {
    set_error("pt_attn_decode: %d pages of %d heads are out of range", a.n_pages, a.Hkv);
    return PT_ERR_INVALID_ARG;
  }
  if (!make_tmap_pages(&mK, a.Kc, a.D, a.ps, heads, 16) || !make_tmap_pages(&mV, a.Vc, a.D, a.ps, heads, 16))
    return PT_ERR_CUDA;
  cudaError_t e = cudaSuccess;
  const int np = (a.D + 63) / 64;
  e = np == 1   ? launch_rows<1>(mK, mV, a, rows, p->sms, s)
      : np == 2 ? launch_rows<2>(mK, mV, a, rows, p->sms, s)
      : np == 3 ? launch_rows<3>(mK, mV, a, rows, p->sms, s)
                : launch_rows<4>(mK, mV, a, rows, p->sms, s);
  if (e == cudaSuccess) e = cudaGetLastError();
  if (e != cudaSuccess) {
    set_error("pt_attn_decode: launch failed: %s", cudaGetErrorString(e));
    return PT_ERR_CUDA;
  }
  return PT_OK;
}

}  // namespace pt
