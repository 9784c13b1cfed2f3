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
#include <vector>

#include "pt.h"
#include "pt_decode.cuh"
#include "pt_internal.h"

namespace pt {
int take_status_decode(cudaStream_t s) {
  const int a = take_status_here(s), b = take_status_decode_tc(s);
  return a < 0 || b < 0 ? -1 : a ? a : b;
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
// CUDA cores: a warp per worker, kSimtR = 4 query rows, 16 tokens a step.
//
// Lanes hold the columns (DL each, VEC of them contiguous), so a token's key
// is one coalesced load, and four keys against four rows leave 16 partial dot
// products per lane.  These are summed over the lanes by halves: each exchange
// adds one half of the values to the partner's and keeps the other, 16
// shuffles for 16 sums where a butterfly for each would take 80, and lane l
// ends with row l/8, token (l/2) mod 4 of the group.  The softmax then runs on
// eight lanes a row.  Bound by memory for the four rows of a small group:
// about 28 instructions a token at head_dim 64, 512 bytes of keys and values.
// ---------------------------------------------------------------------------
template <class E, int DL, int VEC>
__global__ void __launch_bounds__(256, DL >= 16 ? 1 : 2) k_decode_simt(const DecArgs a, const DecClass c) {
  pdl_wait();
  extern __shared__ long long chunk[];
  const long long per = dec_scan<kSimtR, kSimtBT>(a, c, chunk);
  const int lane = threadIdx.x & 31;
  constexpr int R = kSimtR, NV = DL / VEC;
  using V = VecOf<E, VEC>;
  const E* Qp = static_cast<const E*>(a.Q);
  DecWalk<R, kSimtBT> walk(a, c, chunk, (long long)blockIdx.x * 8 + (threadIdx.x >> 5), per);
  DecPiece p;
  const int my_r = lane >> 3;  // the row whose scores this lane holds
  while (walk.next(p)) {
    const int len = dec_len(a, p.node, false);
    int b, e;
    dec_range(a, p.kind, len, b, e);
    float q[R][DL], acc[R][DL];
    int lim_max = 0, lim_min = INT_MAX, my_lim = 0;
    int lim[R];
#pragma unroll
    for (int r = 0; r < R; ++r) {
      const int row = p.rt * R + r;
      lim[r] = 0;
      const E* src = nullptr;
      if (row < p.rows) {
        const DecRow d = dec_row(a, p.node, p.hk, row, len);
        lim[r] = d.lim;
        src = Qp + (long long)(d.s * a.q_len + d.j) * a.q_stride + (long long)d.head * a.D;
      }
      lim_max = max(lim_max, lim[r]);
      lim_min = min(lim_min, lim[r]);
      if (r == my_r) my_lim = lim[r];
#pragma unroll
      for (int i = 0; i < DL; ++i) {
        const int col = (i / VEC * 32 + lane) * VEC + i % VEC;
        q[r][i] = src && col < a.D ? to_f(src[col]) * a.scale_log2 : 0.f;
        acc[r][i] = 0.f;
      }
    }
    float m = -INFINITY, l = 0.f;  // of row my_r, the same on its eight lanes
    for (int t = p.t0; t < p.t1; ++t) {
      const int kv0 = b + t * kSimtBT, n = min(min(kSimtBT, e - kv0), lim_max - kv0);
      if (n <= 0) break;
      // lane i's row of the cache: token kv0 + i
      long long off = 0;
      if (lane < n) {
        const int pi = (kv0 + lane) / a.ps;
        off = (((long long)dec_page(a, p.node, pi) * a.Hkv + p.hk) * a.ps + (kv0 + lane - pi * a.ps)) * a.D;
      }
      float s[4];
#pragma unroll
      for (int gq = 0; gq < 4; ++gq) {
        float d[16];
#pragma unroll
        for (int i = 0; i < 16; ++i) d[i] = 0.f;
        if (gq * 4 < n) {
#pragma unroll
          for (int u = 0; u < 4; ++u) {
            const long long o = __shfl_sync(0xffffffffu, off, gq * 4 + u);
            const E* kp = static_cast<const E*>(a.Kc) + o;
            const bool in = gq * 4 + u < n;
#pragma unroll
            for (int v = 0; v < NV; ++v) {
              const int col = (v * 32 + lane) * VEC;
              V kk;
              if (in && col < a.D) {
                kk = *reinterpret_cast<const V*>(kp + col);
#pragma unroll
                for (int x = 0; x < VEC; ++x)
#pragma unroll
                  for (int r = 0; r < R; ++r) d[r * 4 + u] = fmaf(q[r][v * VEC + x], to_f(kk.e[x]), d[r * 4 + u]);
              }
            }
          }
        }
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
        s[gq] = kv < kv0 + n && kv < my_lim ? d[0] : -INFINITY;
      }
      float mt = fmaxf(fmaxf(s[0], s[1]), fmaxf(s[2], s[3]));
      mt = fmaxf(mt, __shfl_xor_sync(0xffffffffu, mt, 2));
      mt = fmaxf(mt, __shfl_xor_sync(0xffffffffu, mt, 4));
      const float mn = fmaxf(m, mt), ref = mn == -INFINITY ? 0.f : mn;
      const float al = ex2(m - ref);
      m = mn;
      float sum = 0.f;
#pragma unroll
      for (int gq = 0; gq < 4; ++gq) s[gq] = ex2(s[gq] - ref), sum += s[gq];
      sum += __shfl_xor_sync(0xffffffffu, sum, 2);
      sum += __shfl_xor_sync(0xffffffffu, sum, 4);
      l = fmaf(l, al, sum);
#pragma unroll
      for (int r = 0; r < R; ++r) {
        const float ar = __shfl_sync(0xffffffffu, al, r * 8);
#pragma unroll
        for (int i = 0; i < DL; ++i) acc[r][i] *= ar;
      }
      const bool all_kept = kv0 + n <= lim_min;
#pragma unroll
      for (int i = 0; i < kSimtBT; ++i) {
        if (i >= n) break;
        const long long o = __shfl_sync(0xffffffffu, off, i);
        const E* vp = static_cast<const E*>(a.Vc) + o;
        float pr[R];
#pragma unroll
        for (int r = 0; r < R; ++r) pr[r] = __shfl_sync(0xffffffffu, s[i >> 2], r * 8 + (i & 3) * 2);
#pragma unroll
        for (int v = 0; v < NV; ++v) {
          const int col = (v * 32 + lane) * VEC;
          if (col < a.D) {
            const V vv = *reinterpret_cast<const V*>(vp + col);
#pragma unroll
            for (int x = 0; x < VEC; ++x)
#pragma unroll
              for (int r = 0; r < R; ++r)  // a value that the row must not see does not reach it, whatever it is
                if (all_kept || kv0 + i < lim[r])
                  acc[r][v * VEC + x] = fmaf(pr[r], to_f(vv.e[x]), acc[r][v * VEC + x]);
          }
        }
      }
    }
    // the piece's partial result
#pragma unroll
    for (int r = 0; r < R; ++r) {
      if (p.rt * R + r >= p.rows) break;
      const float lr = __shfl_sync(0xffffffffu, l, r * 8), mr = __shfl_sync(0xffffffffu, m, r * 8);
      const float inv = lr == 0.f ? 0.f : 1.f / lr;
      const long long row = p.slot * R + r;
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
// along each segment, so the sum's order is fixed.  A block takes one query
// token's q head; its warps take every fourth piece, lanes the columns.
// ---------------------------------------------------------------------------
struct MergeArgs {
  DecArgs d;
  DecClass c0, c1;    // the classes of the path entries: first, second
  int first;          // class number of c0
  int R0, R1, BT0, BT1;
  const int* path_ptr;
  const int2* path_ent;
  int n_samples;
  void* O;
  float* LSE;
};

template <int CPL>  // columns per lane
__device__ __forceinline__ void merge_row(const MergeArgs& m, int s, int j, int head, int warp, int lane, float& mx,
                                          float& sum, float (&acc)[CPL]) {
  const DecArgs& a = m.d;
  int turn = 0;  // pieces so far, mod 4
  const int hk = head / a.g;
  for (int k = m.path_ptr[s]; k < m.path_ptr[s + 1]; ++k) {
    const int2 en = m.path_ent[k];
    const bool first = (en.x >> 28) == m.first;
    const DecClass& c = first ? m.c0 : m.c1;
    const int R = first ? m.R0 : m.R1, BT = first ? m.BT0 : m.BT1;
    const int si = en.x & ((1 << 28) - 1);
    const int4 sg = c.seg[si];
    int b, e;
    dec_range(a, sg.y, dec_len(a, sg.x, false), b, e);
    const int tiles = (e - b + BT - 1) / BT;
    if (tiles == 0) continue;
    const int row = (en.y * a.q_len + j) * a.g + head - hk * a.g;
    const int rt = row / R, it = rt * a.Hkv + hk;
    const long long per = c.pref[c.nseg], u0 = c.pref[si] + (long long)it * tiles;
    const long long w0 = u0 / per, w1 = (u0 + tiles - 1) / per;
    for (long long w = w0 + ((warp - turn) & 3); w <= w1; w += 4) {
      const long long at = (w + sg.w + it) * R + (row - rt * R);
      const float x = c.lse[at];
      float o[CPL];
#pragma unroll
      for (int i = 0; i < CPL; ++i) o[i] = lane + i * 32 < a.D ? c.opart[at * a.D + lane + i * 32] : 0.f;
      if (x == -INFINITY) continue;
      const float mn = fmaxf(mx, x), al = ex2(mx - mn), f = ex2(x - mn);
      mx = mn;
      sum = fmaf(sum, al, f);
#pragma unroll
      for (int i = 0; i < CPL; ++i) acc[i] = fmaf(acc[i], al, f * o[i]);
    }
    turn = (int)((turn + (w1 - w0 + 1)) & 3);
  }
}

template <class E, int CPL>
__global__ void __launch_bounds__(128) k_decode_merge(const MergeArgs m) {
  pdl_wait();
  __shared__ float sm_m[4], sm_l[4];
  __shared__ float sm_o[4][CPL * 32];
  const DecArgs& a = m.d;
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int head = blockIdx.x % a.Hq, tok = blockIdx.x / a.Hq, s = tok / a.q_len, j = tok - s * a.q_len;
  if (a.q_count) {
    const int n = a.q_count[s];
    if ((n < 0 || n > a.q_len) && threadIdx.x == 0) record_status(PT_STATUS_INVALID);
    if (j >= dec_count(a, s)) return;  // the row stays as it was
  }
  float mx = -INFINITY, sum = 0.f, acc[CPL];
#pragma unroll
  for (int i = 0; i < CPL; ++i) acc[i] = 0.f;
  merge_row<CPL>(m, s, j, head, warp, lane, mx, sum, acc);
  if (lane == 0) sm_m[warp] = mx, sm_l[warp] = sum;
#pragma unroll
  for (int i = 0; i < CPL; ++i) sm_o[warp][lane + i * 32] = acc[i];
  __syncthreads();
  float top = fmaxf(fmaxf(sm_m[0], sm_m[1]), fmaxf(sm_m[2], sm_m[3]));
  float f[4], all = 0.f;
#pragma unroll
  for (int w = 0; w < 4; ++w) {
    f[w] = sm_m[w] == -INFINITY ? 0.f : ex2(sm_m[w] - top);
    all = fmaf(f[w], sm_l[w], all);
  }
  const float inv = all == 0.f ? 0.f : 1.f / all;
  E* O = static_cast<E*>(m.O) + ((long long)tok * a.Hq + head) * a.D;
  for (int col = threadIdx.x; col < a.D; col += 128) {
    float v = 0.f;
#pragma unroll
    for (int w = 0; w < 4; ++w) v = fmaf(f[w], sm_o[w][col], v);
    v *= inv;
    if constexpr (sizeof(E) == 2)
      O[col] = __float2bfloat16_rn(v);
    else
      O[col] = v;
  }
  if (threadIdx.x == 0)
    m.LSE[(long long)head * m.n_samples * a.q_len + tok] = all == 0.f ? -INFINITY : (top + log2f(all)) * 0.69314718055994531f;
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
  const size_t R = cls == kDecSimt ? kSimtR : cls == kDecRows ? kRowsR : kTileR;
  const size_t slots = (size_t)c.nitems + dec_workers(p, cls);
  return pad256(8 * ((size_t)c.nseg + 1)) + pad256(4 * slots * R) + pad256(4 * slots * R * D);
}

DecClass class_args(const pt_decodeplan* p, int cls, int D, char*& ws) {
  const pt_decodeplan::Class& c = p->cls[cls];
  DecClass d = {};
  d.seg = c.seg;
  d.nseg = c.nseg;
  d.nitems = c.nitems;
  if (!c.nitems) return d;
  const size_t R = cls == kDecSimt ? kSimtR : cls == kDecRows ? kRowsR : kTileR;
  const size_t slots = (size_t)c.nitems + dec_workers(p, cls);
  d.pref = reinterpret_cast<long long*>(ws), ws += pad256(8 * ((size_t)c.nseg + 1));
  d.lse = reinterpret_cast<float*>(ws), ws += pad256(4 * slots * R);
  d.opart = reinterpret_cast<float*>(ws), ws += pad256(4 * slots * R * D);
  return d;
}

size_t ws_bytes(const pt_decodeplan* p, int D) {
  size_t n = std::max(class_bytes(p, kDecSimt, D), (size_t)256);
  if (D <= 256) n = std::max(n, class_bytes(p, kDecRows, D) + class_bytes(p, kDecTile, D));
  return n;
}

template <class E>
cudaError_t launch_simt(const DecArgs& a, const DecClass& c, int grid, size_t smem, cudaStream_t s) {
  const int D = a.D;
  auto go = [&](auto kernel) { return launch_pdl(kernel, dim3(grid), dim3(256), smem, s, a, c); };
  if (D <= 32) return go(k_decode_simt<E, 1, 1>);
  if (D <= 64) return D % 2 ? go(k_decode_simt<E, 2, 1>) : go(k_decode_simt<E, 2, 2>);
  if (D <= 128) return D % 4 ? go(k_decode_simt<E, 4, 1>) : go(k_decode_simt<E, 4, 4>);
  if (D <= 256) return D % 4 ? go(k_decode_simt<E, 8, 1>) : go(k_decode_simt<E, 8, 4>);
  return D % 4 ? go(k_decode_simt<E, 16, 1>) : go(k_decode_simt<E, 16, 4>);
}

template <class E>
cudaError_t launch_merge(const MergeArgs& m, cudaStream_t s) {
  const int grid = m.n_samples * m.d.q_len * m.d.Hq, D = m.d.D;
  auto go = [&](auto kernel) { return launch_pdl(kernel, dim3(grid), dim3(128), 0, s, m); };
  if (D <= 64) return go(k_decode_merge<E, 2>);
  if (D <= 128) return go(k_decode_merge<E, 4>);
  if (D <= 256) return go(k_decode_merge<E, 8>);
  return go(k_decode_merge<E, 16>);
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
  if ((long long)S * q_len * Hq > INT_MAX / 2) {
    set_error("%s: %d samples of %d tokens and %d heads are out of range", who, S, q_len, Hq);
    return PT_ERR_INVALID_ARG;
  }
  if (N > kDecMaxSegs) {
    set_error("%s: %d nodes, more than %d", who, N, kDecMaxSegs);
    return PT_ERR_UNSUPPORTED;
  }
  if (path_ptr[0] != 0) {
    set_error("%s: path_ptr[0] must be 0", who);
    return PT_ERR_INVALID_ARG;
  }
  std::vector<int32_t> np(N + 1, 0), leaf(std::max(S, 1), 0), seen(std::max(N, 1), -1);
  std::vector<uint8_t> is_leaf(std::max(N, 1), 0);
  for (int s = 0; s < S; ++s) {
    if (path_ptr[s + 1] <= path_ptr[s]) {
      set_error("%s: sample path %d is empty", who, s);
      return PT_ERR_INVALID_ARG;
    }
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
  // segments of each class, and each node's segments ({class << 28 | index}, at most two)
  std::vector<int4> seg[kDecClasses];
  long long items[kDecClasses] = {0, 0, 0};
  std::vector<int2> of[2];
  of[0].assign(std::max(N, 1), make_int2(-1, -1));
  of[1].assign(std::max(N, 1), make_int2(-1, -1));
  auto add = [&](int cls, int node, int kind, long long rows) {
    const int R = cls == kDecSimt ? kSimtR : cls == kDecRows ? kRowsR : kTileR;
    seg[cls].push_back(make_int4(node, kind, (int)rows, (int)std::min<long long>(items[cls], INT_MAX)));
    items[cls] += (rows + R - 1) / R * Hkv;
    return cls << 28 | (int)(seg[cls].size() - 1);
  };
  for (int i = 0; i < N; ++i) {
    const long long rows = (long long)(np[i + 1] - np[i]) * q_len * g;
    if (!rows) continue;
    of[0][i].x = add(kDecSimt, i, kSegFull, rows);
    of[1][i].x = add(kDecRows, i, kSegFull, rows);
  }
  for (int c = 0; c < kDecClasses; ++c)
    if (items[c] > INT_MAX / 512) {
      set_error("%s: %lld work items are out of range", who, items[c]);
      return PT_ERR_INVALID_ARG;
    }
  std::vector<int32_t> pptr[2];
  std::vector<int2> pent[2];
  for (int v = 0; v < 2; ++v) {
    pptr[v].assign(S + 1, 0);
    for (int s = 0; s < S; ++s) {
      for (int k = path_ptr[s]; k < path_ptr[s + 1]; ++k) {
        const int2 o = of[v][path_nodes[k]];
        if (o.x >= 0) pent[v].push_back(make_int2(o.x, member[k]));
        if (o.y >= 0) pent[v].push_back(make_int2(o.y, member[k]));
      }
      pptr[v][s + 1] = (int32_t)pent[v].size();
    }
  }
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
  const size_t o_np = put(np.data(), 4 * np.size()), o_samp = put(samp.data(), 4 * (size_t)E),
               o_leaf = put(leaf.data(), 4 * (size_t)S);
  size_t o_seg[kDecClasses], o_pp[2], o_pe[2];
  for (int c = 0; c < kDecClasses; ++c) o_seg[c] = put(seg[c].data(), sizeof(int4) * seg[c].size());
  for (int v = 0; v < 2; ++v) {
    o_pp[v] = put(pptr[v].data(), 4 * pptr[v].size());
    o_pe[v] = put(pent[v].data(), sizeof(int2) * pent[v].size());
  }
  pt_decodeplan* p = new pt_decodeplan();
  p->device = dev;
  p->sms = num_sms(dev);
  p->stream = stream;
  p->N = N, p->S = S, p->Hq = Hq, p->Hkv = Hkv, p->q_len = q_len;
  int rc = pool_alloc(&p->mem, host.size(), dev, stream);
  if (rc) {
    delete p;
    return (pt_status)rc;
  }
  char* base = static_cast<char*>(p->mem);
  p->node_ptr = reinterpret_cast<int32_t*>(base + o_np);
  p->node_samp = reinterpret_cast<int32_t*>(base + o_samp);
  p->leaf = reinterpret_cast<int32_t*>(base + o_leaf);
  for (int c = 0; c < kDecClasses; ++c) {
    p->cls[c].seg = reinterpret_cast<int4*>(base + o_seg[c]);
    p->cls[c].nseg = (int32_t)seg[c].size();
    p->cls[c].nitems = (int32_t)items[c];
  }
  for (int v = 0; v < 2; ++v) {
    p->path_ptr[v] = reinterpret_cast<int32_t*>(base + o_pp[v]);
    p->path_ent[v] = reinterpret_cast<int2*>(base + o_pe[v]);
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

extern "C" pt_status pt_attn_decode(const void* Q, int64_t q_stride, const void* Kc, const void* Vc, pt_dtype dtype,
                                    int32_t D, int32_t n_pages, int32_t page_size, const int32_t* tables,
                                    int32_t max_pages, const int32_t* lens, const int32_t* q_count, float scale,
                                    const pt_decodeplan* plan, void* O, float* LSE, void* workspace,
                                    size_t workspace_bytes, cudaStream_t stream) {
  static const char* who = "pt_attn_decode";
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
  a.node_ptr = plan->node_ptr, a.node_samp = plan->node_samp, a.leaf = plan->leaf;
  a.lens = lens, a.tables = tables, a.q_count = q_count;
  a.Q = Q, a.Kc = Kc, a.Vc = Vc, a.q_stride = q_stride;
  a.q_len = plan->q_len, a.Hq = plan->Hq, a.Hkv = plan->Hkv, a.g = plan->Hq / plan->Hkv, a.D = D;
  a.ps = page_size, a.max_pages = max_pages, a.n_pages = n_pages;
  a.scale_log2 = scale * 1.4426950408889634f;
  char* ws = static_cast<char*>(workspace);
  MergeArgs m = {};
  m.n_samples = plan->S;
  m.O = O;
  m.LSE = LSE;
  const bool tc = dtype == PT_BF16 && decode_tc_supported(D, page_size);
  cudaError_t e = cudaSuccess;
  if (tc) {
    m.first = kDecRows;
    m.c0 = class_args(plan, kDecRows, D, ws);
    m.c1 = class_args(plan, kDecTile, D, ws);
    m.R0 = kRowsR, m.BT0 = kRowsBT, m.R1 = kTileR, m.BT1 = kTileBT;
    ProfScope ps(stream, "decode_tc");
    const int rc = decode_tc(plan, a, m.c0, m.c1, stream);
    if (rc) return (pt_status)rc;
  } else {
    m.first = kDecSimt;
    m.c0 = class_args(plan, kDecSimt, D, ws);
    m.R0 = kSimtR, m.BT0 = kSimtBT;
    a.workers = dec_workers(plan, kDecSimt);
    a.min_units = 2;
    const size_t smem = 8 * (((size_t)m.c0.nseg + 31) / 32 + 1);
    ProfScope ps(stream, "decode_simt");
    e = dtype == PT_BF16 ? launch_simt<__nv_bfloat16>(a, m.c0, a.workers / 8, smem, stream)
                         : launch_simt<float>(a, m.c0, a.workers / 8, smem, stream);
    count_launch();
    if (int rc = launch_status(who, e)) return (pt_status)rc;
  }
  m.d = a;
  m.path_ptr = plan->path_ptr[tc ? 1 : 0];
  m.path_ent = plan->path_ent[tc ? 1 : 0];
  {
    ProfScope ps(stream, "decode_merge");
    e = dtype == PT_BF16 ? launch_merge<__nv_bfloat16>(m, stream) : launch_merge<float>(m, stream);
    count_launch();
  }
  return (pt_status)launch_status(who, e);
}
