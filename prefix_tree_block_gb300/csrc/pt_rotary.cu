// pt_rotary.cu -- rotary positions of one or several axes on the heads of a
// projection, and the inverse rotation.
//
// "cp=1 shared-prefix prefix-tree attention for rollouts" (PR description): a
// completion's position ids continue from its prompt's.  pt_fold_positions,
// pt_cache_tables and pt_draft_tree give those ids; this call turns them into
// rotations of Q's and K's columns.
#include <cuda_bf16.h>

#include <algorithm>
#include <climits>

#include "pt.h"
#include "pt_device.cuh"
#include "pt_internal.h"

using namespace pt;

namespace {

struct RotArgs {
  const char* X;
  char* Y;
  long long x_stride, y_stride;  // bytes between tokens
  const long long* pos;          // [axes][T]
  const float* inv_freq;         // [half]
  int cut[3];                    // the first pairs of axes 1, 2 and 3
  int T, H, D, half;
  int tokens, lanes;  // tokens of a CTA; threads that share a token's heads
  int inverse, copy;  // negative angles; whether the columns behind the rotated ones have to be copied
};

// inv_freq / 2 pi as a fraction of 2^64, modulo 1: a position's turns are then
// one wrapping integer product, exact however far the position is.  With f =
// m 2^e, m of 24 bits, and 1 / 2 pi to 128 bits, what is cut off is below 2^-64
// of a turn for each position up to |inv_freq| = 2^20.
__device__ __forceinline__ unsigned long long turns_of(float f) {
  const unsigned bits = __float_as_uint(f);
  const int ex = (int)((bits >> 23) & 255u);
  const unsigned long long m = (bits & 0x7fffffu) | (ex ? 0x800000u : 0u);
  const int e = max(ex, 1) - 150;  // f = m 2^e
  constexpr unsigned long long kHi = 0x28be60db9391054aull, kLo = 0x7f09d5f47d4d3770ull;  // 2^128 / 2 pi
  // m / 2 pi, its integer part and 64 + 64 bits behind the point
  const unsigned long long lo = m * kLo, c = __umul64hi(m, kLo), mid = m * kHi + c;
  const unsigned long long top = __umul64hi(m, kHi) + (mid < c);
  unsigned long long r;
  if (e == 0)
    r = mid;
  else if (e > 0)
    r = e < 64 ? mid << e | lo >> (64 - e) : 0;
  else if (e > -64)
    r = mid >> -e | top << (64 + e);
  else
    r = e > -128 ? top >> (-64 - e) : 0;
  return bits >> 31 ? 0 - r : r;
}

// The angles of a CTA's tokens in shared memory (cosines, then sines, a row of
// `half` each per token), for every head once.
__device__ __forceinline__ void angles(const RotArgs& a, int t0, int n, float* cs, float* sn) {
#pragma unroll 1
  for (int x = threadIdx.x; x < n * a.half; x += blockDim.x) {
    const int t = x / a.half, i = x - t * a.half;
    const int axis = (i >= a.cut[0]) + (i >= a.cut[1]) + (i >= a.cut[2]);
    const float f = a.inv_freq[i];
    const long long turns = (long long)((unsigned long long)a.pos[(long long)axis * a.T + t0 + t] * turns_of(f));
    float s, c;
    sincospif(__ll2float_rn(turns) * 1.0842021724855044e-19f, &s, &c);  // 2^-63: half turns
    if (!(fabsf(f) < 2147483648.f)) s = c = __uint_as_float(0x7fc00000u);  // infinite or NaN
    cs[x] = c;
    sn[x] = a.inverse ? -s : s;
  }
}

template <class E>
__device__ __forceinline__ float up(E x) {
  if constexpr (sizeof(E) == 2)
    return __bfloat162float(x);
  else
    return x;
}
template <class E>
__device__ __forceinline__ E down(float x) {
  if constexpr (sizeof(E) == 2)
    return __float2bfloat16_rn(x);
  else
    return x;
}

template <class E, int V>
struct alignas(sizeof(E) * V) RotVec {
  E e[V];
};

// One pass: every element is read and written once, products in fp32, one
// rounding.  A CTA takes some tokens, all their heads; its angles are computed
// once, while its first vectors are on their way.  V elements a vector; NEAR:
// pairs lie side by side (V of them in two vectors one after the other), else
// half the rotated columns apart.  A thread keeps V pairs' sines and cosines and
// turns them in every `lanes`-th head of one token, U heads in flight.  It holds
// what it loaded until it stores, so Y may be X.
// Bound by memory: 27687 tokens of 40 heads of 128 out of 48 (bf16, three axes, 568
// MB) 89 us, 94% of the copy's bandwidth; 2048 tokens 6.9 us.  One head a thread 137
// us, two 128, four 97 (its angles' share grows); four heads in flight instead of two
// 114 (registers, then CTAs), four CTAs an SM 106 (spills).
template <class E, int V, bool NEAR, int U>
__global__ void __launch_bounds__(V == 1 ? 512 : 256, V == 1 ? 2 : 3) k_rotary(const RotArgs a) {
  using Vec = RotVec<E, V>;
  extern __shared__ float sm[];
  pdl_wait();
  const int t0 = blockIdx.x * a.tokens, n = min(a.tokens, a.T - t0);
  float *cs = sm, *sn = sm + a.tokens * a.half;
  const int per = a.half / V;  // groups of V pairs
  const int x = threadIdx.x / per, i = (threadIdx.x - x * per) * V, t = x / a.lanes, h0 = x - t * a.lanes;
  const long long apart = NEAR ? V : a.half;
  const E* src = reinterpret_cast<const E*>(a.X + (t0 + t) * a.x_stride) + (NEAR ? 2 * i : i);
  E* dst = reinterpret_cast<E*>(a.Y + (t0 + t) * a.y_stride) + (NEAR ? 2 * i : i);
  const int H = t < n ? a.H : 0;  // (no heads for threads behind the last token)
  Vec p[U], q[U];
  auto load = [&](int h) {
#pragma unroll
    for (int u = 0; u < U; ++u)
      if (h + u * a.lanes < H) {
        p[u] = *reinterpret_cast<const Vec*>(src + (h + u * a.lanes) * a.D);
        q[u] = *reinterpret_cast<const Vec*>(src + (h + u * a.lanes) * a.D + apart);
      }
  };
  load(h0);
  angles(a, t0, n, cs, sn);
  __syncthreads();
  if (t < n) {
    float c[V], s[V];
#pragma unroll
    for (int k = 0; k < V; ++k) c[k] = cs[t * a.half + i + k], s[k] = sn[t * a.half + i + k];
#pragma unroll 1
    for (int h = h0; h < H; h += U * a.lanes) {
      if (h != h0) load(h);
#pragma unroll
      for (int u = 0; u < U; ++u)
        if (h + u * a.lanes < H) {
          Vec y, z;
#pragma unroll
          for (int k = 0; k < V; ++k) {
            if constexpr (NEAR && V > 1) {  // pair k: elements 2k and 2k + 1 of the two vectors
              const Vec& w = 2 * k < V ? p[u] : q[u];
              Vec& o = 2 * k < V ? y : z;
              const float f = up(w.e[2 * k % V]), g = up(w.e[2 * k % V + 1]);
              o.e[2 * k % V] = down<E>(f * c[k] - g * s[k]);
              o.e[2 * k % V + 1] = down<E>(g * c[k] + f * s[k]);
            } else {
              const float f = up(p[u].e[k]), g = up(q[u].e[k]);
              y.e[k] = down<E>(f * c[k] - g * s[k]);
              z.e[k] = down<E>(g * c[k] + f * s[k]);
            }
          }
          E* to = dst + (h + u * a.lanes) * a.D;
          *reinterpret_cast<Vec*>(to) = y;
          *reinterpret_cast<Vec*>(to + apart) = z;
        }
    }
  }
  if (a.copy) {  // columns behind the rotated ones
    const int rest = a.D / V - 2 * per, all = n * a.H * rest;
#pragma unroll 1
    for (int y = threadIdx.x; y < all; y += blockDim.x) {
      const int th = y / rest, tt = th / a.H;
      const long long col = (long long)(th - tt * a.H) * a.D + 2 * a.half + (y - th * rest) * V;
      *reinterpret_cast<Vec*>(reinterpret_cast<E*>(a.Y + (t0 + tt) * a.y_stride) + col) =
          *reinterpret_cast<const Vec*>(reinterpret_cast<const E*>(a.X + (t0 + tt) * a.x_stride) + col);
    }
  }
}

template <class E, bool NEAR>
cudaError_t launch(const RotArgs& a, int unit, dim3 grid, int threads, size_t smem, cudaStream_t s) {
  auto go = [&](auto kernel) { return launch_pdl(kernel, grid, dim3(threads), smem, s, a); };
  if (unit == 16) return go(k_rotary<E, 16 / (int)sizeof(E), NEAR, 2>);
  if (unit == 8) return go(k_rotary<E, 8 / (int)sizeof(E), NEAR, 2>);
  return go(k_rotary<E, 1, NEAR, 2>);
}

}  // namespace

extern "C" pt_status pt_rotary(const void* X, int64_t x_stride, pt_dtype dtype, int32_t T, int32_t H, int32_t D,
                               const int64_t* positions, const float* inv_freq, int32_t rot_dim,
                               const int32_t* sections, int32_t n_axes, int32_t interleaved, int32_t inverse, void* Y,
                               int64_t y_stride, cudaStream_t stream) {
  static const char* who = "pt_rotary";
  if (dtype != PT_BF16 && dtype != PT_F32) {
    set_error("%s: unknown dtype %d", who, (int)dtype);
    return PT_ERR_INVALID_ARG;
  }
  const int es = dtype == PT_BF16 ? 2 : 4;
  if (T < 0 || H < 0 || D < 1 || (long long)H * D > INT_MAX / 4) {
    set_error("%s: T = %d, H = %d or D = %d out of range", who, T, H, D);
    return PT_ERR_INVALID_ARG;
  }
  if (rot_dim < 2 || rot_dim > D || rot_dim % 2) {
    set_error("%s: rot_dim = %d must be even and at most the head_dim %d", who, rot_dim, D);
    return PT_ERR_INVALID_ARG;
  }
  if (rot_dim > 1024) {
    set_error("%s: rot_dim = %d, more than 1024", who, rot_dim);
    return PT_ERR_UNSUPPORTED;
  }
  const int half = rot_dim / 2;
  RotArgs a = {};
  if (n_axes < 1 || n_axes > 4) {
    set_error("%s: %d axes, 1 to 4 wanted", who, n_axes);
    return n_axes < 1 ? PT_ERR_INVALID_ARG : PT_ERR_UNSUPPORTED;
  }
  if (n_axes > 1 && !sections) {
    set_error("%s: %d axes without sections", who, n_axes);
    return PT_ERR_INVALID_ARG;
  }
  long long sum = 0;
  for (int i = 0; i < 3; ++i) a.cut[i] = INT_MAX;
  for (int i = 0; sections && i < n_axes; ++i) {
    if (sections[i] < 0) {
      set_error("%s: section %d has %d pairs", who, i, sections[i]);
      return PT_ERR_INVALID_ARG;
    }
    sum += sections[i];
    if (i + 1 < n_axes) a.cut[i] = (int)std::min<long long>(sum, INT_MAX);
  }
  if (sections && sum != half) {
    set_error("%s: the sections have %lld pairs, rot_dim / 2 is %d", who, sum, half);
    return PT_ERR_INVALID_ARG;
  }
  if (x_stride < (int64_t)H * D || y_stride < (int64_t)H * D) {
    set_error("%s: tokens %lld and %lld elements apart, rows of %lld", who, (long long)x_stride, (long long)y_stride,
              (long long)H * D);
    return PT_ERR_INVALID_ARG;
  }
  if (T == 0 || H == 0) return PT_OK;
  if (!X || !Y || !positions || !inv_freq) {
    set_error("%s: a pointer is NULL", who);
    return PT_ERR_INVALID_ARG;
  }
  const uintptr_t x = reinterpret_cast<uintptr_t>(X), y = reinterpret_cast<uintptr_t>(Y);
  const uintptr_t all = x | y | (uintptr_t)(x_stride * es) | (uintptr_t)(y_stride * es) | (uintptr_t)(D * es);
  if (all & (uintptr_t)(es - 1)) {
    set_error("%s: a pointer is not aligned to its elements", who);
    return PT_ERR_INVALID_ARG;
  }
  const bool same = x == y && x_stride == y_stride;
  const uintptr_t nx = ((uintptr_t)(T - 1) * x_stride + (uintptr_t)H * D) * es,
                  ny = ((uintptr_t)(T - 1) * y_stride + (uintptr_t)H * D) * es;
  if (!same && x < y + ny && y < x + nx) {
    // (slices of one buffer whose rows do not meet: equal strides, the rows side by side)
    const long long gap = (long long)(x > y ? x - y : y - x), row = (long long)H * D * es;
    if (x_stride != y_stride || gap % (x_stride * es) < row || x_stride * es - gap % (x_stride * es) < row) {
      set_error("%s: Y overlaps X without being X", who);
      return PT_ERR_INVALID_ARG;
    }
  }
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess) {
    set_error("%s: no CUDA device", who);
    return PT_ERR_CUDA;
  }
  // the widest vectors that the columns, strides and addresses allow
  int unit = 16;
  while (unit > es && ((all & (uintptr_t)(unit - 1)) || half * es % unit)) unit >>= 1;
  if (unit < 8) unit = es;
  a.X = static_cast<const char*>(X), a.Y = static_cast<char*>(Y);
  a.x_stride = x_stride * es, a.y_stride = y_stride * es;
  a.pos = reinterpret_cast<const long long*>(positions);
  a.inv_freq = inv_freq;
  a.T = T, a.H = H, a.D = D, a.half = half;
  a.inverse = inverse != 0;
  a.copy = !same && rot_dim < D;
  // Eight heads a thread or a few more and 256 threads a CTA; fewer heads where that leaves SMs idle (40 heads: one token
  // 2.1 us, 3.3 with eight; 64 tokens 2.2 and 4.3; 2048 tokens 6.9 with eight, 9.0 with one).
  const int per = half / (unit / es), sms = num_sms(dev);
  int each = 8;
  while (each > 1 && (long long)T * ((H + each - 1) / each) * per < 512ll * sms) each /= 2;
  const int most = std::max(1, std::min((H + each - 1) / each, 256 / per));
  a.lanes = 1;  // (a power of two, so that warps are full: 40 heads in four lanes 89 us, in five 93)
  while (2 * a.lanes <= most) a.lanes *= 2;
  // (a CTA's elements are counted in 32 bits; H * D is at most INT_MAX / 4)
  a.tokens = std::max(1, std::min(256 / (per * a.lanes), INT_MAX / 4 / (H * D)));
  const int threads = per * a.lanes * a.tokens;
  const dim3 grid((unsigned)(((long long)T + a.tokens - 1) / a.tokens));
  const size_t smem = (size_t)a.tokens * half * 8;
  cudaError_t e;
  {
    ProfScope ps(stream, "rotary");
    if (dtype == PT_BF16)
      e = interleaved ? launch<__nv_bfloat16, true>(a, unit, grid, threads, smem, stream)
                      : launch<__nv_bfloat16, false>(a, unit, grid, threads, smem, stream);
    else
      e = interleaved ? launch<float, true>(a, unit, grid, threads, smem, stream) : launch<float, false>(a, unit, grid, threads, smem, stream);
    count_launch();
  }
  if (e == cudaSuccess) e = cudaGetLastError();
  if (e != cudaSuccess) {
    set_error("%s: launch failed: %s", who, cudaGetErrorString(e));
    return PT_ERR_CUDA;
  }
  return PT_OK;
}
