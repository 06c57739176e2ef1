// resnorm_impl.cuh -- kernels of the gated residual norm.
//
//   out = alpha h + w z r,   r = rms_b(z),   w_c = scale_c a(q_c) post_c
//   y   = pre out p,         p = rms_b(out)
//
// and, with n_b elements in block b and d = gout + pre p gy - out p^3 / n_b sum_b(gy pre out),
//
//   gh = alpha d,   gz = r (w d - z r / n_b sum_b(w d z r)),   P_c = sum_m d z r,
//   gq_c = scale post a'(q) P_c,   A_c = sum_n a(q) P_c,   gpost = scale A,   gscale = post A,
//   gpre_c = sum_n p sum_m gy out.
//
// Powers of p and r are never formed alone: d = gout + p (pre gy - out (p (p S / n_b))), so that a block of zeros
// under a small eps, or a block of tiny elements, gives gradients as large as they are and no inf * 0.
//
// A thread owns whole channels of a row (u, u + lanes, ... of every block), so the sums over m
// (gates, parameter gradients) stay inside a thread and the only exchange is the block sum of an
// rms.  A channel's 2l+1 components lie side by side, so reading channel by channel would
// touch 2l+1 times the cache lines of a row; rows therefore pass through shared memory (odd
// distances between the channels of neighbouring lanes: no bank conflicts), where each value is read
// once from memory and once written.  A group of warps owns a ring of tiles: while it computes one,
// the copies of the next are in flight.  Results go over the operands that they replace and
// leave in wide runs.
//
// Rows are dealt to groups by index and a channel's partial sums belong to one thread of a
// group, so every sum has a fixed order.
#pragma once

#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include "chain.cuh"
#include "resnorm.h"

namespace cgtp {
namespace {

template <typename A, typename T>
__device__ __forceinline__ A rn_get(const T* p) {
  if constexpr (sizeof(T) == 2) return static_cast<A>(__bfloat162float(*p));
  else return static_cast<A>(*p);
}
// stores v rounded once and returns what is stored
__device__ __forceinline__ float rn_put(float* p, float v) { return *p = v; }
__device__ __forceinline__ double rn_put(double* p, double v) { return *p = v; }
__device__ __forceinline__ float rn_put(__nv_bfloat16* p, float v) {
  *p = __float2bfloat16_rn(v);
  return __bfloat162float(*p);
}

__device__ __forceinline__ float rn_rsqrt(float v) { return rsqrtf(v); }
__device__ __forceinline__ double rn_rsqrt(double v) { return rsqrt(v); }
// 1 / (1 + e^-q) to a few units in the last place for every q; 0 below -87.3, where the value is no normal number.
// e^-q = 2^(hi + lo) with hi the rounded product -q log2(e) and lo what its rounding and the constant's left out (the
// fast exponential leaves lo out, which costs 37 units at q = -30), 2^lo = 1 + lo ln 2.  For a q without such a
// split (infinite, or so far out that 2^hi is 0 or infinite) the correction only has to be positive.  expf in its
// place: 5,000 x 128x0e+128x1o+128x2e backward 46.1 us against 44.7 us, 200,000 x 32x0e+32x1o+32x2e+32x3o 458 against 442.
__device__ __forceinline__ float rn_sigmoid(float q) {
  const float hi = -1.44269502f * q;
  const float lo = fmaf(-1.92596303e-8f, q, fmaf(-1.44269502f, q, -hi));
  const float c = fminf(fabsf(fmaf(lo, 0.693147182f, 1.0f)), 2.0f);
  float e, s;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(e) : "f"(hi));
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(s) : "f"(fmaf(e, c, 1.0f)));
  return s;
}
__device__ __forceinline__ double rn_sigmoid(double q) { return 1.0 / (1.0 + exp(-q)); }

// a(q) and, when asked for, a'(q)
template <typename A>
__device__ __forceinline__ A rn_gate(int act, A q, A* derivative) {
  if (act == CGTP_ACT_IDENTITY) {
    if (derivative) *derivative = A(1);
    return q;
  }
  const A s = rn_sigmoid(q);
  const bool silu = act == CGTP_ACT_SILU;
  if (derivative) *derivative = silu ? s + s * (q * (A(1) - s)) : s * (A(1) - s);
  return silu ? q * s : s;
}

// Per-channel factors: post * scale and pre, in shared memory or read in place.
template <bool STAGED, typename A>
struct RnFactors {
  const A *post, *scale, *pre;   // STAGED: post holds the product, and no pointer is null
  __device__ __forceinline__ A base_at(int c) const {
    if constexpr (STAGED) return post[c];
    return (post ? post[c] : A(1)) * (scale ? scale[c] : A(1));
  }
  __device__ __forceinline__ A pre_at(int c) const {
    if constexpr (STAGED) return pre[c];
    return pre ? pre[c] : A(1);
  }
};

// The threads of a row.  Groups of several warps (ONE = false) exchange sums through `scratch`
// (two banks in turn, so that one barrier separates the uses of a bank).  WHOLE: one warp, 32 lanes a row.
template <typename A, bool ONE, bool WHOLE>
struct RnTeam {
  int t, lanes, warps, barrier;   // place in the row, threads of a row, warps of the group, its named barrier
  A* scratch;
  int bank;

  // distance between a thread's channels
  __device__ __forceinline__ int stride() const { return WHOLE ? 32 : lanes; }
  __device__ __forceinline__ void sync() const {
    if constexpr (ONE) __syncwarp();
    else asm volatile("bar.sync %0, %1;" ::"r"(barrier), "r"(warps * 32) : "memory");
  }
  // Sums of K values over the row's threads; collective over the group.  The branch stays where every row has
  // 32 lanes, too: without it the code around the sums was scheduled worse (200,000 x 576 rows: forward 315 us
  // against 266 us, backward 510 us against 484 us).
  template <int K>
  __device__ __forceinline__ void sum(A (&v)[K]) {
    if (!ONE || lanes == 32) {
#pragma unroll
      for (int o = 16; o; o >>= 1)
#pragma unroll
        for (int i = 0; i < K; ++i) v[i] += __shfl_xor_sync(0xffffffffu, v[i], o);
    } else {
      for (int o = lanes >> 1; o; o >>= 1)
#pragma unroll
        for (int i = 0; i < K; ++i) v[i] += __shfl_xor_sync(0xffffffffu, v[i], o);
    }
    if constexpr (ONE) {
      __syncwarp();
      return;
    }
    A* s = scratch + bank * 4 * kRnWarps;
    bank ^= 1;
    if ((threadIdx.x & 31) == 0)
#pragma unroll
      for (int i = 0; i < K; ++i) s[i * kRnWarps + (t >> 5)] = v[i];
    sync();
#pragma unroll
    for (int i = 0; i < K; ++i) {
      v[i] = s[i * kRnWarps];
      for (int w = 1; w < warps; ++w) v[i] += s[i * kRnWarps + w];
    }
  }
};

template <typename A>
__device__ __forceinline__ A rn_eps(const RnArgs& a) {
  if constexpr (sizeof(A) == 8) return a.eps;
  return a.eps_f;
}
template <typename A>
__device__ __forceinline__ A rn_alpha(const RnArgs& a) {
  if constexpr (sizeof(A) == 8) return a.alpha;
  return a.alpha_f;
}
template <typename A>
__device__ __forceinline__ A rn_inv_n(const RnBlock& b) {
  if constexpr (sizeof(A) == 8) return b.inv_n;
  return b.inv_n_f;
}

// Pointers to one row, in shared memory or in global memory.
template <typename S, typename I, typename O>
struct RnForwardRow {
  const S* h;
  const I *z, *q;
  S* out;
  O* y;
};
template <typename S, typename I, typename O, typename A>
struct RnBackwardRow {
  const S *g, *x;
  const I *gy, *z, *q;
  S* gh;
  O *gz, *gq;
  A* part;
  bool live;   // false: a place without a row (its results stay in its place of the tile)
};

// S: residual stream, I: what comes from a product, O: what goes to one, A: arithmetic and parameters.
// Results may lie over operands: an element is written by the thread that read it, after its last read.
//
// A block's values stay in registers where a thread's share, K channels of D components, is small
// (every operand is then read once from shared memory); larger shares are read again for each pass.
template <int D, int K, bool FULL, typename S, typename I, typename O, typename A, bool STAGED, bool ONE, bool WHOLE>
__device__ __forceinline__ void rn_block_held(const RnArgs& a, const RnBlock b, const RnForwardRow<S, I, O>& row,
                                                const RnFactors<STAGED, A>& f, RnTeam<A, ONE, WHOLE>& team) {
  const A inv_n = rn_inv_n<A>(b), eps = rn_eps<A>(a);
  const bool has_h = FULL || a.t[kRnH].ptr, has_z = FULL || a.t[kRnZ].ptr, gated = FULL || a.t[kRnQ].ptr;
  const bool pre_norm = FULL || a.pre_norm, post_norm = FULL || a.post_norm;
  A v[K][D], w[K];
  A s[1] = {A(0)};
  const I* z = row.z + b.off;
  const S* h = row.h + b.off;
  if (has_z) {
#pragma unroll
    for (int k = 0; k < K; ++k) {
      const int u = team.t + k * team.stride();
      w[k] = A(0);
#pragma unroll
      for (int m = 0; m < D; ++m) v[k][m] = A(0);
      if (FULL || u < b.mul) {
        w[k] = f.base_at(b.coff + u);
        if (gated) w[k] *= rn_gate<A>(a.act, rn_get<A>(row.q + b.coff + u), nullptr);
#pragma unroll
        for (int m = 0; m < D; ++m) {
          v[k][m] = rn_get<A>(z + u * D + m);
          s[0] += v[k][m] * v[k][m];
        }
      }
    }
    if (post_norm) {
      team.sum(s);
      const A r = rn_rsqrt(s[0] * inv_n + eps);
#pragma unroll
      for (int k = 0; k < K; ++k) w[k] *= r;
    }
    s[0] = A(0);
    S* out = row.out + b.off;
    const A alpha = rn_alpha<A>(a);
#pragma unroll
    for (int k = 0; k < K; ++k) {
      const int u = team.t + k * team.stride();
      if (FULL || u < b.mul) {
        if (has_h) {
#pragma unroll
          for (int m = 0; m < D; ++m) v[k][m] = w[k] * v[k][m] + alpha * rn_get<A>(h + u * D + m);
        } else {
#pragma unroll
          for (int m = 0; m < D; ++m) v[k][m] *= w[k];
        }
#pragma unroll
        for (int m = 0; m < D; ++m) {
          v[k][m] = rn_put(out + u * D + m, v[k][m]);
          s[0] += v[k][m] * v[k][m];
        }
      }
    }
  } else {
#pragma unroll
    for (int k = 0; k < K; ++k) {
      const int u = team.t + k * team.stride();
#pragma unroll
      for (int m = 0; m < D; ++m) v[k][m] = A(0);
      if (FULL || u < b.mul) {
#pragma unroll
        for (int m = 0; m < D; ++m) {
          v[k][m] = rn_get<A>(h + u * D + m);
          s[0] += v[k][m] * v[k][m];
        }
      }
    }
  }
  if (!pre_norm) return;
  team.sum(s);
  const A p = rn_rsqrt(s[0] * inv_n + eps);
  O* y = row.y + b.off;
#pragma unroll
  for (int k = 0; k < K; ++k) {
    const int u = team.t + k * team.stride();
    if (FULL || u < b.mul) {
      const A g = p * f.pre_at(b.coff + u);
#pragma unroll
      for (int m = 0; m < D; ++m) rn_put(y + u * D + m, g * v[k][m]);
    }
  }
}

template <int D, typename S, typename I, typename O, typename A, bool STAGED, bool ONE, bool WHOLE>
__device__ __forceinline__ void rn_block_any(const RnArgs& a, const RnBlock b, const RnForwardRow<S, I, O>& row,
                                                 const RnFactors<STAGED, A>& f, RnTeam<A, ONE, WHOLE>& team) {
  const A inv_n = rn_inv_n<A>(b), eps = rn_eps<A>(a), alpha = rn_alpha<A>(a);
  const bool has_h = a.t[kRnH].ptr, has_z = a.t[kRnZ].ptr, gated = a.t[kRnQ].ptr;
  const S* h = row.h + b.off;
  const I *z = row.z + b.off, *q = row.q + b.coff;
  S* out = row.out + b.off;
  O* y = row.y + b.off;
  A r = A(1);
  if (has_z && a.post_norm) {
    A ss[1] = {A(0)};
    for (int u = team.t; u < b.mul; u += team.lanes)
#pragma unroll
      for (int m = 0; m < D; ++m) {
        const A v = rn_get<A>(z + u * D + m);
        ss[0] += v * v;
      }
    team.sum(ss);
    r = rn_rsqrt(ss[0] * inv_n + eps);
  }
  A ss[1] = {A(0)};
  if (has_z) {
    for (int u = team.t; u < b.mul; u += team.lanes) {
      A w = r * f.base_at(b.coff + u);
      if (gated) w *= rn_gate<A>(a.act, rn_get<A>(q + u), nullptr);
#pragma unroll
      for (int m = 0; m < D; ++m) {
        A v = w * rn_get<A>(z + u * D + m);
        if (has_h) v += alpha * rn_get<A>(h + u * D + m);
        v = rn_put(out + u * D + m, v);
        ss[0] += v * v;
      }
    }
  } else {
    for (int u = team.t; u < b.mul; u += team.lanes)
#pragma unroll
      for (int m = 0; m < D; ++m) {
        const A v = rn_get<A>(h + u * D + m);
        ss[0] += v * v;
      }
  }
  if (!a.pre_norm) return;
  team.sum(ss);
  const A p = rn_rsqrt(ss[0] * inv_n + eps);
  const S* x = has_z ? out : h;
  for (int u = team.t; u < b.mul; u += team.lanes) {
    const A w = p * f.pre_at(b.coff + u);
#pragma unroll
    for (int m = 0; m < D; ++m) rn_put(y + u * D + m, w * rn_get<A>(x + u * D + m));
  }
}

template <int D, int K, bool FULL, typename S, typename I, typename O, typename A, bool STAGED, bool ONE, bool WHOLE>
__device__ __forceinline__ void rn_block_held(const RnArgs& a, const RnBlock b,
                                                 const RnBackwardRow<S, I, O, A>& row, const RnFactors<STAGED, A>& f,
                                                 RnTeam<A, ONE, WHOLE>& team) {
  const A inv_n = rn_inv_n<A>(b), eps = rn_eps<A>(a), alpha = rn_alpha<A>(a);
  const bool has_g = FULL || a.t[kRnGout].ptr, has_gh = FULL || a.t[kRnGh].ptr, has_z = FULL || a.t[kRnBz].ptr,
             gated = FULL || a.t[kRnBq].ptr, pre_norm = FULL || a.pre_norm, post_norm = FULL || a.post_norm;
  const S *g = row.g + b.off, *x = row.x + b.off;
  const I *gy = row.gy + b.off, *z = row.z + b.off;
  A d[K][D], xv[K][D], zv[K][D], xy[K], pre[K];   // d starts as gy
  A s[3] = {A(0), A(0), A(0)};                    // sums of x^2, of gy pre x, of z^2
#pragma unroll
  for (int k = 0; k < K; ++k) {
    const int u = team.t + k * team.stride();
    xy[k] = pre[k] = A(0);
#pragma unroll
    for (int m = 0; m < D; ++m) d[k][m] = xv[k][m] = zv[k][m] = A(0);
    if (FULL || u < b.mul) {
      if (pre_norm) {
        pre[k] = f.pre_at(b.coff + u);
#pragma unroll
        for (int m = 0; m < D; ++m) {
          xv[k][m] = rn_get<A>(x + u * D + m);
          d[k][m] = rn_get<A>(gy + u * D + m);
          s[0] += xv[k][m] * xv[k][m];
          xy[k] += xv[k][m] * d[k][m];
        }
        s[1] += pre[k] * xy[k];
      }
      if (has_z) {
#pragma unroll
        for (int m = 0; m < D; ++m) {
          zv[k][m] = rn_get<A>(z + u * D + m);
          s[2] += zv[k][m] * zv[k][m];
        }
      }
    }
  }
  A p = A(0), kx = A(0), r = A(1);
  team.sum(s);
  if (pre_norm) {
    p = rn_rsqrt(s[0] * inv_n + eps);
    kx = p * (p * (s[1] * inv_n));   // times p below
  }
  if (post_norm) r = rn_rsqrt(s[2] * inv_n + eps);
  A along[1] = {A(0)}, w[K];   // sum over the block of w d z r
#pragma unroll
  for (int k = 0; k < K; ++k) {
    const int u = team.t + k * team.stride(), c = b.coff + u;
    w[k] = A(0);
    if (FULL || u < b.mul) {
      if (has_g) {
#pragma unroll
        for (int m = 0; m < D; ++m) d[k][m] = rn_get<A>(g + u * D + m) + p * (pre[k] * d[k][m] - kx * xv[k][m]);
      } else {
#pragma unroll
        for (int m = 0; m < D; ++m) d[k][m] = p * (pre[k] * d[k][m] - kx * xv[k][m]);
      }
      if (row.live && pre_norm) row.part[a.chan + c] += p * xy[k];
      if (has_gh) {
#pragma unroll
        for (int m = 0; m < D; ++m) rn_put(row.gh + b.off + u * D + m, alpha * d[k][m]);
      }
      if (has_z) {
        A P = A(0);
#pragma unroll
        for (int m = 0; m < D; ++m) P += d[k][m] * zv[k][m];
        P *= r;
        const A base = f.base_at(c);
        A act = A(1), der = A(0);
        if (gated) {
          act = rn_gate<A>(a.act, rn_get<A>(row.q + c), &der);
          rn_put(row.gq + c, base * der * P);
        }
        w[k] = base * act;
        along[0] += w[k] * P;
        if (row.live) row.part[c] += act * P;
      }
    }
  }
  if (!has_z) return;
  A kz = A(0);
  if (post_norm) {
    team.sum(along);
    kz = r * (r * (along[0] * inv_n));
  }
#pragma unroll
  for (int k = 0; k < K; ++k) {
    const int u = team.t + k * team.stride();
    if (FULL || u < b.mul) {
      const A wr = w[k] * r;
#pragma unroll
      for (int m = 0; m < D; ++m) rn_put(row.gz + b.off + u * D + m, wr * d[k][m] - kz * zv[k][m]);
    }
  }
}

template <int D, typename S, typename I, typename O, typename A, bool STAGED, bool ONE, bool WHOLE>
__device__ __forceinline__ void rn_block_any(const RnArgs& a, const RnBlock b,
                                                  const RnBackwardRow<S, I, O, A>& row, const RnFactors<STAGED, A>& f,
                                                  RnTeam<A, ONE, WHOLE>& team) {
  const A inv_n = rn_inv_n<A>(b), eps = rn_eps<A>(a), alpha = rn_alpha<A>(a);
  const bool has_g = a.t[kRnGout].ptr, has_gh = a.t[kRnGh].ptr, has_z = a.t[kRnBz].ptr, gated = a.t[kRnBq].ptr;
  const S *g = row.g + b.off, *x = row.x + b.off;
  const I *gy = row.gy + b.off, *z = row.z + b.off, *q = row.q + b.coff;
  S* gh = row.gh + b.off;
  O *gz = row.gz + b.off, *gq = row.gq + b.coff;
  A p = A(0), k = A(0), r = A(1);
  if (a.pre_norm || (has_z && a.post_norm)) {
    A s[3] = {A(0), A(0), A(0)};   // sums of x^2, of gy pre x, of z^2
    for (int u = team.t; u < b.mul; u += team.lanes) {
      if (a.pre_norm) {
        A xy = A(0);
#pragma unroll
        for (int m = 0; m < D; ++m) {
          const A v = rn_get<A>(x + u * D + m);
          s[0] += v * v;
          xy += v * rn_get<A>(gy + u * D + m);
        }
        s[1] += f.pre_at(b.coff + u) * xy;
      }
      if (has_z && a.post_norm)
#pragma unroll
        for (int m = 0; m < D; ++m) {
          const A v = rn_get<A>(z + u * D + m);
          s[2] += v * v;
        }
    }
    team.sum(s);
    if (a.pre_norm) {
      p = rn_rsqrt(s[0] * inv_n + eps);
      k = p * (p * (s[1] * inv_n));   // times p below
    }
    if (has_z && a.post_norm) r = rn_rsqrt(s[2] * inv_n + eps);
  }
  const bool again = has_z && a.post_norm;   // a third pass writes gh and gz
  A along[1] = {A(0)};                       // sum over the block of w d z r
  for (int u = team.t; u < b.mul; u += team.lanes) {
    const int c = b.coff + u;
    const A pre = a.pre_norm ? f.pre_at(c) : A(0);
    A P = A(0), xy = A(0), d[D];
#pragma unroll
    for (int m = 0; m < D; ++m) {
      A v = has_g ? rn_get<A>(g + u * D + m) : A(0);
      if (a.pre_norm) {
        const A e = rn_get<A>(gy + u * D + m), o = rn_get<A>(x + u * D + m);
        v += p * (pre * e - k * o);
        xy += e * o;
      }
      d[m] = v;
      if (has_z) P += v * rn_get<A>(z + u * D + m);
    }
    if (row.live && a.pre_norm) row.part[a.chan + c] += p * xy;
    A w = A(0);
    if (has_z) {
      P *= r;
      const A base = f.base_at(c);
      A act = A(1), der = A(0);
      if (gated) act = rn_gate<A>(a.act, rn_get<A>(q + u), &der);
      w = base * act;
      along[0] += w * P;
      if (row.live) row.part[c] += act * P;
      if (gated) rn_put(gq + u, base * der * P);
    }
    if (!again)
#pragma unroll
      for (int m = 0; m < D; ++m) {
        if (has_gh) rn_put(gh + u * D + m, alpha * d[m]);
        if (has_z) rn_put(gz + u * D + m, w * d[m]);
      }
  }
  if (!again) return;
  team.sum(along);
  const A kz = r * (r * (along[0] * inv_n));
  for (int u = team.t; u < b.mul; u += team.lanes) {
    const int c = b.coff + u;
    const A pre = a.pre_norm ? f.pre_at(c) : A(0);
    A w = r * f.base_at(c);
    if (gated) w *= rn_gate<A>(a.act, rn_get<A>(q + u), nullptr);
#pragma unroll
    for (int m = 0; m < D; ++m) {
      A v = has_g ? rn_get<A>(g + u * D + m) : A(0);
      if (a.pre_norm) v += p * (pre * rn_get<A>(gy + u * D + m) - k * rn_get<A>(x + u * D + m));
      const A e = w * v - kz * rn_get<A>(z + u * D + m);
      if (has_gh) rn_put(gh + u * D + m, alpha * v);
      rn_put(gz + u * D + m, e);
    }
  }
}

// A block by its number of components and the thread's share (rn_share).
#define CGTP_RN_CASE(D, K) \
  case rn_code(D, K): HELD(D, K); break;
#define CGTP_RN_HELD                                                                                          \
  CGTP_RN_CASE(1, 1) CGTP_RN_CASE(1, 2) CGTP_RN_CASE(1, 4) CGTP_RN_CASE(1, 8) CGTP_RN_CASE(3, 1)             \
  CGTP_RN_CASE(3, 2) CGTP_RN_CASE(3, 4) CGTP_RN_CASE(5, 1) CGTP_RN_CASE(5, 2) CGTP_RN_CASE(5, 4)             \
  CGTP_RN_CASE(7, 1) CGTP_RN_CASE(7, 2) CGTP_RN_CASE(9, 1) CGTP_RN_CASE(9, 2) CGTP_RN_CASE(11, 1)            \
  CGTP_RN_CASE(13, 1) CGTP_RN_CASE(15, 1)
#define CGTP_RN_ANY                                                                                           \
  switch (b.D) {                                                                                              \
    case 1: ANY(1); break;                                                                                    \
    case 3: ANY(3); break;                                                                                    \
    case 5: ANY(5); break;                                                                                    \
    case 7: ANY(7); break;                                                                                    \
    case 9: ANY(9); break;                                                                                    \
    case 11: ANY(11); break;                                                                                  \
    case 13: ANY(13); break;                                                                                  \
    default: ANY(15); break;                                                                                  \
  }

template <int KIND, typename Row, typename A, bool STAGED, bool ONE, bool WHOLE>
__device__ __forceinline__ void rn_row(const RnArgs& a, const RnBlock* table, const Row& row, const RnFactors<STAGED, A>& f,
                                       RnTeam<A, ONE, WHOLE>& team) {
  for (int i = 0; i < a.n_blocks; ++i) {
#define HELD(D, K) rn_block_held<D, K, KIND != kRnOne && KIND != kRnMany>(a, b, row, f, team)
    if constexpr (KIND == kRnOne || KIND == kRnMany) {
      // many blocks come from the table in shared memory, others from the kernel's parameters
      RnBlock b;
      if (table) b = table[i];
      else b = a.few[i];
      switch (b.code) { CGTP_RN_HELD }
    } else if constexpr (STAGED) {
      const RnBlock& b = a.few[i];
      switch (b.code) { CGTP_RN_HELD }
#undef HELD
    } else {
      const RnBlock b = table[i];
#define ANY(D) rn_block_any<D>(a, b, row, f, team)
      CGTP_RN_ANY
#undef ANY
    }
  }
}

// row n of tensor i in memory
template <typename T>
__device__ __forceinline__ T* rn_at(const RnArgs& a, int i, int64_t n) {
  return reinterpret_cast<T*>(a.t[i].ptr) + n * a.t[i].ld;
}
// row j of tensor i in a stage (the stage's first byte where the tensor has no region)
template <typename T>
__device__ __forceinline__ T* rn_in(const RnArgs& a, int i, char* stage, int j) {
  return reinterpret_cast<T*>(stage + max(a.t[i].at, 0) + j * a.t[i].pitch);
}

// ---------------------------------------------------------------------------
// Rows staged in shared memory
// ---------------------------------------------------------------------------

// Column i of the sums over rows: gpost = scale A, gscale = post A, gpre.
template <typename A>
__device__ __forceinline__ void rn_put_sums(A v, int i, int chan, const void* post, const void* scale, void* gpost, void* gscale,
                                            void* gpre) {
  if (i < chan) {
    if (gpost) static_cast<A*>(gpost)[i] = scale ? v * static_cast<const A*>(scale)[i] : v;
    if (gscale) static_cast<A*>(gscale)[i] = post ? v * static_cast<const A*>(post)[i] : v;
  } else if (gpre) {
    static_cast<A*>(gpre)[i - chan] = v;
  }
}

// Column i of the partial sums, added in CTA order within each of `segments` threads and then in their order.
template <typename A>
__device__ __forceinline__ void rn_columns(const A* part, int ctas, int chan, const void* post, const void* scale, void* gpost,
                                           void* gscale, void* gpre, A (*sums)[33], int i, int seg, int segments) {
  A v = A(0);
  if (i < 2 * chan)
    for (int k = seg; k < ctas; k += segments) v += __ldcg(part + (int64_t)k * 2 * chan + i);
  const int lane = threadIdx.x & 31;
  sums[seg][lane] = v;
  __syncthreads();
  if (seg == 0 && i < 2 * chan) {
    for (int k = 1; k < segments; ++k) v += sums[k][lane];
    rn_put_sums<A>(v, i, chan, post, scale, gpost, gscale, gpre);
  }
  __syncthreads();
}

// 152 CTAs x 384 sums: 7 us, the latency of 19 loads in a row and a launch.
template <typename A>
__global__ void __launch_bounds__(256) rn_reduce_kernel(const void* part, int ctas, int chan, const void* post, const void* scale,
                                                        void* gpost, void* gscale, void* gpre) {
  __shared__ A sums[8][33];
  chain_enter();
  rn_columns<A>(static_cast<const A*>(part), ctas, chan, post, scale, gpost, gscale, gpre, sums,
                blockIdx.x * 32 + (threadIdx.x & 31), threadIdx.x >> 5, 8);
}

// `bytes` bytes from memory to shared memory in asynchronous copies of V bytes (the rest at once)
template <int V>
__device__ __forceinline__ void rn_copy_in(char* dst, const char* src, int bytes, int t, int threads) {
  uint32_t d = static_cast<uint32_t>(__cvta_generic_to_shared(dst)) + t * V;
  const char* s = src + t * V;
  int left = bytes - t * V;
  for (; left >= V; left -= 4 * threads * V, d += 4 * threads * V, s += 4 * threads * V) {
#pragma unroll
    for (int j = 0; j < 4; ++j)
      if (left - j * threads * V >= V) {
        if constexpr (V == 16) asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(d + j * threads * V), "l"(s + j * threads * V) : "memory");
        else asm volatile("cp.async.ca.shared.global [%0], [%1], %2;" ::"r"(d + j * threads * V), "l"(s + j * threads * V), "n"(V) : "memory");
      }
  }
  if (bytes % V)
    for (int i = bytes / V * V + 2 * t; i < bytes; i += 2 * threads)
      *reinterpret_cast<uint16_t*>(dst + i) = *reinterpret_cast<const uint16_t*>(src + i);
}
template <typename T>
__device__ __forceinline__ void rn_copy_out(char* dst, const char* src, int bytes, int t, int threads) {
  constexpr int V = sizeof(T);
  const char* s = src + t * V;
  char* d = dst + t * V;
  int left = bytes - t * V;
  for (; left >= V; left -= 4 * threads * V, d += 4 * threads * V, s += 4 * threads * V) {
    T v[4];
#pragma unroll
    for (int j = 0; j < 4; ++j)
      if (left - j * threads * V >= V) v[j] = *reinterpret_cast<const T*>(s + j * threads * V);
#pragma unroll
    for (int j = 0; j < 4; ++j)
      if (left - j * threads * V >= V) *reinterpret_cast<T*>(d + j * threads * V) = v[j];
  }
  if (V > 2 && bytes % V)
    for (int i = bytes / V * V + 2 * t; i < bytes; i += 2 * threads)
      *reinterpret_cast<uint16_t*>(dst + i) = *reinterpret_cast<const uint16_t*>(src + i);
}

// Rows [n0, n0 + count) of tensor r between memory and its region of the stage.
template <bool IN>
__device__ __forceinline__ void rn_move(const RnRows& r, char* stage, int n0, int count, int t, int threads) {
  char* mem = r.ptr + n0 * r.ld_bytes;
  char* region = stage + r.at;
  const int runs = r.linear ? 1 : count, bytes = r.width * r.es * (r.linear ? count : 1);
  for (int j = 0; j < runs; ++j, mem += r.ld_bytes, region += r.pitch) {
    if constexpr (IN) {
      if (r.vec == 16) rn_copy_in<16>(region, mem, bytes, t, threads);
      else if (r.vec == 8) rn_copy_in<8>(region, mem, bytes, t, threads);
      else if (r.vec == 4) rn_copy_in<4>(region, mem, bytes, t, threads);
      else for (int i = 2 * t; i < bytes; i += 2 * threads)
        *reinterpret_cast<uint16_t*>(region + i) = *reinterpret_cast<const uint16_t*>(mem + i);
    } else {
      if (r.vec == 16) rn_copy_out<uint4>(mem, region, bytes, t, threads);
      else if (r.vec == 8) rn_copy_out<uint2>(mem, region, bytes, t, threads);
      else if (r.vec == 4) rn_copy_out<uint32_t>(mem, region, bytes, t, threads);
      else rn_copy_out<uint16_t>(mem, region, bytes, t, threads);
    }
  }
}

// The same for NT tensors at once whose tiles are runs of `bytes` bytes, a multiple of 16.
template <int NT>
__device__ __forceinline__ void rn_runs_in(const RnRows* const (&r)[NT], char* stage, int n0, int bytes, int t, int threads) {
  const char* src[NT];
  uint32_t dst[NT];
#pragma unroll
  for (int i = 0; i < NT; ++i) {
    src[i] = r[i]->ptr + n0 * r[i]->ld_bytes + t * 16;
    dst[i] = static_cast<uint32_t>(__cvta_generic_to_shared(stage)) + r[i]->at + t * 16;
  }
  const int run = threads * 16;
  int left = bytes;
  for (; left >= 4 * run; left -= 4 * run) {
#pragma unroll
    for (int j = 0; j < 4; ++j)
#pragma unroll
      for (int i = 0; i < NT; ++i)
        asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(dst[i] + j * run), "l"(src[i] + j * run) : "memory");
#pragma unroll
    for (int i = 0; i < NT; ++i) src[i] += 4 * run, dst[i] += 4 * run;
  }
  for (; left > t * 16; left -= run)
#pragma unroll
    for (int i = 0; i < NT; ++i) {
      asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(dst[i]), "l"(src[i]) : "memory");
      src[i] += run, dst[i] += run;
    }
}
template <int NT>
__device__ __forceinline__ void rn_runs_out(const RnRows* const (&r)[NT], const char* stage, int n0, int bytes, int t, int threads) {
  char* dst[NT];
  const char* src[NT];
#pragma unroll
  for (int i = 0; i < NT; ++i) {
    dst[i] = r[i]->ptr + n0 * r[i]->ld_bytes + t * 16;
    src[i] = stage + r[i]->at + t * 16;
  }
  const int run = threads * 16;
  int left = bytes;
  for (; left >= 4 * run; left -= 4 * run) {
#pragma unroll
    for (int i = 0; i < NT; ++i) {
      uint4 v[4];
#pragma unroll
      for (int j = 0; j < 4; ++j) v[j] = *reinterpret_cast<const uint4*>(src[i] + j * run);
#pragma unroll
      for (int j = 0; j < 4; ++j) *reinterpret_cast<uint4*>(dst[i] + j * run) = v[j];
      src[i] += 4 * run, dst[i] += 4 * run;
    }
  }
  for (; left > t * 16; left -= run)
#pragma unroll
    for (int i = 0; i < NT; ++i) {
      *reinterpret_cast<uint4*>(dst[i]) = *reinterpret_cast<const uint4*>(src[i]);
      src[i] += run, dst[i] += run;
    }
}

// Bound by HBM where blocks fill the warp: 200,000 rows of 64x0e+64x1o+64x2e forward with bfloat16 y 259 us (6.8 TB/s;
// a copy reaches 6.7), backward 482 to 506 us (6.1 to 6.4 TB/s; the cards differ); 60,000 x 128x0e+128x1o+128x2e backward 310 to
// 335 us (5.5 to 5.9 TB/s, nine warps fit).  Elsewhere by instructions: 400,000 x 33x0e+17x1o+5x2e 119 us (2.9 TB/s);
// and by bank conflicts of rows side by side: 2,000,000 x 8x0e+8x1o 300 us (3.8 TB/s).  One CTA an SM, 128 registers a thread:
// what a warp holds of a block is worth more than a second CTA.
template <bool BACKWARD, int KIND, typename S, typename I, typename O, typename A>
__global__ void __launch_bounds__(kRnWarps * 32, 1) rn_staged_kernel(const __grid_constant__ RnArgs a) {
  extern __shared__ __align__(16) char shared[];
  chain_enter();
  constexpr bool ONE = KIND >= kRnOne, FULL = KIND != kRnOne && KIND != kRnMany;
  constexpr bool WHOLE = KIND == kRnOneFull;
  const int warps = ONE ? 1 : a.warps, threads = warps * 32;
  const int g = threadIdx.x / threads, tg = threadIdx.x - g * threads;
  char* mine = shared + g * a.group_bytes;
  A* scratch = reinterpret_cast<A*>(mine + a.stages * a.stage_bytes);
  A* part = scratch + (ONE ? 0 : 8 * kRnWarps);           // [rows at a time][2][C]
  A* factors = reinterpret_cast<A*>(shared + a.groups * a.group_bytes);   // post * scale [C], pre [C]
  const RnFactors<false, A> read{static_cast<const A*>(a.post), static_cast<const A*>(a.scale), static_cast<const A*>(a.pre)};
  for (int i = threadIdx.x; i < a.chan; i += blockDim.x) {
    factors[i] = read.base_at(i);
    factors[a.chan + i] = read.pre_at(i);
  }
  const RnFactors<true, A> f{factors, nullptr, factors + a.chan};
  RnBlock* table = nullptr;
  if (!FULL && a.n_blocks > kRnInline) {
    table = reinterpret_cast<RnBlock*>(shared + a.table_at);
    for (int i = threadIdx.x; i < a.n_blocks; i += blockDim.x) {
      table[i] = a.blocks[i];
      table[i].code = rn_code(table[i].D, rn_share(table[i].D, table[i].mul, a.lanes));
    }
  }
  const int abreast = ONE ? 32 / a.lanes : 1, sub = ONE ? tg / a.lanes : 0;
  RnTeam<A, ONE, WHOLE> team{tg - sub * a.lanes, a.lanes, warps, 1 + g, scratch, 0};
  constexpr int first_out = kRnInputs[BACKWARD], last = BACKWARD ? kRnBackward : kRnForward;
  if constexpr (BACKWARD)
    for (int i = tg; i < abreast * 2 * a.chan; i += threads) part[i] = A(0);
  const int step = a.ctas * a.groups, N = static_cast<int>(a.N), tiles = static_cast<int>(a.tiles);
  int tile = g * a.ctas + blockIdx.x;
  const auto load = [&](int k, char* stage) {
    if (k < tiles) {
      const int n0 = k * a.rows, count = min(a.rows, N - n0);
      const int wide = count * a.dim * static_cast<int>(sizeof(S)), narrow = count * a.chan * static_cast<int>(sizeof(S));
      if (FULL && ((wide | narrow) & 15) == 0) {
        if constexpr (BACKWARD) {
          const RnRows* const many[4] = {&a.t[kRnGout], &a.t[kRnGy], &a.t[kRnX], &a.t[kRnBz]};
          rn_runs_in<4>(many, stage, n0, wide, tg, threads);
        } else {
          const RnRows* const many[2] = {&a.t[kRnH], &a.t[kRnZ]};
          rn_runs_in<2>(many, stage, n0, wide, tg, threads);
        }
        const RnRows* const q[1] = {&a.t[BACKWARD ? kRnBq : kRnQ]};
        rn_runs_in<1>(q, stage, n0, narrow, tg, threads);
      } else {
#pragma unroll
        for (int i = 0; i < first_out; ++i)
          if (FULL || a.t[i].ptr) rn_move<true>(a.t[i], stage, n0, count, tg, threads);
      }
    }
    asm volatile("cp.async.commit_group;" ::: "memory");
  };
  for (int s = 0; s < a.stages; ++s) load(tile + s * step, mine + s * a.stage_bytes);
  __syncthreads();
  for (char* stage = mine; tile < tiles; tile += step) {
    const int n0 = tile * a.rows, count = min(a.rows, N - n0);
    if (a.stages == 1) asm volatile("cp.async.wait_group 0;" ::: "memory");
    else asm volatile("cp.async.wait_group 1;" ::: "memory");
    team.sync();
    for (int j0 = 0; j0 < count; j0 += abreast) {
      const int j = j0 + sub;
      if constexpr (BACKWARD) {
        const RnBackwardRow<S, I, O, A> row{
            rn_in<S>(a, kRnGout, stage, j), rn_in<S>(a, kRnX, stage, j),  rn_in<I>(a, kRnGy, stage, j),
            rn_in<I>(a, kRnBz, stage, j),   rn_in<I>(a, kRnBq, stage, j), rn_in<S>(a, kRnGh, stage, j),
            rn_in<O>(a, kRnGz, stage, j),   rn_in<O>(a, kRnGq, stage, j), part + sub * 2 * a.chan, j < count};
        rn_row<KIND>(a, table, row, f, team);
      } else {
        const RnForwardRow<S, I, O> row{rn_in<S>(a, kRnH, stage, j), rn_in<I>(a, kRnZ, stage, j),
                                        rn_in<I>(a, kRnQ, stage, j), rn_in<S>(a, kRnOut, stage, j),
                                        rn_in<O>(a, kRnY, stage, j)};
        rn_row<KIND>(a, table, row, f, team);
      }
    }
    team.sync();
    const int wide = count * a.dim, narrow = count * a.chan;
    if (FULL && ((wide | narrow) * static_cast<int>(sizeof(O)) & 15) == 0) {
      const RnRows* const to[2] = {&a.t[first_out], &a.t[first_out + 1]};
      if constexpr (sizeof(S) == sizeof(O)) {
        rn_runs_out<2>(to, stage, n0, wide * static_cast<int>(sizeof(S)), tg, threads);
      } else {
        const RnRows* const one[1] = {to[0]};
        const RnRows* const two[1] = {to[1]};
        rn_runs_out<1>(one, stage, n0, wide * static_cast<int>(sizeof(S)), tg, threads);
        rn_runs_out<1>(two, stage, n0, wide * static_cast<int>(sizeof(O)), tg, threads);
      }
      if constexpr (BACKWARD) {
        const RnRows* const gq[1] = {&a.t[kRnGq]};
        rn_runs_out<1>(gq, stage, n0, narrow * static_cast<int>(sizeof(O)), tg, threads);
      }
    } else {
#pragma unroll
      for (int i = first_out; i < last; ++i)
        if (FULL || a.t[i].ptr) rn_move<false>(a.t[i], stage, n0, count, tg, threads);
    }
    team.sync();
    load(tile + a.stages * step, stage);
    stage = a.stages == 1 || stage != mine ? mine : mine + a.stage_bytes;
  }
  if constexpr (BACKWARD) {
    // the CTA's sums: groups in order, and in a group the rows that ran side by side
    __syncthreads();
    A* to = static_cast<A*>(a.part) + (int64_t)blockIdx.x * 2 * a.chan;
    for (int i = threadIdx.x; i < 2 * a.chan; i += blockDim.x) {
      A v = A(0);
      for (int k = 0; k < a.groups; ++k) {
        const A* p = part + (k - g) * (a.group_bytes / static_cast<int>(sizeof(A)));
        for (int j = 0; j < abreast; ++j) v += p[j * 2 * a.chan + i];
      }
      if (a.ctas == 1) rn_put_sums<A>(v, i, a.chan, a.post, a.scale, a.gpost, a.gscale, a.gpre);
      else to[i] = v;
    }
    if (a.ticket) {
      __shared__ bool last;
      __threadfence();
      __syncthreads();   // the groups' sums have been read, too
      if (threadIdx.x == 0) last = atomicAdd(a.ticket, 1u) == gridDim.x - 1;
      __syncthreads();
      if (!last) return;
      __threadfence();
      A(*sums)[33] = reinterpret_cast<A(*)[33]>(shared);
      const int segments = blockDim.x >> 5;
      for (int i = threadIdx.x & 31; i < (2 * a.chan + 31) / 32 * 32; i += 32)
        rn_columns<A>(static_cast<const A*>(a.part), a.ctas, a.chan, a.post, a.scale, a.gpost, a.gscale, a.gpre, sums, i,
                      threadIdx.x >> 5, segments);
      if (threadIdx.x == 0) *a.ticket = 0;
    }
  }
}

// ---------------------------------------------------------------------------
// Rows that do not fit in shared memory, or whose blocks a thread cannot hold: a CTA reads a row in place, and
// again for each pass (from L1 or L2).  20,000 rows of 8192x0e: forward 1.75 ms (1.9 TB/s), backward 4.1 ms (1.3 TB/s).
// ---------------------------------------------------------------------------

template <bool BACKWARD, typename S, typename I, typename O, typename A>
__global__ void __launch_bounds__(kRnDirectWarps * 32) rn_direct_kernel(const __grid_constant__ RnArgs a) {
  __shared__ A scratch[8 * kRnWarps];
  chain_enter();
  RnTeam<A, false, false> team{static_cast<int>(threadIdx.x), kRnDirectWarps * 32, kRnDirectWarps, 1, scratch, 0};
  const RnFactors<false, A> f{static_cast<const A*>(a.post), static_cast<const A*>(a.scale), static_cast<const A*>(a.pre)};
  A* part = static_cast<A*>(a.part) + (int64_t)blockIdx.x * 2 * a.chan;
  if constexpr (BACKWARD) {
    // a channel's sums are kept by the thread that owns the channel
    for (int i = 0; i < a.n_blocks; ++i) {
      const RnBlock b = a.blocks[i];
      for (int u = team.t; u < b.mul; u += team.lanes) part[b.coff + u] = part[a.chan + b.coff + u] = A(0);
    }
  }
  for (int64_t n = blockIdx.x; n < a.N; n += gridDim.x) {
    if constexpr (BACKWARD) {
      const RnBackwardRow<S, I, O, A> row{rn_at<S>(a, kRnGout, n), rn_at<S>(a, kRnX, n), rn_at<I>(a, kRnGy, n),
                                          rn_at<I>(a, kRnBz, n),   rn_at<I>(a, kRnBq, n), rn_at<S>(a, kRnGh, n),
                                          rn_at<O>(a, kRnGz, n),   rn_at<O>(a, kRnGq, n), part, true};
      rn_row<kRnDirect>(a, a.blocks, row, f, team);
    } else {
      const RnForwardRow<S, I, O> row{rn_at<S>(a, kRnH, n), rn_at<I>(a, kRnZ, n), rn_at<I>(a, kRnQ, n),
                                      rn_at<S>(a, kRnOut, n), rn_at<O>(a, kRnY, n)};
      rn_row<kRnDirect>(a, a.blocks, row, f, team);
    }
  }
}

template <bool BACKWARD, int KIND, typename S, typename I, typename O, typename A>
cudaError_t rn_launch_staged(const RnArgs& a, cudaStream_t st) {
  if (smem_cap_cached(reinterpret_cast<const void*>(rn_staged_kernel<BACKWARD, KIND, S, I, O, A>)) < a.smem)
    return cudaErrorInvalidConfiguration;
  return chain_launch(rn_staged_kernel<BACKWARD, KIND, S, I, O, A>, a.ctas, a.groups * a.warps * 32, a.smem, st, a);
}

// FP64 has no kernels of its own for full rows: its tiles are twice as long, its shares spill
template <bool BACKWARD, typename S, typename I, typename O, typename A>
cudaError_t rn_launch(const RnArgs& a, cudaStream_t st) {
  constexpr bool wide = sizeof(A) == 8;
  cudaError_t e;
  switch (a.kind) {
    case kRnOneFull: e = rn_launch_staged<BACKWARD, wide ? kRnOne : kRnOneFull, S, I, O, A>(a, st); break;
    case kRnFewFull: e = rn_launch_staged<BACKWARD, wide ? kRnOne : kRnFewFull, S, I, O, A>(a, st); break;
    case kRnOne: e = rn_launch_staged<BACKWARD, kRnOne, S, I, O, A>(a, st); break;
    case kRnManyFull: e = rn_launch_staged<BACKWARD, wide ? kRnMany : kRnManyFull, S, I, O, A>(a, st); break;
    case kRnMany: e = rn_launch_staged<BACKWARD, kRnMany, S, I, O, A>(a, st); break;
    default:
      e = chain_launch(rn_direct_kernel<BACKWARD, S, I, O, A>, a.ctas, kRnDirectWarps * 32, 0, st, a);
  }
  if (!BACKWARD || e != cudaSuccess || a.ticket || (a.kind != kRnDirect && a.ctas == 1) || !(a.gpost || a.gscale || a.gpre)) return e;
  return chain_launch(rn_reduce_kernel<A>, (2 * a.chan + 31) / 32, 256, 0, st, a.part, a.ctas, a.chan, a.post, a.scale, a.gpost,
                      a.gscale, a.gpre);
}

}  // namespace
}  // namespace cgtp
