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
// A team of threads owns a row; a thread owns channels u, u + team, ... of every block, so the
// sums over m (gates, parameter gradients) stay inside a thread and the only exchange is the
// block sum of an rms.  Rows are dealt to teams by index and a channel's partial sums belong to
// one thread of a team, so every sum has a fixed order.
#pragma once

#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include "resnorm.h"

namespace cgtp {
namespace {

template <typename A>
__device__ __forceinline__ A rn_get(const float* p) {
  return static_cast<A>(*p);
}
template <typename A>
__device__ __forceinline__ A rn_get(const double* p) {
  return static_cast<A>(*p);
}
template <typename A>
__device__ __forceinline__ A rn_get(const __nv_bfloat16* p) {
  return static_cast<A>(__bfloat162float(*p));
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
__device__ __forceinline__ float rn_exp(float v) { return expf(v); }
__device__ __forceinline__ double rn_exp(double v) { return exp(v); }

// a(q) and, when asked for, a'(q)
template <typename A>
__device__ __forceinline__ A rn_gate(int act, A q, A* derivative) {
  if (act == CGTP_ACT_IDENTITY) {
    if (derivative) *derivative = A(1);
    return q;
  }
  const A s = A(1) / (A(1) + rn_exp(-q));
  if (act == CGTP_ACT_SIGMOID) {
    if (derivative) *derivative = s * (A(1) - s);
    return s;
  }
  if (derivative) *derivative = s * (A(1) + q * (A(1) - s));
  return q * s;
}

// Sum over the team.  Every thread of the CTA calls it the same number of times.
template <typename A>
__device__ __forceinline__ A rn_team_sum(A v, int team, A* scratch) {
  const int wide = team < 32 ? team : 32;
  for (int o = wide >> 1; o; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
  if (team <= 32) return v;
  __syncthreads();   // the previous sum has been read
  if ((threadIdx.x & 31) == 0) scratch[threadIdx.x >> 5] = v;
  __syncthreads();
  A t = A(0);
  for (int w = 0; w < kRnThreads / 32; ++w) t += scratch[w];
  return t;
}

template <typename A, typename P>
__device__ __forceinline__ A rn_param(const void* p, int c) {
  return p ? rn_get<A>(static_cast<const P*>(p) + c) : A(1);
}

// S: residual stream, I: what comes from a product, O: what goes to one, A: arithmetic and parameters.
template <typename S, typename I, typename O, typename A, int D>
__device__ __forceinline__ void rn_forward_block(const RnArgs& a, const RnBlock b, int64_t n, bool live, int t,
                                                 A* scratch) {
  const A inv_n = A(1) / static_cast<A>(b.mul * D), eps = static_cast<A>(a.eps);
  const S* h = a.h ? static_cast<const S*>(a.h) + n * a.ld_h + b.off : nullptr;
  const I* z = a.z ? static_cast<const I*>(a.z) + n * a.ld_z + b.off : nullptr;
  const I* q = a.q ? static_cast<const I*>(a.q) + n * a.ld_q + b.coff : nullptr;
  S* out = a.out ? static_cast<S*>(a.out) + n * a.ld_out + b.off : nullptr;
  const int step = a.team;
  A r = A(1);
  if (z && a.post_norm) {
    A ss = A(0);
    for (int u = t; u < b.mul; u += step)
#pragma unroll
      for (int m = 0; m < D; ++m) {
        const A v = rn_get<A>(z + u * D + m);
        ss += v * v;
      }
    r = rn_rsqrt(rn_team_sum(ss, a.team, scratch) * inv_n + eps);
  }
  A ss = A(0);
  for (int u = t; u < b.mul; u += step) {
    if (z) {
      const int c = b.coff + u;
      A w = r * rn_param<A, A>(a.post, c) * rn_param<A, A>(a.scale, c);
      if (q) w *= rn_gate<A>(a.act, rn_get<A>(q + u), nullptr);
#pragma unroll
      for (int m = 0; m < D; ++m) {
        A v = w * rn_get<A>(z + u * D + m);
        if (h) v += static_cast<A>(a.alpha) * rn_get<A>(h + u * D + m);
        if (live) v = rn_put(out + u * D + m, v);
        ss += v * v;
      }
    } else {
#pragma unroll
      for (int m = 0; m < D; ++m) {
        const A v = rn_get<A>(h + u * D + m);
        ss += v * v;
      }
    }
  }
  if (!a.pre_norm) return;
  const A p = rn_rsqrt(rn_team_sum(ss, a.team, scratch) * inv_n + eps);
  if (!live) return;
  const S* x = z ? out : h;
  O* y = static_cast<O*>(a.y) + n * a.ld_y + b.off;
  for (int u = t; u < b.mul; u += step) {
    const A w = p * rn_param<A, A>(a.pre, b.coff + u);
#pragma unroll
    for (int m = 0; m < D; ++m) rn_put(y + u * D + m, w * rn_get<A>(x + u * D + m));
  }
}

template <typename S, typename I, typename O, typename A, int D>
__device__ __forceinline__ void rn_backward_block(const RnArgs& a, const RnBlock b, int64_t n, bool live, int t,
                                                  A* scratch, A* part) {
  const A inv_n = A(1) / static_cast<A>(b.mul * D), eps = static_cast<A>(a.eps);
  const S* g = a.gout ? static_cast<const S*>(a.gout) + n * a.ld_gout + b.off : nullptr;
  const I* gy = a.pre_norm ? static_cast<const I*>(a.gy) + n * a.ld_gy + b.off : nullptr;
  const S* x = a.pre_norm ? static_cast<const S*>(a.x) + n * a.ld_x + b.off : nullptr;
  const I* z = a.z ? static_cast<const I*>(a.z) + n * a.ld_z + b.off : nullptr;
  const I* q = a.q ? static_cast<const I*>(a.q) + n * a.ld_q + b.coff : nullptr;
  S* gh = a.gh ? static_cast<S*>(a.gh) + n * a.ld_gh + b.off : nullptr;
  O* gz = a.z ? static_cast<O*>(a.gz) + n * a.ld_gz + b.off : nullptr;
  O* gq = a.q ? static_cast<O*>(a.gq) + n * a.ld_gq + b.coff : nullptr;
  const int step = a.team;
  A p = A(0), k = A(0), r = A(1);
  if (a.pre_norm) {
    A sx = A(0), sxy = A(0);
    for (int u = t; u < b.mul; u += step) {
      const A pre = rn_param<A, A>(a.pre, b.coff + u);
      A xy = A(0);
#pragma unroll
      for (int m = 0; m < D; ++m) {
        const A v = rn_get<A>(x + u * D + m);
        sx += v * v;
        xy += v * rn_get<A>(gy + u * D + m);
      }
      sxy += pre * xy;
    }
    p = rn_rsqrt(rn_team_sum(sx, a.team, scratch) * inv_n + eps);
    k = p * p * p * inv_n * rn_team_sum(sxy, a.team, scratch);
  }
  if (z && a.post_norm) {
    A sz = A(0);
    for (int u = t; u < b.mul; u += step)
#pragma unroll
      for (int m = 0; m < D; ++m) {
        const A v = rn_get<A>(z + u * D + m);
        sz += v * v;
      }
    r = rn_rsqrt(rn_team_sum(sz, a.team, scratch) * inv_n + eps);
  }
  A along = A(0);   // sum over the block of w d z r
  for (int u = t; u < b.mul; u += step) {
    const int c = b.coff + u;
    const A pre = p * rn_param<A, A>(a.pre, c);
    A P = A(0), xy = A(0), d[D];
#pragma unroll
    for (int m = 0; m < D; ++m) {
      A v = g ? rn_get<A>(g + u * D + m) : A(0);
      if (gy) {
        const A e = rn_get<A>(gy + u * D + m), f = rn_get<A>(x + u * D + m);
        v += pre * e - k * f;
        xy += e * f;
      }
      d[m] = v;
      if (z) P += v * rn_get<A>(z + u * D + m);
    }
    if (live && gh)
#pragma unroll
      for (int m = 0; m < D; ++m) rn_put(gh + u * D + m, static_cast<A>(a.alpha) * d[m]);
    if (live && gy) part[a.chan + c] += p * xy;
    if (z) {
      P *= r;
      const A base = rn_param<A, A>(a.post, c) * rn_param<A, A>(a.scale, c);
      A act = A(1), der = A(0);
      if (q) act = rn_gate<A>(a.act, rn_get<A>(q + u), &der);
      along += base * act * P;
      if (live) {
        part[c] += act * P;
        if (q) rn_put(gq + u, base * der * P);
        if (!a.post_norm)
#pragma unroll
          for (int m = 0; m < D; ++m) rn_put(gz + u * D + m, base * act * d[m]);
      }
    }
  }
  if (!z || !a.post_norm) return;
  const A kz = r * r * inv_n * rn_team_sum(along, a.team, scratch);
  if (!live) return;
  for (int u = t; u < b.mul; u += step) {
    const int c = b.coff + u;
    const A pre = p * rn_param<A, A>(a.pre, c);
    A w = r * rn_param<A, A>(a.post, c) * rn_param<A, A>(a.scale, c);
    if (q) w *= rn_gate<A>(a.act, rn_get<A>(q + u), nullptr);
#pragma unroll
    for (int m = 0; m < D; ++m) {
      A v = g ? rn_get<A>(g + u * D + m) : A(0);
      if (gy) v += pre * rn_get<A>(gy + u * D + m) - k * rn_get<A>(x + u * D + m);
      rn_put(gz + u * D + m, w * v - kz * rn_get<A>(z + u * D + m));
    }
  }
}

#define CGTP_RN_SWITCH(CALL)                                                                                      \
  switch (b.D) {                                                                                                  \
    case 1: CALL(1); break;                                                                                       \
    case 3: CALL(3); break;                                                                                       \
    case 5: CALL(5); break;                                                                                       \
    case 7: CALL(7); break;                                                                                       \
    case 9: CALL(9); break;                                                                                       \
    case 11: CALL(11); break;                                                                                     \
    case 13: CALL(13); break;                                                                                     \
    default: CALL(15); break;                                                                                     \
  }

template <typename S, typename I, typename O, typename A>
__global__ void __launch_bounds__(kRnThreads) rn_forward_kernel(const RnArgs a) {
  __shared__ A scratch[kRnThreads / 32];
  const int teams = kRnThreads / a.team, t = threadIdx.x % a.team;
  const int64_t all = (int64_t)gridDim.x * teams;
  // every thread of a CTA runs the same number of rounds (the sums are collective)
  for (int64_t n0 = (int64_t)blockIdx.x * teams; n0 < a.N; n0 += all) {
    const int64_t mine = n0 + threadIdx.x / a.team;
    const bool live = mine < a.N;
    const int64_t n = live ? mine : a.N - 1;
    for (int i = 0; i < a.n_blocks; ++i) {
      const RnBlock b = a.blocks[i];
#define CGTP_RN_CALL(D) rn_forward_block<S, I, O, A, D>(a, b, n, live, t, scratch)
      CGTP_RN_SWITCH(CGTP_RN_CALL)
#undef CGTP_RN_CALL
    }
  }
}

template <typename S, typename I, typename O, typename A>
__global__ void __launch_bounds__(kRnThreads) rn_backward_kernel(const RnArgs a) {
  __shared__ A scratch[kRnThreads / 32];
  const int teams = kRnThreads / a.team, t = threadIdx.x % a.team;
  const int64_t all = (int64_t)gridDim.x * teams;
  const int64_t slot = (int64_t)blockIdx.x * teams + threadIdx.x / a.team;
  A* part = static_cast<A*>(a.part) + slot * 2 * a.chan;
  for (int i = 0; i < a.n_blocks; ++i) {
    const RnBlock b = a.blocks[i];
    for (int u = t; u < b.mul; u += a.team) part[b.coff + u] = part[a.chan + b.coff + u] = A(0);
  }
  for (int64_t n0 = (int64_t)blockIdx.x * teams; n0 < a.N; n0 += all) {
    const int64_t mine = n0 + threadIdx.x / a.team;
    const bool live = mine < a.N;
    const int64_t n = live ? mine : a.N - 1;
    for (int i = 0; i < a.n_blocks; ++i) {
      const RnBlock b = a.blocks[i];
#define CGTP_RN_CALL(D) rn_backward_block<S, I, O, A, D>(a, b, n, live, t, scratch, part)
      CGTP_RN_SWITCH(CGTP_RN_CALL)
#undef CGTP_RN_CALL
    }
  }
}

// gpost = scale A, gscale = post A, gpre: the teams' partial sums added in team order.
template <typename A>
__global__ void rn_reduce_kernel(const RnArgs a, int slots) {
  const int c = blockIdx.x * blockDim.x + threadIdx.x;
  if (c >= a.chan) return;
  const A* part = static_cast<const A*>(a.part);
  A s = A(0), g = A(0);
  for (int i = 0; i < slots; ++i) {
    s += part[(int64_t)i * 2 * a.chan + c];
    g += part[(int64_t)i * 2 * a.chan + a.chan + c];
  }
  if (a.gpost) static_cast<A*>(a.gpost)[c] = s * rn_param<A, A>(a.scale, c);
  if (a.gscale) static_cast<A*>(a.gscale)[c] = s * rn_param<A, A>(a.post, c);
  if (a.gpre) static_cast<A*>(a.gpre)[c] = g;
}

template <typename S, typename I, typename O, typename A>
cudaError_t rn_launch(const RnArgs& a, bool backward, int ctas, cudaStream_t st) {
  if (!backward) {
    rn_forward_kernel<S, I, O, A><<<ctas, kRnThreads, 0, st>>>(a);
    return cudaGetLastError();
  }
  rn_backward_kernel<S, I, O, A><<<ctas, kRnThreads, 0, st>>>(a);
  cudaError_t e = cudaGetLastError();
  if (e != cudaSuccess || !(a.gpost || a.gscale || a.gpre)) return e;
  rn_reduce_kernel<A><<<(a.chan + 127) / 128, 128, 0, st>>>(a, ctas * (kRnThreads / a.team));
  return cudaGetLastError();
}

}  // namespace
}  // namespace cgtp
