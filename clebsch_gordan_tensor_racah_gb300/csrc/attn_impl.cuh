// attn_impl.cuh -- kernels of the attention along a graph's edges (include/cgtp_attn.h), one translation unit
// an element type.
//
// Mathematics.  For an edge e of receiver n with source s = col[e], head h and its shared head hk = h / group,
//   z = scale <q[n,h], k[s,hk]> + T[bucket(r_e), h] + b[e,h],   a = exp(z - lse[n,h])
//   out[n,h] = sum_e a v[s,hk]                                  (values of sources)
//   w'[e,h]  = a w[e,h]                                         (rows of edges)
// and backward, with dp = <gout[n,h], v[s,hk]> or <gw'[e,h], w[e,h]>,
//   ds = a (dp - sum_e a dp),  gq = scale sum_e ds k,  gk = scale sum ds q,  gv = sum a gout,  gw = a gw'.
// A logit of -infinity leaves its edge out: a weight of zero takes nothing from its edge's rows, whatever they hold.
//
// Split.  A row's threads (a warp, or a CTA) hold `sub` edges at once.  Dot products: a team of threads a
// (edge, head) pair.  Sums over edges: a thread owns vectors of the result's row and runs over the edges, so that
// nothing is reduced and every gathered row is read in wide pieces; where the row has fewer vectors than there are
// threads, several streams of edges are added at the end in a fixed order.  The receivers' kernel of the backward
// writes a and ds (edges x heads); the sources' kernel, over the transpose, only gathers and adds.  Rows longer
// than the graph's chunk are cut into items whose partial results another launch joins in a fixed order.
#pragma once

#include <cuda_bf16.h>

#include <algorithm>
#include <cmath>
#include <type_traits>

#include "attn.h"
#include "chain.cuh"

namespace cgtp {
namespace {

using bf16 = __nv_bfloat16;

// ---------------------------------------------------------------------------
// vectors of elements
// ---------------------------------------------------------------------------
__device__ __forceinline__ float wide(float x) { return x; }
__device__ __forceinline__ double wide(double x) { return x; }
__device__ __forceinline__ float wide(bf16 x) { return __bfloat162float(x); }

template <typename T>
__device__ __forceinline__ T narrow(float x);
template <>
__device__ __forceinline__ float narrow<float>(float x) { return x; }
template <>
__device__ __forceinline__ bf16 narrow<bf16>(float x) { return __float2bfloat16_rn(x); }
__device__ __forceinline__ double narrow_d(double x) { return x; }

template <int BYTES>
struct Raw;
template <>
struct Raw<16> { using type = uint4; };
template <>
struct Raw<8> { using type = uint2; };
template <>
struct Raw<4> { using type = unsigned; };
template <>
struct Raw<2> { using type = unsigned short; };

// V elements, read and written in pieces of at most 16 bytes
template <typename T, int V>
struct Pack {
  static constexpr int kBytes = V * sizeof(T) < 16 ? V * sizeof(T) : 16, kRaws = V * sizeof(T) / kBytes;
  using W = typename Raw<kBytes>::type;
  union {
    W raw[kRaws];
    T e[V];
  };
  __device__ __forceinline__ Pack() {}
  __device__ __forceinline__ void load(const T* p) {
#pragma unroll
    for (int i = 0; i < kRaws; ++i) raw[i] = reinterpret_cast<const W*>(p)[i];
  }
  __device__ __forceinline__ void store(T* p) const {
#pragma unroll
    for (int i = 0; i < kRaws; ++i) reinterpret_cast<W*>(p)[i] = raw[i];
  }
};

template <typename T, typename A>
__device__ __forceinline__ T to(A x) {
  if constexpr (std::is_same<T, A>::value) return x;
  else return narrow<T>(x);
}

template <typename A>
__device__ __forceinline__ A lowest() { return -static_cast<A>(INFINITY); }
__device__ __forceinline__ float expo(float x) { return expf(x); }
__device__ __forceinline__ double expo(double x) { return exp(x); }
__device__ __forceinline__ float loga(float x) { return logf(x); }
__device__ __forceinline__ double loga(double x) { return log(x); }
__device__ __forceinline__ float larger(float a, float b) { return fmaxf(a, b); }
__device__ __forceinline__ double larger(double a, double b) { return fmax(a, b); }

// widths of vectors of a storage type: 16 bytes, half of that for bfloat16, one element
template <typename S>
struct Widths {
  static constexpr int kFull = 16 / sizeof(S), kHalf = sizeof(S) == 2 ? 4 : 16 / sizeof(S);
};
template <typename S, typename F>
__device__ __forceinline__ void with_width(int v, F&& f) {
  if (v == Widths<S>::kFull) f(std::integral_constant<int, Widths<S>::kFull>());
  else if (Widths<S>::kHalf != Widths<S>::kFull && v == Widths<S>::kHalf) f(std::integral_constant<int, Widths<S>::kHalf>());
  else f(std::integral_constant<int, 1>());
}

// ---------------------------------------------------------------------------
// the threads of a row
// ---------------------------------------------------------------------------
template <bool WARP>
struct Group {
  int t, n;
  __device__ __forceinline__ Group() : t(WARP ? threadIdx.x & 31 : threadIdx.x), n(WARP ? 32 : blockDim.x) {}
  __device__ __forceinline__ void sync() const {
    if (WARP) __syncwarp();
    else __syncthreads();
  }
};

struct Item {
  int64_t row;
  int64_t e0, e1;
  int index;   // item of a split row, or -1
};

// f(item) for every piece of work of this group.  First come the items of split rows, the longest work.
template <bool WARP, typename F>
__device__ __forceinline__ void each_item(const AtArgs& a, const Group<WARP>& g, F&& f) {
  const int64_t groups = WARP ? int64_t(gridDim.x) * (blockDim.x / 32) : gridDim.x;
  const int64_t first = WARP ? int64_t(blockIdx.x) * (blockDim.x / 32) + threadIdx.x / 32 : blockIdx.x;
  const int64_t total = a.n_items + (a.phase == kAtSecond ? 0 : a.n_rows);
  for (int64_t w = first; w < total; w += groups) {
    Item it;
    if (w < a.n_items) {
      const Int4 v = a.items[w];
      it = {v.x, v.y, v.z, static_cast<int>(w)};
    } else {
      it.row = w - a.n_items;
      it.e0 = a.rowptr[it.row];
      it.e1 = a.rowptr[it.row + 1];
      it.index = -1;
      if (a.n_items && it.e1 - it.e0 > a.chunk) continue;
    }
    f(it);
    g.sync();
  }
}

// pair / heads for pairs below 2^24 (heads <= 64: the error of the multiplier is below 2^-32 a unit)
__device__ __forceinline__ int pair_edge(const AtArgs& a, int pair) {
  return a.heads == 1 ? pair : static_cast<int>(__umulhi(static_cast<unsigned>(pair), a.heads_magic));
}

// A row of all heads into shared memory, head by head, in the arithmetic's type.
template <typename S, typename A, bool WARP>
__device__ __forceinline__ void stage(const Group<WARP>& g, const AtTab& tab, int heads, const S* row, A* to_) {
  with_width<S>(tab.vec, [&](auto v) {
    constexpr int V = decltype(v)::value;
    for (int c = g.t; c < heads * tab.pieces; c += g.n) {
      Pack<S, V> x;
      x.load(row + tab.dot_full[c]);
#pragma unroll
      for (int j = 0; j < V; ++j) to_[c * V + j] = wide(x.e[j]);
    }
  });
}

// f(i, h, <x[h], rows[idx(i)][h or its shared head]>) for every pair of the cnt edges and the heads, by one
// thread of the pair's team.
template <typename S, typename A, bool WARP, typename F>
__device__ __forceinline__ void dots(const AtArgs& a, const Group<WARP>& g, const AtTab& tab, int team, int cnt, const A* x, const S* rows,
                                     int64_t ld, const int* idx, F&& f) {
  const int total = cnt * a.heads, lane = g.t & (team - 1), teams = g.n / team;
  constexpr int U = 4;
  with_width<S>(tab.vec, [&](auto v) {
    constexpr int V = decltype(v)::value;
    // (every thread of a warp takes the same number of turns: the shuffles need all of them)
    for (int base = 0; base < total; base += U * teams) {
      A sum[U];
      const S* row[U];
      const A* xs[U];
      const int* off[U];
#pragma unroll
      for (int u = 0; u < U; ++u) {
        const int pair = min(base + u * teams + g.t / team, total - 1);
        const int i = pair_edge(a, pair), h = pair - i * a.heads;
        row[u] = rows + int64_t(idx[i]) * ld;
        xs[u] = x + h * tab.pieces * V;
        off[u] = tab.dot_kv + (a.group == 1 ? h : h / a.group) * tab.pieces;
        sum[u] = 0;
      }
      for (int c = lane; c < tab.pieces; c += team) {
        Pack<S, V> y[U];
#pragma unroll
        for (int u = 0; u < U; ++u) y[u].load(row[u] + off[u][c]);
#pragma unroll
        for (int u = 0; u < U; ++u)
#pragma unroll
          for (int j = 0; j < V; ++j) sum[u] += xs[u][c * V + j] * wide(y[u].e[j]);
      }
#pragma unroll
      for (int u = 0; u < U; ++u) {
        for (int o = team / 2; o > 0; o /= 2) sum[u] += __shfl_xor_sync(0xffffffffu, sum[u], o);
        const int pair = base + u * teams + g.t / team;
        if (lane == 0 && pair < total) {
          const int i = pair_edge(a, pair);
          f(i, pair - i * a.heads, sum[u]);
        }
      }
    }
  });
}

// Sums over edges, in the order of the edges within a stream:
//   r[p] = (first ? 0 : keep[p] * rescale[h]) + sum_i coef[i][h] rows[idx(i)][offset]   (over the `ng` heads of a piece)
// and emit(p, head, r) where last, keep[p] = r otherwise.
template <int V, typename S, typename A, bool WARP, typename F>
__device__ __forceinline__ void accumulate(const Group<WARP>& g, int heads, int cnt, int pieces, int ng, const int* tab, const A* coef,
                                           const S* rows, int64_t ld, const int* idx, A* keep, const A* rescale, A* red, bool first,
                                           bool last, F&& emit) {
  const int streams = pieces < g.n && cnt > 1 ? min(g.n / pieces, cnt) : 1;
  const auto finish = [&](int p, int h, A* r) {
    if (!first) {
      const A f = rescale ? rescale[h] : A(1);
#pragma unroll
      for (int j = 0; j < V; ++j) r[j] += f == 0 ? A(0) : keep[p * V + j] * f;
    }
    if (last) {
      emit(p, h, r);
    } else {
#pragma unroll
      for (int j = 0; j < V; ++j) keep[p * V + j] = r[j];
    }
  };
  const auto run = [&](int p, int at, int step, A* r) {
#pragma unroll
    for (int j = 0; j < V; ++j) r[j] = 0;
    for (int q = 0; q < ng; ++q) {
      const int entry = tab[p * ng + q], h = entry >> kAtHeadShift;
      const S* col = rows + (entry & ((1 << kAtHeadShift) - 1));
      constexpr int U = 4;
      int i = at;
      for (; i + (U - 1) * step < cnt; i += U * step) {
        Pack<S, V> y[U];
        A c[U];
#pragma unroll
        for (int u = 0; u < U; ++u) {
          y[u].load(col + int64_t(idx[i + u * step]) * ld);
          c[u] = coef[(i + u * step) * heads + h];
        }
#pragma unroll
        for (int u = 0; u < U; ++u)
          if (c[u] != 0) {
#pragma unroll
            for (int j = 0; j < V; ++j) r[j] += c[u] * wide(y[u].e[j]);
          }
      }
      for (; i < cnt; i += step) {
        Pack<S, V> y;
        y.load(col + int64_t(idx[i]) * ld);
        const A c = coef[i * heads + h];
        if (c != 0) {
#pragma unroll
          for (int j = 0; j < V; ++j) r[j] += c * wide(y.e[j]);
        }
      }
    }
  };
  if (streams == 1) {
    for (int p = g.t; p < pieces; p += g.n) {
      A r[V];
      run(p, 0, 1, r);
      finish(p, tab[p * ng] >> kAtHeadShift, r);
    }
    return;
  }
  const int s = g.t / pieces, p = g.t - s * pieces;
  A r[V];
  if (s < streams) run(p, s, streams, r);
  g.sync();   // `red` may still be read
  if (s > 0 && s < streams) {
#pragma unroll
    for (int j = 0; j < V; ++j) red[(s * pieces + p) * V + j] = r[j];
  }
  g.sync();
  if (s == 0) {
    for (int q = 1; q < streams; ++q) {
#pragma unroll
      for (int j = 0; j < V; ++j) r[j] += red[(q * pieces + p) * V + j];
    }
    finish(p, tab[p * ng] >> kAtHeadShift, r);
  }
}

// For every head, by the lanes of one warp: r = combine over i < cnt of take(i, h), then done(h, r) by one lane.
// f(h, i, lane is the head's first, all) is called in two passes by the caller's lambda through `loop`.
struct HeadLanes {
  int h, slot, slots, width;   // head, first edge and step of this lane; lanes that differ in `width` and above share the head
  bool on;
};
template <bool WARP, typename F>
__device__ __forceinline__ void each_head(const Group<WARP>& g, int heads, F&& f) {
  const int warps = WARP ? 1 : g.n / 32, per = (heads + warps - 1) / warps, w = g.t / 32, lane = g.t & 31;
  for (int h0 = w * per; h0 < min(heads, (w + 1) * per); h0 += 32) {
    const int count = min(min(heads, (w + 1) * per) - h0, 32);
    int width = 1;
    while (width < count) width *= 2;
    HeadLanes l;
    l.width = width;
    l.slots = 32 / width;
    l.slot = lane / width;
    const int k = lane & (width - 1);
    l.on = k < count;
    l.h = h0 + min(k, count - 1);
    f(l);
  }
}
template <typename A>
__device__ __forceinline__ A all_max(const HeadLanes& l, A x) {
  for (int o = l.width; o < 32; o *= 2) x = larger(x, __shfl_xor_sync(0xffffffffu, x, o));
  return x;
}
template <typename A>
__device__ __forceinline__ A all_sum(const HeadLanes& l, A x) {
  for (int o = l.width; o < 32; o *= 2) x += __shfl_xor_sync(0xffffffffu, x, o);
  return x;
}

// number of borders <= r (0 for NaN)
template <typename A>
__device__ __forceinline__ int bucket_of(const A* borders, int n, A r) {
  int lo = 0, hi = n;
  while (lo < hi) {
    const int mid = (lo + hi) / 2;
    if (borders[mid] <= r) lo = mid + 1;
    else hi = mid;
  }
  return lo;
}

// A row's regions of shared memory
template <typename A>
struct Smem {
  A *q, *g, *z, *p, *stat, *acc, *red;
  int *idx, *bucket;
  template <bool WARP>
  __device__ __forceinline__ Smem(const AtArgs& a, const Group<WARP>&) {
    extern __shared__ __align__(16) char at_smem[];
    char* s = at_smem + (WARP ? (threadIdx.x / 32) * a.group_smem : 0);
    q = reinterpret_cast<A*>(s);
    g = reinterpret_cast<A*>(s + a.at_g);
    z = reinterpret_cast<A*>(s + a.at_z);
    p = reinterpret_cast<A*>(s + a.at_p);
    idx = reinterpret_cast<int*>(s + a.at_idx);
    bucket = idx + a.sub;
    stat = reinterpret_cast<A*>(s + a.at_stat);
    acc = reinterpret_cast<A*>(s + a.at_acc);
    red = reinterpret_cast<A*>(s + a.at_red);
  }
};

// Ends of the edges [e, e + cnt) and their buckets.
template <typename A, bool WARP>
__device__ __forceinline__ void load_edges(const AtArgs& a, const Group<WARP>& g, const Smem<A>& sm, int64_t e, int cnt) {
  for (int i = g.t; i < cnt; i += g.n) {
    sm.idx[i] = a.col[e + i];
    if (a.table) sm.bucket[i] = bucket_of(static_cast<const A*>(a.borders), a.n_borders, static_cast<const A*>(a.lengths)[e + i]);
  }
}

// Logits of the edges [e, e + cnt) into z.
template <typename S, typename A, bool WARP>
__device__ __forceinline__ void logits(const AtArgs& a, const Group<WARP>& g, const Smem<A>& sm, int64_t e, int cnt) {
  const A scale = static_cast<A>(a.scale);
  const A *table = static_cast<const A*>(a.table), *bias = static_cast<const A*>(a.bias);
  dots<S, A>(a, g, a.qk, a.team_qk, cnt, sm.q, reinterpret_cast<const S*>(a.k.p), a.k.ld, sm.idx, [&](int i, int h, A s) {
    A b = 0;
    if (table) b = table[sm.bucket[i] * a.heads + h];
    if (bias) b += bias[(e + i) * a.heads + h];
    sm.z[i * a.heads + h] = b == lowest<A>() ? b : s * scale + b;
  });
}

// ---------------------------------------------------------------------------
// forward
// ---------------------------------------------------------------------------

// Running maximum (stat[h]) and sum of exponentials (stat[heads + h]) over the edges in z, which become exp(z -
// maximum); stat[2 heads + h] = factor of what was summed before.
template <typename A, bool WARP>
__device__ __forceinline__ void softmax_step(const AtArgs& a, const Group<WARP>& g, const Smem<A>& sm, int cnt, bool first, bool keep_z) {
  each_head(g, a.heads, [&](const HeadLanes& l) {
    A top = lowest<A>();
    for (int i = l.slot; i < cnt; i += l.slots) top = larger(top, sm.z[i * a.heads + l.h]);
    top = all_max(l, top);
    const A before = first ? lowest<A>() : sm.stat[l.h];
    top = larger(top, before);
    const A shift = top == lowest<A>() ? A(0) : top;
    A sum = 0;
    for (int i = l.slot; i < cnt; i += l.slots) {
      const A p = expo(sm.z[i * a.heads + l.h] - shift);
      // (lanes beyond the last head repeat it and write nothing)
      if (!keep_z && l.on) sm.z[i * a.heads + l.h] = p;
      sum += p;
    }
    sum = all_sum(l, sum);
    __syncwarp();
    if (l.on && l.slot == 0) {
      const A f = first ? A(0) : expo(before - shift);
      sm.stat[l.h] = top;
      sm.stat[a.heads + l.h] = (first ? A(0) : sm.stat[a.heads + l.h] * f) + sum;
      sm.stat[2 * a.heads + l.h] = f;
    }
  });
}

template <typename S, typename R, typename A, bool WARP>
__global__ void attn_forward_kernel(const AtArgs a) {
  chain_enter();
  const Group<WARP> g;
  const Smem<A> sm(a, g);
  const int width = a.heads * a.dv;
  each_item(a, g, [&](const Item& it) {
    stage<S, A>(g, a.qk, a.heads, reinterpret_cast<const S*>(a.q.p) + it.row * a.q.ld, sm.q);
    const bool part = it.index >= 0;
    A* to_part = static_cast<A*>(a.part) + int64_t(it.index) * (width + 2 * a.heads);
    bool first = true;
    int64_t e = it.e0;
    do {
      const int cnt = static_cast<int>(min(int64_t(a.sub), it.e1 - e));
      load_edges(a, g, sm, e, cnt);
      g.sync();
      logits<S>(a, g, sm, e, cnt);
      g.sync();
      softmax_step(a, g, sm, cnt, first, false);
      g.sync();
      const bool last = e + cnt >= it.e1;
      with_width<S>(a.vv.vec, [&](auto v) {
        constexpr int V = decltype(v)::value;
        accumulate<V>(g, a.heads, cnt, a.heads * a.vv.pieces, 1, a.vv.acc, sm.z, reinterpret_cast<const S*>(a.v.p), a.v.ld, sm.idx, sm.acc,
                      sm.stat + 2 * a.heads, sm.red, first, last, [&](int p, int h, const A* r) {
                        if (part) {
#pragma unroll
                          for (int j = 0; j < V; ++j) to_part[p * V + j] = r[j];
                        } else {
                          const A l = sm.stat[a.heads + h], f = l == 0 ? A(0) : A(1) / l;
                          Pack<R, V> y;
#pragma unroll
                          for (int j = 0; j < V; ++j) y.e[j] = to<R>(r[j] * f);
                          y.store(reinterpret_cast<R*>(a.out.p) + it.row * a.out.ld + p * V);
                        }
                      });
      });
      e += cnt;
      first = false;
      if (!last) g.sync();
    } while (e < it.e1);
    for (int h = g.t; h < a.heads; h += g.n) {
      if (part) {
        to_part[width + h] = sm.stat[h];
        to_part[width + a.heads + h] = sm.stat[a.heads + h];
      } else {
        static_cast<A*>(a.lse)[it.row * a.heads + h] = loga(sm.stat[a.heads + h]) + (sm.stat[h] == lowest<A>() ? A(0) : sm.stat[h]);
      }
    }
  });
}

// Joins the parts of a split row: grid (columns / 32, rows); 8 streams of parts a column.
template <typename R, typename A>
__global__ void attn_join_forward_kernel(const AtArgs a) {
  chain_enter();
  __shared__ A red[8][33], red_l[8][33];
  const Int4 j = a.joins[blockIdx.y];
  const int width = a.heads * a.dv, stride = width + 2 * a.heads;
  const int c = blockIdx.x * 32 + threadIdx.x, s = threadIdx.y;
  const A* part = static_cast<const A*>(a.part) + int64_t(j.y) * stride;
  // the columns' heads: those of the vectors in the order of memory, then the statistics'
  const bool value = c < width, stat = c >= width && c < width + a.heads;
  const int h = value ? a.vv.acc[c / a.vv.vec] >> kAtHeadShift : stat ? c - width : 0;
  A top = lowest<A>();
  for (int i = s; i < j.z; i += 8) top = larger(top, part[int64_t(i) * stride + width + h]);
  red[s][threadIdx.x] = top;
  __syncthreads();
  for (int i = 0; i < 8; ++i) top = larger(top, red[i][threadIdx.x]);
  __syncthreads();
  const A shift = top == lowest<A>() ? A(0) : top;
  A sum = 0, l = 0;
  for (int i = s; i < j.z; i += 8) {
    const A* p = part + int64_t(i) * stride;
    const A f = expo(p[width + h] - shift);
    l += f * p[width + a.heads + h];
    if (value && f != 0) sum += f * p[c];
  }
  red[s][threadIdx.x] = sum;
  red_l[s][threadIdx.x] = l;
  __syncthreads();
  if (s) return;
  for (int i = 1; i < 8; ++i) sum += red[i][threadIdx.x], l += red_l[i][threadIdx.x];
  if (value) reinterpret_cast<R*>(a.out.p)[int64_t(j.x) * a.out.ld + c] = to<R>(l == 0 ? A(0) : sum / l);
  if (stat) static_cast<A*>(a.lse)[int64_t(j.x) * a.heads + h] = loga(l) + shift;
}

// sum of parts: out[row][c] = sum_i part[i * stride + at + c]
template <typename R, typename A>
__global__ void attn_join_sum_kernel(const AtArgs a, const AtRows out, int width, int at, int stride) {
  chain_enter();
  __shared__ A red[8][33];
  const Int4 j = a.joins[blockIdx.y];
  const int c = blockIdx.x * 32 + threadIdx.x, s = threadIdx.y;
  const A* part = static_cast<const A*>(a.part) + int64_t(j.y) * stride + at;
  A sum = 0;
  if (c < width)
    for (int i = s; i < j.z; i += 8) sum += part[int64_t(i) * stride + c];
  red[s][threadIdx.x] = sum;
  __syncthreads();
  if (s || c >= width) return;
  for (int i = 1; i < 8; ++i) sum += red[i][threadIdx.x];
  reinterpret_cast<R*>(out.p)[int64_t(j.x) * out.ld + c] = to<R>(sum);
}

// w' = a w for the edges [e, e + cnt) with their weights in z.
template <typename S, typename A, bool WARP>
__device__ __forceinline__ void scale_rows(const AtArgs& a, const Group<WARP>& g, const Smem<A>& sm, int64_t e, int cnt) {
  with_width<S>(a.vv.vec, [&](auto v) {
    constexpr int V = decltype(v)::value, U = 4;
    const int pieces = a.heads * a.vv.pieces;
    const S* in = reinterpret_cast<const S*>(a.v.p) + e * a.v.ld;
    S* out = reinterpret_cast<S*>(a.out.p) + e * a.out.ld;
    int i = g.t / pieces, p = g.t - i * pieces;
    const int di = g.n / pieces, dp = g.n - di * pieces;
    while (i < cnt) {
      Pack<S, V> y[U];
      int at[U], ap[U];
#pragma unroll
      for (int u = 0; u < U; ++u) {
        at[u] = i;
        ap[u] = p;
        if (i < cnt) y[u].load(in + i * a.v.ld + p * V);
        i += di;
        p += dp;
        if (p >= pieces) p -= pieces, ++i;
      }
#pragma unroll
      for (int u = 0; u < U; ++u) {
        if (at[u] >= cnt) continue;
        const A f = sm.z[at[u] * a.heads + (a.vv.acc[ap[u]] >> kAtHeadShift)];
#pragma unroll
        for (int j = 0; j < V; ++j) y[u].e[j] = to<S>(f == 0 ? A(0) : f * wide(y[u].e[j]));
        y[u].store(out + at[u] * a.out.ld + ap[u] * V);
      }
    }
  });
}

// Statistics of a split row from those of its parts: stat[h] = maximum, stat[heads + h] = sum of exponentials.
template <typename A, bool WARP>
__device__ __forceinline__ void joined_stats(const AtArgs& a, const Group<WARP>& g, const Smem<A>& sm, Int4 join) {
  const A* part = static_cast<const A*>(a.part) + int64_t(join.y) * 2 * a.heads;
  each_head(g, a.heads, [&](const HeadLanes& l) {
    A top = lowest<A>();
    for (int i = l.slot; i < join.z; i += l.slots) top = larger(top, part[int64_t(i) * 2 * a.heads + l.h]);
    top = all_max(l, top);
    const A shift = top == lowest<A>() ? A(0) : top;
    A sum = 0;
    for (int i = l.slot; i < join.z; i += l.slots) {
      const A* p = part + int64_t(i) * 2 * a.heads + l.h;
      sum += expo(p[0] - shift) * p[a.heads];
    }
    sum = all_sum(l, sum);
    if (l.on && l.slot == 0) {
      sm.stat[l.h] = top;
      sm.stat[a.heads + l.h] = sum;
    }
  });
}

// Weights of the edges of a row, and the edges' rows times them.  A row that fits `sub` edges is done at once; a
// longer one writes its logits to alpha and comes back for them; a split one does so in two launches.
template <typename S, typename A, bool WARP>
__global__ void attn_edges_forward_kernel(const AtArgs a) {
  chain_enter();
  const Group<WARP> g;
  const Smem<A> sm(a, g);
  A* alpha = static_cast<A*>(a.alpha);
  const auto weigh = [&](int64_t e, int cnt, bool held) {   // z (held: exponentials) -> weights, alpha and rows
    for (int f = g.t; f < cnt * a.heads; f += g.n) {
      const int i = pair_edge(a, f), h = f - i * a.heads;
      const A l = sm.stat[a.heads + h], top = sm.stat[h];
      A p = held ? sm.z[f] : expo(alpha[e * a.heads + f] - (top == lowest<A>() ? A(0) : top));
      p = p == 0 ? A(0) : p / l;
      sm.z[f] = p;
      alpha[e * a.heads + f] = p;
    }
    g.sync();
    scale_rows<S>(a, g, sm, e, cnt);
  };
  each_item(a, g, [&](const Item& it) {
    if (it.e0 == it.e1) return;
    const bool one = it.index < 0 && it.e1 - it.e0 <= a.sub;
    if (a.phase != kAtSecond) {
      stage<S, A>(g, a.qk, a.heads, reinterpret_cast<const S*>(a.q.p) + it.row * a.q.ld, sm.q);
      for (int64_t e = it.e0; e < it.e1; e += a.sub) {
        const int cnt = static_cast<int>(min(int64_t(a.sub), it.e1 - e));
        load_edges(a, g, sm, e, cnt);
        g.sync();
        logits<S>(a, g, sm, e, cnt);
        g.sync();
        if (!one)
          for (int f = g.t; f < cnt * a.heads; f += g.n) alpha[e * a.heads + f] = sm.z[f];
        softmax_step(a, g, sm, cnt, e == it.e0, !one);
        g.sync();
      }
      if (one) {
        weigh(it.e0, static_cast<int>(it.e1 - it.e0), true);
        return;
      }
      if (it.index >= 0) {
        A* part = static_cast<A*>(a.part) + int64_t(it.index) * 2 * a.heads;
        for (int h = g.t; h < 2 * a.heads; h += g.n) part[h] = sm.stat[h];
        return;
      }
    } else {
      joined_stats(a, g, sm, a.joins[a.items[it.index].w]);
      g.sync();
    }
    for (int64_t e = it.e0; e < it.e1; e += a.sub) {
      weigh(e, static_cast<int>(min(int64_t(a.sub), it.e1 - e)), false);
      g.sync();
    }
  });
}

// ---------------------------------------------------------------------------
// backward
// ---------------------------------------------------------------------------

// dp = <gw', w> of the edges' rows and gw = a gw', for the weights in p.
template <typename S, typename R, typename A, bool WARP>
__device__ __forceinline__ void edge_rows_backward(const AtArgs& a, const Group<WARP>& g, const Smem<A>& sm, int64_t e, int cnt) {
  const int total = cnt * a.heads, team = a.team_vv, lane = g.t & (team - 1), teams = g.n / team;
  with_width<S>(a.vv.vec, [&](auto v) {
    constexpr int V = decltype(v)::value, U = 4;
    const S* w = reinterpret_cast<const S*>(a.v.p) + e * a.v.ld;
    const R* gw2 = reinterpret_cast<const R*>(a.gout.p) + e * a.gout.ld;
    R* gw = reinterpret_cast<R*>(a.gv.p) + e * a.gv.ld;
    for (int base = 0; base < total; base += teams) {
      const int pair = base + g.t / team;
      const bool on = pair < total;
      const int i = pair_edge(a, min(pair, total - 1)), h = min(pair, total - 1) - i * a.heads;
      const A f = sm.p[i * a.heads + h];
      const int* off = a.vv.dot_full + h * a.vv.pieces;
      A sum = 0;
      for (int c = lane; c < a.vv.pieces; c += U * team) {
        Pack<S, V> x[U];
        Pack<R, V> y[U];
        int at[U];
#pragma unroll
        for (int u = 0; u < U; ++u) {
          at[u] = c + u * team < a.vv.pieces && on ? off[c + u * team] : -1;
          if (at[u] >= 0) {
            x[u].load(w + i * a.v.ld + at[u]);
            y[u].load(gw2 + i * a.gout.ld + at[u]);
          }
        }
#pragma unroll
        for (int u = 0; u < U; ++u) {
          if (at[u] < 0) continue;
#pragma unroll
          for (int j = 0; j < V; ++j) {
            const A b = wide(y[u].e[j]);
            sum += b * wide(x[u].e[j]);
            y[u].e[j] = to<R>(f == 0 ? A(0) : f * b);
          }
          y[u].store(gw + i * a.gv.ld + at[u]);
        }
      }
      for (int o = team / 2; o > 0; o /= 2) sum += __shfl_xor_sync(0xffffffffu, sum, o);
      if (lane == 0 && on) sm.z[i * a.heads + h] = f == 0 ? A(0) : sum;
    }
  });
}

// The receivers' kernel: a and ds of every edge, and gq.
template <typename S, typename R, typename A, bool WARP, bool EDGES>
__global__ void attn_receive_kernel(const AtArgs a) {
  chain_enter();
  const Group<WARP> g;
  const Smem<A> sm(a, g);
  A *alpha = static_cast<A*>(a.alpha), *ds = static_cast<A*>(a.ds);
  const A scale = static_cast<A>(a.scale);
  // ds of the edges in z (dp) and p (a), for the sums in stat; gq
  const auto second = [&](const Item& it, int64_t e, int cnt, bool first, bool last) {
    for (int f = g.t; f < cnt * a.heads; f += g.n) {
      const int h = f - pair_edge(a, f) * a.heads;
      const A p = sm.p[f], d = p == 0 ? A(0) : p * (sm.z[f] - sm.stat[h]);
      ds[e * a.heads + f] = d;
      sm.z[f] = d;
    }
    g.sync();
    with_width<S>(a.qk.vec, [&](auto v) {
      constexpr int V = decltype(v)::value;
      accumulate<V>(g, a.heads, cnt, a.heads * a.qk.pieces, 1, a.qk.acc, sm.z, reinterpret_cast<const S*>(a.k.p), a.k.ld, sm.idx, sm.acc,
                    static_cast<const A*>(nullptr), sm.red, first, last, [&](int p, int, const A* r) {
                      if (it.index >= 0) {
                        A* part = static_cast<A*>(a.part) + int64_t(it.index) * a.heads * a.dk;
#pragma unroll
                        for (int j = 0; j < V; ++j) part[p * V + j] = r[j] * scale;
                      } else {
                        Pack<R, V> y;
#pragma unroll
                        for (int j = 0; j < V; ++j) y.e[j] = to<R>(r[j] * scale);
                        y.store(reinterpret_cast<R*>(a.gq.p) + it.row * a.gq.ld + p * V);
                      }
                    });
    });
  };
  each_item(a, g, [&](const Item& it) {
    const bool one = it.index < 0 && it.e1 - it.e0 <= a.sub;
    if (a.phase != kAtSecond) {
      if (!EDGES) {
        stage<S, A>(g, a.qk, a.heads, reinterpret_cast<const S*>(a.q.p) + it.row * a.q.ld, sm.q);
        stage<S, A>(g, a.vv, a.heads, reinterpret_cast<const S*>(a.gout.p) + it.row * a.gout.ld, sm.g);
      }
      int64_t e = it.e0;
      do {
        const int cnt = static_cast<int>(min(int64_t(a.sub), it.e1 - e));
        if (EDGES) {
          for (int i = g.t; i < cnt; i += g.n) sm.idx[i] = a.col[e + i];
          for (int f = g.t; f < cnt * a.heads; f += g.n) sm.p[f] = alpha[e * a.heads + f];
          g.sync();
          edge_rows_backward<S, R>(a, g, sm, e, cnt);
        } else {
          load_edges(a, g, sm, e, cnt);
          g.sync();
          logits<S>(a, g, sm, e, cnt);
          g.sync();
          for (int f = g.t; f < cnt * a.heads; f += g.n) {
            const A z = sm.z[f];
            const A p = z == lowest<A>() ? A(0) : expo(z - static_cast<const A*>(a.lse)[it.row * a.heads + (f - pair_edge(a, f) * a.heads)]);
            sm.p[f] = p;
            alpha[e * a.heads + f] = p;
          }
          dots<S, A>(a, g, a.vv, a.team_vv, cnt, sm.g, reinterpret_cast<const S*>(a.v.p), a.v.ld, sm.idx,
                     [&](int i, int h, A s) { sm.z[i * a.heads + h] = s; });
        }
        g.sync();
        if (!one)
          for (int f = g.t; f < cnt * a.heads; f += g.n) ds[e * a.heads + f] = sm.z[f];
        each_head(g, a.heads, [&](const HeadLanes& l) {
          A sum = 0;
          for (int i = l.slot; i < cnt; i += l.slots) {
            const A p = sm.p[i * a.heads + l.h];
            if (p != 0) sum += p * sm.z[i * a.heads + l.h];
          }
          sum = all_sum(l, sum);
          if (l.on && l.slot == 0) sm.stat[l.h] = (e == it.e0 ? A(0) : sm.stat[l.h]) + sum;
        });
        g.sync();
        e += cnt;
      } while (e < it.e1);
      if (one) {
        second(it, it.e0, static_cast<int>(it.e1 - it.e0), true, true);
        return;
      }
      if (it.index >= 0) {
        A* part = static_cast<A*>(a.part_sum) + int64_t(it.index) * a.heads;
        for (int h = g.t; h < a.heads; h += g.n) part[h] = sm.stat[h];
        return;
      }
    } else {
      const Int4 join = a.joins[a.items[it.index].w];
      each_head(g, a.heads, [&](const HeadLanes& l) {
        A sum = 0;
        for (int i = l.slot; i < join.z; i += l.slots) sum += static_cast<const A*>(a.part_sum)[int64_t(join.y + i) * a.heads + l.h];
        sum = all_sum(l, sum);
        if (l.on && l.slot == 0) sm.stat[l.h] = sum;
      });
      g.sync();
    }
    for (int64_t e = it.e0; e < it.e1; e += a.sub) {
      const int cnt = static_cast<int>(min(int64_t(a.sub), it.e1 - e));
      for (int i = g.t; i < cnt; i += g.n) sm.idx[i] = a.col[e + i];
      for (int f = g.t; f < cnt * a.heads; f += g.n) {
        sm.z[f] = ds[e * a.heads + f];
        sm.p[f] = alpha[e * a.heads + f];
      }
      g.sync();
      second(it, e, cnt, e == it.e0, e + cnt >= it.e1);
      g.sync();
    }
  });
}

// The sources' kernel, over the transpose: gk, and gv where VALUES.
template <typename S, typename R, typename A, bool WARP, bool VALUES>
__global__ void attn_send_kernel(const AtArgs a) {
  chain_enter();
  const Group<WARP> g;
  const Smem<A> sm(a, g);
  const A *alpha = static_cast<const A*>(a.alpha), *ds = static_cast<const A*>(a.ds);
  const A scale = static_cast<A>(a.scale);
  const int wk = a.kv * a.dk, stride = wk + (VALUES ? a.kv * a.dv : 0);
  each_item(a, g, [&](const Item& it) {
    const bool part = it.index >= 0;
    A* to_part = static_cast<A*>(a.part) + int64_t(it.index) * stride;
    int64_t e = it.e0;
    do {
      const int cnt = static_cast<int>(min(int64_t(a.sub), it.e1 - e));
      for (int i = g.t; i < cnt; i += g.n) {
        sm.idx[i] = a.col[e + i];
        sm.bucket[i] = a.eid[e + i];
      }
      g.sync();
      for (int f = g.t; f < cnt * a.heads; f += g.n) {
        const int i = pair_edge(a, f);
        const int64_t at = int64_t(sm.bucket[i]) * a.heads + (f - i * a.heads);
        sm.z[f] = ds[at] * scale;
        if (VALUES) sm.p[f] = alpha[at];
      }
      g.sync();
      const bool first = e == it.e0, last = e + cnt >= it.e1;
      with_width<S>(a.qk.vec, [&](auto v) {
        constexpr int V = decltype(v)::value;
        accumulate<V>(g, a.heads, cnt, a.kv * a.qk.pieces, a.group, a.qk.send, sm.z, reinterpret_cast<const S*>(a.q.p), a.q.ld, sm.idx, sm.acc,
                      static_cast<const A*>(nullptr), sm.red, first, last, [&](int p, int, const A* r) {
                        if (part) {
#pragma unroll
                          for (int j = 0; j < V; ++j) to_part[p * V + j] = r[j];
                        } else {
                          Pack<R, V> y;
#pragma unroll
                          for (int j = 0; j < V; ++j) y.e[j] = to<R>(r[j]);
                          y.store(reinterpret_cast<R*>(a.gk.p) + it.row * a.gk.ld + p * V);
                        }
                      });
      });
      if (VALUES)
        with_width<S>(a.vv.vec, [&](auto v) {
          constexpr int V = decltype(v)::value;
          accumulate<V>(g, a.heads, cnt, a.kv * a.vv.pieces, a.group, a.vv.send, sm.p, reinterpret_cast<const S*>(a.gout.p), a.gout.ld, sm.idx,
                        sm.acc + wk, static_cast<const A*>(nullptr), sm.red, first, last, [&](int p, int, const A* r) {
                          if (part) {
#pragma unroll
                            for (int j = 0; j < V; ++j) to_part[wk + p * V + j] = r[j];
                          } else {
                            Pack<R, V> y;
#pragma unroll
                            for (int j = 0; j < V; ++j) y.e[j] = to<R>(r[j]);
                            y.store(reinterpret_cast<R*>(a.gv.p) + it.row * a.gv.ld + p * V);
                          }
                        });
        });
      e += cnt;
      if (!last) g.sync();
    } while (e < it.e1);
  });
}

// Gradient of the bias table: sums of ds by bucket.  A lane always adds to the same head's column of its warp's
// histogram, one column a lane, so that nothing collides and the order is fixed.
template <typename A>
__global__ void attn_table_kernel(const AtArgs a) {
  chain_enter();
  extern __shared__ __align__(16) char at_smem[];
  const int buckets = a.n_borders + 1, cols = a.hist_cols, lane = threadIdx.x & 31, w = threadIdx.x / 32;
  A* hist = reinterpret_cast<A*>(at_smem) + w * buckets * cols;
  for (int i = lane; i < buckets * cols; i += 32) hist[i] = 0;
  __syncwarp();
  const int slots = a.heads < 32 ? 32 / a.heads : 1;
  const int h0 = a.heads < 32 ? lane % a.heads : lane, s = a.heads < 32 ? lane / a.heads : 0;
  const int64_t warps = int64_t(gridDim.x) * (blockDim.x / 32), first = int64_t(blockIdx.x) * (blockDim.x / 32) + w;
  const A *lengths = static_cast<const A*>(a.lengths), *borders = static_cast<const A*>(a.borders), *ds = static_cast<const A*>(a.ds);
  if (s < slots)
    for (int64_t e = first * slots + s; e < a.n_edges; e += warps * slots) {
      const int b = bucket_of(borders, a.n_borders, lengths[e]);
      for (int h = h0; h < a.heads; h += 32) hist[b * cols + (h - h0) + lane] += ds[e * a.heads + h];
    }
  __syncthreads();
  // columns of a head: lanes h, h + heads, ... of each block of 32, over all warps
  const A* all = reinterpret_cast<const A*>(at_smem);
  for (int i = threadIdx.x; i < buckets * a.heads; i += blockDim.x) {
    const int b = i / a.heads, h = i - b * a.heads;
    double sum = 0;
    for (int q = 0; q < static_cast<int>(blockDim.x) / 32; ++q)
      for (int k = 0; k < slots; ++k) sum += all[(q * buckets + b) * cols + h + k * a.heads];
    if (gridDim.x == 1) static_cast<A*>(a.gtable)[i] = static_cast<A>(sum);
    else static_cast<double*>(a.hist)[int64_t(blockIdx.x) * buckets * a.heads + i] = sum;
  }
}

template <typename A>
__global__ void attn_table_sum_kernel(const AtArgs a, int parts) {
  chain_enter();
  __shared__ double red[8][33];
  const int c = blockIdx.x * 32 + threadIdx.x, s = threadIdx.y, width = (a.n_borders + 1) * a.heads;
  double sum = 0;
  if (c < width)
    for (int i = s; i < parts; i += 8) sum += static_cast<const double*>(a.hist)[int64_t(i) * width + c];
  red[s][threadIdx.x] = sum;
  __syncthreads();
  if (s || c >= width) return;
  for (int i = 1; i < 8; ++i) sum += red[i][threadIdx.x];
  static_cast<A*>(a.gtable)[c] = static_cast<A>(sum);
}

// ---------------------------------------------------------------------------
// launches
// ---------------------------------------------------------------------------
template <typename... P, typename... Args>
cudaError_t at_launch(void (*kernel)(P...), dim3 grid, dim3 block, size_t smem, cudaStream_t st, Args&&... args) {
  if (smem > 48 * 1024 && smem_cap_cached(reinterpret_cast<const void*>(kernel)) < 0) return cudaErrorInvalidValue;
  cudaLaunchAttribute attr;
  attr.id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr.val.programmaticStreamSerializationAllowed = 1;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = grid;
  cfg.blockDim = block;
  cfg.dynamicSmemBytes = smem;
  cfg.stream = st;
  cfg.attrs = &attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, kernel, static_cast<P>(args)...);
}

template <typename... P>
cudaError_t at_run(void (*warp)(P...), void (*cta)(P...), const AtArgs& a, cudaStream_t st) {
  return at_launch(a.warp_rows ? warp : cta, dim3(a.grid), dim3(a.block), a.smem, st, a);
}

}  // namespace

#define CGTP_AT_DEFINE(suffix, S, R, A)                                                                                      \
  cudaError_t at_forward_##suffix(const AtArgs& a, cudaStream_t st) {                                                        \
    return at_run(attn_forward_kernel<S, R, A, true>, attn_forward_kernel<S, R, A, false>, a, st);                           \
  }                                                                                                                          \
  cudaError_t at_edges_forward_##suffix(const AtArgs& a, cudaStream_t st) {                                                  \
    return at_run(attn_edges_forward_kernel<S, A, true>, attn_edges_forward_kernel<S, A, false>, a, st);                     \
  }                                                                                                                          \
  cudaError_t at_receive_##suffix(const AtArgs& a, cudaStream_t st) {                                                        \
    return at_run(attn_receive_kernel<S, R, A, true, false>, attn_receive_kernel<S, R, A, false, false>, a, st);             \
  }                                                                                                                          \
  cudaError_t at_edges_receive_##suffix(const AtArgs& a, cudaStream_t st) {                                                  \
    return at_run(attn_receive_kernel<S, R, A, true, true>, attn_receive_kernel<S, R, A, false, true>, a, st);               \
  }                                                                                                                          \
  cudaError_t at_send_##suffix(const AtArgs& a, bool values, cudaStream_t st) {                                              \
    return values ? at_run(attn_send_kernel<S, R, A, true, true>, attn_send_kernel<S, R, A, false, true>, a, st)             \
                  : at_run(attn_send_kernel<S, R, A, true, false>, attn_send_kernel<S, R, A, false, false>, a, st);          \
  }                                                                                                                          \
  cudaError_t at_join_forward_##suffix(const AtArgs& a, cudaStream_t st) {                                                   \
    const int width = a.heads * a.dv + a.heads;                                                                              \
    return at_launch(attn_join_forward_kernel<R, A>, dim3((width + 31) / 32, a.n_joins), dim3(32, 8), 0, st, a);             \
  }                                                                                                                          \
  cudaError_t at_join_sum_##suffix(const AtArgs& a, const AtRows& out, int width, int at, int stride, cudaStream_t st) {     \
    return at_launch(attn_join_sum_kernel<R, A>, dim3((width + 31) / 32, a.n_joins), dim3(32, 8), 0, st, a, out, width, at,  \
                     stride);                                                                                                \
  }                                                                                                                          \
  cudaError_t at_table_##suffix(const AtArgs& a, cudaStream_t st) {                                                          \
    const int buckets = a.n_borders + 1, width = buckets * a.heads;                                                          \
    cudaError_t e = at_launch(attn_table_kernel<A>, dim3(a.hist_ctas), dim3(32 * a.hist_warps),                              \
                              size_t(a.hist_warps) * buckets * a.hist_cols * sizeof(A), st, a);                              \
    if (e != cudaSuccess || a.hist_ctas == 1) return e;                                                                      \
    return at_launch(attn_table_sum_kernel<A>, dim3((width + 31) / 32), dim3(32, 8), 0, st, a, a.hist_ctas);                 \
  }

}  // namespace cgtp
