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
// Split.  A warp takes a row (or a run of its edges; several warps of a CTA share a row where rows are few) and holds
// `sub` edges at once, so that no barrier stands between the steps of a row.  Its lanes are (edge, head, lane of the
// head): the vectors of a head's queries or results stay in registers while the edges pass, a dot product needs
// the shuffles of one head's lanes only, and every gathered row is read in whole sectors.  The receivers' kernel of
// the backward writes ds and a (edges x heads); the sources' kernel, over the transpose, only gathers and adds.  Rows
// longer than the graph's chunk are cut into items whose partial results another launch joins in a fixed order.
// Edge rows, which are most of their bytes, pass through kernels of their own that know nothing of the graph.
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
  __device__ __forceinline__ void clear() {
#pragma unroll
    for (int i = 0; i < kRaws; ++i) raw[i] = W{};
  }
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

// V numbers of the arithmetic.  Pairs of FP32 numbers are multiplied and added together.
template <typename A, int V>
struct Nums {
  A e[V];
  __device__ __forceinline__ void clear() {
#pragma unroll
    for (int k = 0; k < V; ++k) e[k] = 0;
  }
  __device__ __forceinline__ A get(int k) const { return e[k]; }
  __device__ __forceinline__ void set(int k, A x) { e[k] = x; }
  // += f y; a weight of zero takes nothing, whatever y holds
  __device__ __forceinline__ void add(A f, const Nums& y) {
    if (f != 0) {
#pragma unroll
      for (int k = 0; k < V; ++k) e[k] += f * y.e[k];
    }
  }
  __device__ __forceinline__ void add_product(const Nums& x, const Nums& y) {
#pragma unroll
    for (int k = 0; k < V; ++k) e[k] += x.e[k] * y.e[k];
  }
  __device__ __forceinline__ A total() const {
    A s = e[0];
#pragma unroll
    for (int k = 1; k < V; ++k) s += e[k];
    return s;
  }
};
template <>
struct Nums<float, 4> {
  uint64_t p[2];
  static __device__ __forceinline__ uint64_t pair(float a, float b) {
    uint64_t r;
    asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "f"(a), "f"(b));
    return r;
  }
  __device__ __forceinline__ void clear() { p[0] = p[1] = 0; }
  __device__ __forceinline__ float get(int k) const {
    float a, b;
    asm("mov.b64 {%0, %1}, %2;" : "=f"(a), "=f"(b) : "l"(p[k / 2]));
    return k & 1 ? b : a;
  }
  __device__ __forceinline__ void set(int k, float x) { p[k / 2] = k & 1 ? pair(get(k - 1), x) : pair(x, get(k + 1)); }
  __device__ __forceinline__ void add(float f, const Nums& y) {
    asm("{\n\t.reg .pred q;\n\t.reg .b64 ff;\n\tsetp.neu.f32 q, %2, 0f00000000;\n\tmov.b64 ff, {%2, %2};\n\t"
        "@q fma.rn.f32x2 %0, ff, %3, %0;\n\t@q fma.rn.f32x2 %1, ff, %4, %1;\n\t}"
        : "+l"(p[0]), "+l"(p[1])
        : "f"(f), "l"(y.p[0]), "l"(y.p[1]));
  }
  __device__ __forceinline__ void add_product(const Nums& x, const Nums& y) {
    asm("fma.rn.f32x2 %0, %2, %4, %0;\n\tfma.rn.f32x2 %1, %3, %5, %1;" : "+l"(p[0]), "+l"(p[1]) : "l"(x.p[0]), "l"(x.p[1]), "l"(y.p[0]), "l"(y.p[1]));
  }
  __device__ __forceinline__ float total() const { return (get(0) + get(2)) + (get(1) + get(3)); }
};

template <typename A, typename S, int V>
__device__ __forceinline__ Nums<A, V> widened(const Pack<S, V>& y) {
  Nums<A, V> r;
  if constexpr (std::is_same<A, float>::value && V == 4) {
    r.p[0] = r.pair(wide(y.e[0]), wide(y.e[1]));
    r.p[1] = r.pair(wide(y.e[2]), wide(y.e[3]));
  } else {
#pragma unroll
    for (int k = 0; k < V; ++k) r.e[k] = wide(y.e[k]);
  }
  return r;
}

// Widths of vectors of a storage type: 16 bytes (8 for bfloat16, whose elements cost more to widen than to load), or
// one element.  Rows of edges, which are read in the order of memory, take 16 bytes of bfloat16 too.
template <typename S>
constexpr int kWide = sizeof(S) == 8 ? 2 : 4;
template <typename S, typename F>
__device__ __forceinline__ void with_width(int v, F&& f) {
  if (sizeof(S) == 2 && v == 8) f(std::integral_constant<int, 8>());
  else if (v == kWide<S>) f(std::integral_constant<int, kWide<S>>());
  else f(std::integral_constant<int, 1>());
}

// ---------------------------------------------------------------------------
// the warps of a row
// ---------------------------------------------------------------------------

constexpr unsigned kAll = 0xffffffffu;

// One warp a row, or all warps of the CTA.
struct Team {
  bool one;
  int w, warps, lane;   // this warp among the row's
  __device__ __forceinline__ Team(const AtArgs& a)
      : one(a.one), w(a.one ? 0 : threadIdx.x / 32), warps(a.one ? 1 : blockDim.x / 32), lane(threadIdx.x & 31) {}
  __device__ __forceinline__ void sync() const {
    if (one) __syncwarp();
    else __syncthreads();
  }
  __device__ __forceinline__ int thread() const { return w * 32 + lane; }
  __device__ __forceinline__ int threads() const { return warps * 32; }
};

struct Item {
  int64_t row;
  int64_t e0, e1;   // this warp's edges
  int index;        // item of a split row, or -1
};

// f(item) for every piece of work of this team.  First come the items of split rows, the longest work.
template <typename F>
__device__ __forceinline__ void each_item(const AtArgs& a, const Team& t, F&& f) {
  const int64_t teams = t.one ? int64_t(gridDim.x) * (blockDim.x / 32) : gridDim.x;
  const int64_t first = t.one ? int64_t(blockIdx.x) * (blockDim.x / 32) + threadIdx.x / 32 : blockIdx.x;
  const int64_t total = a.n_items + (a.phase == kAtSecond ? 0 : a.n_rows);
  for (int64_t i = first; i < total; i += teams) {
    Item it;
    if (i < a.n_items) {
      const Int4 v = a.items[i];
      it = {v.x, v.y, v.z, static_cast<int>(i)};
    } else {
      it.row = i - a.n_items;
      it.e0 = a.rowptr[it.row];
      it.e1 = a.rowptr[it.row + 1];
      it.index = -1;
      if (a.n_items && it.e1 - it.e0 > a.chunk) continue;
    }
    if (!t.one) {
      const int64_t b = it.e0, len = it.e1 - b;
      it.e0 = b + len * t.w / t.warps;
      it.e1 = b + len * (t.w + 1) / t.warps;
    }
    f(it);
    t.sync();
  }
}

// pair / heads for pairs below 2^24 (heads <= 64: the error of the multiplier is below 2^-32 a unit)
__device__ __forceinline__ int pair_edge(const AtArgs& a, int pair) {
  return a.heads == 1 ? pair : static_cast<int>(__umulhi(static_cast<unsigned>(pair), a.heads_magic));
}

// This lane's place: lane = (edge slot, unit, lane of the unit); the units are heads, groups of heads or shared heads.
struct Place {
  int x, u, s;
  __device__ __forceinline__ Place(const AtLanes& l) {
    const int lane = threadIdx.x & 31;
    x = lane & ((1 << l.width) - 1);
    u = (lane >> l.width) & ((1 << l.units) - 1);
    s = lane >> (l.width + l.units);
  }
};

// The edges of a run are taken U times the edge slots at a time: the lists of edges and weights are filled up to that
// (with the first edge and zeros), so that the loops need no bounds.
__device__ __forceinline__ int filled(int cnt, int step) { return (cnt + step - 1) & -step; }

// z[i][h] = <x[h], rows[idx(i)][shared head]>.  G heads that share a row's vectors are taken together; CB vectors a
// lane stay in registers while the edges pass, U edges in flight.
template <int V, int CB, int U, int G, typename S, typename A>
__device__ __forceinline__ void dots(const AtArgs& a, const AtTab& tab, int cnt, const S* x, const AtRows& rows, const int* idx, A* z) {
  const AtLanes& l = tab.lanes;
  const Place at(l);
  const int units = a.heads / G, pieces = tab.pieces, slots = 32 >> (l.width + l.units), end = filled(cnt, U * slots);
  for (int ub = 0; ub < units; ub += 32) {
    const int h0 = min(ub + at.u, units - 1) * G;
    const bool writes = at.x == 0 && ub + at.u < units;
    const int* full = tab.dot_full + h0 * pieces;
    const int* shared = tab.dot_kv + (a.group == 1 ? h0 : h0 / a.group) * pieces;
#pragma unroll 1
    for (int c0 = 0; c0 < pieces; c0 += CB << l.width) {
      Nums<A, V> xr[G][CB];
      const char* base[CB];
      bool ok[CB];
      Pack<S, V> y[U][CB];
#pragma unroll
      for (int j = 0; j < CB; ++j) {
        const int c = c0 + (j << l.width) + at.x;
        ok[j] = c < pieces;
        base[j] = rows.p + (ok[j] ? shared[c] : 0) * sizeof(S);
#pragma unroll
        for (int q = 0; q < G; ++q) {
          Pack<S, V> v;
          v.clear();
          if (ok[j]) v.load(x + full[q * pieces + c]);
          xr[q][j] = widened<A>(v);
        }
#pragma unroll
        for (int u = 0; u < U; ++u) y[u][j].clear();   // what lanes without a vector multiply by zero
      }
      const int* ip = idx + at.s;
      A* to_ = z + at.s * a.heads + h0;
#pragma unroll 1
      for (int b = 0; b < end; b += U * slots, ip += U * slots, to_ += U * slots * a.heads) {
#pragma unroll
        for (int u = 0; u < U; ++u) {
          const uint64_t off = uint64_t(static_cast<unsigned>(ip[u * slots])) * rows.ld_bytes;
#pragma unroll
          for (int j = 0; j < CB; ++j)
            if (ok[j]) y[u][j].load(reinterpret_cast<const S*>(base[j] + off));
        }
        A sum[U][G];
#pragma unroll
        for (int u = 0; u < U; ++u) {
          Nums<A, V> s[G];
#pragma unroll
          for (int q = 0; q < G; ++q) s[q].clear();
#pragma unroll
          for (int j = 0; j < CB; ++j) {
            const Nums<A, V> w = widened<A>(y[u][j]);
#pragma unroll
            for (int q = 0; q < G; ++q) s[q].add_product(xr[q][j], w);
          }
#pragma unroll
          for (int q = 0; q < G; ++q) sum[u][q] = s[q].total();
        }
#pragma unroll 1
        for (int o = 1 << l.width >> 1; o > 0; o >>= 1)
#pragma unroll
          for (int u = 0; u < U; ++u)
#pragma unroll
            for (int q = 0; q < G; ++q) sum[u][q] += __shfl_xor_sync(kAll, sum[u][q], o);
        if (writes)
#pragma unroll
          for (int u = 0; u < U; ++u)
#pragma unroll
            for (int q = 0; q < G; ++q) {
              A* r = to_ + u * slots * a.heads + q;
              *r = c0 == 0 ? sum[u][q] : *r + sum[u][q];
            }
      }
    }
  }
  __syncwarp();
}

// Sums over edges: r = sum_i coef[i][h] rows[idx(i)][offset of a vector], plus, where this is not the first part of a run,
// what the parts before left in `keep`, times rescale[head].  emit(head, vector's offset, r) by one lane where this is
// the last part.  SEND: the units are shared heads, whose result sums over the heads of their group; otherwise G heads
// that share a row's vectors are taken together.
template <int V, int CB, int U, int G, bool SEND, typename S, typename A, typename F>
__device__ __forceinline__ void sums(const AtArgs& a, const AtTab& tab, int cnt, A* coef, const AtRows& rows, const int* idx, A* keep,
                                     const A* rescale, bool first, bool last, F&& emit) {
  const AtLanes& l = tab.lanes;
  const Place at(l);
  const int units = SEND ? a.kv : a.heads / G, pieces = tab.pieces, slots = 32 >> (l.width + l.units), end = filled(cnt, U * slots);
  for (int f = cnt * a.heads + (threadIdx.x & 31); f < end * a.heads; f += 32) coef[f] = 0;
  __syncwarp();
  for (int ub = 0; ub < units; ub += 32) {
    const bool on = ub + at.u < units;
    const int unit = min(ub + at.u, units - 1);
#pragma unroll 1
    for (int c0 = 0; c0 < pieces; c0 += CB << l.width) {
      Nums<A, V> acc[G][CB];
#pragma unroll
      for (int q = 0; q < G; ++q)
#pragma unroll
        for (int j = 0; j < CB; ++j) acc[q][j].clear();
#pragma unroll 1
      for (int g = 0; g < (SEND ? a.group : 1); ++g) {
        const int h0 = SEND ? unit * a.group + g : unit * G;
        const int* from = SEND ? tab.dot_full + h0 * pieces : tab.dot_kv + (a.group == 1 ? h0 : h0 / a.group) * pieces;
        const char* base[CB];
        bool ok[CB];
        Pack<S, V> y[U][CB];
#pragma unroll
        for (int j = 0; j < CB; ++j) {
          const int c = c0 + (j << l.width) + at.x;
          ok[j] = c < pieces;
          base[j] = rows.p + (ok[j] ? from[c] : 0) * sizeof(S);
#pragma unroll
          for (int u = 0; u < U; ++u) y[u][j].clear();
        }
        const int* ip = idx + at.s;
        const A* fp = coef + at.s * a.heads + h0;
#pragma unroll 1
        for (int b = 0; b < end; b += U * slots, ip += U * slots, fp += U * slots * a.heads) {
          A f[U][G];
#pragma unroll
          for (int u = 0; u < U; ++u) {
            const uint64_t off = uint64_t(static_cast<unsigned>(ip[u * slots])) * rows.ld_bytes;
#pragma unroll
            for (int j = 0; j < CB; ++j)
              if (ok[j]) y[u][j].load(reinterpret_cast<const S*>(base[j] + off));
#pragma unroll
            for (int q = 0; q < G; ++q) f[u][q] = fp[u * slots * a.heads + q];
          }
#pragma unroll
          for (int u = 0; u < U; ++u)
#pragma unroll
            for (int j = 0; j < CB; ++j) {
              const Nums<A, V> w = widened<A>(y[u][j]);
#pragma unroll
              for (int q = 0; q < G; ++q) acc[q][j].add(f[u][q], w);
            }
        }
      }
#pragma unroll 1
      for (int o = 1 << (l.width + l.units); o < 32; o <<= 1)
#pragma unroll
        for (int q = 0; q < G; ++q)
#pragma unroll
          for (int j = 0; j < CB; ++j)
#pragma unroll
            for (int k = 0; k < V; ++k) acc[q][j].set(k, acc[q][j].get(k) + __shfl_xor_sync(kAll, acc[q][j].get(k), o));
      if (at.s == 0 && on)
#pragma unroll
        for (int j = 0; j < CB; ++j) {
          const int c = c0 + (j << l.width) + at.x;
          if (c >= pieces) continue;
#pragma unroll
          for (int q = 0; q < G; ++q) {
            const int h = SEND ? unit : unit * G + q, place = (SEND ? tab.dot_kv : tab.dot_full)[h * pieces + c];
            A r[V];
#pragma unroll
            for (int k = 0; k < V; ++k) r[k] = acc[q][j].get(k);
            if (!first) {
              const A f = rescale ? rescale[h] : A(1);
#pragma unroll
              for (int k = 0; k < V; ++k) r[k] += f == 0 ? A(0) : keep[place + k] * f;
            }
            if (last) {
              emit(h, place, r);
            } else {
#pragma unroll
              for (int k = 0; k < V; ++k) keep[place + k] = r[k];
            }
          }
        }
    }
  }
  __syncwarp();
}

// CTAs of 256 threads that an SM is to hold: registers bound the edges in flight.
template <int G>
constexpr int kResident = G == 1 ? 3 : 2;

// Vectors of a lane that the loops hold at once, and edges in flight: two of each for queries and keys, whose rows are
// short, and for values what the plan's rows fill best (CB, see attn.cu); single elements four at a time; where four
// heads share a vector one, with four edges.
template <int V, int G>
constexpr int kTurn = G == 4 ? 1 : V == 1 ? 4 : 2;
template <int CB, int G>
constexpr int kFlight = G == 4 ? 4 : CB == 2 ? 2 : 1;

// The heads of a warp's lanes for sums over edges x heads in shared memory: lane = (edge slot, head); lanes beyond the
// last head have no edges.
struct HeadLanes {
  int h, slot, slots, width;
  bool on;   // the lane that writes a head's result
};
template <typename F>
__device__ __forceinline__ void each_head(const AtArgs& a, F&& f) {
  const int lane = threadIdx.x & 31;
  for (int h0 = 0; h0 < a.heads; h0 += 32) {
    HeadLanes l;
    l.width = 1 << a.head_lanes;
    l.slots = 32 >> a.head_lanes;
    l.h = h0 + (lane & (l.width - 1));
    const bool mine = l.h < a.heads;
    l.slot = mine ? lane >> a.head_lanes : 1 << 30;
    l.on = mine && l.slot == 0;
    f(l);
  }
}
template <typename A>
__device__ __forceinline__ A all_max(const HeadLanes& l, A x) {
  for (int o = l.width; o < 32; o *= 2) x = larger(x, __shfl_xor_sync(kAll, x, o));
  return x;
}
template <typename A>
__device__ __forceinline__ A all_sum(const HeadLanes& l, A x) {
  for (int o = l.width; o < 32; o *= 2) x += __shfl_xor_sync(kAll, x, o);
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

// A warp's regions of shared memory
template <typename A>
struct Smem {
  A *z, *p, *stat, *acc;
  int *idx, *bucket;
  __device__ __forceinline__ Smem(const AtArgs& a, int warp) {
    extern __shared__ __align__(16) char at_smem[];
    char* s = at_smem + warp * a.warp_smem;
    z = reinterpret_cast<A*>(s);
    p = reinterpret_cast<A*>(s + a.at_p);
    idx = reinterpret_cast<int*>(s + a.at_idx);
    bucket = idx + a.sub + a.pad;
    stat = reinterpret_cast<A*>(s + a.at_stat);
    acc = reinterpret_cast<A*>(s + a.at_acc);
  }
};

// Ends of the edges [e, e + cnt), filled up to what the loops take at a time.
template <typename A>
__device__ __forceinline__ void load_ends(const AtArgs& a, const Smem<A>& sm, int64_t e, int cnt) {
  if (cnt == 0) return;
  for (int i = threadIdx.x & 31; i < cnt + a.pad; i += 32) sm.idx[i] = a.col[e + (i < cnt ? i : 0)];
}

// Inner products of the queries of `row` and the keys of the edges [e, e + cnt), into z.
template <int QV, int G, typename S, typename A>
__device__ __forceinline__ void products(const AtArgs& a, const Smem<A>& sm, int64_t row, int64_t e, int cnt) {
  load_ends(a, sm, e, cnt);
  if (a.table)
    for (int i = threadIdx.x & 31; i < cnt; i += 32)
      sm.bucket[i] = bucket_of(static_cast<const A*>(a.borders), a.n_borders, static_cast<const A*>(a.lengths)[e + i]);
  __syncwarp();
  constexpr int CB = kTurn<QV, G>;
  dots<QV, CB, kFlight<CB, G>, G>(a, a.qk, cnt, reinterpret_cast<const S*>(a.q.p) + row * a.q.ld, a.k, sm.idx, sm.z);
}

// The logit of edge e + i and head h from its inner product.
template <typename A>
__device__ __forceinline__ A logit(const AtArgs& a, const Smem<A>& sm, int64_t e, int i, int h) {
  A b = 0;
  if (a.table) b = static_cast<const A*>(a.table)[sm.bucket[i] * a.heads + h];
  if (a.bias) b += static_cast<const A*>(a.bias)[(e + i) * a.heads + h];
  return b == lowest<A>() ? b : sm.z[i * a.heads + h] * static_cast<A>(a.scale) + b;
}

// ---------------------------------------------------------------------------
// forward
// ---------------------------------------------------------------------------

// Turns the products in z into logits and, unless keep_z, those into exp(z - maximum), with the running maximum (stat[h])
// and sum of exponentials (stat[heads + h]); stat[2 heads + h] = factor of what was summed before.
template <typename A>
__device__ __forceinline__ void softmax_step(const AtArgs& a, const Smem<A>& sm, int64_t e, int cnt, bool first, bool keep_z) {
  each_head(a, [&](const HeadLanes& l) {
    A top = lowest<A>();
    for (int i = l.slot; i < cnt; i += l.slots) {
      const A z = logit(a, sm, e, i, l.h);
      sm.z[i * a.heads + l.h] = z;
      top = larger(top, z);
    }
    top = all_max(l, top);
    const A before = first || l.h >= a.heads ? lowest<A>() : sm.stat[l.h];
    top = larger(top, before);
    const A shift = top == lowest<A>() ? A(0) : top;
    A sum = 0;
    for (int i = l.slot; i < cnt; i += l.slots) {
      const A p = expo(sm.z[i * a.heads + l.h] - shift);
      sum += p;
      if (!keep_z) sm.z[i * a.heads + l.h] = p;
    }
    sum = all_sum(l, sum);
    __syncwarp();
    if (l.on) {
      const A f = first ? A(0) : expo(before - shift);
      sm.stat[l.h] = top;
      sm.stat[a.heads + l.h] = (first ? A(0) : sm.stat[a.heads + l.h] * f) + sum;
      sm.stat[2 * a.heads + l.h] = f;
    }
  });
  __syncwarp();
}

// Joins the statistics of a row's warps: stat of the first warp = maximum, sum; factor[w][h] (stat[2 heads + h] of warp
// w) = exp(its maximum - the row's).
template <typename A>
__device__ __forceinline__ void join_warps(const AtArgs& a, const Team& t) {
  const Smem<A> one(a, 0);
  __syncthreads();
  for (int h = t.thread(); h < a.heads; h += t.threads()) {
    A top = lowest<A>();
    for (int w = 0; w < t.warps; ++w) top = larger(top, Smem<A>(a, w).stat[h]);
    const A shift = top == lowest<A>() ? A(0) : top;
    A sum = 0;
    for (int w = 0; w < t.warps; ++w) {
      const Smem<A> sm(a, w);
      const A f = expo(sm.stat[h] - shift);
      sm.stat[2 * a.heads + h] = f;
      sum += sm.stat[a.heads + h] * f;
    }
    one.stat[h] = top;
    one.stat[a.heads + h] = sum;
  }
  __syncthreads();
}

template <typename S, typename R, typename A, int QV, int VV, int G, int CB>
__global__ void __launch_bounds__(256, kResident<G>) attn_forward_kernel(const AtArgs a) {
  chain_enter();
  const Team t(a);
  const Smem<A> sm(a, threadIdx.x / 32);
  const int width = a.heads * a.dv;
  each_item(a, t, [&](const Item& it) {
    const bool part = it.index >= 0;
    A* to_part = static_cast<A*>(a.part) + int64_t(it.index) * (width + 2 * a.heads);
    R* out = reinterpret_cast<R*>(a.out.p) + it.row * a.out.ld;
    int64_t e = it.e0;
    do {
      const int cnt = static_cast<int>(min(int64_t(a.sub), it.e1 - e));
      products<QV, G, S>(a, sm, it.row, e, cnt);
      softmax_step(a, sm, e, cnt, e == it.e0, false);
      const bool last = e + cnt >= it.e1;
      sums<VV, CB, kFlight<CB, G>, G, false, S>(
          a, a.vv, cnt, sm.z, a.v, sm.idx, sm.acc, sm.stat + 2 * a.heads, e == it.e0, t.one && last,
                  [&](int h, int at, const A* r) {
                    constexpr int V = VV;
                    if (part) {
#pragma unroll
                      for (int k = 0; k < V; ++k) to_part[at + k] = r[k];
                    } else {
                      const A l = sm.stat[a.heads + h], f = l == 0 ? A(0) : A(1) / l;
                      Pack<R, V> y;
#pragma unroll
                      for (int k = 0; k < V; ++k) y.e[k] = to<R>(r[k] * f);
                      y.store(out + at);
                    }
                  });
      e += cnt;
    } while (e < it.e1);
    const Smem<A> one(a, t.one ? threadIdx.x / 32 : 0);
    if (!t.one) {
      join_warps<A>(a, t);
      for (int c = t.thread(); c < width; c += t.threads()) {
        const int h = a.vv.acc[c / a.vv.vec] >> kAtHeadShift;
        A r = 0;
        for (int w = 0; w < t.warps; ++w) {
          const Smem<A> other(a, w);
          const A f = other.stat[2 * a.heads + h];
          if (f != 0) r += f * other.acc[c];
        }
        const A l = one.stat[a.heads + h];
        if (part) to_part[c] = r;
        else out[c] = to<R>(l == 0 ? A(0) : r / l);
      }
    }
    for (int h = t.thread(); h < a.heads; h += t.threads()) {
      const A top = one.stat[h], l = one.stat[a.heads + h];
      if (part) {
        to_part[width + h] = top;
        to_part[width + a.heads + h] = l;
      } else {
        static_cast<A*>(a.lse)[it.row * a.heads + h] = loga(l) + (top == lowest<A>() ? A(0) : top);
      }
    }
  });
}

// Joins the parts of a split row: grid (rows, columns / 32); 8 streams of parts a column.
template <typename R, typename A>
__global__ void attn_join_forward_kernel(const AtArgs a) {
  chain_enter();
  __shared__ A red[8][33], red_l[8][33];
  const Int4 j = a.joins[blockIdx.x];
  const int width = a.heads * a.dv, stride = width + 2 * a.heads;
  const int c = blockIdx.y * 32 + threadIdx.x, s = threadIdx.y;
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
  const Int4 j = a.joins[blockIdx.x];
  const int c = blockIdx.y * 32 + threadIdx.x, s = threadIdx.y;
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

// Weights of the edges of a row.  A run of edges that fits `sub` is done at once; a longer one writes its logits to alpha
// and comes back for them; the items of a split row do so in two launches.
template <typename S, typename A, int QV, int G>
__global__ void __launch_bounds__(256, kResident<G>) attn_weights_kernel(const AtArgs a) {
  chain_enter();
  const Team t(a);
  const Smem<A> sm(a, threadIdx.x / 32), one(a, t.one ? threadIdx.x / 32 : 0);
  A* alpha = static_cast<A*>(a.alpha);
  each_item(a, t, [&](const Item& it) {
    const bool held = t.one && it.index < 0 && it.e1 - it.e0 <= a.sub;
    if (a.phase != kAtSecond) {
      int64_t e = it.e0;
      do {
        const int cnt = static_cast<int>(min(int64_t(a.sub), it.e1 - e));
        products<QV, G, S>(a, sm, it.row, e, cnt);
        softmax_step(a, sm, e, cnt, e == it.e0, !held);
        if (!held)
          for (int f = t.lane; f < cnt * a.heads; f += 32) alpha[e * a.heads + f] = sm.z[f];
        __syncwarp();
        e += cnt;
      } while (e < it.e1);
      if (!t.one) join_warps<A>(a, t);
      if (it.index >= 0) {
        A* part = static_cast<A*>(a.part) + int64_t(it.index) * 2 * a.heads;
        for (int h = t.thread(); h < 2 * a.heads; h += t.threads()) part[h] = one.stat[h];
        return;
      }
    } else {
      // statistics of the row from those of its items, by every warp for itself
      const Int4 join = a.joins[a.items[it.index].w];
      const A* part = static_cast<const A*>(a.part) + int64_t(join.y) * 2 * a.heads;
      each_head(a, [&](const HeadLanes& l) {
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
        if (l.on) {
          sm.stat[l.h] = top;
          sm.stat[a.heads + l.h] = sum;
        }
      });
      __syncwarp();
    }
    const A* stat = a.phase == kAtSecond ? sm.stat : one.stat;
    const int64_t base = it.e0 * a.heads;
    const int count = static_cast<int>(it.e1 - it.e0) * a.heads;   // no run is longer than the graph's chunk
    for (int f = t.lane; f < count; f += 32) {
      const int h = f - pair_edge(a, f) * a.heads;
      const A l = stat[a.heads + h], top = stat[h];
      const A p = held ? sm.z[f] : expo(alpha[base + f] - (top == lowest<A>() ? A(0) : top));
      alpha[base + f] = p == 0 ? A(0) : p / l;
    }
  });
}

// w' = a w: vectors of all rows in the order of memory, four a thread and turn.
template <typename S, typename A>
__global__ void __launch_bounds__(256) attn_scale_rows_kernel(const AtArgs a) {
  chain_enter();
  with_width<S>(a.vv.vec, [&](auto v) {
    constexpr int V = decltype(v)::value, U = 4;
    const int pieces = a.heads * a.vv.pieces;
    const A* alpha = static_cast<const A*>(a.alpha);
    const S* in = reinterpret_cast<const S*>(a.v.p);
    S* out = reinterpret_cast<S*>(a.out.p);
    // place of this CTA's first vector, and the distance to its next
    const int64_t first = int64_t(blockIdx.x) * (256 * U), step = int64_t(gridDim.x) * (256 * U);
    int64_t e0 = first / pieces;
    const int64_t de = step / pieces;
    int p0 = static_cast<int>(first - e0 * pieces);
    const int dp = static_cast<int>(step - de * pieces);
    for (; e0 < a.n_edges; e0 += de, p0 += dp, e0 += p0 >= pieces, p0 -= p0 >= pieces ? pieces : 0) {
      Pack<S, V> y[U];
      int64_t e[U];
      int p[U];
      A f[U];
#pragma unroll
      for (int u = 0; u < U; ++u) {
        const unsigned r = p0 + u * 256 + threadIdx.x;   // below 8192 + 1024: the multiplier's error stays below one
        const int i = pieces == 1 ? r : static_cast<int>(__umulhi(r, a.pieces_magic));
        e[u] = e0 + i;
        p[u] = r - i * pieces;
        if (e[u] < a.n_edges) {
          y[u].load(in + e[u] * a.v.ld + p[u] * V);
          f[u] = alpha[e[u] * a.heads + (a.vv.acc[p[u]] >> kAtHeadShift)];
        }
      }
#pragma unroll
      for (int u = 0; u < U; ++u) {
        if (e[u] >= a.n_edges) continue;
#pragma unroll
        for (int k = 0; k < V; ++k) y[u].e[k] = to<S>(f[u] == 0 ? A(0) : f[u] * wide(y[u].e[k]));
        y[u].store(out + e[u] * a.out.ld + p[u] * V);
      }
    }
  });
}

// ---------------------------------------------------------------------------
// backward
// ---------------------------------------------------------------------------

// gw = a gw' and dp = <gw', w> (into ds): a warp takes the heads of one or more edges at a time.
template <typename S, typename A>
__global__ void __launch_bounds__(256) attn_edge_rows_backward_kernel(const AtArgs a) {
  chain_enter();
  const A* alpha = static_cast<const A*>(a.alpha);
  A* dp = static_cast<A*>(a.ds);
  with_width<S>(a.vv.vec, [&](auto v) {
    constexpr int V = decltype(v)::value, U = 4;
    const int pieces = a.vv.pieces;
    const Place l(a.vv.lanes);
    const int width = 1 << a.vv.lanes.width, slots = 32 >> (a.vv.lanes.width + a.vv.lanes.units);
    const int64_t step = int64_t(gridDim.x) * (blockDim.x / 32) * slots;
    for (int64_t b = (int64_t(blockIdx.x) * (blockDim.x / 32) + threadIdx.x / 32) * slots; b < a.n_edges; b += step) {
      const int64_t e = min(b + l.s, a.n_edges - 1);
      const S* w = reinterpret_cast<const S*>(a.v.p) + e * a.v.ld;
      const A* g = reinterpret_cast<const A*>(a.gout.p) + e * a.gout.ld;
      A* gw = reinterpret_cast<A*>(a.gv.p) + e * a.gv.ld;
      for (int ub = 0; ub < a.heads; ub += 32) {
        const bool on = ub + l.u < a.heads && b + l.s < a.n_edges;
        const int h = min(ub + l.u, a.heads - 1);
        const A f = alpha[e * a.heads + h];
        const int* off = a.vv.dot_full + h * pieces;
        A sum = 0;
        for (int c = l.x; c < pieces; c += U * width) {
          Pack<S, V> x[U];
          Pack<A, V> y[U];
          int at[U];
#pragma unroll
          for (int u = 0; u < U; ++u) {
            at[u] = c + u * width < pieces && on ? off[c + u * width] : -1;
            if (at[u] >= 0) {
              x[u].load(w + at[u]);
              y[u].load(g + at[u]);
            }
          }
#pragma unroll
          for (int u = 0; u < U; ++u) {
            if (at[u] < 0) continue;
#pragma unroll
            for (int k = 0; k < V; ++k) {
              const A d = y[u].e[k];
              sum += d * wide(x[u].e[k]);
              y[u].e[k] = f == 0 ? A(0) : f * d;
            }
            y[u].store(gw + at[u]);
          }
        }
        for (int o = width / 2; o > 0; o /= 2) sum += __shfl_xor_sync(kAll, sum, o);
        if (l.x == 0 && on) dp[e * a.heads + h] = f == 0 ? A(0) : sum;
      }
    }
  });
}

// What the receivers' kernel leaves for the sources': ds and a of every edge and head.
template <typename A>
struct alignas(2 * sizeof(A)) Pair {
  A ds, p;
};

// The receivers' kernel: ds of every edge, and gq.  EDGES: dp comes in ds and a in alpha; otherwise both are
// computed here.
template <typename S, typename R, typename A, int QV, int VV, int G, int CB, bool EDGES>
__global__ void __launch_bounds__(256, kResident<G>) attn_receive_kernel(const AtArgs a) {
  chain_enter();
  const Team t(a);
  const Smem<A> sm(a, threadIdx.x / 32);
  const A scale = static_cast<A>(a.scale);
  Pair<A>* pairs = static_cast<Pair<A>*>(a.pairs);
  const int width = a.heads * a.dk;
  // dp and a of the edges [e, e + cnt) into z and p: from memory where they are there
  const auto fetch = [&](int64_t e, int cnt) {
    load_ends(a, sm, e, cnt);
    for (int f = t.lane; f < cnt * a.heads; f += 32) {
      if (EDGES) {
        sm.z[f] = static_cast<const A*>(a.ds)[e * a.heads + f];
        sm.p[f] = static_cast<const A*>(a.alpha)[e * a.heads + f];
      } else {
        const Pair<A> x = pairs[e * a.heads + f];
        sm.z[f] = x.ds;
        sm.p[f] = x.p;
      }
    }
    __syncwarp();
  };
  each_item(a, t, [&](const Item& it) {
    const bool held = it.e1 - it.e0 <= a.sub && a.phase != kAtSecond;   // z, p and idx hold the whole run
    if (a.phase != kAtSecond) {
      int64_t e = it.e0;
      do {
        const int cnt = static_cast<int>(min(int64_t(a.sub), it.e1 - e));
        if (EDGES) {
          fetch(e, cnt);
        } else {
          products<QV, G, S>(a, sm, it.row, e, cnt);
          const A* lse = static_cast<const A*>(a.lse) + it.row * a.heads;
          for (int f = t.lane; f < cnt * a.heads; f += 32) {
            const int i = pair_edge(a, f), h = f - i * a.heads;
            const A z = logit(a, sm, e, i, h);
            sm.p[f] = z == lowest<A>() ? A(0) : expo(z - lse[h]);
          }
          __syncwarp();
          dots<VV, CB, kFlight<CB, G>, G>(a, a.vv, cnt, reinterpret_cast<const S*>(a.gout.p) + it.row * a.gout.ld, a.v, sm.idx, sm.z);
          if (!held || it.index >= 0)
            for (int f = t.lane; f < cnt * a.heads; f += 32) pairs[e * a.heads + f] = {sm.z[f], sm.p[f]};
        }
        each_head(a, [&](const HeadLanes& l) {
          A sum = 0;
          for (int i = l.slot; i < cnt; i += l.slots) {
            const A p = sm.p[i * a.heads + l.h];
            if (p != 0) sum += p * sm.z[i * a.heads + l.h];
          }
          sum = all_sum(l, sum);
          if (l.on) sm.stat[l.h] = (e == it.e0 ? A(0) : sm.stat[l.h]) + sum;
        });
        __syncwarp();
        e += cnt;
      } while (e < it.e1);
      if (!t.one) {
        __syncthreads();
        A total[2] = {0, 0};   // heads <= 64, at least 32 threads
        for (int j = 0; j < 2; ++j)
          if (t.thread() + j * t.threads() < a.heads)
            for (int w = 0; w < t.warps; ++w) total[j] += Smem<A>(a, w).stat[t.thread() + j * t.threads()];
        __syncthreads();
        for (int j = 0; j < 2; ++j)
          if (t.thread() + j * t.threads() < a.heads)
            for (int w = 0; w < t.warps; ++w) Smem<A>(a, w).stat[t.thread() + j * t.threads()] = total[j];
        __syncthreads();
      }
      if (it.index >= 0) {
        A* part = static_cast<A*>(a.part_sum) + int64_t(it.index) * a.heads;
        for (int h = t.thread(); h < a.heads; h += t.threads()) part[h] = sm.stat[h];
        return;
      }
    } else {
      const Int4 join = a.joins[a.items[it.index].w];
      each_head(a, [&](const HeadLanes& l) {
        A sum = 0;
        for (int i = l.slot; i < join.z; i += l.slots) sum += static_cast<const A*>(a.part_sum)[int64_t(join.y + i) * a.heads + l.h];
        sum = all_sum(l, sum);
        if (l.on) sm.stat[l.h] = sum;
      });
      __syncwarp();
    }
    const auto finish = [&](int at, A x) {   // one element of gq
      if (it.index >= 0) static_cast<A*>(a.part)[int64_t(it.index) * width + at] = x * scale;
      else (reinterpret_cast<R*>(a.gq.p) + it.row * a.gq.ld)[at] = to<R>(x * scale);
    };
    int64_t e = it.e0;
    do {
      const int cnt = static_cast<int>(min(int64_t(a.sub), it.e1 - e));
      if (!held) fetch(e, cnt);
      for (int f = t.lane; f < cnt * a.heads; f += 32) {
        const int h = f - pair_edge(a, f) * a.heads;
        const A p = sm.p[f], d = p == 0 ? A(0) : p * (sm.z[f] - sm.stat[h]);
        sm.z[f] = d;
        if (!EDGES) pairs[e * a.heads + f] = {d, p};
        if (a.ds) static_cast<A*>(a.ds)[e * a.heads + f] = d;
      }
      __syncwarp();
      const bool last = e + cnt >= it.e1;
      constexpr int QB = kTurn<QV, G>;
      sums<QV, QB, kFlight<QB, G>, G, false, S>(
          a, a.qk, cnt, sm.z, a.k, sm.idx, sm.acc, static_cast<const A*>(nullptr), e == it.e0, t.one && last, [&](int, int at, const A* r) {
                    constexpr int V = QV;
                    if (it.index >= 0) {
#pragma unroll
                      for (int k = 0; k < V; ++k) finish(at + k, r[k]);
                    } else {
                      Pack<R, V> y;
#pragma unroll
                      for (int k = 0; k < V; ++k) y.e[k] = to<R>(r[k] * scale);
                      y.store(reinterpret_cast<R*>(a.gq.p) + it.row * a.gq.ld + at);
                    }
                  });
      __syncwarp();
      e += cnt;
    } while (e < it.e1);
    if (!t.one) {
      __syncthreads();
      for (int c = t.thread(); c < width; c += t.threads()) {
        A r = 0;
        for (int w = 0; w < t.warps; ++w) r += Smem<A>(a, w).acc[c];
        finish(c, r);
      }
    }
  });
}

// The sources' kernel, over the transpose: gk, and gv where VALUES.
template <typename S, typename R, typename A, int QV, int VV, int CB, bool VALUES>
__global__ void __launch_bounds__(256, kResident<1>) attn_send_kernel(const AtArgs a) {
  chain_enter();
  const Team t(a);
  const Smem<A> sm(a, threadIdx.x / 32);
  const A scale = static_cast<A>(a.scale);
  const int wk = a.kv * a.dk, stride = wk + (VALUES ? a.kv * a.dv : 0);
  each_item(a, t, [&](const Item& it) {
    const bool part = it.index >= 0;
    A* to_part = static_cast<A*>(a.part) + int64_t(it.index) * stride;
    const auto finish = [&](int at, A x) {   // element `at` of (gk, gv)
      if (part) to_part[at] = x;
      else if (at < wk) (reinterpret_cast<R*>(a.gk.p) + it.row * a.gk.ld)[at] = to<R>(x);
      else (reinterpret_cast<R*>(a.gv.p) + it.row * a.gv.ld)[at - wk] = to<R>(x);
    };
    int64_t e = it.e0;
    do {
      const int cnt = static_cast<int>(min(int64_t(a.sub), it.e1 - e));
      load_ends(a, sm, e, cnt);
      for (int i = t.lane; i < cnt; i += 32) sm.bucket[i] = a.eid[e + i];
      __syncwarp();
      for (int f = t.lane; f < cnt * a.heads; f += 32) {
        const int i = pair_edge(a, f);
        const int64_t at = int64_t(sm.bucket[i]) * a.heads + (f - i * a.heads);
        if (VALUES) {
          const Pair<A> x = static_cast<const Pair<A>*>(a.pairs)[at];
          sm.z[f] = x.ds * scale;
          sm.p[f] = x.p;
        } else {
          sm.z[f] = static_cast<const A*>(a.ds)[at] * scale;
        }
      }
      __syncwarp();
      const bool first = e == it.e0, last = t.one && e + cnt >= it.e1;
      const auto store = [&](auto v, R* row, int from) {
        return [=](int, int at, const A* r) {
          constexpr int V = decltype(v)::value;
          if (part) {
#pragma unroll
            for (int k = 0; k < V; ++k) to_part[from + at + k] = r[k];
          } else {
            Pack<R, V> y;
#pragma unroll
            for (int k = 0; k < V; ++k) y.e[k] = to<R>(r[k]);
            y.store(row + at);
          }
        };
      };
      constexpr int QB = kTurn<QV, 1>;
      const A* none = nullptr;
      sums<QV, QB, kFlight<QB, 1>, 1, true, S>(a, a.qk, cnt, sm.z, a.q, sm.idx, sm.acc, none, first, last,
                                               store(std::integral_constant<int, QV>(), reinterpret_cast<R*>(a.gk.p) + it.row * a.gk.ld, 0));
      if (VALUES)
        sums<VV, CB, kFlight<CB, 1>, 1, true, S>(a, a.vv, cnt, sm.p, a.gout, sm.idx, sm.acc + wk, none, first, last,
                                                 store(std::integral_constant<int, VV>(), reinterpret_cast<R*>(a.gv.p) + it.row * a.gv.ld, wk));
      __syncwarp();
      e += cnt;
    } while (e < it.e1);
    if (!t.one) {
      __syncthreads();
      for (int c = t.thread(); c < stride; c += t.threads()) {
        A r = 0;
        for (int w = 0; w < t.warps; ++w) r += Smem<A>(a, w).acc[c];
        finish(c, r);
      }
    }
  });
}

// Gradient of the bias table: sums of ds by bucket.  A lane always adds to the same head's column of its warp's
// histogram, one column a lane, so that nothing collides and the order is fixed.  ds lies ds_step values apart.
template <typename A>
__global__ void attn_table_kernel(const AtArgs a) {
  chain_enter();
  extern __shared__ __align__(16) char at_smem[];
  const int buckets = a.n_borders + 1, cols = a.hist_cols, lane = threadIdx.x & 31, w = threadIdx.x / 32, warps_here = blockDim.x / 32;
  A* all = reinterpret_cast<A*>(at_smem);
  A* hist = all + w * buckets * cols;
  A* borders = all + warps_here * buckets * cols;
  for (int i = lane; i < buckets * cols; i += 32) hist[i] = 0;
  for (int i = threadIdx.x; i < a.n_borders; i += blockDim.x) borders[i] = static_cast<const A*>(a.borders)[i];
  __syncthreads();
  const int slots = a.heads < 32 ? 32 / a.heads : 1;
  const int h0 = a.heads < 32 ? lane % a.heads : lane, s = a.heads < 32 ? lane / a.heads : 0;
  const int64_t step = int64_t(gridDim.x) * warps_here * slots, first = (int64_t(blockIdx.x) * warps_here + w) * slots + s;
  const A *lengths = static_cast<const A*>(a.lengths), *ds = static_cast<const A*>(a.hist_from);
  constexpr int U = 4;
  if (s < slots)
    for (int64_t e = first; e < a.n_edges; e += U * step) {
      A r[U], d[U][2];
#pragma unroll
      for (int u = 0; u < U; ++u) {
        const int64_t at = e + u * step;
        r[u] = 0;
        d[u][0] = d[u][1] = 0;
        if (at < a.n_edges) {
          r[u] = lengths[at];
          if (h0 < a.heads) d[u][0] = ds[(at * a.heads + h0) * a.hist_step];
          if (h0 + 32 < a.heads) d[u][1] = ds[(at * a.heads + h0 + 32) * a.hist_step];
        }
      }
#pragma unroll
      for (int u = 0; u < U; ++u) {
        if (e + u * step >= a.n_edges) continue;
        A* at = hist + bucket_of(borders, a.n_borders, r[u]) * cols + lane;
        at[0] += d[u][0];
        if (cols > 32) at[32] += d[u][1];
      }
    }
  __syncthreads();
  // columns of a head: lanes h, h + heads, ... of each block of 32, over all warps
  for (int i = threadIdx.x; i < buckets * a.heads; i += blockDim.x) {
    const int b = i / a.heads, h = i - b * a.heads;
    double sum = 0;
    for (int q = 0; q < warps_here; ++q)
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
cudaError_t at_run(void (*kernel)(P...), const AtArgs& a, cudaStream_t st) {
  return at_launch(kernel, dim3(a.grid), dim3(a.block), a.smem, st, a);
}

}  // namespace

// kernel(QV, VV, G, CB) for the call's vectors
template <typename S, typename F>
auto at_variant(const AtArgs& a, F&& f) {
  using std::integral_constant;
  constexpr int W = kWide<S>;
  const integral_constant<int, 1> one{};
  const integral_constant<int, W> w{};
  const integral_constant<int, 2> two{};
  const integral_constant<int, 4> four{};
  const integral_constant<int, 5> five{};
  if (a.four) return f(w, w, four, one);
  if (a.vv.vec == 1) return a.qk.vec == 1 ? f(one, one, one, four) : f(w, one, one, four);
  if (a.qk.vec == 1) return a.vv.turn == 2 ? f(one, w, one, two) : a.vv.turn == 4 ? f(one, w, one, four) : f(one, w, one, five);
  return a.vv.turn == 2 ? f(w, w, one, two) : a.vv.turn == 4 ? f(w, w, one, four) : f(w, w, one, five);
}

#define CGTP_AT_FORWARD(suffix, S, R, A)                                                                                     \
  cudaError_t at_forward_##suffix(const AtArgs& a, cudaStream_t st) {                                                        \
    return at_variant<S>(a, [&](auto qv, auto vv, auto g, auto cb) {                                                         \
      return at_run(attn_forward_kernel<S, R, A, decltype(qv)::value, decltype(vv)::value, decltype(g)::value, decltype(cb)::value>, a, st); \
    });                                                                                                                      \
  }                                                                                                                          \
  cudaError_t at_weights_##suffix(const AtArgs& a, cudaStream_t st) {                                                        \
    constexpr int W = kWide<S>;                                                                                              \
    return at_run(a.four ? attn_weights_kernel<S, A, W, 4> : a.qk.vec == 1 ? attn_weights_kernel<S, A, 1, 1> : attn_weights_kernel<S, A, W, 1>, a, st); \
  }                                                                                                                          \
  cudaError_t at_scale_rows_##suffix(const AtArgs& a, cudaStream_t st) {                                                     \
    return at_launch(attn_scale_rows_kernel<S, A>, dim3(a.grid), dim3(256), 0, st, a);                                       \
  }                                                                                                                          \
  cudaError_t at_join_forward_##suffix(const AtArgs& a, cudaStream_t st) {                                                   \
    const int width = a.heads * a.dv + a.heads;                                                                              \
    return at_launch(attn_join_forward_kernel<R, A>, dim3(a.n_joins, (width + 31) / 32), dim3(32, 8), 0, st, a);             \
  }

#define CGTP_AT_BACKWARD(suffix, S, R, A)                                                                                     \
  cudaError_t at_edge_rows_##suffix(const AtArgs& a, cudaStream_t st) {                                                      \
    return at_launch(attn_edge_rows_backward_kernel<S, A>, dim3(a.grid), dim3(256), 0, st, a);                               \
  }                                                                                                                          \
  cudaError_t at_receive_##suffix(const AtArgs& a, bool edges, cudaStream_t st) {                                            \
    constexpr int W = kWide<S>;                                                                                              \
    if (edges)                                                                                                               \
      return at_run(a.four             ? attn_receive_kernel<S, R, A, W, 1, 4, 1, true>                                      \
                    : a.qk.vec == 1 ? attn_receive_kernel<S, R, A, 1, 1, 1, 1, true>                                         \
                                       : attn_receive_kernel<S, R, A, W, 1, 1, 1, true>,                                     \
                    a, st);                                                                                                  \
    return at_variant<S>(a, [&](auto qv, auto vv, auto g, auto cb) {                                                         \
      return at_run(attn_receive_kernel<S, R, A, decltype(qv)::value, decltype(vv)::value, decltype(g)::value, decltype(cb)::value, false>, a, st); \
    });                                                                                                                      \
  }                                                                                                                          \
  cudaError_t at_send_##suffix(const AtArgs& a, bool values, cudaStream_t st) {                                              \
    constexpr int W = kWide<S>;                                                                                              \
    if (!values) return at_run(a.qk.vec > 1 ? attn_send_kernel<S, R, A, W, 1, 1, false> : attn_send_kernel<S, R, A, 1, 1, 1, false>, a, st); \
    return at_variant<S>(a, [&](auto qv, auto vv, auto g, auto cb) {                                                         \
      constexpr int CB = decltype(g)::value == 4 ? 2 : decltype(cb)::value;                                                  \
      return at_run(attn_send_kernel<S, R, A, decltype(qv)::value, decltype(vv)::value, CB, true>, a, st);                   \
    });                                                                                                                      \
  }                                                                                                                          \
  cudaError_t at_join_sum_##suffix(const AtArgs& a, const AtRows& out, int width, int at, int stride, cudaStream_t st) {     \
    return at_launch(attn_join_sum_kernel<R, A>, dim3(a.n_joins, (width + 31) / 32), dim3(32, 8), 0, st, a, out, width, at,  \
                     stride);                                                                                                \
  }                                                                                                                          \
  cudaError_t at_table_##suffix(const AtArgs& a, cudaStream_t st) {                                                          \
    const int buckets = a.n_borders + 1, width = buckets * a.heads;                                                          \
    cudaError_t e = at_launch(attn_table_kernel<A>, dim3(a.hist_ctas), dim3(32 * a.hist_warps),                              \
                              (size_t(a.hist_warps) * buckets * a.hist_cols + a.n_borders) * sizeof(A), st, a);              \
    if (e != cudaSuccess || a.hist_ctas == 1) return e;                                                                      \
    return at_launch(attn_table_sum_kernel<A>, dim3((width + 31) / 32), dim3(32, 8), 0, st, a, a.hist_ctas);                 \
  }

}  // namespace cgtp
