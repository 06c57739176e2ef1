// adamw.cu -- AdamW over many tensors, with states in the parameters' type or in 8 bits, and
// the global gradient norm (declared in include/cgtp_train.h).
//
// Work is cut into units of up to eight blocks of 128 elements of one tensor (a table made with
// the optimizer: no search in the kernels); a warp takes a unit, a lane 4 elements of a block.  The
// tensors' pointers and decays travel in the kernel's parameters, so that the loads of a unit wait for
// one table entry only, which is read a unit ahead.
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include <algorithm>
#include <cmath>
#include <new>
#include <string>
#include <vector>

#include "cgtp_train.h"
#include "chain.cuh"
#include "internal.h"

struct cgtp_adamw_s {
  int param_dtype = 0, grad_dtype = 0, state = 0, num_sms = 0;
  std::vector<int64_t> numel, begin;   // begin[i]: first block of tensor i
  std::vector<float> decay;
  void* units_dev = nullptr;
  std::vector<int64_t> unit_begin;     // first unit of every kMostTensors-th tensor, and their number
  double* part = nullptr;              // one partial sum of squares per CTA
  unsigned* ticket = nullptr;          // CTAs of the norm that are done
  void* base = nullptr;
  size_t device_bytes = 0;
};

namespace cgtp {
namespace {

constexpr int kBlock = 128;        // elements of a block: 32 lanes x 4
constexpr int kMTop = 15, kVTop = 31;   // largest exponent field of the m and v codes
constexpr int kEMin = 40;          // block exponents below this are raised to it: every code is then a normal float
constexpr int kENan = 255;         // block exponent of a block of NaNs
constexpr int kStepThreads = 256;
constexpr int kWarpsPerCta = kStepThreads / 32;

constexpr int kUnit = 8;           // blocks of a unit at most
constexpr int kMostTensors = 1024, kFewTensors = 64;   // of a launch

struct __align__(16) Unit {
  int tensor;       // within its launch
  unsigned block;   // first block within the tensor
  unsigned state;   // first block within the states
  int elements;     // up to kUnit * kBlock
};

// pointers and decay factors of a launch's tensors
template <int K>
struct Tensors {
  void* p[K];
  const void* g[K];
  void* c[K];
  float decay[K];
};

struct Scalars {
  double lr_decay, b1, one_b1, b2, one_b2, rate, root, eps;
  uint32_t key0, key1;
  int flush;   // move_of<true>
};

// A v below the smallest normal float adds at most sqrt(2^-126) root = 1.1e-19 root to eps: less than 2^-25 of it, half
// the rounding of the sum, where eps is at least 4e-12 root (root: 31.6 in the first step of beta2 = 0.999).
constexpr double kFlushEps = 4e-12;

// Pseudo-random bits of element i (its low 32 bits; key0 holds the high ones too): a Weyl step and two
// multiply-xorshift rounds, of which the last xorshift is left to the two halves below.
__device__ __forceinline__ uint32_t noise_of(uint32_t i, uint32_t key0, uint32_t key1) {
  uint32_t x = i * 0x9E3779B1u + key0;
  x = (x ^ (x >> 15)) * 0xBB67AE85u;
  return (x ^ (x >> 13)) * 0x3C6EF373u + key1;
}
// the upper and the lower 16 bits of x ^ x >> 16, as the upper 16 of 20 bits
__device__ __forceinline__ uint32_t m_noise(uint32_t x) { return x >> 12 & 0xFFFF0u; }
__device__ __forceinline__ uint32_t v_noise(uint32_t x) { return (x << 4 ^ x >> 12) & 0xFFFF0u; }

// A code of a block with exponent E and largest exponent field TOP stands for
//   field f > 0:  2^(E - TOP + f - 127) (1 + mantissa / 8),   field 0:  mantissa 2^(E - TOP + 1 - 130),
// which is 2^(E - TOP) times the float whose bits are the code << 20 (a denormal for field 0).  The
// power goes in as two factors, since it may pass the largest float; both products are exact.
struct Power {
  float first, second;
};
__device__ __forceinline__ Power code_power(int E, int top) {
  const int base = max(E, kEMin) - top, half = base >> 1;
  return {E == kENan ? __uint_as_float(0x7FC00000u) : __uint_as_float(static_cast<uint32_t>(half + 127) << 23),
          __uint_as_float(static_cast<uint32_t>(base - half + 127) << 23)};
}
// bits of the float of byte j of a word of four codes: m (sign and 7 bits) and v (8 bits)
__device__ __forceinline__ float m_bits(uint32_t word, int j) {
  return __uint_as_float(static_cast<uint32_t>(static_cast<int32_t>(word << (24 - 8 * j)) >> 4) & 0x87F00000u);
}
__device__ __forceinline__ float v_bits(uint32_t word, int j) {
  return __uint_as_float((j == 3 ? word >> 4 : word << (20 - 8 * j)) & 0x0FF00000u);
}

// The code of x >= 0 (its bits), rounded up with probability = its distance above the code below it; r: 16 random
// bits, then four zeros, so that the distance counts in whole 2^-16 of a code step, rounded down (2^-17 in the
// mean).  E leaves room for the largest value of the block to be rounded up.
template <int TOP>
__device__ __forceinline__ uint32_t code_of(uint32_t bits, int E, uint32_t r) {
  return (bits + r - (static_cast<uint32_t>(E - TOP) << 23)) >> 20;
}
// The same where x may be below the smallest exponent of the codes; the code is the lowest byte.
template <int TOP>
__device__ __forceinline__ uint32_t code_of_any(uint32_t bits, int E, uint32_t r) {
  const int base = E - TOP;
  const float fine = __fmul_rn(__uint_as_float(bits), __uint_as_float(static_cast<uint32_t>(256 - base) << 23));
  const float noise = __fadd_rn(__uint_as_float(0x3F800000u | r << 3), -1.0f);   // r 2^-20
  const uint32_t low = __float_as_uint(__fadd_rd(__fadd_rn(fine, noise), 8388608.0f));   // 2^23 + the floor
  return bits >= (static_cast<uint32_t>(base + 1) << 23) ? code_of<TOP>(bits, E, r) : low;
}

__device__ __forceinline__ int block_exponent(uint32_t max_bits) {
  return max(static_cast<int>((max_bits + 0xFFFFFu) >> 23), kEMin);
}

template <typename G, typename A>
__device__ __forceinline__ void load4(const G* g, int64_t left, bool wide, A* v) {
  if constexpr (sizeof(G) == 4) {
    if (wide && left >= 4) {
      const float4 t = *reinterpret_cast<const float4*>(g);
      v[0] = t.x, v[1] = t.y, v[2] = t.z, v[3] = t.w;
      return;
    }
  } else if constexpr (sizeof(G) == 8) {
    if (wide && left >= 4) {
      const double2 s = reinterpret_cast<const double2*>(g)[0], t = reinterpret_cast<const double2*>(g)[1];
      v[0] = s.x, v[1] = s.y, v[2] = t.x, v[3] = t.y;
      return;
    }
  } else {
    if (wide && left >= 4) {
      const uint2 t = *reinterpret_cast<const uint2*>(g);
      v[0] = __uint_as_float(t.x << 16), v[1] = __uint_as_float(t.x & 0xFFFF0000u);
      v[2] = __uint_as_float(t.y << 16), v[3] = __uint_as_float(t.y & 0xFFFF0000u);
      return;
    }
  }
#pragma unroll
  for (int i = 0; i < 4; ++i) v[i] = i < left ? static_cast<A>(g[i]) : A(0);
}

template <typename G, typename A>
__device__ __forceinline__ void store4(G* g, int64_t left, bool wide, const A* v) {
  if constexpr (sizeof(G) == 4) {
    if (wide && left >= 4) {
      *reinterpret_cast<float4*>(g) = make_float4(v[0], v[1], v[2], v[3]);
      return;
    }
  } else if constexpr (sizeof(G) == 8) {
    if (wide && left >= 4) {
      reinterpret_cast<double2*>(g)[0] = make_double2(v[0], v[1]);
      reinterpret_cast<double2*>(g)[1] = make_double2(v[2], v[3]);
      return;
    }
  } else {
    if (wide && left >= 4) {
      __nv_bfloat162 s[2] = {__floats2bfloat162_rn(v[0], v[1]), __floats2bfloat162_rn(v[2], v[3])};
      *reinterpret_cast<uint2*>(g) = *reinterpret_cast<uint2*>(s);
      return;
    }
  }
#pragma unroll
  for (int i = 0; i < 4; ++i)
    if (i < left) g[i] = static_cast<G>(v[i]);
}

template <typename G>
__device__ __forceinline__ bool wide_ok(const G* p) {
  return (reinterpret_cast<uintptr_t>(p) & (4 * sizeof(G) > 16 ? 15 : 4 * sizeof(G) - 1)) == 0;
}

// m and v without contraction: every product and sum is rounded as written, so that the codes of
// the 8-bit states do not depend on how the compiler pairs them.  FP32 products in pairs (one instruction for two).
template <typename A>
struct Pair {
  A x, y;
};
__device__ __forceinline__ uint64_t bits_of(Pair<float> v) {
  return static_cast<uint64_t>(__float_as_uint(v.y)) << 32 | __float_as_uint(v.x);
}
__device__ __forceinline__ Pair<float> pair_of(uint64_t b) {
  return {__uint_as_float(static_cast<uint32_t>(b)), __uint_as_float(static_cast<uint32_t>(b >> 32))};
}
__device__ __forceinline__ Pair<float> mul_rn(Pair<float> a, Pair<float> b) {
  uint64_t r;
  asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(bits_of(a)), "l"(bits_of(b)));
  return pair_of(r);
}
// Sums one by one: a paired sum after a paired product came out contracted to one rounding.
__device__ __forceinline__ Pair<float> add_rn(Pair<float> a, Pair<float> b) { return {__fadd_rn(a.x, b.x), __fadd_rn(a.y, b.y)}; }
__device__ __forceinline__ Pair<double> mul_rn(Pair<double> a, Pair<double> b) { return {__dmul_rn(a.x, b.x), __dmul_rn(a.y, b.y)}; }
__device__ __forceinline__ Pair<double> add_rn(Pair<double> a, Pair<double> b) { return {__dadd_rn(a.x, b.x), __dadd_rn(a.y, b.y)}; }
template <typename A>
__device__ __forceinline__ Pair<A> mul_rn(Pair<A> a, A b) {
  return mul_rn(a, Pair<A>{b, b});
}

// rate m / (sqrt(v) root + eps).  FP32: root and reciprocal to a unit in the last place each, the move to a few;
// p's own rounding is larger unless the move is as large as p.  FAST: a v below the smallest normal float counts as
// zero (kFlushEps).
template <bool FAST>
__device__ __forceinline__ float move_of(float m, float v, float rate, float root, float eps) {
  float s, r;
  if constexpr (FAST) {
    asm("sqrt.approx.ftz.f32 %0, %1;" : "=f"(s) : "f"(v));
    asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(s * root + eps));
    return rate * m * r;
  }
  asm("sqrt.approx.f32 %0, %1;" : "=f"(s) : "f"(v));
  return __fdividef(rate * m, s * root + eps);
}
template <bool FAST>
__device__ __forceinline__ double move_of(double m, double v, double rate, double root, double eps) {
  return rate * m / (sqrt(v) * root + eps);
}

// p (1 - decay) - move.  Decay and move are added before anything is rounded to p's size: 1 - decay alone would lose a
// decay below 2^-25, and be off by a tenth at 3e-7.  An infinite p stays (decay p is infinite or 0 * inf).
template <typename A>
__device__ __forceinline__ A moved(A p, A decay, A move) {
  const A t = decay * p + move;
  return fabs(p) < A(INFINITY) ? p - t : p;
}

template <typename A>
struct StepScalars {
  A coef, decay, b1, one_b1, b2, one_b2, rate, root, eps;
  uint32_t key0, key1;
  bool flush;
};

// One block: p, g, m and v of a lane are there; m is m_scale times mv (a power of two or 1) before b1, and so is v.
template <typename A>
__device__ __forceinline__ void step_values(A (&p)[4], const A (&g)[4], A (&m)[4], A (&v)[4], const StepScalars<A>& s,
                                            A m_scale, A v_scale) {
  const A b1 = s.b1 * m_scale, b2 = s.b2 * v_scale;   // exact
#pragma unroll
  for (int i = 0; i < 4; i += 2) {
    const Pair<A> gi = mul_rn(Pair<A>{g[i], g[i + 1]}, s.coef);
    const Pair<A> mn = add_rn(mul_rn(Pair<A>{m[i], m[i + 1]}, b1), mul_rn(gi, s.one_b1));
    const Pair<A> vn = add_rn(mul_rn(Pair<A>{v[i], v[i + 1]}, b2), mul_rn(mul_rn(gi, gi), s.one_b2));
    m[i] = mn.x, m[i + 1] = mn.y, v[i] = vn.x, v[i + 1] = vn.y;
  }
  if (s.flush) {
#pragma unroll
    for (int i = 0; i < 4; ++i) p[i] = moved(p[i], s.decay, move_of<true>(m[i], v[i], s.rate, s.root, s.eps));
  } else {
#pragma unroll
    for (int i = 0; i < 4; ++i) p[i] = moved(p[i], s.decay, move_of<false>(m[i], v[i], s.rate, s.root, s.eps));
  }
}

// Rounds a block's m and v to codes: words of four codes a lane, and the block's exponents.
__device__ __forceinline__ void encode_block(const float (&m)[4], const float (&v)[4], int64_t place, const StepScalars<float>& s,
                                             uint32_t* m_word, uint32_t* v_word, uint32_t* m_exp, uint32_t* v_exp) {
  uint32_t a[4], b[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) a[i] = __float_as_uint(m[i]) & 0x7FFFFFFFu, b[i] = __float_as_uint(v[i]);   // v >= 0, or a NaN
  const uint32_t mb = max(max(a[0], a[1]), max(a[2], a[3])), vb = max(max(b[0], b[1]), max(b[2], b[3]));
  const int me = block_exponent(__reduce_max_sync(0xffffffffu, mb)), ve = block_exponent(__reduce_max_sync(0xffffffffu, vb));
  const uint32_t key = static_cast<uint32_t>(place >> 32) * 0x85A308D3u + s.key0;
  // m has values below its smallest exponent in most blocks where gradients are heavy-tailed; v hardly any but
  // zeros, which the warp looks for once
  const bool v_low = __any_sync(0xffffffffu, min(min(b[0], b[1]), min(b[2], b[3])) < static_cast<uint32_t>(ve - kVTop + 1) << 23);
  uint32_t r[4], cm[4], cv[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    r[i] = noise_of(static_cast<uint32_t>(place) + i, key, s.key1);
    cm[i] = code_of_any<kMTop>(a[i], me, m_noise(r[i]));
  }
  if (v_low) {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      cv[i] = code_of_any<kVTop>(b[i], ve, v_noise(r[i])) & 255u;
      cv[i] = b[i] ? max(cv[i], 1u) : cv[i];
    }
  } else {
#pragma unroll
    for (int i = 0; i < 4; ++i) cv[i] = code_of<kVTop>(b[i], ve, v_noise(r[i]));
  }
  const uint32_t signs = __byte_perm(__byte_perm(__float_as_uint(m[0]), __float_as_uint(m[1]), 0x0073),
                                     __byte_perm(__float_as_uint(m[2]), __float_as_uint(m[3]), 0x0073), 0x5410);
  const uint32_t mc = __byte_perm(__byte_perm(cm[0], cm[1], 0x0040), __byte_perm(cm[2], cm[3], 0x0040), 0x5410) | (signs & 0x80808080u);
  const uint32_t vc = __byte_perm(__byte_perm(cv[0], cv[1], 0x0040), __byte_perm(cv[2], cv[3], 0x0040), 0x5410);
  *m_word = me >= kENan ? 0 : mc;
  *v_word = ve >= kENan ? 0 : vc;
  *m_exp = static_cast<uint32_t>(min(me, kENan));
  *v_exp = static_cast<uint32_t>(min(ve, kENan));
}

template <typename A>
__device__ __forceinline__ StepScalars<A> scalars_of(const Scalars& host, A coef) {
  StepScalars<A> s;
  s.coef = coef;
  s.b1 = static_cast<A>(host.b1), s.one_b1 = static_cast<A>(host.one_b1);
  s.b2 = static_cast<A>(host.b2), s.one_b2 = static_cast<A>(host.one_b2);
  s.rate = static_cast<A>(host.rate), s.root = static_cast<A>(host.root), s.eps = static_cast<A>(host.eps);
  s.key0 = host.key0, s.key1 = host.key1;
  s.flush = host.flush;
  return s;
}

// ---------------------------------------------------------------------------
// States in the parameters' type: a lane holds its elements of NB blocks, and the loads of the next NB are
// in flight while these are computed.  Bound by HBM: 100.7 M FP32 parameters with bfloat16 gradients and copies,
// 28 bytes an element, 425 us (6.6 TB/s; a copy reaches 6.7); without loads ahead 445 us, a block a warp 495 us.
// ---------------------------------------------------------------------------

template <typename A, int NB>
struct Held {
  A p[NB][4], g[NB][4], m[NB][4], v[NB][4];
};

// k: the first block's place in the states; p, g, c point at the lane's elements of it, of which `left` are
// in the tensor.  WHOLE: every element is there and every address allows 16-byte (bfloat16: 8-byte) accesses.
template <typename A, typename G, bool WHOLE, int NB>
__device__ __forceinline__ void get_blocks(Held<A, NB>& h, unsigned k, int left, const A* p, const G* g, const A* m, const A* v) {
#pragma unroll
  for (int b = 0; b < NB; ++b) {
    const int64_t place = (int64_t)(k + b) * kBlock + (threadIdx.x & 31) * 4;
    load4<A, A>(p + b * kBlock, WHOLE ? 4 : left - b * kBlock, WHOLE || wide_ok(p), h.p[b]);
    load4<G, A>(g + b * kBlock, WHOLE ? 4 : left - b * kBlock, WHOLE || wide_ok(g), h.g[b]);
    load4<A, A>(m + place, 4, true, h.m[b]);
    load4<A, A>(v + place, 4, true, h.v[b]);
  }
}
template <typename A, bool WHOLE, int NB>
__device__ __forceinline__ void put_blocks(Held<A, NB>& h, unsigned k, int left, A* p, __nv_bfloat16* c, A* m, A* v,
                                           const StepScalars<A>& s) {
#pragma unroll
  for (int b = 0; b < NB; ++b) {
    const int64_t place = (int64_t)(k + b) * kBlock + (threadIdx.x & 31) * 4;
    const int rest = WHOLE ? 4 : left - b * kBlock;
    step_values<A>(h.p[b], h.g[b], h.m[b], h.v[b], s, A(1), A(1));
    store4<A, A>(p + b * kBlock, rest, WHOLE || wide_ok(p), h.p[b]);
    if constexpr (sizeof(A) == 4)
      if (c) store4<__nv_bfloat16, A>(c + b * kBlock, rest, WHOLE || wide_ok(c), h.p[b]);
    store4<A, A>(m + place, 4, true, h.m[b]);
    store4<A, A>(v + place, 4, true, h.v[b]);
  }
}

template <typename A, typename G, int K>
__global__ void __launch_bounds__(kStepThreads) adamw_kernel(const __grid_constant__ Tensors<K> ts, const Unit* units,
                                                             unsigned n_units, A* m, A* v, const Scalars host, const A* clip) {
  constexpr int NB = sizeof(A) == 8 ? 1 : 2;
  chain_enter();
  const int lane = threadIdx.x & 31;
  const unsigned stride = gridDim.x * kWarpsPerCta;
  unsigned u = blockIdx.x * kWarpsPerCta + (threadIdx.x >> 5);
  if (u >= n_units) return;
  Unit next = units[u];
  const A coef = clip ? clip[1] : A(1);
  if (!isfinite(coef)) return;
  StepScalars<A> s = scalars_of<A>(host, coef);
  const A lr_decay = static_cast<A>(host.lr_decay);
  for (;;) {
    const Unit unit = next;
    u += stride;
    if (u < n_units) next = units[u];
    const G* g = static_cast<const G*>(ts.g[unit.tensor]);
    if (g) {
      s.decay = lr_decay * static_cast<A>(ts.decay[unit.tensor]);
      const int64_t at = (int64_t)unit.block * kBlock + lane * 4;
      A* p = static_cast<A*>(ts.p[unit.tensor]) + at;
      __nv_bfloat16* c = ts.c[unit.tensor] ? static_cast<__nv_bfloat16*>(ts.c[unit.tensor]) + at : nullptr;
      g += at;
      if (unit.elements == kUnit * kBlock && wide_ok(p) && wide_ok(g) && (!c || wide_ok(c))) {
        Held<A, NB> h, ahead;
        get_blocks<A, G, true, NB>(h, unit.state, 4, p, g, m, v);
#pragma unroll 1
        for (int b = 0; b < kUnit; b += NB) {
          if (b + NB < kUnit) get_blocks<A, G, true, NB>(ahead, unit.state + b + NB, 4, p + (b + NB) * kBlock, g + (b + NB) * kBlock, m, v);
          put_blocks<A, true, NB>(h, unit.state + b, 4, p + b * kBlock, c ? c + b * kBlock : nullptr, m, v, s);
          h = ahead;
        }
      } else {
#pragma unroll 1
        for (int b = 0; b * kBlock < unit.elements; ++b) {
          Held<A, 1> h;
          const int left = unit.elements - b * kBlock - lane * 4;
          get_blocks<A, G, false, 1>(h, unit.state + b, left, p + b * kBlock, g + b * kBlock, m, v);
          put_blocks<A, false, 1>(h, unit.state + b, left, p + b * kBlock, c ? c + b * kBlock : nullptr, m, v, s);
        }
      }
    }
    if (u >= n_units) return;
  }
}

// ---------------------------------------------------------------------------
// 8-bit states.  Decoding and rounding take about 300 instructions a block, so a warp that waits for
// its loads costs issue slots: operands come through a ring of asynchronous copies in shared memory, two blocks
// a stage, that runs ahead over the warp's units.  100.7 M parameters, 16 bytes an element: 364 to 371 us (4.4 TB/s) at 365
// warp instructions a block and 2.8 a cycle; loads into registers instead of the ring 470 us at best.
// ---------------------------------------------------------------------------

constexpr int kRing = 3, kStageBlocks = 2;

template <typename G>
struct __align__(16) Stage {
  float p[kStageBlocks * kBlock];
  G g[kStageBlocks * kBlock];
  uint8_t m[kStageBlocks * kBlock], v[kStageBlocks * kBlock];
  float* to;            // the first block's parameters, and their copy
  __nv_bfloat16* copy;
  unsigned state;       // the first block's place in the states
  int elements;         // from there to the end of the unit
  float decay;
  int wide;             // whole blocks at aligned addresses
};

__device__ __forceinline__ void copy_async16(void* shared, const void* global) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(static_cast<uint32_t>(__cvta_generic_to_shared(shared))), "l"(global) : "memory");
}
__device__ __forceinline__ void copy_async8(void* shared, const void* global) {
  asm volatile("cp.async.ca.shared.global [%0], [%1], 8;" ::"r"(static_cast<uint32_t>(__cvta_generic_to_shared(shared))), "l"(global) : "memory");
}

// The warp's units in order, a stage's blocks at a time.
template <typename G, int K>
struct Feed {
  const Tensors<K>& ts;
  const Unit* units;
  unsigned n_units, stride, next_index;
  Unit unit, next;
  int block;            // next block of the unit
  const uint8_t *m, *v;
  float lr_decay;

  __device__ __forceinline__ void advance() {
    unit = next;
    block = 0;
    next_index += stride;
    next.elements = 0;
    if (next_index < n_units) next = units[next_index];
  }
  // fills a stage; false behind the last unit
  __device__ __forceinline__ bool fill(Stage<G>& st) {
    const int lane = threadIdx.x & 31;
    while (block * kBlock >= unit.elements || !ts.g[unit.tensor]) {
      if (next.elements == 0) return false;
      advance();
    }
    const int elements = unit.elements - block * kBlock;
    const int64_t at = (int64_t)(unit.block + block) * kBlock;
    float* p = static_cast<float*>(ts.p[unit.tensor]) + at;
    const G* g = static_cast<const G*>(ts.g[unit.tensor]) + at;
    __nv_bfloat16* c = ts.c[unit.tensor] ? static_cast<__nv_bfloat16*>(ts.c[unit.tensor]) + at : nullptr;
    const unsigned state = unit.state + block;
    const bool wide = elements >= kStageBlocks * kBlock && wide_ok(p) && wide_ok(g) && (!c || wide_ok(c));
    if (lane == 0) {
      st.to = p, st.copy = c;
      st.state = state, st.elements = elements;
      st.decay = lr_decay * ts.decay[unit.tensor];
      st.wide = wide;
    }
    if (wide) {
#pragma unroll
      for (int b = 0; b < kStageBlocks; ++b) {
        copy_async16(st.p + b * kBlock + lane * 4, p + b * kBlock + lane * 4);
        if constexpr (sizeof(G) == 4) copy_async16(st.g + b * kBlock + lane * 4, g + b * kBlock + lane * 4);
        else copy_async8(st.g + b * kBlock + lane * 4, g + b * kBlock + lane * 4);
      }
      // 16 lanes the codes of m, 16 those of v
      const uint8_t* codes = (lane < 16 ? m : v) + (int64_t)state * kBlock + (lane & 15) * 16;
      copy_async16((lane < 16 ? st.m : st.v) + (lane & 15) * 16, codes);
    } else {
      for (int i = lane; i < min(elements, kStageBlocks * kBlock); i += 32) st.p[i] = p[i], st.g[i] = g[i];
      const int words = min(kStageBlocks, (elements + kBlock - 1) / kBlock) * (kBlock / 4);
      for (int i = lane; i < words; i += 32) {
        reinterpret_cast<uint32_t*>(st.m)[i] = reinterpret_cast<const uint32_t*>(m + (int64_t)state * kBlock)[i];
        reinterpret_cast<uint32_t*>(st.v)[i] = reinterpret_cast<const uint32_t*>(v + (int64_t)state * kBlock)[i];
      }
    }
    block += kStageBlocks;
    return true;
  }
};

template <typename G, int K>
__global__ void __launch_bounds__(kStepThreads, 3) adamw8_kernel(const __grid_constant__ Tensors<K> ts, const Unit* units,
                                                                 unsigned n_units, uint8_t* m_, uint8_t* v_, uint8_t* m_exp,
                                                                 uint8_t* v_exp, const Scalars host, const float* clip) {
  extern __shared__ __align__(16) unsigned char shared[];
  chain_enter();
  const int lane = threadIdx.x & 31;
  Stage<G>* ring = reinterpret_cast<Stage<G>*>(shared) + (threadIdx.x >> 5) * kRing;
  const unsigned first = blockIdx.x * kWarpsPerCta + (threadIdx.x >> 5);
  if (first >= n_units) return;
  const float coef = clip ? clip[1] : 1.0f;
  if (!isfinite(coef)) return;
  StepScalars<float> s = scalars_of<float>(host, coef);
  Feed<G, K> feed{ts, units, n_units, gridDim.x * kWarpsPerCta, first, {}, units[first], 0, m_, v_, static_cast<float>(host.lr_decay)};
  feed.advance();
  int filled = 0, done = 0;
  bool more = true;
#pragma unroll
  for (int i = 0; i < kRing - 1; ++i) {
    more = more && feed.fill(ring[i]);
    filled += more;
    asm volatile("cp.async.commit_group;" ::: "memory");
  }
  __syncwarp();
  // exponents of a stage's blocks: lanes 0 and 1 those of m, 2 and 3 those of v, a stage ahead
  static_assert(kStageBlocks == 2, "lanes 0 to 3 hold the exponents of a stage");
  const auto exponent_at = [&](const Stage<G>& st) { return (lane < 2 ? m_exp : v_exp) + st.state + (lane & 1); };
  const auto exponents = [&](const Stage<G>& st) -> uint32_t {
    return lane < 4 && (lane & 1) * kBlock < st.elements ? *exponent_at(st) : 0u;
  };
  uint32_t e = done < filled ? exponents(ring[0]) : 0u;
  for (int at = 0; done < filled; ++done, at = at + 1 == kRing ? 0 : at + 1) {
    const int free = at == 0 ? kRing - 1 : at - 1;   // the stage of the last turn
    more = more && feed.fill(ring[free]);
    filled += more;
    asm volatile("cp.async.commit_group;" ::: "memory");
    asm volatile("cp.async.wait_group %0;" ::"n"(kRing - 1) : "memory");
    __syncwarp();
    const Stage<G>& st = ring[at];
    const uint32_t e_now = e;
    if (done + 1 < filled) e = exponents(ring[at + 1 == kRing ? 0 : at + 1]);
    s.decay = st.decay;
    uint32_t e_new = 0;
    const Power power = code_power(static_cast<int>(e_now), lane < 2 ? kMTop : kVTop);   // of lanes 0 to 3
    const int64_t first_place = (int64_t)st.state * kBlock + lane * 4;
    uint32_t *m_words = reinterpret_cast<uint32_t*>(m_ + first_place), *v_words = reinterpret_cast<uint32_t*>(v_ + first_place);
    const int elements = st.elements;
    float* const first_to = st.to + lane * 4;
    __nv_bfloat16* const first_copy = st.copy ? st.copy + lane * 4 : nullptr;
    const bool wide = st.wide;
#pragma unroll
    for (int b = 0; b < kStageBlocks; ++b) {
      if (b * kBlock < elements) {
        const int left = elements - b * kBlock - lane * 4;
        float p[4], g[4], m[4], v[4];
        load4<float, float>(st.p + b * kBlock + lane * 4, 4, true, p);
        load4<G, float>(st.g + b * kBlock + lane * 4, 4, true, g);
        const uint32_t mw = reinterpret_cast<const uint32_t*>(st.m + b * kBlock)[lane], vw = reinterpret_cast<const uint32_t*>(st.v + b * kBlock)[lane];
        const Power mp{__shfl_sync(0xffffffffu, power.first, b), __shfl_sync(0xffffffffu, power.second, b)};
        const Power vp{__shfl_sync(0xffffffffu, power.first, 2 + b), __shfl_sync(0xffffffffu, power.second, 2 + b)};
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          m[i] = m_bits(mw, i) * mp.first;
          v[i] = v_bits(vw, i) * vp.first;
        }
        step_values<float>(p, g, m, v, s, mp.second, vp.second);
        float* to = first_to + b * kBlock;
        __nv_bfloat16* copy = first_copy ? first_copy + b * kBlock : nullptr;
        if (wide) {
          store4<float, float>(to, 4, true, p);
          if (copy) store4<__nv_bfloat16, float>(copy, 4, true, p);
        } else {
          store4<float, float>(to, left, wide_ok(to), p);
          if (copy) store4<__nv_bfloat16, float>(copy, left, wide_ok(copy), p);
#pragma unroll
          for (int i = 0; i < 4; ++i)
            if (i >= left) m[i] = v[i] = 0.0f;   // the place behind the tensor's end
        }
        uint32_t m_word, v_word, me, ve;
        encode_block(m, v, first_place + b * kBlock, s, &m_word, &v_word, &me, &ve);
        m_words[b * (kBlock / 4)] = m_word;
        v_words[b * (kBlock / 4)] = v_word;
        e_new = lane == b ? me : lane == 2 + b ? ve : e_new;
      }
    }
    if (lane < 4 && (lane & 1) * kBlock < elements) *exponent_at(st) = static_cast<uint8_t>(e_new);
    __syncwarp();
  }
}

// Bound by HBM: 100.7 M elements, 10 bytes each, 150 us (6.7 TB/s).
__global__ void __launch_bounds__(kStepThreads) state_values_kernel(const uint8_t* m, const uint8_t* v, const uint8_t* m_exp,
                                                                    const uint8_t* v_exp, float* m_out, float* v_out, int64_t n4) {
  chain_enter();
  const int64_t i = (int64_t)blockIdx.x * kStepThreads + threadIdx.x;
  if (i >= n4) return;
  const uint32_t mc = reinterpret_cast<const uint32_t*>(m)[i], vc = reinterpret_cast<const uint32_t*>(v)[i];
  const Power mp = code_power(m_exp[i >> 5], kMTop), vp = code_power(v_exp[i >> 5], kVTop);
  float a[4], b[4];
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    a[j] = __fmul_rn(__fmul_rn(m_bits(mc, j), mp.first), mp.second);
    b[j] = __fmul_rn(__fmul_rn(v_bits(vc, j), vp.first), vp.second);
  }
  reinterpret_cast<float4*>(m_out)[i] = make_float4(a[0], a[1], a[2], a[3]);
  reinterpret_cast<float4*>(v_out)[i] = make_float4(b[0], b[1], b[2], b[3]);
}

__device__ __forceinline__ double cta_sum(double v) {
  __shared__ double warp_sum[kWarpsPerCta];
  for (int o = 16; o; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
  __syncthreads();
  if ((threadIdx.x & 31) == 0) warp_sum[threadIdx.x >> 5] = v;
  __syncthreads();
  double t = 0.0;
  for (int w = 0; w < kWarpsPerCta; ++w) t += warp_sum[w];
  return t;
}

// Bound by HBM reads: 100.7 M FP32 gradients 67 us (6.0 TB/s).
// Sum of squares of the CTA's units: a thread's own in A, the rest in FP64.  The last CTA of the last launch
// (a counter; the order of the sums does not depend on it) adds the CTAs' sums and leaves the counter at zero.
template <typename A, typename G, int K>
__global__ void __launch_bounds__(kStepThreads) norm_kernel(const __grid_constant__ Tensors<K> ts, const Unit* units,
                                                            unsigned n_units, double* part, int before, bool last,
                                                            unsigned* ticket, double max_norm, A* out) {
  chain_enter();
  const int lane = threadIdx.x & 31;
  A sum[4] = {A(0), A(0), A(0), A(0)};
  for (unsigned u = blockIdx.x * kWarpsPerCta + (threadIdx.x >> 5); u < n_units; u += gridDim.x * kWarpsPerCta) {
    const Unit unit = units[u];
    const G* g = static_cast<const G*>(ts.g[unit.tensor]);
    if (!g) continue;
    g += (int64_t)unit.block * kBlock + lane * 4;
    A v[kUnit][4];
    if (unit.elements == kUnit * kBlock && wide_ok(g)) {
#pragma unroll
      for (int b = 0; b < kUnit; ++b) load4<G, A>(g + b * kBlock, 4, true, v[b]);
    } else {
#pragma unroll
      for (int b = 0; b < kUnit; ++b) load4<G, A>(g + b * kBlock, unit.elements - b * kBlock - lane * 4, wide_ok(g), v[b]);
    }
#pragma unroll
    for (int b = 0; b < kUnit; ++b)
#pragma unroll
      for (int i = 0; i < 4; ++i) sum[i] += v[b][i] * v[b][i];
  }
  const double mine = cta_sum(static_cast<double>((sum[0] + sum[1]) + (sum[2] + sum[3])));
  __shared__ bool finish;
  if (threadIdx.x == 0) {
    part[before + blockIdx.x] = mine;
    __threadfence();
    finish = last && atomicAdd(ticket, 1u) == gridDim.x - 1;
  }
  __syncthreads();
  if (!finish) return;
  __threadfence();
  const int count = before + static_cast<int>(gridDim.x);
  double v = 0.0;
  for (int i = threadIdx.x; i < count; i += kStepThreads) v += __ldcg(part + i);
  v = cta_sum(v);
  if (threadIdx.x != 0) return;
  *ticket = 0;
  const double norm = sqrt(v);
  out[0] = static_cast<A>(norm);
  out[1] = isfinite(norm) ? static_cast<A>(norm > max_norm ? max_norm / norm : 1.0) : static_cast<A>(nan(""));
}

constexpr int kNormCtasPerSm = 8, kStepCtasPerSm = 8;

cgtp_status launched(cudaError_t e, const char* what) {
  return e == cudaSuccess ? CGTP_OK : fail(CGTP_ECUDA, std::string(what) + ": " + cudaGetErrorString(e));
}

template <int K>
void fill(Tensors<K>* a, const cgtp_adamw_s* o, int t0, int n, void* const* params, const void* const* grads, void* const* copies) {
  for (int i = 0; i < n; ++i) {
    a->p[i] = params ? params[t0 + i] : nullptr;
    a->g[i] = grads[t0 + i];
    a->c[i] = copies ? copies[t0 + i] : nullptr;
    a->decay[i] = o->decay[t0 + i];
  }
}

struct StepArgs {
  void *m, *v;
  uint8_t *m_exp, *v_exp;
  Scalars s;
  const void* clip;
};

int ctas_for(const cgtp_adamw_s* o, int64_t units, int per_sm) {
  return static_cast<int>(std::max<int64_t>(1, std::min<int64_t>((units + kWarpsPerCta - 1) / kWarpsPerCta, int64_t(o->num_sms) * per_sm)));
}

template <typename A, typename G, bool EIGHT, int K>
cgtp_status step_launch(const cgtp_adamw_s* o, int t0, int n, void* const* params, const void* const* grads,
                        void* const* copies, const StepArgs& a, cudaStream_t st) {
  Tensors<K> ts;
  fill(&ts, o, t0, n, params, grads, copies);
  const int64_t u0 = o->unit_begin[t0 / kMostTensors], u1 = o->unit_begin[t0 / kMostTensors + 1];
  if (u1 == u0) return CGTP_OK;
  const Unit* units = static_cast<const Unit*>(o->units_dev) + u0;
  const unsigned n_units = static_cast<unsigned>(u1 - u0);
  if constexpr (EIGHT) {
    constexpr int bytes = kWarpsPerCta * kRing * sizeof(Stage<G>);
    if (smem_cap_cached(reinterpret_cast<const void*>(adamw8_kernel<G, K>)) < bytes) return fail(CGTP_ECUDA, "adamw step: shared memory");
    return launched(chain_launch(adamw8_kernel<G, K>, ctas_for(o, n_units, 3), kStepThreads, bytes, st, ts, units, n_units, a.m, a.v,
                                 a.m_exp, a.v_exp, a.s, a.clip),
                    "adamw step");
  } else {
    return launched(chain_launch(adamw_kernel<A, G, K>, ctas_for(o, n_units, kStepCtasPerSm), kStepThreads, 0, st, ts, units, n_units,
                                 a.m, a.v, a.s, a.clip),
                    "adamw step");
  }
}

template <typename A, typename G, bool EIGHT>
cgtp_status step_all(const cgtp_adamw_s* o, void* const* params, const void* const* grads, void* const* copies,
                     const StepArgs& a, cudaStream_t st) {
  const int all = static_cast<int>(o->numel.size());
  for (int t0 = 0; t0 < all; t0 += kMostTensors) {
    const int n = std::min(kMostTensors, all - t0);
    const cgtp_status s = n <= kFewTensors ? step_launch<A, G, EIGHT, kFewTensors>(o, t0, n, params, grads, copies, a, st)
                                           : step_launch<A, G, EIGHT, kMostTensors>(o, t0, n, params, grads, copies, a, st);
    if (s != CGTP_OK) return s;
  }
  return CGTP_OK;
}

template <typename A, typename G>
cgtp_status norm_all(const cgtp_adamw_s* o, const void* const* grads, double max_norm, void* out, cudaStream_t st) {
  const int all = static_cast<int>(o->numel.size());
  int before = 0;
  for (int t0 = 0; t0 < all; t0 += kMostTensors) {
    const int n = std::min(kMostTensors, all - t0);
    const int64_t u0 = o->unit_begin[t0 / kMostTensors], u1 = o->unit_begin[t0 / kMostTensors + 1];
    const int ctas = ctas_for(o, u1 - u0, kNormCtasPerSm);
    const bool last = t0 + n == all;
    cudaError_t e = cudaSuccess;
    const auto run = [&](auto few, auto kernel) {
      decltype(few) ts;
      fill(&ts, o, t0, n, nullptr, grads, nullptr);
      e = chain_launch(kernel, ctas, kStepThreads, 0, st, ts, static_cast<const Unit*>(o->units_dev) + u0, u1 - u0, o->part, before, last,
                       o->ticket, max_norm, out);
    };
    if (n <= kFewTensors) run(Tensors<kFewTensors>{}, norm_kernel<A, G, kFewTensors>);
    else run(Tensors<kMostTensors>{}, norm_kernel<A, G, kMostTensors>);
    const cgtp_status s = launched(e, "gradient norm");
    if (s != CGTP_OK) return s;
    before += ctas;
  }
  return CGTP_OK;
}

int es_of(int dtype) { return dtype == CGTP_F64 ? 8 : dtype == CGTP_BF16 ? 2 : 4; }

cgtp_status element(const void* p, int es, const char* name, size_t i) {
  if (reinterpret_cast<uintptr_t>(p) % es)
    return fail(CGTP_EINVAL, std::string("pointer not aligned to its element: ") + name + " " + std::to_string(i));
  return CGTP_OK;
}

cgtp_status buffer(const void* p, const char* name) {
  if (!p) return fail(CGTP_EINVAL, std::string("null pointer: ") + name);
  if (reinterpret_cast<uintptr_t>(p) % 16) return fail(CGTP_EINVAL, std::string("pointer not 16-byte aligned: ") + name);
  return CGTP_OK;
}

// the step's key: seed and t through two multiply-xorshift rounds
uint64_t step_key(uint64_t seed, int64_t t) {
  uint64_t z = seed + static_cast<uint64_t>(t) * 0x9E3779B97F4A7C15ull;
  z = (z ^ (z >> 29)) * 0xBB67AE8584CAA73Bull;
  z = (z ^ (z >> 32)) * 0x9E3779B97F4A7C15ull;
  return z ^ (z >> 29);
}

cgtp_status create(cgtp_adamw_s* o, int n, const int64_t* numel, const float* decay_scale) {
  o->begin.push_back(0);
  for (int i = 0; i < n; ++i) {
    if (numel[i] < 0) return fail(CGTP_EINVAL, "a tensor has fewer than 0 elements");
    if (numel[i] > (int64_t(1) << 36)) return fail(CGTP_EUNSUPPORTED, "a tensor has more than 2^36 elements");
    if (decay_scale && !std::isfinite(decay_scale[i])) return fail(CGTP_EINVAL, "decay_scale must be finite");
    o->numel.push_back(numel[i]);
    o->begin.push_back(o->begin.back() + (numel[i] + kBlock - 1) / kBlock);
    if (o->begin.back() > (int64_t(1) << 31) - 1) return fail(CGTP_EUNSUPPORTED, "more than 2^31 - 1 blocks of 128 elements");
  }
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess ||
      cudaDeviceGetAttribute(&o->num_sms, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess) {
    cudaGetLastError();
    return fail(CGTP_ECUDA, "no CUDA device");
  }
  o->decay.assign(n, 1.0f);
  if (decay_scale) o->decay.assign(decay_scale, decay_scale + n);
  // one allocation: the ticket (in the place of a unit), the units, the partial sums
  std::vector<Unit> units(1, Unit{});
  for (int i = 0; i < n; ++i) {
    if (i % kMostTensors == 0) o->unit_begin.push_back(static_cast<int64_t>(units.size()) - 1);
    for (int64_t b = 0; b < o->begin[i + 1] - o->begin[i]; b += kUnit)
      units.push_back({i % kMostTensors, static_cast<unsigned>(b), static_cast<unsigned>(o->begin[i] + b),
                       static_cast<int>(std::min<int64_t>(kUnit * kBlock, numel[i] - b * kBlock))});
  }
  o->unit_begin.push_back(static_cast<int64_t>(units.size()) - 1);
  const size_t parts = size_t(o->num_sms) * kNormCtasPerSm * (o->unit_begin.size() - 1);
  const size_t b_units = units.size() * sizeof(Unit), bytes = b_units + parts * sizeof(double);
  if (cudaMalloc(&o->base, bytes) != cudaSuccess) {
    cudaGetLastError();
    return fail(CGTP_ENOMEM, "optimizer table allocation failed");
  }
  o->device_bytes = bytes;
  o->ticket = static_cast<unsigned*>(o->base);
  o->units_dev = static_cast<Unit*>(o->base) + 1;
  o->part = reinterpret_cast<double*>(static_cast<unsigned char*>(o->base) + b_units);
  if (!upload(o->base, units.data(), b_units)) {
    cudaGetLastError();
    return fail(CGTP_ECUDA, "optimizer table upload failed");
  }
  return CGTP_OK;
}

}  // namespace
}  // namespace cgtp

using namespace cgtp;

extern "C" {

cgtp_status cgtp_adamw_create(cgtp_adamw* out, int n_tensors, const int64_t* numel, const float* decay_scale,
                              int param_dtype, int grad_dtype, int state) {
  clear_error();
  if (!out) return fail(CGTP_EINVAL, "null optimizer output pointer");
  *out = nullptr;
  if (n_tensors < 1 || !numel) return fail(CGTP_EINVAL, "an optimizer needs at least one tensor");
  if (param_dtype != CGTP_F32 && param_dtype != CGTP_F64) return fail(CGTP_EINVAL, "param_dtype must be CGTP_F32 or CGTP_F64");
  if (grad_dtype != param_dtype && !(grad_dtype == CGTP_BF16 && param_dtype == CGTP_F32))
    return fail(CGTP_EINVAL, "grad_dtype must be param_dtype, or CGTP_BF16 with CGTP_F32 parameters");
  if (state != CGTP_STATE_FULL && state != CGTP_STATE_8BIT) return fail(CGTP_EINVAL, "state must be CGTP_STATE_FULL or CGTP_STATE_8BIT");
  if (state == CGTP_STATE_8BIT && param_dtype != CGTP_F32) return fail(CGTP_EUNSUPPORTED, "8-bit states need CGTP_F32 parameters");
  cgtp_adamw_s* o = new (std::nothrow) cgtp_adamw_s();
  if (!o) return fail(CGTP_ENOMEM, "host allocation failed");
  o->param_dtype = param_dtype;
  o->grad_dtype = grad_dtype;
  o->state = state;
  cgtp_status s;
  try {
    s = create(o, n_tensors, numel, decay_scale);
  } catch (const std::bad_alloc&) {
    s = fail(CGTP_ENOMEM, "host allocation failed");
  }
  if (s != CGTP_OK) {
    cgtp_adamw_destroy(o);
    return s;
  }
  *out = o;
  return CGTP_OK;
}

void cgtp_adamw_destroy(cgtp_adamw o) {
  if (!o) return;
  if (o->base) cudaFree(o->base);
  delete o;
}

cgtp_status cgtp_adamw_info(cgtp_adamw o, int64_t* state_numel) {
  clear_error();
  if (!o) return fail(CGTP_EINVAL, "null optimizer");
  if (state_numel) *state_numel = o->begin.back() * kBlock;
  return CGTP_OK;
}

cgtp_status cgtp_adamw_device_bytes(cgtp_adamw o, int64_t* bytes) {
  clear_error();
  if (!o || !bytes) return fail(CGTP_EINVAL, "null argument");
  *bytes = static_cast<int64_t>(o->device_bytes);
  return CGTP_OK;
}

cgtp_status cgtp_adamw_step(cgtp_adamw o, void* const* params, const void* const* grads, void* const* copies, void* m,
                            void* v, void* m_exp, void* v_exp, double lr, double beta1, double beta2, double eps,
                            double weight_decay, int64_t step, uint64_t seed, const void* clip, void* stream) {
  clear_error();
  if (!o) return fail(CGTP_EINVAL, "null optimizer");
  if (!params || !grads) return fail(CGTP_EINVAL, "null pointer list");
  if (!(beta1 >= 0.0 && beta1 < 1.0 && beta2 >= 0.0 && beta2 < 1.0)) return fail(CGTP_EINVAL, "betas must be in [0, 1)");
  if (!std::isfinite(lr) || !std::isfinite(weight_decay) || !(eps >= 0.0) || !std::isfinite(eps))
    return fail(CGTP_EINVAL, "lr, weight_decay and eps must be finite, eps >= 0");
  if (step < 1) return fail(CGTP_EINVAL, "steps are counted from 1");
  if (copies && o->param_dtype != CGTP_F32) return fail(CGTP_EUNSUPPORTED, "bfloat16 copies need CGTP_F32 parameters");
  const int ep = es_of(o->param_dtype), eg = es_of(o->grad_dtype);
  cgtp_status s;
  for (size_t i = 0; i < o->numel.size(); ++i) {
    if (o->numel[i] == 0 || !grads[i]) continue;
    if (!params[i]) return fail(CGTP_EINVAL, "null pointer: parameter " + std::to_string(i));
    if ((s = element(params[i], ep, "parameter", i)) || (s = element(grads[i], eg, "gradient", i)) ||
        (copies && (s = element(copies[i], 2, "copy", i))))
      return s;
  }
  if ((s = element(clip, ep, "clip", 0))) return s;
  if (o->begin.back() == 0) return CGTP_OK;
  if ((s = buffer(m, "m")) || (s = buffer(v, "v"))) return s;
  const bool eight = o->state == CGTP_STATE_8BIT;
  if (eight && (!m_exp || !v_exp)) return fail(CGTP_EINVAL, "8-bit states need m_exp and v_exp");
  const uint64_t key = step_key(seed, step);
  const double t = static_cast<double>(step);
  const double root = 1.0 / std::sqrt(1.0 - std::pow(beta2, t));
  StepArgs a{m, v, static_cast<uint8_t*>(m_exp), static_cast<uint8_t*>(v_exp),
             Scalars{lr * weight_decay, beta1, 1.0 - beta1, beta2, 1.0 - beta2, lr / (1.0 - std::pow(beta1, t)), root, eps,
                     static_cast<uint32_t>(key), static_cast<uint32_t>(key >> 32), eps >= kFlushEps * root},
             clip};
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  if (o->param_dtype == CGTP_F64) return step_all<double, double, false>(o, params, grads, copies, a, st);
  if (o->grad_dtype == CGTP_BF16)
    return eight ? step_all<float, __nv_bfloat16, true>(o, params, grads, copies, a, st)
                 : step_all<float, __nv_bfloat16, false>(o, params, grads, copies, a, st);
  return eight ? step_all<float, float, true>(o, params, grads, copies, a, st)
               : step_all<float, float, false>(o, params, grads, copies, a, st);
}

cgtp_status cgtp_grad_norm(cgtp_adamw o, const void* const* grads, double max_norm, void* out, void* stream) {
  clear_error();
  if (!o) return fail(CGTP_EINVAL, "null optimizer");
  if (!grads || !out) return fail(CGTP_EINVAL, "null pointer");
  if (!(max_norm > 0.0)) return fail(CGTP_EINVAL, "max_norm must be > 0");
  cgtp_status s;
  if ((s = element(out, es_of(o->param_dtype), "out", 0))) return s;
  for (size_t i = 0; i < o->numel.size(); ++i)
    if (o->numel[i] && (s = element(grads[i], es_of(o->grad_dtype), "gradient", i))) return s;
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  if (o->param_dtype == CGTP_F64) return norm_all<double, double>(o, grads, max_norm, out, st);
  if (o->grad_dtype == CGTP_BF16) return norm_all<float, __nv_bfloat16>(o, grads, max_norm, out, st);
  return norm_all<float, float>(o, grads, max_norm, out, st);
}

cgtp_status cgtp_adamw_state_values(cgtp_adamw o, const void* m, const void* v, const void* m_exp, const void* v_exp,
                                    float* m_out, float* v_out, void* stream) {
  clear_error();
  if (!o) return fail(CGTP_EINVAL, "null optimizer");
  if (o->state != CGTP_STATE_8BIT) return fail(CGTP_EUNSUPPORTED, "the states are not 8-bit codes");
  const int64_t n4 = o->begin.back() * (kBlock / 4);
  if (n4 == 0) return CGTP_OK;
  cgtp_status s;
  if ((s = buffer(m, "m")) || (s = buffer(v, "v")) || (s = buffer(m_out, "m_out")) || (s = buffer(v_out, "v_out"))) return s;
  if (!m_exp || !v_exp) return fail(CGTP_EINVAL, "null pointer: m_exp or v_exp");
  const unsigned ctas = static_cast<unsigned>((n4 + kStepThreads - 1) / kStepThreads);
  return launched(chain_launch(state_values_kernel, ctas, kStepThreads, 0, static_cast<cudaStream_t>(stream), m, v, m_exp, v_exp, m_out,
                               v_out, n4),
                  "optimizer state values");
}

}  // extern "C"
