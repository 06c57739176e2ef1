// adamw.cu -- AdamW over many tensors, with states in the parameters' type or in 8 bits, and
// the global gradient norm (declared in include/cgtp_train.h).
//
// Work is cut into blocks of 128 elements, numbered over all tensors; a warp takes a block, a
// lane 4 elements of it.  The tensors' pointers travel in the kernel's parameters.
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include <algorithm>
#include <cmath>
#include <new>
#include <string>
#include <vector>

#include "cgtp_train.h"
#include "internal.h"

struct cgtp_adamw_s {
  int param_dtype = 0, grad_dtype = 0, state = 0, num_sms = 0;
  std::vector<int64_t> numel, begin;   // begin[i]: first block of tensor i
  int64_t* begin_dev = nullptr;
  int64_t* numel_dev = nullptr;
  float* decay_dev = nullptr;
  double* part = nullptr;              // one partial sum of squares per CTA
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

struct Table {
  const int64_t *begin, *numel;
  const float* decay;
};

// pointers of tensors [t0, t0 + n)
template <int K>
struct Pointers {
  void* p[K];
  const void* g[K];
  void* c[K];
};

struct Scalars {
  double lr_decay, b1, one_b1, b2, one_b2, rate, root, eps;
  uint32_t key0, key1;
};

// index of the tensor that holds block k: the last one that begins at or before it
__device__ __forceinline__ int tensor_of(const int64_t* begin, int lo, int hi, int64_t k) {
  while (hi - lo > 1) {
    const int mid = (lo + hi) >> 1;
    if (__ldg(begin + mid) <= k) lo = mid;
    else hi = mid;
  }
  return lo;
}

// 32 pseudo-random bits of element i: a Weyl step and two multiply-xorshift rounds
__device__ __forceinline__ uint32_t noise_of(uint64_t i, uint32_t key0, uint32_t key1) {
  uint32_t x = static_cast<uint32_t>(i) * 0x9E3779B1u + static_cast<uint32_t>(i >> 32) * 0x85A308D3u + key0;
  x = (x ^ (x >> 15)) * 0xBB67AE85u;
  x = (x ^ (x >> 13)) * 0x3C6EF373u + key1;
  return x ^ (x >> 16);
}

// A code of a block with exponent E and largest exponent field TOP stands for
//   field f > 0:  2^(E - TOP + f - 127) (1 + mantissa / 8),   field 0:  mantissa 2^(E - TOP + 1 - 130).
template <int TOP>
__device__ __forceinline__ float code_value(uint32_t code, int E) {
  const int base = max(E, kEMin) - TOP;
  const float low = static_cast<float>(code) * __uint_as_float(static_cast<uint32_t>(base - 2) << 23);
  const float v = code >= 8 ? __uint_as_float((static_cast<uint32_t>(base) << 23) + (code << 20)) : low;
  return E == kENan ? __uint_as_float(0x7FC00000u) : v;
}

// The code of x >= 0, rounded up with probability = its distance above the code below it; r: 20 random bits.
// E leaves room for the largest value of the block to be rounded up.
template <int TOP>
__device__ __forceinline__ uint32_t code_of(float x, int E, uint32_t r) {
  const int base = E - TOP;
  const uint32_t bits = __float_as_uint(x);
  const float fine = x * __uint_as_float(static_cast<uint32_t>(256 - base) << 23);
  const uint32_t low = static_cast<uint32_t>(floorf(__fadd_rn(fine, static_cast<float>(r) * 9.5367431640625e-7f)));
  return bits >= (static_cast<uint32_t>(base + 1) << 23) ? ((bits + r) >> 20) - (static_cast<uint32_t>(base) << 3) : low;
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
// the 8-bit states do not depend on how the compiler pairs them.
__device__ __forceinline__ float mul_rn(float a, float b) { return __fmul_rn(a, b); }
__device__ __forceinline__ double mul_rn(double a, double b) { return __dmul_rn(a, b); }
__device__ __forceinline__ float add_rn(float a, float b) { return __fadd_rn(a, b); }
__device__ __forceinline__ double add_rn(double a, double b) { return __dadd_rn(a, b); }

template <typename A, typename G, bool EIGHT, int K>
__global__ void __launch_bounds__(kStepThreads) adamw_kernel(const __grid_constant__ Pointers<K> ptrs, const Table tab, int t0,
                                                         int n, int64_t k0, int64_t k1, void* m_, void* v_, uint8_t* m_exp,
                                                         uint8_t* v_exp, const Scalars s, const A* clip) {
  const int lane = threadIdx.x & 31;
  const int64_t k = k0 + (int64_t)blockIdx.x * kWarpsPerCta + (threadIdx.x >> 5);
  if (k >= k1) return;
  const A coef = clip ? __ldg(clip + 1) : A(1);
  if (!isfinite(coef)) return;
  const int t = tensor_of(tab.begin, t0, t0 + n, k);
  const int64_t at = (k - __ldg(tab.begin + t)) * kBlock + lane * 4;
  const int64_t left = __ldg(tab.numel + t) - at;
  const G* g = static_cast<const G*>(ptrs.g[t - t0]);
  if (!g) return;
  A* p = static_cast<A*>(ptrs.p[t - t0]) + at;
  g += at;
  const int64_t place = k * kBlock + lane * 4;
  A pv[4], gv[4], mv[4], vv[4];
  load4<A, A>(p, left, wide_ok(p), pv);
  load4<G, A>(g, left, wide_ok(g), gv);
  if constexpr (EIGHT) {
    const uint32_t mc = *reinterpret_cast<const uint32_t*>(static_cast<const uint8_t*>(m_) + place);
    const uint32_t vc = *reinterpret_cast<const uint32_t*>(static_cast<const uint8_t*>(v_) + place);
    const int me = m_exp[k], ve = v_exp[k];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const float a = code_value<kMTop>(mc >> (8 * i) & 127u, me);
      mv[i] = mc >> (8 * i) & 128u ? -a : a;
      vv[i] = code_value<kVTop>(vc >> (8 * i) & 255u, ve);
    }
  } else {
    load4<A, A>(static_cast<const A*>(m_) + place, 4, true, mv);
    load4<A, A>(static_cast<const A*>(v_) + place, 4, true, vv);
  }
  const A keep = A(1) - static_cast<A>(s.lr_decay) * static_cast<A>(__ldg(tab.decay + t));
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const A gi = mul_rn(gv[i], coef);
    mv[i] = add_rn(mul_rn(mv[i], static_cast<A>(s.b1)), mul_rn(gi, static_cast<A>(s.one_b1)));
    vv[i] = add_rn(mul_rn(vv[i], static_cast<A>(s.b2)), mul_rn(mul_rn(gi, gi), static_cast<A>(s.one_b2)));
    pv[i] = pv[i] * keep - static_cast<A>(s.rate) * mv[i] / (sqrt(vv[i]) * static_cast<A>(s.root) + static_cast<A>(s.eps));
  }
  store4<A, A>(p, left, wide_ok(p), pv);
  if constexpr (sizeof(A) == 4) {
    if (ptrs.c[t - t0]) {
      __nv_bfloat16* c = static_cast<__nv_bfloat16*>(ptrs.c[t - t0]) + at;
      store4<__nv_bfloat16, A>(c, left, wide_ok(c), pv);
    }
  }
  if constexpr (EIGHT) {
    uint32_t mb = 0, vb = 0;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      if (i >= left) mv[i] = vv[i] = 0.0f;   // the place behind the tensor's end
      mb = max(mb, __float_as_uint(mv[i]) & 0x7FFFFFFFu);
      vb = max(vb, __float_as_uint(vv[i]) & 0x7FFFFFFFu);
    }
    const int me = block_exponent(__reduce_max_sync(0xffffffffu, mb));
    const int ve = block_exponent(__reduce_max_sync(0xffffffffu, vb));
    uint32_t mc = 0, vc = 0;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const uint32_t r = noise_of(static_cast<uint64_t>(place + i), s.key0, s.key1);
      const uint32_t a = code_of<kMTop>(fabsf(mv[i]), me, (r >> 16) << 4) | (mv[i] < 0.0f ? 128u : 0u);
      uint32_t b = code_of<kVTop>(vv[i], ve, (r & 0xFFFFu) << 4);
      b = vv[i] > 0.0f ? max(b, 1u) : b;
      mc |= a << (8 * i);
      vc |= b << (8 * i);
    }
    if (me >= kENan) mc = 0;
    if (ve >= kENan) vc = 0;
    *reinterpret_cast<uint32_t*>(static_cast<uint8_t*>(m_) + place) = mc;
    *reinterpret_cast<uint32_t*>(static_cast<uint8_t*>(v_) + place) = vc;
    if (lane == 0) {
      m_exp[k] = static_cast<uint8_t>(min(me, kENan));
      v_exp[k] = static_cast<uint8_t>(min(ve, kENan));
    }
  } else {
    store4<A, A>(static_cast<A*>(m_) + place, left, true, mv);
    store4<A, A>(static_cast<A*>(v_) + place, left, true, vv);
  }
}

__global__ void __launch_bounds__(kStepThreads) state_values_kernel(const uint8_t* m, const uint8_t* v, const uint8_t* m_exp,
                                                                const uint8_t* v_exp, float* m_out, float* v_out, int64_t n4) {
  const int64_t i = (int64_t)blockIdx.x * kStepThreads + threadIdx.x;
  if (i >= n4) return;
  const uint32_t mc = reinterpret_cast<const uint32_t*>(m)[i], vc = reinterpret_cast<const uint32_t*>(v)[i];
  const int me = m_exp[i >> 5], ve = v_exp[i >> 5];
  float a[4], b[4];
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    const float t = code_value<kMTop>(mc >> (8 * j) & 127u, me);
    a[j] = mc >> (8 * j) & 128u ? -t : t;
    b[j] = code_value<kVTop>(vc >> (8 * j) & 255u, ve);
  }
  reinterpret_cast<float4*>(m_out)[i] = make_float4(a[0], a[1], a[2], a[3]);
  reinterpret_cast<float4*>(v_out)[i] = make_float4(b[0], b[1], b[2], b[3]);
}

__device__ __forceinline__ double cta_sum(double v) {
  __shared__ double warp_sum[kWarpsPerCta];
  for (int o = 16; o; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
  if ((threadIdx.x & 31) == 0) warp_sum[threadIdx.x >> 5] = v;
  __syncthreads();
  double t = 0.0;
  for (int w = 0; w < kWarpsPerCta; ++w) t += warp_sum[w];
  return t;
}

// sum of squares of the CTA's blocks: a thread's own in A, the rest in FP64
template <typename A, typename G, int K>
__global__ void __launch_bounds__(kStepThreads) square_sum_kernel(const __grid_constant__ Pointers<K> ptrs, const Table tab, int t0,
                                                              int n, int64_t k0, int64_t k1, double* part) {
  const int lane = threadIdx.x & 31;
  A sum = A(0);
  for (int64_t k = k0 + (int64_t)blockIdx.x * kWarpsPerCta + (threadIdx.x >> 5); k < k1; k += (int64_t)gridDim.x * kWarpsPerCta) {
    const int t = tensor_of(tab.begin, t0, t0 + n, k);
    const G* g = static_cast<const G*>(ptrs.g[t - t0]);
    if (!g) continue;
    const int64_t at = (k - __ldg(tab.begin + t)) * kBlock + lane * 4;
    A v[4];
    load4<G, A>(g + at, __ldg(tab.numel + t) - at, wide_ok(g + at), v);
#pragma unroll
    for (int i = 0; i < 4; ++i) sum += v[i] * v[i];
  }
  const double total = cta_sum(static_cast<double>(sum));
  if (threadIdx.x == 0) part[blockIdx.x] = total;
}

template <typename A>
__global__ void __launch_bounds__(kStepThreads) norm_kernel(const double* part, int count, double max_norm, A* out) {
  double v = 0.0;
  for (int i = threadIdx.x; i < count; i += kStepThreads) v += part[i];
  v = cta_sum(v);
  if (threadIdx.x != 0) return;
  const double norm = sqrt(v);
  out[0] = static_cast<A>(norm);
  out[1] = isfinite(norm) ? static_cast<A>(norm > max_norm ? max_norm / norm : 1.0) : static_cast<A>(nan(""));
}

constexpr int kMostTensors = 1024, kFewTensors = 64;
constexpr int kNormCtasPerSm = 8;

cgtp_status launched(const char* what) {
  const cudaError_t e = cudaGetLastError();
  return e == cudaSuccess ? CGTP_OK : fail(CGTP_ECUDA, std::string(what) + ": " + cudaGetErrorString(e));
}

Table table(const cgtp_adamw_s* o) { return {o->begin_dev, o->numel_dev, o->decay_dev}; }

template <int K>
void fill(Pointers<K>* a, int t0, int n, void* const* params, const void* const* grads, void* const* copies) {
  for (int i = 0; i < n; ++i) {
    a->p[i] = params ? params[t0 + i] : nullptr;
    a->g[i] = grads[t0 + i];
    a->c[i] = copies ? copies[t0 + i] : nullptr;
  }
}

struct StepArgs {
  void *m, *v;
  uint8_t *m_exp, *v_exp;
  Scalars s;
  const void* clip;
};

template <typename A, typename G, bool EIGHT, int K>
cgtp_status step_launch(const cgtp_adamw_s* o, int t0, int n, void* const* params, const void* const* grads,
                        void* const* copies, const StepArgs& a, cudaStream_t st) {
  Pointers<K> ptrs;
  fill(&ptrs, t0, n, params, grads, copies);
  const int64_t k0 = o->begin[t0], k1 = o->begin[t0 + n];
  if (k1 == k0) return CGTP_OK;
  const int64_t ctas = (k1 - k0 + kWarpsPerCta - 1) / kWarpsPerCta;
  adamw_kernel<A, G, EIGHT, K><<<static_cast<unsigned>(ctas), kStepThreads, 0, st>>>(
      ptrs, table(o), t0, n, k0, k1, a.m, a.v, a.m_exp, a.v_exp, a.s, static_cast<const A*>(a.clip));
  return launched("adamw step");
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

template <typename A, typename G, int K>
cgtp_status norm_launch(const cgtp_adamw_s* o, int t0, int n, const void* const* grads, int ctas, double* part,
                        cudaStream_t st) {
  Pointers<K> ptrs;
  fill(&ptrs, t0, n, nullptr, grads, nullptr);
  square_sum_kernel<A, G, K><<<ctas, kStepThreads, 0, st>>>(ptrs, table(o), t0, n, o->begin[t0], o->begin[t0 + n], part);
  return launched("gradient norm");
}

template <typename A, typename G>
cgtp_status norm_all(const cgtp_adamw_s* o, const void* const* grads, double max_norm, void* out, cudaStream_t st) {
  const int all = static_cast<int>(o->numel.size());
  int count = 0;
  for (int t0 = 0; t0 < all; t0 += kMostTensors) {
    const int n = std::min(kMostTensors, all - t0);
    const int64_t blocks = o->begin[t0 + n] - o->begin[t0];
    const int ctas = static_cast<int>(std::max<int64_t>(
        1, std::min<int64_t>((blocks + kWarpsPerCta - 1) / kWarpsPerCta, o->num_sms * kNormCtasPerSm)));
    const cgtp_status s = n <= kFewTensors ? norm_launch<A, G, kFewTensors>(o, t0, n, grads, ctas, o->part + count, st)
                                           : norm_launch<A, G, kMostTensors>(o, t0, n, grads, ctas, o->part + count, st);
    if (s != CGTP_OK) return s;
    count += ctas;
  }
  norm_kernel<A><<<1, kStepThreads, 0, st>>>(o->part, count, max_norm, static_cast<A*>(out));
  return launched("gradient norm");
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
  const std::vector<float> decay = decay_scale ? std::vector<float>(decay_scale, decay_scale + n) : std::vector<float>(n, 1.0f);
  const size_t parts = size_t(o->num_sms) * kNormCtasPerSm * ((n + kMostTensors - 1) / kMostTensors);
  const size_t b_begin = (n + 1) * sizeof(int64_t), b_numel = n * sizeof(int64_t), b_part = parts * sizeof(double);
  const size_t bytes = b_begin + b_numel + b_part + n * sizeof(float);
  if (cudaMalloc(&o->base, bytes) != cudaSuccess) {
    cudaGetLastError();
    return fail(CGTP_ENOMEM, "optimizer table allocation failed");
  }
  o->device_bytes = bytes;
  unsigned char* at = static_cast<unsigned char*>(o->base);
  o->begin_dev = reinterpret_cast<int64_t*>(at);
  o->numel_dev = reinterpret_cast<int64_t*>(at + b_begin);
  o->part = reinterpret_cast<double*>(at + b_begin + b_numel);
  o->decay_dev = reinterpret_cast<float*>(at + b_begin + b_numel + b_part);
  if (cudaMemcpy(o->begin_dev, o->begin.data(), b_begin, cudaMemcpyHostToDevice) != cudaSuccess ||
      cudaMemcpy(o->numel_dev, o->numel.data(), b_numel, cudaMemcpyHostToDevice) != cudaSuccess ||
      cudaMemcpy(o->decay_dev, decay.data(), n * sizeof(float), cudaMemcpyHostToDevice) != cudaSuccess) {
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
  StepArgs a{m, v, static_cast<uint8_t*>(m_exp), static_cast<uint8_t*>(v_exp),
             Scalars{lr * weight_decay, beta1, 1.0 - beta1, beta2, 1.0 - beta2, lr / (1.0 - std::pow(beta1, t)),
                     1.0 / std::sqrt(1.0 - std::pow(beta2, t)), eps, static_cast<uint32_t>(key),
                     static_cast<uint32_t>(key >> 32)},
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
  state_values_kernel<<<ctas, kStepThreads, 0, static_cast<cudaStream_t>(stream)>>>(
      static_cast<const uint8_t*>(m), static_cast<const uint8_t*>(v), static_cast<const uint8_t*>(m_exp),
      static_cast<const uint8_t*>(v_exp), m_out, v_out, n4);
  return launched("optimizer state values");
}

}  // extern "C"
