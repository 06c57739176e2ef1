// resnorm.cu -- the gated residual norm's plan, argument checks and launches
// (declared in include/cgtp_train.h; kernels in resnorm_impl.cuh).
#include <cuda_runtime.h>

#include <algorithm>
#include <cmath>
#include <new>
#include <string>

#include "resnorm.h"

namespace cgtp {
namespace {

int es_stream(const cgtp_resnorm_s* p) {
  return p->dtype == CGTP_F64 ? 8 : p->dtype == CGTP_BF16 && (p->flags & CGTP_RESNORM_STORAGE) ? 2 : 4;
}
int es_go(const cgtp_resnorm_s* p) { return p->dtype == CGTP_F64 ? 8 : p->dtype == CGTP_BF16 ? 2 : 4; }
int es_param(const cgtp_resnorm_s* p) { return p->dtype == CGTP_F64 ? 8 : 4; }

// one row tensor: element alignment and a row distance of at least `width` (0: contiguous)
cgtp_status rows(const void* ptr, int64_t* ld, int64_t width, int es, const char* name) {
  if (!ptr) return CGTP_OK;
  if (reinterpret_cast<uintptr_t>(ptr) % es) return fail(CGTP_EINVAL, std::string("pointer not aligned to its element: ") + name);
  if (*ld == 0) *ld = width;
  if (*ld < width) return fail(CGTP_EINVAL, std::string("rows overlap (row distance below the row length): ") + name);
  return CGTP_OK;
}

cgtp_status param(const void* ptr, int es, const char* name) {
  if (reinterpret_cast<uintptr_t>(ptr) % es) return fail(CGTP_EINVAL, std::string("pointer not aligned to its element: ") + name);
  return CGTP_OK;
}

int ctas_for(const cgtp_resnorm_s* p, int64_t N) {
  const int teams = kRnThreads / p->team;
  return static_cast<int>(std::min<int64_t>((N + teams - 1) / teams, p->teams_max / teams));
}

RnArgs base_args(const cgtp_resnorm_s* p, int64_t N) {
  RnArgs a;
  a.N = N;
  a.blocks = p->blocks_dev;
  a.n_blocks = static_cast<int>(p->blocks.size());
  a.dim = static_cast<int>(p->dim);
  a.chan = static_cast<int>(p->chan);
  a.act = p->act;
  a.team = p->team;
  a.pre_norm = p->flags & CGTP_RESNORM_PRE;
  a.post_norm = p->flags & CGTP_RESNORM_POST;
  a.alpha = p->alpha;
  a.eps = p->eps;
  a.part = p->part;
  return a;
}

cgtp_status launch(const cgtp_resnorm_s* p, const RnArgs& a, bool backward, int ctas, cudaStream_t st) {
  const cudaError_t e = p->dtype == CGTP_F64                          ? rn_launch_f64(a, backward, ctas, st)
                        : p->dtype == CGTP_F32                        ? rn_launch_f32(a, backward, ctas, st)
                        : (p->flags & CGTP_RESNORM_STORAGE)           ? rn_launch_bf16s(a, backward, ctas, st)
                                                                      : rn_launch_bf16(a, backward, ctas, st);
  return e == cudaSuccess ? CGTP_OK : fail(CGTP_ECUDA, std::string("resnorm: ") + cudaGetErrorString(e));
}

cgtp_status create(cgtp_resnorm_s* p, const char* irreps) {
  std::vector<Irrep> ir;
  std::string err;
  if (!parse_irreps(irreps, &ir, &err)) return fail(CGTP_EINVAL, err);
  int widest = 1;
  for (const Irrep& i : ir) {
    if (i.mul < 1) return fail(CGTP_EINVAL, "irreps blocks of a norm must have a channel");
    p->blocks.push_back({static_cast<int>(p->dim), static_cast<int>(p->chan), i.mul, 2 * i.l + 1});
    p->dim += int64_t(i.mul) * (2 * i.l + 1);
    p->chan += i.mul;
    widest = std::max(widest, i.mul);
    if (p->dim > (1 << 20)) return fail(CGTP_EUNSUPPORTED, "rows of more than 1048576 elements");
  }
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess ||
      cudaDeviceGetAttribute(&p->num_sms, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess) {
    cudaGetLastError();
    return fail(CGTP_ECUDA, "no CUDA device");
  }
  p->team = 1;
  while (p->team < 32 && p->team < widest) p->team *= 2;
  if (p->dim > 4096) p->team = kRnThreads;
  p->teams_max = p->num_sms * 8 * (kRnThreads / p->team);
  const size_t tab = p->blocks.size() * sizeof(RnBlock);
  const size_t part = size_t(p->teams_max) * 2 * p->chan * es_param(p);
  if (cudaMalloc(reinterpret_cast<void**>(&p->blocks_dev), tab) != cudaSuccess || cudaMalloc(&p->part, part) != cudaSuccess) {
    cudaGetLastError();
    return fail(CGTP_ENOMEM, "norm table allocation failed");
  }
  p->device_bytes = tab + part;
  if (cudaMemcpy(p->blocks_dev, p->blocks.data(), tab, cudaMemcpyHostToDevice) != cudaSuccess) {
    cudaGetLastError();
    return fail(CGTP_ECUDA, "norm table upload failed");
  }
  return CGTP_OK;
}

}  // namespace
}  // namespace cgtp

using namespace cgtp;

extern "C" {

cgtp_status cgtp_resnorm_create(cgtp_resnorm* out, const char* irreps, int dtype, int flags, int act, double alpha,
                                double eps) {
  clear_error();
  if (!out) return fail(CGTP_EINVAL, "null plan output pointer");
  *out = nullptr;
  if (dtype != CGTP_F32 && dtype != CGTP_F64 && dtype != CGTP_BF16)
    return fail(CGTP_EINVAL, "dtype must be CGTP_F32, CGTP_F64 or CGTP_BF16");
  if (flags & ~(CGTP_RESNORM_POST | CGTP_RESNORM_PRE | CGTP_RESNORM_STORAGE)) return fail(CGTP_EINVAL, "unknown flag");
  if (act < CGTP_ACT_NONE || act > CGTP_ACT_SILU) return fail(CGTP_EINVAL, "unknown gate activation");
  if (!(eps >= 0.0) || !std::isfinite(eps) || !std::isfinite(alpha)) return fail(CGTP_EINVAL, "eps must be >= 0, alpha and eps finite");
  cgtp_resnorm_s* p = new (std::nothrow) cgtp_resnorm_s();
  if (!p) return fail(CGTP_ENOMEM, "host allocation failed");
  p->dtype = dtype;
  p->flags = flags;
  p->act = act;
  p->alpha = alpha;
  p->eps = eps;
  cgtp_status s;
  try {
    s = create(p, irreps);
  } catch (const std::bad_alloc&) {
    s = fail(CGTP_ENOMEM, "host allocation failed");
  }
  if (s != CGTP_OK) {
    cgtp_resnorm_destroy(p);
    return s;
  }
  *out = p;
  return CGTP_OK;
}

void cgtp_resnorm_destroy(cgtp_resnorm p) {
  if (!p) return;
  if (p->blocks_dev) cudaFree(p->blocks_dev);
  if (p->part) cudaFree(p->part);
  delete p;
}

cgtp_status cgtp_resnorm_info(cgtp_resnorm p, int64_t* dim, int64_t* channels, int* blocks) {
  clear_error();
  if (!p) return fail(CGTP_EINVAL, "null plan");
  if (dim) *dim = p->dim;
  if (channels) *channels = p->chan;
  if (blocks) *blocks = static_cast<int>(p->blocks.size());
  return CGTP_OK;
}

cgtp_status cgtp_resnorm_device_bytes(cgtp_resnorm p, int64_t* bytes) {
  clear_error();
  if (!p || !bytes) return fail(CGTP_EINVAL, "null argument");
  *bytes = static_cast<int64_t>(p->device_bytes);
  return CGTP_OK;
}

cgtp_status cgtp_resnorm_forward(cgtp_resnorm p, int64_t N, const void* h, int64_t ld_h, const void* z, int64_t ld_z,
                                 const void* q, int64_t ld_q, const void* post, const void* scale, const void* pre,
                                 void* out, int64_t ld_out, void* y, int64_t ld_y, void* stream) {
  clear_error();
  if (!p) return fail(CGTP_EINVAL, "null plan");
  if (N < 0) return fail(CGTP_EINVAL, "N must be >= 0");
  RnArgs a = base_args(p, N);
  if (N > 0) {
    if (!z && !h) return fail(CGTP_EINVAL, "null pointer: h and z");
    if (!z && out) return fail(CGTP_EINVAL, "out needs z (without it the stream is h)");
    if (z && !out) return fail(CGTP_EINVAL, "null pointer: out");
    if (a.pre_norm != (y != nullptr)) return fail(CGTP_EINVAL, "y is written exactly with CGTP_RESNORM_PRE");
    if (!z && !y) return fail(CGTP_EINVAL, "nothing to compute: neither z nor y");
    if (z && p->act != CGTP_ACT_NONE && !q) return fail(CGTP_EINVAL, "null pointer: q");
  }
  const int es = es_stream(p), go = es_go(p), ep = es_param(p);
  cgtp_status s;
  if ((s = rows(h, &ld_h, p->dim, es, "h")) || (s = rows(z, &ld_z, p->dim, es, "z")) ||
      (s = rows(q, &ld_q, p->chan, es, "q")) || (s = rows(out, &ld_out, p->dim, es, "out")) ||
      (s = rows(y, &ld_y, p->dim, go, "y")) || (s = param(post, ep, "post")) || (s = param(scale, ep, "scale")) ||
      (s = param(pre, ep, "pre")))
    return s;
  if (N == 0) return CGTP_OK;
  a.h = h, a.ld_h = ld_h;
  a.z = z, a.ld_z = ld_z;
  a.q = z && p->act != CGTP_ACT_NONE ? q : nullptr, a.ld_q = ld_q;
  a.post = post, a.scale = scale, a.pre = pre;
  a.out = out, a.ld_out = ld_out;
  a.y = y, a.ld_y = ld_y;
  return launch(p, a, false, ctas_for(p, N), static_cast<cudaStream_t>(stream));
}

cgtp_status cgtp_resnorm_backward(cgtp_resnorm p, int64_t N, const void* gout, int64_t ld_gout, const void* gy,
                                  int64_t ld_gy, const void* x, int64_t ld_x, const void* z, int64_t ld_z,
                                  const void* q, int64_t ld_q, const void* post, const void* scale, const void* pre,
                                  void* gh, int64_t ld_gh, void* gz, int64_t ld_gz, void* gq, int64_t ld_gq,
                                  void* gpost, void* gscale, void* gpre, void* stream) {
  clear_error();
  if (!p) return fail(CGTP_EINVAL, "null plan");
  if (N < 0) return fail(CGTP_EINVAL, "N must be >= 0");
  RnArgs a = base_args(p, N);
  const bool gated = z && p->act != CGTP_ACT_NONE;
  if (N > 0) {
    if (a.pre_norm != (gy != nullptr)) return fail(CGTP_EINVAL, "gy is read exactly with CGTP_RESNORM_PRE");
    if (a.pre_norm && !x) return fail(CGTP_EINVAL, "null pointer: x");
    if (!gout && !gy) return fail(CGTP_EINVAL, "null pointer: gout and gy");
    if (gated && !q) return fail(CGTP_EINVAL, "null pointer: q");
    if ((z != nullptr) != (gz != nullptr)) return fail(CGTP_EINVAL, "gz is written exactly when z is given");
    if (gated != (gq != nullptr)) return fail(CGTP_EINVAL, "gq is written exactly when q is read");
  }
  const int es = es_stream(p), go = es_go(p), ep = es_param(p);
  cgtp_status s;
  if ((s = rows(gout, &ld_gout, p->dim, es, "gout")) || (s = rows(gy, &ld_gy, p->dim, es, "gy")) ||
      (s = rows(x, &ld_x, p->dim, es, "x")) || (s = rows(z, &ld_z, p->dim, es, "z")) ||
      (s = rows(q, &ld_q, p->chan, es, "q")) || (s = rows(gh, &ld_gh, p->dim, es, "gh")) ||
      (s = rows(gz, &ld_gz, p->dim, go, "gz")) || (s = rows(gq, &ld_gq, p->chan, go, "gq")) ||
      (s = param(post, ep, "post")) || (s = param(scale, ep, "scale")) || (s = param(pre, ep, "pre")) ||
      (s = param(gpost, ep, "gpost")) || (s = param(gscale, ep, "gscale")) || (s = param(gpre, ep, "gpre")))
    return s;
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  if (N == 0) {
    for (void* g : {gpost, gscale, gpre})
      if (g && cudaMemsetAsync(g, 0, p->chan * ep, st) != cudaSuccess) {
        cudaGetLastError();
        return fail(CGTP_ECUDA, "resnorm: clearing a parameter gradient failed");
      }
    return CGTP_OK;
  }
  a.gout = gout, a.ld_gout = ld_gout;
  a.gy = gy, a.ld_gy = ld_gy;
  a.x = x, a.ld_x = ld_x;
  a.z = z, a.ld_z = ld_z;
  a.q = gated ? q : nullptr, a.ld_q = ld_q;
  a.post = post, a.scale = scale, a.pre = pre;
  a.gh = gh, a.ld_gh = ld_gh;
  a.gz = gz, a.ld_gz = ld_gz;
  a.gq = gated ? gq : nullptr, a.ld_gq = ld_gq;
  a.gpost = gpost, a.gscale = gscale, a.gpre = gpre;
  return launch(p, a, true, ctas_for(p, N), st);
}

}  // extern "C"
