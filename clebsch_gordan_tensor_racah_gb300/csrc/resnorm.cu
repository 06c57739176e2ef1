// resnorm.cu -- the gated residual norm's plan, argument checks and launches
// (declared in include/cgtp_train.h; kernels in resnorm_impl.cuh).
#include <cuda_runtime.h>

#include <algorithm>
#include <cmath>
#include <cstring>
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

RnArgs base_args(const cgtp_resnorm_s* p, int64_t N) {
  RnArgs a;
  a.N = N;
  a.blocks = p->blocks_dev;
  a.n_blocks = static_cast<int>(p->blocks.size());
  std::copy(p->blocks.begin(), p->blocks.begin() + std::min<size_t>(p->blocks.size(), kRnInline), a.few);
  a.dim = static_cast<int>(p->dim);
  a.chan = static_cast<int>(p->chan);
  a.act = p->act;
  a.pre_norm = p->flags & CGTP_RESNORM_PRE;
  a.post_norm = p->flags & CGTP_RESNORM_POST;
  a.alpha = p->alpha;
  a.eps = p->eps;
  a.alpha_f = static_cast<float>(p->alpha);
  a.eps_f = static_cast<float>(p->eps);
  a.part = p->part;
  return a;
}

void set(RnRows* r, const void* ptr, int64_t ld, int64_t width, int es) {
  r->ptr = const_cast<char*>(static_cast<const char*>(ptr));
  r->ld = ld;
  r->ld_bytes = ld * es;
  r->width = static_cast<int>(width);
  r->es = es;
}

// widest copy (16, 8, 4 or 2 bytes) that divides every offset in `bits`
int widest_copy(uint64_t bits) { return bits % 16 == 0 ? 16 : bits % 8 == 0 ? 8 : bits % 4 == 0 ? 4 : 2; }

int round16(int64_t v) { return static_cast<int>((v + 15) / 16 * 16); }

// Regions of a stage for tiles of `rows` rows.  An input whose rows lie side by side keeps that
// layout (one run of bytes a tile); other rows start at multiples of 16 bytes.  A result takes
// the region of an operand that is dead, element by element, when it is written (see the kernels).
int lay_out(RnArgs* a, bool backward, int rows) {
  int at = 0;
  const auto own = [&](RnRows* r) {
    const int dense = r->width * r->es;
    r->linear = r->ld == r->width;
    r->pitch = r->linear ? dense : round16(dense);
    r->at = at;
    at = round16(at + int64_t(rows) * r->pitch);
  };
  const auto over = [&](RnRows* r, const RnRows& in) {
    r->at = in.at;
    r->pitch = in.pitch;
    r->linear = r->ld == r->width && r->pitch == r->width * r->es;
  };
  RnRows* t = a->t;
  for (int i = 0; i < kRnInputs[backward]; ++i)
    if (t[i].ptr) own(&t[i]);
  if (!backward) {
    if (t[kRnOut].ptr) over(&t[kRnOut], t[kRnH].ptr ? t[kRnH] : t[kRnZ]);
    if (t[kRnY].ptr) {
      if (t[kRnZ].ptr && t[kRnH].ptr) over(&t[kRnY], t[kRnZ]);
      else if (!t[kRnZ].ptr && t[kRnY].es == t[kRnH].es) over(&t[kRnY], t[kRnH]);
      else own(&t[kRnY]);
    }
  } else {
    if (t[kRnGh].ptr) {
      if (t[kRnGout].ptr) over(&t[kRnGh], t[kRnGout]);
      else own(&t[kRnGh]);
    }
    if (t[kRnGz].ptr) {
      if (t[kRnGy].ptr && t[kRnGz].es == t[kRnGy].es) over(&t[kRnGz], t[kRnGy]);
      else own(&t[kRnGz]);
    }
    if (t[kRnGq].ptr) {
      if (t[kRnGq].es == t[kRnBq].es) over(&t[kRnGq], t[kRnBq]);
      else own(&t[kRnGq]);
    }
  }
  for (int i = 0; i < (backward ? kRnBackward : kRnForward); ++i) {
    RnRows& r = t[i];
    if (!r.ptr) continue;
    uint64_t bits = reinterpret_cast<uintptr_t>(r.ptr) | uint64_t(r.ld) * r.es * (r.linear ? rows : 1);
    if (!r.linear) bits |= r.pitch;
    r.vec = widest_copy(bits);
  }
  return at;
}

// How rows are dealt out (see resnorm_impl.cuh): the cheapest of the launches that fit, by the
// instructions that a row costs and the warps that hide their latency.
//   instructions: an element of a thread's share, a channel, a step of the block sums and the fixed part of a
//     block, fitted to counters of the kernels (a row of 64x0e+64x1o+64x2e: 1,328 backward, 885 forward);
//     half as many again where operands are missing, blocks do not fill the lanes or copies are ragged.
//   rate: grows with the warps of an SM as w / (w + 8).
// Measured on both sides (GB300, share of the copy bandwidth):
//   threads a row: 32x0e+32x1o+32x2e+32x3o, 200,000 rows: 32 threads 96% / 90% (forward / backward), 16 threads
//     90% / 81%; 8x0e+8x1o, 2,000,000 rows: 8 threads 44% / 46%, 4 threads 57% / 49%, 2 threads 35% / 28% (16
//     rows a warp start in the same bank: 4 threads are the fewest); 33x0e+17x1o+5x2e forward: 32 threads 21%, 16
//     threads 28%, 8 threads 46%; 128x0e+128x1o+128x2e backward, 60,000 rows: 32 threads 90%, 64 threads 74%.
//   stages: two where that leaves as many warps, else one: 64x0e+64x1o+64x2e forward, 200,000 rows: two 100%, one 83%;
//     128x0e+128x1o+128x2e backward: two (4 warps) 62%, one (9 warps) 90%.
void deal(const cgtp_resnorm_s* p, RnArgs* a, bool backward) {
  const int n_rows = backward ? kRnBackward : kRnForward, ep = es_param(p);
  const bool listed = p->blocks.size() <= kRnInline;
  const int factors = round16(2 * p->chan * ep) + (listed ? 0 : round16(p->blocks.size() * sizeof(RnBlock)));
  double best = 0.0;
  int fewest = 1;
  while (fewest < 4 && fewest < p->widest) fewest *= 2;
  for (int team = fewest; team <= 32 * kRnWarps; team *= 2) {   // threads of a row
    const int warps = std::max(1, team / 32), abreast = std::max(1, 32 / team);
    if (team > fewest && team >= 2 * p->widest) break;
    // Rows of a tile: as many as run side by side, and enough that a tile of every contiguous tensor
    // starts at a multiple of 16 bytes.
    int rows = abreast;
    for (int i = 0; i < n_rows; ++i)
      while (a->t[i].ptr && a->t[i].ld == a->t[i].width && (int64_t(rows) * a->t[i].width * a->t[i].es) % 16) rows *= 2;
    bool held = true, fills = listed;
    double work = 0.0;
    for (const RnBlock& b : p->blocks) {
      const int share = rn_share(b.D, b.mul, team);
      held &= share > 0;
      fills &= b.mul == share * team;
      work += share * ((backward ? 15 : 9) * b.D + (backward ? 40 : 25)) + (backward ? 8 : 4) * std::log2(std::min(team, 32)) +
              (warps > 1 ? 120 : 0) + 40;
    }
    if (!held) continue;
    const int stage = lay_out(a, backward, rows);
    bool full = fills && a->pre_norm && a->post_norm;
    for (int i = 0; i < n_rows; ++i) full &= a->t[i].ptr && a->t[i].vec == 16 && (a->t[i].linear || rows == 1);
    const int64_t kept = (warps > 1 ? 8 * kRnWarps : 0) + (backward ? int64_t(abreast) * 2 * p->chan : 0);
    for (int stages = kRnMaxStages; stages >= 1; --stages) {
      const int64_t group = int64_t(stages) * stage + round16(kept * ep);
      const int groups = static_cast<int>(std::min<int64_t>((p->smem_cap - factors) / group, kRnWarps / warps));
      if (groups <= 0) continue;
      const int busy = groups * warps;
      const double rate = double(busy) / (busy + 8) / (work * warps / abreast * (!full ? 1.5 : team < 32 ? 1.35 : 1.0));
      if (rate <= best) continue;
      best = rate;
      a->kind = warps > 1 ? (full ? kRnManyFull : kRnMany) : !full ? kRnOne : team == 32 ? kRnOneFull : kRnFewFull;
      a->stages = stages;
      a->warps = warps;
      a->lanes = team;
      a->groups = groups;
      a->rows = rows;
      a->group_bytes = static_cast<int>(group);
    }
  }
  if (a->kind == kRnDirect) {
    a->ctas = static_cast<int>(std::min<int64_t>(a->N, int64_t(p->num_sms) * kRnCtasPerSm));
    return;
  }
  a->stage_bytes = lay_out(a, backward, a->rows);
  // as many turns of the grid as the tiles need, with no more groups than those turns keep busy
  const int64_t tiles = (a->N + a->rows - 1) / a->rows;
  const int64_t turns = (tiles + int64_t(p->num_sms) * a->groups - 1) / (int64_t(p->num_sms) * a->groups);
  // (a backward of so few rows runs in one CTA, whose sums are the sums over all rows)
  const bool one = backward && tiles <= a->groups;
  a->groups = static_cast<int>(one ? tiles : (tiles + p->num_sms * turns - 1) / (p->num_sms * turns));
  a->table_at = a->groups * a->group_bytes + round16(2 * p->chan * ep);
  a->smem = a->groups * a->group_bytes + factors;
  a->tiles = tiles;
  a->ctas = one ? 1 : static_cast<int>(std::min<int64_t>(a->tiles, p->num_sms));
  for (size_t i = 0; listed && i < p->blocks.size(); ++i)
    a->few[i].code = rn_code(a->few[i].D, rn_share(a->few[i].D, a->few[i].mul, a->lanes));
}

cgtp_status launch(const cgtp_resnorm_s* p, RnArgs& a, bool backward, cudaStream_t st) {
  deal(p, &a, backward);
  const int sums_smem = 33 * a.groups * a.warps * es_param(p);   // of the last CTA
  if (backward && a.kind != kRnDirect && (a.gpost || a.gscale || a.gpre) && a.ctas > 1 &&
      int64_t(a.ctas) * 2 * a.chan <= kRnTailSums &&
      sums_smem <= a.smem)
    a.ticket = p->ticket;
  const auto run = p->dtype == CGTP_F64                ? (backward ? rn_backward_f64 : rn_forward_f64)
                   : p->dtype == CGTP_F32              ? (backward ? rn_backward_f32 : rn_forward_f32)
                   : (p->flags & CGTP_RESNORM_STORAGE) ? (backward ? rn_backward_bf16s : rn_forward_bf16s)
                                                       : (backward ? rn_backward_bf16 : rn_forward_bf16);
  const cudaError_t e = run(a, st);
  return e == cudaSuccess ? CGTP_OK : fail(CGTP_ECUDA, std::string("resnorm: ") + cudaGetErrorString(e));
}

cgtp_status create(cgtp_resnorm_s* p, const char* irreps) {
  std::vector<Irrep> ir;
  std::string err;
  if (!parse_irreps(irreps, &ir, &err)) return fail(CGTP_EINVAL, err);
  for (const Irrep& i : ir) {
    if (i.mul < 1) return fail(CGTP_EINVAL, "irreps blocks of a norm must have a channel");
    const double inv_n = 1.0 / (double(i.mul) * (2 * i.l + 1));
    p->blocks.push_back({static_cast<int>(p->dim), static_cast<int>(p->chan), i.mul, 2 * i.l + 1, 0,
                         static_cast<float>(inv_n), inv_n});
    p->dim += int64_t(i.mul) * (2 * i.l + 1);
    p->chan += i.mul;
    p->widest = std::max(p->widest, i.mul);
    if (p->dim > (1 << 20)) return fail(CGTP_EUNSUPPORTED, "rows of more than 1048576 elements");
  }
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess ||
      cudaDeviceGetAttribute(&p->num_sms, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess ||
      cudaDeviceGetAttribute(&p->smem_cap, cudaDevAttrMaxSharedMemoryPerBlockOptin, dev) != cudaSuccess) {
    cudaGetLastError();
    return fail(CGTP_ECUDA, "no CUDA device");
  }
  p->smem_cap -= 512;   // the kernels' static shared memory
  // one allocation: the ticket, the block table, the partial sums
  const size_t tab = p->blocks.size() * sizeof(RnBlock), head = (16 + tab + 255) / 256 * 256;
  const size_t part = size_t(p->num_sms) * kRnCtasPerSm * 2 * p->chan * es_param(p);
  std::vector<char> table(16 + tab, 0);
  std::memcpy(table.data() + 16, p->blocks.data(), tab);
  if (cudaMalloc(&p->base, head + part) != cudaSuccess) {
    cudaGetLastError();
    return fail(CGTP_ENOMEM, "norm table allocation failed");
  }
  p->device_bytes = head + part;
  p->ticket = static_cast<unsigned*>(p->base);
  p->blocks_dev = reinterpret_cast<RnBlock*>(static_cast<char*>(p->base) + 16);
  p->part = static_cast<char*>(p->base) + head;
  if (!upload(p->base, table.data(), table.size())) {
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
  if (p->base) cudaFree(p->base);
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
  if (N >= (int64_t(1) << 30)) return fail(CGTP_EUNSUPPORTED, "N must be below 2^30");
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
  set(&a.t[kRnH], h, ld_h, p->dim, es);
  set(&a.t[kRnZ], z, ld_z, p->dim, es);
  set(&a.t[kRnQ], z && p->act != CGTP_ACT_NONE ? q : nullptr, ld_q, p->chan, es);
  set(&a.t[kRnOut], out, ld_out, p->dim, es);
  set(&a.t[kRnY], y, ld_y, p->dim, go);
  a.post = post, a.scale = scale, a.pre = pre;
  return launch(p, a, false, static_cast<cudaStream_t>(stream));
}

cgtp_status cgtp_resnorm_backward(cgtp_resnorm p, int64_t N, const void* gout, int64_t ld_gout, const void* gy,
                                  int64_t ld_gy, const void* x, int64_t ld_x, const void* z, int64_t ld_z,
                                  const void* q, int64_t ld_q, const void* post, const void* scale, const void* pre,
                                  void* gh, int64_t ld_gh, void* gz, int64_t ld_gz, void* gq, int64_t ld_gq,
                                  void* gpost, void* gscale, void* gpre, void* stream) {
  clear_error();
  if (!p) return fail(CGTP_EINVAL, "null plan");
  if (N < 0) return fail(CGTP_EINVAL, "N must be >= 0");
  if (N >= (int64_t(1) << 30)) return fail(CGTP_EUNSUPPORTED, "N must be below 2^30");
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
  if (!z) a.alpha = 1.0, a.alpha_f = 1.0f;   // the stream is h itself
  set(&a.t[kRnGout], gout, ld_gout, p->dim, es);
  set(&a.t[kRnGy], gy, ld_gy, p->dim, es);
  set(&a.t[kRnX], a.pre_norm ? x : nullptr, ld_x, p->dim, es);
  set(&a.t[kRnBz], z, ld_z, p->dim, es);
  set(&a.t[kRnBq], gated ? q : nullptr, ld_q, p->chan, es);
  set(&a.t[kRnGh], gh, ld_gh, p->dim, es);
  set(&a.t[kRnGz], gz, ld_gz, p->dim, go);
  set(&a.t[kRnGq], gq, ld_gq, p->chan, go);
  a.post = post, a.scale = scale, a.pre = pre;
  a.gpost = gpost, a.gscale = gscale, a.gpre = gpre;
  return launch(p, a, true, st);
}

}  // extern "C"
