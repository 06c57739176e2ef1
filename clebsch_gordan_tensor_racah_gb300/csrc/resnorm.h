// resnorm.h -- what the gated residual norm's plan, launcher and kernels share (not public).
#pragma once

#include <cstdint>

#include "cgtp_train.h"
#include "internal.h"

namespace cgtp {

// One irreps block of a row: channels [coff, coff + mul), elements [off, off + mul * D).
struct RnBlock {
  int off, coff, mul, D;
};

// Arguments of one launch.  Row distances are in elements.
struct RnArgs {
  int64_t N = 0;
  const void *h = nullptr, *z = nullptr, *q = nullptr, *gout = nullptr, *gy = nullptr, *x = nullptr;
  int64_t ld_h = 0, ld_z = 0, ld_q = 0, ld_gout = 0, ld_gy = 0, ld_x = 0;
  const void *post = nullptr, *scale = nullptr, *pre = nullptr;
  void *out = nullptr, *y = nullptr, *gh = nullptr, *gz = nullptr, *gq = nullptr;
  int64_t ld_out = 0, ld_y = 0, ld_gh = 0, ld_gz = 0, ld_gq = 0;
  void *gpost = nullptr, *gscale = nullptr, *gpre = nullptr;
  const RnBlock* blocks = nullptr;
  void* part = nullptr;   // per team: [2][C] partial sums (see resnorm_impl.cuh)
  int n_blocks = 0, dim = 0, chan = 0, act = 0;
  int team = 32;          // threads of a row: a power of two up to 32, or the whole CTA
  bool post_norm = false, pre_norm = false;
  double alpha = 1.0, eps = 0.0;
};

}  // namespace cgtp

struct cgtp_resnorm_s {
  int dtype = 0, flags = 0, act = 0;
  double alpha = 1.0, eps = 0.0;
  int64_t dim = 0, chan = 0;
  std::vector<cgtp::RnBlock> blocks;
  cgtp::RnBlock* blocks_dev = nullptr;
  void* part = nullptr;
  int num_sms = 0, team = 32, teams_max = 0;
  size_t device_bytes = 0;
};

namespace cgtp {

// resnorm_*.cu: one translation unit per set of element types
cudaError_t rn_launch_f32(const RnArgs& a, bool backward, int ctas, cudaStream_t st);
cudaError_t rn_launch_f64(const RnArgs& a, bool backward, int ctas, cudaStream_t st);
cudaError_t rn_launch_bf16(const RnArgs& a, bool backward, int ctas, cudaStream_t st);
cudaError_t rn_launch_bf16s(const RnArgs& a, bool backward, int ctas, cudaStream_t st);

constexpr int kRnThreads = 256;

}  // namespace cgtp
