// resnorm.h -- what the gated residual norm's plan, launcher and kernels share (not public).
#pragma once

#include <cstdint>

#include "cgtp_train.h"
#include "internal.h"

namespace cgtp {

// One irreps block of a row: channels [coff, coff + mul), elements [off, off + mul * D).
struct RnBlock {
  int off, coff, mul, D;
  int code;            // rn_code, set for a launch
  float inv_n_f;       // 1 / (mul D)
  double inv_n;
};

// A row tensor of a launch (distances in elements) and its place in a staged tile.
struct RnRows {
  char* ptr = nullptr;
  int64_t ld = 0, ld_bytes = 0;
  int width = 0, es = 0;    // elements of a row, bytes of an element
  int at = -1, pitch = 0;   // first byte and row distance in bytes of its region of a stage; -1: no region
  int vec = 0;              // bytes of a copy between the region and memory
  bool linear = false;      // the rows of a tile are one run of bytes on both sides
};

enum { kRnH, kRnZ, kRnQ, kRnOut, kRnY, kRnForward };                                    // forward
enum { kRnGout, kRnGy, kRnX, kRnBz, kRnBq, kRnGh, kRnGz, kRnGq, kRnBackward };          // backward
constexpr int kRnInputs[2] = {3, 5};
constexpr int kRnMaxRows = kRnBackward;

constexpr int kRnInline = 64;
// kRnOne: a warp a row, or several rows a warp.  kRnMany: several warps a row.  ..Full: every operand there, tiles that are runs of 16-byte pieces, blocks that fill the lanes (and a
// warp a row; kRnFewFull: several rows a warp).  kRnDirect: rows in place, a CTA a row,
// any number and size of blocks.
enum RnKind { kRnDirect, kRnMany, kRnManyFull, kRnOne, kRnFewFull, kRnOneFull };

// Arguments of one launch.
struct RnArgs {
  int64_t N = 0, tiles = 0;
  RnRows t[kRnMaxRows];
  const void *post = nullptr, *scale = nullptr, *pre = nullptr;
  void *gpost = nullptr, *gscale = nullptr, *gpre = nullptr;
  const RnBlock* blocks = nullptr;   // device table; also in `few` where they fit there
  RnBlock few[kRnInline];
  void* part = nullptr;       // [CTAs][2][C] partial sums: of a(q) P, of gpre
  unsigned* ticket = nullptr; // CTAs that are done, where the last one adds the partial sums (null: another launch does)
  int n_blocks = 0, dim = 0, chan = 0, act = 0;
  bool post_norm = false, pre_norm = false;
  double alpha = 1.0, eps = 0.0;
  float alpha_f = 1.0f, eps_f = 0.0f;
  // how rows are dealt out
  int kind = 0;               // RnKind
  int stages = 1;             // tiles of a group in shared memory
  int lanes = 32;             // threads of a row: a power of two below a warp, or 32 * warps
  int warps = 1;              // warps of a group
  int groups = 1;             // groups of a CTA
  int rows = 1;               // rows of a tile
  int stage_bytes = 0, group_bytes = 0, table_at = 0, smem = 0, ctas = 1;
};

}  // namespace cgtp

struct cgtp_resnorm_s {
  int dtype = 0, flags = 0, act = 0;
  double alpha = 1.0, eps = 0.0;
  int64_t dim = 0, chan = 0;
  int widest = 1;             // channels of the widest block
  std::vector<cgtp::RnBlock> blocks;
  void* base = nullptr;       // the device allocation that holds the next three
  cgtp::RnBlock* blocks_dev = nullptr;
  void* part = nullptr;
  unsigned* ticket = nullptr;
  int num_sms = 0, smem_cap = 0;
  size_t device_bytes = 0;
};

namespace cgtp {

// resnorm_*.cu: one translation unit per set of element types and direction
#define CGTP_RN_DECLARE(name)                                   \
  cudaError_t rn_forward_##name(const RnArgs& a, cudaStream_t st); \
  cudaError_t rn_backward_##name(const RnArgs& a, cudaStream_t st);
CGTP_RN_DECLARE(f32)
CGTP_RN_DECLARE(f64)
CGTP_RN_DECLARE(bf16)
CGTP_RN_DECLARE(bf16s)
#undef CGTP_RN_DECLARE

#ifdef __CUDACC__
#define CGTP_HOST_DEVICE __host__ __device__
#else
#define CGTP_HOST_DEVICE
#endif

// Channels of a block that a thread keeps in registers: mul / lanes rounded up to a share that the
// kernels have code for (at most about 20 values), or 0.
CGTP_HOST_DEVICE inline int rn_share(int D, int mul, int lanes) {
  const int share = mul <= lanes ? 1 : mul <= 2 * lanes ? 2 : mul <= 4 * lanes ? 4 : mul <= 8 * lanes ? 8 : 0;
  return share <= (D == 1 ? 8 : D <= 5 ? 4 : D <= 9 ? 2 : 1) ? share : 0;
}
// Number of the code for blocks of D components and a share: CGTP_RN_HELD counts the same way.
CGTP_HOST_DEVICE constexpr int rn_code(int D, int share) {
  return (D <= 3 ? (D == 1 ? 0 : 4) : D <= 7 ? (D == 5 ? 7 : 10) : D == 9 ? 12 : 14 + (D - 11) / 2) +
         (share >= 8 ? 3 : share >= 4 ? 2 : share - 1);
}

// Partial sums (CTAs x 2 C) that the last CTA of a backward adds itself: up to 16 loads a thread, which is
// less than another launch (2,000 rows of 8x0e+8x1o).  Above, the launch takes 6 us and one CTA would take longer.
constexpr int kRnTailSums = 8192;
constexpr int kRnMaxStages = 2;     // tiles of a group in shared memory
constexpr int kRnWarps = 16;        // warps of a CTA at most
constexpr int kRnDirectWarps = 8;   // warps of a row that is too long for shared memory
constexpr int kRnCtasPerSm = 4;     // of the unstaged kernels

}  // namespace cgtp
