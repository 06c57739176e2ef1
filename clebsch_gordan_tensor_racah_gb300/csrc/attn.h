// attn.h -- shared definitions of the attention along a graph's edges (attn.cu, attn_impl.cuh).
#pragma once

#include <cuda_runtime.h>

#include <cstdint>
#include <vector>

#include "internal.h"

namespace cgtp {

constexpr int kAtMaxHeads = 64;
constexpr int kAtMaxRow = 8192;       // elements of a row of all heads
constexpr int kAtMaxBorders = 511;
constexpr int kAtHeadShift = 24;      // table entries: element offset | head << 24

// Tables of one irreps string for vectors of V elements (see attn.cu): per head ("dot", head-major) and in the
// order of memory ("acc").
struct AtTab {
  int vec = 1;                   // elements of a vector
  int pieces = 0;                // vectors of one head
  const int* dot_full = nullptr; // [heads * pieces] offsets in rows of all heads
  const int* dot_kv = nullptr;   // [kv * pieces] offsets in rows of the shared heads
  const int* acc = nullptr;      // [heads * pieces] by place in a full row: offset in the shared row | head
  const int* send = nullptr;     // [kv * pieces][group] by place in a shared row: offset in the full row | head
};

struct AtRows {
  char* p = nullptr;
  int64_t ld = 0;   // elements
};

struct AtArgs {
  int heads = 0, kv = 0, group = 1;
  uint32_t heads_magic = 0;      // ceil(2^32 / heads)
  int dk = 0, dv = 0;            // elements of a head
  double scale = 1.0;
  AtTab qk, vv;
  int n_borders = 0;
  const void* borders = nullptr;
  // graph: rows are receivers, or sources for the sender kernel
  const int32_t* rowptr = nullptr;
  const int32_t* col = nullptr;    // the other end of each edge
  const int32_t* eid = nullptr;    // sender kernel: the edge's place in the receivers' order
  int64_t n_rows = 0, n_edges = 0;
  const Int4* items = nullptr;     // pieces of split rows: row, first edge, last edge, part
  const Int4* joins = nullptr;     // split rows: row, first part, number of parts
  int n_items = 0, n_joins = 0, chunk = 0;
  // tensors
  AtRows q, k, v, out, gout, gq, gk, gv;
  const void *lengths = nullptr, *table = nullptr, *bias = nullptr;
  void *lse = nullptr, *alpha = nullptr, *ds = nullptr, *gtable = nullptr;
  void* part = nullptr;            // partial results of split rows
  void* part_sum = nullptr;        // edge rows, backward: partial sums of split rows [parts][heads]
  void* hist = nullptr;            // partial sums of the bias table [ctas][buckets * heads]
  // launch
  int phase = 0;
  int sub = 0;                     // edges held at once
  int team_qk = 1, team_vv = 1;    // threads of one dot product
  int warp_rows = 0;               // a warp a row; otherwise a CTA a row
  int group_smem = 0;              // bytes of shared memory of a row's threads
  int at_g = 0, at_z = 0, at_p = 0, at_idx = 0, at_stat = 0, at_acc = 0, at_red = 0;  // regions, in bytes
  unsigned grid = 0, block = 0;
  size_t smem = 0;
  int hist_ctas = 0, hist_warps = 0, hist_cols = 0;
};

// phases of a kernel
enum : int { kAtWhole = 0, kAtFirst = 1, kAtSecond = 2 };

#define CGTP_AT_DECLARE(suffix)                                              \
  cudaError_t at_forward_##suffix(const AtArgs&, cudaStream_t);              \
  cudaError_t at_edges_forward_##suffix(const AtArgs&, cudaStream_t);        \
  cudaError_t at_receive_##suffix(const AtArgs&, cudaStream_t);              \
  cudaError_t at_edges_receive_##suffix(const AtArgs&, cudaStream_t);        \
  cudaError_t at_send_##suffix(const AtArgs&, bool values, cudaStream_t);    \
  cudaError_t at_join_forward_##suffix(const AtArgs&, cudaStream_t);         \
  cudaError_t at_join_sum_##suffix(const AtArgs&, const AtRows&, int width, int at, int stride, cudaStream_t); \
  cudaError_t at_table_##suffix(const AtArgs&, cudaStream_t);
CGTP_AT_DECLARE(f32)
CGTP_AT_DECLARE(f64)
CGTP_AT_DECLARE(bf16)
CGTP_AT_DECLARE(bf16s)
#undef CGTP_AT_DECLARE

}  // namespace cgtp

struct cgtp_attn_s {
  int dtype = 0, flags = 0;
  int heads = 0, kv = 0, dk = 0, dv = 0;
  double scale = 1.0;
  int n_borders = 0;
  const void* borders = nullptr;
  cgtp::AtTab qk[3], vv[3];      // by width of a vector, widest first; the last is one element
  int n_qk = 0, n_vv = 0;
  void* base = nullptr;
  size_t device_bytes = 0;
  int device = 0, num_sms = 0, smem_cap = 0;
};
