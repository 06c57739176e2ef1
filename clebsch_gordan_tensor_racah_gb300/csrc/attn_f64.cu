// attn_f64.cu -- attention along a graph's edges: FP64 tensors.
#include "attn_impl.cuh"

namespace cgtp {
CGTP_AT_DEFINE(f64, double, double, double)
}  // namespace cgtp
