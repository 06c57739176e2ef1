// attn_f64_fwd.cu -- attention along a graph's edges, forward, FP64 tensors.
#include "attn_impl.cuh"

namespace cgtp {
CGTP_AT_FORWARD(f64, double, double, double)
}  // namespace cgtp
