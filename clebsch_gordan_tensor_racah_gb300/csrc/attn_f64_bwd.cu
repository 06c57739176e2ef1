// attn_f64_bwd.cu -- attention along a graph's edges, backward, FP64 tensors.
#include "attn_impl.cuh"

namespace cgtp {
CGTP_AT_BACKWARD(f64, double, double, double)
}  // namespace cgtp
