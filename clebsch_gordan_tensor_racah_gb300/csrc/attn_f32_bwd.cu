// attn_f32_bwd.cu -- attention along a graph's edges, backward, FP32 tensors.
#include "attn_impl.cuh"

namespace cgtp {
CGTP_AT_BACKWARD(f32, float, float, float)
}  // namespace cgtp
