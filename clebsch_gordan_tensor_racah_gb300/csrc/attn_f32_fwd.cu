// attn_f32_fwd.cu -- attention along a graph's edges, forward, FP32 tensors.
#include "attn_impl.cuh"

namespace cgtp {
CGTP_AT_FORWARD(f32, float, float, float)
}  // namespace cgtp
