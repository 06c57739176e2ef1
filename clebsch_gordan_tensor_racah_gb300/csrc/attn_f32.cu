// attn_f32.cu -- attention along a graph's edges: FP32 tensors.
#include "attn_impl.cuh"

namespace cgtp {
CGTP_AT_DEFINE(f32, float, float, float)
}  // namespace cgtp
