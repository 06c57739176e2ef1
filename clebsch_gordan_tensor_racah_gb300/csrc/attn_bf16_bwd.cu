// attn_bf16_bwd.cu -- attention along a graph's edges, backward, bfloat16 inputs, FP32 results.
#include "attn_impl.cuh"

namespace cgtp {
CGTP_AT_BACKWARD(bf16, bf16, float, float)
}  // namespace cgtp
