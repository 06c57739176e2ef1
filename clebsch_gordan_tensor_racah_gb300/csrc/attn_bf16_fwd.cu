// attn_bf16_fwd.cu -- attention along a graph's edges, forward, bfloat16 inputs, FP32 results.
#include "attn_impl.cuh"

namespace cgtp {
CGTP_AT_FORWARD(bf16, bf16, float, float)
}  // namespace cgtp
