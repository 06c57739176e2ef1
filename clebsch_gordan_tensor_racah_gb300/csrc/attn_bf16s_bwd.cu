// attn_bf16s_bwd.cu -- attention along a graph's edges, backward, bfloat16 inputs and results.
#include "attn_impl.cuh"

namespace cgtp {
CGTP_AT_BACKWARD(bf16s, bf16, bf16, float)
}  // namespace cgtp
