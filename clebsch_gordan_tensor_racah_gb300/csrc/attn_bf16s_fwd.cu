// attn_bf16s_fwd.cu -- attention along a graph's edges, forward, bfloat16 inputs and results.
#include "attn_impl.cuh"

namespace cgtp {
CGTP_AT_FORWARD(bf16s, bf16, bf16, float)
}  // namespace cgtp
