// attn_bf16s.cu -- attention along a graph's edges: bfloat16 inputs and results.
#include "attn_impl.cuh"

namespace cgtp {
CGTP_AT_DEFINE(bf16s, bf16, bf16, float)
}  // namespace cgtp
