// attn_bf16.cu -- attention along a graph's edges: bfloat16 inputs, FP32 results.
#include "attn_impl.cuh"

namespace cgtp {
CGTP_AT_DEFINE(bf16, bf16, float, float)
}  // namespace cgtp
