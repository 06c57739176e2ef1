// resnorm_bf16_bwd.cu -- gated residual norm, backward, bfloat16 where the next product reads and FP32 elsewhere.
#include "resnorm_impl.cuh"

cudaError_t cgtp::rn_backward_bf16(const RnArgs& a, cudaStream_t st) {
  return rn_launch<true, float, float, __nv_bfloat16, float>(a, st);
}
