// resnorm_bf16_fwd.cu -- gated residual norm, forward, bfloat16 where the next product reads and FP32 elsewhere.
#include "resnorm_impl.cuh"

cudaError_t cgtp::rn_forward_bf16(const RnArgs& a, cudaStream_t st) {
  return rn_launch<false, float, float, __nv_bfloat16, float>(a, st);
}
