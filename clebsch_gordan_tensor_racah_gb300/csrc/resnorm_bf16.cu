// resnorm_bf16.cu -- gated residual norm, bfloat16 where the next product reads and FP32 elsewhere.
#include "resnorm_impl.cuh"

cudaError_t cgtp::rn_launch_bf16(const RnArgs& a, bool backward, cudaStream_t st) {
  return rn_launch<float, float, __nv_bfloat16, float>(a, backward, st);
}
