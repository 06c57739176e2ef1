// resnorm_bf16s.cu -- gated residual norm, every row tensor in bfloat16.
#include "resnorm_impl.cuh"

cudaError_t cgtp::rn_launch_bf16s(const RnArgs& a, bool backward, cudaStream_t st) {
  return rn_launch<__nv_bfloat16, __nv_bfloat16, __nv_bfloat16, float>(a, backward, st);
}
