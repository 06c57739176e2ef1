// resnorm_bf16s_bwd.cu -- gated residual norm, backward, every row tensor in bfloat16.
#include "resnorm_impl.cuh"

cudaError_t cgtp::rn_backward_bf16s(const RnArgs& a, cudaStream_t st) {
  return rn_launch<true, __nv_bfloat16, __nv_bfloat16, __nv_bfloat16, float>(a, st);
}
