// resnorm_bf16s_fwd.cu -- gated residual norm, forward, every row tensor in bfloat16.
#include "resnorm_impl.cuh"

cudaError_t cgtp::rn_forward_bf16s(const RnArgs& a, cudaStream_t st) {
  return rn_launch<false, __nv_bfloat16, __nv_bfloat16, __nv_bfloat16, float>(a, st);
}
