// resnorm_f32_fwd.cu -- gated residual norm, forward, FP32 tensors.
#include "resnorm_impl.cuh"

cudaError_t cgtp::rn_forward_f32(const RnArgs& a, cudaStream_t st) {
  return rn_launch<false, float, float, float, float>(a, st);
}
