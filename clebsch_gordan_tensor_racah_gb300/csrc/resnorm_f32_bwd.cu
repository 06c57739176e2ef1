// resnorm_f32_bwd.cu -- gated residual norm, backward, FP32 tensors.
#include "resnorm_impl.cuh"

cudaError_t cgtp::rn_backward_f32(const RnArgs& a, cudaStream_t st) {
  return rn_launch<true, float, float, float, float>(a, st);
}
