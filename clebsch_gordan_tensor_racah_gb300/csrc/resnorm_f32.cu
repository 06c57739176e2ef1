// resnorm_f32.cu -- gated residual norm, FP32 tensors.
#include "resnorm_impl.cuh"

cudaError_t cgtp::rn_launch_f32(const RnArgs& a, bool backward, cudaStream_t st) {
  return rn_launch<float, float, float, float>(a, backward, st);
}
