// resnorm_f64.cu -- gated residual norm, FP64 tensors.
#include "resnorm_impl.cuh"

cudaError_t cgtp::rn_launch_f64(const RnArgs& a, bool backward, cudaStream_t st) {
  return rn_launch<double, double, double, double>(a, backward, st);
}
