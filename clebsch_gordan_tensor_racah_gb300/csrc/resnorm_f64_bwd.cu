// resnorm_f64_bwd.cu -- gated residual norm, backward, FP64 tensors.
#include "resnorm_impl.cuh"

cudaError_t cgtp::rn_backward_f64(const RnArgs& a, cudaStream_t st) {
  return rn_launch<true, double, double, double, double>(a, st);
}
