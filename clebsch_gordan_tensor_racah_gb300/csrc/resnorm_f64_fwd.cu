// resnorm_f64_fwd.cu -- gated residual norm, forward, FP64 tensors.
#include "resnorm_impl.cuh"

cudaError_t cgtp::rn_forward_f64(const RnArgs& a, cudaStream_t st) {
  return rn_launch<false, double, double, double, double>(a, st);
}
