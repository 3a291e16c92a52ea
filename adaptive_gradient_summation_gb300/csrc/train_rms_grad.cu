// train_rms_grad.cu -- the gradient of the root-mean-square norm (kernels: adasum_norm.cuh).
#include "adasum_norm.cuh"

namespace adasum {

int launch_rms_grad(const NormGradArgs& a, int dtype, bool vec, const WorkerRows& rows, const ParamGradArgs& p, cudaStream_t stream) {
  return launch_norm_grad_of<kRms>(a, dtype, vec, rows, p, stream);
}

}  // namespace adasum
