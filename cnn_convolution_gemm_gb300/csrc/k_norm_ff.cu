// Norms around a residual block, x and x' in fp32, z, gate and h in fp32.
#include "k_norm.cuh"

cudaError_t launch_norm_ff(const NormArgs& a, cudaStream_t st) {
  return gb::norm::launch<float, float>(a, st);
}
