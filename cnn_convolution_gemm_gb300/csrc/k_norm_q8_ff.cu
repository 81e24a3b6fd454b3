// Norms around a residual block with h in 8 bits, x and x' in fp32, z and gate in fp32.
#include "k_norm.cuh"

cudaError_t launch_norm_q8_ff(const NormArgs& a, cudaStream_t st) {
  return gb::norm::launch<float, float, float, true>(a, st);
}
