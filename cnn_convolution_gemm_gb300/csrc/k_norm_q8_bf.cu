// Norms around a residual block with h in 8 bits, x and x' in bf16, z and gate in fp32.
#include "k_norm.cuh"

cudaError_t launch_norm_q8_bf(const NormArgs& a, cudaStream_t st) {
  return gb::norm::launch<__nv_bfloat16, float, float, true>(a, st);
}
