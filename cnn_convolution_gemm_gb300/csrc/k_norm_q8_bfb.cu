// Norms around a residual block with h in 8 bits, x and x' in bf16, z in fp32, gate in bf16.
#include "k_norm.cuh"

cudaError_t launch_norm_q8_bfb(const NormArgs& a, cudaStream_t st) {
  return gb::norm::launch<__nv_bfloat16, float, __nv_bfloat16, true>(a, st);
}
