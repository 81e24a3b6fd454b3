// Norms around a residual block with h in 8 bits, x and x' in fp32, z and gate in bf16.
#include "k_norm.cuh"

cudaError_t launch_norm_q8_fb(const NormArgs& a, cudaStream_t st) {
  return gb::norm::launch<float, __nv_bfloat16, __nv_bfloat16, true>(a, st);
}
