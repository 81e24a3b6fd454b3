// Norms around a residual block, x and x' in bf16, z in fp32, gate and h in bf16.
#include "k_norm.cuh"

cudaError_t launch_norm_bfb(const NormArgs& a, cudaStream_t st) {
  return gb::norm::launch<__nv_bfloat16, float, __nv_bfloat16, false>(a, st);
}
