// Norms around a residual block, x and x' in bf16, z, gate and h in fp32.
#include "k_norm.cuh"

cudaError_t launch_norm_bf(const NormArgs& a, cudaStream_t st) {
  return gb::norm::launch<__nv_bfloat16, float, float, false>(a, st);
}
