// Norms around a residual block, x and x' in bf16, z, gate and h in bf16.
#include "k_norm.cuh"

cudaError_t launch_norm_bb(const NormArgs& a, cudaStream_t st) {
  return gb::norm::launch<__nv_bfloat16, __nv_bfloat16>(a, st);
}
