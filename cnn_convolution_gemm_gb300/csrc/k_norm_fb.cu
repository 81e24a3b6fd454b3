// Norms around a residual block, x and x' in fp32, z, gate and h in bf16.
#include "k_norm.cuh"

cudaError_t launch_norm_fb(const NormArgs& a, cudaStream_t st) {
  return gb::norm::launch<float, __nv_bfloat16>(a, st);
}
