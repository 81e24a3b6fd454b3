// Product with integer 4-bit weights, tiles of up to 160 rows of X.
#include "k_w4_gemm.cuh"

cudaError_t launch_w4_gemm_160(const W4Gemm& g, const W4Operand& x, cudaStream_t st) {
  return gb::w4::gemm::launch<160>(g, x, st);
}
