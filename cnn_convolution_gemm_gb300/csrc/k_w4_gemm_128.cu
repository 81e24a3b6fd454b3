// Product with integer 4-bit weights, tiles of up to 128 rows of X.
#include "k_w4_gemm.cuh"

cudaError_t launch_w4_gemm_128(const W4Gemm& g, const W4Operand& x, cudaStream_t st) {
  return gb::w4::gemm::launch<128>(g, x, st);
}
