// dense_f16.cu: the dense products of f16 operands.
#include "dense_host.cuh"

int moe::dense_product_f16(int kind, const DenseOperand& P, const DenseOperand& Q, const DenseArgs& g, cudaStream_t st) {
  return dense_product<__half>(kind, P, Q, g, st);
}
int moe::dense_backward_f16(const DenseOperand (&P)[2], const DenseOperand (&Q)[2], const DenseArgs (&g)[2], cudaStream_t st) {
  return launch_backward<__half>(P, Q, g, st);
}
