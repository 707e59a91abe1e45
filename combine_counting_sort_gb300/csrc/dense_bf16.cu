// dense_bf16.cu: the dense products of bf16 operands.
#include "dense_host.cuh"

int moe::dense_product_bf16(int kind, const DenseOperand& P, const DenseOperand& Q, const DenseArgs& g, cudaStream_t st) {
  return dense_product<__nv_bfloat16>(kind, P, Q, g, st);
}
int moe::dense_backward_bf16(const DenseOperand (&P)[2], const DenseOperand (&Q)[2], const DenseArgs (&g)[2], cudaStream_t st) {
  return launch_backward<__nv_bfloat16>(P, Q, g, st);
}
