// few_w4_32.cu: the decoding kernels for 4-bit weights with groups of 32.
#include "few_layer.cuh"
#include "few_matvec.cuh"

namespace moe {
template int launch_matvec<32>(const MatvecArgs&, int, cudaStream_t);
template int launch_layer<32>(const LayerArgs&, int, cudaStream_t);
}  // namespace moe
