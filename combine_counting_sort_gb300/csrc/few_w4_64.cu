// few_w4_64.cu: the decoding kernels for 4-bit weights with groups of 64.
#include "few_layer.cuh"
#include "few_matvec.cuh"

namespace moe {
template int launch_matvec<64>(const MatvecArgs&, int, cudaStream_t);
template int launch_layer<64>(const LayerArgs&, int, cudaStream_t);
}  // namespace moe
