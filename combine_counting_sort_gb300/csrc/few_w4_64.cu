// few_w4_64.cu: the decoding kernels for 4-bit weights with groups of 64.
#include "few_kernels.cuh"

namespace moe {
template int launch_matvec<64>(const MatvecArgs&, int, cudaStream_t);
template int launch_layer<64>(const LayerArgs&, int, cudaStream_t);
}  // namespace moe
