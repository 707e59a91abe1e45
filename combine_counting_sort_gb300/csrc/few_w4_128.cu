// few_w4_128.cu: the decoding kernels for 4-bit weights with groups of 128.
#include "few_layer.cuh"
#include "few_matvec.cuh"

namespace moe {
template int launch_matvec<128>(const MatvecArgs&, int, cudaStream_t);
template int launch_layer<128>(const LayerArgs&, int, cudaStream_t);
}  // namespace moe
