// few_fp8.cu: the whole-layer kernels for FP8 weights with 128 x 128 scales.
#include "few_layer.cuh"

namespace moe {
template int launch_layer<0>(const LayerArgs&, int, cudaStream_t);
}  // namespace moe
