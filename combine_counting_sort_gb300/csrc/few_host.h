// few_host.h: arguments of the decoding kernels and their launches per weight form.
#pragma once

#include "few_plan.h"
#include "host_util.h"

namespace moe {

struct MatvecArgs {
  CUtensorMap map_w, map_x;   // wide and tensor kernels: whole tiles, and 64 columns of all tokens
  const uint16_t* x;
  const uint8_t* W;
  uint16_t* y;
  int32_t* status;
  int T, N, K;
  int slices;          // wide kernel: of a stage; tensor kernel: blocks that share rows
  uint32_t smem_bytes;
};

struct LayerArgs {
  CUtensorMap map1, map2;   // FP8 weights: 128 bytes x 16 rows x 128-column slices
  const uint16_t *x, *router;
  const uint8_t *W1, *W2;
  const float *W1_scale, *W2_scale;
  int32_t* ids;
  float* w;
  uint16_t* out;
  int32_t* counters;   // arrivals of the grid's blocks at its meetings, and at the end
  float* logits;       // [splits][T, E] sums over runs of columns
  uint8_t *x8, *h8;    // token records of x [T] and of the activations [T k], K / 128 of kTokenRecord bytes each
  float* h;            // [T k, F] activations times their route's weight
  int32_t* status;
  int T, H, E, k, F;
  int splits;          // runs of columns of the logits
  int cols;            // tokens of a segment, at most
  uint32_t smem_bytes;
};

// A tensor map of up to three dimensions, innermost first; strides in bytes of dimensions 1 and 2.
inline bool encode_few_map(CUtensorMap* map, CUtensorMapDataType type, CUtensorMapSwizzle swizzle, const void* base, int rank,
                           const uint64_t* dims, const uint64_t* strides, const uint32_t* box) {
  auto enc = tensor_map_encoder();
  if (!enc) return false;
  cuuint64_t d[3], st[2];
  cuuint32_t b[3], one[3] = {1, 1, 1};
  for (int i = 0; i < rank; ++i) { d[i] = dims[i]; b[i] = box[i]; }
  for (int i = 0; i + 1 < rank; ++i) st[i] = strides[i];
  return enc(map, type, (cuuint32_t)rank, const_cast<void*>(base), d, st, b, one, CU_TENSOR_MAP_INTERLEAVE_NONE, swizzle,
             CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

// GROUP 0: FP8 (the layer only); 32, 64, 128: 4-bit.
template <int GROUP> int launch_matvec(const MatvecArgs& a, int nsm, cudaStream_t s);
template <int GROUP> int launch_layer(const LayerArgs& a, int nsm, cudaStream_t s);

// Row tiles per item: the fewest (rounds over the SMs) x (row tiles), and of
// those the most row tiles, since a stage's tokens are shared by its row tiles.
inline int few_row_tiles(int tiles, int nsm, int most = 3) {
  int best = 1, cost = 1 << 30;
  for (int rt = 1; rt <= most; ++rt) {
    const int groups = (tiles + rt - 1) / rt, c = (groups + nsm - 1) / nsm * rt;
    if (c <= cost) { cost = c; best = rt; }
  }
  return best;
}

// Launch with all the shared memory a block can have; `cluster` blocks share rows.
template <class Kernel, class Args>
int few_launch(Kernel kernel, Args& a, int threads, int blocks, bool cooperative, cudaStream_t s, int cluster = 1) {
  int dev = 0, smem = 0;
  if (cudaGetDevice(&dev) != cudaSuccess) return MOE_ERR_CUDA;
  if (cudaDeviceGetAttribute(&smem, cudaDevAttrMaxSharedMemoryPerBlockOptin, dev) != cudaSuccess) return MOE_ERR_CUDA;
  if (smem < (int)kFewMinSmem) return MOE_ERR_UNSUPPORTED;
  if (cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, smem) != cudaSuccess) return MOE_ERR_CUDA;
  auto args = a;
  args.smem_bytes = smem;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(blocks);
  cfg.blockDim = dim3(threads);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = s;
  cudaLaunchAttribute attr[2];
  if (cooperative) {
    attr[0].id = cudaLaunchAttributeCooperative;
    attr[0].val.cooperative = 1;
  } else {
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
  }
  attr[1].id = cudaLaunchAttributeClusterDimension;
  attr[1].val.clusterDim.x = cluster;
  attr[1].val.clusterDim.y = attr[1].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = cluster > 1 ? 2 : 1;
  return cudaLaunchKernelEx(&cfg, kernel, args) == cudaSuccess ? MOE_OK : MOE_ERR_CUDA;
}

}  // namespace moe
