// few_host.h: arguments of the decoding kernels and their launches per weight form.
#pragma once

#include "host_util.h"

namespace moe {

constexpr int kFewMinSmem = 200 * 1024;   // what the largest stages and tables need

struct MatvecArgs {
  const uint16_t* x;
  const uint8_t* W;
  uint16_t* y;
  int32_t* status;
  int T, N, K;
  uint32_t smem_bytes;
};

struct LayerArgs {
  const uint16_t *x, *router;
  const uint8_t *W1, *W2;
  const float *W1_scale, *W2_scale;
  int32_t* ids;
  float* w;
  uint16_t* out;
  int32_t* counters;   // [0] blocks done with the logits, [1] with the activations, [2] with everything
  float* logits;       // [T, E]
  uint16_t* h;         // [rows, F] bf16 activations times their route's weight
  int32_t* status;
  int T, H, E, k, F;
  uint32_t smem_bytes;
};

// GROUP 0: FP8 (the layer only); 32, 64, 128: 4-bit.
template <int GROUP> int launch_matvec(const MatvecArgs& a, int nsm, cudaStream_t s);
template <int GROUP> int launch_layer(const LayerArgs& a, int nsm, cudaStream_t s);

}  // namespace moe
