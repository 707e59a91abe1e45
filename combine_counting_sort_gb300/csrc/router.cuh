// router.cuh: the router's top-k of one token by one warp.
#pragma once

#include "common.cuh"

namespace moe {

// k rounds of a warp-wide arg-max over E <= 32 * VPL logits (largest logit, ties
// to the lower expert id), then softmax weights over the selected logits, summed
// in slot order.  Lane j < k returns slot j's id and weight.
template <int VPL>
MOE_DEV int warp_topk(const float* logits, int E, int k, int lane, float* weight) {
  float v[VPL];
#pragma unroll
  for (int i = 0; i < VPL; ++i) {
    const int e = i * 32 + lane;
    v[i] = e < E ? __ldcg(logits + e) : -INFINITY;
  }
  bool used[VPL];
#pragma unroll
  for (int i = 0; i < VPL; ++i) used[i] = (i * 32 + lane) >= E;
  float sel_l0 = 0.f, my_l = 0.f;
  int my_id = 0;
  for (int j = 0; j < k; ++j) {
    float best = -INFINITY;
    int bid = 0x7fffffff;
#pragma unroll
    for (int i = 0; i < VPL; ++i) {
      const int e = i * 32 + lane;
      if (!used[i] && (v[i] > best || (v[i] == best && e < bid))) { best = v[i]; bid = e; }
    }
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) {
      const float ob = __shfl_xor_sync(0xffffffffu, best, o);
      const int oi = __shfl_xor_sync(0xffffffffu, bid, o);
      if (ob > best || (ob == best && oi < bid)) { best = ob; bid = oi; }
    }
#pragma unroll
    for (int i = 0; i < VPL; ++i)
      if (i * 32 + lane == bid) used[i] = true;
    if (j == 0) sel_l0 = best;
    if (lane == j) { my_l = best; my_id = bid; }
  }
  const float ex = lane < k ? expf(my_l - sel_l0) : 0.f;
  float sum = 0.f;
  for (int j = 0; j < k; ++j) sum += __shfl_sync(0xffffffffu, ex, j);   // slots in order
  *weight = ex / sum;
  return my_id;
}

}  // namespace moe
