// router.cuh: the router's top-k of one token by one warp.
#pragma once

#include "common.cuh"

namespace moe {

// k rounds of a warp-wide arg-max over E <= 32 * VPL logits (largest logit, ties
// to the lower expert id), then softmax weights over the selected logits, summed
// in slot order.  Lane j < k returns slot j's id and weight.
// The logits are compared as unsigned keys of the same order (0: none, a NaN, or
// taken), so that a round is two warp reductions of one instruction each.
template <int VPL>
MOE_DEV int warp_topk(const float* logits, int E, int k, int lane, float* weight) {
  uint32_t key[VPL];
#pragma unroll
  for (int i = 0; i < VPL; ++i) {
    const int e = i * 32 + lane;
    const float v = (e < E ? __ldcg(logits + e) : NAN) + 0.f;   // -0 and 0 are the same
    const uint32_t u = __float_as_uint(v);
    key[i] = v != v ? 0u : (u >> 31 ? ~u : u | 0x80000000u);
  }
  float sel_l0 = 0.f, my_l = 0.f;
  int my_id = 0;
  for (int j = 0; j < k; ++j) {
    uint32_t best = 0;
#pragma unroll
    for (int i = 0; i < VPL; ++i) best = max(best, key[i]);
    best = __reduce_max_sync(0xffffffffu, best);
    uint32_t id = 0x7fffffffu;
#pragma unroll
    for (int i = VPL - 1; i >= 0; --i)
      if (key[i] == best) id = (uint32_t)(i * 32 + lane);
    id = best == 0 ? 0x7fffffffu : __reduce_min_sync(0xffffffffu, id);
#pragma unroll
    for (int i = 0; i < VPL; ++i)
      if ((uint32_t)(i * 32 + lane) == id) key[i] = 0;
    const float l = best == 0 ? -INFINITY : __uint_as_float(best >> 31 ? best & 0x7FFFFFFFu : ~best);
    if (j == 0) sel_l0 = l;
    if (lane == j) { my_l = l; my_id = (int)id; }
  }
  const float ex = lane < k ? expf(my_l - sel_l0) : 0.f;
  float sum = 0.f;
  for (int j = 0; j < k; ++j) sum += __shfl_sync(0xffffffffu, ex, j);   // slots in order
  *weight = ex / sum;
  return my_id;
}

}  // namespace moe
