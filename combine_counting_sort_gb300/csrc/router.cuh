// router.cuh: the router's top-k of one token by one warp.
#pragma once

#include "common.cuh"

namespace moe {

constexpr int kRouterMaxRuns = 4;

// k rounds of a warp-wide arg-max over E <= 32 * VPL logits (largest logit, ties
// to the lower expert id), then softmax weights over the selected logits, summed
// in slot order.  Lane j < k returns slot j's id and weight.  A logit is the sum of
// `runs` <= kRouterMaxRuns values, `run` apart, in their order.
// The logits are compared as unsigned keys of the same order (0: none, a NaN, or
// taken), so that a round is two warp reductions of one instruction each.
template <int VPL>
MOE_DEV int warp_topk(const float* logits, size_t run, int runs, int E, int k, int lane, float* weight) {
  float v[VPL];
#pragma unroll
  for (int i = 0; i < VPL; ++i) v[i] = i * 32 + lane < E ? __ldcg(logits + i * 32 + lane) : NAN;
  if (runs > 1) {   // all loads in flight together
    float u[kRouterMaxRuns - 1][VPL];
#pragma unroll
    for (int r = 1; r < kRouterMaxRuns; ++r)
#pragma unroll
      for (int i = 0; i < VPL; ++i) u[r - 1][i] = r < runs && i * 32 + lane < E ? __ldcg(logits + r * run + i * 32 + lane) : 0.f;
#pragma unroll
    for (int r = 1; r < kRouterMaxRuns; ++r)
#pragma unroll
      for (int i = 0; i < VPL; ++i) v[i] += u[r - 1][i];
  }
  uint32_t key[VPL];
#pragma unroll
  for (int i = 0; i < VPL; ++i) {
    const uint32_t b = __float_as_uint(v[i] + 0.f);   // -0 and 0 are the same
    key[i] = v[i] != v[i] ? 0u : (b >> 31 ? ~b : b | 0x80000000u);
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
