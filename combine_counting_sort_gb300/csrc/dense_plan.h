// dense_plan.h: which kernel a dense product takes, and in what shape (host
// only; no CUDA).
#pragma once

#include <stdint.h>

#include <algorithm>

namespace moe {

struct DensePlan {
  bool pair;   // 256 x 256 tiles on CTA pairs; otherwise:
  int nt;      // rows i a tile
  int stages;  // ring stages
  int split;   // CTAs that share a tile's contraction
};

inline DensePlan dense_plan(long long I, long long J, long long K, bool gated, bool p_mn, int sms) {
  const long long KB = (K + 63) / 64;
  const long long tj = (J + (gated ? 63 : 127)) / (gated ? 64 : 128);
  DensePlan best = {true, 0, 0, 0};
  const long long ptiles = (I + 255) / 256 * ((J + (gated ? 127 : 255)) / (gated ? 128 : 256));
  double cost = (double)((ptiles + sms / 2 - 1) / (sms / 2)) * KB * 540.0 + 6000.0;
  for (int nt = p_mn ? 64 : 16; nt <= 256; nt *= 2) {
    const long long ti = (I + nt - 1) / nt;
    for (int split = 1; split <= 8 && split <= KB; ++split) {
      const long long ctas = ti * tj * split;
      const int stage = 16384 + nt * 128;
      // two CTAs an SM where the ring allows it and there are as many; a whole SM's ring for one
      const int per_sm = nt <= 64 && ctas > sms ? 2 : 1;
      const long long share = (KB + split - 1) / split;
      // (no more stages than are filled, but room for the tile's sums)
      const int stages = std::max((nt * 512 + stage - 1) / stage, (int)std::min<long long>(share, std::min(12, (per_sm == 2 ? 104 : 220) * 1024 / stage)));
      const double kb = (double)share;
      const double waves = (double)((ctas + (long long)sms * per_sm - 1) / ((long long)sms * per_sm));
      const double busy = std::min<double>((double)ctas, (double)sms * per_sm) / sms;
      const double per_kb = std::max(2.0 * nt, stage / 30.0) * std::max(1.0, busy);
      const double c = waves * (kb * per_kb + 1500.0 + 6.0 * nt) + 3000.0 + (split > 1 ? 1000.0 : 0.0);
      if (c < cost) {
        cost = c;
        best = {false, nt, stages, split};
      }
    }
  }
  return best;
}

}  // namespace moe
