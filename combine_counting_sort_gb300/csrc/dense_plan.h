// dense_plan.h: which kernel a dense product takes, and in what shape (host
// only; no CUDA).
//
// Every shape that fits is given its time by a model of the two kernels, and the
// least is taken.  The model's constants are a least-squares fit (in the logarithm, 14%
// rms) to 2800 timings of 220 products: 1 to 4000 rows, 64 to 8000 columns, contractions of 64 to
// 7120, every direction and epilogue.  What it picks takes 3% more than the best shape
// timed, on average; by waves and bytes alone it was 12%.
#pragma once

#include <stdint.h>

#include <algorithm>

namespace moe {

constexpr int kDFewMaxStages = 12;
constexpr int kDFewMaxSplit = 8;

struct DensePlan {
  bool pair;   // 256 x 256 tiles on CTA pairs; otherwise:
  int nt;      // rows i a tile
  int stages;  // ring stages
  int split;   // CTAs that share a tile's contraction
};

// What a product asks of its kernel.
struct DenseShape {
  long long I, J, K;
  bool gated, p_mn;          // P with rows contiguous (64 of them a copy)
  bool aux, residual, vec;   // of the epilogue: a second output, a third input, 16-byte vectors
};

// What the device holds at once: CTAs in clusters of c that fill an SM (cta[0][c]) or
// half of one (cta[1][c]), and pairs.
struct DenseDevice {
  int sms, pairs;
  int cta[2][kDFewMaxSplit + 1];
};

// Shared memory of the few-row kernel's ring: half an SM's for tiles of up to 64 rows where there
// are more CTAs than SMs, otherwise all of it; no more stages than are filled, but room for the tile's sums.
inline int dfew_stages(int nt, long long share, bool half) {
  const int stage = 16384 + nt * 128, fit = std::min(kDFewMaxStages, (half ? 104 : 220) * 1024 / stage);
  return std::max((nt * 512 + stage - 1) / stage, (int)std::min<long long>(share, fit));
}

inline DensePlan dense_plan(const DenseShape& s, const DenseDevice& d) {
  const long long KB = (s.K + 63) / 64, columns = s.gated ? 64 : 128;
  const double odd = s.vec ? 0.0 : 1.0, res = s.residual ? 1.0 : 0.0, aux = s.aux ? 1.0 : 0.0, two = s.gated ? 2.0 : 1.0;
  // pairs: a tile's epilogue runs under the next tile's products, all but the last one's (ns)
  const long long tiles = (s.I + 255) / 256 * ((s.J + 2 * columns - 1) / (2 * columns));
  const double rounds = (double)((tiles + d.pairs - 1) / d.pairs);
  const double epilogue = (2427.0 + 1637.0 * res + 1950.0 * aux) * (1.0 + 1.1 * odd);
  DensePlan best = {true, 0, 0, 0};
  double cost = 2212.0 + std::max(rounds * KB * 286.0, (rounds - 1.0) * epilogue) + epilogue;
  for (int nt = s.p_mn ? 64 : 16; nt <= 256; nt *= 2) {
    const long long all = (s.I + nt - 1) / nt * ((s.J + columns - 1) / columns);
    for (int split = 1; split <= kDFewMaxSplit && split <= KB; ++split) {
      const long long ctas = all * split, share = (KB + split - 1) / split;
      const bool half = nt <= 64 && ctas > d.sms;
      const long long room = d.cta[half][split];
      if (room < split) continue;
      const double waves = (double)((ctas + room - 1) / room), at_once = (double)std::min(ctas, room);
      const double on_sm = half ? std::min(2.0, std::max(1.0, at_once / d.sms)) : 1.0;
      // 64 of k: the products, this SM's reads, all SMs' reads
      const double stage = 16384.0 + nt * 128.0;
      const double per_k = std::max({1.755 * nt * on_sm, stage * on_sm / 90.0, stage * at_once / d.sms / 91.0});
      const double rows = (double)((std::min<long long>(nt, s.I) + (long long)(8 * two) * split - 1) / ((long long)(8 * two) * split));   // a thread's
      const double end = 798.0 + rows * (29.4 * two + 78.0 * res + 40.7 * aux * two) * (1.0 + 1.43 * odd) + 3.2 * nt * on_sm +
                         (split > 1 ? 14.2 * std::min<long long>(nt, s.I) * on_sm : 0.0);
      const double c = 941.0 + (split > 1 ? 655.0 : 0.0) + 107.0 * split + waves * (577.0 + share * per_k + end);
      if (c < cost) {
        cost = c;
        best = {false, nt, dfew_stages(nt, share, half), split};
      }
    }
  }
  return best;
}

}  // namespace moe
