// dense_plan.h: which kernel a dense product takes, and in what shape (host
// only; no CUDA).
//
// Every shape that fits is given its time by a model of the two kernels, and the
// least is taken.  The model's constants are fitted to 9500 timings of 550 products (1 to
// 4000 rows, 64 to 12000 columns, contractions of 64 to 7120, every direction and
// epilogue; operands in memory where they are larger than L2), first to the times, then for
// what the choice costs: 3% over the best shape timed, on average, and 33% at most; by waves and
// bytes alone it was 12%.
#pragma once

#include <stdint.h>

#include <algorithm>
#include <cmath>

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

inline bool same_shape(const DenseShape& a, const DenseShape& b) {
  return a.I == b.I && a.J == b.J && a.K == b.K && a.gated == b.gated && a.p_mn == b.p_mn && a.aux == b.aux && a.residual == b.residual && a.vec == b.vec;
}

// Where a shape's plan is kept.
constexpr int kPlanSlots = 64;
inline int plan_slot(const DenseShape& s) {
  const uint64_t h = ((uint64_t)s.I * 1000003u + (uint64_t)s.J) * 1000003u + (uint64_t)s.K + s.aux * 7u + s.residual * 13u + s.vec * 29u;
  return (int)(h * 0x9E3779B97F4A7C15ull >> 58);
}

// What the device holds at once: CTAs in clusters of c that fill an SM (cta[0][c]) or
// half of one (cta[1][c]), and pairs.
struct DenseDevice {
  int sms, pairs;
  int cta[2][kDFewMaxSplit + 1];
};

// Shared memory of the few-row kernel's ring: half an SM's for tiles of up to 64 rows where there
// are more CTAs than the SMs hold one each of, otherwise all of it; no more stages than are filled, but room for the tile's sums.
inline int dfew_stages(int nt, long long share, bool half) {
  const int stage = 16384 + nt * 128, fit = std::min(kDFewMaxStages, (half ? 104 : 220) * 1024 / stage);
  return std::max((nt * 512 + stage - 1) / stage, (int)std::min<long long>(share, fit));
}

// CTAs of the few-row kernel
inline long long dfew_ctas(const DenseShape& s, int nt, int split) {
  const long long columns = s.gated ? 64 : 128;
  return (s.I + nt - 1) / nt * ((s.J + columns - 1) / columns) * split;
}

// Time (ns) of the few-row kernel in one of its shapes, `ctas` being launched in all, in clusters of `cluster`,
// two an SM or one; below 0 where the device cannot hold the clusters.
inline double dfew_cost(const DenseShape& s, const DenseDevice& d, int nt, int split, long long ctas, int cluster, bool half) {
  const long long KB = (s.K + 63) / 64;
  const double odd = s.vec ? 0.0 : 1.0, res = s.residual ? 1.0 : 0.0, aux = s.aux ? 1.0 : 0.0, two = s.gated ? 2.0 : 1.0;
  // more bytes than L2 keeps until they are used again; rows j read by two tiles of i come twice
  const double bytes = 2.0 * (s.I * s.K + two * s.J * s.K + s.I * s.J * (1.0 + res + two * aux));
  const bool cold = bytes > 12e6;
  const long long share = (KB + split - 1) / split, room = d.cta[half][cluster];
  if (room < cluster) return -1.0;
  const double waves = (double)((ctas + room - 1) / room), at_once = (double)std::min(ctas, room);
  const double on_sm = half ? std::min(2.0, std::max(1.0, at_once / d.sms)) : 1.0;
  // 64 of k: the products, this SM's reads, all SMs' reads, this SM's reads from memory
  const double stage = 16384.0 + nt * 128.0;
  const double per_k = std::max({1.9 * nt * on_sm, stage * on_sm / 94.4, stage * at_once / d.sms / 78.6, cold ? 16384.0 * on_sm / 76.3 : 0.0});
  // memory, which wants some 256 CTAs of small tiles to keep it busy
  const double memory = (bytes + (cold && nt < s.I ? 2.0 * two * s.J * s.K : 0.0)) / 6200.0 * (1.0 + (nt <= 32 ? 0.173 : 0.0) * std::max(0.0, 1.0 - at_once / 256.0));
  const double held = (double)std::min<long long>(nt, s.I), rows = std::ceil(held / (8.0 * two * split));   // a tile's, a thread's
  const double end = 1249.0 + rows * (12.7 * two + 158.0 * res + 66.8 * aux * two) * (1.0 + 0.367 * odd) + 3.42 * nt * on_sm +
                     (split > 1 ? 13.8 * held * on_sm : 0.0);
  const double alone = cold && !half && nt <= 32 ? 836.0 : 0.0;   // one small ring an SM: its start and end are not another one's work
  return 785.0 + alone + (split > 1 ? 495.0 : 0.0) + 126.5 * split + std::max(waves * (434.0 + share * per_k), memory) + end + (waves - 1.0) * 0.944 * end;
}

inline double dpair_cost(const DenseShape& s, const DenseDevice& d) {
  const long long KB = (s.K + 63) / 64, columns = s.gated ? 128 : 256;
  const double odd = s.vec ? 0.0 : 1.0, res = s.residual ? 1.0 : 0.0, aux = s.aux ? 1.0 : 0.0;
  // a tile's epilogue runs under the next tile's products, all but the last one's
  const long long tiles = (s.I + 255) / 256 * ((s.J + columns - 1) / columns);
  const double rounds = (double)((tiles + d.pairs - 1) / d.pairs);
  const double epilogue = (2944.0 + 1022.0 * res + 3042.0 * aux) * (1.0 + 0.411 * odd) + 4937.0 * res * odd;
  return 960.0 + std::max(rounds * KB * 389.4, (rounds - 1.0) * epilogue) + epilogue;
}

// f(nt) for the rows a tile may have
template <typename F>
void for_tiles(const DenseShape& s, F&& f) {
  const int least = s.p_mn ? 64 : 16;
  for (int nt = least; nt <= 256 && (nt <= std::max(least, 32) || nt < 2 * s.I); nt *= 2) f(nt);   // (not half of its rows empty)
}

inline DensePlan dense_plan(const DenseShape& s, const DenseDevice& d, double* time = nullptr) {
  DensePlan best = {true, 0, 0, 0};
  double cost = dpair_cost(s, d);
  const long long KB = (s.K + 63) / 64;
  for_tiles(s, [&](int nt) {
    for (int split = 1; split <= kDFewMaxSplit && split <= KB; ++split) {
      const long long ctas = dfew_ctas(s, nt, split);
      const bool half = nt <= 64 && ctas > d.cta[0][split];
      const double c = dfew_cost(s, d, nt, split, ctas, split, half);
      if (c >= 0.0 && c < cost) {
        cost = c;
        best = {false, nt, dfew_stages(nt, (KB + split - 1) / split, half), split};
      }
    }
  });
  if (time) *time = cost;
  return best;
}

// Two products that need nothing of one another, in one launch where that is quicker than one after
// the other.  Clusters are as large as the larger split, which is a multiple of the other one.
inline bool dense_plan_both(const DenseShape (&s)[2], const DenseDevice& d, DensePlan (&plan)[2]) {
  double apart[2];
  plan[0] = dense_plan(s[0], d, &apart[0]);
  plan[1] = dense_plan(s[1], d, &apart[1]);
  double cost = apart[0] + apart[1];
  bool both = false;
  const long long KB[2] = {(s[0].K + 63) / 64, (s[1].K + 63) / 64};
  for (int a = 1; a <= kDFewMaxSplit && a <= KB[0]; ++a)
    for (int b = 1; b <= kDFewMaxSplit && b <= KB[1]; ++b) {
      const int cluster = std::max(a, b);
      if (cluster % std::min(a, b)) continue;
      for_tiles(s[0], [&](int nt0) {
        for_tiles(s[1], [&](int nt1) {
          const long long c0 = dfew_ctas(s[0], nt0, a), c1 = dfew_ctas(s[1], nt1, b);
          const long long ctas = (c0 + cluster - 1) / cluster * cluster + (c1 + cluster - 1) / cluster * cluster;
          const bool half = nt0 <= 64 && nt1 <= 64 && ctas > d.cta[0][cluster];
          const double t0 = dfew_cost(s[0], d, nt0, a, ctas, cluster, half), t1 = dfew_cost(s[1], d, nt1, b, ctas, cluster, half);
          if (t0 < 0.0 || t1 < 0.0 || std::max(t0, t1) >= cost) return;
          cost = std::max(t0, t1);
          both = true;
          plan[0] = {false, nt0, dfew_stages(nt0, (KB[0] + a - 1) / a, half), a};
          plan[1] = {false, nt1, dfew_stages(nt1, (KB[1] + b - 1) / b, half), b};
        });
      });
    }
  return both;
}

}  // namespace moe
