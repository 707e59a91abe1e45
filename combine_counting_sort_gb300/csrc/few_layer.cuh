// few_layer.cuh: a whole MoE layer for a few tokens, in one launch (few_slice.cuh: its
// products).  What bounds it is memory, but for some 12 us: until the routes are
// known, no weight can be on its way.
//
// Measured, us and share of the copy bandwidth that the weights were read at (H 7168, F 2048, 8 of 256
// experts): FP8, 1 token 66 (79%), 16 tokens 640 (103%), 64 tokens 1458 (99%); 4-bit, groups of
// 128, 1 token 52 (53%), 64 tokens 1031 (72%); groups of 32, 8 tokens 267 (79%).  One token's 66
// us in ns, by a block's own clock: records 670, logits 1570, meeting 1470, routes 1820, tables 1890 (the
// block's meetings around them included), gate and up 33700, meeting and records 6100, down
// 15200; the 4-bit products take 25200 and 11000, bound by the hand-over of stages that hold half the
// bytes and by widening.  With H or F of a few hundred the stages are
// mostly empty and the fixed 12 us are most of the time (8 experts, 256 x 256: 12.8 us).
#pragma once

#include <type_traits>

#include "few_slice.cuh"
#include "router.cuh"

namespace moe {

constexpr int kFewOwnTopk = 2 * kFewAllWarps;   // tokens whose routes every block selects for itself

// ---------------------------------------------------------------- copies

struct LayerMatrix {
  const uint8_t* p;        // 4-bit: the expert's tiles
  const CUtensorMap* map;  // FP8: all experts' rows
  const float* scale;
  int row0, K;             // FP8: the expert's first row
};

// Copy `tiles` row tiles (the rt-th at row tile tile0 + rt % PER * step + rt / PER) of the 128-column
// slices [kt0, kt0 + nk) into the stage at `st`; whole warp.
template <int GROUP, int SP, int PER>
MOE_DEV void copy_weights(const LayerMatrix& W, int tile0, int step, int tiles, int kt0, int nk, uint32_t st, uint32_t scales,
                          uint32_t bar, int lane) {
  using F = FewForm<GROUP, SP>;
  static_assert(F::kW4 || SP == 1, "a box has 8 slices");
  const int KT = W.K / 128;
  if (F::kW4) {
    if (lane == 0) mbar_arrive_expect_tx(bar, tiles * nk * F::kTile);
    __syncwarp();
    if (lane < tiles) bulk_load_once(st + lane * F::kRowTile, W.p + ((size_t)(tile0 + lane % PER * step + lane / PER) * KT + kt0) * F::kTile, nk * F::kTile, bar);
  } else {
    // a box of min(8, K / 128) slices; slices past K count as bytes and are filled with zeros
    if (lane == 0) mbar_arrive_expect_tx(bar, tiles * min(kFewWarps, KT) * 2048);
    __syncwarp();
    if (lane < tiles) tma_load_3d_once(st + lane * F::kRowTile, W.map, 0, W.row0 + (tile0 + lane % PER * step + lane / PER) * 16, kt0, bar);
    for (int i = lane; i < tiles * kFewWarps; i += 32) {
      const int rt = i / kFewWarps, kt = i % kFewWarps;
      const bool on = kt < nk;
      const float* src = W.scale + (size_t)((tile0 + rt % PER * step + rt / PER) >> 3) * KT + (on ? kt0 + kt : kt0);
      cp_async4(scales + 4 * i, src, on ? 4 : 0);
    }
    cp_async_arrive(bar);
  }
}

// Copy the records [kt0, kt0 + nk) of `cols` tokens, token c's at record_of(c).
template <int PITCH, class RecordOf>
MOE_DEV void copy_tokens(RecordOf record_of, int cols, int kt0, int nk, uint32_t tok, uint32_t bar, int lane) {
  if (lane == 0) mbar_arrive_expect_tx(bar, cols * nk * kTokenRecord);
  __syncwarp();
  if (lane < cols) bulk_load(tok + lane * PITCH, record_of(lane) + (size_t)kt0 * kTokenRecord, nk * kTokenRecord, bar);
}

// ---------------------------------------------------------------- routes

// Tables of the routes in shared memory, sized by the P = T k pairs.  A segment is
// one expert and up to A.cols of the tokens routed to it; row r of the activations
// belongs to one (token, expert).  An expert's segments follow one another, so that what its weights
// are copied for again comes out of L2 (64 tokens on all of 8 experts, FP8: 354 MB read from memory,
// the weights' own bytes, in 303 us; one pass over them would take 52).
struct FewTables {
  uint64_t* seg_mask;
  int *seg_expert, *seg_row;
  float* row_weight;
  uint8_t* row_token;
  MOE_DEV FewTables(unsigned char* p, int P) {
    seg_mask = reinterpret_cast<uint64_t*>(p);
    seg_expert = reinterpret_cast<int*>(seg_mask + P);
    seg_row = seg_expert + P;
    row_weight = reinterpret_cast<float*>(seg_row + P);
    row_token = reinterpret_cast<uint8_t*>(row_weight + P);
  }
};

// The logits as products of bf16 MMAs: units of 16 experts x 8 tokens x one of `splits`
// equal runs of columns, one unit to a block.  Each warp takes every eighth chunk of
// 32 columns, of which lane t of a row (or token) reads columns 8 t .. in one go (the
// column order inside an MMA is free as long as both operands follow it).  The
// warps' sums meet in shared memory; the runs' sums go to logits[run][t][e].
MOE_DEV void few_logits(const LayerArgs& A, float* part, int tid, int warp, int lane) {
  const int rows = (A.E + 15) / 16, blocks = (A.T + 7) / 8, chunks = A.H / 32;
  for (int unit = blockIdx.x; unit < rows * blocks * A.splits; unit += gridDim.x) {
    const int e0 = unit % rows * 16, t0 = unit / rows % blocks * 8, run = unit / rows / blocks;
    if (warp < kFewWarps) {
      const int g = lane >> 2;
      const uint16_t* r0 = A.router + (size_t)min(e0 + g, A.E - 1) * A.H + 8 * (lane & 3);
      const uint16_t* r1 = A.router + (size_t)min(e0 + g + 8, A.E - 1) * A.H + 8 * (lane & 3);
      const uint16_t* x = A.x + (size_t)min(t0 + g, A.T - 1) * A.H + 8 * (lane & 3);
      float s[2][4] = {};
      const int end = (run + 1) * chunks / A.splits;
#pragma unroll 4
      for (int c = run * chunks / A.splits + warp; c < end; c += kFewWarps) {
        const uint4 a0 = __ldg(reinterpret_cast<const uint4*>(r0 + c * 32)), a1 = __ldg(reinterpret_cast<const uint4*>(r1 + c * 32));
        const uint4 b = __ldg(reinterpret_cast<const uint4*>(x + c * 32));
        const uint32_t m0[4] = {a0.x, a1.x, a0.y, a1.y}, m1[4] = {a0.z, a1.z, a0.w, a1.w};
        mma_bf16(s[0], m0, b.x, b.y);
        mma_bf16(s[1], m1, b.z, b.w);
      }
#pragma unroll
      for (int i = 0; i < 4; ++i)
        part[(warp * 8 + 2 * (lane & 3) + (i & 1)) * kFewColPitch + g + 8 * (i >> 1)] = s[0][i] + s[1][i];
    }
    __syncthreads();
    if (tid < 128) {
      const int e = e0 + (tid & 15), t = t0 + (tid >> 4);
      if (e < A.E && t < A.T) A.logits[((size_t)run * A.T + t) * A.E + e] = get_sum(part, 8, tid & 15, tid >> 4);
    }
    __syncthreads();
  }
}

// Bounded wait of one thread for `n` arrivals on a counter of the whole grid.
MOE_DEV bool grid_wait(const int32_t* ctr, int n, volatile int* abort_flag, int32_t* status) {
  const uint64_t t0 = globaltimer_ns();
  while (ld_acquire_gpu(ctr) < n) {
    if (*abort_flag) return false;
    if (globaltimer_ns() - t0 > kFewTimeoutNs) {
      *abort_flag = 1;
      set_status(status, MOE_ERR_TIMEOUT);
      return false;
    }
  }
  return true;
}

// The grid's blocks meet: what each wrote before is seen by all after.
MOE_DEV void few_meet(const LayerArgs& A, int counter, FewShared* sh, int tid) {
  __threadfence();
  __syncthreads();
  if (tid == 0) {
    red_release_gpu_add(A.counters + counter, 1);
    grid_wait(A.counters + counter, gridDim.x, &sh->abort_flag, A.status);
  }
  __syncthreads();
}

// The tables of at most 32 pairs, by one warp: lane p is pair p, the lowest lane of those
// with the same expert makes its segment.
MOE_DEV void few_tables_small(const LayerArgs& A, FewShared* sh, const FewTables& tb, const int* ids, const float* w, int lane) {
  const int P = A.T * A.k, t = lane / A.k;
  const int e = lane < P ? ids[lane] : -1;
  if (e >= A.E && blockIdx.x == 0) set_status(A.status, MOE_ERR_EXPERT_ID);
  const bool on = e >= 0 && e < A.E;
  const uint32_t same = __match_any_sync(0xffffffffu, on ? e : -1 - lane);
  uint32_t tokens = 0;
  float sum = 0.f;
  bool again = false;   // the token names the expert in an earlier slot too
  for (int p = 0; p < P; ++p) {
    const float wp = __shfl_sync(0xffffffffu, lane < P ? w[lane] : 0.f, p);
    if ((same >> p) & 1) {
      tokens |= 1u << (p / A.k);
      if (p / A.k == t) {
        again |= p < lane;
        sum += wp;   // in slot order
      }
    }
  }
  const bool leads = on && lane == __ffs(same) - 1;
  const int c = leads ? __popc(tokens) : 0, s = (c + A.cols - 1) / A.cols;
  int incl = c | s << 16;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int v = __shfl_up_sync(0xffffffffu, incl, o);
    if (lane >= o) incl += v;
  }
  int row = (incl & 0xFFFF) - c, seg = (incl >> 16) - s;
  const int first = __shfl_sync(0xffffffffu, row, __ffs(same) - 1);
  const int most = __reduce_max_sync(0xffffffffu, c), all = __shfl_sync(0xffffffffu, incl, 31);
  if (leads) {
    for (uint32_t m = tokens; m;) {
      uint32_t take = m;
      if (__popc(m) > A.cols) {
        take = 0;
        for (int b = 0; b < A.cols; ++b) take |= (m ^ take) & (~(m ^ take) + 1);   // the lowest bit left
      }
      m ^= take;
      tb.seg_mask[seg] = take;
      tb.seg_expert[seg] = e;
      tb.seg_row[seg++] = row;
      row += __popc(take);
    }
  }
  if (on && !again) {
    const int r = first + __popc(tokens & ((1u << t) - 1));
    tb.row_token[r] = (uint8_t)t;
    tb.row_weight[r] = sum;
  }
  if (lane == 0) {
    sh->rows = all & 0xFFFF;
    sh->segs = all >> 16;
    sh->cap = max(1, min(most, A.cols));
  }
}

// The tables from the pairs' ids and weights (in shared memory).  scratch: E masks,
// E first rows, a count per warp.
MOE_DEV void few_tables(const LayerArgs& A, FewShared* sh, const FewTables& tb, const int* ids, const float* w,
                        unsigned char* scratch, int tid, int warp, int lane) {
  const int P = A.T * A.k;
  if (P <= 32) {   // 0.4 us, and 1.7 us the other way
    if (warp == 0) few_tables_small(A, sh, tb, ids, w, lane);
    return;
  }
  uint64_t* mask = reinterpret_cast<uint64_t*>(scratch);
  int* first = reinterpret_cast<int*>(mask + A.E);
  int* totals = first + A.E;
  if (tid == 0) sh->cap = 1;
  for (int e = tid; e < A.E; e += kFewThreads) mask[e] = 0;
  __syncthreads();
  for (int p = tid; p < P; p += kFewThreads) {
    const int e = ids[p];
    if (e >= A.E) {
      if (blockIdx.x == 0) set_status(A.status, MOE_ERR_EXPERT_ID);
    } else if (e >= 0) {
      atomicOr(reinterpret_cast<unsigned long long*>(&mask[e]), 1ull << (p / A.k));   // a set: any order
    }
  }
  __syncthreads();
  // thread i: experts 4 i .. 4 i + 3; rows in the low half of a count, segments in the high
  static_assert(4 * kFewThreads >= 1024, "");
  int counts = 0, most = 0;
  uint64_t m4[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    m4[i] = 4 * tid + i < A.E ? mask[4 * tid + i] : 0;
    const int c = __popcll(m4[i]);
    counts += c | ((c + A.cols - 1) / A.cols) << 16;
    most = max(most, c);
  }
  int incl = counts;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int v = __shfl_up_sync(0xffffffffu, incl, o);
    if (lane >= o) incl += v;
  }
  most = __reduce_max_sync(0xffffffffu, most);
  if (lane == 31) totals[warp] = incl;
  if (lane == 0 && most > 1) atomicMax(&sh->cap, min(most, A.cols));
  __syncthreads();
  int at = incl - counts;
  for (int i = 0; i < warp; ++i) at += totals[i];
  int row = at & 0xFFFF, seg = at >> 16;
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    uint64_t m = m4[i];
    if (4 * tid + i < A.E) first[4 * tid + i] = row;
    while (m) {
      uint64_t take = m;
      if (__popcll(m) > A.cols) {
        take = 0;
        for (int b = 0; b < A.cols; ++b) take |= (m ^ take) & (~(m ^ take) + 1);   // the lowest bit left
      }
      m ^= take;
      tb.seg_mask[seg] = take;
      tb.seg_expert[seg] = 4 * tid + i;
      tb.seg_row[seg++] = row;
      row += __popcll(take);
    }
  }
  if (tid == kFewThreads - 1) {
    sh->rows = row;
    sh->segs = seg;
  }
  __syncthreads();
  for (int p = tid; p < P; p += kFewThreads) {   // a token that names an expert again adds to its weight, in slot order
    const int e = ids[p], t = p / A.k;
    if (e < 0 || e >= A.E) continue;
    bool again = false;
    float sum = 0.f;
    for (int i = t * A.k; i < (t + 1) * A.k; ++i) {
      if (ids[i] == e) {
        again |= i < p;
        sum += w[i];
      }
    }
    if (!again) {
      const int r = first[e] + __popcll(mask[e] & ((1ull << t) - 1));
      tb.row_token[r] = (uint8_t)t;
      tb.row_weight[r] = sum;
    }
  }
}

template <int GROUP>
MOE_DEV LayerMatrix expert_matrix(const uint8_t* W, const CUtensorMap* map, const float* scale, int e, int N, int K) {
  if (GROUP != 0) return LayerMatrix{W + (size_t)e * w4_matrix_bytes(N, K, GROUP ? GROUP : 128), nullptr, nullptr, 0, K};
  return LayerMatrix{nullptr, map, scale + (size_t)e * (N / 128) * (K / 128), e * N, K};
}

// ---------------------------------------------------------------- gate and up, down

template <int GROUP, int RT2, bool DIRECT, int SP>
MOE_DEV void layer_products(const LayerArgs& A, unsigned char* sm, const FewTables& tb, uint32_t after_tables, uint32_t zero, int tid,
                            int warp, int lane) {
  using F = FewForm<GROUP, SP>;
  constexpr int kPairs = layer_pairs(GROUP, SP, DIRECT);   // gate and up row tiles of a stage
  FewShared* sh = reinterpret_cast<FewShared*>(sm);
  const int HT = A.H / 128, FT = A.F / 128;
  const int segs = sh->segs, cap = sh->cap;
  // The sums on their way to the finishing warps.  Down: DIRECT one buffer,
  // [row tile][warp][token]; else as gate and up, and the output's sums [T][16 RT2].
  const LayerRoom room = layer_room(GROUP, SP, RT2, DIRECT, A.T, A.T * A.k, cap, A.smem_bytes);
  FewRing way = few_sums_ring(sm, after_tables, room.buf, room.bufs);
  float* sums = reinterpret_cast<float*>(sm + after_tables + room.sums);
  const uint32_t tok = room.tok, sco = room.scale;
  FewRing ring = few_ring(sm, after_tables + room.sums + room.out, A.smem_bytes, room.stage);
  const int fitems = A.F / (16 * kPairs), items1 = segs * fitems, steps1 = (HT + F::kSlices - 1) / F::kSlices;
  const int htiles = A.H / 16, items2 = (htiles + RT2 - 1) / RT2, steps2 = (FT + F::kSlices - 1) / F::kSlices;

  if (warp == kFewWarps) {
    int issued = 0, partial = 0;
    bool ok = __all_sync(0xffffffffu, !sh->abort_flag);
    fence_proxy_async_global();
    for (int item = blockIdx.x; ok && item < items1; item += gridDim.x) {
      const int seg = item / fitems, f = item % fitems;
      const LayerMatrix W = expert_matrix<GROUP>(A.W1, &A.map1, A.W1_scale, tb.seg_expert[seg], 2 * A.F, A.H);
      const int cols = __popcll(tb.seg_mask[seg]), row = tb.seg_row[seg];
      for (int s = 0; s < steps1; ++s) {
        ok = ring_wait(ring.empty_bar(), ring.phase ^ 1, &sh->abort_flag, A.status);
        if (!ok) break;
        const int kt0 = s * F::kSlices, nk = min(F::kSlices, HT - kt0);
        copy_weights<GROUP, SP, 2>(W, f * kPairs, A.F / 16, 2 * kPairs, kt0, nk, ring.stage(), ring.stage() + sco, ring.full_bar(), lane);
        copy_tokens<F::kTokPitch>([&](int c) { return A.x8 + (size_t)tb.row_token[row + c] * HT * kTokenRecord; }, cols, kt0, nk,
                    ring.stage() + tok, ring.full_bar(), lane);
        ring.next();
        ++issued;
      }
    }
    // The down weights do not wait for the activations, only their token copies do.
    const int mine = items2 > (int)blockIdx.x ? (items2 - 1 - blockIdx.x) / gridDim.x + 1 : 0;
    const int total = mine * segs * steps2;
    FewRing late = ring;   // the stage whose activations come next
    int item = blockIdx.x, seg = 0, s = 0, lseg = 0, ls = 0;
    int begun = 0, filled = 0;
    bool met = false;
    while (ok && filled < total) {
      while (begun < total && (met ? begun == filled : begun < ring.stages)) {
        ok = ring_wait(ring.empty_bar(), ring.phase ^ 1, &sh->abort_flag, A.status);
        if (!ok) break;
        const LayerMatrix W = expert_matrix<GROUP>(A.W2, &A.map2, A.W2_scale, tb.seg_expert[seg], A.H, A.F);
        const int kt0 = s * F::kSlices, nk = min(F::kSlices, FT - kt0);
        copy_weights<GROUP, SP, 1>(W, item * RT2, 0, min(RT2, htiles - item * RT2), kt0, nk, ring.stage(), ring.stage() + sco,
                            ring.full_bar(), lane);
        ring.next();
        ++begun;
        ++issued;
        ++partial;
        if (++s == steps2) {
          s = 0;
          if (++seg == segs) { seg = 0; item += gridDim.x; }
        }
      }
      if (!ok) break;
      if (!met) {
        ok = __all_sync(0xffffffffu, grid_wait(A.counters + 2, gridDim.x, &sh->abort_flag, A.status));
        if (!ok) break;
        fence_proxy_async_global();   // the records were written by ordinary stores
        met = true;
      }
      const int kt0 = ls * F::kSlices, nk = min(F::kSlices, FT - kt0);
      const uint8_t* h8 = A.h8 + (size_t)tb.seg_row[lseg] * FT * kTokenRecord;
      copy_tokens<F::kTokPitch>([&](int c) { return h8 + (size_t)c * FT * kTokenRecord; }, __popcll(tb.seg_mask[lseg]), kt0, nk,
                  late.stage() + tok, late.full_bar(), lane);
      late.next();
      ++filled;
      --partial;
      if (++ls == steps2) {
        ls = 0;
        if (++lseg == segs) lseg = 0;
      }
    }
    drain(ring, issued, partial, lane);
  } else {
    const bool finisher = warp > kFewWarps;
    const int fid = tid - 32 * (kFewWarps + 1);   // of a finishing thread
    bool ok = consumer_sync_all(!sh->abort_flag);
    auto wait = [&](uint32_t bar, uint32_t parity) { return ok = ring_wait(bar, parity, &sh->abort_flag, A.status); };
    auto arrive = [&](uint32_t bar) {
      __syncwarp();
      if (lane == 0) mbar_arrive(bar);
    };

    if (finisher) {
      for (int item = blockIdx.x; ok && item < items1; item += gridDim.x) {
        const int seg = item / fitems, f = item % fitems;
        const int cols = __popcll(tb.seg_mask[seg]), first = tb.seg_row[seg];
        for (int pair = 0; pair < kPairs; ++pair, way.next()) {
          if (!(ok = ring_wait_idle(way.full_bar(), way.phase, &sh->abort_flag, A.status))) break;
          const float* r = reinterpret_cast<const float*>(sm + way.stage());
          for (int i = fid; i < 16 * cols; i += kFewFinishThreads) {
            const int row = i & 15, c = i >> 4;
            const float g = get_sum(r, cap, row, c) * F::kSumScale, u = get_sum(r + kFewWarps * cap * kFewColPitch, cap, row, c) * F::kSumScale;
            A.h[(size_t)(first + c) * A.F + (f * kPairs + pair) * 16 + row] = g / (1.f + expf(-g)) * u * tb.row_weight[first + c];
          }
          arrive(way.empty_bar());
        }
      }
      __threadfence();
      finish_sync();
      if (fid == 0) {
        red_release_gpu_add(A.counters + 1, 1);
        ok = ok && grid_wait(A.counters + 1, gridDim.x, &sh->abort_flag, A.status);
      }
    } else {
      for (int item = blockIdx.x; ok && item < items1; item += gridDim.x) {
        const int cols = __popcll(tb.seg_mask[item / fitems]);
        auto item_sums = [&](auto nt) {
          constexpr int NT = decltype(nt)::value;
          const LaneTokens<NT> lt((1u << cols) - 1, F::kTokPitch, lane);
          float acc[kPairs][2][NT][4] = {};
          for (int s = 0; s < steps1; ++s, ring.next()) {
            if (!wait(ring.full_bar(), ring.phase)) return;
            const uint32_t st = ring.stage();
#pragma unroll
            for (int i = warp; i < F::kSlices; i += kFewWarps)
              if (s * F::kSlices + i < HT) {
#pragma unroll
                for (int pair = 0; pair < kPairs; ++pair)
                  few_slice<GROUP, SP, 2, NT>(st + 2 * pair * F::kRowTile, st + sco, st + tok + i * kTokenRecord, zero, lt, i, lane, acc[pair]);
              }
            arrive(ring.empty_bar());
          }
#pragma unroll
          for (int pair = 0; pair < kPairs; ++pair) {
            if (!wait(way.empty_bar(), way.phase ^ 1)) return;
            put_sums<2, NT>(reinterpret_cast<float*>(sm + way.stage()), cap, cols, warp, lane, acc[pair]);
            arrive(way.full_bar());
            way.next();
          }
        };
        if (SP == 2 || DIRECT || cols <= 8)
          item_sums(std::integral_constant<int, 1>());
        else
          item_sums(std::integral_constant<int, 2>());
      }
    }
    ok = consumer_sync_all(ok);
    if (ok) {
      for (int i = (finisher ? warp - 1 : warp) * gridDim.x + blockIdx.x; i < sh->rows * FT; i += (kFewAllWarps - 1) * gridDim.x) {
        const float4 h = __ldcg(reinterpret_cast<const float4*>(A.h + (size_t)i * 128) + lane);
        const float v[4] = {h.x, h.y, h.z, h.w};
        put_record<GROUP>(v, A.h8 + (size_t)i * kTokenRecord, lane);
      }
    }
    fence_proxy_async_global();   // ordinary stores here, bulk copies there
    __threadfence();
    ok = consumer_sync_all(ok);
    if (tid == 0) red_release_gpu_add(A.counters + 2, 1);

    // Down.  DIRECT: one item's sums at a time, in one buffer; its barriers are those of
    // buffer 0, of which all fillings so far are over.
    if (DIRECT) {
      const int filled = (items1 > (int)blockIdx.x ? (items1 - 1 - blockIdx.x) / gridDim.x + 1 : 0) + 1 >> 1;   // of buffer 0
      way.slot = 0;
      way.phase = filled & 1;
      way.stages = 1;
    }
    if (finisher) {
      constexpr int kParts = kFewFinishThreads / (16 * RT2);   // threads to a row: a token's is t % kParts
      const int row = fid % (16 * RT2), part = fid / (16 * RT2);
      for (int item = blockIdx.x; ok && item < items2; item += gridDim.x) {
        const int nrt = min(RT2, htiles - item * RT2);
        if constexpr (DIRECT) {
          if (!(ok = ring_wait_idle(way.full_bar(), way.phase, &sh->abort_flag, A.status))) break;
          const float* r = reinterpret_cast<const float*>(sm + way.stage());
          for (int i = fid; i < 16 * nrt * A.T; i += kFewFinishThreads) {
            const int t = i / (16 * nrt), o = i % (16 * nrt);
            A.out[(size_t)t * A.H + item * RT2 * 16 + o] =
                to_bf16(get_sum(r + (o >> 4) * kFewWarps * A.T * kFewColPitch, A.T, o & 15, t) * F::kSumScale);
          }
          arrive(way.empty_bar());
          way.next();
        } else {
          for (int t = part; t < A.T; t += kParts) sums[t * 16 * RT2 + row] = 0.f;
          for (int seg = 0; seg < segs; ++seg, way.next()) {
            if (!(ok = ring_wait_idle(way.full_bar(), way.phase, &sh->abort_flag, A.status))) break;
            const int cols = __popcll(tb.seg_mask[seg]), first = tb.seg_row[seg];
            const float* r = reinterpret_cast<const float*>(sm + way.stage()) + (row >> 4) * kFewWarps * cap * kFewColPitch;
            for (int c = 0; c < cols; ++c) {
              const int t = tb.row_token[first + c];
              if (t % kParts == part) sums[t * 16 * RT2 + row] += get_sum(r, cap, row & 15, c);
            }
            arrive(way.empty_bar());
          }
          if (!ok) break;
          if (row < 16 * nrt)
            for (int t = part; t < A.T; t += kParts) A.out[(size_t)t * A.H + item * RT2 * 16 + row] = to_bf16(sums[t * 16 * RT2 + row] * F::kSumScale);
        }
      }
    } else {
      for (int item = blockIdx.x; ok && item < items2; item += gridDim.x) {
        if constexpr (DIRECT) {
          float acc[RT2][1][4] = {};
          for (int seg = 0; ok && seg < segs; ++seg) {
            const LaneTokens<1> lt((uint32_t)tb.seg_mask[seg], F::kTokPitch, lane);
            for (int s = 0; s < steps2; ++s, ring.next()) {
              if (!wait(ring.full_bar(), ring.phase)) break;
#pragma unroll
              for (int i = warp; i < F::kSlices; i += kFewWarps)
                if (s * F::kSlices + i < FT) few_slice<GROUP, SP, RT2, 1, true>(ring.stage(), ring.stage() + sco, ring.stage() + tok + i * kTokenRecord, zero, lt, i, lane, acc);
              arrive(ring.empty_bar());
            }
          }
          if (!ok || !wait(way.empty_bar(), way.phase ^ 1)) break;
          put_sums<RT2, 1>(reinterpret_cast<float*>(sm + way.stage()), A.T, A.T, warp, lane, acc);
          arrive(way.full_bar());
          way.next();
        } else {
          for (int seg = 0; ok && seg < segs; ++seg) {
            const int cols = __popcll(tb.seg_mask[seg]);
            auto segment_sums = [&](auto nt) {
              constexpr int NT = decltype(nt)::value;
              const LaneTokens<NT> lt((1u << cols) - 1, F::kTokPitch, lane);
              float acc[RT2][NT][4] = {};
              for (int s = 0; s < steps2; ++s, ring.next()) {
                if (!wait(ring.full_bar(), ring.phase)) return;
#pragma unroll
                for (int i = warp; i < F::kSlices; i += kFewWarps)
                  if (s * F::kSlices + i < FT) few_slice<GROUP, SP, RT2, NT>(ring.stage(), ring.stage() + sco, ring.stage() + tok + i * kTokenRecord, zero, lt, i, lane, acc);
                arrive(ring.empty_bar());
              }
              if (!wait(way.empty_bar(), way.phase ^ 1)) return;
              put_sums<RT2, NT>(reinterpret_cast<float*>(sm + way.stage()), cap, cols, warp, lane, acc);
              arrive(way.full_bar());
              way.next();
            };
            if (SP == 2 || cols <= 8)
              segment_sums(std::integral_constant<int, 1>());
            else
              segment_sums(std::integral_constant<int, 2>());
          }
        }
      }
    }
  }
}

// ---------------------------------------------------------------- the kernel

// One cooperative launch, one block per SM:
//   tokens to records, and logits; the grid meets; every block selects the
//   routes for itself and builds the same tables;
//   gate and up: items (segment, 16 features), the two row tiles of a stage
//   being the gate's and the up's rows of the same features;
//   the grid meets, the activations become records, the grid meets again;
//   meanwhile the ring already fills with the next weights;
//   down: items (RT2 row tiles of the output), each over all segments with the
//   sums of every token on chip, so the output is written once, without atomics,
//   in a fixed order.
// DIRECT (T <= 8): a token is a column of the down products, and its sums over all
// experts stay in registers (an expert adds to its own tokens' only).  Otherwise the columns are a segment's tokens, and the
// segments' sums are added up in shared memory.
template <int GROUP, int RT2, bool DIRECT>
__global__ void __launch_bounds__(kFewThreads, 1) layer_few_kernel(const __grid_constant__ LayerArgs A) {
  extern __shared__ __align__(1024) unsigned char sm[];
  FewShared* sh = reinterpret_cast<FewShared*>(sm);
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int P = A.T * A.k, HT = A.H / 128;
  const FewTables tb(sm + kTablesAt, P);
  const uint32_t after_tables = few_tables_end(P);
  const uint32_t zero = smem_u32(sm) + kZeroAt;
  unsigned char* scratch = sm + after_tables;   // until the ring takes it
  int* ids = reinterpret_cast<int*>(scratch);
  float* w = reinterpret_cast<float*>(ids + P);
  unsigned char* scratch2 = reinterpret_cast<unsigned char*>(w + P);

  few_barriers(sm, tid, FewForm<GROUP, 1>::kArrivals);
  if (tid < kTokenRecord / 4) reinterpret_cast<int*>(sm + kZeroAt)[tid] = 0;
  for (int i = warp * gridDim.x + blockIdx.x; i < A.T * HT; i += kFewAllWarps * gridDim.x) {
    const uint2 x = __ldg(reinterpret_cast<const uint2*>(A.x + (size_t)i * 128) + lane);   // the tokens' rows are blocks of 128 in a row
    const float v[4] = {bf16_lo(x.x), bf16_hi(x.x), bf16_lo(x.y), bf16_hi(x.y)};
    put_record<GROUP>(v, A.x8 + (size_t)i * kTokenRecord, lane);
  }
  if (A.router) few_logits(A, reinterpret_cast<float*>(scratch), tid, warp, lane);
  fence_proxy_async_global();   // the records are read by bulk copies
  few_meet(A, 0, sh, tid);
  if (A.router) {
    // Few tokens: every block selects for all of them.  Many: each block for its own, and the
    // grid meets once more (1.4 us; a warp takes 2 to 3 us for its first token and 1.5 for each
    // one more).
    const bool shared_out = A.T > kFewOwnTopk;
    for (int t = shared_out ? (int)blockIdx.x + (warp ? A.T : 0) : warp; t < A.T; t += shared_out ? gridDim.x : kFewAllWarps) {
      float wt;
      const float* l = A.logits + (size_t)t * A.E;
      const size_t run = (size_t)A.T * A.E;
      const int id = A.E <= 256 ? warp_topk<8>(l, run, A.splits, A.E, A.k, lane, &wt) : warp_topk<32>(l, run, A.splits, A.E, A.k, lane, &wt);
      if (lane < A.k) {
        if (!shared_out) {
          ids[t * A.k + lane] = id;
          w[t * A.k + lane] = wt;
        }
        if (shared_out || blockIdx.x == 0) {
          A.ids[t * A.k + lane] = id;
          A.w[t * A.k + lane] = wt;
        }
      }
    }
    if (shared_out) few_meet(A, 3, sh, tid);
  }
  if (!A.router || A.T > kFewOwnTopk) {
    for (int p = tid; p < P; p += kFewThreads) {
      ids[p] = __ldcg(A.ids + p);
      w[p] = __ldcg(A.w + p);
    }
  }
  __syncthreads();
  few_tables(A, sh, tb, ids, w, scratch2, tid, warp, lane);
  fence_proxy_async_shared();   // the ring's copies overwrite the scratch
  __syncthreads();

  if (layer_slices(GROUP, RT2, DIRECT, A.T, P, sh->cap, A.smem_bytes) == 2)
    layer_products<GROUP, RT2, DIRECT, GROUP != 0 ? 2 : 1>(A, sm, tb, after_tables, zero, tid, warp, lane);
  else if (GROUP == 0 || !DIRECT)
    layer_products<GROUP, RT2, DIRECT, 1>(A, sm, tb, after_tables, zero, tid, warp, lane);
  // the last block to leave clears the counters for the next call
  __syncthreads();
  if (tid == 0 && atomicAdd(A.counters + 4, 1) == (int)gridDim.x - 1) {
    for (int i = 0; i < 5; ++i) A.counters[i] = 0;
    __threadfence();
  }
}

template <int GROUP, int RT2>
int launch_layer_rt(const LayerArgs& args, int nsm, cudaStream_t s) {
  LayerArgs a = args;
  a.cols = layer_cols(GROUP, RT2, a.T <= 8, a.T, a.T * a.k, kFewMinSmem);
  return a.T <= 8 ? few_launch(layer_few_kernel<GROUP, RT2, true>, a, kFewThreads, nsm, true, s)
                  : few_launch(layer_few_kernel<GROUP, RT2, false>, a, kFewThreads, nsm, true, s);
}
template <int GROUP>
int launch_layer(const LayerArgs& a, int nsm, cudaStream_t s) {
  switch (few_row_tiles(a.H / 16, nsm)) {
    case 1: return launch_layer_rt<GROUP, 1>(a, nsm, s);
    case 2: return launch_layer_rt<GROUP, 2>(a, nsm, s);
    default: return launch_layer_rt<GROUP, 3>(a, nsm, s);
  }
}

}  // namespace moe
