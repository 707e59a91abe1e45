// few_kernels.cuh: the decoding kernels, instantiated per weight form.
#pragma once

#include "few.cuh"
#include "few_host.h"
#include "router.cuh"

namespace moe {

// Barriers of the ring and the block's flags at the start of shared memory.
struct FewShared {
  uint64_t full[kFewMaxStages], empty[kFewMaxStages];
  volatile int abort_flag;
  int segs, cap, rows;
};
static_assert(sizeof(FewShared) <= 256, "");

// Ring geometry in the `bytes` of shared memory behind offset `at`, barriers
// initialised by the calling thread 0; the caller synchronises the block.
MOE_DEV FewRing few_ring(unsigned char* sm, uint32_t at, uint32_t smem_bytes, uint32_t stage_bytes, int arrivals) {
  FewShared* sh = reinterpret_cast<FewShared*>(sm);
  FewRing r;
  at = (at + 127) & ~127u;
  r.base = smem_u32(sm) + at;
  r.stage_bytes = stage_bytes;
  r.full = smem_u32(sh->full);
  r.empty = smem_u32(sh->empty);
  r.stages = min((int)((smem_bytes - at) / stage_bytes), kFewMaxStages);
  r.slot = r.phase = 0;
  if (threadIdx.x == 0) {
    for (int i = 0; i < r.stages; ++i) {
      mbar_init(r.full + 8 * i, arrivals);
      mbar_init(r.empty + 8 * i, kFewWarps);
    }
    fence_mbar_init();
  }
  return r;
}

// The copying warp's end: every stage it has begun is complete before the block
// leaves.  `issued` stages were begun in all; the last `partial` of them still
// lack their tokens (an abandoned wait), whose arrivals are made up for.
MOE_DEV void drain(FewRing r, int issued, int partial, int lane) {
  // r is positioned behind the last stage begun
  const int n = min(issued, r.stages);
  for (int i = 0; i < n; ++i) {
    if (r.slot == 0) { r.slot = r.stages; r.phase ^= 1; }
    --r.slot;
    if (i < partial && lane == 0) mbar_arrive(r.full_bar());
    const uint64_t t0 = globaltimer_ns();   // bounded; it runs out only if a copy never lands
    while (!mbar_try_wait(r.full_bar(), r.phase) && globaltimer_ns() - t0 < kFewTimeoutNs) {}
  }
}

// ---------------------------------------------------------------- matrix-vector products

// Work items: (group of RT row tiles, pass of up to 16 tokens), the passes of a
// group next to one another so that the second finds the weights in L2.
template <int GROUP, int RT>
__global__ void __launch_bounds__(kFewThreads, 1) matvec_kernel(const MatvecArgs A) {
  extern __shared__ __align__(128) unsigned char sm[];
  using F = FewForm<GROUP>;
  FewShared* sh = reinterpret_cast<FewShared*>(sm);
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int tiles = (A.N + 15) / 16, groups = (tiles + RT - 1) / RT;
  const int passes = (A.T + kFewMaxCols - 1) / kFewMaxCols, per = (A.T + passes - 1) / passes;
  const int items = groups * passes, KT = (A.K + 127) / 128, steps = (KT + kFewWarps - 1) / kFewWarps;
  const int nt = per > 8 ? 2 : 1;
  float* red = reinterpret_cast<float*>(sm + 256);
  const int red_floats = kFewWarps * RT * nt * 128;
  FewRing ring = few_ring(sm, 256 + 2 * red_floats * 4, A.smem_bytes, few_stage_bytes<GROUP>(RT, per), F::kArrivals);
  if (tid == 0) sh->abort_flag = 0;
  __syncthreads();
  const uint32_t tok = RT * F::kRowTile;

  if (warp == kFewWarps) {
    int issued = 0;
    for (int item = blockIdx.x; item < items; item += gridDim.x) {
      const int group = item / passes, t0 = item % passes * per, cols = min(per, A.T - t0);
      const FewMatrix W{A.W, nullptr, A.K};
      for (int s = 0; s < steps; ++s) {
        if (!ring_wait(ring.empty_bar(), ring.phase ^ 1, &sh->abort_flag, A.status)) goto done;
        const int kt0 = s * kFewWarps, nk = min(kFewWarps, KT - kt0);
        copy_weights<GROUP>(W, group * RT, 1, min(RT, tiles - group * RT), kt0, nk, ring.stage(), 0, ring.full_bar(), lane);
        copy_tokens<GROUP>([&](int c) { return A.x + (size_t)(t0 + c) * A.K; }, cols, A.K, kt0, nk, ring.stage() + tok,
                           ring.full_bar(), lane);
        ring.next();
        ++issued;
      }
    }
  done:
    drain(ring, issued, 0, lane);
    return;
  }

  int buf = 0;
  bool ok = true;
  for (int item = blockIdx.x; item < items; item += gridDim.x) {
    const int group = item / passes, t0 = item % passes * per, cols = min(per, A.T - t0);
    const int nrt = min(RT, tiles - group * RT);
    float acc[RT][2][4] = {};
    for (int s = 0; s < steps; ++s) {
      ok = ring_wait(ring.full_bar(), ring.phase, &sh->abort_flag, A.status);
      if (!ok) break;
      if (s * kFewWarps + warp < KT) {
        const uint32_t st = ring.stage();
        const int c = lane >> 2;
        const uint32_t t0r = c < cols ? st + tok + c * F::kTokPitch : 0, t1r = c + 8 < cols ? st + tok + (c + 8) * F::kTokPitch : 0;
        if (cols <= 8) {
          const uint32_t rows[1] = {t0r};
          slice_columns<GROUP, RT, 1, 2>(st, 0, rows, warp, lane, nrt, acc);
        } else {
          const uint32_t rows[2] = {t0r, t1r};
          slice_columns<GROUP, RT, 2, 2>(st, 0, rows, warp, lane, nrt, acc);
        }
      }
      __syncwarp();
      if (lane == 0) mbar_arrive(ring.empty_bar());
      ring.next();
    }
    float* r = red + buf * red_floats;
#pragma unroll
    for (int rt = 0; rt < RT; ++rt)
#pragma unroll
      for (int j = 0; j < 2; ++j)
        if (j < nt) put_block(r, RT * nt, warp, rt * nt + j, lane, acc[rt][j]);
    // two buffers: a warp reaches the next item's meeting only after it has read this one's
    if (!consumer_sync_all(ok)) return;
    for (int i = tid; i < nrt * 16 * cols; i += 256) {
      const int row = i % (nrt * 16), c = i / (nrt * 16);
      const int n = group * RT * 16 + row;
      if (n < A.N) A.y[(size_t)(t0 + c) * A.N + n] = to_bf16(get_sum(r, RT * nt, (row >> 4) * nt + (c >> 3), row & 15, c & 7));
    }
    buf ^= 1;
  }
}

// ---------------------------------------------------------------- the layer

// Tables of the routes in shared memory, sized by the P = T k pairs.  A segment is
// one expert and up to 16 of the tokens routed to it; row r of the activations
// belongs to one (token, expert).
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

// logits[t, e] for the experts of this block: each warp takes every eighth chunk of
// 256 columns, the partial sums meet in shared memory in the warps' order.
MOE_DEV void few_logits(const LayerArgs& A, float* part, int tid, int warp, int lane) {
  for (int e = blockIdx.x; e < A.E; e += gridDim.x) {
    if (warp < kFewWarps) {
      for (int t = 0; t < A.T; ++t) {
        float s = 0.f;
        for (int c = warp * 256 + lane * 8; c < A.H; c += kFewWarps * 256) {
          const uint4 r = __ldg(reinterpret_cast<const uint4*>(A.router + (size_t)e * A.H + c));
          const uint4 v = __ldg(reinterpret_cast<const uint4*>(A.x + (size_t)t * A.H + c));
          const uint32_t rw[4] = {r.x, r.y, r.z, r.w}, vw[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
          for (int i = 0; i < 4; ++i) s = fmaf(bf16_hi(rw[i]), bf16_hi(vw[i]), fmaf(bf16_lo(rw[i]), bf16_lo(vw[i]), s));
        }
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) s += __shfl_xor_sync(0xffffffffu, s, o);
        if (lane == 0) part[warp * A.T + t] = s;
      }
    }
    __syncthreads();
    if (tid < A.T) {
      float s = 0.f;
      for (int w = 0; w < kFewWarps; ++w) s += part[w * A.T + tid];
      A.logits[(size_t)tid * A.E + e] = s;
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

// The tables from the pairs' ids and weights (in shared memory).  scratch: E masks,
// E first rows.
MOE_DEV void few_tables(const LayerArgs& A, FewShared* sh, const FewTables& tb, const int* ids, const float* w,
                        unsigned char* scratch, int tid, int warp, int lane) {
  const int P = A.T * A.k;
  uint64_t* mask = reinterpret_cast<uint64_t*>(scratch);
  int* first = reinterpret_cast<int*>(mask + A.E);
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
  if (warp == 0) {
    int rows = 0, segs = 0, most = 0;
    for (int e0 = 0; e0 < A.E; e0 += 32) {
      const int e = e0 + lane;
      uint64_t m = e < A.E ? mask[e] : 0;
      const int c = __popcll(m), s = (c + kFewMaxCols - 1) / kFewMaxCols;
      int incl = c | s << 16;   // at most 1024 rows and 1024 segments
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const int v = __shfl_up_sync(0xffffffffu, incl, o);
        if (lane >= o) incl += v;
      }
      const int row = rows + (incl & 0xFFFF) - c, seg = segs + (incl >> 16) - s;
      if (e < A.E) first[e] = row;
      for (int i = 0; i < s; ++i) {
        uint64_t take = m;
        if (__popcll(m) > kFewMaxCols) {
          take = 0;
          for (int b = 0; b < kFewMaxCols; ++b) {
            const uint64_t low = m & (~m + 1);
            take |= low;
            m ^= low;
          }
        }
        tb.seg_mask[seg + i] = take;
        tb.seg_expert[seg + i] = e;
        tb.seg_row[seg + i] = row + i * kFewMaxCols;
      }
      most = max(most, c);
      const int all = __shfl_sync(0xffffffffu, incl, 31);
      rows += all & 0xFFFF;
      segs += all >> 16;
    }
    most = __reduce_max_sync(0xffffffffu, most);
    if (lane == 0) {
      sh->segs = segs;
      sh->rows = rows;
      sh->cap = min(most, kFewMaxCols);
    }
  }
  __syncthreads();
  if (tid < A.T) {   // a token that names an expert again adds to its weight, in slot order
    for (int j = 0; j < A.k; ++j) {
      const int e = ids[tid * A.k + j];
      if (e < 0 || e >= A.E) continue;
      bool again = false;
      for (int i = 0; i < j; ++i) again |= ids[tid * A.k + i] == e;
      const int row = first[e] + __popcll(mask[e] & ((1ull << tid) - 1));
      tb.row_token[row] = (uint8_t)tid;
      tb.row_weight[row] = again ? tb.row_weight[row] + w[tid * A.k + j] : w[tid * A.k + j];
    }
  }
}

template <int GROUP>
MOE_DEV FewMatrix expert_matrix(const uint8_t* W, const float* scale, int e, int N, int K) {
  if (GROUP != 0) return FewMatrix{W + (size_t)e * w4_matrix_bytes(N, K, GROUP ? GROUP : 128), nullptr, K};
  return FewMatrix{W + (size_t)e * N * K, scale + (size_t)e * (N / 128) * (K / 128), K};
}

// One cooperative launch, one block per SM:
//   routes: logits, one grid-wide meeting, then every block selects for itself
//   and builds the same tables;
//   gate and up: items (segment, 16 features), the RT = 2 row tiles of a stage
//   being the gate's and the up's rows of the same features;
//   one grid-wide meeting, during which the ring already fills with
//   the next weights;
//   down: items (RT2 row tiles of the output), each over all segments with the
//   sums of every token in registers, so the output is written once, without
//   atomics, in a fixed order.
// NT: blocks of 8 token columns that the down sums cover (T <= 8 NT).
template <int GROUP, int RT2, int NT>
__global__ void __launch_bounds__(kFewThreads, 1) layer_few_kernel(const LayerArgs A) {
  extern __shared__ __align__(128) unsigned char sm[];
  using F = FewForm<GROUP>;
  constexpr int kRT = RT2 > 2 ? RT2 : 2;
  FewShared* sh = reinterpret_cast<FewShared*>(sm);
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int P = A.T * A.k;
  const FewTables tb(sm + 256, P);
  const uint32_t after_tables = (256 + P * 21 + 127) & ~127;
  unsigned char* scratch = sm + after_tables;   // until the ring takes it
  int* ids = reinterpret_cast<int*>(scratch);
  float* w = reinterpret_cast<float*>(ids + P);
  unsigned char* scratch2 = reinterpret_cast<unsigned char*>(w + P);

  if (tid == 0) sh->abort_flag = 0;
  if (A.router) {
    few_logits(A, reinterpret_cast<float*>(scratch), tid, warp, lane);   // ends with __syncthreads
    if (tid == 0) {
      __threadfence();
      red_release_gpu_add(A.counters, 1);
      grid_wait(A.counters, gridDim.x, &sh->abort_flag, A.status);
    }
    __syncthreads();
    for (int t = warp; t < A.T; t += kFewWarps + 1) {
      float wt;
      const float* l = A.logits + (size_t)t * A.E;
      const int id = A.E <= 256 ? warp_topk<8>(l, A.E, A.k, lane, &wt) : warp_topk<32>(l, A.E, A.k, lane, &wt);
      if (lane < A.k) {
        ids[t * A.k + lane] = id;
        w[t * A.k + lane] = wt;
        if (blockIdx.x == 0) {
          A.ids[t * A.k + lane] = id;
          A.w[t * A.k + lane] = wt;
        }
      }
    }
  } else {
    for (int p = tid; p < P; p += kFewThreads) {
      ids[p] = A.ids[p];
      w[p] = A.w[p];
    }
  }
  __syncthreads();
  few_tables(A, sh, tb, ids, w, scratch2, tid, warp, lane);
  fence_proxy_async_shared();   // the ring's copies overwrite the scratch
  __syncthreads();

  const int segs = sh->segs, cap = max(sh->cap, 1), nt = cap > 8 ? 2 : 1;
  float* red = reinterpret_cast<float*>(sm + after_tables);
  const int red_floats = kFewWarps * 2 * nt * 128;
  FewRing ring = few_ring(sm, after_tables + 2 * red_floats * 4, A.smem_bytes, few_stage_bytes<GROUP>(kRT, cap), F::kArrivals);
  __syncthreads();
  const uint32_t tok = kRT * F::kRowTile, sco = tok + cap * F::kTokPitch;
  const int ftiles = A.F / 16, items1 = segs * ftiles, steps1 = (A.H / 128 + kFewWarps - 1) / kFewWarps;
  const int htiles = A.H / 16, items2 = (htiles + RT2 - 1) / RT2, steps2 = (A.F / 128 + kFewWarps - 1) / kFewWarps;

  if (warp == kFewWarps) {
    int issued = 0, partial = 0;
    bool ok = __all_sync(0xffffffffu, !sh->abort_flag);
    for (int item = blockIdx.x; ok && item < items1; item += gridDim.x) {
      const int seg = item / ftiles, f = item % ftiles;
      const FewMatrix W = expert_matrix<GROUP>(A.W1, A.W1_scale, tb.seg_expert[seg], 2 * A.F, A.H);
      const int cols = __popcll(tb.seg_mask[seg]), row = tb.seg_row[seg];
      for (int s = 0; s < steps1; ++s) {
        ok = ring_wait(ring.empty_bar(), ring.phase ^ 1, &sh->abort_flag, A.status);
        if (!ok) break;
        const int kt0 = s * kFewWarps, nk = min(kFewWarps, A.H / 128 - kt0);
        copy_weights<GROUP>(W, f, ftiles, 2, kt0, nk, ring.stage(), ring.stage() + sco, ring.full_bar(), lane);
        copy_tokens<GROUP>([&](int c) { return A.x + (size_t)tb.row_token[row + c] * A.H; }, cols, A.H, kt0, nk,
                           ring.stage() + tok, ring.full_bar(), lane);
        ring.next();
        ++issued;
      }
    }
    // The down weights do not wait for the activations, only their token copies do.
    const int mine = items2 > (int)blockIdx.x ? (items2 - 1 - blockIdx.x) / gridDim.x + 1 : 0;
    const int total = mine * segs * steps2;
    FewRing late = ring;   // the stage whose activations come next
    int item = blockIdx.x, seg = 0, s = 0, litem_seg = 0, ls = 0;
    int begun = 0, filled = 0;
    bool met = false;
    while (ok && filled < total) {
      while (begun < total && (met ? begun == filled : begun < ring.stages)) {
        ok = ring_wait(ring.empty_bar(), ring.phase ^ 1, &sh->abort_flag, A.status);
        if (!ok) break;
        const FewMatrix W = expert_matrix<GROUP>(A.W2, A.W2_scale, tb.seg_expert[seg], A.H, A.F);
        const int kt0 = s * kFewWarps, nk = min(kFewWarps, A.F / 128 - kt0);
        copy_weights<GROUP>(W, item * RT2, 1, min(RT2, htiles - item * RT2), kt0, nk, ring.stage(), ring.stage() + sco,
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
        ok = grid_wait(A.counters + 1, gridDim.x, &sh->abort_flag, A.status);
        ok = __all_sync(0xffffffffu, ok);
        if (!ok) break;
        fence_proxy_async_global();   // the activations were written by ordinary stores
        met = true;
      }
      const int kt0 = ls * kFewWarps, nk = min(kFewWarps, A.F / 128 - kt0);
      const uint16_t* h = A.h + (size_t)tb.seg_row[litem_seg] * A.F;
      copy_tokens<GROUP>([&](int c) { return h + (size_t)c * A.F; }, __popcll(tb.seg_mask[litem_seg]), A.F, kt0, nk,
                         late.stage() + tok, late.full_bar(), lane);
      late.next();
      ++filled;
      --partial;
      if (++ls == steps2) {
        ls = 0;
        if (++litem_seg == segs) litem_seg = 0;
      }
    }
    drain(ring, issued, partial, lane);
  } else {
    bool ok = consumer_sync_all(!sh->abort_flag);
    int buf = 0;
    for (int item = blockIdx.x; ok && item < items1; item += gridDim.x) {
      const int seg = item / ftiles, f = item % ftiles;
      const int cols = __popcll(tb.seg_mask[seg]), row = tb.seg_row[seg];
      float acc[2][2][4] = {};
      for (int s = 0; s < steps1; ++s) {
        ok = ring_wait(ring.full_bar(), ring.phase, &sh->abort_flag, A.status);
        if (!ok) break;
        if (s * kFewWarps + warp < A.H / 128) {
          const uint32_t st = ring.stage();
          const int c = lane >> 2;
          const uint32_t r0 = c < cols ? st + tok + c * F::kTokPitch : 0, r1 = c + 8 < cols ? st + tok + (c + 8) * F::kTokPitch : 0;
          if (cols <= 8) {
            const uint32_t rows[1] = {r0};
            slice_columns<GROUP, 2, 1, 2>(st, st + sco, rows, warp, lane, 2, acc);
          } else {
            const uint32_t rows[2] = {r0, r1};
            slice_columns<GROUP, 2, 2, 2>(st, st + sco, rows, warp, lane, 2, acc);
          }
        }
        __syncwarp();
        if (lane == 0) mbar_arrive(ring.empty_bar());
        ring.next();
      }
      float* r = red + buf * red_floats;
#pragma unroll
      for (int rt = 0; rt < 2; ++rt)
#pragma unroll
        for (int j = 0; j < 2; ++j)
          if (j < nt) put_block(r, 2 * nt, warp, rt * nt + j, lane, acc[rt][j]);
      // two buffers: a warp reaches the next item's meeting only after it has read this one's
      ok = consumer_sync_all(ok);
      if (ok && tid < 16 * cols) {
        const int i = tid & 15, c = tid >> 4;
        const float g = get_sum(r, 2 * nt, c >> 3, i, c & 7), u = get_sum(r, 2 * nt, nt + (c >> 3), i, c & 7);
        A.h[(size_t)(row + c) * A.F + f * 16 + i] = to_bf16(g / (1.f + expf(-g)) * u * tb.row_weight[row + c]);
      }
      buf ^= 1;
    }
    // the activations: ordinary stores here, bulk copies there
    fence_proxy_async_global();
    __threadfence();
    ok = consumer_sync_all(ok);
    if (tid == 0) red_release_gpu_add(A.counters + 1, 1);

    const int first_red = kFewWarps * 2 * 128;   // two blocks per buffer
    buf = 0;
    for (int item = blockIdx.x; ok && item < items2; item += gridDim.x) {
      const int nrt = min(RT2, htiles - item * RT2);
      float acc[RT2][NT][4] = {};
      for (int seg = 0; ok && seg < segs; ++seg) {
        const uint64_t mask = tb.seg_mask[seg];
        for (int s = 0; s < steps2; ++s) {
          ok = ring_wait(ring.full_bar(), ring.phase, &sh->abort_flag, A.status);
          if (!ok) break;
          if (s * kFewWarps + warp < A.F / 128) {
            const uint32_t st = ring.stage();
            if (NT == 1) {
              const int t = lane >> 2;
              const uint32_t rows[1] = {(mask >> t) & 1 ? st + tok + __popcll(mask & ((1ull << t) - 1)) * F::kTokPitch : 0};
              slice_columns<GROUP, RT2, 1, NT>(st, st + sco, rows, warp, lane, nrt, acc);
            } else {
              slice_masked<GROUP, RT2, NT>(st, st + sco, st + tok, mask, warp, lane, nrt, acc);
            }
          }
          __syncwarp();
          if (lane == 0) mbar_arrive(ring.empty_bar());
          ring.next();
        }
      }
      ok = consumer_sync_all(ok);
      if (!ok) break;
#pragma unroll
      for (int b0 = 0; b0 < RT2 * NT; b0 += 2) {
        // block b is row tile b % RT2 of token block b / RT2: the blocks past the batch come last
        if (8 * (b0 / RT2) < A.T) {
          float* r = red + buf * first_red;
#pragma unroll
          for (int i = 0; i < 2; ++i)
            if (b0 + i < RT2 * NT) put_block(r, 2, warp, i, lane, acc[(b0 + i) % RT2][(b0 + i) / RT2]);
          consumer_sync();
          const int b = b0 + (tid >> 7), rt = b % RT2, t = 8 * (b / RT2) + ((tid >> 4) & 7), i = tid & 15;
          if (b < RT2 * NT && rt < nrt && t < A.T)
            A.out[(size_t)t * A.H + (item * RT2 + rt) * 16 + i] = to_bf16(get_sum(r, 2, tid >> 7, i, t & 7));
          buf ^= 1;
        }
      }
    }
  }
  // the last block to leave clears the counters for the next call
  __syncthreads();
  if (tid == 0 && atomicAdd(A.counters + 2, 1) == (int)gridDim.x - 1) {
    A.counters[0] = A.counters[1] = A.counters[2] = 0;
    __threadfence();
  }
}

// ---------------------------------------------------------------- launches

// Row tiles per item: the fewest (rounds over the SMs) x (row tiles), and of
// those the most row tiles, since a stage's tokens are shared by its row tiles.
inline int few_row_tiles(int tiles, int nsm) {
  int best = 1, cost = 1 << 30;
  for (int rt = 1; rt <= 3; ++rt) {
    const int groups = (tiles + rt - 1) / rt, c = (groups + nsm - 1) / nsm * rt;
    if (c <= cost) { cost = c; best = rt; }
  }
  return best;
}

template <class Kernel, class Args>
int few_launch(Kernel kernel, Args a, int blocks, bool cooperative, cudaStream_t s) {
  int dev = 0, smem = 0;
  if (cudaGetDevice(&dev) != cudaSuccess) return MOE_ERR_CUDA;
  if (cudaDeviceGetAttribute(&smem, cudaDevAttrMaxSharedMemoryPerBlockOptin, dev) != cudaSuccess) return MOE_ERR_CUDA;
  if (smem < kFewMinSmem) return MOE_ERR_UNSUPPORTED;
  if (cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, smem) != cudaSuccess) return MOE_ERR_CUDA;
  a.smem_bytes = smem;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(blocks);
  cfg.blockDim = dim3(kFewThreads);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = s;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeCooperative;
  attr[0].val.cooperative = cooperative ? 1 : 0;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, kernel, a) == cudaSuccess ? MOE_OK : MOE_ERR_CUDA;
}

template <int GROUP, int RT>
int launch_matvec_rt(const MatvecArgs& a, int nsm, cudaStream_t s) {
  const int groups = ((a.N + 15) / 16 + RT - 1) / RT, passes = (a.T + kFewMaxCols - 1) / kFewMaxCols;
  return few_launch(matvec_kernel<GROUP, RT>, a, std::min(groups * passes, nsm), false, s);
}
template <int GROUP>
int launch_matvec(const MatvecArgs& a, int nsm, cudaStream_t s) {
  switch (few_row_tiles((a.N + 15) / 16, nsm)) {
    case 1: return launch_matvec_rt<GROUP, 1>(a, nsm, s);
    case 2: return launch_matvec_rt<GROUP, 2>(a, nsm, s);
    default: return launch_matvec_rt<GROUP, 3>(a, nsm, s);
  }
}

template <int GROUP, int RT2>
int launch_layer_rt(const LayerArgs& a, int nsm, cudaStream_t s) {
  return a.T <= 8 ? few_launch(layer_few_kernel<GROUP, RT2, 1>, a, nsm, true, s)
                  : few_launch(layer_few_kernel<GROUP, RT2, 8>, a, nsm, true, s);
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
