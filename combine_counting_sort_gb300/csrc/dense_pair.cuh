// dense_pair.cuh: the dense product for many rows, on CTA pairs.
//
// A 2-CTA cluster takes 256 x 256 tiles of out (gated: 256 x 128, the tile's
// other 128 columns being the up rows) and runs tcgen05.mma.cta_group::2 with
// M = N = 256: each CTA loads its 128 rows of P and its half of Q's 256 rows, 32
// KiB for 64 of k, so an SM takes in 64 bytes per cycle of tensor work instead of
// the 96 of a 128 x 256 tile on its own.  Persistent: tiles are walked in a
// static order, 8 tiles of i beside one another so that what runs at one time
// shares its operands in L2, and two accumulators in tensor memory let a
// tile's epilogue run under the next tile's products.
//
// Roles per CTA (384 threads): warp 0 streams stages of both operands, warp 1 of
// the even CTA issues the products, warps 4-11 of both CTAs hold the epilogue (two
// warps a quarter of the rows, each half the columns).
//
// Bound by the tensor cores (8192 x 2048 x 7168 gated: 247 us, 1.95 PFLOP/s, in a graph; one call after
// another, under the power cap, 286; with factors 260) until an epilogue takes longer than a tile's
// products: 4096 x 7168 x 2048 65 us, with gelu_tanh 68, slope 74 and residual 83 (tensor pipe 77%
// of the active cycles); 4096 x 7168 x 512 32, the floor 15.5.
#pragma once

#include "dense.cuh"

namespace moe {

constexpr int kDPairThreads = 384;
constexpr int kDPairEpiWarp0 = 4, kDPairEpiWarps = 8;
constexpr int kDPairStages = 6;
constexpr uint32_t kDPairStageBytes = 4 * kDenseChunk;   // 128 rows of P, 128 of Q

struct DPairShared {
  uint64_t full[kDPairStages], empty[kDPairStages], tfull[2], tempty[2], drain;
  uint32_t tmem_base;
  int abort_flag;
};

constexpr size_t kDPairSmemBytes = 1024 + kDPairStages * kDPairStageBytes + kDPairEpiWarps * 2 * kBlockBytes + sizeof(DPairShared);
static_assert(kDPairSmemBytes <= 227 * 1024, "shared memory of one CTA");

struct DTile {
  int i0, j0;   // first row and column
};

// Tile t: groups of 8 tiles of i; within a group j outer, i inner.
MOE_DEV DTile dense_tile(int t, int ti, int tj, int tile_j) {
  const int g = t / (8 * tj), r = t - g * 8 * tj;
  const int rows = min(8, ti - 8 * g);
  DTile x;
  x.i0 = (8 * g + r % rows) * 256;
  x.j0 = r / rows * tile_j;
  return x;
}

// One operand's 128 rows from row r0, 64 of k from k0.
template <bool MN>
MOE_DEV void load_operand_pair(uint32_t dst, const CUtensorMap* map, int r0, int k0, uint32_t bar) {
  if (!MN) {
    tma_load_2d_pair(dst, map, k0, r0, bar);
  } else {
    tma_load_2d_pair(dst, map, r0, k0, bar);
    tma_load_2d_pair(dst + kDenseChunk, map, r0 + 64, k0, bar);
  }
}

// AUX: what the backward pass needs is written too.
template <typename T, bool PMN, bool QMN, int EPI, bool AUX>
__global__ void __launch_bounds__(kDPairThreads, 1)
    dense_pair_kernel(const __grid_constant__ CUtensorMap tmP, const __grid_constant__ CUtensorMap tmQ,
                      const __grid_constant__ DenseArgs g) {
  extern __shared__ uint8_t smem_raw[];
  uint8_t* stages = reinterpret_cast<uint8_t*>(((uintptr_t)smem_raw + 1023) & ~(uintptr_t)1023);
  uint8_t* epi_stage = stages + kDPairStages * kDPairStageBytes;
  DPairShared* sh = reinterpret_cast<DPairShared*>(epi_stage + kDPairEpiWarps * 2 * kBlockBytes);
  const int warp = threadIdx.x >> 5;
  const uint32_t rank = cluster_ctarank();
  const uint64_t tmo = g.timeout_ns;

  if (threadIdx.x == 0) {
    tma_prefetch_desc(&tmP);
    tma_prefetch_desc(&tmQ);
    for (int s = 0; s < kDPairStages; ++s) {
      mbar_init(smem_u32(&sh->full[s]), 1);    // even CTA: its producer's expect_tx arrival
      mbar_init(smem_u32(&sh->empty[s]), 1);   // the even CTA's commit, multicast
    }
    for (int p = 0; p < 2; ++p) {
      mbar_init(smem_u32(&sh->tfull[p]), 1);
      mbar_init(smem_u32(&sh->tempty[p]), 2 * kDPairEpiWarps);   // even CTA: both CTAs' epilogue warps
    }
    mbar_init(smem_u32(&sh->drain), 1);
    sh->abort_flag = 0;
    fence_mbar_init();
  }
  cluster_sync();
  if (warp == 1) {
    tmem_alloc_pair(smem_u32(&sh->tmem_base), 512);
    tmem_relinquish_pair();
  }
  tc_fence_before();
  cluster_sync();
  tc_fence_after();
  grid_launch_next();
  grid_wait_previous();

  constexpr int kTileJ = EPI == kEpiGated ? 128 : 256;
  const int ti = (g.I + 255) / 256, tj = (g.J + kTileJ - 1) / kTileJ, tiles = ti * tj;
  const int KB = (g.K + kDenseBK - 1) / kDenseBK;
  const int cluster = (int)blockIdx.x >> 1, clusters = (int)gridDim.x >> 1;

  if (warp == 0) {
    const uint32_t full_even = mapa_shared(smem_u32(&sh->full[0]), 0);
    uint32_t it = 0;
    bool ok = true;
    for (int t = cluster; t < tiles && ok; t += clusters) {
      const DTile x = dense_tile(t, ti, tj, kTileJ);
      // gated: the even CTA holds the gate rows, the odd one the up rows J further on
      const int q0 = EPI == kEpiGated ? x.j0 + (rank ? g.J : 0) : x.j0 + (int)rank * 128;
      for (int kb = 0; kb < KB; ++kb, ++it) {
        const int s = (int)(it % kDPairStages);
        ok = mbar_wait(smem_u32(&sh->empty[s]), ((it / kDPairStages) & 1u) ^ 1u, &sh->abort_flag, g.status, tmo);
        if (!ok) break;
        if (elect_one()) {
          if (rank == 0) mbar_arrive_expect_tx(smem_u32(&sh->full[s]), 2 * kDPairStageBytes);
          const uint32_t full = full_even + 8u * (uint32_t)s, dst = smem_u32(stages + (size_t)s * kDPairStageBytes);
          load_operand_pair<PMN>(dst, &tmP, x.i0 + (int)rank * 128, kb * kDenseBK, full);
          load_operand_pair<QMN>(dst + 2 * kDenseChunk, &tmQ, q0, kb * kDenseBK, full);
        }
        __syncwarp();
      }
    }
    // both CTAs' copies complete on the even CTA's barriers: none in flight at the end
    if (rank == 0) {
      int dummy = 0;
      for (uint32_t i = it > (uint32_t)kDPairStages ? it - kDPairStages : 0u; i < it; ++i)
        mbar_wait(smem_u32(&sh->full[i % kDPairStages]), (i / kDPairStages) & 1u, &dummy, nullptr, tmo);
    }
  } else if (warp == 1 && rank == 0) {
    constexpr uint32_t idesc = idesc_f16<T>(256, 256, PMN, QMN);
    const uint32_t tmem = sh->tmem_base;
    uint32_t it = 0;
    bool ok = true, issued = false;
    int n = 0;
    for (int t = cluster; t < tiles && ok; t += clusters, ++n) {
      const uint32_t p = (uint32_t)n & 1u;
      ok = mbar_wait(smem_u32(&sh->tempty[p]), (((uint32_t)n >> 1) & 1u) ^ 1u, &sh->abort_flag, g.status, tmo);
      if (!ok) break;
      tc_fence_after();
      for (int kb = 0; kb < KB; ++kb, ++it) {
        const int s = (int)(it % kDPairStages);
        ok = mbar_wait(smem_u32(&sh->full[s]), (it / kDPairStages) & 1u, &sh->abort_flag, g.status, tmo);
        if (!ok) break;
        tc_fence_after();
        const uint32_t a0 = smem_u32(stages + (size_t)s * kDPairStageBytes), b0 = a0 + 2 * kDenseChunk;
        if (elect_one()) {
#pragma unroll
          for (int k = 0; k < kDenseBK / 16; ++k)
            umma_f16_pair(tmem + p * 256, operand_desc<PMN>(a0, k), operand_desc<QMN>(b0, k), idesc, kb > 0 || k > 0 ? 1u : 0u);
          umma_commit_pair_multicast(smem_u32(&sh->empty[s]), (uint16_t)0x3);
          if (kb == KB - 1) umma_commit_pair_multicast(smem_u32(&sh->tfull[p]), (uint16_t)0x3);
        }
        __syncwarp();
        issued = true;
      }
    }
    if (issued) {   // no product may be in flight when tensor memory is freed
      int dummy = 0;
      if (elect_one()) umma_commit_pair_multicast(smem_u32(&sh->drain), (uint16_t)0x1);
      __syncwarp();
      mbar_wait(smem_u32(&sh->drain), 0u, &dummy, nullptr, tmo);
    }
  } else if (warp >= kDPairEpiWarp0) {
    const int q = warp & 3, half = (warp - kDPairEpiWarp0) >> 2;
    uint8_t* stage = epi_stage + (warp - kDPairEpiWarp0) * 2 * kBlockBytes;
    const uint32_t tmem = sh->tmem_base + ((uint32_t)(32 * q) << 16);
    const uint32_t tempty_even = mapa_shared(smem_u32(&sh->tempty[0]), 0);
    T* out = static_cast<T*>(g.out);
    T* aux = static_cast<T*>(g.aux);
    constexpr int kChunks = kTileJ / 2 / 32;   // of this warp
    int n = 0;
    for (int t = cluster; t < tiles; t += clusters, ++n) {
      const uint32_t p = (uint32_t)n & 1u;
      const DTile x = dense_tile(t, ti, tj, kTileJ);
      const int i0 = x.i0 + (int)rank * 128 + 32 * q, jw = x.j0 + half * (kTileJ / 2);
      ResidualAhead ahead;
      if (EPI == kEpiLinear) fetch_residual<T>(ahead, g, i0, jw);
      if (!mbar_wait(smem_u32(&sh->tfull[p]), ((uint32_t)n >> 1) & 1u, &sh->abort_flag, g.status, tmo)) break;
      tc_fence_after();
#pragma unroll 1
      for (int c = 0; c < kChunks; ++c) {
        const int col = half * (kTileJ / 2) + 32 * c, j0 = jw + 32 * c;
        f32x2 v[16], u[16];
        if (EPI == kEpiLinear) drain_biased<T>(tmem + p * 256 + col, v, g, j0);
        else drain_block(tmem + p * 256 + col, v);
        if (EPI == kEpiGated) drain_block(tmem + p * 256 + 128 + col, u);
        if (c == kChunks - 1) {   // the accumulator is read: the next tile may have it
          tc_fence_before();
          __syncwarp();
          if (elect_one()) mbar_arrive_cluster_relaxed(tempty_even + 8u * p);
          __syncwarp();
        }
        if (i0 >= g.I || j0 >= g.J) continue;
        if (EPI == kEpiGated) {
          if (AUX) {
            f32x2 f[16];
            with_act(g.act, [&](auto act) {
#pragma unroll
              for (int e = 0; e < 16; ++e) {
                f32x2 y, s;
                act_pair<decltype(act)::value>(v[e], y, s);
                v[e] = y;
                f[e] = mul2(s, u[e]);
                u[e] = mul2(y, u[e]);
              }
            });
            store_block(f, aux, 2LL * g.J, i0, j0, g.I, g.J, g.vec, stage);
            store_block(v, aux + g.J, 2LL * g.J, i0, j0, g.I, g.J, g.vec, stage);
          } else {
            with_act(g.act, [&](auto act) {
#pragma unroll
              for (int e = 0; e < 16; ++e) {
                f32x2 y, s;
                act_pair<decltype(act)::value>(v[e], y, s);
                u[e] = mul2(y, u[e]);
              }
            });
          }
          store_block(u, out, g.J, i0, j0, g.I, g.J, g.vec, stage);
        } else if (EPI == kEpiLinear) {
          if (g.residual) put_residual(ahead, g, i0, j0, stage + kBlockBytes);
          if (c + 1 < kChunks) fetch_residual<T>(ahead, g, i0, j0 + 32);
          if (AUX) {
            f32x2 f[16];
            with_act(g.act, [&](auto act) {
#pragma unroll
              for (int e = 0; e < 16; ++e) act_pair<decltype(act)::value>(v[e], v[e], f[e]);
            });
            store_block(f, aux, g.J, i0, j0, g.I, g.J, g.vec, stage);
          } else {
            with_act(g.act, [&](auto act) {
#pragma unroll
              for (int e = 0; e < 16; ++e) {
                f32x2 s;
                act_pair<decltype(act)::value>(v[e], v[e], s);
              }
            });
          }
          if (g.residual) add_residual<T>(v, stage + kBlockBytes);
          store_block(v, out, g.J, i0, j0, g.I, g.J, g.vec, stage);
        } else {
          store_block(v, out, g.J, i0, j0, g.I, g.J, g.vec, stage);
        }
      }
    }
  }
  tc_fence_before();
  cluster_sync();   // both CTAs done: no product, copy, commit or arrival still aimed at either
  if (warp == 1) {
    tc_fence_after();
    tmem_dealloc_pair(sh->tmem_base, 512);
  }
}

}  // namespace moe
