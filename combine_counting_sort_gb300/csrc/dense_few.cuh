// dense_few.cuh: the dense product for few rows (or few tiles): bound by
// reading Q, or by how many SMs have work.
//
// Roles are swapped against dense_pair.cuh: 128 rows j of Q (gated: 64 gate rows
// and the 64 up rows beside them) are the tensor core's M, and nt = 16 to 256
// rows i of P its N, so one row i costs a product of 128 x 16 and not one of 128 x
// 128.  The contraction is split over the CTAs of a cluster: each streams its
// share of k through a ring of stages into its own accumulator, then all lay their
// sums in shared memory, and each CTA adds up its part of the outputs over the
// cluster, in the CTAs' order, and finishes it.  No atomics, no workspace, one
// launch; results do not change from run to run.
//
// Two blocks an SM stream weights at 6.4 TB/s where there are enough of them (48 x 32768 x 7168
// 73.5 us); a call's fixed cost is launch 2 us, set-up 0.5, the first copy 1, the end 1 to 2.  One row
// of 7168 x 2048 takes 8.3 us (4.3 of them the weights' bytes).  The sums come by loads from the other
// SMs, 16 bytes a cycle; bulk copies between the SMs were no faster (11.5 us against 10.4 for 64 rows).
#pragma once

#include "dense.cuh"
#include "dense_plan.h"

namespace moe {

constexpr int kDFewThreads = 256;

struct DFewShared {
  uint64_t full[kDFewMaxStages], empty[kDFewMaxStages], tfull;
  uint32_t tmem_base;
  int abort_flag;
};

inline uint32_t dfew_stage_bytes(int nt) { return 2 * kDenseChunk + (uint32_t)nt * 128; }
inline size_t dfew_smem_bytes(int nt, int stages) { return 1024 + (size_t)stages * dfew_stage_bytes(nt) + sizeof(DFewShared); }

struct DFewPlan {
  int nt, stages, split;   // rows a tile, ring stages, CTAs a tile
  int cluster;             // CTAs a cluster: one tile's, or several tiles'
  int ti, tiles;           // tiles of i, and in all
};

MOE_DEV float ld_shared_cluster_f32(uint32_t addr) {
  float v;
  asm volatile("ld.shared::cluster.f32 %0, [%1];" : "=f"(v) : "r"(addr) : "memory");
  return v;
}

// 16 consecutive fp32 TMEM columns of this thread's lane.
MOE_DEV void tmem_drain16(uint32_t taddr, float (&v)[16]) {
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x16.b32 {%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15}, [%16];\n\t"
      "tcgen05.wait::ld.sync.aligned;"
      : "=f"(v[0]), "=f"(v[1]), "=f"(v[2]), "=f"(v[3]), "=f"(v[4]), "=f"(v[5]), "=f"(v[6]), "=f"(v[7]), "=f"(v[8]),
        "=f"(v[9]), "=f"(v[10]), "=f"(v[11]), "=f"(v[12]), "=f"(v[13]), "=f"(v[14]), "=f"(v[15])
      : "r"(taddr)
      : "memory");
}

struct Quad {
  uint32_t w[4];
};

// A thread's four columns of a tile's row.  They lie beside one another, 8 bytes a lane, where vectors
// fit (VEC), and where sums come from another SM, 16 bytes a lane.  Otherwise (APART) they lie as many
// columns apart as there are lanes on a row, so that lanes are neighbours in memory.
template <typename T, bool VEC, bool APART, int QUADS>
struct Columns {
  int r, n;   // the first column, and how many of the four the row has
  MOE_DEV Columns(int left) {
    r = (int)threadIdx.x % QUADS * (APART ? 1 : 4);
    n = min(4, APART ? (left - r + QUADS - 1) / QUADS : left - r);
  }
  static MOE_DEV int at(int e) { return APART ? e * QUADS : e; }
  // p: the first column's value.  As it comes, so that nothing waits for it here: two to a
  // word (PAIRED), or one.
  template <bool PAIRED = VEC>
  MOE_DEV Quad load(const T* p) const {
    Quad q;
    if (PAIRED) {
      const uint2 v = *reinterpret_cast<const uint2*>(p);
      q.w[0] = v.x;
      q.w[1] = v.y;
    } else {
#pragma unroll
      for (int e = 0; e < 4; ++e) q.w[e] = e < n ? reinterpret_cast<const uint16_t*>(p)[at(e)] : 0u;
    }
    return q;
  }
  template <bool PAIRED = VEC>
  static MOE_DEV f32x2 pair(const Quad& q, int k) { return Pairs<T>::one(PAIRED ? q.w[k] : q.w[2 * k] | q.w[2 * k + 1] << 16); }
  MOE_DEV void store(const f32x2* v, T* p) const {
    const T o[4] = {from_f32<T>(lo2(v[0])), from_f32<T>(hi2(v[0])), from_f32<T>(lo2(v[1])), from_f32<T>(hi2(v[1]))};
    if (VEC) {
      *reinterpret_cast<uint2*>(p) = *reinterpret_cast<const uint2*>(o);
    } else {
#pragma unroll
      for (int e = 0; e < 4; ++e)
        if (e < n) p[at(e)] = o[e];
    }
  }
  // sums of this CTA's or (REMOTE) another one's shared memory, `from` being the first column's
  template <bool REMOTE>
  static MOE_DEV void sums(uint32_t from, float* f) {
    if (!APART) {
      if (REMOTE) asm volatile("ld.shared::cluster.v4.f32 {%0, %1, %2, %3}, [%4];" : "=f"(f[0]), "=f"(f[1]), "=f"(f[2]), "=f"(f[3]) : "r"(from) : "memory");
      else asm volatile("ld.shared.v4.f32 {%0, %1, %2, %3}, [%4];" : "=f"(f[0]), "=f"(f[1]), "=f"(f[2]), "=f"(f[3]) : "r"(from) : "memory");
    } else {
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        if (REMOTE) asm volatile("ld.shared::cluster.f32 %0, [%1];" : "=f"(f[e]) : "r"(from + 4u * at(e)) : "memory");
        else asm volatile("ld.shared.f32 %0, [%1];" : "=f"(f[e]) : "r"(from + 4u * at(e)) : "memory");
      }
    }
  }
};

// A thread's bias and its first row's residual, fetched while the products run.
struct FinishAhead {
  Quad bias, residual;
};

template <typename T, int EPI, bool VEC, bool SPLIT>
MOE_DEV void fetch_ahead(FinishAhead& ahead, const DenseArgs& g, int split, int rank, int i0, int j0, int rows) {
  const Columns<T, VEC, !VEC && !SPLIT, 32> cols(g.J - j0);
  if (cols.n <= 0) return;
  const int j = j0 + cols.r, t = rank * 8 + (int)threadIdx.x / 32;
  if (g.bias) ahead.bias = cols.template load<false>(static_cast<const T*>(g.bias) + j);
  if (g.residual && t < rows) ahead.residual = cols.load(static_cast<const T*>(g.residual) + (long long)(i0 + t) * g.J + j);
}

// What finishes a tile: this thread's columns of the rows t0, t0 + step, ... below `rows`, the sums
// of the tile's CTAs (from the cluster's CTA `first` on) added up in their order.  U rows at a time, C CTAs' sums of each in flight:
// few rows want all CTAs' at once, many rows several of their own (a load from another SM takes
// some 300 cycles, one of global memory 600).
template <typename T, int EPI, bool VEC, bool SPLIT, int U, int C>
MOE_DEV void finish_rows(const DenseArgs& g, const FinishAhead& ahead, uint32_t sums, int first, int split, int rank, int i0, int j0, int rows) {
  constexpr int QUADS = EPI == kEpiGated ? 16 : 32;
  const Columns<T, VEC, !VEC && !SPLIT, QUADS> cols(g.J - j0);
  if (cols.n <= 0) return;
  const int j = j0 + cols.r, t0 = (SPLIT ? rank * (kDFewThreads / QUADS) : 0) + (int)threadIdx.x / QUADS, step = (SPLIT ? split : 1) * (kDFewThreads / QUADS);
  sums += (uint32_t)cols.r * 4u;
#pragma unroll 1
  for (int t = t0; t < rows; t += U * step) {
    Quad add[U];
    f32x2 v[U][2], w[U][2];
#pragma unroll
    for (int u = 0; u < U; ++u) {
      v[u][0] = v[u][1] = w[u][0] = w[u][1] = 0;
      if (EPI != kEpiLinear || !g.residual) continue;
      if (u == 0 && t == t0) add[u] = ahead.residual;
      else if (t + u * step < rows) add[u] = cols.load(static_cast<const T*>(g.residual) + (long long)(i0 + t + u * step) * g.J + j);
    }
#pragma unroll 1
    for (int c0 = 0; c0 < (SPLIT ? split : 1); c0 += C) {
      float a[C][U][4], b[C][U][4];
#pragma unroll
      for (int c = 0; c < C; ++c) {
        const uint32_t from = SPLIT ? mapa_shared(sums, (uint32_t)(first + min(c0 + c, split - 1))) : sums;
#pragma unroll
        for (int u = 0; u < U; ++u)
          if (t + u * step < rows && (C == 1 || c0 + c < split)) {
            cols.template sums<SPLIT>(from + (uint32_t)(t + u * step) * 512u, a[c][u]);
            if (EPI == kEpiGated) cols.template sums<SPLIT>(from + (uint32_t)(t + u * step) * 512u + 256u, b[c][u]);
          }
      }
#pragma unroll
      for (int c = 0; c < C; ++c)
#pragma unroll
        for (int u = 0; u < U; ++u)
          if (t + u * step < rows && (C == 1 || c0 + c < split)) {
            v[u][0] = add2(v[u][0], pack_f32x2(a[c][u][0], a[c][u][1]));
            v[u][1] = add2(v[u][1], pack_f32x2(a[c][u][2], a[c][u][3]));
            if (EPI == kEpiGated) {
              w[u][0] = add2(w[u][0], pack_f32x2(b[c][u][0], b[c][u][1]));
              w[u][1] = add2(w[u][1], pack_f32x2(b[c][u][2], b[c][u][3]));
            }
          }
    }
    with_act(EPI == kEpiPlain ? MOE_ACT_NONE : g.act, [&](auto act) {
#pragma unroll
      for (int u = 0; u < U; ++u) {
        if (t + u * step >= rows) break;
        const long long i = i0 + t + u * step;
        f32x2 s[2];
#pragma unroll
        for (int k = 0; k < 2; ++k) {
          if (EPI == kEpiLinear && g.bias) v[u][k] = add2(v[u][k], cols.template pair<false>(ahead.bias, k));
          act_pair<decltype(act)::value>(v[u][k], v[u][k], s[k]);
        }
        if (EPI == kEpiGated) {
          if (g.aux) {
            T* aux = static_cast<T*>(g.aux) + 2 * i * g.J + j;
            const f32x2 f[2] = {mul2(s[0], w[u][0]), mul2(s[1], w[u][1])};
            cols.store(f, aux);
            cols.store(v[u], aux + g.J);
          }
#pragma unroll
          for (int k = 0; k < 2; ++k) v[u][k] = mul2(v[u][k], w[u][k]);
        } else if (EPI == kEpiLinear) {
          if (g.aux) cols.store(s, static_cast<T*>(g.aux) + i * g.J + j);
          if (g.residual) {
            v[u][0] = add2(v[u][0], cols.template pair<VEC>(add[u], 0));
            v[u][1] = add2(v[u][1], cols.template pair<VEC>(add[u], 1));
          }
        }
        cols.store(v[u], static_cast<T*>(g.out) + i * g.J + j);
      }
    });
  }
}

template <typename T, int EPI, bool VEC>
MOE_DEV void finish(const DenseArgs& g, const FinishAhead& ahead, uint32_t sums, int first, int split, int rank, int i0, int j0, int rows) {
  constexpr int G = EPI == kEpiGated ? 2 : 1;
  if (split == 1) finish_rows<T, EPI, VEC, false, 4 / G, 1>(g, ahead, sums, first, split, rank, i0, j0, rows);
  else if (rows <= split * 8 * G) finish_rows<T, EPI, VEC, true, 1, kDFewMaxSplit>(g, ahead, sums, first, split, rank, i0, j0, rows);
  else finish_rows<T, EPI, VEC, true, 4 / G, 2>(g, ahead, sums, first, split, rank, i0, j0, rows);
}

// CTA `cta` of a product: Q's rows j are the M operand, P's rows i the N operand.
template <typename T, bool PMN, bool QMN, int EPI>
MOE_DEV void dense_few_cta(const CUtensorMap& tmP, const CUtensorMap& tmQ, const DenseArgs& g, const DFewPlan& plan, int cta) {
  extern __shared__ uint8_t smem_raw[];
  uint8_t* ring = reinterpret_cast<uint8_t*>(((uintptr_t)smem_raw + 1023) & ~(uintptr_t)1023);
  const uint32_t stage_bytes = 2 * kDenseChunk + (uint32_t)plan.nt * 128;
  DFewShared* sh = reinterpret_cast<DFewShared*>(ring + (size_t)plan.stages * stage_bytes);
  const int warp = threadIdx.x >> 5;
  const int split = plan.split, in_cluster = plan.cluster > 1 ? (int)cluster_ctarank() : 0, rank = in_cluster % split;
  const int tile = cta / split;
  if (tile >= plan.tiles) {   // fills up a cluster
    cluster_sync();
    cluster_sync();
    return;
  }
  constexpr int kRows = EPI == kEpiGated ? 64 : 128;   // columns of out a tile
  const int i0 = tile % plan.ti * plan.nt, j0 = tile / plan.ti * kRows;
  const int KB = (g.K + kDenseBK - 1) / kDenseBK;
  const int kb0 = (int)((long long)KB * rank / split), kb1 = (int)((long long)KB * (rank + 1) / split);
  const uint32_t cols = plan.nt < 32 ? 32u : (uint32_t)plan.nt;

  // The copying warp sets up the barriers by itself and fills the ring before it meets the others,
  // so the first copies do not wait for tensor memory.
  if (warp == 0) {
    const int lane = (int)threadIdx.x & 31;
    if (lane == 0) {
      tma_prefetch_desc(&tmP);
      tma_prefetch_desc(&tmQ);
      mbar_init(smem_u32(&sh->tfull), 1);
      sh->abort_flag = 0;
    }
    if (lane < plan.stages) {
      mbar_init(smem_u32(&sh->full[lane]), 1);
      mbar_init(smem_u32(&sh->empty[lane]), 1);
    }
    fence_mbar_init();
    __syncwarp();
  } else if (warp == 1) {
    tmem_alloc(smem_u32(&sh->tmem_base), cols);
    tmem_relinquish();
  }
  grid_launch_next();
  grid_wait_previous();
  // one k's stage of both operands into the ring
  auto copy_stage = [&](int kb, int s) {
    const uint32_t full = smem_u32(&sh->full[s]), q = smem_u32(ring + (size_t)s * stage_bytes), p = q + 2 * kDenseChunk;
    mbar_arrive_expect_tx(full, stage_bytes);
    const int k0 = kb * kDenseBK;
    tma_load_2d(q, &tmQ, QMN ? j0 : k0, QMN ? k0 : j0, full);
    if (QMN) tma_load_2d(q + kDenseChunk, &tmQ, j0 + 64, k0, full);
    else if (EPI == kEpiGated) tma_load_2d(q + kDenseChunk, &tmQ, k0, g.J + j0, full);
    if (PMN)
      for (int c = 0; c < plan.nt / 64; ++c) tma_load_2d(p + c * kDenseChunk, &tmP, i0 + 64 * c, k0, full);
    else
      tma_load_2d(p, &tmP, k0, i0, full);
  };
  const int first = min(plan.stages, kb1 - kb0);
  if (warp == 0) {
    if (elect_one())
      for (int s = 0; s < first; ++s) copy_stage(kb0 + s, s);
    __syncwarp();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = sh->tmem_base;

  const int tv = min(plan.nt, g.I - i0);
  FinishAhead ahead = {};
  if (EPI == kEpiLinear) {
    if (g.vec) fetch_ahead<T, EPI, true, false>(ahead, g, split, rank, i0, j0, tv);
    else if (split > 1) fetch_ahead<T, EPI, false, true>(ahead, g, split, rank, i0, j0, tv);
    else fetch_ahead<T, EPI, false, false>(ahead, g, split, rank, i0, j0, tv);
    if (g.residual && warp >= 2) {   // the rows behind the first into L2
      const int width = min(kRows, g.J - j0) * 2;
      for (int e = (int)threadIdx.x - 64 + 16; e < 2 * tv; e += kDFewThreads - 64)
        if ((e & 1) * 128 < width) prefetch_l2(static_cast<const T*>(g.residual) + (long long)(i0 + (e >> 1)) * g.J + j0 + (e & 1) * 64);
    }
  }

  if (warp == 0) {
    if (elect_one()) {
      int s = 0, issued = first;
      uint32_t ph = 0;
      for (int kb = kb0 + first; kb < kb1; ++kb) {
        if (!mbar_wait(smem_u32(&sh->empty[s]), ph, &sh->abort_flag, g.status, g.timeout_ns)) break;
        copy_stage(kb, s);
        ++issued;
        if (++s == plan.stages) { s = 0; ph ^= 1u; }
      }
      // no copy may be in flight at the end, even where a wait gave up
      int dummy = 0;
      for (int i = max(0, issued - plan.stages); i < issued; ++i)
        mbar_wait(smem_u32(&sh->full[i % plan.stages]), (uint32_t)(i / plan.stages) & 1u, &dummy, nullptr, g.timeout_ns);
    }
    __syncwarp();
  } else if (warp == 1) {
    const uint32_t idesc = idesc_f16<T>(128, 0, QMN, PMN) | ((uint32_t)(plan.nt >> 3) << 17);
    int s = 0;
    uint32_t ph = 0;
    bool ok = true;
    for (int kb = kb0; kb < kb1; ++kb) {
      ok = mbar_wait(smem_u32(&sh->full[s]), ph, &sh->abort_flag, g.status, g.timeout_ns);
      if (!ok) break;
      tc_fence_after();
      const uint32_t q = smem_u32(ring + (size_t)s * stage_bytes), p = q + 2 * kDenseChunk;
      if (elect_one()) {
#pragma unroll
        for (int k = 0; k < kDenseBK / 16; ++k)
          umma_f16(tmem, operand_desc<QMN>(q, k), operand_desc<PMN>(p, k), idesc, kb > kb0 || k > 0 ? 1u : 0u);
        umma_commit(smem_u32(&sh->empty[s]));
      }
      __syncwarp();
      if (++s == plan.stages) { s = 0; ph ^= 1u; }
    }
    // every product issued is complete (also where a wait gave up: nothing may be in flight at the end)
    if (elect_one()) umma_commit(smem_u32(&sh->tfull));
    __syncwarp();
  }
  // tfull comes even after a wait that gave up
  int dummy = 0;
  mbar_wait(smem_u32(&sh->tfull), 0u, &dummy, g.status, g.timeout_ns + g.timeout_ns / 2);
  tc_fence_after();

  // this CTA's sums, [i][j] with j contiguous, over the ring (every stage has been read)
  float* sums = reinterpret_cast<float*>(ring);
  {
    const int q = warp & 3, row = 32 * q + (threadIdx.x & 31);
    for (int c = (warp >> 2) * 16; c < tv; c += 32) {
      float v[16];
      tmem_drain16(tmem + ((uint32_t)(32 * q) << 16) + c, v);
#pragma unroll
      for (int e = 0; e < 16; ++e) sums[(c + e) * 128 + row] = v[e];
    }
  }
  tc_fence_before();
  if (plan.cluster > 1) cluster_sync();
  else __syncthreads();
  if (warp == 1) {
    tc_fence_after();
    tmem_dealloc(tmem, cols);
  }

  if (g.vec) finish<T, EPI, true>(g, ahead, smem_u32(sums), in_cluster - rank, split, rank, i0, j0, tv);
  else finish<T, EPI, false>(g, ahead, smem_u32(sums), in_cluster - rank, split, rank, i0, j0, tv);
  if (plan.cluster > 1) cluster_sync();   // no CTA leaves while another reads its sums
}

template <typename T, bool PMN, bool QMN, int EPI>
__global__ void __launch_bounds__(kDFewThreads, 2)
    dense_few_kernel(const __grid_constant__ CUtensorMap tmP, const __grid_constant__ CUtensorMap tmQ,
                     const __grid_constant__ DenseArgs g, const __grid_constant__ DFewPlan plan) {
  dense_few_cta<T, PMN, QMN, EPI>(tmP, tmQ, g, plan, (int)blockIdx.x);
}

// dx = d W (the first `first` CTAs) and dW = d^T x in one launch
struct DBoth {
  CUtensorMap P[2], Q[2];
  DenseArgs g[2];
  DFewPlan plan[2];
  int first;
};
template <typename T>
__global__ void __launch_bounds__(kDFewThreads, 2) dense_both_kernel(const __grid_constant__ DBoth b) {
  const int cta = (int)blockIdx.x;
  if (cta < b.first) dense_few_cta<T, false, true, kEpiPlain>(b.P[0], b.Q[0], b.g[0], b.plan[0], cta);
  else dense_few_cta<T, true, true, kEpiPlain>(b.P[1], b.Q[1], b.g[1], b.plan[1], cta - b.first);
}

}  // namespace moe
