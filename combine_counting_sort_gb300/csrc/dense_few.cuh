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
#pragma once

#include "dense.cuh"

namespace moe {

constexpr int kDFewThreads = 256;
constexpr int kDFewMaxStages = 12;
constexpr int kDFewMaxSplit = 8;

struct DFewShared {
  uint64_t full[kDFewMaxStages], empty[kDFewMaxStages], tfull;
  uint32_t tmem_base;
  int abort_flag;
};

inline uint32_t dfew_stage_bytes(int nt) { return 2 * kDenseChunk + (uint32_t)nt * 128; }
inline size_t dfew_smem_bytes(int nt, int stages) { return 1024 + (size_t)stages * dfew_stage_bytes(nt) + sizeof(DFewShared); }

struct DFewPlan {
  int nt, stages, split;   // tokens a tile, ring stages, CTAs a cluster
  int ti;                  // tiles of i
};

MOE_DEV float4 ld_shared_cluster_f32x4(uint32_t addr) {
  float4 v;
  asm volatile("ld.shared::cluster.v4.f32 {%0, %1, %2, %3}, [%4];" : "=f"(v.x), "=f"(v.y), "=f"(v.z), "=f"(v.w) : "r"(addr) : "memory");
  return v;
}
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

// Four values, n of them there, 8 bytes at a time where they lie so.
template <typename T>
MOE_DEV uint2 load_quad(const T* p, int n, bool vec) {
  if (vec) return *reinterpret_cast<const uint2*>(p);
  const uint16_t* q = reinterpret_cast<const uint16_t*>(p);
  const uint32_t a = q[0], b = n > 1 ? q[1] : 0u, c = n > 2 ? q[2] : 0u, d = n > 3 ? q[3] : 0u;
  return make_uint2(a | b << 16, c | d << 16);
}
template <typename T>
MOE_DEV void store_quad(const f32x2* v, T* p, int n, bool vec) {
  const T o[4] = {from_f32<T>(lo2(v[0])), from_f32<T>(hi2(v[0])), from_f32<T>(lo2(v[1])), from_f32<T>(hi2(v[1]))};
  if (vec) {
    *reinterpret_cast<uint2*>(p) = *reinterpret_cast<const uint2*>(o);
  } else {
#pragma unroll
    for (int e = 0; e < 4; ++e)
      if (e < n) p[e] = o[e];
  }
}

// What finishes a tile: this thread's four columns of the rows t0, t0 + step, ..., summed over the
// CTAs' sums in their order (one row's loads from all of them in flight).  bias and
// the first row's residual were fetched while the products ran; the next row's is on its way while a
// row is worked on.  Rolled up: the code runs a few times only, and then its length counts.
template <typename T>
struct FinishAhead {
  uint2 bias, residual;
};

template <typename T, int EPI>
MOE_DEV void finish_rows(const DenseArgs& g, const FinishAhead<T>& ahead, uint32_t sums, int split, int i0, int j, int r, int t0, int step, int rows) {
  const int n = min(4, g.J - j);
  if (n <= 0) return;
  uint32_t peer[kDFewMaxSplit];
#pragma unroll
  for (int c = 0; c < kDFewMaxSplit; ++c) peer[c] = c < split ? mapa_shared(sums + r * 4u, (uint32_t)c) : 0u;
  uint2 next = ahead.residual;
#pragma unroll 1
  for (int t = t0; t < rows; t += step) {
    const long long i = i0 + t;
    const uint2 add = next;
    if (EPI == kEpiLinear && g.residual && t + step < rows) next = load_quad(static_cast<const T*>(g.residual) + (i + step) * g.J + j, n, g.vec);
    float4 a[kDFewMaxSplit], b[kDFewMaxSplit];
#pragma unroll
    for (int c = 0; c < kDFewMaxSplit; ++c)
      if (c < split) {
        a[c] = ld_shared_cluster_f32x4(peer[c] + (uint32_t)t * 512u);
        if (EPI == kEpiGated) b[c] = ld_shared_cluster_f32x4(peer[c] + (uint32_t)t * 512u + 256u);
      }
    f32x2 v[2] = {0, 0}, w[2] = {0, 0};
#pragma unroll
    for (int c = 0; c < kDFewMaxSplit; ++c)
      if (c < split) {
        v[0] = add2(v[0], pack_f32x2(a[c].x, a[c].y));
        v[1] = add2(v[1], pack_f32x2(a[c].z, a[c].w));
        if (EPI == kEpiGated) {
          w[0] = add2(w[0], pack_f32x2(b[c].x, b[c].y));
          w[1] = add2(w[1], pack_f32x2(b[c].z, b[c].w));
        }
      }
    if (EPI == kEpiLinear && g.bias) {
      v[0] = add2(v[0], Pairs<T>::one(ahead.bias.x));
      v[1] = add2(v[1], Pairs<T>::one(ahead.bias.y));
    }
    f32x2 s[2];
    with_act(EPI == kEpiPlain ? MOE_ACT_NONE : g.act, [&](auto act) {
#pragma unroll
      for (int k = 0; k < 2; ++k) act_pair<decltype(act)::value>(v[k], v[k], s[k]);
    });
    if (EPI == kEpiGated) {
      if (g.aux) {
        const f32x2 f[2] = {mul2(s[0], w[0]), mul2(s[1], w[1])};
        T* aux = static_cast<T*>(g.aux) + 2 * i * g.J + j;
        store_quad(f, aux, n, g.vec);
        store_quad(v, aux + g.J, n, g.vec);
      }
#pragma unroll
      for (int k = 0; k < 2; ++k) v[k] = mul2(v[k], w[k]);
    } else if (EPI == kEpiLinear) {
      if (g.aux) store_quad(s, static_cast<T*>(g.aux) + i * g.J + j, n, g.vec);
      if (g.residual) {
        v[0] = add2(v[0], Pairs<T>::one(add.x));
        v[1] = add2(v[1], Pairs<T>::one(add.y));
      }
    }
    store_quad(v, static_cast<T*>(g.out) + i * g.J + j, n, g.vec);
  }
}

// Q's rows j are the M operand, P's rows i the N operand.
template <typename T, bool PMN, bool QMN, int EPI>
__global__ void __launch_bounds__(kDFewThreads)
    dense_few_kernel(const __grid_constant__ CUtensorMap tmP, const __grid_constant__ CUtensorMap tmQ,
                     const __grid_constant__ DenseArgs g, const DFewPlan plan) {
  extern __shared__ uint8_t smem_raw[];
  uint8_t* ring = reinterpret_cast<uint8_t*>(((uintptr_t)smem_raw + 1023) & ~(uintptr_t)1023);
  const uint32_t stage_bytes = 2 * kDenseChunk + (uint32_t)plan.nt * 128;
  DFewShared* sh = reinterpret_cast<DFewShared*>(ring + (size_t)plan.stages * stage_bytes);
  const int warp = threadIdx.x >> 5;
  const int split = plan.split, rank = split > 1 ? (int)cluster_ctarank() : 0;
  const int tile = (int)blockIdx.x / split;
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

  // what this thread finishes: four columns of the rows t0, t0 + step, ...
  constexpr int kQuads = kRows / 4;
  const int tv = min(plan.nt, g.I - i0), r = (int)threadIdx.x % kQuads * 4;
  const int t0 = rank * (kDFewThreads / kQuads) + (int)threadIdx.x / kQuads, step = split * (kDFewThreads / kQuads);
  FinishAhead<T> ahead = {};
  if (EPI == kEpiLinear && j0 + r < g.J) {
    const int n = min(4, g.J - j0 - r);
    if (g.bias) ahead.bias = load_quad(static_cast<const T*>(g.bias) + j0 + r, n, g.bias_vec);
    if (g.residual && t0 < tv) ahead.residual = load_quad(static_cast<const T*>(g.residual) + (long long)(i0 + t0) * g.J + j0 + r, n, g.vec);
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
  if (split > 1) cluster_sync();
  else __syncthreads();
  if (warp == 1) {
    tc_fence_after();
    tmem_dealloc(tmem, cols);
  }

  finish_rows<T, EPI>(g, ahead, smem_u32(sums), split, i0, j0 + r, r, t0, step, tv);
  if (split > 1) cluster_sync();   // no CTA leaves while another reads its sums
}

}  // namespace moe
