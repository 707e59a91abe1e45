// few_matvec.cuh: products of up to 64 tokens with one 4-bit matrix.
//
// Codes are widened by one AND: the bits 0x000c and 0x00c0 read as bf16 are
// c * 2^-133 and 16 c * 2^-133 (bf16 is linear from its subnormals to the end of the
// first binade), so the four pairs of a word's eight codes take four ANDs and a
// shift.  The tokens are multiplied by 2^64, or by 2^60 where the code
// carries the 16, which keeps the products within fp32's normal range for any
// token value between 2^-57 and 2^63; the sums are multiplied by 2^69 at the
// end.  The 8 that every code has too much is taken out by the tensor core: a
// group's sum starts from -8 times its tokens.
// Both the AND and the shift run at 64 lanes a clock, so widening by the usual
// 0x4300 | c and a subtraction (11 instructions per 8 codes) held the kernel at
// the ALU's rate, below that of memory.
#pragma once

#include "few.cuh"
#include "few_host.h"

namespace moe {

constexpr int kMatvecCols = 16;   // tokens per pass over a stage

template <int GROUP>
struct MatvecForm {
  static constexpr int kTile = w4_tile_bytes(GROUP);
  static constexpr int kRowTile = kFewWarps * kTile;   // bytes of a row tile in a stage
  // bf16 token rows; 64 mod 128 bytes, so that the 2 rows x 64 bytes of a
  // quarter-warp's 16-byte reads fall on distinct banks
  static constexpr int kTokPitch = 2 * 128 * kFewWarps + 64;
};

// One stage's slice of a warp: RT row tiles times NT blocks of 8 tokens, the lane's
// token of a block at `row` (0: none; `b` then stays the zeros that the caller
// put there).  A stage with fewer row tiles holds older ones in their place,
// whose sums are not used.
template <int GROUP, int RT, int NT>
MOE_DEV void matvec_slice(uint32_t st, const uint32_t (&row)[2], int slice, int lane,
                          uint32_t (&b)[2][16], float (&acc)[RT][2][4]) {
  using F = MatvecForm<GROUP>;
  constexpr int kCount = FewGroups<GROUP>::kCount, kMmas = 8 / kCount;
  uint4 lo[RT], hi[RT];
  float s[RT][kCount][2];
#pragma unroll
  for (int rt = 0; rt < RT; ++rt) {
    const uint32_t w = st + rt * F::kRowTile + slice * F::kTile;
    lo[rt] = lds128(w + lane * 16);
    hi[rt] = lds128(w + 512 + lane * 16);
#pragma unroll
    for (int q = 0; q < kCount; ++q) {
      const uint32_t sc = w + kW4Codes + 32 * q + 2 * (lane >> 2);
      s[rt][q][0] = lds_bf16(sc);
      s[rt][q][1] = lds_bf16(sc + 16);
    }
  }
#pragma unroll
  for (int j = 0; j < NT; ++j) {
    if (row[j]) {
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const uint4 v = lds128(row[j] + slice * 256 + (4 * i + (lane & 3)) * 16);
        const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
        for (int p = 0; p < 4; ++p)
          asm("mul.rn.bf16x2 %0, %1, %2;" : "=r"(b[j][4 * i + p]) : "r"(w[p]), "r"(p & 1 ? 0x5D805D80u : 0x5F805F80u));
      }
    }
  }
  __syncwarp();
  // The MMAs of the row tiles, and those of the eights, are chains of their own: an
  // MMA's result takes some 20 cycles, and with two warps to a scheduler nothing
  // else would fill them.
  const uint32_t minus8[4] = {0x80088008u, 0x80088008u, 0x80808080u, 0x80808080u};   // -8, -128 times 2^-133
#pragma unroll
  for (int q = 0; q < kCount; ++q) {
    float part[RT][NT][4] = {}, eights[NT][4] = {};
#pragma unroll
    for (int m = q * kMmas; m < (q + 1) * kMmas; ++m) {
#pragma unroll
      for (int j = 0; j < NT; ++j) mma_bf16(eights[j], minus8, b[j][2 * m], b[j][2 * m + 1]);
#pragma unroll
      for (int rt = 0; rt < RT; ++rt) {
        const uint32_t l[4] = {lo[rt].x, lo[rt].y, lo[rt].z, lo[rt].w}, h[4] = {hi[rt].x, hi[rt].y, hi[rt].z, hi[rt].w};
        const uint32_t wl = l[m >> 1] >> (m & 1 ? 8 : 0), wh = h[m >> 1] >> (m & 1 ? 8 : 0);
        const uint32_t a[4] = {wl & 0x000F000Fu, wh & 0x000F000Fu, wl & 0x00F000F0u, wh & 0x00F000F0u};
#pragma unroll
        for (int j = 0; j < NT; ++j) mma_bf16(part[rt][j], a, b[j][2 * m], b[j][2 * m + 1]);
      }
    }
#pragma unroll
    for (int rt = 0; rt < RT; ++rt)
#pragma unroll
      for (int j = 0; j < NT; ++j)
#pragma unroll
        for (int i = 0; i < 4; ++i) acc[rt][j][i] = fmaf(part[rt][j][i] + eights[j][i], s[rt][q][i >> 1], acc[rt][j][i]);
  }
}

// Work items: (group of RT row tiles, pass of up to 16 tokens), the passes of a
// group next to one another so that the second finds the weights in L2.
template <int GROUP, int RT>
__global__ void __launch_bounds__(kFewThreads, 1) matvec_kernel(const MatvecArgs A) {
  extern __shared__ __align__(1024) unsigned char sm[];
  using F = MatvecForm<GROUP>;
  FewShared* sh = reinterpret_cast<FewShared*>(sm);
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int tiles = (A.N + 15) / 16, groups = (tiles + RT - 1) / RT;
  const int passes = (A.T + kMatvecCols - 1) / kMatvecCols, per = (A.T + passes - 1) / passes;
  const int items = groups * passes, KT = (A.K + 127) / 128, steps = (KT + kFewWarps - 1) / kFewWarps;
  const int tile_floats = kFewWarps * per * kFewColPitch, bufs = per <= 8 ? 2 : 1;
  constexpr uint32_t tok = RT * F::kRowTile;
  FewRing way = few_sums_ring(sm, 256, RT * tile_floats * 4, bufs);
  FewRing ring = few_ring(sm, 256 + bufs * RT * tile_floats * 4, A.smem_bytes, (tok + per * F::kTokPitch + 127) & ~127u);
  few_barriers(sm, tid, 2);
  __syncthreads();

  if (warp == kFewWarps) {
    int issued = 0;
    bool ok = true;
    for (int item = blockIdx.x; ok && item < items; item += gridDim.x) {
      const int group = item / passes, t0 = item % passes * per, cols = min(per, A.T - t0), nrt = min(RT, tiles - group * RT);
      for (int s = 0; s < steps; ++s) {
        ok = ring_wait(ring.empty_bar(), ring.phase ^ 1, &sh->abort_flag, A.status);
        if (!ok) break;
        const int kt0 = s * kFewWarps, nk = min(kFewWarps, KT - kt0), valid = min(nk * 128, A.K - kt0 * 128);
        const uint32_t st = ring.stage(), bar = ring.full_bar();
        if (valid < nk * 128) {   // zeros past K: the codes there are zero, the products must be too
          for (int c = 0; c < cols; ++c)
            for (int i = valid * 2 + lane * 16; i < nk * 256; i += 512)
              asm volatile("st.shared.v4.u32 [%0], {%1,%1,%1,%1};" :: "r"(st + tok + c * F::kTokPitch + i), "r"(0) : "memory");
          fence_proxy_async_shared();   // a later stage's bulk copy may overwrite them
          __syncwarp();
        }
        if (lane == 0) {
          mbar_arrive_expect_tx(bar, nrt * nk * F::kTile);
          mbar_arrive_expect_tx(bar, cols * valid * 2);
        }
        __syncwarp();
        if (lane < nrt)
          bulk_load(st + lane * F::kRowTile, A.W + ((size_t)(group * RT + lane) * KT + kt0) * F::kTile, nk * F::kTile, bar);
        if (lane < cols) bulk_load(st + tok + lane * F::kTokPitch, A.x + (size_t)(t0 + lane) * A.K + kt0 * 128, valid * 2, bar);
        ring.next();
        ++issued;
      }
    }
    drain(ring, issued, 0, lane);
    return;
  }

  if (warp > kFewWarps) {
    const int fid = tid - 32 * (kFewWarps + 1);
    for (int item = blockIdx.x; item < items; item += gridDim.x, way.next()) {
      if (!ring_wait_idle(way.full_bar(), way.phase, &sh->abort_flag, A.status)) return;
      const int group = item / passes, t0 = item % passes * per, cols = min(per, A.T - t0), nrt = min(RT, tiles - group * RT);
      const float* r = reinterpret_cast<const float*>(sm + way.stage());
      for (int i = fid; i < nrt * 16 * cols; i += kFewFinishThreads) {
        const int row = i % (nrt * 16), c = i / (nrt * 16), n = group * RT * 16 + row;
        if (n < A.N)
          A.y[(size_t)(t0 + c) * A.N + n] = to_bf16(get_sum(r + (row >> 4) * tile_floats, per, row & 15, c) * 0x1p69f);
      }
      __syncwarp();
      if (lane == 0) mbar_arrive(way.empty_bar());
    }
    return;
  }

  for (int item = blockIdx.x; item < items; item += gridDim.x, way.next()) {
    const int t0 = item % passes * per, cols = min(per, A.T - t0);
    float acc[RT][2][4] = {};
    uint32_t b[2][16] = {};
    for (int s = 0; s < steps; ++s, ring.next()) {
      if (!ring_wait(ring.full_bar(), ring.phase, &sh->abort_flag, A.status)) return;
      if (s * kFewWarps + warp < KT) {
        const uint32_t st = ring.stage();
        const int c = lane >> 2;
        const uint32_t row[2] = {c < cols ? st + tok + c * F::kTokPitch : 0, c + 8 < cols ? st + tok + (c + 8) * F::kTokPitch : 0};
        if (cols <= 8)
          matvec_slice<GROUP, RT, 1>(st, row, warp, lane, b, acc);
        else
          matvec_slice<GROUP, RT, 2>(st, row, warp, lane, b, acc);
      }
      __syncwarp();
      if (lane == 0) mbar_arrive(ring.empty_bar());
    }
    if (!ring_wait(way.empty_bar(), way.phase ^ 1, &sh->abort_flag, A.status)) return;
    float* red = reinterpret_cast<float*>(sm + way.stage());
#pragma unroll
    for (int rt = 0; rt < RT; ++rt)
#pragma unroll
      for (int j = 0; j < 2; ++j)
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const int col = 8 * j + 2 * (lane & 3) + (i & 1);
          if (col < cols) red[rt * tile_floats + (warp * per + col) * kFewColPitch + (lane >> 2) + 8 * (i >> 1)] = acc[rt][j][i];
        }
    __syncwarp();
    if (lane == 0) mbar_arrive(way.full_bar());
  }
}

template <int GROUP, int RT>
int launch_matvec_rt(const MatvecArgs& a, int nsm, cudaStream_t s) {
  const int groups = ((a.N + 15) / 16 + RT - 1) / RT, passes = (a.T + kMatvecCols - 1) / kMatvecCols;
  return few_launch(matvec_kernel<GROUP, RT>, a, kFewThreads, std::min(groups * passes, nsm), false, s);
}
template <int GROUP>
int launch_matvec(const MatvecArgs& a, int nsm, cudaStream_t s) {
  switch (few_row_tiles((a.N + 15) / 16, nsm)) {
    case 1: return launch_matvec_rt<GROUP, 1>(a, nsm, s);
    case 2: return launch_matvec_rt<GROUP, 2>(a, nsm, s);
    default: return launch_matvec_rt<GROUP, 3>(a, nsm, s);
  }
}

}  // namespace moe
