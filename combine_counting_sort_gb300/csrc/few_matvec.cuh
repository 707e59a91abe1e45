// few_matvec.cuh: products of up to 64 tokens with one 4-bit matrix, in three kernels.
//
// matvec_few_kernel, one token, or up to four on few columns or many rows: every block makes
// the records of all tokens for itself while its first weights are on their way, and a
// stage holds weights alone (few_slice.cuh: the products).  Bound by memory and the products with
// many rows (152064 x 4096, groups of 64, one token: 57.3 us, 5.8 TB/s), with few by the way through the
// block: launch, records, first copies, sums (4096 x 7168, groups of 128: 6.65 us, of which the
// weights are 2.2; a microsecond more with the records' loads one after the other).
//
// matvec_wide_kernel, up to 16 tokens and few rows: a block of eight warps is KS slices of 128
// columns x 8 / KS groups of 32 rows, each warp all tokens (one or two blocks of 8) on its 32
// rows, so that a code is widened once for all of them: to bf16, 0x4300 | c less 136.  With
// few rows the slices are many, so that every SM has work, and their sums meet in shared
// memory; with many rows they are few, since every block reads all tokens.  A copy costs
// some 70 cycles of an SM's copies whatever its size, so a stage's weights are one box of
// whole tiles, its tokens another (with one to 64 columns 4096 x 7168 and 8 tokens took 7.8 us).
//
// matvec_tensor_kernel (few_tensor.cuh), the rest: more than 16 tokens, or more rows than four
// row tiles per SM.
#pragma once

#include "few_slice.cuh"
#include "few_tensor.cuh"

namespace moe {

constexpr int kMatvecTokenRoom = 96 * 1024;   // of the few kernel's records beside two stages of two row tiles; half of it beside three

__host__ __device__ __forceinline__ int matvec_token_pitch(int KT) { return ((KT * kTokenRecord + 127) & ~127) + 64; }

template <int GROUP, int RT>
__global__ void __launch_bounds__(kFewThreads, 1) matvec_few_kernel(const __grid_constant__ MatvecArgs A) {
  extern __shared__ __align__(1024) unsigned char sm[];
  using F = FewForm<GROUP, 2>;
  FewShared* sh = reinterpret_cast<FewShared*>(sm);
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int tiles = (A.N + 15) / 16, items = (tiles + RT - 1) / RT;
  const int KT = (A.K + 127) / 128, steps = (KT + F::kSlices - 1) / F::kSlices, pitch = matvec_token_pitch(KT);
  constexpr uint32_t kTokensAt = kZeroAt + kTokenRecord;
  const uint32_t zero = smem_u32(sm) + kZeroAt, tokens = smem_u32(sm) + kTokensAt;
  const int tile_floats = kFewWarps * A.T * kFewColPitch;
  const uint32_t sums_at = kTokensAt + A.T * pitch;
  FewRing way = few_sums_ring(sm, sums_at, RT * tile_floats * 4, 2);
  FewRing ring = few_ring(sm, sums_at + 2 * RT * tile_floats * 4, A.smem_bytes, (RT * F::kRowTile + 127) & ~127u);
  grid_launch_next();
  few_barriers(sm, tid, 1);
  if (tid < kTokenRecord / 4) reinterpret_cast<int*>(sm + kZeroAt)[tid] = 0;
  __syncthreads();
  grid_wait_previous();

  if (warp == kFewWarps) {
    int issued = 0;
    bool ok = true;
    for (int item = blockIdx.x; ok && item < items; item += gridDim.x) {
      const int nrt = min(RT, tiles - item * RT);
      for (int s = 0; s < steps; ++s) {
        ok = ring_wait(ring.empty_bar(), ring.phase ^ 1, &sh->abort_flag, A.status);
        if (!ok) break;
        const int kt0 = s * F::kSlices, nk = min(F::kSlices, KT - kt0);
        const uint32_t st = ring.stage(), bar = ring.full_bar();
        if (lane == 0) mbar_arrive_expect_tx(bar, nrt * nk * F::kTile);
        __syncwarp();
        if (lane < nrt)
          bulk_load_once(st + lane * F::kRowTile, A.W + ((size_t)(item * RT + lane) * KT + kt0) * F::kTile, nk * F::kTile, bar);
        ring.next();
        ++issued;
      }
    }
    drain(ring, issued, 0, lane);
    return;
  }

  constexpr int kBatch = 6;   // records of a warp whose loads are in flight together
  for (int i0 = warp > kFewWarps ? warp - 1 : warp; i0 < A.T * KT; i0 += kBatch * (kFewAllWarps - 1)) {
    uint2 x[kBatch];
#pragma unroll
    for (int b = 0; b < kBatch; ++b) {
      const int i = i0 + b * (kFewAllWarps - 1), t = i / KT, k = i % KT * 128 + 4 * lane;   // K is a multiple of 32
      x[b] = t < A.T && k < A.K ? __ldg(reinterpret_cast<const uint2*>(A.x + (size_t)t * A.K + k)) : make_uint2(0, 0);
    }
#pragma unroll
    for (int b = 0; b < kBatch; ++b) {
      const int i = i0 + b * (kFewAllWarps - 1), t = i / KT;
      if (t >= A.T) break;
      const float v[4] = {bf16_lo(x[b].x), bf16_hi(x[b].x), bf16_lo(x[b].y), bf16_hi(x[b].y)};
      put_record<GROUP>(v, sm + kTokensAt + t * pitch + i % KT * kTokenRecord, lane);
    }
  }
  consumer_sync_all(true);

  if (warp > kFewWarps) {
    const int fid = tid - 32 * (kFewWarps + 1);
    for (int item = blockIdx.x; item < items; item += gridDim.x, way.next()) {
      if (!ring_wait_idle(way.full_bar(), way.phase, &sh->abort_flag, A.status)) return;
      const int rows = 16 * min(RT, tiles - item * RT);
      const float* r = reinterpret_cast<const float*>(sm + way.stage());
      for (int i = fid; i < rows * A.T; i += kFewFinishThreads) {
        const int row = i % rows, t = i / rows, n = item * RT * 16 + row;
        if (n < A.N) A.y[(size_t)t * A.N + n] = to_bf16(get_sum(r + (row >> 4) * tile_floats, A.T, row & 15, t) * F::kSumScale);
      }
      __syncwarp();
      if (lane == 0) mbar_arrive(way.empty_bar());
    }
    return;
  }

  const LaneTokens<1> lt((1u << A.T) - 1, pitch, lane);
  for (int item = blockIdx.x; item < items; item += gridDim.x, way.next()) {
    float acc[RT][1][4] = {};
    for (int s = 0; s < steps; ++s, ring.next()) {
      if (!ring_wait(ring.full_bar(), ring.phase, &sh->abort_flag, A.status)) return;
#pragma unroll
      for (int i = warp; i < F::kSlices; i += kFewWarps) {
        const int kt = s * F::kSlices + i;
        if (kt < KT) few_slice<GROUP, 2, RT, 1>(ring.stage(), 0, tokens + kt * kTokenRecord, zero, lt, i, lane, acc);
      }
      __syncwarp();
      if (lane == 0) mbar_arrive(ring.empty_bar());
    }
    if (!ring_wait(way.empty_bar(), way.phase ^ 1, &sh->abort_flag, A.status)) return;
    put_sums<RT, 1>(reinterpret_cast<float*>(sm + way.stage()), A.T, A.T, warp, lane, acc);
    __syncwarp();
    if (lane == 0) mbar_arrive(way.full_bar());
  }
}

// ---------------------------------------------------------------- more tokens

constexpr int kWideThreads = (kFewWarps + 1) * 32;

MOE_DEV bool wide_sync_all(bool ok) {
  uint32_t all;
  asm volatile(
      "{\n\t.reg .pred p, q;\n\t"
      "setp.ne.b32 p, %1, 0;\n\t"
      "bar.red.and.pred q, 3, 256, p;\n\t"
      "selp.u32 %0, 1, 0, q;\n\t}"
      : "=r"(all) : "r"((uint32_t)ok) : "memory");
  return all != 0;
}

// Two row tiles' 64 columns [64 half, 64 half + 64) of a slice times NT blocks of 8 tokens.
// tok: these columns of token lane / 4, 128 bytes in TMA's swizzle, and `token_pitch` to the next.
template <int GROUP, int NT>
MOE_DEV void wide_half(uint32_t w, uint32_t row_tile, uint32_t tok, uint32_t token_pitch, int half, int lane, float (&acc)[2][NT][4]) {
  constexpr int kGroups = GROUP == 32 ? 2 : 1, kMmas = 4 / kGroups;   // groups that these columns touch
  uint32_t a[2][4][4];
  float s[2][kGroups][2];
#pragma unroll
  for (int rt = 0; rt < 2; ++rt) {
    const uint32_t p = w + rt * row_tile + lane * 16 + 8 * half;
    uint32_t c[2][2];   // row g's words, row g + 8's
    asm volatile("ld.shared.v2.u32 {%0,%1}, [%2];" : "=r"(c[0][0]), "=r"(c[0][1]) : "r"(p));
    asm volatile("ld.shared.v2.u32 {%0,%1}, [%2];" : "=r"(c[1][0]), "=r"(c[1][1]) : "r"(p + 512));
#pragma unroll
    for (int m = 0; m < 4; ++m)
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        uint32_t v;
        asm("lop3.b32 %0, %1, %2, %3, 0xEA;" : "=r"(v) : "r"(c[i & 1][m >> 1] >> (4 * (2 * (m & 1) + (i >> 1)))), "n"(0x000F000F), "n"(0x43004300));
        asm("sub.rn.bf16x2 %0, %1, %2;" : "=r"(a[rt][m][i]) : "r"(v), "r"(0x43084308));
      }
#pragma unroll
    for (int q = 0; q < kGroups; ++q) {
      const uint32_t sc = w + rt * row_tile + kW4Codes + 32 * (64 * half / GROUP + q) + 2 * (lane >> 2);
      s[rt][q][0] = lds_bf16(sc);
      s[rt][q][1] = lds_bf16(sc + 16);
    }
  }
#pragma unroll
  for (int j = 0; j < NT; ++j) {   // without a branch, so that the blocks' loads and MMAs overlap
    const uint32_t chunk = (lane & 3) ^ ((tok >> 7) & 7), at = tok + 8 * token_pitch * j;
    const uint4 u = lds128(at + 16 * chunk), v = lds128(at + 16 * (chunk ^ 4));
    const uint32_t b[8] = {u.x, u.y, u.z, u.w, v.x, v.y, v.z, v.w};
#pragma unroll
    for (int q = 0; q < kGroups; ++q) {
      float part[2][4] = {};
#pragma unroll
      for (int m = q * kMmas; m < (q + 1) * kMmas; ++m)
#pragma unroll
        for (int rt = 0; rt < 2; ++rt) mma_bf16(part[rt], a[rt][m], b[2 * m], b[2 * m + 1]);
#pragma unroll
      for (int rt = 0; rt < 2; ++rt)
#pragma unroll
        for (int i = 0; i < 4; ++i) acc[rt][j][i] = fmaf(part[rt][i], s[rt][q][i >> 1], acc[rt][j][i]);
    }
  }
}

// The tokens of a stage as one box [token][64 columns]; otherwise [64 columns][token], a box
// each, where 64 does not divide K (the first would reach into the next token) or the boxes are
// few (8 tokens x 4096 x 7168, eight slices: 7.0 us as one, 7.8 as 16; x 7168 x 2048, two
// slices: 5.1 as one, 5.0 as four: two tokens then share banks).
__host__ __device__ __forceinline__ bool wide_whole(int K, int slices) { return K % 64 == 0 && slices >= 4; }

template <int GROUP, int NT>
__global__ void __launch_bounds__(kWideThreads, 1) matvec_wide_kernel(const __grid_constant__ MatvecArgs A) {
  extern __shared__ __align__(1024) unsigned char sm[];
  constexpr int kTile = w4_tile_bytes(GROUP);
  FewShared* sh = reinterpret_cast<FewShared*>(sm);
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int KS = A.slices, RT = 2 * (kFewWarps / KS);   // slices and row tiles of a stage: 16 tiles of weights
  const int tiles = (A.N + 15) / 16, items = (tiles + RT - 1) / RT, KT = (A.K + 127) / 128, steps = (KT + KS - 1) / KS;
  constexpr uint32_t kRedAt = 256, kBox = NT * 8 * 128;   // a box of tokens: 64 columns of NT * 8, those past T zeros
  const uint32_t row_tile = KS * kTile, tok = (RT * row_tile + 1023) & ~1023u;
  const bool whole = wide_whole(A.K, KS);
  const uint32_t token_pitch = whole ? 2 * KS * 128 : 128, half_pitch = whole ? 128 : kBox;
  float4* red = reinterpret_cast<float4*>(sm + kRedAt);   // [warp][row tile][lane]
  FewRing ring = few_ring(sm, kRedAt + kFewWarps * 2 * 512, A.smem_bytes, tok + 2 * KS * kBox);
  grid_launch_next();
  few_barriers(sm, tid, 1);
  __syncthreads();
  grid_wait_previous();

  if (warp == kFewWarps) {
    int issued = 0;
    bool ok = true;
    for (int item = blockIdx.x; ok && item < items; item += gridDim.x) {
      for (int s = 0; s < steps; ++s) {
        ok = ring_wait(ring.empty_bar(), ring.phase ^ 1, &sh->abort_flag, A.status);
        if (!ok) break;
        // boxes that reach past the matrix or the tokens are filled with zeros, and count as bytes
        if (lane == 0) mbar_arrive_expect_tx(ring.full_bar(), 16 * kTile + 2 * KS * kBox);
        __syncwarp();
        if (lane == 0) tma_load_3d_once(ring.stage(), &A.map_w, 0, s * KS, item * RT, ring.full_bar());
        if (whole) {
          if (lane == 0) tma_load_3d(ring.stage() + tok, &A.map_x, 0, 2 * s * KS, 0, ring.full_bar());
        } else if (lane < 2 * KS) tma_load_2d(ring.stage() + tok + lane * kBox, &A.map_x, (2 * s * KS + lane) * 64, 0, ring.full_bar());
        ring.next();
        ++issued;
      }
    }
    drain(ring, issued, 0, lane);
    return;
  }

  const int slice = warp % KS, group = warp / KS;
  bool ok = true;
  for (int item = blockIdx.x; item < items; item += gridDim.x) {
    const int nrt = tiles - item * RT;
    float acc[2][NT][4] = {};
    for (int s = 0; s < steps; ++s, ring.next()) {
      ok = ring_wait(ring.full_bar(), ring.phase, &sh->abort_flag, A.status);
      if (!ok) break;
      if (s * KS + slice < KT && 2 * group < nrt) {
        const uint32_t w = ring.stage() + 2 * group * row_tile + slice * kTile;
        const uint32_t t = ring.stage() + tok + 2 * slice * half_pitch + (lane >> 2) * token_pitch;
        wide_half<GROUP, NT>(w, row_tile, t, token_pitch, 0, lane, acc);
        wide_half<GROUP, NT>(w, row_tile, t + half_pitch, token_pitch, 1, lane, acc);
      }
      __syncwarp();
      if (lane == 0) mbar_arrive(ring.empty_bar());
    }
    if (!wide_sync_all(ok)) return;
#pragma unroll
    for (int j = 0; j < NT; ++j) {
      if (8 * j < A.T) {
        if (KS > 1) {
          if (slice > 0) {
#pragma unroll
            for (int rt = 0; rt < 2; ++rt)
              red[(warp * 2 + rt) * 32 + lane] = make_float4(acc[rt][j][0], acc[rt][j][1], acc[rt][j][2], acc[rt][j][3]);
          }
          wide_sync_all(true);
        }
        if (slice == 0) {
#pragma unroll
          for (int rt = 0; rt < 2; ++rt) {
            float v[4] = {acc[rt][j][0], acc[rt][j][1], acc[rt][j][2], acc[rt][j][3]};
            for (int i = 1; i < KS; ++i) {   // the slices in their order
              const float4 o = red[((warp + i) * 2 + rt) * 32 + lane];
              v[0] += o.x; v[1] += o.y; v[2] += o.z; v[3] += o.w;
            }
#pragma unroll
            for (int i = 0; i < 4; ++i) {
              const int t = 8 * j + 2 * (lane & 3) + (i & 1), n = (item * RT + 2 * group + rt) * 16 + (lane >> 2) + 8 * (i >> 1);
              if (t < A.T && n < A.N) A.y[(size_t)t * A.N + n] = to_bf16(v[i]);
            }
          }
        }
        if (KS > 1) wide_sync_all(true);   // the meeting place is free again
      }
    }
  }
}

// Slices of the wide kernel's stages: the fewest stages over the rounds that the SMs make,
// each as long as its copies (some 40 bytes a clock, with the tokens out of L2) or
// its MMAs (16 clocks per tile and block of tokens, and 600 beside them).
inline int wide_slices(int tiles, int KT, int nt, int nsm) {
  int best = 1;
  long long cost = 1LL << 60;
  for (int ks = 1; ks <= 8; ks *= 2) {
    const int rows = 2 * (8 / ks), rounds = ((tiles + rows - 1) / rows + nsm - 1) / nsm;
    const long long stage = std::max((16 * 1100 + 2 * ks * nt * 1024) / 40, 16 * nt * 16 + 600);
    const long long c = (long long)rounds * ((KT + ks - 1) / ks) * stage;
    if (c < cost) { cost = c; best = ks; }
  }
  return best;
}

template <int GROUP, int RT>
int launch_matvec_few(const MatvecArgs& a, int nsm, cudaStream_t s) {
  const int items = ((a.N + 15) / 16 + RT - 1) / RT;
  return few_launch(matvec_few_kernel<GROUP, RT>, a, kFewThreads, std::min(items, nsm), false, s);
}
template <int GROUP>
int launch_matvec(const MatvecArgs& args, int nsm, cudaStream_t s) {
  const int tiles = (args.N + 15) / 16;
  const int KT = (args.K + 127) / 128, records = args.T * matvec_token_pitch(KT);
  // The records cost a block some 20 ns each; the other kernels take the tokens as they are.
  // Groups of 128, few / other kernel: one token x 4096 x 7168 6.65 / 6.9 us, x 32768 x 7168
  // 26.4 / 29.2; two x 4096 x 4096 (64 records) 4.8 / 5.2, x 4096 x 7168 (112) 7.2 / 7.0, x 32768 x
  // 7168 27.4 / 29.2; three x 32768 x 7168 28.4 / 29.1; four x 2048 x 2048 (64) 2.95 / 3.65, x 4096 x
  // 7168 (224) 9.1 / 6.9, x 32768 x 4096 18.7 / 18.4; six x 2048 x 2048 (96) 3.7 / 3.7.
  if (records <= kMatvecTokenRoom && (args.T == 1 || (args.T <= 4 && (args.T * KT <= 64 || tiles > 4 * nsm)))) {
    switch (few_row_tiles(tiles, nsm, records <= kMatvecTokenRoom / 2 ? 3 : 2)) {
      case 1: return launch_matvec_few<GROUP, 1>(args, nsm, s);
      case 2: return launch_matvec_few<GROUP, 2>(args, nsm, s);
      default: return launch_matvec_few<GROUP, 3>(args, nsm, s);
    }
  }
  // Groups of 128, wide / tensor kernel: 16 tokens x 8192 x 4096 9.1 / 11.7 us, x 16384 x 4096
  // 14.5 / 13.3, x 32768 x 7168 48 / 29; 32 tokens x 1024 x 1024 5.7 / 4.5, x 4096 x 7168
  // 12.7 / 11.8, x 32768 x 7168 59 / 31.
  if (args.T > 16 || tiles > 4 * nsm) return launch_matvec_tensor<GROUP>(args, nsm, s);
  MatvecArgs a = args;
  const int nt = (a.T + 7) / 8;
  a.slices = wide_slices(tiles, KT, nt, nsm);
  const int rows = 2 * (8 / a.slices), blocks = std::min((tiles + rows - 1) / rows, nsm);
  constexpr int kTile = w4_tile_bytes(GROUP);
  const uint64_t wd[3] = {kTile / 8, (uint64_t)KT, (uint64_t)tiles}, ws[2] = {kTile, (uint64_t)KT * kTile};
  const uint32_t wb[3] = {kTile / 8, (uint32_t)a.slices, (uint32_t)rows};
  const bool whole = wide_whole(a.K, a.slices);
  const uint64_t xd[3] = {64, (uint64_t)a.K / 64, (uint64_t)a.T}, xs[2] = {128, (uint64_t)a.K * 2};
  const uint32_t xb[3] = {64, 2 * (uint32_t)a.slices, (uint32_t)nt * 8};
  const uint64_t xd2[2] = {(uint64_t)a.K, (uint64_t)a.T}, xs2[1] = {(uint64_t)a.K * 2};
  const uint32_t xb2[2] = {64, (uint32_t)nt * 8};
  if (!encode_few_map(&a.map_w, CU_TENSOR_MAP_DATA_TYPE_UINT64, CU_TENSOR_MAP_SWIZZLE_NONE, a.W, 3, wd, ws, wb) ||
      !encode_few_map(&a.map_x, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, CU_TENSOR_MAP_SWIZZLE_128B, a.x, whole ? 3 : 2, whole ? xd : xd2, whole ? xs : xs2,
                      whole ? xb : xb2))
    return MOE_ERR_CUDA;
  return nt == 1 ? few_launch(matvec_wide_kernel<GROUP, 1>, a, kWideThreads, blocks, false, s)
                 : few_launch(matvec_wide_kernel<GROUP, 2>, a, kWideThreads, blocks, false, s);
}

}  // namespace moe
