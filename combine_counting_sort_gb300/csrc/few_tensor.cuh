// few_tensor.cuh: products of 2 to 64 tokens with one 4-bit matrix on the fifth-generation
// tensor cores.
//
// y[t][n] = sum over groups q of scale[n][q] * sum over the group's k of (code[n][k] - 8) * x[t][k].
//
// A block takes 256 matrix rows, two times the MMA's 128, and all tokens, and walks K in
// slices of 128 columns.  Sixteen widening warps turn a slice's codes into bf16 and put them
// into tensor memory, where the MMA reads them as its A operand (a thread's TMEM lane is one row:
// 64 32-bit columns); the tokens are its B operand as TMA brings them.  Codes and tokens are
// exact in bf16, and a group's MMAs add up in fp32 in tensor memory; eight summing warps multiply
// the groups' sums by the rows' scales in fp32 and add them to their registers.  One warp copies, two
// issue the MMAs.  Nothing widened goes back to shared memory, and the roles wait for one another
// only through rings: the stages, two A buffers and two or four units of sums per 128 rows.
//
// With few rows a cluster of blocks shares them, each a run of the slices; their sums meet
// in shared memory and every block adds up its share of the tokens, the runs in their order.
//
// Measured, us for 32768 x 7168: groups of 128, 16 / 32 / 64 tokens 29.3 / 31.3 / 36.1 (48 / 59 /
// 95 with the weights as the A operand of mma.sync); groups of 64, 48 tokens 39.3 (75.5);
// groups of 32, 64 tokens 60 (111).  What bounds it: with groups of 128 the ALU, 112 ANDs,
// shifts and selections per 32 rows and slice at 16 lanes a clock, of which it is 64% busy, and
// 128 items for 152 SMs; with 152 items it reads 4.8 TB/s.  With smaller groups the summing
// warps, whose 256 additions per row and slice (groups of 32, 64 tokens) wait for each unit.
// What it took: one warp per 128 rows for the MMAs, with nothing but waits and MMAs in one
// elected thread (71 to 44 us at 48 tokens); the MMAs' addresses in uniform registers; sixteen
// widening warps and not eight (35 to 29 us at 16 tokens).  The columns of sums split over
// sixteen summing warps, and two additions per instruction, gained nothing.
#pragma once

#include "few.cuh"
#include "few_host.h"

namespace moe {

constexpr int kTensorRows = 256;   // of a block
constexpr int kTensorThreads = kTensorWarps * 32;
static_assert(tensor_split_fits(65536 / kTensorThreads / 8 * 8), "register split exceeds launch");

// 16 TMEM columns of this thread's lane; complete behind the next tmem_got of the same registers.
MOE_DEV void tmem_get(uint32_t taddr, float (&v)[16]) {
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x16.b32 {%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15}, [%16];"
      : "=f"(v[0]), "=f"(v[1]), "=f"(v[2]), "=f"(v[3]), "=f"(v[4]), "=f"(v[5]), "=f"(v[6]), "=f"(v[7]),
        "=f"(v[8]), "=f"(v[9]), "=f"(v[10]), "=f"(v[11]), "=f"(v[12]), "=f"(v[13]), "=f"(v[14]), "=f"(v[15])
      : "r"(taddr)
      : "memory");
}
MOE_DEV void tmem_got(float (&v)[16]) {
  asm volatile(
      "tcgen05.wait::ld.sync.aligned;"
      : "+f"(v[0]), "+f"(v[1]), "+f"(v[2]), "+f"(v[3]), "+f"(v[4]), "+f"(v[5]), "+f"(v[6]), "+f"(v[7]),
        "+f"(v[8]), "+f"(v[9]), "+f"(v[10]), "+f"(v[11]), "+f"(v[12]), "+f"(v[13]), "+f"(v[14]), "+f"(v[15])
      :: "memory");
}
// 16 columns into TMEM; complete at the next wait::st.
MOE_DEV void tmem_put(uint32_t taddr, const uint32_t (&v)[16]) {
  asm volatile(
      "tcgen05.st.sync.aligned.32x32b.x16.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15, %16};"
      :: "r"(taddr),
         "r"(v[0]), "r"(v[1]), "r"(v[2]), "r"(v[3]), "r"(v[4]), "r"(v[5]), "r"(v[6]), "r"(v[7]),
         "r"(v[8]), "r"(v[9]), "r"(v[10]), "r"(v[11]), "r"(v[12]), "r"(v[13]), "r"(v[14]), "r"(v[15])
      : "memory");
}

// D[tmem] (+)= A[tmem] * B[smem]^T, bf16 operands, fp32 sums.
MOE_DEV void umma_bf16_ta(uint32_t d_tmem, uint32_t a_tmem, uint64_t bdesc, uint32_t idesc, uint32_t accumulate) {
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "setp.ne.b32 p, %4, 0;\n\t"
      "tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p;\n\t}"
      :: "r"(d_tmem), "r"(a_tmem), "l"(bdesc), "r"(idesc), "r"(accumulate) : "memory");
}
// Instruction descriptor of kind::f16: fp32 D (bits 4-5 = 1), A and B bf16 (bits 7-9, 10-12
// = 1), both K-major, N >> 3 in bits 17-22, M >> 4 in bits 24-28.
__host__ __device__ constexpr uint32_t idesc_bf16_f32(int M, int N) {
  return (1u << 4) | (1u << 7) | (1u << 10) | ((uint32_t)(N >> 3) << 17) | ((uint32_t)(M >> 4) << 24);
}

// A 32-bit register's pair of codes as bf16 (c - 8) / 64.  The bits c and 16 c read as bf16 are
// c * 2^-133 and c * 2^-129 (bf16 is linear from its subnormals to the end of the first
// binade), so one AND and one multiply-add widen two codes, both exactly.
MOE_DEV uint32_t widen_low(uint32_t word) {
  uint32_t v;
  asm("fma.rn.bf16x2 %0, %1, %2, %3;" : "=r"(v) : "r"(word & 0x000F000Fu), "r"(0x7F007F00u), "r"(0xBE00BE00u));
  return v;
}
MOE_DEV uint32_t widen_high(uint32_t word) {
  uint32_t v;
  asm("fma.rn.bf16x2 %0, %1, %2, %3;" : "=r"(v) : "r"(word & 0x00F000F0u), "r"(0x7D007D00u), "r"(0xBE00BE00u));
  return v;
}
constexpr float kTensorSumScale = 64.f;   // what the sums lack

struct TensorShared {   // behind FewShared
  uint64_t a_full[4], a_empty[4];   // [buffer][block of rows]
  uint64_t d_full[8], d_empty[8];   // units of sums
  uint64_t done[2];
  uint32_t tmem;
};
static_assert(sizeof(TensorShared) <= 256, "");

template <int GROUP, int NT>
__global__ void __launch_bounds__(kTensorThreads, 1) matvec_tensor_kernel(const __grid_constant__ MatvecArgs A) {
  extern __shared__ __align__(1024) unsigned char sm[];
  constexpr int kTile = w4_tile_bytes(GROUP), kGroups = FewGroups<GROUP>::kCount;
  constexpr int kN = 8 * NT, kPer = kN > 32 ? 1 : kGroups < 64 / kN ? kGroups : 64 / kN;   // groups per unit of sums
  constexpr int kUnits = kPer * kN <= 32 ? 4 : 2;                                          // units per block of rows
  constexpr uint32_t kBox = kN * 128;   // 64 columns of all tokens, those past T zeros
  constexpr uint32_t kTok = tensor_tokens_at(GROUP), kStage = tensor_stage(GROUP, kN);
  static_assert(tensor_stages(GROUP, kN, kFewMinSmem) >= kTensorMinStages, "the widening warps' waits");
  constexpr uint32_t kAcols = 64, kSums = 4 * kAcols;   // columns of an A buffer; where the sums' units begin,
  constexpr uint32_t kPitch = (512 - kSums) / (2 * kUnits);   // and from one to the next
  static_assert(kPitch >= kPer * kN, "");
  FewShared* sh = reinterpret_cast<FewShared*>(sm);
  TensorShared* ts = reinterpret_cast<TensorShared*>(sm + 256);
  const int tid = threadIdx.x, warp = __shfl_sync(0xffffffffu, tid >> 5, 0), lane = tid & 31;   // uniform: the MMAs' operands are
  const int C = A.slices, rank = C > 1 ? (int)cluster_ctarank() : 0;   // blocks that share 256 rows
  const int tiles = (A.N + 15) / 16, items = (tiles + 15) / 16, KT = (A.K + 127) / 128;
  const int kt_begin = KT * rank / C, steps = KT * (rank + 1) / C - kt_begin;
  const int first = blockIdx.x / C, stride = gridDim.x / C;
  const int mine = (items - 1 - first) / stride * steps + steps;   // slices of this block's items
  FewRing ring = few_ring(sm, 512, A.smem_bytes, kStage);
  grid_launch_next();
  few_barriers(sm, tid, 1, 8);   // the summing warps free a stage
  if (tid >= 32 && tid < 40) {
    const int i = tid - 32;
    if (i < 4) {
      mbar_init(smem_u32(ts->a_full + i), 4);
      mbar_init(smem_u32(ts->a_empty + i), 1);
    }
    mbar_init(smem_u32(ts->d_full + i), 1);
    mbar_init(smem_u32(ts->d_empty + i), 4);
    if (i < 2) mbar_init(smem_u32(ts->done + i), 1);
    fence_mbar_init();
  }
  if (warp == kTensorMma) {
    tmem_alloc(smem_u32(&ts->tmem), 512);
    tmem_relinquish();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = ts->tmem;
  grid_wait_previous();

  auto wait = [&](uint32_t bar, uint32_t parity) { return ring_wait(bar, parity, &sh->abort_flag, A.status); };
  auto arrive = [&](uint32_t bar) {
    __syncwarp();
    if (lane == 0) mbar_arrive(bar);
  };
  const int block = (warp >> 2) & 1, quad = warp & 3;   // of the widening and the summing warps
  const uint32_t tile = (8 * block + 2 * quad + (lane >> 4)) * kTile;   // of this thread's row
  // The block's meeting at the end of every role (no tensor operation or copy is in flight behind it).
  auto meet = [] {
    tc_fence_before();
    asm volatile("bar.sync 1, %0;" :: "n"(kTensorThreads) : "memory");
    tc_fence_after();
  };

  if (warp >= kTensorCopy) regs_dealloc<kTensorRestRegs>();
  if (warp == kTensorCopy) {
    int issued = 0;
    bool ok = true;
    for (int item = first; ok && item < items; item += stride) {
      for (int s = 0; s < steps; ++s) {
        if (!(ok = wait(ring.empty_bar(), ring.phase ^ 1))) break;
        // boxes that reach past the matrix or the tokens are filled with zeros, and count as bytes
        if (lane == 0) {
          mbar_arrive_expect_tx(ring.full_bar(), 16 * kTile + 2 * kBox);
          tma_load_3d_once(ring.stage(), &A.map_w, 0, kt_begin + s, item * 16, ring.full_bar());
          tma_load_2d(ring.stage() + kTok, &A.map_x, (kt_begin + s) * 128, 0, ring.full_bar());
          tma_load_2d(ring.stage() + kTok + kBox, &A.map_x, (kt_begin + s) * 128 + 64, 0, ring.full_bar());
        }
        __syncwarp();
        ring.next();
        ++issued;
      }
    }
    drain(ring, issued, 0, lane);
    meet();
  } else if (warp > kTensorCopy) {   // one warp per 128 rows, all of it by one thread: the waits are its time
    constexpr uint32_t kIdesc = idesc_bf16_f32(128, kN);
    if (warp < kTensorMma + 2 && elect_one()) {
      const int b = warp - kTensorMma;
      const uint32_t a_full = smem_u32(ts->a_full + b), a_empty = smem_u32(ts->a_empty + b);
      const uint32_t d_full = smem_u32(ts->d_full + b * kUnits), d_empty = smem_u32(ts->d_empty + b * kUnits);
      const uint32_t sums = tmem + kSums + b * kUnits * kPitch, codes = tmem + b * kAcols;
      auto wait1 = [&](uint32_t bar, uint32_t parity) { return mbar_wait(bar, parity, &sh->abort_flag, A.status, kFewTimeoutNs); };
      bool ok = true;
      int unit = 0, unit_phase = 1, slot = 0;
      uint64_t tok = sw128_kmajor_desc(ring.base + kTok);
      for (int n = 0; ok && n < mine; ++n) {
        const int buf = n & 1;
        if (!wait1(a_full + 16 * buf, (n >> 1) & 1)) break;   // the stage is full: the codes came out of it
#pragma unroll
        for (int q = 0; q < kGroups; q += kPer) {
          ok = wait1(d_empty + 8 * unit, unit_phase);
          if (!ok) break;
          tc_fence_after();
#pragma unroll
          for (int k = q * (GROUP / 16); k < (q + kPer) * (GROUP / 16); ++k)
            umma_bf16_ta(sums + unit * kPitch + (k * 16 / GROUP - q) * kN, codes + buf * 2 * kAcols + 8 * k,
                         tok + (((k >> 2) * kBox + (k & 3) * 32) >> 4), kIdesc, k % (GROUP / 16) > 0);
          umma_commit(d_full + 8 * unit);
          if (q + kPer == kGroups) umma_commit(a_empty + 16 * buf);
          if (++unit == kUnits) { unit = 0; unit_phase ^= 1; }
        }
        tok += kStage >> 4;
        if (++slot == ring.stages) { slot = 0; tok = sw128_kmajor_desc(ring.base + kTok); }
      }
      // no MMA may be in flight when tensor memory is freed
      umma_commit(smem_u32(ts->done + b));
      int none = 0;
      mbar_wait(smem_u32(ts->done + b), 0, &none, A.status, kFewTimeoutNs);
    }
    __syncwarp();
    meet();
    if (warp == kTensorMma) tmem_dealloc(tmem, 512);
  } else if (warp < kTensorSum) {
    regs_dealloc<kTensorWidenRegs>();
    const uint32_t at = tile + (lane & 15) * 64;
    const int rot = (lane >> 1) & 3;   // the row's four 16-byte chunks in an order without bank conflicts
    uint32_t w[4][4];                  // [chunk t][word j]: columns 32 j + 8 t ..
    const int odd_slices = warp >> 3;  // each warp every second slice, for one of the A buffers
    const uint32_t a = tmem + ((uint32_t)(32 * quad) << 16) + (odd_slices * 2 + block) * kAcols;
    const uint32_t full = smem_u32(ts->a_full + odd_slices * 2 + block), empty = smem_u32(ts->a_empty + odd_slices * 2 + block);
    if (odd_slices) ring.next();   // kTensorMinStages: why its waits are safe with an odd number of stages
    for (int n = odd_slices; n < mine; n += 2) {
      if (!wait(ring.full_bar(), ring.phase)) break;
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const uint4 v = lds128(ring.stage() + at + 16 * ((i + rot) & 3));
        w[i][0] = v.x; w[i][1] = v.y; w[i][2] = v.z; w[i][3] = v.w;
      }
#pragma unroll
      for (int j = 0; j < 4; ++j) {   // the chunks in their places
        const uint32_t a0 = w[0][j], a1 = w[1][j], a2 = w[2][j], a3 = w[3][j];
        const bool odd = rot & 1, two = rot & 2;
        const uint32_t b0 = odd ? a3 : a0, b1 = odd ? a0 : a1, b2 = odd ? a1 : a2, b3 = odd ? a2 : a3;
        w[0][j] = two ? b2 : b0;
        w[1][j] = two ? b3 : b1;
        w[2][j] = two ? b0 : b2;
        w[3][j] = two ? b1 : b3;
      }
      if (!wait(empty, ((n >> 1) & 1) ^ 1)) break;
      tc_fence_after();
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        uint32_t v[16];
#pragma unroll
        for (int t = 0; t < 4; ++t) {
          const uint32_t lo = w[t][j], hi = lo >> 8;
          v[4 * t] = widen_low(lo);
          v[4 * t + 1] = widen_high(lo);
          v[4 * t + 2] = widen_low(hi);
          v[4 * t + 3] = widen_high(hi);
        }
        tmem_put(a + 16 * j, v);
      }
      asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory");
      tc_fence_before();
      arrive(full);
      ring.next();
      ring.next();
    }
    meet();
  } else {
    regs_alloc<kTensorSumRegs>();
    float acc[kN];
    const uint32_t d_full = smem_u32(ts->d_full + block * kUnits), d_empty = smem_u32(ts->d_empty + block * kUnits);
    const uint32_t sums = tmem + ((uint32_t)(32 * quad) << 16) + kSums + block * kUnits * kPitch;
    bool ok = true;
    int unit = 0, unit_phase = 0;
    for (int item = first; ok && item < items; item += stride) {
#pragma unroll
      for (int c = 0; c < kN; ++c) acc[c] = 0.f;
      for (int s = 0; s < steps; ++s, ring.next()) {
        if (!(ok = wait(ring.full_bar(), ring.phase))) break;
        float scale[kGroups];
#pragma unroll
        for (int q = 0; q < kGroups; ++q) scale[q] = lds_bf16(ring.stage() + tile + kW4Codes + 32 * q + 2 * (lane & 15));
#pragma unroll
        for (int q = 0; q < kGroups; q += kPer) {
          if (!(ok = wait(d_full + 8 * unit, unit_phase))) break;
          if (q + kPer == kGroups) arrive(ring.empty_bar());   // the MMAs have read the tokens, and before that the codes were
          tc_fence_after();
          const uint32_t d = sums + unit * kPitch;
          float v[2][16];   // a read is on its way while the one before is added
          tmem_get(d, v[0]);
#pragma unroll
          for (int c = 0; c < kPer * kN; c += 16) {
            float (&now)[16] = v[c / 16 & 1];
            tmem_got(now);
            if (c + 16 < kPer * kN) {
              tmem_get(d + c + 16, v[(c / 16 + 1) & 1]);
            } else {
              tc_fence_before();
              arrive(d_empty + 8 * unit);
            }
#pragma unroll
            for (int i = 0; i < 16; ++i) acc[c % kN + i] = fmaf(now[i], scale[q + c / kN], acc[c % kN + i]);
          }
          if (++unit == kUnits) { unit = 0; unit_phase ^= 1; }
        }
        if (!ok) break;
      }
      const int row = item * kTensorRows + 128 * block + 32 * quad + lane;
      if (ok && C == 1 && row < A.N) {
#pragma unroll
        for (int t = 0; t < kN; ++t)
          if (t < A.T) A.y[(size_t)t * A.N + row] = to_bf16(acc[t] * kTensorSumScale);
      }
    }
    meet();
    if (C > 1) {   // the ring is done with and holds the sums, [token][row]
#pragma unroll
      for (int t = 0; t < kN; ++t)
        asm volatile("st.shared.f32 [%0], %1;" :: "r"(ring.base + 4 * (t * kTensorRows + 128 * block + 32 * quad + lane)), "f"(acc[t]) : "memory");
    }
  }

  if (C > 1) {   // one item per cluster
    __syncwarp();
    cluster_sync();
    const int row = first * kTensorRows + (tid & 255);
    if (tid < 512 && row < A.N && !sh->abort_flag) {
      for (int t = rank + C * (tid >> 8); t < A.T; t += 2 * C) {
        float sum = 0.f;
        for (int r = 0; r < C; ++r) {
          float v;
          asm volatile("ld.shared::cluster.f32 %0, [%1];" : "=f"(v) : "r"(mapa_shared(ring.base + 4 * (t * kTensorRows + (tid & 255)), r)) : "memory");
          sum += v;
        }
        A.y[(size_t)t * A.N + row] = to_bf16(sum * kTensorSumScale);
      }
    }
    __syncwarp();
    cluster_sync();   // no block leaves while another reads its sums
  }
}

// Blocks that share 256 rows: the largest cluster of which the SMs take one for every item at
// once.  On 152 SMs 15 of eight, 36 of four and 76 of two ran at once; 16 of eight took 16.9 us
// for 4096 x 7168 and 32 tokens where 16 of four take 11.7, 38 of four 18.4 us for 9728 x 4096
// where 38 of two take 13.5.
inline int tensor_cluster(int items, int KT, int nsm) {
  int c = items * 10 <= nsm ? 8 : items * 4 + 8 <= nsm ? 4 : items * 2 <= nsm ? 2 : 1;
  while (c > KT) c /= 2;
  return c;
}

template <int GROUP, int NT>
int launch_tensor_nt(const MatvecArgs& a, int blocks, cudaStream_t s) {
  static const bool split_ok = [] {
    cudaFuncAttributes f;
    return cudaFuncGetAttributes(&f, matvec_tensor_kernel<GROUP, NT>) == cudaSuccess && tensor_split_fits(f.numRegs);
  }();
  if (!split_ok) return MOE_ERR_UNSUPPORTED;
  return few_launch(matvec_tensor_kernel<GROUP, NT>, a, kTensorThreads, blocks, false, s, a.slices);
}

template <int GROUP>
int launch_matvec_tensor(const MatvecArgs& args, int nsm, cudaStream_t s) {
  MatvecArgs a = args;
  const int tiles = (a.N + 15) / 16, items = (tiles + 15) / 16, KT = (a.K + 127) / 128, nt = (a.T + 15) / 16 * 2;
  a.slices = tensor_cluster(items, KT, nsm);
  const int blocks = a.slices > 1 ? items * a.slices : std::min(items, nsm);
  constexpr int kTile = w4_tile_bytes(GROUP);
  const uint64_t wd[3] = {kTile / 8, (uint64_t)KT, (uint64_t)tiles}, ws[2] = {kTile, (uint64_t)KT * kTile};
  const uint32_t wb[3] = {kTile / 8, 1, 16};
  const uint64_t xd[2] = {(uint64_t)a.K, (uint64_t)a.T}, xs[1] = {(uint64_t)a.K * 2};
  const uint32_t xb[2] = {64, (uint32_t)nt * 8};
  if (!encode_few_map(&a.map_w, CU_TENSOR_MAP_DATA_TYPE_UINT64, CU_TENSOR_MAP_SWIZZLE_NONE, a.W, 3, wd, ws, wb) ||
      !encode_few_map(&a.map_x, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, CU_TENSOR_MAP_SWIZZLE_128B, a.x, 2, xd, xs, xb))
    return MOE_ERR_CUDA;
  switch (nt) {
    case 2: return launch_tensor_nt<GROUP, 2>(a, blocks, s);
    case 4: return launch_tensor_nt<GROUP, 4>(a, blocks, s);
    case 6: return launch_tensor_nt<GROUP, 6>(a, blocks, s);
    default: return launch_tensor_nt<GROUP, 8>(a, blocks, s);
  }
}

}  // namespace moe
