// few.cuh: the streaming engine of the decoding kernels (few tokens, all of the
// time goes into reading weights once).
//
// A CTA is eight computing warps and one copying warp.  The copying warp walks
// the CTA's work and keeps a ring of shared-memory stages full with bulk copies
// (cp.async.bulk, counted on an mbarrier per stage): per stage RT row tiles of
// 16 weight rows x 1024 columns, and the same 1024 columns of the tokens that
// the weights multiply.  Each computing warp takes one 128-column slice of a
// stage: it reads its codes as the A operand of mma.sync.m16n8k16 (16 weight
// rows), widens them to bf16 in registers (exactly: 4-bit integers and e4m3
// values are bf16 values) and multiplies them with up to 8 tokens per MMA.
// Group scales are applied to the fp32 sum of a group.  The eight partial sums
// of a row meet in shared memory once a row tile is complete, in a fixed order.
//
// mma.sync and not tcgen05: the tensor work is the weights times 8 columns,
// far below either's rate, and the operands must pass through registers to be
// widened anyway; what bounds these kernels is memory, then the instructions
// that widen the codes.
#pragma once

#include "common.cuh"
#include "w4.cuh"

namespace moe {

constexpr int kFewWarps = 8;                       // computing warps
constexpr int kFewThreads = (kFewWarps + 1) * 32;  // and the copying warp
constexpr int kFewStageCols = kFewWarps * 128;     // weight columns per stage
constexpr int kFewMaxCols = 16;                    // tokens per pass over a stage
constexpr int kFewMaxStages = 12;
constexpr uint64_t kFewTimeoutNs = 1000000000ull;  // bound of every wait

// Untiled bulk copy global -> shared (16-byte aligned, size a multiple of 16).
MOE_DEV void bulk_load(uint32_t dst, const void* src, uint32_t bytes, uint32_t bar) {
  asm volatile("cp.async.bulk.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1], %2, [%3];"
               :: "r"(dst), "l"(reinterpret_cast<uint64_t>(src)), "r"(bytes), "r"(bar) : "memory");
}
// This thread's earlier cp.async copies arrive on `bar` when they are complete.
MOE_DEV void cp_async_arrive(uint32_t bar) {
  asm volatile("cp.async.mbarrier.arrive.noinc.shared::cta.b64 [%0];" :: "r"(bar) : "memory");
}

MOE_DEV void mma_bf16(float (&d)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
  asm("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
      : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
      : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}

MOE_DEV uint4 lds128(uint32_t a) {
  uint4 v;
  asm volatile("ld.shared.v4.u32 {%0,%1,%2,%3}, [%4];" : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w) : "r"(a));
  return v;
}
MOE_DEV float lds_f32(uint32_t a) {
  float v;
  asm volatile("ld.shared.f32 %0, [%1];" : "=f"(v) : "r"(a));
  return v;
}
MOE_DEV float lds_bf16(uint32_t a) {
  uint16_t v;
  asm volatile("ld.shared.u16 %0, [%1];" : "=h"(v) : "r"(a));
  return bf16_lo(v);
}

// ---------------------------------------------------------------- weight forms

// Geometry of a stage for GROUP (0: FP8 rows with 128 x 128 scales; else 4-bit tiles).
template <int GROUP>
struct FewForm {
  static constexpr bool kW4 = GROUP != 0;
  static constexpr int kTile = w4_tile_bytes(kW4 ? GROUP : 128);
  // FP8 rows are copied one by one with a pitch that is 64 mod 128 bytes, so the
  // 8 rows x 64 bytes of a quarter-warp's 16-byte reads fall on distinct banks.
  static constexpr int kRowPitch = kFewStageCols + 64;
  static constexpr int kRowTile = kW4 ? kFewWarps * kTile : 16 * kRowPitch;   // bytes of a row tile in a stage
  // Tokens: bf16 rows; the quarter-warp's reads are 16 bytes apart (4-bit: pitch
  // 64 mod 128) or 32 bytes apart (FP8: pitch 16 mod 128 fills the gaps).
  static constexpr int kTokPitch = 2 * kFewStageCols + (kW4 ? 64 : 16);
  static constexpr int kScaleBytes = kW4 ? 0 : 4 * kFewWarps;                 // per row tile
  // arrivals that complete a stage: weights, tokens, and the lanes' scale copies
  static constexpr int kArrivals = kW4 ? 2 : 34;
};

// One MMA's A operand: columns m of the lane's 8 MMA slots from the code words of
// rows g (lo) and g + 8 (hi).
template <int GROUP>
MOE_DEV void widen(const uint32_t* lo, const uint32_t* hi, int m, uint32_t (&a)[4]) {
  if (GROUP != 0) {
    // nibble pairs as 128 + code in bf16 (0x4300 | code), minus 136
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const uint32_t w = (i & 1 ? hi : lo)[m >> 1] >> (4 * (2 * (m & 1) + (i >> 1)));
      uint32_t v;
      asm("lop3.b32 %0, %1, %2, %3, 0xEA;" : "=r"(v) : "r"(w), "n"(0x000F000F), "n"(0x43004300));
      asm("sub.rn.bf16x2 %0, %1, %2;" : "=r"(a[i]) : "r"(v), "r"(0x43084308));
    }
  } else {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const uint32_t w = (i & 1 ? hi : lo)[m];
      const float2 f = e4m3x2_to_float2((uint16_t)(i >> 1 ? w >> 16 : w & 0xFFFFu));
      a[i] = pack_bf16x2(f.x, f.y);
    }
  }
}

// The lane's code words of a row tile's slice: 4 (4-bit) or 8 (FP8) words per row.
template <int GROUP>
MOE_DEV void load_codes(uint32_t wst, int warp, int lane, uint32_t (&lo)[8], uint32_t (&hi)[8]) {
  using F = FewForm<GROUP>;
  if (F::kW4) {
    const uint32_t a = wst + warp * F::kTile + lane * 16;
    const uint4 l = lds128(a), h = lds128(a + 512);
    lo[0] = l.x; lo[1] = l.y; lo[2] = l.z; lo[3] = l.w;
    hi[0] = h.x; hi[1] = h.y; hi[2] = h.z; hi[3] = h.w;
  } else {
    const uint32_t a = wst + (lane >> 2) * F::kRowPitch + warp * 128 + (lane & 3) * 16;
#pragma unroll
    for (int j = 0; j < 2; ++j) {
      const uint4 l = lds128(a + 64 * j), h = lds128(a + 8 * F::kRowPitch + 64 * j);
      lo[4 * j] = l.x; lo[4 * j + 1] = l.y; lo[4 * j + 2] = l.z; lo[4 * j + 3] = l.w;
      hi[4 * j] = h.x; hi[4 * j + 1] = h.y; hi[4 * j + 2] = h.z; hi[4 * j + 3] = h.w;
    }
  }
}

// The B operands of the lane's 8 MMAs: its columns of one token's slice.
template <int GROUP>
MOE_DEV void load_token(uint32_t row, int warp, int lane, uint32_t (&b)[16]) {
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    const uint32_t a = row + warp * 256 + (FewForm<GROUP>::kW4 ? (4 * j + (lane & 3)) * 16 : (4 * (j >> 1) + (lane & 3)) * 32 + 16 * (j & 1));
    const uint4 v = lds128(a);
    b[4 * j] = v.x; b[4 * j + 1] = v.y; b[4 * j + 2] = v.z; b[4 * j + 3] = v.w;
  }
}

// Scales of group q of a row tile's slice for rows g and g + 8.
template <int GROUP>
MOE_DEV float2 load_scales(uint32_t wst, uint32_t sst, int rt, int warp, int lane, int q) {
  using F = FewForm<GROUP>;
  if (F::kW4) {
    const uint32_t a = wst + warp * F::kTile + kW4Codes + 32 * q + 2 * (lane >> 2);
    return make_float2(lds_bf16(a), lds_bf16(a + 16));
  }
  const float s = lds_f32(sst + 4 * (kFewWarps * rt + warp));
  return make_float2(s, s);
}

constexpr int few_group_mmas(int group) { return group == 32 ? 2 : group == 64 ? 4 : 8; }

// One stage's slice of a warp: RT row tiles times NT blocks of 8 token columns,
// the columns' rows in `trow` (0: no such column).
template <int GROUP, int RT, int NT, int NTA>
MOE_DEV void slice_columns(uint32_t wst, uint32_t sst, const uint32_t (&trow)[NT], int warp, int lane, int tiles,
                         float (&acc)[RT][NTA][4]) {
  using F = FewForm<GROUP>;
  uint32_t b[NT][16];
#pragma unroll
  for (int j = 0; j < NT; ++j) {
#pragma unroll
    for (int i = 0; i < 16; ++i) b[j][i] = 0;
    if (trow[j]) load_token<GROUP>(trow[j], warp, lane, b[j]);
  }
#pragma unroll
  for (int rt = 0; rt < RT; ++rt) {
    if (rt < tiles) {
      const uint32_t w = wst + rt * F::kRowTile;
      uint32_t lo[8], hi[8];
      load_codes<GROUP>(w, warp, lane, lo, hi);
      float part[NT][4];
#pragma unroll
      for (int m = 0; m < 8; ++m) {
        uint32_t a[4];
        widen<GROUP>(lo, hi, m, a);
        if (m % few_group_mmas(GROUP) == 0) {
#pragma unroll
          for (int j = 0; j < NT; ++j) part[j][0] = part[j][1] = part[j][2] = part[j][3] = 0.f;
        }
#pragma unroll
        for (int j = 0; j < NT; ++j) mma_bf16(part[j], a, b[j][2 * m], b[j][2 * m + 1]);
        if ((m + 1) % few_group_mmas(GROUP) == 0) {
          const float2 s = load_scales<GROUP>(w, sst, rt, warp, lane, m / few_group_mmas(GROUP));
#pragma unroll
          for (int j = 0; j < NT; ++j) {
            acc[rt][j][0] = fmaf(part[j][0], s.x, acc[rt][j][0]);
            acc[rt][j][1] = fmaf(part[j][1], s.x, acc[rt][j][1]);
            acc[rt][j][2] = fmaf(part[j][2], s.y, acc[rt][j][2]);
            acc[rt][j][3] = fmaf(part[j][3], s.y, acc[rt][j][3]);
          }
        }
      }
    }
  }
}

// As slice_columns for tokens spread over NT blocks of columns of which few are in
// use (bit t of `mask`: token t): the widened codes stay in registers, each
// block in use passes over them.  Token t's row is the number of bits below t.
template <int GROUP, int RT, int NT>
MOE_DEV void slice_masked(uint32_t wst, uint32_t sst, uint32_t tok, uint64_t mask, int warp, int lane, int tiles,
                          float (&acc)[RT][NT][4]) {
  using F = FewForm<GROUP>;
#pragma unroll
  for (int rt = 0; rt < RT; ++rt) {
    if (rt < tiles) {
      const uint32_t w = wst + rt * F::kRowTile;
      uint32_t lo[8], hi[8], a[8][4];
      load_codes<GROUP>(w, warp, lane, lo, hi);
#pragma unroll
      for (int m = 0; m < 8; ++m) widen<GROUP>(lo, hi, m, a[m]);
#pragma unroll
      for (int j = 0; j < NT; ++j) {
        if ((mask >> (8 * j)) & 0xFF) {
          const int t = 8 * j + (lane >> 2);
          uint32_t b[16];
#pragma unroll
          for (int i = 0; i < 16; ++i) b[i] = 0;
          if ((mask >> t) & 1) load_token<GROUP>(tok + __popcll(mask & ((1ull << t) - 1)) * F::kTokPitch, warp, lane, b);
          float part[4];
#pragma unroll
          for (int m = 0; m < 8; ++m) {
            if (m % few_group_mmas(GROUP) == 0) part[0] = part[1] = part[2] = part[3] = 0.f;
            mma_bf16(part, a[m], b[2 * m], b[2 * m + 1]);
            if ((m + 1) % few_group_mmas(GROUP) == 0) {
              const float2 s = load_scales<GROUP>(w, sst, rt, warp, lane, m / few_group_mmas(GROUP));
              acc[rt][j][0] = fmaf(part[0], s.x, acc[rt][j][0]);
              acc[rt][j][1] = fmaf(part[1], s.x, acc[rt][j][1]);
              acc[rt][j][2] = fmaf(part[2], s.y, acc[rt][j][2]);
              acc[rt][j][3] = fmaf(part[3], s.y, acc[rt][j][3]);
            }
          }
        }
      }
    }
  }
}

// ---------------------------------------------------------------- the ring

struct FewRing {
  uint32_t base, stage_bytes, full, empty;   // shared addresses; full / empty: barriers 8 bytes apart
  int stages;
  int slot, phase;
  MOE_DEV uint32_t stage() const { return base + slot * stage_bytes; }
  MOE_DEV uint32_t full_bar() const { return full + 8 * slot; }
  MOE_DEV uint32_t empty_bar() const { return empty + 8 * slot; }
  MOE_DEV void next() {
    if (++slot == stages) { slot = 0; phase ^= 1; }
  }
};

// A warp's bounded wait: one outcome for all lanes.
MOE_DEV bool ring_wait(uint32_t bar, uint32_t parity, volatile int* abort_flag, int32_t* status) {
  return __all_sync(0xffffffffu, mbar_wait(bar, parity, abort_flag, status, kFewTimeoutNs));
}

template <int GROUP>
MOE_DEV uint32_t few_stage_bytes(int rt, int cols) {
  using F = FewForm<GROUP>;
  return (uint32_t)((rt * (F::kRowTile + F::kScaleBytes) + cols * F::kTokPitch + 127) & ~127);
}

// Where weight copies come from: one matrix of N rows (whole row tiles) and K columns.
struct FewMatrix {
  const uint8_t* p;
  const float* scale;
  int K;
};

// Copy `tiles` row tiles (the rt-th at row tile index tile0 + rt * tile_step) of
// 128-column slices [kt0, kt0 + nk) into the stage at `st`; whole warp.  `rt_cap`
// is the stage's room in row tiles, `sst` where its scales go.
template <int GROUP>
MOE_DEV void copy_weights(const FewMatrix& W, int tile0, int tile_step, int tiles, int kt0, int nk, uint32_t st, uint32_t sst,
                          uint32_t bar, int lane) {
  using F = FewForm<GROUP>;
  const int KT = (W.K + 127) / 128;
  if (F::kW4) {
    if (lane == 0) mbar_arrive_expect_tx(bar, tiles * nk * F::kTile);
    __syncwarp();
    if (lane < tiles)
      bulk_load(st + lane * F::kRowTile, W.p + ((size_t)(tile0 + lane * tile_step) * KT + kt0) * F::kTile, nk * F::kTile, bar);
  } else {
    if (lane == 0) mbar_arrive_expect_tx(bar, tiles * 16 * nk * 128);
    __syncwarp();
    for (int i = lane; i < tiles * 16; i += 32) {
      const int rt = i >> 4, r = i & 15;
      bulk_load(st + rt * F::kRowTile + r * F::kRowPitch,
                W.p + ((size_t)(tile0 + rt * tile_step) * 16 + r) * W.K + kt0 * 128, nk * 128, bar);
    }
    for (int i = lane; i < tiles * kFewWarps; i += 32) {
      const int rt = i / kFewWarps, kt = i % kFewWarps;
      const bool on = kt < nk;
      const float* src = W.scale + (size_t)((tile0 + rt * tile_step) >> 3) * KT + (on ? kt0 + kt : kt0);
      cp_async4(sst + 4 * i, src, on ? 4 : 0);
    }
    cp_async_arrive(bar);
  }
}

// Copy columns [128 kt0, 128 (kt0 + nk)) of `cols` token rows (row c at rows + c's
// index times pitch elements) behind the weights; K may end inside the last slice.
template <int GROUP, class RowOf>
MOE_DEV void copy_tokens(RowOf row_of, int cols, int K, int kt0, int nk, uint32_t tok, uint32_t bar, int lane) {
  using F = FewForm<GROUP>;
  const int valid = min(nk * 128, K - kt0 * 128);
  if (F::kW4 && valid < nk * 128) {   // zeros past K: the codes there are zero, the products must be too
    for (int c = 0; c < cols; ++c)
      for (int i = valid * 2 + lane * 16; i < nk * 256; i += 512)
        asm volatile("st.shared.v4.u32 [%0], {%1,%1,%1,%1};" :: "r"(tok + c * F::kTokPitch + i), "r"(0) : "memory");
    fence_proxy_async_shared();   // a later stage's bulk copy may overwrite them
    __syncwarp();
  }
  if (lane == 0) mbar_arrive_expect_tx(bar, cols * valid * 2);
  __syncwarp();
  if (lane < cols) bulk_load(tok + lane * F::kTokPitch, row_of(lane) + kt0 * 128, valid * 2, bar);
}

// ---------------------------------------------------------------- sums over the warps

// Each warp's accumulators of one 16 x 8 block, as they lie in the lanes.
MOE_DEV void put_block(float* red, int blocks, int warp, int block, int lane, const float (&c)[4]) {
  reinterpret_cast<float4*>(red)[(warp * blocks + block) * 32 + lane] = make_float4(c[0], c[1], c[2], c[3]);
}
// The sum over the warps, in their order, of row r (0..15) and column c (0..7).
MOE_DEV float get_sum(const float* red, int blocks, int block, int r, int c) {
  const int at = (4 * (r & 7) + (c >> 1)) * 4 + 2 * (r >> 3) + (c & 1);
  float s = 0.f;
#pragma unroll
  for (int w = 0; w < kFewWarps; ++w) s += red[(w * blocks + block) * 128 + at];
  return s;
}

MOE_DEV void consumer_sync() { asm volatile("bar.sync 1, 256;" ::: "memory"); }
// The computing warps' meeting that also tells all of them whether any gave up, so that
// they leave together.
MOE_DEV bool consumer_sync_all(bool ok) {
  uint32_t all;
  asm volatile(
      "{\n\t.reg .pred p, q;\n\t"
      "setp.ne.b32 p, %1, 0;\n\t"
      "bar.red.and.pred q, 1, 256, p;\n\t"
      "selp.u32 %0, 1, 0, q;\n\t}"
      : "=r"(all) : "r"((uint32_t)ok) : "memory");
  return all != 0;
}
MOE_DEV uint16_t to_bf16(float v) {
  const __nv_bfloat16 b = __float2bfloat16_rn(v);
  return *reinterpret_cast<const uint16_t*>(&b);
}

}  // namespace moe
