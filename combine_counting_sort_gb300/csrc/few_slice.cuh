// few_slice.cuh: weights times tokens on a stage's slices.
//
// The products run on f16 MMAs with fp32 sums.  An e4m3 code is one of the f16
// values (one conversion per two codes).  A pair of 4-bit codes takes an AND and a
// multiply-add, and two pairs a shift: the bits 0x000c and 0x00c0 read as f16 are c * 2^-24 and
// 16 c * 2^-24 (f16 is linear from its subnormals to the end of the first binade), of which
// the multiply-add makes (c - 8) * 2^-9, exactly; the sums are multiplied by 2^9 at the
// end.  (Taking the 8 out of a group's sum instead, as 8 times the sum of the token's values,
// saves the multiply-adds but loses the low bits of that sum to a large value that
// meets a weight of zero.)
//
// A token's 128 values share a power of two 2^e that brings their largest magnitude
// into [2^14, 2^15): a bf16 value is then an f16 value as it is, down to 2^-31 of the
// block's largest, and smaller ones are within 2^-39 of that largest.  The layer's activations
// between its products, fp32 values, are rounded to f16's 11 bits this way, those below
// 2^-28 of the largest to within 2^-39 of it.  (A second f16 for what that leaves out would double
// the MMAs and the records; with out in bf16 the error against 64 bits is 1% more for the rounding.)
//
// What bounds it: memory.  Per tile of 16 x 128 weights a warp spends 40 ANDs and
// shifts and 32 multiply-adds (4-bit) or 32 conversions (FP8), 8 MMAs per 8 tokens
// and some 30 other instructions.  A stage of 6 x 8 tiles of FP8 took 1150 cycles with the
// conversions as the compiler unpacks them, 640 as written here (a stage's bytes: 610).
#pragma once

#include <cuda_fp16.h>

#include "few.cuh"
#include "few_host.h"

namespace moe {

// SP: 128-column slices of a stage per warp.
template <int GROUP, int SP>
struct FewForm {
  static constexpr bool kW4 = GROUP != 0;
  static constexpr int kTile = few_tile_bytes(GROUP);
  static_assert(!kW4 || kTile == w4_tile_bytes(kW4 ? GROUP : 128), "");
  static constexpr int kSlices = kFewWarps * SP;
  // 4-bit: the slices' tiles as they lie in memory.  FP8: per slice 16 rows of
  // 128 bytes in TMA's 128-byte swizzle, which ldmatrix reads without bank conflicts.
  static constexpr int kRowTile = kSlices * kTile;
  static constexpr int kTokPitch = few_token_pitch(kSlices);
  // arrivals that complete a stage: weights, tokens, and the lanes' scale copies
  static constexpr int kArrivals = kW4 ? 2 : 34;
  static constexpr float kSumScale = kW4 ? 0x1p9f : 1.f;   // what the sums lack
};
// ---------------------------------------------------------------- token records

// Four consecutive values v (columns 4 lane ..) of a warp's 128 into the record at
// `rec`: the 16 bytes at 64 i + 16 t are the B operands that lane t of a column reads for
// the MMAs 2i and 2i + 1.  4-bit: columns 32 i + 8 t ...  FP8: columns 32 i + 4 t .. and
// 32 i + 16 + 4 t .., which ldmatrix gives to lane t.  Behind the values: the scale.
template <int GROUP>
MOE_DEV void put_record(const float (&v)[4], uint8_t* rec, int lane) {
  uint32_t big = 0;
#pragma unroll
  for (int i = 0; i < 4; ++i) big = max(big, __float_as_uint(v[i]) & 0x7FFFFFFFu);
  big = __reduce_max_sync(0xffffffffu, big);
  const int e = max((int)(big >> 23) - 127 - 14, -125);
  const float down = __uint_as_float((uint32_t)(127 - e) << 23);
  const __half2 a = __floats2half2_rn(v[0] * down, v[1] * down), b = __floats2half2_rn(v[2] * down, v[3] * down);
  const int at = GROUP != 0 ? 8 * lane : 64 * (lane >> 3) + 16 * (lane & 3) + 8 * ((lane >> 2) & 1);
  *reinterpret_cast<uint2*>(rec + at) = make_uint2(*reinterpret_cast<const uint32_t*>(&a), *reinterpret_cast<const uint32_t*>(&b));
  if (lane == 0) *reinterpret_cast<float*>(rec + 256) = __uint_as_float((uint32_t)(127 + e) << 23);
}

// ---------------------------------------------------------------- products

// The codes of a row tile's slice: 4-bit: the lane's words of row g (0-3) and of row
// g + 8 (4-7).  FP8: words m and m + 8 are columns 16 m + 4 t .. of row g and of row g + 8.
template <int GROUP>
MOE_DEV void load_codes(uint32_t wst, int slice, int lane, uint32_t (&c)[GROUP ? 8 : 16]) {
  using F = FewForm<GROUP, 1>;
  if constexpr (F::kW4) {
    const uint32_t p = wst + slice * F::kTile + lane * 16;
    const uint4 l = lds128(p), h = lds128(p + 512);
    c[0] = l.x; c[1] = l.y; c[2] = l.z; c[3] = l.w;
    c[4] = h.x; c[5] = h.y; c[6] = h.z; c[7] = h.w;
  } else {
    const uint32_t row = wst + slice * 2048 + (lane & 15) * 128;
#pragma unroll
    for (int j = 0; j < 4; ++j)   // 16-byte chunks 2j (lanes 0-15 give the rows' addresses) and 2j + 1
      asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0,%1,%2,%3}, [%4];"
                   : "=r"(c[2 * j]), "=r"(c[2 * j + 8]), "=r"(c[2 * j + 1]), "=r"(c[2 * j + 9])
                   : "r"(row + (((2 * j + (lane >> 4)) ^ (lane & 7)) << 4)) : "memory");
  }
}

// Four e4m3 codes as f16 values: the first two, and the others.
MOE_DEV void widen_e4m3(uint32_t codes, uint32_t& lo, uint32_t& hi) {
  asm("{\n\t.reg .b16 l, h;\n\t"
      "mov.b32 {l, h}, %2;\n\t"
      "cvt.rn.f16x2.e4m3x2 %0, l;\n\t"
      "cvt.rn.f16x2.e4m3x2 %1, h;\n\t}"
      : "=r"(lo), "=r"(hi) : "r"(codes));
}

// Two pairs of 4-bit codes, at the low and at the high nibbles of a word's lower bytes, as f16 (c - 8) * 2^-9:
// c * 2^-24 times 2^15, 16 c * 2^-24 times 2^11, less 2^-6.
MOE_DEV void widen_w4(uint32_t word, uint32_t& lo, uint32_t& hi) {
  asm("fma.rn.f16x2 %0, %1, %2, %3;" : "=r"(lo) : "r"(word & 0x000F000Fu), "r"(0x78007800u), "r"(0xA400A400u));
  asm("fma.rn.f16x2 %0, %1, %2, %3;" : "=r"(hi) : "r"(word & 0x00F000F0u), "r"(0x68006800u), "r"(0xA400A400u));
}

// The A operand of MMA m of a slice.
template <int GROUP>
MOE_DEV void widen(const uint32_t (&c)[GROUP ? 8 : 16], int m, uint32_t (&a)[4]) {
  if constexpr (GROUP != 0) {
    const uint32_t l = c[m >> 1] >> (m & 1 ? 8 : 0), h = c[4 + (m >> 1)] >> (m & 1 ? 8 : 0);
    widen_w4(l, a[0], a[2]);
    widen_w4(h, a[1], a[3]);
  } else {
    widen_e4m3(c[m], a[0], a[2]);
    widen_e4m3(c[m + 8], a[1], a[3]);
  }
}

// The scales of a row tile's slice for rows g and g + 8, per group.
template <int GROUP, int SP>
MOE_DEV void load_scales(uint32_t wst, uint32_t scales, int rt, int slice, int lane, float (&s)[FewGroups<GROUP>::kCount][2]) {
  using F = FewForm<GROUP, SP>;
#pragma unroll
  for (int q = 0; q < FewGroups<GROUP>::kCount; ++q) {
    if (F::kW4) {
      const uint32_t sc = wst + slice * F::kTile + kW4Codes + 32 * q + 2 * (lane >> 2);
      s[q][0] = lds_bf16(sc);
      s[q][1] = lds_bf16(sc + 16);
    } else {
      s[q][0] = s[q][1] = lds_f32(scales + 4 * (F::kSlices * rt + slice));
    }
  }
}

// Where a lane finds its columns' tokens behind the first one's records, for NT blocks of 8 columns: its B
// operand's (column 8 j + lane / 4) and those of its sums (8 j + 2 (lane % 4) and the
// next); -1 where a column has none.  Bit c of `mask` says that column c has a
// token, and the number of bits below it which one in the row it is, `pitch` apart.
template <int NT>
struct LaneTokens {
  int b[NT], x[NT][2];
  MOE_DEV LaneTokens(uint32_t mask, int pitch, int lane) {
    auto at = [&](int c) { return (mask >> c) & 1 ? __popc(mask & ((1u << c) - 1)) * pitch : -1; };
#pragma unroll
    for (int j = 0; j < NT; ++j) {
      b[j] = at(8 * j + (lane >> 2));
      x[j][0] = at(8 * j + 2 * (lane & 3));
      x[j][1] = at(8 * j + 2 * (lane & 3) + 1);
    }
  }
};

// One stage's slice of a warp: RT row tiles times NT blocks of 8 columns, added to
// acc (rows g and g + 8 of the lane's two columns of a block).  The first token's record
// of these columns is at `tokens`; columns without a token read the zeros at `zero`.  The MMAs of the row tiles are chains of their own:
// an MMA's result takes some 20 cycles, and with two warps to a scheduler little else
// fills them.  A stage with fewer row tiles holds older ones in their place, whose
// sums are not used.  OWN: the sums of a column without a token stay as they are: they are
// used, and zeros times weights that are infinite or NaN are NaN.
template <int GROUP, int SP, int RT, int NT, bool OWN = false>
MOE_DEV void few_slice(uint32_t st, uint32_t scales, uint32_t tokens, uint32_t zero, const LaneTokens<NT>& lt, int slice, int lane,
                       float (&acc)[RT][NT][4]) {
  using F = FewForm<GROUP, SP>;
  constexpr int kCount = FewGroups<GROUP>::kCount, kMmas = 8 / kCount;
  uint32_t c[RT][GROUP ? 8 : 16], b[NT][16];
  float s[RT][kCount][2], xs[NT][2];
#pragma unroll
  for (int j = 0; j < NT; ++j) {
    const uint32_t p = lt.b[j] < 0 ? zero : tokens + lt.b[j];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const uint4 v = lds128(p + 64 * i + 16 * (lane & 3));
      b[j][4 * i] = v.x; b[j][4 * i + 1] = v.y; b[j][4 * i + 2] = v.z; b[j][4 * i + 3] = v.w;
    }
  }
#pragma unroll
  for (int rt = 0; rt < RT; ++rt) {
    load_codes<GROUP>(st + rt * F::kRowTile, slice, lane, c[rt]);
    load_scales<GROUP, SP>(st + rt * F::kRowTile, scales, rt, slice, lane, s[rt]);
  }
#pragma unroll
  for (int j = 0; j < NT; ++j)
#pragma unroll
    for (int i = 0; i < 2; ++i) xs[j][i] = lds_f32((lt.x[j][i] < 0 ? zero : tokens + lt.x[j][i]) + 256);
  float v[RT][NT][4];
#pragma unroll
  for (int q = 0; q < kCount; ++q) {
    float part[RT][NT][4];
#pragma unroll
    for (int rt = 0; rt < RT; ++rt)
#pragma unroll
      for (int j = 0; j < NT; ++j)
#pragma unroll
        for (int i = 0; i < 4; ++i) part[rt][j][i] = 0.f;
#pragma unroll
    for (int m = q * kMmas; m < (q + 1) * kMmas; ++m)
#pragma unroll
      for (int rt = 0; rt < RT; ++rt) {
        uint32_t a[4];
        widen<GROUP>(c[rt], m, a);
#pragma unroll
        for (int j = 0; j < NT; ++j) mma_f16(part[rt][j], a, b[j][2 * m], b[j][2 * m + 1]);
      }
#pragma unroll
    for (int rt = 0; rt < RT; ++rt)
#pragma unroll
      for (int j = 0; j < NT; ++j)
#pragma unroll
        for (int i = 0; i < 4; ++i)
          v[rt][j][i] = q == 0 ? part[rt][j][i] * s[rt][q][i >> 1] : fmaf(part[rt][j][i], s[rt][q][i >> 1], v[rt][j][i]);
  }
#pragma unroll
  for (int rt = 0; rt < RT; ++rt)
#pragma unroll
    for (int j = 0; j < NT; ++j)
#pragma unroll
      for (int i = 0; i < 4; ++i)
        if (!OWN || lt.x[j][i & 1] >= 0) acc[rt][j][i] = fmaf(v[rt][j][i], xs[j][i & 1], acc[rt][j][i]);
}

// A warp's sums of RT row tiles into the meeting place `red`: [row tile][warp][column].
template <int RT, int NT>
MOE_DEV void put_sums(float* red, int pitch, int cols, int warp, int lane, const float (&acc)[RT][NT][4]) {
#pragma unroll
  for (int rt = 0; rt < RT; ++rt)
#pragma unroll
    for (int j = 0; j < NT; ++j)
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const int c = 8 * j + 2 * (lane & 3) + (i & 1);
        if (c < cols) red[((rt * kFewWarps + warp) * pitch + c) * kFewColPitch + (lane >> 2) + 8 * (i >> 1)] = acc[rt][j][i];
      }
}

}  // namespace moe
