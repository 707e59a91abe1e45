// few_plan.h: how the decoding layer's kernel divides its shared memory, for the host and
// the device.
//
// Behind the barriers, the record of zeros and the routes' tables lie the sums on their
// way to the finishing warps, the output's sums, and a ring of stages, each the weights of some
// row tiles, the records of a segment's tokens and (FP8) the weights' scales.  With one stage
// nothing is copied while a stage is multiplied, so what is chosen leaves two.  64 tokens, H 7168,
// F 2048, one stage / two, us: 8 of 256 experts, 8 tokens to one of them, 4-bit with groups
// of 128 1660 / 1020, of 32 1822 / 1107; 8 of 32 experts, 16 tokens a segment, FP8 587 / 385;
// 16 of 64 experts, FP8 1139 / 783 (segments of up to 15).
#pragma once

#include <stdint.h>

#ifdef __CUDACC__
#define MOE_PLAN __host__ __device__ constexpr
#else
#define MOE_PLAN constexpr
#endif

namespace moe {

constexpr int kFewWarps = 8;                       // computing warps, one or two 128-column slices of a stage each
constexpr int kFewMaxStages = 12;
constexpr uint32_t kFewMinSmem = 227 * 1024;       // a block has at least as much
// Bytes of the record that holds 128 values of a token as the MMAs take them: f16
// values, the scale, and 12 bytes of alignment.
constexpr int kTokenRecord = 272;
// A warp's sums of one row tile: column c of rows 0..15 lies at 20 c floats of the warp's part,
// so that the stores of a warp, at 40 t + g floats for t = 0..3 and g = 0..7, do not meet in a bank.
constexpr int kFewColPitch = 20;
constexpr int kLayerCols = 16;                     // tokens per pass over a stage, at most
constexpr uint32_t kZeroAt = 256, kTablesAt = kZeroAt + (kTokenRecord + 15) / 16 * 16;

// Where the tables of T k = `pairs` pairs end.
MOE_PLAN uint32_t few_tables_end(int pairs) { return (kTablesAt + pairs * 21 + 127) & ~127u; }

// Bytes of a row tile's slice of 128 columns, and from one token's records to the next in a stage, 64
// mod 128: the 2 tokens x 64 bytes of a quarter-warp's reads then fall on distinct banks.
MOE_PLAN int few_tile_bytes(int group) { return group ? 1024 + 32 * (128 / group) : 2048; }
MOE_PLAN int few_token_pitch(int slices) { return slices * kTokenRecord + 64; }

struct LayerRoom {
  int bufs;             // buffers of sums
  uint32_t buf, sums;   // bytes of one, and of all
  uint32_t out;         // of the output's sums
  uint32_t tok, scale;  // where a stage's tokens and scales lie
  uint32_t stage;
  int stages;
};

// Weights of a row tile of a stage: sp slices of 128 columns per warp.  rt2: row tiles of a down
// stage.  Gate and up: one row tile of each, or two where the slices are few and the tokens many
// (4-bit, sp 1, not direct): these then serve twice the weights.  cap: columns of the
// fullest segment.  The sums take two buffers where the columns are few and two stages remain.
MOE_PLAN int layer_pairs(int group, int sp, bool direct) { return group != 0 && !direct && sp == 1 ? 2 : 1; }
MOE_PLAN LayerRoom layer_room(int group, int sp, int rt2, bool direct, int T, int pairs, int cap, uint32_t smem) {
  LayerRoom r = {};
  const int gate_up = 2 * layer_pairs(group, sp, direct), rt = rt2 > gate_up ? rt2 : gate_up;
  const uint32_t align = group ? 128 : 1024;
  r.tok = rt * kFewWarps * sp * few_tile_bytes(group);
  r.scale = r.tok + cap * few_token_pitch(kFewWarps * sp);
  r.stage = (r.scale + (group ? 0 : rt * 4 * kFewWarps * sp) + align - 1) / align * align;
  r.buf = kFewWarps * (direct || rt2 < 2 ? 2 : rt2) * cap * kFewColPitch * 4;
  r.out = direct ? 0 : T * 16 * rt2 * 4;
  for (r.bufs = direct || cap <= 8 ? 2 : 1;; r.bufs = 1) {
    r.sums = r.bufs * r.buf;
    const uint32_t down = kFewWarps * rt2 * T * kFewColPitch * 4;   // direct: one item's, [row tile][warp][token]
    if (direct && down > r.sums) r.sums = down;
    const uint32_t at = (few_tables_end(pairs) + r.sums + r.out + 1023) & ~1023u;
    r.stages = at < smem ? (int)((smem - at) / r.stage) : 0;
    if (r.stages > kFewMaxStages) r.stages = kFewMaxStages;
    if (direct || r.bufs == 1 || r.stages >= 2) return r;
  }
}

// 4-bit stages are short of work: handing one over takes some 300 cycles of a warp's 900.  Two
// slices per warp halve that, where no expert has more than 8 tokens and two such stages
// fit beside one another.
MOE_PLAN int layer_slices(int group, int rt2, bool direct, int T, int pairs, int cap, uint32_t smem) {
  return group != 0 && (direct || (cap <= 8 && layer_room(group, 2, rt2, false, T, pairs, cap, smem).stages >= 2)) ? 2 : 1;
}

// Tokens of a segment, at most: as many as leave two stages of them (15 for FP8 weights with three
// row tiles and more than some 800 pairs, else 16).
MOE_PLAN int layer_cols(int group, int rt2, bool direct, int T, int pairs, uint32_t smem) {
  int cols = kLayerCols;
  while (!direct && cols > 8 && layer_room(group, 1, rt2, false, T, pairs, cols, smem).stages < 2) --cols;
  return cols;
}

// The tensor kernel's warps (few_tensor.cuh): 0-15 widen, 16-23 sum, 24 copies, 25 and 26 issue
// MMAs, 27 makes up a warpgroup; their registers by setmaxnreg.  Its inc draws on what the block was
// launched with and waits for it without end, so a kernel with fewer registers a thread
// than the split needs (72) must not be launched.
constexpr int kTensorSum = 16, kTensorCopy = 24, kTensorMma = 25, kTensorWarps = 28;
constexpr int kTensorWidenRegs = 56, kTensorSumRegs = 120, kTensorRestRegs = 40;
MOE_PLAN bool tensor_split_fits(int regs) {
  return kTensorSum * kTensorWidenRegs + (kTensorCopy - kTensorSum) * kTensorSumRegs + (kTensorWarps - kTensorCopy) * kTensorRestRegs <=
         kTensorWarps * regs;
}

// Its ring: stages of 16 row tiles' slice of 128 columns and that of n tokens (8 to 64), behind 1 KB of barriers.
// Its two sets of widening warps wait for every second stage each.  With an odd number of stages
// a slot changes sets from round to round, and a wait by parity would take the round before
// last's fill for this one's, did the wait for an A buffer two slices earlier not imply that slice
// i - 4 is done, and so slice i - stages: with four stages or more.
constexpr int kTensorMinStages = 4;
MOE_PLAN uint32_t tensor_tokens_at(int group) { return (16 * few_tile_bytes(group) + 1023) & ~1023u; }
MOE_PLAN uint32_t tensor_stage(int group, int n) { return tensor_tokens_at(group) + 2 * n * 128; }
MOE_PLAN int tensor_stages(int group, int n, uint32_t smem) {
  const int s = (smem - 1024) / tensor_stage(group, n);
  return s < kFewMaxStages ? s : kFewMaxStages;
}

}  // namespace moe
