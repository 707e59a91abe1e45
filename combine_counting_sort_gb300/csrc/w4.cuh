// w4.cuh: the laid-out form of 4-bit weights.
//
// A matrix [N, K] is a row-major grid of tiles of 16 rows x 128 columns, each
// one contiguous run of bytes: 1024 bytes of codes, then 128/group rows of 16
// bf16 scales (one per matrix row).  What the matrix lacks of a whole tile has
// code 8 (value 0) and scale 0.
//
// The codes lie in the order in which mma.sync.m16n8k16 takes its A operand:
// 16 bytes per lane and half (rows 0-7, rows 8-15), so one 16-byte read per
// lane and half brings a lane's 32 codes of row g = lane / 4 without bank
// conflicts.  Word j of those 16 bytes holds columns 32 j + 8 t + 0..7
// (t = lane % 4): nibble p is column 2p and nibble p + 4 column 2p + 1, so
// that (word >> 4p) & 0x000F000F is the pair of neighbours that one 32-bit A
// register holds.  The column order inside an MMA is free as long as the B
// operand follows it: its lane t reads the same 8 columns, 16 bytes of bf16.
#pragma once

#include "common.cuh"

namespace moe {

constexpr int kW4Codes = 1024;   // bytes of codes in a tile
constexpr int kW4Rows = 16, kW4Cols = 128;

__host__ __device__ __forceinline__ constexpr int w4_tile_bytes(int group) {
  return kW4Codes + 32 * (kW4Cols / group);
}
__host__ __device__ __forceinline__ constexpr bool w4_group_ok(int group) {
  return group == 32 || group == 64 || group == 128;
}
__host__ __device__ __forceinline__ constexpr size_t w4_matrix_bytes(int N, int K, int group) {
  return (size_t)((N + 15) / 16) * ((K + 127) / 128) * w4_tile_bytes(group);
}

}  // namespace moe
