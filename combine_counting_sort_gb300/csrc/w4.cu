// w4.cu: 4-bit weights with group scales: quantise, lay out, read back.
#include "host_util.h"
#include "w4.cuh"

namespace moe {

// All three kernels: one warp per tile, the warps of a block on neighbouring tiles of a
// row of tiles.  Quantising and packing, lane 4g + t owns rows g and 8 + g and columns 32 j + 8 t + 0..7: 16
// bytes of bf16 per j, 4 lanes on 64 bytes of a row, and 16 bytes of codes per half.
// Bound by memory (quantising: 2.5 bytes a weight, and some 8 instructions).  16 matrices of 4096 x
// 7168, groups of 128: quantised in 178 us (6.7 TB/s), packed in 100 us, read back in 310
// us, almost all of it the 1.88 GB written.
constexpr int kW4Warps = 8;

struct W4Tile {
  int e, nt, kt, lane;
  bool on;
  size_t at;   // tile index
  MOE_DEV W4Tile(int KT, int NT) {
    kt = blockIdx.x * kW4Warps + (threadIdx.x >> 5);
    nt = blockIdx.y;
    e = blockIdx.z;
    lane = threadIdx.x & 31;
    on = kt < KT;
    at = ((size_t)e * NT + nt) * KT + kt;
  }
};

// The code of w in a scale s: rint of the quotient, plus 8.  The quotient by the
// reciprocal and one correction (Markstein's division step, "Computation of
// elementary functions on the IBM RISC System/6000 processor", 1990): it is the
// exact quotient wherever that is an fp32 value, so wherever it lies half way
// between two codes, and else within an ulp, while the quotient of two bf16
// values nearest to half way, but not on it, is 2^-10 from it.  1.5 * 2^23 + 8 brings the
// rounded integer, ties to even, into the low bits.
MOE_DEV uint32_t w4_code(float w, float s, float inv) {
  const float q0 = __fmul_rn(w, inv);
  const float q = __fmaf_rn(__fmaf_rn(-q0, s, w), inv, q0);
  return __float_as_uint(__fadd_rn(q, 12582920.f)) & 15u;
}
// Scales outside [2^-100, 2^100], whose reciprocal or residual may leave fp32's normal
// range: by division.  A scale of zero: 8.
MOE_DEV uint32_t w4_code_far(float w, float s) {
  if (!(s > 0.f)) return 8u;
  return (uint32_t)((int)fminf(fmaxf(rintf(__fdiv_rn(w, s)), -8.f), 7.f) + 8);
}

template <int GROUP>
__global__ void __launch_bounds__(kW4Warps * 32) quant_w4_kernel(const uint16_t* __restrict__ W, int N, int K, int KT,
                                                                 uint8_t* __restrict__ Wp) {
  constexpr int kGroups = kW4Cols / GROUP, kPer = 4 / kGroups;   // words j per group
  const W4Tile T(KT, gridDim.y);
  if (!T.on) return;
  const int g = T.lane >> 2, t = T.lane & 3;
  uint4 v[2][4];
#pragma unroll
  for (int h = 0; h < 2; ++h)
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const int n = T.nt * kW4Rows + 8 * h + g, c = T.kt * kW4Cols + 32 * j + 8 * t;   // K is a multiple of 32
      v[h][j] = n < N && c < K ? __ldcs(reinterpret_cast<const uint4*>(W + ((size_t)T.e * N + n) * K + c)) : make_uint4(0, 0, 0, 0);
    }
  uint8_t* tile = Wp + T.at * w4_tile_bytes(GROUP);
#pragma unroll
  for (int h = 0; h < 2; ++h) {
    uint32_t code[4];
#pragma unroll
    for (int q = 0; q < kGroups; ++q) {
      // magnitudes of bf16 values order like their bits, a NaN above all
      uint32_t m = 0;
#pragma unroll
      for (int j = q * kPer; j < (q + 1) * kPer; ++j) {
        const uint32_t w[4] = {v[h][j].x, v[h][j].y, v[h][j].z, v[h][j].w};
#pragma unroll
        for (int i = 0; i < 4; ++i) m = __vmaxu2(m, w[i] & 0x7FFF7FFFu);
      }
      m = max(m & 0xFFFFu, m >> 16);
      m = max(m, __shfl_xor_sync(0xffffffffu, m, 1));
      m = max(m, __shfl_xor_sync(0xffffffffu, m, 2));
      const __nv_bfloat16 sb = __float2bfloat16_rn(__fdiv_rn(__uint_as_float(m << 16), 7.0f));
      const uint16_t bits = *reinterpret_cast<const uint16_t*>(&sb);
      if (t == 0) *reinterpret_cast<uint16_t*>(tile + kW4Codes + 2 * (16 * q + 8 * h + g)) = bits;
      const float s = bf16_lo(bits);
      if (s >= 0x1p-100f && s <= 0x1p100f) {
        const float inv = __frcp_rn(s);
#pragma unroll
        for (int j = q * kPer; j < (q + 1) * kPer; ++j) {
          const uint32_t w[4] = {v[h][j].x, v[h][j].y, v[h][j].z, v[h][j].w};
          code[j] = 0;
#pragma unroll
          for (int i = 0; i < 4; ++i)
            code[j] |= w4_code(bf16_lo(w[i]), s, inv) << (4 * i) | w4_code(bf16_hi(w[i]), s, inv) << (4 * i + 16);
        }
      } else {
#pragma unroll
        for (int j = q * kPer; j < (q + 1) * kPer; ++j) {
          const uint32_t w[4] = {v[h][j].x, v[h][j].y, v[h][j].z, v[h][j].w};
          code[j] = 0;
#pragma unroll 1
          for (int i = 0; i < 4; ++i) {
            const uint32_t u = i == 0 ? w[0] : i == 1 ? w[1] : i == 2 ? w[2] : w[3];
            code[j] |= w4_code_far(bf16_lo(u), s) << (4 * i) | w4_code_far(bf16_hi(u), s) << (4 * i + 16);
          }
        }
      }
    }
    reinterpret_cast<uint4*>(tile)[32 * h + T.lane] = make_uint4(code[0], code[1], code[2], code[3]);
  }
}

// Eight codes in the columns' order -> the tile's: nibble 2p to p, 2p + 1 to p + 4.
MOE_DEV uint32_t w4_reorder(uint32_t c) {
  uint32_t even = c & 0x0F0F0F0Fu, odd = (c >> 4) & 0x0F0F0F0Fu;
  even = (even | even >> 4) & 0x00FF00FFu;
  odd = (odd | odd >> 4) & 0x00FF00FFu;
  return ((even | even >> 8) & 0xFFFFu) | (odd | odd >> 8) << 16;
}

// Codes and scales of a checkpoint, laid out.
template <int GROUP>
__global__ void __launch_bounds__(kW4Warps * 32) pack_w4_kernel(const uint8_t* __restrict__ codes, const uint16_t* __restrict__ scale,
                                                                int N, int K, int KT, uint8_t* __restrict__ Wp) {
  const W4Tile T(KT, gridDim.y);
  if (!T.on) return;
  const int g = T.lane >> 2, t = T.lane & 3;
  uint8_t* tile = Wp + T.at * w4_tile_bytes(GROUP);
#pragma unroll
  for (int h = 0; h < 2; ++h) {
    uint32_t code[4];
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const int n = T.nt * kW4Rows + 8 * h + g, c = T.kt * kW4Cols + 32 * j + 8 * t;
      code[j] = n < N && c < K ? w4_reorder(__ldcs(reinterpret_cast<const uint32_t*>(codes + (((size_t)T.e * N + n) * K + c) / 2)))
                               : 0x88888888u;
    }
    reinterpret_cast<uint4*>(tile)[32 * h + T.lane] = make_uint4(code[0], code[1], code[2], code[3]);
  }
  for (int i = T.lane; i < kW4Rows * (kW4Cols / GROUP); i += 32) {
    const int n = T.nt * kW4Rows + i % kW4Rows, q = T.kt * (kW4Cols / GROUP) + i / kW4Rows;
    *reinterpret_cast<uint16_t*>(tile + kW4Codes + 2 * i) =
        n < N && q < K / GROUP ? scale[((size_t)T.e * N + n) * (K / GROUP) + q] : (uint16_t)0;
  }
}

// The values that the codes stand for, in fp32 (exact: 4 bits times 8 bits).  Here a lane
// owns columns 4 lane .. of every row, so that a store is 512 bytes in a row; the
// codes of a row are 64 bytes in a row, two lanes to a word.
template <int GROUP>
__global__ void __launch_bounds__(kW4Warps * 32) dequant_w4_kernel(const uint8_t* __restrict__ Wp, int N, int K, int KT,
                                                                   float* __restrict__ W) {
  const W4Tile T(KT, gridDim.y);
  if (!T.on) return;
  const uint8_t* tile = Wp + T.at * w4_tile_bytes(GROUP);
  const int c = 4 * T.lane, n0 = T.nt * kW4Rows, col = T.kt * kW4Cols + c;
  uint32_t code[kW4Rows];
  uint16_t scale[kW4Rows];
#pragma unroll
  for (int r = 0; r < kW4Rows; ++r) {
    code[r] = __ldcs(reinterpret_cast<const uint32_t*>(tile) + 4 * (32 * (r >> 3) + 4 * (r & 7) + ((c & 31) >> 3)) + (c >> 5));
    scale[r] = *reinterpret_cast<const uint16_t*>(tile + kW4Codes + 2 * (16 * (c / GROUP) + r));
  }
  if (col >= K) return;
#pragma unroll
  for (int r = 0; r < kW4Rows; ++r) {
    if (n0 + r >= N) break;
    const uint32_t w = code[r] >> (8 * (T.lane & 1));
    const float s = bf16_lo(scale[r]);
    float v[4];
#pragma unroll
    for (int i = 0; i < 4; ++i)   // 2^23 + code, less 2^23 + 8
      v[i] = (__uint_as_float(0x4B000000u | ((w >> (16 * (i & 1) + 4 * (i >> 1))) & 15u)) - 8388616.f) * s;
    __stcs(reinterpret_cast<float4*>(W + ((size_t)T.e * N + n0 + r) * K + col), make_float4(v[0], v[1], v[2], v[3]));
  }
}

}  // namespace moe

using namespace moe;

static int check_w4(int E, int N, int K, int group) {
  if (!w4_group_ok(group)) return MOE_ERR_INVALID_ARG;
  if (E < 1 || E > 65535 || N < 1 || N > MOE_W4_MAX_N || K < group || K % group || K > MOE_W4_MAX_K) return MOE_ERR_INVALID_ARG;
  return MOE_OK;
}

static dim3 w4_grid(int E, int N, int K) { return dim3(((K + 127) / 128 + kW4Warps - 1) / kW4Warps, (N + 15) / 16, E); }

#define W4_LAUNCH(kernel, ...)                                                                              \
  do {                                                                                                      \
    const dim3 grid = w4_grid(E, N, K);                                                                     \
    cudaStream_t s = (cudaStream_t)stream;                                                                  \
    if (group == 32) kernel<32><<<grid, kW4Warps * 32, 0, s>>>(__VA_ARGS__);                                \
    else if (group == 64) kernel<64><<<grid, kW4Warps * 32, 0, s>>>(__VA_ARGS__);                           \
    else kernel<128><<<grid, kW4Warps * 32, 0, s>>>(__VA_ARGS__);                                           \
  } while (0)

extern "C" int moe_w4_packed_bytes(int N, int K, int group, size_t* bytes) {
  if (!bytes) return MOE_ERR_INVALID_ARG;
  const int rc = check_w4(1, N, K, group);
  if (rc) return rc;
  *bytes = w4_matrix_bytes(N, K, group);
  return MOE_OK;
}

extern "C" int moe_quant_weights_w4(const uint16_t* W, int E, int N, int K, int group, uint8_t* Wp,
                                    moe_stream_t stream) {
  if (!W || !Wp || !aligned16(W) || !aligned16(Wp)) return MOE_ERR_INVALID_ARG;
  const int rc = check_w4(E, N, K, group);
  if (rc) return rc;
  W4_LAUNCH(quant_w4_kernel, W, N, K, (K + 127) / 128, Wp);
  return cudaGetLastError() == cudaSuccess ? MOE_OK : MOE_ERR_CUDA;
}

extern "C" int moe_pack_weights_w4(const uint8_t* codes, const uint16_t* scale, int E, int N, int K, int group,
                                   uint8_t* Wp, moe_stream_t stream) {
  if (!codes || !scale || !Wp || !aligned16(Wp) || ((uintptr_t)scale & 1) || ((uintptr_t)codes & 3)) return MOE_ERR_INVALID_ARG;
  const int rc = check_w4(E, N, K, group);
  if (rc) return rc;
  W4_LAUNCH(pack_w4_kernel, codes, scale, N, K, (K + 127) / 128, Wp);
  return cudaGetLastError() == cudaSuccess ? MOE_OK : MOE_ERR_CUDA;
}

extern "C" int moe_dequant_weights_w4(const uint8_t* Wp, int E, int N, int K, int group, float* W,
                                      moe_stream_t stream) {
  if (!Wp || !W || !aligned16(Wp) || !aligned16(W)) return MOE_ERR_INVALID_ARG;
  const int rc = check_w4(E, N, K, group);
  if (rc) return rc;
  W4_LAUNCH(dequant_w4_kernel, Wp, N, K, (K + 127) / 128, W);
  return cudaGetLastError() == cudaSuccess ? MOE_OK : MOE_ERR_CUDA;
}
