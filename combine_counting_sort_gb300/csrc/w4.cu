// w4.cu: 4-bit weights with group scales: quantise, lay out, read back.
#include "host_util.h"
#include "w4.cuh"

namespace moe {

// Byte b of word (half, lane = 4g + t, j) of a tile's codes: the nibbles of row
// 8 half + g, columns 32j + 8t + 4 (b % 2) + b / 2 (low) and two further (high).
// A thread builds one 16-byte read of the matmul: the 32 codes of one row and t.

// The bf16 scale of a group whose largest magnitude is `am`, and a value's code:
// round to nearest even of the fp32 quotient, both exact roundings of the rule
// (am / 7 and w / scale of two 8-bit significands are never within 2^-17 of a
// rounding boundary without lying on it).  Infinite or NaN maxima give a
// scale that is not finite, which the products then show.
MOE_DEV uint16_t w4_scale(float am) {
  const __nv_bfloat16 s = __float2bfloat16_rn(__fdiv_rn(am, 7.0f));
  return *reinterpret_cast<const uint16_t*>(&s);
}
MOE_DEV uint32_t w4_code(float w, float scale) {
  if (!(scale > 0.f)) return 8u;
  const float q = rintf(__fdiv_rn(w, scale));
  return (uint32_t)((int)fminf(fmaxf(q, -8.f), 7.f) + 8);
}

// One block per tile: 128 threads stage 16 x 128 values in shared memory, reduce
// the group maxima, then 64 threads write 16 bytes of codes each.
__global__ void __launch_bounds__(128) quant_w4_kernel(const uint16_t* __restrict__ W, int N, int K, int group,
                                                       uint8_t* __restrict__ Wp) {
  __shared__ float v[kW4Rows][kW4Cols + 1];
  __shared__ float sc[kW4Rows][4];
  const int kt = blockIdx.x, nt = blockIdx.y, e = blockIdx.z, tid = threadIdx.x;
  const int KT = gridDim.x, NT = gridDim.y, G = kW4Cols / group;
  uint8_t* tile = Wp + (((size_t)e * NT + nt) * KT + kt) * w4_tile_bytes(group);
  const int c = kt * kW4Cols + tid;
  for (int r = 0; r < kW4Rows; ++r) {
    const int n = nt * kW4Rows + r;
    v[r][tid] = n < N && c < K ? bf16_lo(W[((size_t)e * N + n) * K + c]) : 0.f;
  }
  __syncthreads();
  if (tid < kW4Rows * G) {
    const int r = tid % kW4Rows, g = tid / kW4Rows;
    float am = 0.f;
    for (int i = 0; i < group; ++i) {
      const float a = fabsf(v[r][g * group + i]);
      am = a > am || a != a ? a : am;   // a NaN stays
    }
    const uint16_t s = w4_scale(am);
    sc[r][g] = bf16_lo(s);
    *reinterpret_cast<uint16_t*>(tile + kW4Codes + 2 * (16 * g + r)) = s;
  }
  __syncthreads();
  if (tid < 64) {
    const int half = tid >> 5, lane = tid & 31, r = 8 * half + (lane >> 2), t = lane & 3;
    uint32_t w[4];
    for (int j = 0; j < 4; ++j) {
      const int k0 = 32 * j + 8 * t;
      w[j] = 0;
      for (int p = 0; p < 4; ++p) {
        w[j] |= w4_code(v[r][k0 + 2 * p], sc[r][k0 / group]) << (4 * p);
        w[j] |= w4_code(v[r][k0 + 2 * p + 1], sc[r][k0 / group]) << (4 * p + 16);
      }
    }
    reinterpret_cast<uint4*>(tile)[tid] = make_uint4(w[0], w[1], w[2], w[3]);
  }
}

// Codes and scales of a checkpoint, laid out: one thread per 32 codes.
__global__ void __launch_bounds__(64) pack_w4_kernel(const uint8_t* __restrict__ codes, const uint16_t* __restrict__ scale,
                                                     int N, int K, int group, uint8_t* __restrict__ Wp) {
  const int kt = blockIdx.x, nt = blockIdx.y, e = blockIdx.z, tid = threadIdx.x;
  const int KT = gridDim.x, NT = gridDim.y, G = kW4Cols / group;
  uint8_t* tile = Wp + (((size_t)e * NT + nt) * KT + kt) * w4_tile_bytes(group);
  const int half = tid >> 5, lane = tid & 31, t = lane & 3;
  const int n = nt * kW4Rows + 8 * half + (lane >> 2);
  uint32_t w[4];
  for (int j = 0; j < 4; ++j) {
    const int k0 = kt * kW4Cols + 32 * j + 8 * t;
    w[j] = 0x88888888u;
    if (n < N && k0 < K) {   // K is a multiple of the group, so 8 columns are in or out together
      w[j] = 0;
      const uint8_t* src = codes + (((size_t)e * N + n) * K + k0) / 2;
      for (int p = 0; p < 4; ++p) w[j] |= (uint32_t)(src[p] & 15) << (4 * p) | (uint32_t)(src[p] >> 4) << (4 * p + 16);
    }
  }
  reinterpret_cast<uint4*>(tile)[tid] = make_uint4(w[0], w[1], w[2], w[3]);
  if (tid < kW4Rows * G) {
    const int r = tid % kW4Rows, g = tid / kW4Rows;
    const int nr = nt * kW4Rows + r, kg = kt * G + g;
    *reinterpret_cast<uint16_t*>(tile + kW4Codes + 2 * (16 * g + r)) =
        nr < N && kg < K / group ? scale[((size_t)e * N + nr) * (K / group) + kg] : (uint16_t)0;
  }
}

// The values that the codes stand for, in fp32 (exact: 4 bits times 8 bits).
__global__ void __launch_bounds__(128) dequant_w4_kernel(const uint8_t* __restrict__ Wp, int N, int K, int group,
                                                         float* __restrict__ W) {
  const int kt = blockIdx.x, nt = blockIdx.y, e = blockIdx.z;
  const uint8_t* tile = Wp + (((size_t)e * gridDim.y + nt) * gridDim.x + kt) * w4_tile_bytes(group);
  const int c = kt * kW4Cols + threadIdx.x;
  if (c >= K) return;
  for (int r = 0; r < kW4Rows && nt * kW4Rows + r < N; ++r)
    W[((size_t)e * N + nt * kW4Rows + r) * K + c] = w4_value(tile, r, threadIdx.x, group);
}

}  // namespace moe

using namespace moe;

static int check_w4(int E, int N, int K, int group) {
  if (!w4_group_ok(group)) return MOE_ERR_INVALID_ARG;
  if (E < 1 || E > 65535 || N < 1 || N > MOE_W4_MAX_N || K < group || K % group || K > MOE_W4_MAX_K) return MOE_ERR_INVALID_ARG;
  return MOE_OK;
}

static dim3 w4_grid(int E, int N, int K) { return dim3((K + 127) / 128, (N + 15) / 16, E); }

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
  quant_w4_kernel<<<w4_grid(E, N, K), 128, 0, (cudaStream_t)stream>>>(W, N, K, group, Wp);
  return cudaGetLastError() == cudaSuccess ? MOE_OK : MOE_ERR_CUDA;
}

extern "C" int moe_pack_weights_w4(const uint8_t* codes, const uint16_t* scale, int E, int N, int K, int group,
                                   uint8_t* Wp, moe_stream_t stream) {
  if (!codes || !scale || !Wp || !aligned16(Wp) || ((uintptr_t)scale & 1)) return MOE_ERR_INVALID_ARG;
  const int rc = check_w4(E, N, K, group);
  if (rc) return rc;
  pack_w4_kernel<<<w4_grid(E, N, K), 64, 0, (cudaStream_t)stream>>>(codes, scale, N, K, group, Wp);
  return cudaGetLastError() == cudaSuccess ? MOE_OK : MOE_ERR_CUDA;
}

extern "C" int moe_dequant_weights_w4(const uint8_t* Wp, int E, int N, int K, int group, float* W,
                                      moe_stream_t stream) {
  if (!Wp || !W || !aligned16(Wp) || !aligned16(W)) return MOE_ERR_INVALID_ARG;
  const int rc = check_w4(E, N, K, group);
  if (rc) return rc;
  dequant_w4_kernel<<<w4_grid(E, N, K), 128, 0, (cudaStream_t)stream>>>(Wp, N, K, group, W);
  return cudaGetLastError() == cudaSuccess ? MOE_OK : MOE_ERR_CUDA;
}
