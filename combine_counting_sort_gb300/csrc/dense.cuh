// dense.cuh: 16-bit matrix products on tcgen05 for the dense operators beside
// the experts, with the operators' arithmetic in their epilogues.
//
//   out[i][j] = sum_k P[i][k] * Q[j][k],  fp32 accumulation in tensor memory
//
// Either operand may lie in memory with k contiguous ("K-major") or with i (or
// j) contiguous ("MN-major"): the tensor core reads both from shared memory, so
// the backward products d W and d^T x need no transposed copies.
//
//   linear  out = act(sum + bias) + residual, and act' beside it
//   gated   Q holds gate rows and up rows: out = act(gate sum) * up sum, and
//           the two factors of the backward pass beside it
//   plain   out = sum (the backward products)
//
// Two kernels share these pieces: dense_pair.cuh (256 x 256 tiles on CTA
// pairs, for many rows) and dense_few.cuh (128 of j against few i, the
// contraction split over a cluster).
#pragma once

#include <type_traits>

#include "dtype.cuh"
#include "tmem_drain.cuh"

namespace moe {

enum { kEpiPlain = 0, kEpiLinear = 1, kEpiGated = 2 };

constexpr int kDenseBK = 64;                     // contraction per stage: 128 bytes, one swizzle row
constexpr uint32_t kDenseChunk = 64 * 128;       // 64 rows (or 64 k) of 128 bytes

struct DenseArgs {
  int I, J, K;             // J: columns of out (gated: F)
  void* out;               // [I][J], 16-bit
  const void* bias;        // [J] or null
  const void* residual;    // [I][J] or null
  void* aux;               // slope [I][J], gated factors [I][2 J], or null
  int act;
  int vec;                 // out, residual and aux take 16-byte vectors
  int bias_vec;            // bias too
  int32_t* status;
  uint64_t timeout_ns;
};

// ---------------------------------------------------------------- descriptors and MMA

// kind::f16: fp32 D (bits 4-5 = 1), A and B f16 (0) or bf16 (1) in bits 7-9 and
// 10-12, their majors in bits 15 and 16 (1: MN-major), N >> 3 in bits 17-22, M >> 4
// in bits 24-28.
template <typename T>
constexpr uint32_t idesc_f16(int M, int N, bool a_mn, bool b_mn) {
  const uint32_t f = std::is_same<T, __nv_bfloat16>::value ? 1u : 0u;
  return (1u << 4) | (f << 7) | (f << 10) | ((a_mn ? 1u : 0u) << 15) | ((b_mn ? 1u : 0u) << 16) |
         ((uint32_t)(N >> 3) << 17) | ((uint32_t)(M >> 4) << 24);
}

// Shared-memory descriptor of k16 (16 values of k) of an operand tile at `base`.
// K-major: rows of 128 bytes, swizzled in atoms of 8 rows; k16 starts 32 bytes on.
// MN-major: chunks of 64 rows i, each 64 k of 128 bytes; 8 k make an atom of 1024
// bytes (the stride offset), the next 64 rows lie a chunk on (the leading offset).
template <bool MN>
MOE_DEV uint64_t operand_desc(uint32_t base, int k16) {
  if (!MN) return sw128_kmajor_desc(base + k16 * 32);
  return (uint64_t)(((base + k16 * 2048) & 0x3FFFFu) >> 4) | ((uint64_t)(kDenseChunk >> 4) << 16) | ((uint64_t)(1024 >> 4) << 32) |
         ((uint64_t)1 << 46) | ((uint64_t)2 << 61);
}

MOE_DEV void umma_f16(uint32_t d_tmem, uint64_t adesc, uint64_t bdesc, uint32_t idesc, uint32_t accumulate) {
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "setp.ne.b32 p, %4, 0;\n\t"
      "tcgen05.mma.cta_group::1.kind::f16 [%0], %1, %2, %3, p;\n\t}"
      :: "r"(d_tmem), "l"(adesc), "l"(bdesc), "r"(idesc), "r"(accumulate) : "memory");
}

MOE_DEV void umma_f16_pair(uint32_t d_tmem, uint64_t adesc, uint64_t bdesc, uint32_t idesc, uint32_t accumulate) {
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "setp.ne.b32 p, %4, 0;\n\t"
      "tcgen05.mma.cta_group::2.kind::f16 [%0], %1, %2, %3, p;\n\t}"
      :: "r"(d_tmem), "l"(adesc), "l"(bdesc), "r"(idesc), "r"(accumulate) : "memory");
}

// ---------------------------------------------------------------- activations

// act(a) and act'(a) in fp32.
template <int ACT>
MOE_DEV float2 act_slope(float a) {
  if (ACT == MOE_ACT_RELU) return make_float2(a < 0.f ? 0.f : a, a > 0.f ? 1.f : 0.f);
  if (ACT == MOE_ACT_SILU) {
    const float s = __fdividef(1.f, 1.f + __expf(-a));
    return make_float2(a * s, s * (1.f + a * (1.f - s)));
  }
  if (ACT == MOE_ACT_GELU) {   // erfc: no cancellation for a far below zero
    const float cdf = 0.5f * erfcf(-0.70710678f * a);
    return make_float2(a * cdf, cdf + a * (0.39894228f * __expf(-0.5f * a * a)));
  }
  if (ACT == MOE_ACT_GELU_TANH) {   // (1 + tanh z) / 2 = 1 / (1 + exp(-2 z))
    const float z2 = 1.5957691f * a * fmaf(0.044715f * a, a, 1.f);
    const float s = __fdividef(1.f, 1.f + __expf(-z2)), r = 1.f - s;
    return make_float2(a * s, s + (r > 0.f ? a * s * r * (1.5957691f * fmaf(0.134145f * a, a, 1.f)) : 0.f));
  }
  return make_float2(a, 1.f);
}

template <int ACT>
struct ActTag {
  static constexpr int value = ACT;
};

// f(ActTag<act>): one branch outside the loops over elements.
template <typename F>
MOE_DEV void with_act(int act, F&& f) {
  switch (act) {
    case MOE_ACT_RELU: f(ActTag<MOE_ACT_RELU>()); break;
    case MOE_ACT_SILU: f(ActTag<MOE_ACT_SILU>()); break;
    case MOE_ACT_GELU: f(ActTag<MOE_ACT_GELU>()); break;
    case MOE_ACT_GELU_TANH: f(ActTag<MOE_ACT_GELU_TANH>()); break;
    default: f(ActTag<MOE_ACT_NONE>()); break;
  }
}

// ---------------------------------------------------------------- 32 x 32 blocks between registers and rows
//
// A warp reads its accumulators with lane l holding 32 columns of row i0 + l.  Stored
// like that, one access would touch 32 rows for 16 bytes each; so a block goes through
// 4 KB of shared memory of the warp's own, and each access covers whole sectors of
// few rows: with vectors 64 bytes of 8 rows, and where no vector fits (an odd row
// length, an unaligned start) 32 neighbouring values of one row.  Chunks of 16 bytes
// are swizzled so that neither side meets a bank twice.

constexpr uint32_t kBlockBytes = 32 * 32 * 4;

// The block rounded to T, to rows of `out`.
template <typename T>
MOE_DEV void store_block(const float (&v)[32], T* out, long long ld, int i0, int j0, int I, int J, bool vec, uint8_t* stage) {
  const int lane = threadIdx.x & 31;
  __syncwarp();   // the last block has left the stage
#pragma unroll
  for (int c = 0; c < 4; ++c) {
    Vec<T, 8> o;
#pragma unroll
    for (int e = 0; e < 8; ++e) o.v[e] = from_f32<T>(v[8 * c + e]);
    *reinterpret_cast<Vec<T, 8>*>(stage + lane * 64 + ((c ^ (lane >> 1)) & 3) * 16) = o;
  }
  __syncwarp();
  if (vec) {
    const int c = lane & 3;
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      const int r = 8 * k + (lane >> 2);
      if (i0 + r < I && j0 + 8 * c < J)
        *reinterpret_cast<uint4*>(out + (long long)(i0 + r) * ld + j0 + 8 * c) =
            *reinterpret_cast<const uint4*>(stage + r * 64 + ((c ^ (r >> 1)) & 3) * 16);
    }
  } else if (j0 + lane < J) {
    const int rows = min(32, I - i0);
#pragma unroll 8
    for (int r = 0; r < rows; ++r)
      out[(long long)(i0 + r) * ld + j0 + lane] =
          *reinterpret_cast<const T*>(stage + r * 64 + (((lane >> 3) ^ (r >> 1)) & 3) * 16 + (lane & 7) * 2);
  }
}

// act(block + bias) + residual to rows of g.out, and act' to rows of g.aux.  The
// arithmetic is done where the columns lie beside one another, so bias and residual are
// read in whole sectors too; `pre` holds them, fetched ahead (vectors only).
template <typename T>
struct LinearAhead {
  Vec<T, 8> bias, res[4];
};

template <typename T>
MOE_DEV void linear_fetch(LinearAhead<T>& pre, const DenseArgs& g, int i0, int j0) {
  const int lane = threadIdx.x & 31, j = j0 + 8 * (lane & 3);
  if (!g.vec || j >= g.J) return;
  if (g.bias && g.bias_vec) pre.bias = *reinterpret_cast<const Vec<T, 8>*>(static_cast<const T*>(g.bias) + j);
  if (g.residual)
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      const int i = i0 + 8 * k + (lane >> 2);
      if (i < g.I) pre.res[k] = *reinterpret_cast<const Vec<T, 8>*>(static_cast<const T*>(g.residual) + (long long)i * g.J + j);
    }
}

template <typename T>
MOE_DEV void linear_block(const float (&v)[32], const LinearAhead<T>& pre, const DenseArgs& g, int i0, int j0, uint8_t* stage) {
  const int lane = threadIdx.x & 31;
  T* out = static_cast<T*>(g.out);
  T* aux = static_cast<T*>(g.aux);
  const T* bias = static_cast<const T*>(g.bias);
  const T* residual = static_cast<const T*>(g.residual);
  __syncwarp();
#pragma unroll
  for (int c = 0; c < 8; ++c)
    *reinterpret_cast<float4*>(stage + lane * 128 + ((c ^ lane) & 7) * 16) = make_float4(v[4 * c], v[4 * c + 1], v[4 * c + 2], v[4 * c + 3]);
  __syncwarp();
  if (g.vec) {
    const int c = lane & 3, j = j0 + 8 * c;
    if (j >= g.J) return;
    float b[8];
#pragma unroll
    for (int e = 0; e < 8; ++e) b[e] = !bias ? 0.f : to_f32(g.bias_vec ? pre.bias.v[e] : bias[j + e]);
    with_act(g.act, [&](auto act) {
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        const int r = 8 * k + (lane >> 2), i = i0 + r;
        if (i >= g.I) continue;
        const float4 lo = *reinterpret_cast<const float4*>(stage + r * 128 + (((2 * c) ^ r) & 7) * 16);
        const float4 hi = *reinterpret_cast<const float4*>(stage + r * 128 + (((2 * c + 1) ^ r) & 7) * 16);
        const float a[8] = {lo.x, lo.y, lo.z, lo.w, hi.x, hi.y, hi.z, hi.w};
        const long long at = (long long)i * g.J + j;
        Vec<T, 8> y, s;
#pragma unroll
        for (int e = 0; e < 8; ++e) {
          const float2 f = act_slope<decltype(act)::value>(a[e] + b[e]);
          s.v[e] = from_f32<T>(f.y);
          y.v[e] = from_f32<T>(residual ? f.x + to_f32(pre.res[k].v[e]) : f.x);
        }
        if (aux) *reinterpret_cast<Vec<T, 8>*>(aux + at) = s;
        *reinterpret_cast<Vec<T, 8>*>(out + at) = y;
      }
    });
  } else {
    const int j = j0 + lane, rows = min(32, g.I - i0);
    if (j >= g.J) return;
    const float b = bias ? to_f32(bias[j]) : 0.f;
    with_act(g.act, [&](auto act) {
#pragma unroll 8
      for (int r = 0; r < rows; ++r) {
        const float a = *reinterpret_cast<const float*>(stage + r * 128 + (((lane >> 2) ^ r) & 7) * 16 + (lane & 3) * 4);
        const long long at = (long long)(i0 + r) * g.J + j;
        const float2 f = act_slope<decltype(act)::value>(a + b);
        if (aux) aux[at] = from_f32<T>(f.y);
        out[at] = from_f32<T>(residual ? f.x + to_f32(residual[at]) : f.x);
      }
    });
  }
}

}  // namespace moe
