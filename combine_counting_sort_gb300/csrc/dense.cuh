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

// act(a) and act'(a) in fp32, two values at a time.
//   silu       s = 1 / (1 + exp(-a)):  a s,  s + a s (1 - s)
//   gelu_tanh  (1 + tanh z) / 2 = 1 / (1 + exp(-2 z)) = s, 2 z = c a (1 + 0.044715 a^2):  a s,  s + a s (1 - s) (2 z)'
//   gelu       the normal distribution's tail q(|a|) = exp(-a^2 / 2) t (c1 + t (c2 + ...)), t = 1 / (1 + 0.36 |a|): seven
//              terms, least largest error of the ratio over |a| <= 14 (2^-20, so small values far below zero
//              keep their digits); the density comes of the same exponential
// One exponential and one reciprocal each, both by the approximate instructions (2^-22 of
// the value): 8 issue cycles each for a warp, so they bound the epilogue's arithmetic.
MOE_DEV float ex2(float v) { float r; asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(v)); return r; }
MOE_DEV float rcp(float v) { float r; asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(v)); return r; }
MOE_DEV f32x2 ex2_pair(f32x2 v) { return pack_f32x2(ex2(lo2(v)), ex2(hi2(v))); }
MOE_DEV f32x2 rcp_pair(f32x2 v) { return pack_f32x2(rcp(lo2(v)), rcp(hi2(v))); }

template <int ACT>
MOE_DEV void act_pair(f32x2 a, f32x2& y, f32x2& slope) {
  constexpr float kLog2e = 1.44269504f;
  const f32x2 one = both(1.f);
  if (ACT == MOE_ACT_RELU) {
    const float l = lo2(a), h = hi2(a);
    const float yl = l < 0.f ? 0.f : l, yh = h < 0.f ? 0.f : h;   // (a NaN stays, in the slope too)
    y = pack_f32x2(yl, yh);
    slope = pack_f32x2(l > 0.f ? 1.f : yl, h > 0.f ? 1.f : yh);
  } else if (ACT == MOE_ACT_SILU) {
    const f32x2 s = rcp_pair(add2(ex2_pair(mul2(a, both(-kLog2e))), one));
    y = mul2(a, s);
    slope = fma2(y, fma2(s, both(-1.f), one), s);
  } else if (ACT == MOE_ACT_GELU_TANH) {
    constexpr float c = 1.59576912f, d = 0.044715f * c;   // 2 sqrt(2 / pi)
    const f32x2 a2 = mul2(a, a);
    const f32x2 s = rcp_pair(add2(ex2_pair(mul2(a, fma2(a2, both(-d * kLog2e), both(-c * kLog2e)))), one));
    y = mul2(a, s);
    // (a^2 kept finite: where it overflows, 1 - s is 0 long since, and 0 times infinity is no slope)
    const f32x2 b2 = pack_f32x2(fminf(lo2(a2), 1e30f), fminf(hi2(a2), 1e30f));
    slope = fma2(mul2(y, fma2(s, both(-1.f), one)), fma2(b2, both(3.f * d), both(c)), s);
  } else if (ACT == MOE_ACT_GELU) {
    const f32x2 b = pack_f32x2(fabsf(lo2(a)), fabsf(hi2(a)));
    const f32x2 e = ex2_pair(mul2(mul2(a, a), both(-0.5f * kLog2e)));
    const f32x2 t = rcp_pair(fma2(b, both(0.36f), one));
    f32x2 q = fma2(t, both(0.0470560688f), both(-0.179763952f));
    q = fma2(q, t, both(0.180953031f));
    q = fma2(q, t, both(0.0265499758f));
    q = fma2(q, t, both(0.13971904f));
    q = fma2(q, t, both(0.141772491f));
    q = fma2(q, t, both(0.143713043f));
    q = mul2(mul2(q, t), e);
    const f32x2 p = fma2(q, both(-1.f), one);
    const f32x2 cdf = pack_f32x2(lo2(a) < 0.f ? lo2(q) : lo2(p), hi2(a) < 0.f ? hi2(q) : hi2(p));
    y = mul2(a, cdf);
    slope = fma2(mul2(a, e), both(0.39894228f), cdf);
  } else {
    y = a;
    slope = one;
  }
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

MOE_DEV void prefetch_l2(const void* p) { asm volatile("prefetch.global.L2 [%0];" ::"l"(p)); }

// ---------------------------------------------------------------- 32 x 32 blocks between registers and rows
//
// A warp holds its accumulators with lane l having 32 columns of row i0 + l, and works
// on them there.  Moved like that, one access would touch 32 rows for 16 bytes each; so
// blocks go, in the type's 16 bits, through 2 KB of shared memory, and each access covers
// whole sectors of few rows: with vectors 64 bytes of 8 rows, and where no vector fits (an
// odd row length, an unaligned start) 32 neighbouring values of one row.  Chunks of
// 16 bytes are swizzled so that neither side meets a bank twice.  (Working on the block
// where its columns lie beside one another, through fp32 in shared memory: 36 us against
// 21 for 4096 x 7168 x 512.)

constexpr uint32_t kBlockBytes = 32 * 64;

// where chunk c (8 columns) of row r is
MOE_DEV uint32_t block_at(int r, int c) { return (uint32_t)(r * 64 + ((c ^ (r >> 1)) & 3) * 16); }

// 32 columns of this lane's accumulator row, in pairs
MOE_DEV void drain_block(uint32_t taddr, f32x2 (&v)[16]) {
  float f[32];
  tmem_drain32(taddr, f);
#pragma unroll
  for (int e = 0; e < 16; ++e) v[e] = pack_f32x2(f[2 * e], f[2 * e + 1]);
}

// A block from its stage to rows that start anywhere: 16-byte stores between a row's first and last boundary,
// the values of each out of the two vectors of the stage that hold them; the eight values beside them one
// by one.  (12 stores instead of the 32 of a value a lane, which take some 6 cycles each.)  Not inlined: beside
// it the stores of whole vectors took 36 us instead of 30 at 4096 x 7168 x 512.
template <typename T>
__device__ __noinline__ void store_odd_block(T* out, long long ld, int i0, int j0, int I, int J, const uint8_t* stage) {
  const int lane = threadIdx.x & 31;
  if (j0 + 32 <= J) {
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      const int r = 8 * k + (lane >> 2), c = lane & 3;
      T* row = out + (long long)(i0 + r) * ld + j0;
      const int head = (8 - vector_offset(row)) & 7;
      if (i0 + r < I && (head == 0 || c < 3)) {
        const uint4 lo = *reinterpret_cast<const uint4*>(stage + block_at(r, c)), hi = *reinterpret_cast<const uint4*>(stage + block_at(r, (c + 1) & 3));
        *reinterpret_cast<uint4*>(row + head + 8 * c) = shifted8(lo, hi, head);
      }
    }
    T edge[8];
#pragma unroll
    for (int k = 0; k < 8; ++k) {
      const int r = 4 * k + (lane >> 3), q = lane & 7;
      const int head = (8 - vector_offset(out + (long long)(i0 + r) * ld + j0)) & 7, col = q < head ? q : 24 + q;
      edge[k] = *reinterpret_cast<const T*>(stage + block_at(r, col >> 3) + (col & 7) * 2);
    }
#pragma unroll
    for (int k = 0; k < 8; ++k) {
      const int r = 4 * k + (lane >> 3), q = lane & 7;
      T* row = out + (long long)(i0 + r) * ld + j0;
      const int head = (8 - vector_offset(row)) & 7;
      if (i0 + r < I && head) row[q < head ? q : 24 + q] = edge[k];
    }
  } else if (j0 + lane < J) {
#pragma unroll
    for (int k = 0; k < 32; k += 8) {   // eight rows read before they are written: the compiler may not swap the two
      T v[8];
#pragma unroll
      for (int r = 0; r < 8; ++r) v[r] = *reinterpret_cast<const T*>(stage + block_at(k + r, lane >> 3) + (lane & 7) * 2);
#pragma unroll
      for (int r = 0; r < 8; ++r)
        if (i0 + k + r < I) out[(long long)(i0 + k + r) * ld + j0 + lane] = v[r];
    }
  }
}

// The block rounded to T, to rows of `out`.
template <typename T>
MOE_DEV void store_block(const f32x2 (&v)[16], T* out, long long ld, int i0, int j0, int I, int J, bool vec, uint8_t* stage) {
  const int lane = threadIdx.x & 31;
  __syncwarp();   // the last block has left the stage
#pragma unroll
  for (int c = 0; c < 4; ++c) *reinterpret_cast<uint4*>(stage + block_at(lane, c)) = Pairs<T>::put(v + 4 * c);
  __syncwarp();
  if (vec) {
    const int c = lane & 3;
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      const int r = 8 * k + (lane >> 2);
      if (i0 + r < I && j0 + 8 * c < J)
        *reinterpret_cast<uint4*>(out + (long long)(i0 + r) * ld + j0 + 8 * c) = *reinterpret_cast<const uint4*>(stage + block_at(r, c));
    }
  } else {
    store_odd_block(out, ld, i0, j0, I, J, stage);
  }
}

// A block's residual as its rows lie: 16 bytes of rows 8 k + lane / 4, fetched ahead of its use.  Rows
// that start anywhere are asked for in L2 then, and loaded where they are used.
struct ResidualAhead {
  uint4 v[4];
};

template <typename T>
MOE_DEV void fetch_residual(ResidualAhead& a, const DenseArgs& g, int i0, int j0) {
  const int lane = threadIdx.x & 31;
  if (!g.residual || j0 >= g.J) return;
  const T* p = static_cast<const T*>(g.residual) + (long long)i0 * g.J + j0;
  if (g.vec) {
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      const int r = 8 * k + (lane >> 2), c = 8 * (lane & 3);
      if (i0 + r < g.I && j0 + c < g.J) a.v[k] = *reinterpret_cast<const uint4*>(p + (long long)r * g.J + c);
    }
  } else if (i0 + lane < g.I) {
    const T* row = p + (long long)lane * g.J;
    prefetch_l2(row);
    prefetch_l2(row + min(32, g.J - j0) - 1);
  }
}

// 32 columns of the accumulator plus their bias, which every lane reads whole (from L1 but for a
// tile's first rows) while the accumulator comes.
template <typename T>
MOE_DEV void drain_biased(uint32_t taddr, f32x2 (&v)[16], const DenseArgs& g, int j0) {
  const T* bias = static_cast<const T*>(g.bias) + j0;
  if (g.bias && g.bias_vec && j0 + 32 <= g.J) {
    uint4 b[4];
#pragma unroll
    for (int c = 0; c < 4; ++c) b[c] = reinterpret_cast<const uint4*>(bias)[c];
    drain_block(taddr, v);
#pragma unroll
    for (int c = 0; c < 4; ++c) {
      f32x2 f[4];
      Pairs<T>::get(b[c], f);
#pragma unroll
      for (int e = 0; e < 4; ++e) v[4 * c + e] = add2(v[4 * c + e], f[e]);
    }
  } else {
    drain_block(taddr, v);
    if (g.bias)
#pragma unroll
      for (int c = 0; c < 16; ++c) {
        const int n = g.J - j0 - 2 * c;
        v[c] = add2(v[c], pack_f32x2(n > 0 ? to_f32(bias[2 * c]) : 0.f, n > 1 ? to_f32(bias[2 * c + 1]) : 0.f));
      }
  }
}

// The residual's block into shared memory, and from there to the lanes of its rows.  (Rows that start
// anywhere: not inlined either.)
static __device__ __noinline__ void put_odd_residual(const uint16_t* p, int i0, int j0, int I, int J, uint8_t* stage) {
  const int lane = threadIdx.x & 31, c = lane & 3;
  const long long total = (long long)I * J, at = (long long)(i0 + (lane >> 2)) * J + j0 + 8 * c;
  const auto there = [&](int k) { return i0 + 8 * k + (lane >> 2) < I && j0 + 8 * c < J; };
  Unaligned u[4] = {};
#pragma unroll
  for (int k = 0; k < 4; ++k) load_unaligned(u[k], p, at + 8LL * k * J, total, there(k));
#pragma unroll
  for (int k = 0; k < 4; ++k)
    if (there(k)) *reinterpret_cast<uint4*>(stage + block_at(8 * k + (lane >> 2), c)) = shifted(u[k], p, at + 8LL * k * J, total);
}

MOE_DEV void put_residual(const ResidualAhead& a, const DenseArgs& g, int i0, int j0, uint8_t* stage) {
  const int lane = threadIdx.x & 31;
  if (g.vec) {
#pragma unroll
    for (int k = 0; k < 4; ++k) *reinterpret_cast<uint4*>(stage + block_at(8 * k + (lane >> 2), lane & 3)) = a.v[k];
  } else {
    put_odd_residual(static_cast<const uint16_t*>(g.residual), i0, j0, g.I, g.J, stage);
  }
}

template <typename T>
MOE_DEV void add_residual(f32x2 (&v)[16], const uint8_t* stage) {
  const int lane = threadIdx.x & 31;
  __syncwarp();
#pragma unroll
  for (int c = 0; c < 4; ++c) {
    f32x2 r[4];
    Pairs<T>::get(*reinterpret_cast<const uint4*>(stage + block_at(lane, c)), r);
#pragma unroll
    for (int e = 0; e < 4; ++e) v[4 * c + e] = add2(v[4 * c + e], r[e]);
  }
  __syncwarp();
}

}  // namespace moe
