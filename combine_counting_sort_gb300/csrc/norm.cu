// norm.cu: layer norm over each row of [T, H], forward and backward.
//
//   n = (x - mean) * rstd,  rstd = 1 / sqrt(var + eps),  y = n * weight + bias
//   g = dy * weight,  dx = rstd * (g - mean(g) - n * mean(g * n))
//   dweight = sum_t dy * n,  dbias = sum_t dy
//
// Memory bound: forward reads x and writes y, backward reads x and dy and
// writes dx, once each.  A row lies in the registers of the threads that work
// on it, so mean and variance are taken in two passes over registers (no
// cancellation for rows far from zero) while memory is read once.  All sums
// are fp32, in a fixed order: results do not change from run to run.
#include "dtype.cuh"
#include "host_util.h"

namespace moe {

constexpr int kNormMaxH = MOE_NORM_MAX_H;

template <int TPR>
struct RowGroup {   // TPR threads of a block that work on one row
  static constexpr int kWarps = TPR / 32;
  // Sum of (a, b) over the group; every thread gets it.  `scratch` holds one
  // float2 per warp of the block; the caller alternates between two of them.
  static MOE_DEV float2 sum(float a, float b, float2* scratch) {
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) {
      a += __shfl_xor_sync(0xffffffffu, a, o);
      b += __shfl_xor_sync(0xffffffffu, b, o);
    }
    if (kWarps == 1) return make_float2(a, b);
    const int warp = threadIdx.x >> 5, first = (threadIdx.x / TPR) * kWarps;
    if ((threadIdx.x & 31) == 0) scratch[warp] = make_float2(a, b);
    if (TPR == (int)blockDim.x) __syncthreads();
    else asm volatile("bar.sync %0, %1;" ::"r"((int)(threadIdx.x / TPR) + 1), "n"(TPR) : "memory");
    a = b = 0.f;
    // every lane sums the warps' values in the same order
    const int lane = threadIdx.x & 31;
    if (lane < kWarps) { const float2 v = scratch[first + lane]; a = v.x; b = v.y; }
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) {
      a += __shfl_xor_sync(0xffffffffu, a, o);
      b += __shfl_xor_sync(0xffffffffu, b, o);
    }
    return make_float2(a, b);
  }
};

// weight or bias values j, .., j + V - 1 as fp32: the rows' type or fp32 (where
// V > 1, 16-byte aligned), `none` where there is no such tensor.
template <typename T, int V>
MOE_DEV void param(const void* p, bool f32, int j, float none, float* out) {
  if (!p) {
#pragma unroll
    for (int v = 0; v < V; ++v) out[v] = none;
  } else if (f32) {
    constexpr int L = V < 4 ? V : 4;
#pragma unroll
    for (int v = 0; v < V; v += L) {
      const Vec<float, L> a = *reinterpret_cast<const Vec<float, L>*>(static_cast<const float*>(p) + j + v);
#pragma unroll
      for (int i = 0; i < L; ++i) out[v + i] = a.v[i];
    }
  } else {
    const Vec<T, V> a = *reinterpret_cast<const Vec<T, V>*>(static_cast<const T*>(p) + j);
#pragma unroll
    for (int v = 0; v < V; ++v) out[v] = to_f32(a.v[v]);
  }
}

struct NormArgs {
  const void* x;
  const void* dy;
  const void* weight;
  const void* bias;
  bool wf32;
  int T, H;
  float eps;
  void* y;      // y, or dx
  float* mean;
  float* rstd;
  float* part;  // backward: [groups][2][H] sums of each group's rows
};

// ---------------------------------------------------------------- forward

// TPR threads a row, NV vectors of V values each: H <= TPR * NV * V.
template <typename T, int V, int NV, int TPR, int BLOCK>
__global__ void __launch_bounds__(BLOCK) norm_fwd_kernel(const NormArgs p) {
  using Vc = Vec<T, V>;
  __shared__ float2 scratch[2][BLOCK / 32];
  const int tid = threadIdx.x % TPR;
  const long long row = (long long)blockIdx.x * (BLOCK / TPR) + threadIdx.x / TPR;
  const bool live = row < p.T;
  const T* x = static_cast<const T*>(p.x) + (live ? row : 0) * p.H;
  Vc raw[NV];
  float s = 0.f;
#pragma unroll
  for (int i = 0; i < NV; ++i) {
    const int j = (i * TPR + tid) * V;
    if (j < p.H) raw[i] = *reinterpret_cast<const Vc*>(x + j);
  }
#pragma unroll
  for (int i = 0; i < NV; ++i)
    if ((i * TPR + tid) * V < p.H) {
#pragma unroll
      for (int v = 0; v < V; ++v) s += to_f32(raw[i].v[v]);
    }
  const float mean = RowGroup<TPR>::sum(s, 0.f, scratch[0]).x / (float)p.H;
  float q = 0.f;
#pragma unroll
  for (int i = 0; i < NV; ++i)
    if ((i * TPR + tid) * V < p.H) {
#pragma unroll
      for (int v = 0; v < V; ++v) {
        const float d = to_f32(raw[i].v[v]) - mean;
        q = fmaf(d, d, q);
      }
    }
  const float var = RowGroup<TPR>::sum(q, 0.f, scratch[1]).x / (float)p.H;
  const float rstd = 1.f / sqrtf(var + p.eps);
  if (!live) return;
  if (tid == 0) {
    if (p.mean) p.mean[row] = mean;
    if (p.rstd) p.rstd[row] = rstd;
  }
  T* y = static_cast<T*>(p.y) + row * p.H;
#pragma unroll
  for (int i = 0; i < NV; ++i) {
    const int j = (i * TPR + tid) * V;
    if (j < p.H) {
      float w[V], b[V];
      param<T, V>(p.weight, p.wf32, j, 1.f, w);
      param<T, V>(p.bias, p.wf32, j, 0.f, b);
      Vc o;
#pragma unroll
      for (int v = 0; v < V; ++v) o.v[v] = from_f32<T>(fmaf((to_f32(raw[i].v[v]) - mean) * rstd, w[v], b[v]));
      *reinterpret_cast<Vc*>(y + j) = o;
    }
  }
}

// ---------------------------------------------------------------- backward

// A group of TPR threads walks rows g, g + groups, ... and keeps its columns'
// sums for dweight and dbias in registers; the next row's loads are in flight
// while this one is worked on.
template <typename T, int V, int NV, int TPR, int BLOCK>
__global__ void __launch_bounds__(BLOCK) norm_bwd_kernel(const NormArgs p) {
  using Vc = Vec<T, V>;
  __shared__ float2 scratch[2][BLOCK / 32];
  const int tid = threadIdx.x % TPR;
  const int groups = gridDim.x * (BLOCK / TPR), g = blockIdx.x * (BLOCK / TPR) + threadIdx.x / TPR;
  const float inv = 1.f / (float)p.H;
  Vc rx[NV], rd[NV];
  float w[NV * V], dw[NV * V] = {}, db[NV * V] = {};
#pragma unroll
  for (int i = 0; i < NV; ++i)
    if ((i * TPR + tid) * V < p.H) param<T, V>(p.weight, p.wf32, (i * TPR + tid) * V, 1.f, w + i * V);
  auto load = [&](long long row) {
    const T* x = static_cast<const T*>(p.x) + row * p.H;
    const T* dy = static_cast<const T*>(p.dy) + row * p.H;
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      const int j = (i * TPR + tid) * V;
      if (j < p.H) {
        rx[i] = *reinterpret_cast<const Vc*>(x + j);
        rd[i] = *reinterpret_cast<const Vc*>(dy + j);
      }
    }
  };
  if (g < p.T) load(g);
  int turn = 0;
  for (long long row = g; row < p.T; row += groups, turn ^= 1) {
    const float mean = p.mean[row], rstd = p.rstd[row];
    Vc cx[NV], cd[NV];
#pragma unroll
    for (int i = 0; i < NV; ++i) { cx[i] = rx[i]; cd[i] = rd[i]; }
    if (row + groups < p.T) load(row + groups);
    float s1 = 0.f, s2 = 0.f;
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      const int j = (i * TPR + tid) * V;
      if (j < p.H) {
#pragma unroll
        for (int v = 0; v < V; ++v) {
          const float n = (to_f32(cx[i].v[v]) - mean) * rstd, d = to_f32(cd[i].v[v]);
          const float gr = d * w[i * V + v];
          s1 += gr;
          s2 = fmaf(gr, n, s2);
          dw[i * V + v] = fmaf(d, n, dw[i * V + v]);
          db[i * V + v] += d;
        }
      }
    }
    const float2 s = RowGroup<TPR>::sum(s1, s2, scratch[turn]);
    const float m1 = s.x * inv, m2 = s.y * inv;
    T* dx = static_cast<T*>(p.y) + row * p.H;
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      const int j = (i * TPR + tid) * V;
      if (j < p.H) {
        Vc o;
#pragma unroll
        for (int v = 0; v < V; ++v) {
          const float n = (to_f32(cx[i].v[v]) - mean) * rstd;
          const float gr = to_f32(cd[i].v[v]) * w[i * V + v];
          o.v[v] = from_f32<T>(rstd * (gr - m1 - n * m2));
        }
        *reinterpret_cast<Vc*>(dx + j) = o;
      }
    }
  }
  float* pw = p.part + (long long)g * 2 * p.H;
#pragma unroll
  for (int i = 0; i < NV; ++i)
#pragma unroll
    for (int v = 0; v < V; ++v) {
      const int j = (i * TPR + tid) * V + v;
      if (j < p.H) {
        pw[j] = dw[i * V + v];
        pw[p.H + j] = db[i * V + v];
      }
    }
}

// dweight (blockIdx.y 0) and dbias (1): the groups' sums added up.  A block
// takes 32 columns, its 16 warps every 16th group.
template <typename T>
__global__ void __launch_bounds__(512) norm_sums_kernel(const float* part, int groups, int H, bool wf32, void* dweight,
                                                        void* dbias) {
  __shared__ float acc[16][32];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int j = blockIdx.x * 32 + lane;
  void* out = blockIdx.y ? dbias : dweight;
  if (!out) return;
  float s = 0.f;
  if (j < H)
    for (int g = warp; g < groups; g += 16) s += part[((long long)g * 2 + blockIdx.y) * H + j];
  acc[warp][lane] = s;
  __syncthreads();
  if (warp == 0 && j < H) {
    s = 0.f;
#pragma unroll
    for (int w = 0; w < 16; ++w) s += acc[w][lane];
    if (wf32) static_cast<float*>(out)[j] = s;
    else static_cast<T*>(out)[j] = from_f32<T>(s);
  }
}

template <typename T, int V, int NV, int TPR>
int launch_fwd(const NormArgs& p, cudaStream_t st) {
  constexpr int BLOCK = TPR < 256 ? 256 : TPR;
  const long long blocks = ((long long)p.T + BLOCK / TPR - 1) / (BLOCK / TPR);
  norm_fwd_kernel<T, V, NV, TPR, BLOCK><<<(unsigned)blocks, BLOCK, 0, st>>>(p);
  return cudaGetLastError() == cudaSuccess ? MOE_OK : MOE_ERR_CUDA;
}

// E values a thread
template <typename T, int V, int E>
int fwd_of(const NormArgs& p, cudaStream_t st) {
  if (p.H <= 32 * E) return launch_fwd<T, V, E / V, 32>(p, st);
  if (p.H <= 128 * E) return launch_fwd<T, V, E / V, 128>(p, st);
  if (p.H <= 256 * E) return launch_fwd<T, V, E / V, 256>(p, st);
  return launch_fwd<T, V, E / V, 1024>(p, st);
}

template <typename T>
int fwd_typed(const NormArgs& p, bool vec, cudaStream_t st) {
  constexpr int V = kVec16<T>;
  if (!vec) return fwd_of<T, 1, 32>(p, st);
  // few rows: more threads a row, since one row's latency is the time
  if (p.T <= 2 * 152 && p.H <= 1024 * 8) return fwd_of<T, V, 8>(p, st);
  return fwd_of<T, V, 32>(p, st);
}

// Backward: threads a row by its length, 16 values a thread.
constexpr int kBwdE = 16;
inline int bwd_tpr(int H) { return H <= 32 * kBwdE ? 32 : H <= 128 * kBwdE ? 128 : H <= 512 * kBwdE ? 512 : 1024; }
inline int bwd_block(int tpr) { return tpr < 256 ? 256 : tpr; }

// Groups that walk the rows: a block or two for each SM, no more than rows.
inline long long bwd_blocks(int T, int H) {
  const int tpr = bwd_tpr(H), per = bwd_block(tpr) / tpr;
  return std::min<long long>(((long long)T + per - 1) / per, tpr >= 512 ? 152 : 304);
}

template <typename T, int V, int TPR>
int launch_bwd(const NormArgs& p, void* dweight, void* dbias, cudaStream_t st) {
  constexpr int BLOCK = TPR < 256 ? 256 : TPR;
  const int blocks = (int)bwd_blocks(p.T, p.H), groups = blocks * (BLOCK / TPR);
  norm_bwd_kernel<T, V, kBwdE / V, TPR, BLOCK><<<blocks, BLOCK, 0, st>>>(p);
  if (dweight || dbias)
    norm_sums_kernel<T><<<dim3((p.H + 31) / 32, 2), 512, 0, st>>>(p.part, groups, p.H, p.wf32, dweight, dbias);
  return cudaGetLastError() == cudaSuccess ? MOE_OK : MOE_ERR_CUDA;
}

template <typename T, int V>
int bwd_of(const NormArgs& p, void* dweight, void* dbias, cudaStream_t st) {
  switch (bwd_tpr(p.H)) {
    case 32: return launch_bwd<T, V, 32>(p, dweight, dbias, st);
    case 128: return launch_bwd<T, V, 128>(p, dweight, dbias, st);
    case 512: return launch_bwd<T, V, 512>(p, dweight, dbias, st);
    default: return launch_bwd<T, V, 1024>(p, dweight, dbias, st);
  }
}

inline size_t elem_bytes(int dtype) { return dtype == MOE_F32 ? 4 : 2; }

inline bool norm_shape_ok(int T, int H) { return T >= 0 && H >= 1 && H <= kNormMaxH; }

// a tensor of this type starts where its elements may start
inline bool elem_aligned(const void* p, int dtype) { return (uintptr_t)p % elem_bytes(dtype) == 0; }

}  // namespace moe

using namespace moe;

extern "C" int moe_layernorm(const void* x, int T, int H, int dtype, const void* weight, const void* bias, int wdtype, float eps,
                             void* y, float* mean, float* rstd, moe_stream_t stream) {
  if (!norm_shape_ok(T, H) || dtype < MOE_BF16 || dtype > MOE_F32 || (wdtype != dtype && wdtype != MOE_F32) || !(eps >= 0.f))
    return MOE_ERR_INVALID_ARG;
  if (T == 0) return MOE_OK;
  if (!x || !y) return MOE_ERR_INVALID_ARG;
  if (!elem_aligned(x, dtype) || !elem_aligned(y, dtype) || !elem_aligned(weight, wdtype) || !elem_aligned(bias, wdtype) ||
      !elem_aligned(mean, MOE_F32) || !elem_aligned(rstd, MOE_F32))
    return MOE_ERR_INVALID_ARG;
  NormArgs p = {x, nullptr, weight, bias, wdtype == MOE_F32, T, H, eps, y, mean, rstd, nullptr};
  const bool vec = aligned16(x) && aligned16(y) && aligned16(weight) && aligned16(bias) && (H * elem_bytes(dtype)) % 16 == 0;
  cudaStream_t st = (cudaStream_t)stream;
  if (dtype == MOE_BF16) return fwd_typed<__nv_bfloat16>(p, vec, st);
  if (dtype == MOE_F16) return fwd_typed<__half>(p, vec, st);
  return fwd_typed<float>(p, vec, st);
}

extern "C" int moe_layernorm_bwd_ws_bytes(int T, int H, size_t* bytes) {
  if (!bytes || !norm_shape_ok(T, H)) return MOE_ERR_INVALID_ARG;
  const int tpr = bwd_tpr(H);
  *bytes = (size_t)bwd_blocks(T, H) * (bwd_block(tpr) / tpr) * 2 * H * sizeof(float);
  return MOE_OK;
}

extern "C" int moe_layernorm_bwd(const void* dy, const void* x, int T, int H, int dtype, const void* weight, int wdtype,
                                 const float* mean, const float* rstd, void* dx, void* dweight, void* dbias, void* ws,
                                 size_t ws_bytes, moe_stream_t stream) {
  if (!norm_shape_ok(T, H) || dtype < MOE_BF16 || dtype > MOE_F32 || (wdtype != dtype && wdtype != MOE_F32)) return MOE_ERR_INVALID_ARG;
  if (!elem_aligned(weight, wdtype) || !elem_aligned(dweight, wdtype) || !elem_aligned(dbias, wdtype)) return MOE_ERR_INVALID_ARG;
  cudaStream_t st = (cudaStream_t)stream;
  if (T == 0) {   // sums over no rows
    if (dweight && cudaMemsetAsync(dweight, 0, H * elem_bytes(wdtype), st) != cudaSuccess) return MOE_ERR_CUDA;
    if (dbias && cudaMemsetAsync(dbias, 0, H * elem_bytes(wdtype), st) != cudaSuccess) return MOE_ERR_CUDA;
    return MOE_OK;
  }
  size_t need = 0;
  moe_layernorm_bwd_ws_bytes(T, H, &need);
  if (!dy || !x || !mean || !rstd || !dx || !ws || ws_bytes < need) return MOE_ERR_INVALID_ARG;
  if (!elem_aligned(x, dtype) || !elem_aligned(dy, dtype) || !elem_aligned(dx, dtype) || !elem_aligned(mean, MOE_F32) ||
      !elem_aligned(rstd, MOE_F32) || !aligned16(ws))
    return MOE_ERR_INVALID_ARG;
  NormArgs p = {x, dy, weight, nullptr, wdtype == MOE_F32, T, H, 0.f, dx, const_cast<float*>(mean), const_cast<float*>(rstd),
                static_cast<float*>(ws)};
  const bool vec = aligned16(x) && aligned16(dy) && aligned16(dx) && aligned16(weight) && (H * elem_bytes(dtype)) % 16 == 0;
  if (dtype == MOE_BF16)
    return vec ? bwd_of<__nv_bfloat16, 8>(p, dweight, dbias, st) : bwd_of<__nv_bfloat16, 1>(p, dweight, dbias, st);
  if (dtype == MOE_F16) return vec ? bwd_of<__half, 8>(p, dweight, dbias, st) : bwd_of<__half, 1>(p, dweight, dbias, st);
  return vec ? bwd_of<float, 4>(p, dweight, dbias, st) : bwd_of<float, 1>(p, dweight, dbias, st);
}
