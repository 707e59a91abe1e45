// norm_bwd.cu: layer norm's backward pass.
//
//   n = (x - mean) * rstd,  g = dy * weight
//   dx = rstd * (g - mean_H(g) - n * mean_H(g * n)),  dweight = sum_t dy * n,  dbias = sum_t dy
//
// Memory bound: reads x and dy and writes dx once.  One block an SM walks the
// rows; each thread keeps its columns' sums for dweight and dbias in registers
// over all of its rows.  Blocks write those sums to the workspace (2 H fp32 each,
// 152 of them: 2% of the rows' bytes at 8192 rows), and a second kernel adds
// them up in the blocks' order: no atomics, the same result every time.
#include "norm.cuh"

namespace moe {

// B rows at a time: their loads, their products and above all the exchanges between
// warps overlap.
template <typename T, typename W, int TPR, int NV, int B, int D, bool MASK>
__global__ void __launch_bounds__(kNormThreads, 1) norm_bwd_kernel(const NormArgs p) {
  constexpr int V = kVec16<T>, P = V / 2, WARPS = TPR / 32, GROUPS = kNormThreads / TPR;
  extern __shared__ uint8_t ring[];   // [D][B][x, dy][NV][threads] vectors, then the weights
  __shared__ float2 stats[2][B][kNormThreads / 32];
  const int grp = (int)threadIdx.x / TPR, lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const long long groups = (long long)gridDim.x * GROUPS, g = (long long)blockIdx.x * GROUPS + grp;
  const RowPart<T, TPR, NV, MASK> part(p.H, g);
  constexpr uint32_t STEP = kNormThreads * 16, HALF = NV * STEP, ROW = 2 * HALF, SLOT = B * ROW;
  uint8_t* mine = ring + threadIdx.x * 16;
  const uint32_t mine_at = smem_u32(mine);
  const long long stride = groups * p.H;
  long long at = g * p.H + part.first, next_row = g;   // the next row to fetch, and its vector 0
  const T *x = static_cast<const T*>(p.x), *dy = static_cast<const T*>(p.dy);
  T* dst = static_cast<T*>(p.y) + at;
  auto fetch = [&](int slot) {
#pragma unroll
    for (int r = 0; r < B; ++r) {
      if (next_row < p.T) {
        part.fetch(x + at, next_row == p.T - 1, mine_at + slot * SLOT + r * ROW, STEP);
        part.fetch(dy + at, next_row == p.T - 1, mine_at + slot * SLOT + r * ROW + HALF, STEP);
      }
      next_row += groups;
      at += stride;
    }
    cp_async_commit();
  };
#pragma unroll
  for (int d = 0; d < D - 1; ++d) fetch(d);
  W* const ws = reinterpret_cast<W*>(ring + D * SLOT);
  ParamVec<T, W> w[MASK ? NV : 1];
  if (MASK) {
#pragma unroll
    for (int i = 0; i < NV; ++i) w[i] = part.template params<W>(p.weight, 1.f, i);
  } else {
    copy_params(ws, p.weight, 1.f, p.H);
    __syncthreads();
  }
  f32x2 dw[NV][P], db[NV][P];
#pragma unroll
  for (int i = 0; i < NV; ++i)
#pragma unroll
    for (int e = 0; e < P; ++e) dw[i][e] = db[i][e] = 0;
  const float inv_h = 1.f / (float)p.H;
  float mean[B], rstd[B];
#pragma unroll
  for (int r = 0; r < B; ++r) {
    const long long row = g + r * groups;
    mean[r] = row < p.T ? p.mean[row] : 0.f;
    rstd[r] = row < p.T ? p.rstd[row] : 0.f;
  }

  int slot = 0, turn = 0;
  for (long long row = g; row < p.T; row += B * groups, turn ^= 1) {
    float mean_next[B], rstd_next[B];
#pragma unroll
    for (int r = 0; r < B; ++r) {
      const long long n = row + (B + r) * groups;
      mean_next[r] = n < p.T ? p.mean[n] : 0.f;
      rstd_next[r] = n < p.T ? p.rstd[n] : 0.f;
    }
    cp_async_wait<D - 2>();
    f32x2 dev[B][NV][P], gr[B][NV][P], s1[B], s2[B];
#pragma unroll
    for (int r = 0; r < B; ++r) s1[r] = s2[r] = 0;
#pragma unroll
    for (int i = 0; i < NV; ++i)
      if (part.any(i)) {
        f32x2 wp[P];
        if (MASK) w[i].get(wp);
        else reinterpret_cast<const ParamVec<T, W>*>(ws + part.col(i))->get(wp);
#pragma unroll
        for (int r = 0; r < B; ++r) {
          if (r && row + r * groups >= p.T) continue;   // the whole group
          f32x2 d[P];
          const f32x2 r2 = both(rstd[r]);
          const uint8_t* at_row = mine + slot * SLOT + r * ROW + i * STEP;
          Pairs<T>::get(*reinterpret_cast<const uint4*>(at_row), dev[r][i]);
          Pairs<T>::get(*reinterpret_cast<const uint4*>(at_row + HALF), d);
#pragma unroll
          for (int e = 0; e < P; ++e) dev[r][i][e] = add2(dev[r][i][e], both(-mean[r]));
          if (MASK) {
            part.mask(i, dev[r][i]);
            part.mask(i, d);
          }
#pragma unroll
          for (int e = 0; e < P; ++e) {
            gr[r][i][e] = mul2(d[e], wp[e]);
            s1[r] = add2(s1[r], gr[r][i][e]);
            s2[r] = fma2(gr[r][i][e], dev[r][i][e], s2[r]);
            dw[i][e] = fma2(mul2(d[e], r2), dev[r][i][e], dw[i][e]);
            db[i][e] = add2(db[i][e], d[e]);
          }
        }
      }
    fetch(slot == 0 ? D - 1 : slot - 1);   // into the slot read a turn ago
    slot = slot == D - 1 ? 0 : slot + 1;

    float a[B], b[B];
#pragma unroll
    for (int r = 0; r < B; ++r) {
      a[r] = sum2(s1[r]);
      b[r] = sum2(s2[r]);
    }
#pragma unroll
    for (int k = 16; k > 0; k >>= 1)
#pragma unroll
      for (int r = 0; r < B; ++r) {
        a[r] += __shfl_xor_sync(0xffffffffu, a[r], k);
        b[r] += __shfl_xor_sync(0xffffffffu, b[r], k);
      }
    if (WARPS > 1) {
      if (lane == 0)
#pragma unroll
        for (int r = 0; r < B; ++r) stats[turn][r][warp] = make_float2(a[r], b[r]);
      group_sync<TPR>();
#pragma unroll
      for (int r = 0; r < B; ++r) {
        const float2 o = stats[turn][r][grp * WARPS + lane % WARPS];
        a[r] = o.x;
        b[r] = o.y;
      }
#pragma unroll
      for (int k = WARPS / 2; k > 0; k >>= 1)
#pragma unroll
        for (int r = 0; r < B; ++r) {
          a[r] += __shfl_xor_sync(0xffffffffu, a[r], k);
          b[r] += __shfl_xor_sync(0xffffffffu, b[r], k);
        }
    }
#pragma unroll
    for (int r = 0; r < B; ++r) {
      // dx = rstd * g - rstd * mean(g) - dev * rstd^2 * mean(g n),  mean(g n) = rstd * mean(g dev)
      const f32x2 r2 = both(rstd[r]), c1 = both(-rstd[r] * (a[r] * inv_h)), c2 = both(-rstd[r] * (rstd[r] * (rstd[r] * (b[r] * inv_h))));
      if (r == 0 || row + r * groups < p.T) {
#pragma unroll
        for (int i = 0; i < NV; ++i)
          if (part.any(i)) {
            f32x2 o[P];
#pragma unroll
            for (int e = 0; e < P; ++e) o[e] = fma2(dev[r][i][e], c2, fma2(gr[r][i][e], r2, c1));
            part.store(dst, i, Pairs<T>::put(o));
          }
      }
      dst += stride;
      mean[r] = mean_next[r];
      rstd[r] = rstd_next[r];
    }
  }
  cp_async_wait<0>();

  // the block's sums: its groups one after another over shared memory, or straight from registers
  float* out = p.part + (long long)blockIdx.x * 2 * p.H;
  float* acc = GROUPS > 1 ? reinterpret_cast<float*>(ring) : out;
  __syncthreads();
#pragma unroll 1
  for (int k = 0; k < GROUPS; ++k) {
    if (k == grp) {
#pragma unroll
      for (int i = 0; i < NV; ++i)
#pragma unroll
        for (int e = 0; e < V; ++e) {
          const int j = part.col(i) + e;
          if (j < 0 || j >= p.H) continue;
          const float a = e % 2 ? hi2(dw[i][e / 2]) : lo2(dw[i][e / 2]), b = e % 2 ? hi2(db[i][e / 2]) : lo2(db[i][e / 2]);
          acc[j] = k ? acc[j] + a : a;
          acc[p.H + j] = k ? acc[p.H + j] + b : b;
        }
    }
    if (GROUPS > 1) __syncthreads();
  }
  if (GROUPS > 1)
    for (int j = threadIdx.x; j < 2 * p.H; j += kNormThreads) out[j] = acc[j];
}

// dweight (blockIdx.y 0) and dbias (1): the blocks' sums added up.  A block
// takes 32 columns, its 16 warps every 16th of the sums.
template <typename W>
__global__ void __launch_bounds__(512) norm_sums_kernel(const float* part, int n, int H, W* dweight, W* dbias) {
  __shared__ float acc[16][32];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int j = blockIdx.x * 32 + lane;
  W* out = blockIdx.y ? dbias : dweight;
  if (!out) return;
  float s = 0.f;
  if (j < H) {
#pragma unroll 10
    for (int g = warp; g < n; g += 16) s += part[((long long)g * 2 + blockIdx.y) * H + j];
  }
  acc[warp][lane] = s;
  __syncthreads();
  if (warp == 0 && j < H) {
    s = 0.f;
#pragma unroll
    for (int k = 0; k < 16; ++k) s += acc[k][lane];
    out[j] = from_f32<W>(s);
  }
}

// Tensors that do not start on 16 bytes, fp32 rows beyond 8192 values (and the
// odd lengths just below 16384): a block a row for dx, and a thread a column for the sums.
template <typename T, typename W>
__global__ void __launch_bounds__(kNormThreads) norm_bwd_any_kernel(const NormArgs p) {
  __shared__ float scratch[kNormThreads / 32];
  const long long row = blockIdx.x;
  const T *x = static_cast<const T*>(p.x) + row * p.H, *dy = static_cast<const T*>(p.dy) + row * p.H;
  T* dx = static_cast<T*>(p.y) + row * p.H;
  const float mean = p.mean[row], rstd = p.rstd[row];
  float a = 0.f, b = 0.f;
  for (int j = threadIdx.x; j < p.H; j += kNormThreads) {
    const float g = to_f32(dy[j]) * param<W>(p.weight, j, 1.f);
    a += g;
    b = fmaf(g, (to_f32(x[j]) - mean) * rstd, b);
  }
  a = block_sum(a, scratch) / (float)p.H;
  b = block_sum(b, scratch) / (float)p.H;
  for (int j = threadIdx.x; j < p.H; j += kNormThreads) {
    const float g = to_f32(dy[j]) * param<W>(p.weight, j, 1.f), n = (to_f32(x[j]) - mean) * rstd;
    dx[j] = from_f32<T>(rstd * (g - a - n * b));
  }
}

// columns' sums of the rows blockIdx.y, blockIdx.y + gridDim.y, ... into part[blockIdx.y]
template <typename T>
__global__ void __launch_bounds__(256) norm_sums_any_kernel(const NormArgs p) {
  const int j = blockIdx.x * 256 + threadIdx.x;
  if (j >= p.H) return;
  float a = 0.f, b = 0.f;
  for (long long row = blockIdx.y; row < p.T; row += gridDim.y) {
    const float d = to_f32(static_cast<const T*>(p.dy)[row * p.H + j]);
    a = fmaf(d, (to_f32(static_cast<const T*>(p.x)[row * p.H + j]) - p.mean[row]) * p.rstd[row], a);
    b += d;
  }
  p.part[((long long)blockIdx.y * 2) * p.H + j] = a;
  p.part[((long long)blockIdx.y * 2 + 1) * p.H + j] = b;
}

template <typename W>
int launch_sums(const NormArgs& p, int n, void* dweight, void* dbias, cudaStream_t st) {
  if (dweight || dbias)
    norm_sums_kernel<W><<<dim3((p.H + 31) / 32, 2), 512, 0, st>>>(p.part, n, p.H, static_cast<W*>(dweight), static_cast<W*>(dbias));
  return cudaGetLastError() == cudaSuccess ? MOE_OK : MOE_ERR_CUDA;
}

template <typename T, typename W, int TPR, int NV, int B, int D, bool MASK>
int launch_bwd(const NormArgs& p, void* dweight, void* dbias, cudaStream_t st) {
  constexpr size_t ring = (size_t)D * B * 2 * NV * kNormThreads * 16;
  static_assert(kNormThreads / TPR == 1 || ring >= (size_t)2 * TPR * NV * kVec16<T> * 4, "a row's sums fit the ring");
  const size_t smem = ring + (MASK ? 0 : (size_t)p.H * sizeof(W));
  auto kernel = norm_bwd_kernel<T, W, TPR, NV, B, D, MASK>;
  static const cudaError_t attr = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, 227 * 1024 - 1024);
  if (attr != cudaSuccess) return MOE_ERR_CUDA;
  const int blocks = norm_blocks(p.T, kNormThreads / TPR, 1, device_sm_count());
  kernel<<<blocks, kNormThreads, smem, st>>>(p);
  return launch_sums<W>(p, blocks, dweight, dbias, st);
}

template <typename T, typename W>
int launch_bwd_any(const NormArgs& p, void* dweight, void* dbias, cudaStream_t st) {
  // the sums first: dx may be x or dy
  const int n = std::min(p.T, kNormMaxBlocks);
  if (dweight || dbias) norm_sums_any_kernel<T><<<dim3((p.H + 255) / 256, n), 256, 0, st>>>(p);
  norm_bwd_any_kernel<T, W><<<p.T, kNormThreads, 0, st>>>(p);
  return launch_sums<W>(p, n, dweight, dbias, st);
}

template <typename T, typename W, bool MASK>
int norm_bwd(const NormArgs& p, void* dweight, void* dbias, cudaStream_t st) {
  // 16 values a thread; B and D as shared memory holds x and dy of D * B rows beside the weights.
  // Where a block works on one row, two at a time; else its groups overlap already.
  constexpr int V = kVec16<T>, NV = 16 / V, D = sizeof(T) == 2 ? 4 : 3;
  switch (norm_tpr(p.H, V, 16)) {
    case 32: return launch_bwd<T, W, 32, NV, 1, D, MASK>(p, dweight, dbias, st);
    case 64: return launch_bwd<T, W, 64, NV, 1, D, MASK>(p, dweight, dbias, st);
    case 128: return launch_bwd<T, W, 128, NV, 1, D, MASK>(p, dweight, dbias, st);
    case 256: return launch_bwd<T, W, 256, NV, 1, D, MASK>(p, dweight, dbias, st);
    case 512: return launch_bwd<T, W, 512, NV, sizeof(T) == 2 ? 2 : 1, 3, MASK>(p, dweight, dbias, st);
    case 1024:
      if (sizeof(T) == 2) return launch_bwd<T, W, 512, sizeof(T) == 2 ? 2 * NV : NV, 1, 2, MASK>(p, dweight, dbias, st);
    default: break;
  }
  return launch_bwd_any<T, W>(p, dweight, dbias, st);
}

template <typename T, typename W>
int norm_bwd(const NormArgs& p, void* dweight, void* dbias, cudaStream_t st) {
  if (!aligned16(p.x) || !aligned16(p.dy) || !aligned16(p.y)) return launch_bwd_any<T, W>(p, dweight, dbias, st);
  return p.H % kVec16<T> ? norm_bwd<T, W, true>(p, dweight, dbias, st) : norm_bwd<T, W, false>(p, dweight, dbias, st);
}

}  // namespace moe

using namespace moe;

extern "C" int moe_layernorm_bwd_ws_bytes(int T, int H, size_t* bytes) {
  if (!bytes || !norm_shape_ok(T, H)) return MOE_ERR_INVALID_ARG;
  // sums of as many blocks as any type's rows and any such device take
  *bytes = (size_t)std::max(1, std::min(T, kNormMaxBlocks)) * 2 * H * sizeof(float);
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
  if (device_sm_count() > kNormMaxBlocks) return MOE_ERR_UNSUPPORTED;
  const NormArgs p = {x, dy, weight, nullptr, T, H, 0.f, dx, const_cast<float*>(mean), const_cast<float*>(rstd), static_cast<float*>(ws)};
  if (dtype == MOE_F32) return norm_bwd<float, float>(p, dweight, dbias, st);
  if (dtype == MOE_BF16)
    return wdtype == MOE_F32 ? norm_bwd<__nv_bfloat16, float>(p, dweight, dbias, st) : norm_bwd<__nv_bfloat16, __nv_bfloat16>(p, dweight, dbias, st);
  return wdtype == MOE_F32 ? norm_bwd<__half, float>(p, dweight, dbias, st) : norm_bwd<__half, __half>(p, dweight, dbias, st);
}
