// norm_bwd.cu: layer norm's backward pass.
//
//   n = (x - mean) * rstd,  g = dy * weight
//   dx = rstd * (g - mean_H(g) - n * mean_H(g * n)),  dweight = sum_t dy * n,  dbias = sum_t dy
//
// Memory bound: reads x and dy and writes dx once (few rows: norm_bwd_few.cu).  Two blocks an SM walk the
// rows; each thread keeps its columns' sums for dweight and dbias in registers
// over all of its rows.  Blocks write those sums to the workspace (2 H fp32 each,
// 304 of them: 5% of the rows' bytes at 8192 rows), and a second kernel adds
// them up in the blocks' order: no atomics, the same result every time.
#include "norm.cuh"

namespace moe {

// x and dy are read from the ring twice, before and after the row's sums are
// known, so that registers hold the column sums of 32 values a thread and two
// blocks an SM still fit: one block's exchange between warps runs under the other's work.
template <typename T, typename W, int TPR, int BLOCK, int NV, int D, bool MASK>
__global__ void __launch_bounds__(BLOCK, 512 / BLOCK) norm_bwd_kernel(const NormArgs p) {
  constexpr int V = kVec16<T>, P = V / 2, WARPS = TPR / 32, GROUPS = BLOCK / TPR;
  extern __shared__ uint8_t ring[];   // [D][x, dy][NV][threads] vectors, then the weights
  __shared__ float2 stats[2][BLOCK / 32];
  const int grp = (int)threadIdx.x / TPR, lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int groups = gridDim.x * GROUPS, g = blockIdx.x * GROUPS + grp;
  const RowPart<T, TPR, NV, MASK> part(p.H, g);
  constexpr uint32_t STEP = BLOCK * 16, HALF = NV * STEP, SLOT = 2 * HALF;
  grid_launch_next();
  grid_wait_previous();
  uint8_t* mine = ring + threadIdx.x * 16;
  const uint32_t mine_at = smem_u32(mine);
  const long long stride = (long long)groups * p.H;
  long long at = (long long)g * p.H + part.first;   // vector 0 of the next row to fetch
  const T *x = static_cast<const T*>(p.x), *dy = static_cast<const T*>(p.dy);
  T* dst = static_cast<T*>(p.y) + at;
#pragma unroll
  for (int d = 0; d < D - 1; ++d, at += stride) {
    const long long row = g + (long long)d * groups;
    if (row < p.T) {
      part.fetch(x + at, row >= p.tail, mine_at + d * SLOT, STEP);
      part.fetch(dy + at, row >= p.tail, mine_at + d * SLOT + HALF, STEP);
    }
    cp_async_commit();
  }
  W* const ws = reinterpret_cast<W*>(ring + D * SLOT);
  ParamVec<T, W> w[MASK ? NV : 1];
  if (MASK) {
#pragma unroll
    for (int i = 0; i < NV; ++i) w[i] = part.template params<W>(p.weight, 1.f, i);
  } else {
    copy_params<BLOCK>(ws, p.weight, 1.f, p.H);
    __syncthreads();
  }
  auto weights = [&](int i, f32x2* out) {
    if (MASK) w[i].get(out);
    else reinterpret_cast<const ParamVec<T, W>*>(ws + part.col(i))->get(out);
  };
  f32x2 dw[NV][P], db[NV][P];
#pragma unroll
  for (int i = 0; i < NV; ++i)
#pragma unroll
    for (int e = 0; e < P; ++e) dw[i][e] = db[i][e] = 0;
  const float inv_h = 1.f / (float)p.H;
  float mean = g < p.T ? p.mean[g] : 0.f, rstd = g < p.T ? p.rstd[g] : 0.f;

  int slot = 0, turn = 0;
  for (long long row = g; row < p.T; row += groups, turn ^= 1) {
    const bool more = row + groups < p.T;
    const float mean_next = more ? p.mean[row + groups] : 0.f, rstd_next = more ? p.rstd[row + groups] : 0.f;
    cp_async_wait<D - 2>();
    const f32x2 r2 = both(rstd), m2 = both(-mean);
    const uint8_t* here = mine + slot * SLOT;
    f32x2 s1 = 0, s2 = 0;
#pragma unroll
    for (int i = 0; i < NV; ++i)
      if (part.any(i)) {
        f32x2 d[P], dev[P], wp[P];
        Pairs<T>::get(*reinterpret_cast<const uint4*>(here + i * STEP), dev);
        Pairs<T>::get(*reinterpret_cast<const uint4*>(here + HALF + i * STEP), d);
        weights(i, wp);
#pragma unroll
        for (int e = 0; e < P; ++e) dev[e] = add2(dev[e], m2);
        if (MASK) {
          part.mask(i, dev);
          part.mask(i, d);
        }
#pragma unroll
        for (int e = 0; e < P; ++e) {
          const f32x2 gr = mul2(d[e], wp[e]);
          s1 = add2(s1, gr);
          s2 = fma2(gr, dev[e], s2);
          dw[i][e] = fma2(mul2(d[e], r2), dev[e], dw[i][e]);
          db[i][e] = add2(db[i][e], d[e]);
        }
      }
    float a = warp_sum(sum2(s1)), b = warp_sum(sum2(s2));
    if (WARPS > 1) {
      if (lane == 0) stats[turn][warp] = make_float2(a, b);
      group_sync<TPR, BLOCK>();
      const float2 o = stats[turn][grp * WARPS + lane % WARPS];
      a = o.x;
      b = o.y;
#pragma unroll
      for (int k = WARPS / 2; k > 0; k >>= 1) {
        a += __shfl_xor_sync(0xffffffffu, a, k);
        b += __shfl_xor_sync(0xffffffffu, b, k);
      }
    }
    // dx = rstd * g - rstd * mean(g) - dev * rstd^2 * mean(g n),  mean(g n) = rstd * mean(g dev)
    const f32x2 c1 = both(-rstd * (a * inv_h)), c2 = both(-rstd * (rstd * (rstd * (b * inv_h))));
#pragma unroll
    for (int i = 0; i < NV; ++i)
      if (part.any(i)) {
        f32x2 d[P], dev[P], wp[P];
        Pairs<T>::get(*reinterpret_cast<const uint4*>(here + i * STEP), dev);
        Pairs<T>::get(*reinterpret_cast<const uint4*>(here + HALF + i * STEP), d);
        weights(i, wp);
#pragma unroll
        for (int e = 0; e < P; ++e) d[e] = fma2(add2(dev[e], m2), c2, fma2(mul2(d[e], r2), wp[e], c1));
        part.store(dst, i, Pairs<T>::put(d));
      }
    const long long ahead = row + (long long)(D - 1) * groups;
    const int next = slot == 0 ? D - 1 : slot - 1;   // the slot read a row ago
    if (ahead < p.T) {
      part.fetch(x + at, ahead >= p.tail, mine_at + next * SLOT, STEP);
      part.fetch(dy + at, ahead >= p.tail, mine_at + next * SLOT + HALF, STEP);
    }
    cp_async_commit();
    at += stride;
    dst += stride;
    slot = slot == D - 1 ? 0 : slot + 1;
    mean = mean_next;
    rstd = rstd_next;
  }
  cp_async_wait<0>();

  // The block's sums: each group lays its own in shared memory as its vectors lie, and the
  // block adds them up column by column, in the groups' order.
  constexpr int SPAN = TPR * NV * V;
  float* sums = reinterpret_cast<float*>(ring);   // [groups][2][SPAN]
  __syncthreads();
#pragma unroll
  for (int i = 0; i < NV; ++i)
    if (part.any(i)) {
      float* a = sums + (size_t)grp * 2 * SPAN + (i * TPR + part.tid) * V;
#pragma unroll
      for (int e = 0; e < P; e += 2) {
        *reinterpret_cast<float4*>(a + 2 * e) = make_float4(lo2(dw[i][e]), hi2(dw[i][e]), lo2(dw[i][e + 1]), hi2(dw[i][e + 1]));
        *reinterpret_cast<float4*>(a + SPAN + 2 * e) = make_float4(lo2(db[i][e]), hi2(db[i][e]), lo2(db[i][e + 1]), hi2(db[i][e + 1]));
      }
    }
  __syncthreads();
  float* out = p.part + (long long)blockIdx.x * 2 * p.H;
  for (int j = threadIdx.x; j < p.H; j += BLOCK) {
    float a = 0.f, b = 0.f;
#pragma unroll
    for (int k = 0; k < GROUPS; ++k) {
      const int shift = MASK ? (int)((long long)(blockIdx.x * GROUPS + k) * p.H % V) : 0;
      const float* s = sums + (size_t)k * 2 * SPAN + j + shift;
      a += s[0];
      b += s[SPAN];
    }
    out[j] = a;
    out[p.H + j] = b;
  }
}

// dweight (blockIdx.y 0) and dbias (1): the blocks' sums added up.  A block
// takes 32 columns, its 16 warps every 16th of the sums.
template <typename W>
__global__ void __launch_bounds__(512) norm_sums_kernel(const float* part, int n, int H, W* dweight, W* dbias) {
  __shared__ float acc[16][32];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int j = blockIdx.x * 32 + lane;
  W* out = blockIdx.y ? dbias : dweight;
  grid_launch_next();
  grid_wait_previous();
  if (!out) return;
  float s = 0.f;
  if (j < H) {
#pragma unroll
    for (int k = 0; k < kNormMaxBlocks / 16; ++k)   // all loads in flight at once
      if (16 * k + warp < n) s += part[((long long)(16 * k + warp) * 2 + blockIdx.y) * H + j];
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
__global__ void __launch_bounds__(512) norm_bwd_any_kernel(const NormArgs p) {
  __shared__ float scratch[16];
  const long long row = blockIdx.x;
  const T *x = static_cast<const T*>(p.x) + row * p.H, *dy = static_cast<const T*>(p.dy) + row * p.H;
  T* dx = static_cast<T*>(p.y) + row * p.H;
  grid_launch_next();
  grid_wait_previous();
  const float mean = p.mean[row], rstd = p.rstd[row];
  float a = 0.f, b = 0.f;
  for (int j = threadIdx.x; j < p.H; j += 512) {
    const float g = to_f32(dy[j]) * param<W>(p.weight, j, 1.f);
    a += g;
    b = fmaf(g, (to_f32(x[j]) - mean) * rstd, b);
  }
  a = block_sum<512>(a, scratch) / (float)p.H;
  b = block_sum<512>(b, scratch) / (float)p.H;
  for (int j = threadIdx.x; j < p.H; j += 512) {
    const float g = to_f32(dy[j]) * param<W>(p.weight, j, 1.f), n = (to_f32(x[j]) - mean) * rstd;
    dx[j] = from_f32<T>(rstd * (g - a - n * b));
  }
}

// columns' sums of the rows blockIdx.y, blockIdx.y + gridDim.y, ... into part[blockIdx.y]
template <typename T>
__global__ void __launch_bounds__(256) norm_sums_any_kernel(const NormArgs p) {
  const int j = blockIdx.x * 256 + threadIdx.x;
  grid_launch_next();
  grid_wait_previous();
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
  if (!dweight && !dbias) return MOE_OK;
  const float* part = p.part;
  return launch_next(norm_sums_kernel<W>, dim3((p.H + 31) / 32, 2), 512, 0, st, 1, 1, part, n, p.H, static_cast<W*>(dweight), static_cast<W*>(dbias));
}

template <typename T, typename W, int TPR, int NV, int D, bool MASK>
int launch_bwd(const NormArgs& p, void* dweight, void* dbias, cudaStream_t st) {
  constexpr int BLOCK = TPR == 512 ? 512 : 256;
  constexpr size_t ring = (size_t)D * 2 * NV * BLOCK * 16;
  static_assert(ring >= (size_t)2 * BLOCK * NV * kVec16<T> * 4, "the groups' sums fit the ring");
  const size_t smem = ring + (MASK ? 0 : (size_t)p.H * sizeof(W));
  auto kernel = norm_bwd_kernel<T, W, TPR, BLOCK, NV, D, MASK>;
  static OncePerDevice limit;
  if (!limit(current_device(), [&] { return cuda_ok(cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, 227 * 1024 - 1024)); }))
    return MOE_ERR_CUDA;
  const int blocks = norm_blocks(p.T, BLOCK / TPR, BLOCK == 256 && smem <= 112 * 1024 ? 2 : 1, device_sm_count());
  const int rc = launch_next(kernel, dim3(blocks), BLOCK, smem, st, 1, 1, p);
  return rc ? rc : launch_sums<W>(p, blocks, dweight, dbias, st);
}

template <typename T, typename W>
int launch_bwd_any(const NormArgs& p, void* dweight, void* dbias, cudaStream_t st) {
  // the sums first: dx may be x or dy
  const int n = std::min(p.T, kNormMaxBlocks);
  int rc = dweight || dbias ? launch_next(norm_sums_any_kernel<T>, dim3((p.H + 255) / 256, n), 256, 0, st, 1, 1, p) : MOE_OK;
  if (rc == MOE_OK) rc = launch_next(norm_bwd_any_kernel<T, W>, dim3(p.T), 512, 0, st, 1, 1, p);
  return rc ? rc : launch_sums<W>(p, n, dweight, dbias, st);
}

template <typename T, typename W, bool MASK>
int norm_bwd(const NormArgs& p, void* dweight, void* dbias, cudaStream_t st) {
  // 32 values a thread (fp32 rows: 16, whose ring is as large); D turns beside the weights in
  // shared memory, twice an SM where a row takes at most 256 threads
  constexpr int V = kVec16<T>, E = sizeof(T) == 2 ? 32 : 16, NV = E / V;
  switch (norm_tpr(p.H, V, E)) {
    case 32: return launch_bwd<T, W, 32, NV, 3, MASK>(p, dweight, dbias, st);
    case 64: return launch_bwd<T, W, 64, NV, 3, MASK>(p, dweight, dbias, st);
    case 128: return launch_bwd<T, W, 128, NV, 3, MASK>(p, dweight, dbias, st);
    case 256:
      if (MASK || 3 * 32 * 1024 + p.H * sizeof(W) <= 112 * 1024) return launch_bwd<T, W, 256, NV, 3, MASK>(p, dweight, dbias, st);
      return launch_bwd<T, W, 256, NV, 2, MASK>(p, dweight, dbias, st);
    case 512: return launch_bwd<T, W, 512, NV, sizeof(T) == 2 ? 2 : 3, MASK>(p, dweight, dbias, st);
    default: break;
  }
  return launch_bwd_any<T, W>(p, dweight, dbias, st);
}

template <typename T, typename W>
int norm_bwd(const NormArgs& p, void* dweight, void* dbias, cudaStream_t st) {
  if (!aligned16(p.x) || !aligned16(p.dy) || !aligned16(p.y) || !aligned16(p.weight)) return launch_bwd_any<T, W>(p, dweight, dbias, st);
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
    if (dweight && !cuda_ok(cudaMemsetAsync(dweight, 0, H * elem_bytes(wdtype), st))) return MOE_ERR_CUDA;
    if (dbias && !cuda_ok(cudaMemsetAsync(dbias, 0, H * elem_bytes(wdtype), st))) return MOE_ERR_CUDA;
    return MOE_OK;
  }
  size_t need = 0;
  moe_layernorm_bwd_ws_bytes(T, H, &need);
  if (!dy || !x || !mean || !rstd || !dx || !ws || ws_bytes < need) return MOE_ERR_INVALID_ARG;
  if (!elem_aligned(x, dtype) || !elem_aligned(dy, dtype) || !elem_aligned(dx, dtype) || !elem_aligned(mean, MOE_F32) ||
      !elem_aligned(rstd, MOE_F32) || !aligned16(ws))
    return MOE_ERR_INVALID_ARG;
  if (2 * device_sm_count() > kNormMaxBlocks) return MOE_ERR_UNSUPPORTED;
  const NormArgs p = {x, dy, weight, nullptr, T, H, 0.f, dx, const_cast<float*>(mean), const_cast<float*>(rstd), static_cast<float*>(ws), norm_tail(T, H, dtype)};
  // Few rows, and no more than 12 of them to a thread of a strip (22: 14.3 us against 9.8 at 5719 x 143; 10: 7.0 against
  // 11.6 at 1200 x 2048).  dx over x or dy would change what the strips' blocks read.
  const int vec = dtype == MOE_F32 ? 4 : 8, tpr = norm_tpr(H, vec, vec);
  if (tpr <= 1024 && few_rows(T, tpr) && T <= 12 * std::max(256, tpr) && dx != x && dx != dy && aligned16(x) && aligned16(dy) && aligned16(dx) && aligned16(weight))
    return norm_bwd_few(dtype, wdtype, p, dweight, dbias, st);
  if (dtype == MOE_F32) return norm_bwd<float, float>(p, dweight, dbias, st);
  if (dtype == MOE_BF16)
    return wdtype == MOE_F32 ? norm_bwd<__nv_bfloat16, float>(p, dweight, dbias, st) : norm_bwd<__nv_bfloat16, __nv_bfloat16>(p, dweight, dbias, st);
  return wdtype == MOE_F32 ? norm_bwd<__half, float>(p, dweight, dbias, st) : norm_bwd<__half, __half>(p, dweight, dbias, st);
}
