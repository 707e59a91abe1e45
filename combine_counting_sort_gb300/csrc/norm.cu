// norm.cu: layer norm over each row of [T, H], forward.
//
//   n = (x - mean) * rstd,  rstd = 1 / sqrt(var + eps),  y = n * weight + bias
//
// Memory bound: reads x and writes y once.  Mean and variance come from one
// exchange between a row's warps: each takes its own mean, then its squares about
// that mean, and the warps' means and squares are joined about the row's mean, so
// nothing cancels for rows far from zero: their means are right to the last bit (warp_stats), and
// n is made of deviations, for x * rstd - mean * rstd would round at the size of mean * rstd.  A row of
// equal values has n = 0.  Sums are fp32 in a fixed order.
#include "norm.cuh"

namespace moe {

constexpr int kFwdThreads = 512;
// Blocks an SM: two, unless registers hold weights and biases too.
template <typename T, int NV, bool MASK>
constexpr int kFwdPerSm = !MASK && NV * kVec16<T> <= 32 ? 2 : 1;

// A warp's mean and squares about it.  `mean` is off by the roundings of a sum of n values; further than four
// deviations from zero they are not small beside a deviation, and the sum of the thread's deviations, which
// `deviations` gives, moves it.  (Taken for every row: 90.3 us against 87.7 at
// 8192 x 7168 fp32.)
template <typename F>
MOE_DEV float2 warp_stats(float mean, float squares, float inv_n, F&& deviations) {
  if (mean * mean > 16.f * inv_n * squares) {
    const float r = warp_sum(deviations()), move = r * inv_n, q = fmaf(-move, r, squares);
    return make_float2(mean + move, q < 0.f ? 0.f : q);
  }
  return make_float2(mean, squares);
}

template <typename T, typename W, int TPR, int NV, int D, bool MASK>
__global__ void __launch_bounds__(kFwdThreads, kFwdPerSm<T, NV, MASK>) norm_fwd_kernel(const NormArgs p) {
  constexpr int V = kVec16<T>, P = V / 2, BLOCK = kFwdThreads, WARPS = TPR / 32, GROUPS = BLOCK / TPR;
  extern __shared__ uint8_t ring[];   // [D][NV][threads] vectors
  __shared__ float2 stats[2][BLOCK / 32];
  __shared__ float counts[BLOCK / 32];
  const int grp = (int)threadIdx.x / TPR, lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const long long groups = (long long)gridDim.x * GROUPS, g = (long long)blockIdx.x * GROUPS + grp;
  const RowPart<T, TPR, NV, MASK> part(p.H, g);
  constexpr uint32_t STEP = BLOCK * 16, SLOT = NV * STEP;
  grid_launch_next();
  grid_wait_previous();
  uint8_t* mine = ring + threadIdx.x * 16;
  const uint32_t mine_at = smem_u32(mine);
  const long long stride = groups * p.H;
  const T* src = static_cast<const T*>(p.x) + g * p.H + part.first;   // vector 0 of the next row to fetch
  T* dst = static_cast<T*>(p.y) + g * p.H + part.first;
  // (4000 x 8001: 37.8 us with branches, 32.4 without; rows of whole vectors are slower without, 49 against 45)
  if (MASK)
#pragma unroll
    for (int d = 0; d < D; ++d) part.clear_absent(mine + d * SLOT, STEP);
#pragma unroll
  for (int d = 0; d < D - 1; ++d, src += stride) {
    if (g + d * groups < p.T) part.fetch(src, g + d * groups >= p.tail, mine_at + d * SLOT, STEP);
    cp_async_commit();
  }
  W* const ws = reinterpret_cast<W*>(ring + D * SLOT);
  W* const bs = ws + p.H;
  ParamVec<T, W> w[MASK ? NV : 1], b[MASK ? NV : 1];
  if (!MASK) {
    copy_params<BLOCK>(ws, p.weight, 1.f, p.H);
    copy_params<BLOCK>(bs, p.bias, 0.f, p.H);
  }
  int mine_n = 0;
#pragma unroll
  for (int i = 0; i < NV; ++i) {
    if (MASK) {
      w[i] = part.template params<W>(p.weight, 1.f, i);
      b[i] = part.template params<W>(p.bias, 0.f, i);
    }
    mine_n += max(0, part.hi(i) - part.lo(i));
  }
  // values of a row in each warp: the same for every row
  const float warp_n = warp_sum((float)mine_n), warp_inv = warp_n > 0.f ? 1.f / warp_n : 0.f;
  if (lane == 0) counts[warp] = warp_n;
  __syncthreads();
  const int peer = grp * WARPS + lane % WARPS;   // the warp whose sums this lane joins
  const float peer_n = counts[peer], inv_h = 1.f / (float)p.H;

  int slot = 0, turn = 0;
  for (long long row = g; row < p.T; row += groups, turn ^= 1) {
    cp_async_wait<D - 2>();
    f32x2 v[NV][P];
    f32x2 s = 0;
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      if (!MASK && !part.any(i)) continue;
      Pairs<T>::get(*reinterpret_cast<const uint4*>(mine + slot * SLOT + i * STEP), v[i]);
      part.mask(i, v[i]);
#pragma unroll
      for (int e = 0; e < P; ++e) s = add2(s, v[i][e]);
    }
    const int next = slot == 0 ? D - 1 : slot - 1;   // the slot read a row ago
    const long long ahead = row + (D - 1) * groups;
    if (ahead < p.T) part.fetch(src, ahead >= p.tail, mine_at + next * SLOT, STEP);
    cp_async_commit();
    src += stride;
    slot = slot == D - 1 ? 0 : slot + 1;

    const float m = warp_sum(sum2(s)) * warp_inv;
    f32x2 q = 0;
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      if (!MASK && !part.any(i)) continue;
#pragma unroll
      for (int e = 0; e < P; ++e) v[i][e] = add2(v[i][e], both(-m));
      part.mask(i, v[i]);
#pragma unroll
      for (int e = 0; e < P; ++e) q = fma2(v[i][e], v[i][e], q);
    }
    const float2 own = warp_stats(m, warp_sum(sum2(q)), warp_inv, [&] {
      f32x2 r = 0;
#pragma unroll
      for (int i = 0; i < NV; ++i) {
        if (!MASK && !part.any(i)) continue;
#pragma unroll
        for (int e = 0; e < P; ++e) r = add2(r, v[i][e]);
      }
      return sum2(r);
    });
    float mean = own.x, var = own.y * inv_h;
    if (WARPS > 1) {
      if (lane == 0) stats[turn][warp] = own;
      group_sync<TPR, BLOCK>();
      const float2 o = stats[turn][peer];
      const float from = stats[turn][grp * WARPS].x;   // the first warp's mean
      float t = peer_n * (o.x - from);
#pragma unroll
      for (int k = WARPS / 2; k > 0; k >>= 1) t += __shfl_xor_sync(0xffffffffu, t, k);
      mean = fmaf(t, inv_h, from);
      const float off = o.x - mean;
      t = fmaf(peer_n * off, off, o.y);
#pragma unroll
      for (int k = WARPS / 2; k > 0; k >>= 1) t += __shfl_xor_sync(0xffffffffu, t, k);
      var = t * inv_h;
    }
    const float rstd = 1.f / sqrtf(var + p.eps);
    // from the deviations about the warp's mean: their distance to the row's is of their own size
    const f32x2 r2 = both(rstd), off = both((m - mean) * rstd);
    if (part.tid == 0) {
      if (p.mean) p.mean[row] = mean;
      if (p.rstd) p.rstd[row] = rstd;
    }
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      if (!MASK && !part.any(i)) continue;
      f32x2 wp[P], bp[P], o[P];
      if (MASK) {
        w[i].get(wp);
        b[i].get(bp);
      } else {
        reinterpret_cast<const ParamVec<T, W>*>(ws + part.col(i))->get(wp);
        reinterpret_cast<const ParamVec<T, W>*>(bs + part.col(i))->get(bp);
      }
#pragma unroll
      for (int e = 0; e < P; ++e) o[e] = fma2(fma2(v[i][e], r2, off), wp[e], bp[e]);
      if (part.any(i)) part.store(dst, i, Pairs<T>::put(o));
    }
    dst += stride;
  }
  cp_async_wait<0>();
}

// Few rows: all of them at once, everything loaded straight into registers (one vector
// a thread, TPR threads a row), since the latency of one row is the time.
// What is held between the passes stays packed, so that an SM holds 1536 threads and more.
template <typename T, typename W, int TPR, bool MASK>
__global__ void __launch_bounds__(TPR < 256 ? 256 : TPR, (TPR <= 64 ? 4 : TPR <= 256 ? 6 : TPR == 512 ? 3 : 2)) norm_fwd_few_kernel(const NormArgs p) {
  constexpr int V = kVec16<T>, P = V / 2, WARPS = TPR / 32, BLOCK = TPR < 256 ? 256 : TPR;
  __shared__ float2 stats[BLOCK / 32];
  __shared__ float counts[BLOCK / 32];
  const int grp = (int)threadIdx.x / TPR, lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const long long row = (long long)blockIdx.x * (BLOCK / TPR) + grp;
  const RowPart<T, TPR, 1, MASK> part(p.H, row);
  const T* src = static_cast<const T*>(p.x) + row * p.H + part.first;
  uint4 raw = make_uint4(0, 0, 0, 0);
  ParamVec<T, W> w, b;
  grid_launch_next();
  grid_wait_previous();
  if (row >= p.T) return;   // (a whole group)
  if (MASK) {
    // a row's first and last vectors have its neighbours' values too, but none behind the tensor
    uint4 wr[2] = {}, br[2] = {};
    const bool there = part.any(0), inside = part.readable(0, row >= p.tail) == V;
    load_if(raw, src, there && inside);
    part.template params_begin<W>(p.weight, 0, wr);
    part.template params_begin<W>(p.bias, 0, br);
    if (there) {
      if (!inside) {
        f32x2 v[P];
#pragma unroll
        for (int e = 0; e < P; ++e)
          v[e] = pack_f32x2(2 * e >= part.lo(0) && 2 * e < part.hi(0) ? to_f32(src[2 * e]) : 0.f,
                            2 * e + 1 >= part.lo(0) && 2 * e + 1 < part.hi(0) ? to_f32(src[2 * e + 1]) : 0.f);
        raw = Pairs<T>::put(v);
      }
      w = part.template params_end<W>(p.weight, 1.f, 0, wr);
      b = part.template params_end<W>(p.bias, 0.f, 0, br);
    }
  } else if (part.any(0)) {
    raw = *reinterpret_cast<const uint4*>(src);
    if (p.weight) w = *reinterpret_cast<const ParamVec<T, W>*>(static_cast<const W*>(p.weight) + part.col(0));
    else w = part.template params<W>(p.weight, 1.f, 0);
    if (p.bias) b = *reinterpret_cast<const ParamVec<T, W>*>(static_cast<const W*>(p.bias) + part.col(0));
    else b = part.template params<W>(p.bias, 0.f, 0);
  }
  const float n = warp_sum((float)max(0, part.hi(0) - part.lo(0))), inv_n = n > 0.f ? 1.f / n : 0.f, inv_h = 1.f / (float)p.H;
  f32x2 v[P], s = 0;
  Pairs<T>::get(raw, v);
  if (part.any(0)) part.mask(0, v);
#pragma unroll
  for (int e = 0; e < P; ++e) s = add2(s, v[e]);
  const float m = warp_sum(sum2(s)) * inv_n;
  f32x2 d[P], q = 0, r = 0;
#pragma unroll
  for (int e = 0; e < P; ++e) d[e] = add2(v[e], both(-m));
  if (part.any(0)) {
    part.mask(0, d);
#pragma unroll
    for (int e = 0; e < P; ++e) {
      q = fma2(d[e], d[e], q);
      r = add2(r, d[e]);
    }
  }
  const float2 own = warp_stats(m, warp_sum(sum2(q)), inv_n, [&] { return sum2(r); });
  float mean = own.x, var = own.y * inv_h;
  if (WARPS > 1) {
    if (lane == 0) {
      stats[warp] = own;
      counts[warp] = n;
    }
    group_sync<TPR, BLOCK>();
    const int peer = grp * WARPS + lane;
    const float2 o = lane < WARPS ? stats[peer] : make_float2(0.f, 0.f);
    const float on = lane < WARPS ? counts[peer] : 0.f;
    const float from = __shfl_sync(0xffffffffu, o.x, 0);   // the first warp's mean
    mean = fmaf(warp_sum(on * (o.x - from)), inv_h, from);
    const float off = o.x - mean;
    var = warp_sum(fmaf(on * off, off, o.y)) * inv_h;
  }
  const float rstd = 1.f / sqrtf(var + p.eps);
  if (part.tid == 0) {
    if (p.mean) p.mean[row] = mean;
    if (p.rstd) p.rstd[row] = rstd;
  }
  if (part.any(0)) {
    f32x2 wp[P], bp[P];
    Pairs<T>::get(raw, v);
    w.get(wp);
    b.get(bp);
#pragma unroll
    for (int e = 0; e < P; ++e) v[e] = fma2(mul2(add2(v[e], both(-mean)), both(rstd)), wp[e], bp[e]);
    part.store(static_cast<T*>(p.y) + row * p.H + part.first, 0, Pairs<T>::put(v));
  }
}

// Tensors that do not start on 16 bytes (and the odd lengths just below 16384): a
// block a row, read three times.
template <typename T, typename W>
__global__ void __launch_bounds__(512) norm_fwd_any_kernel(const NormArgs p) {
  __shared__ float scratch[16];
  const long long row = blockIdx.x;
  const T* x = static_cast<const T*>(p.x) + row * p.H;
  T* y = static_cast<T*>(p.y) + row * p.H;
  float s = 0.f;
  grid_launch_next();
  grid_wait_previous();
  for (int j = threadIdx.x; j < p.H; j += 512) s += to_f32(x[j]);
  const float m = block_sum<512>(s, scratch) / (float)p.H;
  float r = 0.f;
  s = 0.f;
  for (int j = threadIdx.x; j < p.H; j += 512) {
    const float d = to_f32(x[j]) - m;
    s = fmaf(d, d, s);
    r += d;
  }
  r = block_sum<512>(r, scratch) / (float)p.H;
  const float mean = m + r, rstd = 1.f / sqrtf(fmaxf(fmaf(-r, r, block_sum<512>(s, scratch) / (float)p.H), 0.f) + p.eps);
  if (threadIdx.x == 0) {
    if (p.mean) p.mean[row] = mean;
    if (p.rstd) p.rstd[row] = rstd;
  }
  for (int j = threadIdx.x; j < p.H; j += 512)
    y[j] = from_f32<T>(fmaf((to_f32(x[j]) - mean) * rstd, param<W>(p.weight, j, 1.f), param<W>(p.bias, j, 0.f)));
}

template <typename T, typename W, int TPR, int NV, int D, bool MASK>
int launch_fwd(const NormArgs& p, cudaStream_t st) {
  const size_t smem = (size_t)D * NV * kFwdThreads * 16 + (MASK ? 0 : 2 * (size_t)p.H * sizeof(W));
  auto kernel = norm_fwd_kernel<T, W, TPR, NV, D, MASK>;
  static OncePerDevice limit;
  if (!limit(current_device(), [&] { return cuda_ok(cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, 227 * 1024 - 1024)); }))
    return MOE_ERR_CUDA;
  const int per_sm = smem <= 112 * 1024 ? kFwdPerSm<T, NV, MASK> : 1;
  return launch_next(kernel, dim3(norm_blocks(p.T, kFwdThreads / TPR, per_sm, device_sm_count())), kFwdThreads, smem, st, 1, 1, p);
}

template <typename T, typename W>
int launch_fwd_any(const NormArgs& p, cudaStream_t st) {
  return launch_next(norm_fwd_any_kernel<T, W>, dim3(p.T), 512, 0, st, 1, 1, p);
}

template <typename T, typename W, int TPR, bool MASK>
int launch_fwd_few(const NormArgs& p, cudaStream_t st) {
  constexpr int BLOCK = TPR < 256 ? 256 : TPR, ROWS = BLOCK / TPR;
  return launch_next(norm_fwd_few_kernel<T, W, TPR, MASK>, dim3((p.T + ROWS - 1) / ROWS), BLOCK, 0, st, 1, 1, p);
}

template <typename T, typename W, bool MASK>
int norm_fwd(const NormArgs& p, cudaStream_t st) {
  constexpr int V = kVec16<T>;
  switch (norm_tpr(p.H, V, V)) {
    case 32: if (few_rows(p.T, 32)) return launch_fwd_few<T, W, 32, MASK>(p, st); break;
    case 64: if (few_rows(p.T, 64)) return launch_fwd_few<T, W, 64, MASK>(p, st); break;
    case 128: if (few_rows(p.T, 128)) return launch_fwd_few<T, W, 128, MASK>(p, st); break;
    case 256: if (few_rows(p.T, 256)) return launch_fwd_few<T, W, 256, MASK>(p, st); break;
    case 512: if (few_rows(p.T, 512)) return launch_fwd_few<T, W, 512, MASK>(p, st); break;
    case 1024: if (few_rows(p.T, 1024)) return launch_fwd_few<T, W, 1024, MASK>(p, st); break;
    default: break;
  }
  // Values a thread: as many as leave two blocks an SM room in registers and shared memory.
  // (One block of 1024 threads with a turn more in its ring: 50.8 us against 46.9 at 8192 x 7168.)
  constexpr int E = sizeof(T) == 2 ? 32 : 16, NV = E / V, D = 2;
  switch (norm_tpr(p.H, V, E)) {
    case 32: return launch_fwd<T, W, 32, NV, D, MASK>(p, st);
    case 64: return launch_fwd<T, W, 64, NV, D, MASK>(p, st);
    case 128: return launch_fwd<T, W, 128, NV, D, MASK>(p, st);
    case 256: return launch_fwd<T, W, 256, NV, D, MASK>(p, st);
    case 512: return launch_fwd<T, W, 512, NV, D, MASK>(p, st);
    case 1024:   // fp32 beyond 8192 values: weights and biases in registers, for they do not fit beside the ring
      if (sizeof(T) == 4) return launch_fwd<T, W, 512, sizeof(T) == 4 ? 2 * NV : NV, D, true>(p, st);
    default: return launch_fwd_any<T, W>(p, st);
  }
}

template <typename T, typename W>
int norm_fwd(const NormArgs& p, cudaStream_t st) {
  if (!aligned16(p.x) || !aligned16(p.y) || !aligned16(p.weight) || !aligned16(p.bias)) return launch_fwd_any<T, W>(p, st);
  return p.H % kVec16<T> ? norm_fwd<T, W, true>(p, st) : norm_fwd<T, W, false>(p, st);
}

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
  const NormArgs p = {x, nullptr, weight, bias, T, H, eps, y, mean, rstd, nullptr, norm_tail(T, H, dtype)};
  cudaStream_t st = (cudaStream_t)stream;
  if (dtype == MOE_F32) return norm_fwd<float, float>(p, st);
  if (dtype == MOE_BF16) return wdtype == MOE_F32 ? norm_fwd<__nv_bfloat16, float>(p, st) : norm_fwd<__nv_bfloat16, __nv_bfloat16>(p, st);
  return wdtype == MOE_F32 ? norm_fwd<__half, float>(p, st) : norm_fwd<__half, __half>(p, st);
}
