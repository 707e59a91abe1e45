// norm_bwd_few.cu: layer norm's backward pass for few rows, in one launch.
//
// The rows' dx and the columns' sums need nothing of one another, so some blocks
// take rows, all at once with a vector a thread, and others take strips of
// columns over all rows, which they read a second time (out of L2).  Against each
// block's sums in a workspace and a second kernel, whose bytes are a row's of
// fp32 for each block: 300 x 7168 13.0 us against 7.3 here, one row 7.2 against 2.0.
//
// A strip is 8 vectors wide; the blocks of a cluster share its rows and add up
// their sums through distributed shared memory in rank order.
#include "norm.cuh"

namespace moe {

// This lane's vector of a row that starts anywhere (UNALIGNED), or on a vector.  By predicated
// loads; what lies beyond the tensor is fetched value by value, when it is taken.
template <typename T, bool UNALIGNED>
struct StripVec {
  uint4 lo, hi;
  MOE_DEV static int off(long long at) { return (int)(at % kVec16<T>); }   // (the tensor itself starts on 16 bytes)
  MOE_DEV static bool inside(long long at, long long total) { return at - off(at) + 2 * kVec16<T> <= total; }
  MOE_DEV void load(const T* p, long long at, long long total, bool there) {
    if (!UNALIGNED) {
      load_if(lo, p + at, there);
    } else {
      const T* v = p + at - off(at);
      load_if(lo, v, there && inside(at, total));
      load_if(hi, v + kVec16<T>, there && inside(at, total));
    }
  }
  MOE_DEV uint4 take(const T* p, long long at, long long total) const {
    if (!UNALIGNED) return lo;
    if (!inside(at, total)) {
      constexpr int V = kVec16<T>;
      f32x2 f[V / 2];
#pragma unroll
      for (int e = 0; e < V / 2; ++e)
        f[e] = pack_f32x2(at + 2 * e < total ? to_f32(p[at + 2 * e]) : 0.f, at + 2 * e + 1 < total ? to_f32(p[at + 2 * e + 1]) : 0.f);
      return Pairs<T>::put(f);
    }
    return sizeof(T) == 2 ? shifted8(lo, hi, off(at)) : shifted8(lo, hi, 2 * off(at));
  }
};

template <typename T, typename W, int TPR, bool MASK>
__global__ void __launch_bounds__(TPR < 256 ? 256 : TPR, TPR <= 256 ? 4 : 1024 / TPR)
    norm_bwd_few_kernel(const __grid_constant__ NormArgs p, W* dweight, W* dbias, int strip_blocks, int cluster) {
  constexpr int V = kVec16<T>, P = V / 2, BLOCK = TPR < 256 ? 256 : TPR, WARPS = BLOCK / 32;
  const T *x = static_cast<const T*>(p.x), *dy = static_cast<const T*>(p.dy);
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  grid_launch_next();
  grid_wait_previous();

  if ((int)blockIdx.x < strip_blocks) {   // ---- a strip of columns
    constexpr int COLS = 8 * V, SLOTS = BLOCK / 8, ROWS = 2;
    __shared__ float sums[WARPS][2][COLS];
    __shared__ float total[2][COLS];
    const int rank = (int)blockIdx.x % cluster, j0 = (int)blockIdx.x / cluster * COLS;
    const int j = j0 + (int)(threadIdx.x % 8) * V, step = SLOTS * cluster;
    const long long all = (long long)p.T * p.H;
    f32x2 dw[P], db[P];
#pragma unroll
    for (int e = 0; e < P; ++e) dw[e] = db[e] = 0;
    for (long long i = rank * SLOTS + (int)threadIdx.x / 8; i < p.T; i += (long long)ROWS * step) {
      StripVec<T, MASK> xs[ROWS] = {}, ds[ROWS] = {};
      float mean[ROWS], rstd[ROWS];
#pragma unroll
      for (int r = 0; r < ROWS; ++r) {
        const long long row = i + r * step;
        const bool there = row < p.T && j < p.H;
        xs[r].load(x, row * p.H + j, all, there);
        ds[r].load(dy, row * p.H + j, all, there);
        mean[r] = there ? p.mean[row] : 0.f;
        rstd[r] = there ? p.rstd[row] : 0.f;
      }
#pragma unroll
      for (int r = 0; r < ROWS; ++r) {
        const long long row = i + r * step;
        if (row >= p.T || j >= p.H) break;
        f32x2 d[P], dev[P];
        Pairs<T>::get(xs[r].take(x, row * p.H + j, all), dev);
        Pairs<T>::get(ds[r].take(dy, row * p.H + j, all), d);
#pragma unroll
        for (int e = 0; e < P; ++e) {
          dw[e] = fma2(mul2(d[e], both(rstd[r])), add2(dev[e], both(-mean[r])), dw[e]);
          db[e] = add2(db[e], d[e]);
        }
      }
    }
    // the warp's four rows, the block's warps, the cluster's blocks
#pragma unroll
    for (int e = 0; e < P; ++e)
#pragma unroll
      for (int o = 8; o <= 16; o *= 2) {
        dw[e] = add2(dw[e], pack_f32x2(__shfl_xor_sync(0xffffffffu, lo2(dw[e]), o), __shfl_xor_sync(0xffffffffu, hi2(dw[e]), o)));
        db[e] = add2(db[e], pack_f32x2(__shfl_xor_sync(0xffffffffu, lo2(db[e]), o), __shfl_xor_sync(0xffffffffu, hi2(db[e]), o)));
      }
    if (lane < 8)
#pragma unroll
      for (int e = 0; e < P; ++e) {
        *reinterpret_cast<f32x2*>(&sums[warp][0][lane * V + 2 * e]) = dw[e];
        *reinterpret_cast<f32x2*>(&sums[warp][1][lane * V + 2 * e]) = db[e];
      }
    __syncthreads();
    const int which = (int)threadIdx.x / COLS, c = (int)threadIdx.x % COLS;
    float s = 0.f;
    if (which < 2) {
#pragma unroll
      for (int w = 0; w < WARPS; ++w) s += sums[w][which][c];
      total[which][c] = s;
    }
    if (cluster > 1) cluster_sync();
    W* out = which ? dbias : dweight;
    if (rank == 0 && which < 2 && j0 + c < p.H && out) {
      if (cluster > 1) {
        s = 0.f;
        for (int r = 0; r < cluster; ++r) {
          float v;
          asm volatile("ld.shared::cluster.f32 %0, [%1];" : "=f"(v) : "r"(mapa_shared(smem_u32(&total[which][c]), (uint32_t)r)) : "memory");
          s += v;
        }
      }
      out[j0 + c] = from_f32<W>(s);
    }
    if (cluster > 1) cluster_sync();
    return;
  }

  // ---- rows
  __shared__ float2 stats[WARPS];
  const int grp = (int)threadIdx.x / TPR;
  const long long row = (long long)((int)blockIdx.x - strip_blocks) * (BLOCK / TPR) + grp;
  if (row >= p.T) return;   // (a whole group)
  const RowPart<T, TPR, 1, MASK> part(p.H, row);
  const long long at = row * p.H + part.first;
  // a row's first and last vectors have its neighbours' values too, but none behind the tensor
  const bool there = part.any(0), inside = part.readable(0, row >= p.tail) == V;
  uint4 xr = make_uint4(0, 0, 0, 0), dr = xr, wr[2] = {};
  ParamVec<T, W> w;
  load_if(xr, x + at, there && inside);
  load_if(dr, dy + at, there && inside);
  if (MASK) part.template params_begin<W>(p.weight, 0, wr);
  else if (there && p.weight) w = *reinterpret_cast<const ParamVec<T, W>*>(static_cast<const W*>(p.weight) + part.col(0));
  const float mean = p.mean[row], rstd = p.rstd[row];
  f32x2 s1 = 0, s2 = 0, dev[P], g[P];
  if (there) {
    if (!inside) {
      f32x2 a[P], b[P];
#pragma unroll
      for (int e = 0; e < P; ++e) {
        const bool l = 2 * e >= part.lo(0) && 2 * e < part.hi(0), h = 2 * e + 1 >= part.lo(0) && 2 * e + 1 < part.hi(0);
        a[e] = pack_f32x2(l ? to_f32(x[at + 2 * e]) : 0.f, h ? to_f32(x[at + 2 * e + 1]) : 0.f);
        b[e] = pack_f32x2(l ? to_f32(dy[at + 2 * e]) : 0.f, h ? to_f32(dy[at + 2 * e + 1]) : 0.f);
      }
      xr = Pairs<T>::put(a);
      dr = Pairs<T>::put(b);
    }
    if (MASK) w = part.template params_end<W>(p.weight, 1.f, 0, wr);
    else if (!p.weight) w = part.template params<W>(nullptr, 1.f, 0);
    f32x2 wp[P];
    Pairs<T>::get(xr, dev);
    Pairs<T>::get(dr, g);
    w.get(wp);
#pragma unroll
    for (int e = 0; e < P; ++e) {
      dev[e] = add2(dev[e], both(-mean));
      g[e] = mul2(g[e], wp[e]);
    }
    part.mask(0, dev);
    part.mask(0, g);
#pragma unroll
    for (int e = 0; e < P; ++e) {
      s1 = add2(s1, g[e]);
      s2 = fma2(g[e], dev[e], s2);
    }
  }
  float a = warp_sum(sum2(s1)), b = warp_sum(sum2(s2));
  if (TPR > 32) {
    if (lane == 0) stats[warp] = make_float2(a, b);
    group_sync<TPR, BLOCK>();
    const float2 o = lane < TPR / 32 ? stats[grp * (TPR / 32) + lane] : make_float2(0.f, 0.f);
    a = warp_sum(o.x);
    b = warp_sum(o.y);
  }
  if (!there) return;
  // dx = rstd * g - rstd * mean(g) - dev * rstd^2 * mean(g n),  mean(g n) = rstd * mean(g dev)
  const float inv_h = 1.f / (float)p.H;
  const f32x2 c1 = both(-rstd * (a * inv_h)), c2 = both(-rstd * (rstd * (rstd * (b * inv_h))));
#pragma unroll
  for (int e = 0; e < P; ++e) g[e] = fma2(dev[e], c2, fma2(g[e], both(rstd), c1));
  part.store(static_cast<T*>(p.y) + at, 0, Pairs<T>::put(g));
}

template <typename T, typename W, int TPR, bool MASK>
int launch_few(const NormArgs& p, void* dweight, void* dbias, cudaStream_t st) {
  constexpr int BLOCK = TPR < 256 ? 256 : TPR, ROWS = BLOCK / TPR, COLS = 8 * kVec16<T>;
  const int strips = dweight || dbias ? (p.H + COLS - 1) / COLS : 0;
  // blocks to a strip: four rows a thread, where so many strips leave room for them
  const int wanted = (p.T + BLOCK / 8 * 4 - 1) / (BLOCK / 8 * 4), room = std::max(1, 2 * device_sm_count() / std::max(1, strips));
  const int cluster = strips ? std::min({8, wanted, room}) : 1;
  const int blocks = (strips * cluster + (p.T + ROWS - 1) / ROWS + cluster - 1) / cluster * cluster;
  return launch_next(norm_bwd_few_kernel<T, W, TPR, MASK>, dim3((unsigned)blocks), BLOCK, 0, st, (unsigned)cluster, 1, p, static_cast<W*>(dweight),
                     static_cast<W*>(dbias), strips * cluster, cluster);
}

template <typename T, typename W, bool MASK>
int few(const NormArgs& p, void* dweight, void* dbias, cudaStream_t st) {
  constexpr int V = kVec16<T>;
  switch (norm_tpr(p.H, V, V)) {
    case 32: return launch_few<T, W, 32, MASK>(p, dweight, dbias, st);
    case 64: return launch_few<T, W, 64, MASK>(p, dweight, dbias, st);
    case 128: return launch_few<T, W, 128, MASK>(p, dweight, dbias, st);
    case 256: return launch_few<T, W, 256, MASK>(p, dweight, dbias, st);
    case 512: return launch_few<T, W, 512, MASK>(p, dweight, dbias, st);
    default: return launch_few<T, W, 1024, MASK>(p, dweight, dbias, st);
  }
}

template <typename T, typename W>
int few(const NormArgs& p, void* dweight, void* dbias, cudaStream_t st) {
  return p.H % kVec16<T> ? few<T, W, true>(p, dweight, dbias, st) : few<T, W, false>(p, dweight, dbias, st);
}

int norm_bwd_few(int dtype, int wdtype, const NormArgs& p, void* dweight, void* dbias, cudaStream_t st) {
  if (dtype == MOE_F32) return few<float, float>(p, dweight, dbias, st);
  if (dtype == MOE_BF16)
    return wdtype == MOE_F32 ? few<__nv_bfloat16, float>(p, dweight, dbias, st) : few<__nv_bfloat16, __nv_bfloat16>(p, dweight, dbias, st);
  return wdtype == MOE_F32 ? few<__half, float>(p, dweight, dbias, st) : few<__half, __half>(p, dweight, dbias, st);
}

}  // namespace moe
