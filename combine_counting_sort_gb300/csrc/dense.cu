// dense.cu: moe_linear and moe_gated with their backward passes, and the
// elementwise kernels in front of the backward products.
#include "dense_host.cuh"

namespace moe {

// ---------------------------------------------------------------- d = dy * slope and dbias
//
// Memory bound: reads dy and slope, writes d.  A block of 256 threads takes 8 LANES columns,
// LANES threads to a row, eight columns a thread, a few rows in flight; the blocks of a
// cluster (gridDim.y of them) share the rows, and add up their column sums through
// distributed shared memory in rank order.  d's rows are padded to whole vectors.  Rows of
// dy and slope of any length (SHIFT) start anywhere: their eight values are shifted out of
// the two vectors that hold them (857 x 5141 with the sums: 36 us value by value).

template <typename T, bool SHIFT, int LANES>
__global__ void __launch_bounds__(256, 2)
    dense_d_kernel(const T* dy, const T* slope, int I, int J, T* d, long long ldd, T* dbias) {
  constexpr int SLOTS = 256 / LANES, COLS = 8 * LANES, ROWS = SHIFT ? 2 : 4;
  __shared__ float sums[SLOTS][COLS];
  __shared__ float total[COLS];
  const int lane = threadIdx.x % LANES, slot = threadIdx.x / LANES, j0 = blockIdx.x * COLS, j = j0 + 8 * lane;
  const long long rows = I;
  f32x2 acc[4] = {0, 0, 0, 0};
  grid_launch_next();
  grid_wait_previous();
  const int step = SLOTS * gridDim.y;
  const uint16_t *py = reinterpret_cast<const uint16_t*>(dy), *ps = reinterpret_cast<const uint16_t*>(slope);
  // (columns from J on, up to whole vectors, are written with whatever is there: nothing reads them)
  if (j < J)
    for (long long i = blockIdx.y * SLOTS + slot; i < I; i += (long long)ROWS * step) {
      uint4 a[ROWS], s[ROWS];
      if (SHIFT) {
        Unaligned ua[ROWS] = {}, us[ROWS] = {};
#pragma unroll
        for (int r = 0; r < ROWS; ++r) {
          const long long at = min(i + r * step, rows - 1) * J + j;
          load_unaligned(ua[r], py, at, rows * J);
          if (slope) load_unaligned(us[r], ps, at, rows * J);
        }
#pragma unroll
        for (int r = 0; r < ROWS; ++r) {
          const long long at = min(i + r * step, rows - 1) * J + j;
          a[r] = shifted(ua[r], py, at, rows * J);
          if (slope) s[r] = shifted(us[r], ps, at, rows * J);
        }
      } else {
#pragma unroll
        for (int r = 0; r < ROWS; ++r)
          if (i + r * step < I) {
            a[r] = *reinterpret_cast<const uint4*>(py + (i + r * step) * J + j);
            if (slope) s[r] = *reinterpret_cast<const uint4*>(ps + (i + r * step) * J + j);
          }
      }
#pragma unroll
      for (int r = 0; r < ROWS; ++r)
        if (i + r * step < I) {
          f32x2 f[4], g[4];
          Pairs<T>::get(a[r], f);
          if (slope) {
            Pairs<T>::get(s[r], g);
#pragma unroll
            for (int e = 0; e < 4; ++e) f[e] = mul2(f[e], g[e]);
          }
#pragma unroll
          for (int e = 0; e < 4; ++e) acc[e] = add2(acc[e], f[e]);
          if (d) *reinterpret_cast<uint4*>(d + (i + r * step) * ldd + j) = Pairs<T>::put(f);
        }
    }
  if (!dbias) return;
#pragma unroll
  for (int e = 0; e < 4; ++e) *reinterpret_cast<f32x2*>(&sums[slot][8 * lane + 2 * e]) = acc[e];
  __syncthreads();
  if (threadIdx.x < COLS) {
    float s = 0.f;
#pragma unroll
    for (int w = 0; w < SLOTS; ++w) s += sums[w][threadIdx.x];
    total[threadIdx.x] = s;
  }
  cluster_sync();
  if (blockIdx.y == 0 && threadIdx.x < COLS && j0 + (int)threadIdx.x < J) {
    float s = 0.f;
    const uint32_t at = smem_u32(&total[threadIdx.x]);
    for (uint32_t r = 0; r < gridDim.y; ++r) s += ld_shared_cluster_f32(mapa_shared(at, r));
    dbias[j0 + threadIdx.x] = from_f32<T>(s);
  }
  cluster_sync();
}

// d = [dh * factors[:, :F], dh * factors[:, F:]].  (Rows of odd lengths value by value: half of d's own
// lie across its vectors.)
template <typename T, int V>
__global__ void __launch_bounds__(256) gated_d_kernel(const T* dh, const T* factors, int I, int F, T* d, long long ldd) {
  const int j = (blockIdx.x * 256 + threadIdx.x) * V;
  grid_launch_next();
  grid_wait_previous();
  if (j >= F) return;
  constexpr int ROWS = 2;   // in flight
  for (long long i = blockIdx.y; i < I; i += (long long)ROWS * gridDim.y) {
    Vec<T, V> a[ROWS], p[ROWS], q[ROWS];
#pragma unroll
    for (int r = 0; r < ROWS; ++r) {
      const long long at = i + r * (long long)gridDim.y;
      if (at < I) {
        a[r] = *reinterpret_cast<const Vec<T, V>*>(dh + at * F + j);
        p[r] = *reinterpret_cast<const Vec<T, V>*>(factors + at * 2 * F + j);
        q[r] = *reinterpret_cast<const Vec<T, V>*>(factors + at * 2 * F + F + j);
      }
    }
#pragma unroll
    for (int r = 0; r < ROWS; ++r) {
      const long long at = i + r * (long long)gridDim.y;
      if (at >= I) break;
      Vec<T, V> o, u;
#pragma unroll
      for (int v = 0; v < V; ++v) {
        const float f = to_f32(a[r].v[v]);
        o.v[v] = from_f32<T>(f * to_f32(p[r].v[v]));
        u.v[v] = from_f32<T>(f * to_f32(q[r].v[v]));
      }
      *reinterpret_cast<Vec<T, V>*>(d + at * ldd + j) = o;
      *reinterpret_cast<Vec<T, V>*>(d + at * ldd + F + j) = u;
    }
  }
}

template <typename T, int LANES>
int launch_d_lanes(const void* dy, const void* slope, int I, int J, void* d, long long ldd, void* dbias, cudaStream_t st) {
  const bool vec = J % 8 == 0 && aligned16(dy) && aligned16(slope);
  const int strips = (J + 8 * LANES - 1) / (8 * LANES), slots = 256 / LANES;
  // as many blocks as run at once: two an SM, or an eighth fewer in the clusters of up to 8 that add up their
  // sums, which do not fill every part of the device (857 x 5141: 8.6 us, 13.4 with two an SM)
  const int sms = device_sm_count(), all = dbias ? sms * 7 / 4 : 2 * sms;
  const long long want = std::max(1, all / strips), cap = dbias ? 8 : all;
  const int ys = (int)std::min({cap, want, ((long long)I + slots - 1) / slots});
  auto kernel = vec ? dense_d_kernel<T, false, LANES> : dense_d_kernel<T, true, LANES>;
  return launch_next(kernel, dim3((unsigned)strips, (unsigned)ys), 256, 0, st, 1, dbias ? (unsigned)ys : 1u, static_cast<const T*>(dy),
                     static_cast<const T*>(slope), I, J, static_cast<T*>(d), ldd, static_cast<T*>(dbias));
}

// Columns a block: 256 bytes of a row, or less where the clusters of so many strips would not fill the device.
template <typename T>
int launch_d(const void* dy, const void* slope, int I, int J, void* d, long long ldd, void* dbias, cudaStream_t st) {
  const int clusters = device_sm_count() / 8;
  if (!dbias || J > clusters * 128) return launch_d_lanes<T, 16>(dy, slope, I, J, d, ldd, dbias, st);
  if (J > clusters * 64) return launch_d_lanes<T, 8>(dy, slope, I, J, d, ldd, dbias, st);
  return launch_d_lanes<T, 4>(dy, slope, I, J, d, ldd, dbias, st);
}

template <typename T>
int launch_gated_d(const void* dh, const void* factors, int I, int F, void* d, long long ldd, cudaStream_t st) {
  const bool vec = F % 8 == 0 && aligned16(dh) && aligned16(factors);
  const int per = vec ? 2048 : 256, strips = (F + per - 1) / per;
  const dim3 grid((unsigned)strips, (unsigned)std::min(I, std::max(1, 16 * device_sm_count() / strips)));
  auto kernel = vec ? gated_d_kernel<T, 8> : gated_d_kernel<T, 1>;
  return launch_next(kernel, grid, 256, 0, st, 1, 1, static_cast<const T*>(dh), static_cast<const T*>(factors), I, F, static_cast<T*>(d), ldd);
}

constexpr int kDenseMaxT = 1 << 24;

inline bool dense_shape_ok(int T, int N, int K) {
  return T >= 0 && T <= kDenseMaxT && N >= 1 && N <= MOE_DENSE_MAX && K >= 8 && K <= MOE_DENSE_MAX && K % 8 == 0;
}
inline bool half_type(int dtype) { return dtype == MOE_BF16 || dtype == MOE_F16; }
inline bool aligned2(const void* p) { return ((uintptr_t)p & 1) == 0; }
inline bool aligned256(const void* p) { return ((uintptr_t)p & 255) == 0; }
inline long long padded(int n) { return ((long long)n + 7) / 8 * 8; }

int dense(int kind, int dtype, const DenseOperand& P, const DenseOperand& Q, const DenseArgs& g, cudaStream_t st) {
  return dtype == MOE_BF16 ? dense_product_bf16(kind, P, Q, g, st) : dense_product_f16(kind, P, Q, g, st);
}

// dx = d W and dW = d^T x; d is [T, n] with rows of ldd
int dense_backward(int dtype, const void* d, long long ldd, int T, int n, const void* x, int K, const void* W, void* dx, void* dW,
                   int32_t* status, cudaStream_t st) {
  const DenseOperand P[2] = {{d, false, T, ldd}, {d, true, n, ldd}}, Q[2] = {{W, true, K, K}, {x, true, K, K}};
  const DenseArgs g[2] = {{T, K, n, dx, nullptr, nullptr, nullptr, MOE_ACT_NONE, aligned16(dx), 0, status, 0},
                          {n, K, T, dW, nullptr, nullptr, nullptr, MOE_ACT_NONE, aligned16(dW), 0, status, 0}};
  if (dx && dW) return dtype == MOE_BF16 ? dense_backward_bf16(P, Q, g, st) : dense_backward_f16(P, Q, g, st);
  if (dx) return dense(kDenseDx, dtype, P[0], Q[0], g[0], st);
  return dW ? dense(kDenseDw, dtype, P[1], Q[1], g[1], st) : MOE_OK;
}

}  // namespace moe

using namespace moe;

extern "C" int moe_linear(const void* x, int T, int K, const void* W, int N, int dtype, const void* bias, const void* residual, int act,
                          void* y, void* slope, int32_t* status, moe_stream_t stream) {
  if (!dense_shape_ok(T, N, K) || !half_type(dtype) || act < MOE_ACT_NONE || act > MOE_ACT_GELU_TANH) return MOE_ERR_INVALID_ARG;
  if (T == 0) return MOE_OK;
  if (!x || !W || !y || !aligned16(x) || !aligned16(W) || !aligned2(y) || !aligned2(bias) || !aligned2(residual) || !aligned2(slope))
    return MOE_ERR_INVALID_ARG;
  const bool vec = N % 8 == 0 && aligned16(y) && aligned16(residual) && aligned16(slope);
  DenseArgs g = {T, N, K, y, bias, residual, slope, act, vec, N % 8 == 0 && aligned16(bias), status, 0};
  return dense(kDenseLinear, dtype, {x, false, T, K}, {W, false, N, K}, g, (cudaStream_t)stream);
}

extern "C" int moe_linear_bwd_ws_bytes(int T, int N, int K, size_t* bytes) {
  if (!bytes || !dense_shape_ok(T, N, K)) return MOE_ERR_INVALID_ARG;
  *bytes = (size_t)T * padded(N) * 2;
  return MOE_OK;
}

extern "C" int moe_linear_bwd(const void* dy, const void* x, int T, int K, const void* W, int N, int dtype, const void* slope, void* dx,
                              void* dW, void* dbias, void* ws, size_t ws_bytes, int32_t* status, moe_stream_t stream) {
  if (!dense_shape_ok(T, N, K) || !half_type(dtype)) return MOE_ERR_INVALID_ARG;
  if (!aligned2(dx) || !aligned2(dW) || !aligned2(dbias)) return MOE_ERR_INVALID_ARG;
  cudaStream_t st = (cudaStream_t)stream;
  if (T == 0) {   // sums over no rows
    if (dW && !cuda_ok(cudaMemsetAsync(dW, 0, (size_t)N * K * 2, st))) return MOE_ERR_CUDA;
    if (dbias && !cuda_ok(cudaMemsetAsync(dbias, 0, (size_t)N * 2, st))) return MOE_ERR_CUDA;
    return MOE_OK;
  }
  size_t need = 0;
  moe_linear_bwd_ws_bytes(T, N, K, &need);
  if (!dy || !aligned2(dy) || !aligned2(slope) || !ws || !aligned256(ws) || ws_bytes < need) return MOE_ERR_INVALID_ARG;
  if ((dx && (!W || !aligned16(W))) || (dW && (!x || !aligned16(x)))) return MOE_ERR_INVALID_ARG;
  // without an activation dy itself is d, where the copy engine can read its rows
  const bool direct = !slope && N % 8 == 0 && aligned16(dy);
  const bool products = dx || dW;
  if (dbias || (products && !direct)) {
    void* d = products && !direct ? ws : nullptr;
    const int rc = dtype == MOE_BF16 ? launch_d<__nv_bfloat16>(dy, slope, T, N, d, padded(N), dbias, st)
                                     : launch_d<__half>(dy, slope, T, N, d, padded(N), dbias, st);
    if (rc) return rc;
  }
  return dense_backward(dtype, direct ? dy : ws, padded(N), T, N, x, K, W, dx, dW, status, st);
}

extern "C" int moe_gated(const void* x, int T, int H, const void* W1, int F, int dtype, int act, void* h, void* factors, int32_t* status,
                         moe_stream_t stream) {
  if (F < 1 || F > MOE_DENSE_MAX / 2 || !dense_shape_ok(T, 2 * F, H) || !half_type(dtype) || act < MOE_ACT_NONE || act > MOE_ACT_GELU_TANH)
    return MOE_ERR_INVALID_ARG;
  if (T == 0) return MOE_OK;
  if (!x || !W1 || !h || !aligned16(x) || !aligned16(W1) || !aligned2(h) || !aligned2(factors)) return MOE_ERR_INVALID_ARG;
  DenseArgs g = {T, F, H, h, nullptr, nullptr, factors, act, F % 8 == 0 && aligned16(h) && aligned16(factors), 0, status, 0};
  return dense(kDenseGated, dtype, {x, false, T, H}, {W1, false, 2LL * F, H}, g, (cudaStream_t)stream);
}

extern "C" int moe_gated_bwd_ws_bytes(int T, int F, int H, size_t* bytes) {
  if (!bytes || F < 1 || F > MOE_DENSE_MAX / 2 || !dense_shape_ok(T, 2 * F, H)) return MOE_ERR_INVALID_ARG;
  *bytes = (size_t)T * padded(2 * F) * 2;
  return MOE_OK;
}

extern "C" int moe_gated_bwd(const void* dh, const void* x, int T, int H, const void* W1, int F, int dtype, const void* factors, void* dx,
                             void* dW1, void* ws, size_t ws_bytes, int32_t* status, moe_stream_t stream) {
  if (F < 1 || F > MOE_DENSE_MAX / 2 || !dense_shape_ok(T, 2 * F, H) || !half_type(dtype)) return MOE_ERR_INVALID_ARG;
  if (!aligned2(dx) || !aligned2(dW1)) return MOE_ERR_INVALID_ARG;
  cudaStream_t st = (cudaStream_t)stream;
  if (T == 0) {   // sums over no rows
    if (dW1 && !cuda_ok(cudaMemsetAsync(dW1, 0, (size_t)2 * F * H * 2, st))) return MOE_ERR_CUDA;
    return MOE_OK;
  }
  size_t need = 0;
  moe_gated_bwd_ws_bytes(T, F, H, &need);
  if (!dh || !factors || !aligned2(dh) || !aligned2(factors) || !ws || !aligned256(ws) || ws_bytes < need) return MOE_ERR_INVALID_ARG;
  if ((dx && (!W1 || !aligned16(W1))) || (dW1 && (!x || !aligned16(x)))) return MOE_ERR_INVALID_ARG;
  if (!dx && !dW1) return MOE_OK;
  const int rc = dtype == MOE_BF16 ? launch_gated_d<__nv_bfloat16>(dh, factors, T, F, ws, padded(2 * F), st)
                                   : launch_gated_d<__half>(dh, factors, T, F, ws, padded(2 * F), st);
  if (rc) return rc;
  return dense_backward(dtype, ws, padded(2 * F), T, 2 * F, x, H, W1, dx, dW1, status, st);
}
