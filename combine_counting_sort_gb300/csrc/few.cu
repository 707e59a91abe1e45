// few.cu: decoding kernels: 4-bit matrix-vector products and a whole MoE layer
// for a few tokens.
#include "host_util.h"
#include "w4.cuh"

namespace moe {

// Column k of row n of a weight matrix, either form.
struct WeightView {
  const uint8_t* p;
  const float* scale;   // FP8 only
  int N, K, group;      // group 0: FP8 with 128 x 128 scales
  MOE_DEV WeightView expert(int e) const {
    WeightView v = *this;
    if (group == 0) {
      v.p += (size_t)e * N * K;
      v.scale += (size_t)e * (N / 128) * (K / 128);
    } else {
      v.p += (size_t)e * w4_matrix_bytes(N, K, group);
    }
    return v;
  }
  MOE_DEV float at(int n, int k) const {
    if (group == 0) return e4m3x2_to_float2(p[(size_t)n * K + k]).x * scale[(size_t)(n / 128) * (K / 128) + k / 128];
    return w4_value(p + ((size_t)(n / 16) * ((K + 127) / 128) + k / 128) * w4_tile_bytes(group), n % 16, k % 128, group);
  }
};

MOE_DEV float warp_sum(float v) {
  for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
  return v;
}
MOE_DEV float bf16_at(const uint16_t* p, size_t i) { return bf16_lo(p[i]); }
MOE_DEV uint16_t to_bf16(float v) {
  const __nv_bfloat16 b = __float2bfloat16_rn(v);
  return *reinterpret_cast<const uint16_t*>(&b);
}

// One warp per output value.
__global__ void __launch_bounds__(256) matvec_kernel(const uint16_t* __restrict__ x, int T, WeightView W,
                                                     uint16_t* __restrict__ y) {
  const int n = blockIdx.x * 8 + (threadIdx.x >> 5), t = blockIdx.y, lane = threadIdx.x & 31;
  if (n >= W.N) return;
  float s = 0.f;
  for (int k = lane; k < W.K; k += 32) s = fmaf(bf16_at(x, (size_t)t * W.K + k), W.at(n, k), s);
  s = warp_sum(s);
  if (lane == 0) y[(size_t)t * W.N + n] = to_bf16(s);
}

__global__ void __launch_bounds__(256) few_logits_kernel(const uint16_t* __restrict__ x, int H, const uint16_t* __restrict__ router,
                                                         int E, float* __restrict__ logits) {
  const int e = blockIdx.x * 8 + (threadIdx.x >> 5), t = blockIdx.y, lane = threadIdx.x & 31;
  if (e >= E) return;
  float s = 0.f;
  for (int k = lane; k < H; k += 32) s = fmaf(bf16_at(x, (size_t)t * H + k), bf16_at(router, (size_t)e * H + k), s);
  s = warp_sum(s);
  if (lane == 0) logits[(size_t)t * E + e] = s;
}

// a[pair, f] = bf16(w * silu(gate) * up); one warp per value.
__global__ void __launch_bounds__(256) few_gate_up_kernel(const uint16_t* __restrict__ x, int k, int E, WeightView W1,
                                                          const int32_t* __restrict__ ids, const float* __restrict__ w,
                                                          uint16_t* __restrict__ a, int32_t* status) {
  const int F = W1.N / 2, H = W1.K;
  const int f = blockIdx.x * 8 + (threadIdx.x >> 5), p = blockIdx.y, lane = threadIdx.x & 31;
  const int e = ids[p];
  if (e >= E && lane == 0) set_status(status, MOE_ERR_EXPERT_ID);
  if (e < 0 || e >= E || f >= F) return;
  const WeightView W = W1.expert(e);
  float g = 0.f, u = 0.f;
  for (int c = lane; c < H; c += 32) {
    const float v = bf16_at(x, (size_t)(p / k) * H + c);
    g = fmaf(v, W.at(f, c), g);
    u = fmaf(v, W.at(F + f, c), u);
  }
  g = warp_sum(g);
  u = warp_sum(u);
  if (lane == 0) a[(size_t)p * F + f] = to_bf16(g / (1.f + expf(-g)) * u * w[p]);
}

__global__ void __launch_bounds__(256) few_down_kernel(const uint16_t* __restrict__ a, int k, int E, WeightView W2,
                                                       const int32_t* __restrict__ ids, uint16_t* __restrict__ out) {
  const int H = W2.N, F = W2.K;
  const int h = blockIdx.x * 8 + (threadIdx.x >> 5), t = blockIdx.y, lane = threadIdx.x & 31;
  if (h >= H) return;
  float s = 0.f;
  for (int j = 0; j < k; ++j) {
    const int e = ids[t * k + j];
    if (e < 0 || e >= E) continue;
    const WeightView W = W2.expert(e);
    for (int c = lane; c < F; c += 32) s = fmaf(bf16_at(a, (size_t)(t * k + j) * F + c), W.at(h, c), s);
  }
  s = warp_sum(s);
  if (lane == 0) out[(size_t)t * H + h] = to_bf16(s);
}

}  // namespace moe

using namespace moe;

extern "C" int moe_matvec_w4(const uint16_t* x, int T, int K, const uint8_t* Wp, int N, int group, uint16_t* y,
                             int32_t* status, moe_stream_t stream) {
  if (!x || !Wp || !y || !status || !aligned16(x) || !aligned16(Wp) || ((uintptr_t)y & 1)) return MOE_ERR_INVALID_ARG;
  if (T < 1 || T > MOE_FEW_MAX_TOKENS) return MOE_ERR_INVALID_ARG;
  size_t bytes;
  const int rc = moe_w4_packed_bytes(N, K, group, &bytes);
  if (rc) return rc;
  matvec_kernel<<<dim3((N + 7) / 8, T), 256, 0, (cudaStream_t)stream>>>(x, T, WeightView{Wp, nullptr, N, K, group}, y);
  return cudaGetLastError() == cudaSuccess ? MOE_OK : MOE_ERR_CUDA;
}

// Workspace: 256 bytes of counters, the logits, then the activations.
static size_t few_logits_bytes(int T, int E) { return ((size_t)T * E * 4 + 255) / 256 * 256; }

static int check_few(int T, int k, int E, int H, int F) {
  if (T < 1 || T > MOE_FEW_MAX_TOKENS || k < 1 || k > 32 || T * k > MOE_FEW_MAX_PAIRS || E < k || E > 1024) return MOE_ERR_INVALID_ARG;
  if (H < 128 || H % 128 || H > 32768 || F < 128 || F % 128 || F > 32768) return MOE_ERR_INVALID_ARG;
  return MOE_OK;
}

extern "C" int moe_layer_few_ws_bytes(int T, int k, int E, int H, int F, size_t* bytes) {
  if (!bytes) return MOE_ERR_INVALID_ARG;
  const int rc = check_few(T, k, E, H, F);
  if (rc) return rc;
  *bytes = 256 + few_logits_bytes(T, E) + (size_t)T * k * F * 2;
  return MOE_OK;
}

extern "C" int moe_layer_few(const uint16_t* x, int T, int H, const uint16_t* router, int E, int k, const uint8_t* W1,
                             const float* W1_scale, const uint8_t* W2, const float* W2_scale, int F, int group,
                             int32_t* topk_ids, float* topk_w, uint16_t* out, void* ws, size_t ws_bytes,
                             int32_t* status, moe_stream_t stream) {
  size_t need;
  int rc = moe_layer_few_ws_bytes(T, k, E, H, F, &need);
  if (rc) return rc;
  if (!x || !W1 || !W2 || !topk_ids || !topk_w || !out || !ws || !status || ws_bytes < need) return MOE_ERR_INVALID_ARG;
  if (group != 0 && !w4_group_ok(group)) return MOE_ERR_INVALID_ARG;
  if ((group == 0) != (W1_scale != nullptr) || (group == 0) != (W2_scale != nullptr)) return MOE_ERR_INVALID_ARG;
  if (!aligned16(x) || !aligned16(router) || !aligned16(W1) || !aligned16(W2) || !aligned16(W1_scale) ||
      !aligned16(W2_scale) || !aligned16(out) || ((uintptr_t)ws & 255))
    return MOE_ERR_INVALID_ARG;
  cudaStream_t s = (cudaStream_t)stream;
  float* logits = reinterpret_cast<float*>((char*)ws + 256);
  uint16_t* a = reinterpret_cast<uint16_t*>((char*)ws + 256 + few_logits_bytes(T, E));
  if (router) {
    few_logits_kernel<<<dim3((E + 7) / 8, T), 256, 0, s>>>(x, H, router, E, logits);
    rc = moe_router_topk(logits, T, E, k, topk_ids, topk_w, stream);
    if (rc) return rc;
  }
  few_gate_up_kernel<<<dim3((F + 7) / 8, T * k), 256, 0, s>>>(x, k, E, WeightView{W1, W1_scale, 2 * F, H, group}, topk_ids,
                                                              topk_w, a, status);
  few_down_kernel<<<dim3((H + 7) / 8, T), 256, 0, s>>>(a, k, E, WeightView{W2, W2_scale, H, F, group}, topk_ids, out);
  return cudaGetLastError() == cudaSuccess ? MOE_OK : MOE_ERR_CUDA;
}
