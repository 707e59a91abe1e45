// few.cu: entry points of the decoding kernels: 4-bit matrix-vector products and a
// whole MoE layer for a few tokens.
#include "few_host.h"
#include "w4.cuh"

using namespace moe;

extern "C" int moe_matvec_w4(const uint16_t* x, int T, int K, const uint8_t* Wp, int N, int group, uint16_t* y,
                             int32_t* status, moe_stream_t stream) {
  if (!x || !Wp || !y || !status || !aligned16(x) || !aligned16(Wp) || ((uintptr_t)y & 1)) return MOE_ERR_INVALID_ARG;
  if (T < 1 || T > MOE_FEW_MAX_TOKENS) return MOE_ERR_INVALID_ARG;
  size_t bytes;
  const int rc = moe_w4_packed_bytes(N, K, group, &bytes);
  if (rc) return rc;
  const int nsm = device_sm_count();
  if (nsm <= 0) return MOE_ERR_CUDA;
  MatvecArgs a{x, Wp, y, status, T, N, K, 0};
  cudaStream_t s = (cudaStream_t)stream;
  return group == 32 ? launch_matvec<32>(a, nsm, s) : group == 64 ? launch_matvec<64>(a, nsm, s) : launch_matvec<128>(a, nsm, s);
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
  const int nsm = device_sm_count();
  if (nsm <= 0) return MOE_ERR_CUDA;
  LayerArgs a;
  a.x = x; a.router = router;
  a.W1 = W1; a.W2 = W2; a.W1_scale = W1_scale; a.W2_scale = W2_scale;
  a.ids = topk_ids; a.w = topk_w; a.out = out;
  a.counters = reinterpret_cast<int32_t*>(ws);
  a.logits = reinterpret_cast<float*>((char*)ws + 256);
  a.h = reinterpret_cast<uint16_t*>((char*)ws + 256 + few_logits_bytes(T, E));
  a.status = status;
  a.T = T; a.H = H; a.E = E; a.k = k; a.F = F;
  cudaStream_t s = (cudaStream_t)stream;
  switch (group) {
    case 0: return launch_layer<0>(a, nsm, s);
    case 32: return launch_layer<32>(a, nsm, s);
    case 64: return launch_layer<64>(a, nsm, s);
    default: return launch_layer<128>(a, nsm, s);
  }
}
