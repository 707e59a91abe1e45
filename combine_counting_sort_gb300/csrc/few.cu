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
  MatvecArgs a = {};
  a.x = x; a.W = Wp; a.y = y; a.status = status;
  a.T = T; a.N = N; a.K = K;
  cudaStream_t s = (cudaStream_t)stream;
  return group == 32 ? launch_matvec<32>(a, nsm, s) : group == 64 ? launch_matvec<64>(a, nsm, s) : launch_matvec<128>(a, nsm, s);
}

// Workspace: 256 bytes of counters, then what LayerArgs names, each at a multiple of 256 bytes.
constexpr int kFewMaxSplits = 4;   // kRouterMaxRuns
struct FewWorkspace {
  size_t logits, x8, h8, h, bytes;
  FewWorkspace(int T, int k, int E, int H, int F) {
    size_t at = 256;
    auto take = [&at](size_t n) { const size_t p = at; at += (n + 255) / 256 * 256; return p; };
    logits = take((size_t)kFewMaxSplits * T * E * 4);
    x8 = take((size_t)T * (H / 128) * kTokenRecord);
    h8 = take((size_t)T * k * (F / 128) * kTokenRecord);
    h = take((size_t)T * k * F * 4);
    bytes = at;
  }
};

// The FP8 weights of all experts as {128 bytes, rows, slices of 128 columns}; a box
// holds 16 rows of up to 8 slices.
static bool weight_map(CUtensorMap* map, const uint8_t* W, int E, int N, int K) {
  const uint64_t dims[3] = {128, (uint64_t)E * N, (uint64_t)(K / 128)}, strides[2] = {(uint64_t)K, 128};
  const uint32_t box[3] = {128, 16, (uint32_t)std::min(8, K / 128)};
  return encode_u8_map(map, W, 3, dims, strides, box);
}

static int check_few(int T, int k, int E, int H, int F) {
  if (T < 1 || T > MOE_FEW_MAX_TOKENS || k < 1 || k > 32 || T * k > MOE_FEW_MAX_PAIRS || E < k || E > 1024) return MOE_ERR_INVALID_ARG;
  if (H < 128 || H % 128 || H > 32768 || F < 128 || F % 128 || F > 32768) return MOE_ERR_INVALID_ARG;
  return MOE_OK;
}

extern "C" int moe_layer_few_ws_bytes(int T, int k, int E, int H, int F, size_t* bytes) {
  if (!bytes) return MOE_ERR_INVALID_ARG;
  const int rc = check_few(T, k, E, H, F);
  if (rc) return rc;
  *bytes = FewWorkspace(T, k, E, H, F).bytes;
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
  LayerArgs a = {};
  a.x = x; a.router = router;
  a.W1 = W1; a.W2 = W2; a.W1_scale = W1_scale; a.W2_scale = W2_scale;
  a.ids = topk_ids; a.w = topk_w; a.out = out;
  a.counters = reinterpret_cast<int32_t*>(ws);
  const FewWorkspace at(T, k, E, H, F);
  char* base = reinterpret_cast<char*>(ws);
  a.logits = reinterpret_cast<float*>(base + at.logits);
  a.x8 = reinterpret_cast<uint8_t*>(base + at.x8);
  a.h8 = reinterpret_cast<uint8_t*>(base + at.h8);
  a.h = reinterpret_cast<float*>(base + at.h);
  a.status = status;
  a.T = T; a.H = H; a.E = E; a.k = k; a.F = F;
  // the logits' units fill the grid once if there are few
  a.splits = std::max(1, std::min(kFewMaxSplits, nsm / ((E + 15) / 16 * ((T + 7) / 8))));
  cudaStream_t s = (cudaStream_t)stream;
  switch (group) {
    case 0:
      if (!weight_map(&a.map1, W1, E, 2 * F, H) || !weight_map(&a.map2, W2, E, H, F)) return MOE_ERR_CUDA;
      return launch_layer<0>(a, nsm, s);
    case 32: return launch_layer<32>(a, nsm, s);
    case 64: return launch_layer<64>(a, nsm, s);
    default: return launch_layer<128>(a, nsm, s);
  }
}
