// dense_host.cuh: the launches of one dense product, for one 16-bit type.
#pragma once

#include "dense_few.cuh"
#include "dense_pair.cuh"
#include "dense_plan.h"
#include "host_util.h"

namespace moe {

constexpr uint64_t kDenseTimeoutNs = 2000000000ull;

// One operand: `rows` of i (or j) by g.K of k; ld is the length of its rows in memory.
struct DenseOperand {
  const void* p;
  bool mn;         // rows contiguous in memory, k strided
  long long rows, ld;
};

// Swizzled map of one operand: boxes of 64 k x `box` rows, or 64 rows x 64 k.
template <typename T>
bool encode_operand(CUtensorMap* map, const DenseOperand& o, int K, int box) {
  auto enc = tensor_map_encoder();
  if (!enc) return false;
  cuuint64_t d[2] = {(cuuint64_t)(o.mn ? o.rows : K), (cuuint64_t)(o.mn ? K : o.rows)}, s[1] = {(cuuint64_t)o.ld * 2};
  cuuint32_t b[2] = {64, (cuuint32_t)(o.mn ? 64 : box)}, es[2] = {1, 1};
  return enc(map, std::is_same<T, __half>::value ? CU_TENSOR_MAP_DATA_TYPE_FLOAT16 : CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 2,
             const_cast<void*>(o.p), d, s, b, es, CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B,
             CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

// CTAs that the device holds at once in clusters of c; below 0 where it cannot be said.
template <typename K>
int resident_ctas(K kernel, int threads, size_t smem, int c) {
  cudaLaunchConfig_t cfg = {};
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim.x = (unsigned)c;
  attr[0].val.clusterDim.y = attr[0].val.clusterDim.z = 1;
  cfg.gridDim = dim3((unsigned)(c * 512));
  cfg.blockDim = dim3((unsigned)threads);
  cfg.dynamicSmemBytes = smem;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  int n = 0;
  return cuda_ok(cudaOccupancyMaxActiveClusters(&n, kernel, &cfg)) ? n * c : -1;
}

// What the current device holds, by one of the kernels (all take the same threads and shared memory),
// whose limits of shared memory are set there; its status.
template <typename K, typename P>
int ask_device(K few, P pair, DenseDevice* d) {
  if (!device_has_tcgen05()) return MOE_ERR_UNSUPPORTED;
  if (!cuda_ok(cudaFuncSetAttribute(few, cudaFuncAttributeMaxDynamicSharedMemorySize, 227 * 1024)) ||
      !cuda_ok(cudaFuncSetAttribute(pair, cudaFuncAttributeMaxDynamicSharedMemorySize, 227 * 1024)))
    return MOE_ERR_CUDA;
  d->sms = device_sm_count();
  d->pairs = std::min(resident_ctas(pair, kDPairThreads, kDPairSmemBytes, 2), d->sms) / 2;
  if (d->pairs < 1) return MOE_ERR_CUDA;
  for (int c = 1; c <= kDFewMaxSplit; ++c) {
    const int n = resident_ctas(few, kDFewThreads, dfew_smem_bytes(128, 6), c);
    if (n < 0) return MOE_ERR_CUDA;
    d->cta[0][c] = n;
    d->cta[1][c] = 2 * n;   // (of kernels with tensor memory the query says one a SM whatever their size; two run)
  }
  return MOE_OK;
}

// Asked once on each device.
class DenseDevices {
 public:
  template <typename K, typename P>
  int get(int dev, K few, P pair, DenseDevice* d) {
    if (dev >= 64) return ask_device(few, pair, d);
    int rc = MOE_ERR_CUDA;
    if (!once_(dev, [&] { return (rc = ask_device(few, pair, &kept_[dev])) == MOE_OK; })) return rc;
    *d = kept_[dev];
    return MOE_OK;
  }

 private:
  OncePerDevice once_;
  DenseDevice kept_[64];
};

template <typename T, bool PMN, bool QMN, int EPI, bool AUX>
int launch_pair(const CUtensorMap& tmP, const CUtensorMap& tmQ, const DenseArgs& g, int pairs, cudaStream_t st) {
  auto kernel = dense_pair_kernel<T, PMN, QMN, EPI, AUX>;
  static OncePerDevice limit;
  if (!limit(current_device(), [&] { return cuda_ok(cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)kDPairSmemBytes)); }))
    return MOE_ERR_CUDA;
  constexpr int kTileJ = EPI == kEpiGated ? 128 : 256;
  const long long tiles = ((long long)g.I + 255) / 256 * (((long long)g.J + kTileJ - 1) / kTileJ);
  if (tiles > 0x3FFFFFFF) return MOE_ERR_UNSUPPORTED;
  return launch_next(kernel, dim3(2 * (unsigned)std::min<long long>(pairs, tiles)), kDPairThreads, kDPairSmemBytes, st, 2, 1, tmP, tmQ, g);
}

inline DenseShape shape_of(const DenseArgs& g, bool gated, bool p_mn) {
  return {g.I, g.J, g.K, gated, p_mn, g.aux != nullptr, g.residual != nullptr, g.vec != 0};
}

// The plans of the shapes that a thread asked for last (a plan takes longer than a launch), each for its device.
struct DensePlans {
  int device;
  DenseShape shape[2];
  DensePlan plan[2];
  bool both;
};

// The kernel's form of a plan; the CTAs that it takes, in whole clusters.
inline long long few_ctas(const DenseArgs& g, const DensePlan& plan, int rows, int cluster, DFewPlan* fp) {
  fp->nt = plan.nt;
  fp->stages = plan.stages;
  fp->split = plan.split;
  fp->cluster = cluster;
  fp->ti = (int)(((long long)g.I + plan.nt - 1) / plan.nt);
  const long long tiles = (long long)fp->ti * (((long long)g.J + rows - 1) / rows);
  fp->tiles = (int)std::min<long long>(tiles, 0x7FFFFFFF);
  return (tiles * plan.split + cluster - 1) / cluster * cluster;
}

template <typename T, bool PMN, bool QMN, int EPI>
int launch_dense(const DenseOperand& P, const DenseOperand& Q, DenseArgs g, cudaStream_t st) {
  auto kernel = dense_few_kernel<T, PMN, QMN, EPI>;
  static DenseDevices devices;
  const int dev = current_device();
  DenseDevice device;
  if (const int rc = devices.get(dev, kernel, dense_pair_kernel<T, PMN, QMN, EPI, false>, &device)) return rc;
  g.timeout_ns = kDenseTimeoutNs;
  const DenseShape shape = shape_of(g, EPI == kEpiGated, PMN);
  static thread_local DensePlans kept[kPlanSlots] = {};
  DensePlans& at = kept[plan_slot(shape)];
  if (at.device != dev || !same_shape(at.shape[0], shape)) {
    at.plan[0] = dense_plan(shape, device);
    at.device = dev;
    at.shape[0] = shape;
  }
  const DensePlan plan = at.plan[0];
  CUtensorMap tmP, tmQ;
  if (plan.pair) {
    if (!encode_operand<T>(&tmP, P, g.K, 128) || !encode_operand<T>(&tmQ, Q, g.K, 128)) return MOE_ERR_CUDA;
    if (EPI != kEpiPlain && g.aux) return launch_pair<T, PMN, QMN, EPI, EPI != kEpiPlain>(tmP, tmQ, g, device.pairs, st);
    return launch_pair<T, PMN, QMN, EPI, false>(tmP, tmQ, g, device.pairs, st);
  }
  if (!encode_operand<T>(&tmP, P, g.K, plan.nt) || !encode_operand<T>(&tmQ, Q, g.K, EPI == kEpiGated ? 64 : 128)) return MOE_ERR_CUDA;
  DFewPlan fp;
  const long long ctas = few_ctas(g, plan, EPI == kEpiGated ? 64 : 128, plan.split, &fp);
  if (ctas > 0x7FFFFFFF) return MOE_ERR_UNSUPPORTED;
  return launch_next(kernel, dim3((unsigned)ctas), kDFewThreads, dfew_smem_bytes(plan.nt, plan.stages), st, (unsigned)plan.split, 1, tmP, tmQ, g, fp);
}

// dx = d W and dW = d^T x, in one launch where that is quicker
template <typename T>
int launch_backward(const DenseOperand (&P)[2], const DenseOperand (&Q)[2], const DenseArgs (&g)[2], cudaStream_t st) {
  auto kernel = dense_both_kernel<T>;
  static DenseDevices devices;
  const int dev = current_device();
  DenseDevice device;
  if (const int rc = devices.get(dev, kernel, dense_pair_kernel<T, false, true, kEpiPlain, false>, &device)) return rc;
  const DenseShape s[2] = {shape_of(g[0], false, false), shape_of(g[1], false, true)};
  static thread_local DensePlans kept[kPlanSlots] = {};
  DensePlans& at = kept[plan_slot(s[0])];
  if (at.device != dev || !same_shape(at.shape[0], s[0]) || !same_shape(at.shape[1], s[1])) {
    at.both = dense_plan_both(s, device, at.plan);
    at.device = dev;
    at.shape[0] = s[0];
    at.shape[1] = s[1];
  }
  const DensePlan(&plan)[2] = at.plan;
  if (!at.both) {
    const int rc = launch_dense<T, false, true, kEpiPlain>(P[0], Q[0], g[0], st);
    return rc ? rc : launch_dense<T, true, true, kEpiPlain>(P[1], Q[1], g[1], st);
  }
  const int cluster = std::max(plan[0].split, plan[1].split);
  DBoth b;
  long long ctas[2];
  for (int i = 0; i < 2; ++i) {
    if (!encode_operand<T>(&b.P[i], P[i], g[i].K, plan[i].nt) || !encode_operand<T>(&b.Q[i], Q[i], g[i].K, 128)) return MOE_ERR_CUDA;
    b.g[i] = g[i];
    b.g[i].timeout_ns = kDenseTimeoutNs;
    ctas[i] = few_ctas(g[i], plan[i], 128, cluster, &b.plan[i]);
  }
  if (ctas[0] + ctas[1] > 0x7FFFFFFF) return MOE_ERR_UNSUPPORTED;
  b.first = (int)ctas[0];
  const size_t smem = std::max(dfew_smem_bytes(plan[0].nt, plan[0].stages), dfew_smem_bytes(plan[1].nt, plan[1].stages));
  return launch_next(kernel, dim3((unsigned)(ctas[0] + ctas[1])), kDFewThreads, smem, st, (unsigned)cluster, 1, b);
}

// The products that the operators take: x W^T (linear, gated), d W and d^T x.
enum { kDenseLinear = 0, kDenseGated = 1, kDenseDx = 2, kDenseDw = 3 };

template <typename T>
int dense_product(int kind, const DenseOperand& P, const DenseOperand& Q, const DenseArgs& g, cudaStream_t st) {
  switch (kind) {
    case kDenseLinear: return launch_dense<T, false, false, kEpiLinear>(P, Q, g, st);
    case kDenseGated: return launch_dense<T, false, false, kEpiGated>(P, Q, g, st);
    case kDenseDx: return launch_dense<T, false, true, kEpiPlain>(P, Q, g, st);
    default: return launch_dense<T, true, true, kEpiPlain>(P, Q, g, st);
  }
}

int dense_product_bf16(int kind, const DenseOperand& P, const DenseOperand& Q, const DenseArgs& g, cudaStream_t st);
int dense_product_f16(int kind, const DenseOperand& P, const DenseOperand& Q, const DenseArgs& g, cudaStream_t st);
int dense_backward_bf16(const DenseOperand (&P)[2], const DenseOperand (&Q)[2], const DenseArgs (&g)[2], cudaStream_t st);
int dense_backward_f16(const DenseOperand (&P)[2], const DenseOperand (&Q)[2], const DenseArgs (&g)[2], cudaStream_t st);

}  // namespace moe
