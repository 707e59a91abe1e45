// dense_host.cuh: the launches of one dense product, for one 16-bit type.
#pragma once

#include "dense_few.cuh"
#include "dense_pair.cuh"
#include "dense_plan.h"
#include "host_util.h"

namespace moe {

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

// CTAs that the device holds at once in clusters of c; 0 where it cannot be said.
template <typename K>
int resident_ctas(K kernel, int threads, size_t smem, int c) {
  if (cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, 227 * 1024) != cudaSuccess) return 0;
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
  return cudaOccupancyMaxActiveClusters(&n, kernel, &cfg) == cudaSuccess ? n * c : 0;
}

// What the device holds, by one of the kernels (all take the same threads and shared memory).  Asked once.
template <typename K, typename P>
DenseDevice dense_device(K few, P pair) {
  DenseDevice d = {};
  d.sms = device_sm_count();
  d.pairs = std::min(resident_ctas(pair, kDPairThreads, kDPairSmemBytes, 2), d.sms) / 2;
  for (int c = 1; c <= kDFewMaxSplit; ++c) {
    d.cta[0][c] = resident_ctas(few, kDFewThreads, dfew_smem_bytes(128, 6), c);
    d.cta[1][c] = 2 * d.cta[0][c];   // (of kernels with tensor memory the query says one a SM whatever their size; two run)
  }
  return d;
}

template <typename T, bool PMN, bool QMN, int EPI, bool AUX>
int launch_pair(const CUtensorMap& tmP, const CUtensorMap& tmQ, const DenseArgs& g, int pairs, cudaStream_t st) {
  auto kernel = dense_pair_kernel<T, PMN, QMN, EPI, AUX>;
  static const cudaError_t attr = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)kDPairSmemBytes);
  if (attr != cudaSuccess) return MOE_ERR_CUDA;
  constexpr int kTileJ = EPI == kEpiGated ? 128 : 256;
  const long long tiles = ((long long)g.I + 255) / 256 * (((long long)g.J + kTileJ - 1) / kTileJ);
  if (tiles > 0x3FFFFFFF) return MOE_ERR_UNSUPPORTED;
  return launch_next(kernel, dim3(2 * (unsigned)std::min<long long>(pairs, tiles)), kDPairThreads, kDPairSmemBytes, st, 2, 1, tmP, tmQ, g);
}

template <typename T, bool PMN, bool QMN, int EPI>
int launch_dense(const DenseOperand& P, const DenseOperand& Q, DenseArgs g, cudaStream_t st) {
  if (!device_has_tcgen05()) return MOE_ERR_UNSUPPORTED;
  auto kernel = dense_few_kernel<T, PMN, QMN, EPI>;
  static const DenseDevice device = dense_device(kernel, dense_pair_kernel<T, PMN, QMN, EPI, false>);
  if (device.pairs < 1) return MOE_ERR_CUDA;
  g.timeout_ns = 2000000000ull;
  const DensePlan plan = dense_plan({g.I, g.J, g.K, EPI == kEpiGated, PMN, g.aux != nullptr, g.residual != nullptr, g.vec != 0}, device);
  CUtensorMap tmP, tmQ;
  if (plan.pair) {
    if (!encode_operand<T>(&tmP, P, g.K, 128) || !encode_operand<T>(&tmQ, Q, g.K, 128)) return MOE_ERR_CUDA;
    if (EPI != kEpiPlain && g.aux) return launch_pair<T, PMN, QMN, EPI, EPI != kEpiPlain>(tmP, tmQ, g, device.pairs, st);
    return launch_pair<T, PMN, QMN, EPI, false>(tmP, tmQ, g, device.pairs, st);
  }
  if (!encode_operand<T>(&tmP, P, g.K, plan.nt) || !encode_operand<T>(&tmQ, Q, g.K, EPI == kEpiGated ? 64 : 128)) return MOE_ERR_CUDA;
  constexpr int kRows = EPI == kEpiGated ? 64 : 128;
  DFewPlan fp;
  fp.nt = plan.nt;
  fp.stages = plan.stages;
  fp.split = plan.split;
  fp.ti = (int)(((long long)g.I + plan.nt - 1) / plan.nt);
  const long long ctas = (long long)fp.ti * (((long long)g.J + kRows - 1) / kRows) * plan.split;
  if (ctas > 0x7FFFFFFF) return MOE_ERR_UNSUPPORTED;
  return launch_next(kernel, dim3((unsigned)ctas), kDFewThreads, dfew_smem_bytes(plan.nt, plan.stages), st, (unsigned)plan.split, 1, tmP, tmQ, g, fp);
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

}  // namespace moe
