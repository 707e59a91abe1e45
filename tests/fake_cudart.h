// A CUDA runtime that launches nothing, for tests of the library's host code on a machine without a GPU:
// linked with the library's own objects in place of libcudart.  Devices differ in their SMs; what a device
// refuses a real one refuses too (more dynamic shared memory than the kernel was given there).
#pragma once

#include <cuda.h>
#include <cuda_runtime.h>
#include <stdint.h>
#include <stdio.h>
#include <stdlib.h>

#include <map>
#include <utility>
#include <vector>

struct FakeLaunch {
  int device;
  const void* kernel;
  dim3 grid, block;
  size_t smem;
};

struct FakeCuda {
  int device = 0;
  int sms[4] = {152, 20, 152, 152};
  int fail_attribute = 0, fail_occupancy = 0, fail_launch = 0;   // so many of the next calls fail
  cudaError_t last = cudaSuccess;
  std::map<std::pair<int, const void*>, size_t> limit;
  std::vector<FakeLaunch> launches;
  cudaError_t done(cudaError_t e) {
    if (e != cudaSuccess) last = e;
    return e;
  }
  size_t allowed(const void* kernel) {
    auto it = limit.find({device, kernel});
    return it == limit.end() ? 48 * 1024 : it->second;
  }
};
inline FakeCuda& fake() {
  static FakeCuda f;
  return f;
}

extern "C" {
cudaError_t cudaGetDevice(int* d) { *d = fake().device; return cudaSuccess; }
cudaError_t cudaGetLastError() { const cudaError_t e = fake().last; fake().last = cudaSuccess; return e; }
cudaError_t cudaDeviceGetAttribute(int* v, cudaDeviceAttr a, int dev) {
  if (a == cudaDevAttrMultiProcessorCount) *v = fake().sms[dev];
  else if (a == cudaDevAttrComputeCapabilityMajor) *v = 10;
  else return fake().done(cudaErrorInvalidValue);
  return cudaSuccess;
}
cudaError_t cudaFuncSetAttribute(const void* f, cudaFuncAttribute a, int v) {
  if (fake().fail_attribute > 0 && fake().fail_attribute--) return fake().done(cudaErrorMemoryAllocation);
  if (a == cudaFuncAttributeMaxDynamicSharedMemorySize) fake().limit[{fake().device, f}] = (size_t)v;
  return cudaSuccess;
}
cudaError_t cudaOccupancyMaxActiveClusters(int* n, const void* f, const cudaLaunchConfig_t* c) {
  if (fake().fail_occupancy > 0 && fake().fail_occupancy--) return fake().done(cudaErrorMemoryAllocation);
  if (c->dynamicSmemBytes > fake().allowed(f)) return fake().done(cudaErrorInvalidValue);
  *n = fake().sms[fake().device] / (int)c->attrs[0].val.clusterDim.x;
  return cudaSuccess;
}
cudaError_t cudaLaunchKernelExC(const cudaLaunchConfig_t* c, const void* f, void**) {
  if (fake().fail_launch > 0 && fake().fail_launch--) return fake().done(cudaErrorInvalidResourceHandle);
  if (c->dynamicSmemBytes > fake().allowed(f)) return fake().done(cudaErrorInvalidValue);
  fake().launches.push_back({fake().device, f, c->gridDim, c->blockDim, c->dynamicSmemBytes});
  return cudaSuccess;
}
cudaError_t cudaMemsetAsync(void*, int, size_t, cudaStream_t) { return cudaSuccess; }
static CUresult fake_encode(CUtensorMap*, CUtensorMapDataType, cuuint32_t, void*, const cuuint64_t*, const cuuint64_t*, const cuuint32_t*,
                            const cuuint32_t*, CUtensorMapInterleave, CUtensorMapSwizzle, CUtensorMapL2promotion, CUtensorMapFloatOOBfill) {
  return CUDA_SUCCESS;
}
cudaError_t cudaGetDriverEntryPointByVersion(const char*, void** p, unsigned, unsigned long long, cudaDriverEntryPointQueryResult* q) {
  *p = (void*)fake_encode;
  if (q) *q = cudaDriverEntryPointSuccess;
  return cudaSuccess;
}
// what the compiler's own start-up code and <<< >>> call
void** __cudaRegisterFatBinary(void*) { static void* h; return &h; }
void __cudaRegisterFatBinaryEnd(void**) {}
void __cudaUnregisterFatBinary(void**) {}
void __cudaRegisterFunction(void**, const char*, char*, const char*, int, uint3*, uint3*, dim3*, dim3*, int*) {}
unsigned __cudaPushCallConfiguration(dim3, dim3, size_t, void*) { return 0; }
cudaError_t __cudaPopCallConfiguration(dim3*, dim3*, size_t*, void*) { return cudaSuccess; }
cudaError_t __cudaGetKernel(void**, const void*) { return cudaSuccess; }
cudaError_t __cudaLaunchKernel(void*, dim3, dim3, void**, size_t, void*) {   // by <<< >>>
  if (fake().fail_launch > 0 && fake().fail_launch--) return fake().done(cudaErrorInvalidResourceHandle);
  return cudaSuccess;
}
}

#define EXPECT(cond)                                                        \
  do {                                                                      \
    if (!(cond)) {                                                          \
      printf("line %d: %s\n", __LINE__, #cond);                             \
      exit(1);                                                              \
    }                                                                       \
  } while (0)
