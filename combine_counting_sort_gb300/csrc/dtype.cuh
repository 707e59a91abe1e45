// dtype.cuh: bf16, f16 and f32 values as the dense operators load and store
// them: one conversion each way, and vectors of 16 bytes.
#pragma once

#include <cuda_fp16.h>

#include "common.cuh"

namespace moe {

template <typename T>
MOE_DEV float to_f32(T v);
template <>
MOE_DEV float to_f32<float>(float v) { return v; }
template <>
MOE_DEV float to_f32<__half>(__half v) { return __half2float(v); }
template <>
MOE_DEV float to_f32<__nv_bfloat16>(__nv_bfloat16 v) { return __bfloat162float(v); }

template <typename T>
MOE_DEV T from_f32(float v);
template <>
MOE_DEV float from_f32<float>(float v) { return v; }
template <>
MOE_DEV __half from_f32<__half>(float v) { return __float2half_rn(v); }
template <>
MOE_DEV __nv_bfloat16 from_f32<__nv_bfloat16>(float v) { return __float2bfloat16_rn(v); }

// V consecutive values: V = 1, or as many as 16 bytes hold.
template <typename T, int V>
struct alignas(V == 1 ? sizeof(T) : 16) Vec {
  static_assert(V == 1 || V * sizeof(T) == 16, "one value or 16 bytes");
  T v[V];
};

template <typename T>
constexpr int kVec16 = 16 / (int)sizeof(T);

}  // namespace moe
