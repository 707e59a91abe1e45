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

// 16 bytes by a predicated load: no branch, so nothing waits for it here.
MOE_DEV void load_if(uint4& v, const void* p, bool there) {
  asm volatile("{\n\t.reg .pred p;\n\tsetp.ne.b32 p, %5, 0;\n\t@p ld.global.v4.b32 {%0, %1, %2, %3}, [%4];\n\t}"
               : "+r"(v.x), "+r"(v.y), "+r"(v.z), "+r"(v.w) : "l"(p), "r"((int)there));
}

// 16-bit values from the vector boundary at or before p
MOE_DEV int vector_offset(const void* p) { return (int)((uintptr_t)p & 15) >> 1; }

// Eight 16-bit values from value `off` (0 to 7) of two vectors on.
MOE_DEV uint4 shifted8(const uint4& lo, const uint4& hi, int off) {
  uint32_t w[8] = {lo.x, lo.y, lo.z, lo.w, hi.x, hi.y, hi.z, hi.w};
#pragma unroll
  for (int k = 0; k < 6; ++k) w[k] = off & 4 ? w[k + 2] : w[k];
#pragma unroll
  for (int k = 0; k < 5; ++k) w[k] = off & 2 ? w[k + 1] : w[k];
  const int bits = (off & 1) * 16;
  return make_uint4(__funnelshift_r(w[0], w[1], bits), __funnelshift_r(w[1], w[2], bits), __funnelshift_r(w[2], w[3], bits),
                    __funnelshift_r(w[3], w[4], bits));
}

// The two vectors that hold eight values from element `at` of p's `total`, as they come: by
// predicated loads, so that nothing waits for them before they are shifted.  At the tensor's
// ends, where a vector would reach beyond it, the values are fetched one by one then.  (One
// vector a lane and the other from the next lane: 4.2 us against 2.0 for two rows, 15.4 against 13.4 for 857.)
struct Unaligned {
  uint4 lo, hi;
  int off;   // -1: one by one
};
MOE_DEV void load_unaligned(Unaligned& u, const uint16_t* p, long long at, long long total, bool wanted = true) {
  const int off = (int)((uintptr_t)(p + at) & 15) >> 1;
  const bool inside = at >= off && at - off + 16 <= total;
  const uint4* v = reinterpret_cast<const uint4*>(p + at - off);
  load_if(u.lo, v, inside && wanted);
  load_if(u.hi, v + 1, inside && wanted);
  u.off = inside ? off : -1;
}
MOE_DEV uint4 shifted(const Unaligned& u, const uint16_t* p, long long at, long long total) {
  if (u.off < 0) {
    uint32_t w[8];
#pragma unroll
    for (int k = 0; k < 8; ++k) w[k] = at + k < total ? p[at + k] : 0u;
    return make_uint4(w[0] | w[1] << 16, w[2] | w[3] << 16, w[4] | w[5] << 16, w[6] | w[7] << 16);
  }
  return shifted8(u.lo, u.hi, u.off);
}

// ---------------------------------------------------------------- pairs of fp32 (.f32x2 instructions)

using f32x2 = unsigned long long;
MOE_DEV f32x2 add2(f32x2 a, f32x2 b) { f32x2 r; asm("add.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b)); return r; }
MOE_DEV f32x2 mul2(f32x2 a, f32x2 b) { f32x2 r; asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b)); return r; }
MOE_DEV f32x2 fma2(f32x2 a, f32x2 b, f32x2 c) {
  f32x2 r;
  asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r) : "l"(a), "l"(b), "l"(c));
  return r;
}
MOE_DEV f32x2 both(float v) { return pack_f32x2(v, v); }
MOE_DEV float lo2(f32x2 v) { return __uint_as_float((uint32_t)v); }
MOE_DEV float hi2(f32x2 v) { return __uint_as_float((uint32_t)(v >> 32)); }
MOE_DEV float sum2(f32x2 v) { return lo2(v) + hi2(v); }

// 16 bytes of T as pairs
template <typename T>
struct Pairs;
template <>
struct Pairs<float> {
  static constexpr int N = 2;
  static MOE_DEV void get(const uint4& r, f32x2* out) {
    out[0] = (f32x2)r.x | ((f32x2)r.y << 32);
    out[1] = (f32x2)r.z | ((f32x2)r.w << 32);
  }
  static MOE_DEV uint4 put(const f32x2* v) {
    return make_uint4((uint32_t)v[0], (uint32_t)(v[0] >> 32), (uint32_t)v[1], (uint32_t)(v[1] >> 32));
  }
};
template <>
struct Pairs<__nv_bfloat16> {
  static constexpr int N = 4;
  static MOE_DEV f32x2 one(uint32_t v) { return pack_f32x2(bf16_lo(v), bf16_hi(v)); }
  static MOE_DEV void get(const uint4& r, f32x2* out) { out[0] = one(r.x); out[1] = one(r.y); out[2] = one(r.z); out[3] = one(r.w); }
  static MOE_DEV uint4 put(const f32x2* v) {
    return make_uint4(pack_bf16x2_from_pair(v[0]), pack_bf16x2_from_pair(v[1]), pack_bf16x2_from_pair(v[2]), pack_bf16x2_from_pair(v[3]));
  }
};
template <>
struct Pairs<__half> {
  static constexpr int N = 4;
  static MOE_DEV f32x2 one(uint32_t v) {
    const float2 f = __half22float2(*reinterpret_cast<const __half2*>(&v));
    return pack_f32x2(f.x, f.y);
  }
  static MOE_DEV uint32_t pack(f32x2 v) {
    const __half2 h = __floats2half2_rn(lo2(v), hi2(v));
    return *reinterpret_cast<const uint32_t*>(&h);
  }
  static MOE_DEV void get(const uint4& r, f32x2* out) { out[0] = one(r.x); out[1] = one(r.y); out[2] = one(r.z); out[3] = one(r.w); }
  static MOE_DEV uint4 put(const f32x2* v) { return make_uint4(pack(v[0]), pack(v[1]), pack(v[2]), pack(v[3])); }
};

}  // namespace moe
