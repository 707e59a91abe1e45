// norm.cuh: what the forward and the backward pass of layer norm share.
//
// A row lies in the registers of the TPR threads that work on it, NV vectors of
// 16 bytes a thread, so memory is read once whatever the formula passes over.  A
// group of TPR threads walks the rows g, g + groups, ...; each thread keeps
// the next rows' vectors coming by cp.async into a ring in shared memory that
// it alone reads, so nothing is waited for but a thread's own copies.
//
// Rows whose length is no whole number of vectors start inside one.  `groups` is a
// multiple of 8, so all rows of a group start at the same place s inside a
// vector: a thread's columns are the same in each of them, and weights and column
// sums stay in registers there too.  The vectors at a row's ends are masked,
// and stored value by value.
#pragma once

#include <string.h>

#include <type_traits>

#include "dtype.cuh"
#include "host_util.h"

namespace moe {

constexpr int kNormMaxBlocks = 320;   // of the backward pass, two an SM

struct NormArgs {
  const void* x;
  const void* dy;
  const void* weight;
  const void* bias;
  int T, H;
  float eps;
  void* y;      // y, or dx
  float* mean;
  float* rstd;
  float* part;  // backward: [blocks][2][H] sums of each block's rows
  int tail;     // norm_tail
};

// A row's last vector reaches up to V - 1 values into the rows behind it, but not past the tensor's end: from
// this row on, where fewer are left (the last row; more of them where rows are shorter than a vector), it
// is read up to its row's end.
inline int norm_tail(int T, int H, int dtype) {
  const int V = dtype == MOE_F32 ? 4 : 8;
  return T - (V - 1 + H - 1) / H;
}

// A vector's worth of weights: W's own 16 bytes where W is the rows' type, else fp32.
// Rows of whole vectors read them from a copy in shared memory; those of MASK, whose
// vectors start at another column in each group, keep them in registers.
template <typename T, typename W>
struct ParamVec {
  f32x2 p[kVec16<T> / 2];
  MOE_DEV void set(const f32x2* v) {
#pragma unroll
    for (int e = 0; e < kVec16<T> / 2; ++e) p[e] = v[e];
  }
  MOE_DEV void get(f32x2* out) const {
#pragma unroll
    for (int e = 0; e < kVec16<T> / 2; ++e) out[e] = p[e];
  }
};
template <typename T>
struct ParamVec<T, T> {
  uint4 p;
  MOE_DEV void set(const f32x2* v) { p = Pairs<T>::put(v); }   // exact: the values come from T
  MOE_DEV void get(f32x2* out) const { Pairs<T>::get(p, out); }
};

// ---------------------------------------------------------------- a thread's part of its group's rows

// 16 bytes global -> shared, of which the first `bytes` are read and the rest are zeros.
MOE_DEV void cp_async16(uint32_t dst, const void* src, uint32_t bytes) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(reinterpret_cast<uint64_t>(src)), "r"(bytes) : "memory");
}

#define MOE_BOTH __host__ __device__ __forceinline__

// MASK: rows of no whole number of vectors, whose first and last vectors are shared
// with the rows beside them.
template <typename T, int TPR, int NV, bool MASK>
struct RowPart {
  static constexpr int V = kVec16<T>;
  int H, tid, first;   // first: column of this thread's vector 0

  MOE_BOTH RowPart(int H_, long long first_row, int tid_) : H(H_), tid(tid_), first(tid_ * V - (MASK ? (int)(first_row * H_ % V) : 0)) {}
  MOE_DEV RowPart(int H_, long long first_row) : RowPart(H_, first_row, (int)threadIdx.x % TPR) {}
  // first column of vector i, and the part [lo, hi) of it that is this row's
  MOE_BOTH int col(int i) const { return first + i * TPR * V; }
  MOE_BOTH int lo(int i) const { return max(0, -col(i)); }
  MOE_BOTH int hi(int i) const { return min(V, H - col(i)); }
  MOE_BOTH bool any(int i) const { return col(i) < H; }
  MOE_BOTH bool whole(int i) const { return !MASK || (col(i) >= 0 && col(i) + V <= H); }

  // values of vector i that are read, from the vector's start on, in a row that is one of the tail's (norm_tail) or not
  MOE_BOTH int readable(int i, bool tail) const { return MASK && tail ? hi(i) : V; }

  // Start copying this thread's vectors of a row into its slots, `step` bytes apart; `src` is vector 0.
  MOE_DEV void fetch(const T* src, bool tail, uint32_t slot, uint32_t step) const {
#pragma unroll
    for (int i = 0; i < NV; ++i)
      if (any(i)) cp_async16(slot + i * step, src + i * TPR * V, (uint32_t)(readable(i, tail) * sizeof(T)));
  }
  // zeros into the slots of vectors that the rows do not have: work on masked rows then needs no branches
  MOE_DEV void clear_absent(uint8_t* slot, uint32_t step) const {
#pragma unroll
    for (int i = 0; i < NV; ++i)
      if (!any(i)) *reinterpret_cast<uint4*>(slot + i * step) = make_uint4(0, 0, 0, 0);
  }
  // store vector i of the row whose vector 0 is at `dst`
  MOE_DEV void store(T* dst, int i, const uint4& v) const {
    T* p = dst + i * TPR * V;
    if (whole(i)) {
      *reinterpret_cast<uint4*>(p) = v;
    } else {
      const uint32_t w[4] = {v.x, v.y, v.z, v.w};
      const int a = lo(i), b = hi(i);
#pragma unroll
      for (int e = 0; e < V; ++e)
        if (e >= a && e < b) {
          if (sizeof(T) == 4) reinterpret_cast<uint32_t*>(p)[e] = w[e % 4];
          else reinterpret_cast<uint16_t*>(p)[e] = (uint16_t)(w[e / 2] >> (16 * (e % 2)));
        }
    }
  }
  // zeros where vector i is not this row's
  MOE_DEV void mask(int i, f32x2* v) const {
    if (whole(i)) return;
    const int a = lo(i), b = hi(i);
#pragma unroll
    for (int e = 0; e < V / 2; ++e)
      v[e] = pack_f32x2(2 * e >= a && 2 * e < b ? lo2(v[e]) : 0.f, 2 * e + 1 >= a && 2 * e + 1 < b ? hi2(v[e]) : 0.f);
  }
  // This thread's weights (or biases) of vector i, for registers; unspecified outside the row.  16-bit
  // ones come out of the two vectors that hold them, which `begin` loads and `end` waits for.
  template <typename W>
  MOE_DEV bool params_packed(const void* src, int i) const {
    const int c = col(i), off = c & 7;
    return sizeof(W) == 2 && src && c >= off && c - off + 16 <= H;
  }
  template <typename W>
  MOE_DEV void params_begin(const void* src, int i, uint4 (&raw)[2]) const {
    const bool there = params_packed<W>(src, i);
    const W* p = static_cast<const W*>(src) + (col(i) & ~7);
    load_if(raw[0], p, there);
    load_if(raw[1], p + 8, there);
  }
  template <typename W>
  MOE_DEV ParamVec<T, W> params_end(const void* src, float none, int i, const uint4 (&raw)[2]) const {
    ParamVec<T, W> r;
    if (params_packed<W>(src, i)) {
      const uint4 packed = shifted8(raw[0], raw[1], col(i) & 7);
      memcpy(&r, &packed, sizeof(uint4));
      return r;
    }
    const W* p = static_cast<const W*>(src);
    f32x2 v[V / 2];
#pragma unroll
    for (int e = 0; e < V; e += 2) {
      const int j = col(i) + e;
      const float a = j >= 0 && j < H ? (p ? to_f32(p[j]) : none) : 0.f;
      const float b = j + 1 >= 0 && j + 1 < H ? (p ? to_f32(p[j + 1]) : none) : 0.f;
      v[e / 2] = pack_f32x2(a, b);
    }
    r.set(v);
    return r;
  }
  template <typename W>
  MOE_DEV ParamVec<T, W> params(const void* src, float none, int i) const {
    uint4 raw[2] = {};
    params_begin<W>(src, i, raw);
    return params_end<W>(src, none, i, raw);
  }
};

MOE_DEV float warp_sum(float v) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
  return v;
}

// The sum over a block, for every thread.
template <int BLOCK>
MOE_DEV float block_sum(float v, float* scratch) {
  v = warp_sum(v);
  __syncthreads();
  if ((threadIdx.x & 31) == 0) scratch[threadIdx.x >> 5] = v;
  __syncthreads();
  return warp_sum((threadIdx.x & 31) < BLOCK / 32 ? scratch[threadIdx.x & 31] : 0.f);
}

// weight or bias value j, `none` where there is no such tensor
template <typename W>
MOE_DEV float param(const void* p, int j, float none) { return p ? to_f32(static_cast<const W*>(p)[j]) : none; }

// [H] weights (or biases) into shared memory, H of them being whole vectors
template <int BLOCK, typename W>
MOE_DEV void copy_params(W* dst, const void* src, float none, int H) {
  if (src) {
    for (int j = threadIdx.x; j < H / kVec16<W>; j += BLOCK) reinterpret_cast<uint4*>(dst)[j] = static_cast<const uint4*>(src)[j];
  } else {
    for (int j = threadIdx.x; j < H; j += BLOCK) dst[j] = from_f32<W>(none);
  }
}

// All threads of this thread's group.  Barriers 1 to 15, and the block's own for the last of 16
// groups (whose kernel has no barrier of the block after this).
template <int TPR, int BLOCK>
MOE_DEV void group_sync() {
  static_assert(TPR == 32 || BLOCK / TPR <= 16, "named barriers");
  if (TPR == BLOCK) __syncthreads();
  else if (TPR == 32) __syncwarp();
  else asm volatile("bar.sync %0, %1;" ::"r"(((int)threadIdx.x / TPR + 1) % 16), "n"(TPR) : "memory");
}

// Columns that a row's vectors cover, wherever it starts inside its first one.
inline int norm_span(int H, int vec) { return H % vec == 0 ? H : (H + 2 * (vec - 1)) / vec * vec; }
// threads a row at `values` values a thread
inline int norm_tpr(int H, int vec, int values) {
  int tpr = 32;
  while (tpr * values < norm_span(H, vec)) tpr *= 2;
  return tpr;
}

// Rows few enough to be taken all at once: up to two and a half times the threads that run at once (four times: 16.7 us against 9.2 at 9728 x 1024, 18.0
// against 12.9 at 4864 x 1111; never: 5.7 against 4.0 at 304 x 7168).
inline bool few_rows(int T, int tpr) { return 2LL * T * tpr <= 5 * 2048LL * device_sm_count(); }

int norm_bwd_few(int dtype, int wdtype, const NormArgs& p, void* dweight, void* dbias, cudaStream_t st);

inline size_t elem_bytes(int dtype) { return dtype == MOE_F32 ? 4 : 2; }
inline bool norm_shape_ok(int T, int H) { return T >= 0 && H >= 1 && H <= MOE_NORM_MAX_H; }
// a tensor of this type starts where its elements may start
inline bool elem_aligned(const void* p, int dtype) { return (uintptr_t)p % elem_bytes(dtype) == 0; }

// Blocks: `per_sm` on each SM (their number a multiple of 8), or as many as the rows need.
inline int norm_blocks(int T, int groups_a_block, int per_sm, int sms) {
  const long long full = (long long)(sms / 8 * 8) * per_sm, need = ((long long)T + groups_a_block - 1) / groups_a_block;
  return (int)std::max(1LL, std::min(full, need));
}

}  // namespace moe
