// few.cuh: the streaming engine of the decoding kernels (few tokens, all of the
// time goes into reading weights once).
//
// A CTA is eight computing warps, one copying warp and three finishing warps.  The
// copying warp walks the CTA's work and keeps a ring of shared-memory stages full with bulk copies
// and TMA loads (counted on an mbarrier per stage): per stage RT row tiles of 16
// weight rows x 1024 or 2048 columns, and (the layer) the same columns of the tokens that
// the weights multiply.  Each computing warp takes one or two 128-column slices of a stage.
// The eight partial sums of a row go to the finishing warps through shared memory once
// a row tile is complete; they add them in a fixed order and write the results while
// the computing warps go on (a block-wide meeting per item had cost a tenth).
//
// The layer's products, and a matrix's with few tokens, run on mma.sync and not on tcgen05:
// the tensor work is the weights times 8 columns, far below either's rate, while 4-bit codes
// have to pass through registers to be widened and FP8 sums to be scaled per 128 columns.
// More tokens on one matrix take tcgen05 (few_tensor.cuh).
#pragma once

#include "common.cuh"
#include "few_plan.h"
#include "w4.cuh"

namespace moe {

constexpr int kFewFinish = 3;                      // finishing warps
constexpr int kFewAllWarps = kFewWarps + 1 + kFewFinish, kFewThreads = kFewAllWarps * 32;
constexpr int kFewFinishThreads = 32 * kFewFinish;
constexpr uint64_t kFewTimeoutNs = 1000000000ull;  // bound of every wait

// Untiled bulk copy global -> shared (16-byte aligned, size a multiple of 16).
MOE_DEV void bulk_load(uint32_t dst, const void* src, uint32_t bytes, uint32_t bar) {
  asm volatile("cp.async.bulk.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1], %2, [%3];"
               :: "r"(dst), "l"(reinterpret_cast<uint64_t>(src)), "r"(bytes), "r"(bar) : "memory");
}
// As bulk_load and tma_load_3d for weights, which are read once, or again soon after (an expert's
// next 16 tokens): first to leave L2, so that the tokens, the tables and the kernel's own code stay (they are few, and
// each miss of theirs is waited for).
MOE_DEV uint64_t evict_first_policy() {
  uint64_t p;
  asm("createpolicy.fractional.L2::evict_first.b64 %0, 1.0;" : "=l"(p));
  return p;
}
MOE_DEV void bulk_load_once(uint32_t dst, const void* src, uint32_t bytes, uint32_t bar) {
  asm volatile("cp.async.bulk.shared::cluster.global.mbarrier::complete_tx::bytes.L2::cache_hint [%0], [%1], %2, [%3], %4;"
               :: "r"(dst), "l"(reinterpret_cast<uint64_t>(src)), "r"(bytes), "r"(bar), "l"(evict_first_policy()) : "memory");
}
MOE_DEV void tma_load_3d_once(uint32_t dst, const CUtensorMap* map, int x, int y, int z, uint32_t bar) {
  asm volatile(
      "cp.async.bulk.tensor.3d.shared::cluster.global.mbarrier::complete_tx::bytes.L2::cache_hint [%0], [%1, {%2, %3, %4}], [%5], %6;"
      :: "r"(dst), "l"(reinterpret_cast<uint64_t>(map)), "r"(x), "r"(y), "r"(z), "r"(bar), "l"(evict_first_policy()) : "memory");
}
// This thread's earlier cp.async copies arrive on `bar` when they are complete.
MOE_DEV void cp_async_arrive(uint32_t bar) {
  asm volatile("cp.async.mbarrier.arrive.noinc.shared::cta.b64 [%0];" :: "r"(bar) : "memory");
}

// d (16 x 8, fp32) += a (16 rows x 16) * b (16 x 8 columns).
// (mma.sync with e4m3 operands is no way around widening: on sm_103a it is two f16
// MMAs behind twelve conversions.)
MOE_DEV void mma_bf16(float (&d)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
  asm("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
      : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
      : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}
MOE_DEV void mma_f16(float (&d)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
  asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
      : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
      : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}

// Loads by shared address (a generic pointer's loads take the slower path through L1).
MOE_DEV uint4 lds128(uint32_t a) {
  uint4 v;
  asm volatile("ld.shared.v4.u32 {%0,%1,%2,%3}, [%4];" : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w) : "r"(a));
  return v;
}
MOE_DEV float lds_f32(uint32_t a) {
  float v;
  asm volatile("ld.shared.f32 %0, [%1];" : "=f"(v) : "r"(a));
  return v;
}
MOE_DEV float lds_bf16(uint32_t a) {
  uint16_t v;
  asm volatile("ld.shared.u16 %0, [%1];" : "=h"(v) : "r"(a));
  return bf16_lo(v);
}

MOE_DEV uint16_t to_bf16(float v) {
  const __nv_bfloat16 b = __float2bfloat16_rn(v);
  return *reinterpret_cast<const uint16_t*>(&b);
}

template <int GROUP>
struct FewGroups {
  static constexpr int kCount = GROUP == 32 ? 4 : GROUP == 64 ? 2 : 1;   // scales per row and 128-column slice
};

// ---------------------------------------------------------------- the ring

// Barriers of the ring and the block's flags at the start of shared memory.
struct FewShared {
  uint64_t full[kFewMaxStages], empty[kFewMaxStages];
  uint64_t sums_full[2], sums_empty[2];
  volatile int abort_flag;
  int segs, cap, rows;
};
static_assert(sizeof(FewShared) <= 256, "");

struct FewRing {
  uint32_t base, stage_bytes, full, empty;   // shared addresses; full / empty: barriers 8 bytes apart
  int stages;
  int slot, phase;
  MOE_DEV uint32_t stage() const { return base + slot * stage_bytes; }
  MOE_DEV uint32_t full_bar() const { return full + 8 * slot; }
  MOE_DEV uint32_t empty_bar() const { return empty + 8 * slot; }
  MOE_DEV void next() {
    if (++slot == stages) { slot = 0; phase ^= 1; }
  }
};

// All barriers and the abort flag, by the block's first threads; the caller
// synchronises the block.  `arrivals` complete a stage, `readers` free it.
MOE_DEV void few_barriers(unsigned char* sm, int tid, int arrivals, int readers = kFewWarps) {
  FewShared* sh = reinterpret_cast<FewShared*>(sm);
  if (tid < kFewMaxStages) {
    mbar_init(smem_u32(sh->full + tid), arrivals);
    mbar_init(smem_u32(sh->empty + tid), readers);
    if (tid < 2) {
      mbar_init(smem_u32(sh->sums_full + tid), kFewWarps);
      mbar_init(smem_u32(sh->sums_empty + tid), kFewFinish);
    }
    fence_mbar_init();
  }
  if (tid == 0) sh->abort_flag = 0;
}

// A ring in the shared memory [at, smem_bytes).
MOE_DEV FewRing few_ring(unsigned char* sm, uint32_t at, uint32_t smem_bytes, uint32_t stage_bytes) {
  FewShared* sh = reinterpret_cast<FewShared*>(sm);
  FewRing r;
  at = (at + 1023) & ~1023u;
  r.base = smem_u32(sm) + at;
  r.stage_bytes = stage_bytes;
  r.full = smem_u32(sh->full);
  r.empty = smem_u32(sh->empty);
  r.stages = min((int)((smem_bytes - at) / stage_bytes), kFewMaxStages);
  r.slot = r.phase = 0;
  return r;
}

// The way of the sums from the computing to the finishing warps: one or two buffers of
// `stage_bytes` at sm + at.
MOE_DEV FewRing few_sums_ring(unsigned char* sm, uint32_t at, uint32_t bytes, int buffers) {
  FewShared* sh = reinterpret_cast<FewShared*>(sm);
  FewRing r;
  r.base = at;
  r.stage_bytes = bytes;
  r.full = smem_u32(sh->sums_full);
  r.empty = smem_u32(sh->sums_empty);
  r.stages = buffers;
  r.slot = r.phase = 0;
  return r;
}

// A warp's bounded wait: one outcome for all lanes.
MOE_DEV bool ring_wait(uint32_t bar, uint32_t parity, volatile int* abort_flag, int32_t* status) {
  return __all_sync(0xffffffffu, mbar_wait(bar, parity, abort_flag, status, kFewTimeoutNs));
}

// The same for a warp with time to spare: it sleeps between looks, since warps that poll
// take issue slots from those that compute.
MOE_DEV bool ring_wait_idle(uint32_t bar, uint32_t parity, volatile int* abort_flag, int32_t* status) {
  const uint64_t t0 = globaltimer_ns();
  while (!__all_sync(0xffffffffu, mbar_try_wait(bar, parity))) {
    __nanosleep(64);
    bool over = *abort_flag;
    if (!over && globaltimer_ns() - t0 > kFewTimeoutNs) {
      *abort_flag = 1;
      set_status(status, MOE_ERR_TIMEOUT);
      over = true;
    }
    if (__any_sync(0xffffffffu, over)) return false;
  }
  return true;
}

// The copying warp's end: every stage it has begun is complete before the block
// leaves.  `issued` stages were begun in all; the last `partial` of them still
// lack their tokens (an abandoned wait), whose arrivals are made up for.
MOE_DEV void drain(FewRing r, int issued, int partial, int lane) {
  // r is positioned behind the last stage begun
  const int n = min(issued, r.stages);
  for (int i = 0; i < n; ++i) {
    if (r.slot == 0) { r.slot = r.stages; r.phase ^= 1; }
    --r.slot;
    if (i < partial && lane == 0) mbar_arrive(r.full_bar());
    const uint64_t t0 = globaltimer_ns();   // bounded; it runs out only if a copy never lands
    while (!mbar_try_wait(r.full_bar(), r.phase) && globaltimer_ns() - t0 < kFewTimeoutNs) {}
  }
}

// ---------------------------------------------------------------- sums over the warps

// The sum over the warps, in their order.
MOE_DEV float get_sum(const float* red, int pitch, int row, int col) {
  float s = 0.f;
#pragma unroll
  for (int w = 0; w < kFewWarps; ++w) s += red[(w * pitch + col) * kFewColPitch + row];
  return s;
}

// The meeting of all warps but the copying one, which also tells all of them whether any
// gave up, so that they leave together.
MOE_DEV bool consumer_sync_all(bool ok) {
  uint32_t all;
  asm volatile(
      "{\n\t.reg .pred p, q;\n\t"
      "setp.ne.b32 p, %1, 0;\n\t"
      "bar.red.and.pred q, 1, %2, p;\n\t"
      "selp.u32 %0, 1, 0, q;\n\t}"
      : "=r"(all) : "r"((uint32_t)ok), "n"(kFewThreads - 32) : "memory");
  return all != 0;
}
MOE_DEV void finish_sync() { asm volatile("bar.sync 2, %0;" :: "n"(kFewFinishThreads) : "memory"); }

}  // namespace moe
