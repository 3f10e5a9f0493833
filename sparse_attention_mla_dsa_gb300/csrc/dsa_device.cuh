// dsa_device.cuh -- device-side building blocks shared by the DSA kernels:
// the sticky error word, bounded mbarrier waits, TMA, tcgen05 (UMMA + TMEM)
// and the legacy warp-level MMA used by the gather-attend.
//
// All tensor-core and bulk-copy access is written as inline PTX for sm_103a.
#pragma once

#include <cuda.h>
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>
#include <stdint.h>

#include "dsa.h"

namespace dsa {

// ------------------------------------------------------------------ error word
// err[0] = first DSA_DEVERR_* code, err[1] = row it concerned, err[2] = count.
__device__ __forceinline__ void record_error(int* err, int code, int row) {
  if (err == nullptr) return;
  if (atomicCAS(&err[0], 0, code) == 0) atomicExch(&err[1], row);
  atomicAdd(&err[2], 1);
}

// Order-preserving key of a float score: a larger score gives a larger
// unsigned key; -0.0 is folded onto +0.0 first.  Scores must not be NaN.
__device__ __forceinline__ uint32_t order_key(float f) {
  const uint32_t u = __float_as_uint(__fadd_rn(f, 0.0f));
  return (u & 0x80000000u) ? ~u : (u | 0x80000000u);
}

// ------------------------------------------------------------------ timers / waits
__device__ __forceinline__ uint64_t global_ns() {
  uint64_t t;
  asm volatile("mov.u64 %0, %%globaltimer;" : "=l"(t));
  return t;
}

__device__ __forceinline__ uint32_t smem_u32(const void* p) {
  return static_cast<uint32_t>(__cvta_generic_to_shared(p));
}

__device__ __forceinline__ void mbar_init(uint64_t* bar, uint32_t count) {
  asm volatile("mbarrier.init.shared::cta.b64 [%0], %1;" ::"r"(smem_u32(bar)), "r"(count)
               : "memory");
}

__device__ __forceinline__ void fence_mbar_init() {
  asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
}

__device__ __forceinline__ void fence_proxy_async_smem() {
  asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
}

__device__ __forceinline__ void mbar_arrive_expect_tx(uint64_t* bar, uint32_t bytes) {
  asm volatile("mbarrier.arrive.expect_tx.shared::cta.b64 _, [%0], %1;" ::"r"(smem_u32(bar)),
               "r"(bytes)
               : "memory");
}

__device__ __forceinline__ void mbar_arrive(uint64_t* bar) {
  asm volatile("mbarrier.arrive.shared::cta.b64 _, [%0];" ::"r"(smem_u32(bar)) : "memory");
}

__device__ __forceinline__ bool mbar_try_wait(uint64_t* bar, uint32_t parity) {
  uint32_t ok;
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "mbarrier.try_wait.parity.shared::cta.b64 p, [%1], %2;\n\t"
      "selp.u32 %0, 1, 0, p;\n\t}"
      : "=r"(ok)
      : "r"(smem_u32(bar)), "r"(parity)
      : "memory");
  return ok != 0;
}

// The same poll with a bound on how long the hardware may suspend the
// thread inside it.
__device__ __forceinline__ bool mbar_try_wait_hint(uint64_t* bar, uint32_t parity, uint32_t hint_ns) {
  uint32_t ok;
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "mbarrier.try_wait.parity.shared::cta.b64 p, [%1], %2, %3;\n\t"
      "selp.u32 %0, 1, 0, p;\n\t}"
      : "=r"(ok)
      : "r"(smem_u32(bar)), "r"(parity), "r"(hint_ns)
      : "memory");
  return ok != 0;
}

// Limits below this are short: every poll is bounded (32 ns suspend) and
// followed by a look at the clock, so the limit holds to within a poll.
constexpr uint64_t kShortWaitNs = 1000ull * 1000ull;
// Longest time a poll may leave the thread suspended.
constexpr uint32_t kSuspendHintNs = 1000;

// The polling loop of mbar_wait, out of line so that the kernels' wait sites
// stay small (a wait that gets here is waiting anyway).
static __device__ __noinline__ bool mbar_wait_polls(uint64_t* bar, uint32_t parity, uint64_t limit_ns) {
  const uint64_t t0 = global_ns();
  if (limit_ns < kShortWaitNs) {
    for (uint32_t i = 0; i < (1u << 30); ++i) {
      if (mbar_try_wait_hint(bar, parity, 32)) return true;
      if (global_ns() - t0 > limit_ns) return false;
    }
    return false;
  }
  for (uint32_t i = 1; i < (1u << 30); ++i) {
    if (mbar_try_wait_hint(bar, parity, kSuspendHintNs)) return true;
    if ((i & 255u) == 0 && global_ns() - t0 > limit_ns) return false;
  }
  return false;
}

// Wait for the phase with the given parity to complete.  Gives up after
// `limit_ns` of wall time (checked every 256 polls, every poll for a short
// limit) or 2^30 polls, whichever comes first, and returns false then.  A
// thread whose phase cannot complete before the kernel before has ended calls
// grid_dep_wait() first: that kernel's time is not this one's stall.
__device__ __forceinline__ bool mbar_wait(uint64_t* bar, uint32_t parity, uint64_t limit_ns) {
  if (limit_ns >= kShortWaitNs && mbar_try_wait(bar, parity)) return true;
  return mbar_wait_polls(bar, parity, limit_ns);
}

// ------------------------------------------------------------------ dependent launch
// With programmatic stream serialisation a kernel may start while the one
// before it in the stream is still running.  grid_dep_wait() blocks until the
// previous kernel has completed and its writes are visible; every kernel here
// calls it before it reads a predecessor's output or overwrites a buffer a
// predecessor may still read.  grid_dep_launch() lets the next kernel start.
// Both are no-ops for kernels launched without the attribute.  grid_dep_wait()
// holds up its whole warp, so whole warps call it: not one lane in its role (which
// leaves the operands of MMAs and copies in registers of the warp), nor the others
// while it is there (__syncwarp first).
__device__ __forceinline__ void grid_dep_wait() { asm volatile("griddepcontrol.wait;" ::: "memory"); }
// Data written by an earlier kernel of the chain must be read with loads the
// compiler keeps after grid_dep_wait(): plain loads, or these.  The
// read-only-path intrinsics (__ldg, __ldcg, ...) are treated as loads of
// memory that never changes and may be hoisted above the wait.
__device__ __forceinline__ float2 ld_dep_f2(const float2* p) {
  float2 v;
  asm volatile("ld.global.cg.v2.f32 {%0,%1}, [%2];" : "=f"(v.x), "=f"(v.y) : "l"(p) : "memory");
  return v;
}
__device__ __forceinline__ float4 ld_dep_f4(const float4* p) {
  float4 v;
  asm volatile("ld.global.cg.v4.f32 {%0,%1,%2,%3}, [%4];"
               : "=f"(v.x), "=f"(v.y), "=f"(v.z), "=f"(v.w)
               : "l"(p)
               : "memory");
  return v;
}
__device__ __forceinline__ uint2 ld_dep_u2(const uint2* p) {
  uint2 v;
  asm volatile("ld.global.cg.v2.u32 {%0,%1}, [%2];" : "=r"(v.x), "=r"(v.y) : "l"(p) : "memory");
  return v;
}
__device__ __forceinline__ uint4 ld_dep_u4(const uint4* p) {
  uint4 v;
  asm volatile("ld.global.cg.v4.u32 {%0,%1,%2,%3}, [%4];"
               : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w)
               : "l"(p)
               : "memory");
  return v;
}
// One thread's call counts for its CTA.  A kernel with tensor memory makes it from
// the warp that allocates, behind the allocation, and nowhere else: tcgen05.alloc
// waits without a limit until the SM has the columns, and a CTA of the next kernel
// that took them first would keep them until this kernel has ended.
__device__ __forceinline__ void grid_dep_launch() {
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
}

// ------------------------------------------------------------------ TMA
__device__ __forceinline__ void tma_prefetch_map(const CUtensorMap* map) {
  asm volatile("prefetch.tensormap [%0];" ::"l"(reinterpret_cast<uint64_t>(map)) : "memory");
}

__device__ __forceinline__ uint64_t l2_policy_evict_first() {
  uint64_t p;
  asm volatile("createpolicy.fractional.L2::evict_first.b64 %0, 1.0;" : "=l"(p));
  return p;
}

// L2 prefetches.  They move no data into the SM and complete on nothing, so
// they may be issued before grid_dep_wait(): L2 is where every write of the
// device lands, so a later load after the wait still sees the newest value.
// One box of a tiled tensor (same coordinates as a load):
__device__ __forceinline__ void tma_prefetch_l2_2d(const CUtensorMap* map, int32_t x, int32_t y) {
  asm volatile("cp.async.bulk.prefetch.tensor.2d.L2.global.tile [%0, {%1, %2}];" ::"l"(
                   reinterpret_cast<uint64_t>(map)),
               "r"(x), "r"(y)
               : "memory");
}
// The 128-byte line holding `p`:
__device__ __forceinline__ void prefetch_l2(const void* p) {
  asm volatile("prefetch.global.L2 [%0];" ::"l"(p) : "memory");
}

// 2-D tiled load of one box into shared memory, completing on `bar`.
__device__ __forceinline__ void tma_load_2d(void* dst, const CUtensorMap* map, uint64_t* bar,
                                            int32_t x, int32_t y, uint64_t policy) {
  asm volatile(
      "cp.async.bulk.tensor.2d.shared::cluster.global.mbarrier::complete_tx::bytes.L2::cache_hint"
      " [%0], [%1, {%2, %3}], [%4], %5;" ::"r"(smem_u32(dst)),
      "l"(reinterpret_cast<uint64_t>(map)), "r"(x), "r"(y), "r"(smem_u32(bar)), "l"(policy)
      : "memory");
}

// ------------------------------------------------------------------ tcgen05
// By one warp: takes the CTA's tensor memory, then lets the next kernel start (in
// this order, see grid_dep_launch).
__device__ __forceinline__ void tmem_alloc_then_launch(uint32_t* dst, uint32_t ncols) {
  asm volatile(
      "tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;\n\t"
      "tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;" ::"r"(smem_u32(dst)),
      "r"(ncols)
      : "memory");
  grid_dep_launch();
}
// The same for a pair of CTAs (one warp of each), whose tensor memory is taken together.
__device__ __forceinline__ void tmem_alloc_pair_then_launch(uint32_t* dst, uint32_t ncols) {
  asm volatile(
      "tcgen05.alloc.cta_group::2.sync.aligned.shared::cta.b32 [%0], %1;\n\t"
      "tcgen05.relinquish_alloc_permit.cta_group::2.sync.aligned;" ::"r"(smem_u32(dst)),
      "r"(ncols)
      : "memory");
  grid_dep_launch();
}
// (Behind a barrier of the CTA, where the lanes of a warp need not be together.)
__device__ __forceinline__ void tmem_dealloc(uint32_t taddr, uint32_t ncols) {
  __syncwarp();
  asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(taddr), "r"(ncols)
               : "memory");
}
__device__ __forceinline__ void tc_fence_before() {
  asm volatile("tcgen05.fence::before_thread_sync;" ::: "memory");
}
__device__ __forceinline__ void tc_fence_after() {
  asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory");
}

// Shared-memory matrix descriptor of a K-major operand in the 128-byte
// swizzled layout: rows of 128 B (64 bf16 of K), 8-row groups 1024 B apart,
// tile base 1024-byte aligned.  A K step of 16 elements inside the 128-byte
// row advances the start address by 32 B.
__device__ __forceinline__ uint64_t umma_desc_sw128_kmajor(uint32_t saddr) {
  uint64_t d = 0;
  d |= static_cast<uint64_t>((saddr & 0x3FFFFu) >> 4);  // start address  [0,14)
  d |= static_cast<uint64_t>(1) << 16;                  // leading offset (unused here)
  d |= static_cast<uint64_t>(1024 >> 4) << 32;          // stride offset: 8 rows x 128 B
  d |= static_cast<uint64_t>(1) << 46;                  // descriptor version
  d |= static_cast<uint64_t>(2) << 61;                  // 128-byte swizzle
  return d;
}

// Instruction descriptor, kind::f16 with BF16 A and B, FP32 accumulate, both
// operands K-major, M x N tile.
__host__ __device__ constexpr uint32_t umma_idesc_bf16(int m, int n) {
  return (1u << 4)                                   // D = F32
         | (1u << 7)                                 // A = BF16
         | (1u << 10)                                // B = BF16
         | (static_cast<uint32_t>(n >> 3) << 17)     // N
         | (static_cast<uint32_t>(m >> 4) << 24);    // M
}

// D[tmem] (+)= A[smem] * B[smem]^T, issued by one thread.
__device__ __forceinline__ void umma_bf16(uint32_t d_tmem, uint64_t adesc, uint64_t bdesc,
                                          uint32_t idesc, uint32_t accumulate) {
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "setp.ne.b32 p, %4, 0;\n\t"
      "tcgen05.mma.cta_group::1.kind::f16 [%0], %1, %2, %3, p;\n\t}" ::"r"(d_tmem),
      "l"(adesc), "l"(bdesc), "r"(idesc), "r"(accumulate)
      : "memory");
}

// Arrive on `bar` once every tcgen05 op issued so far by this thread is done.
__device__ __forceinline__ void umma_commit(uint64_t* bar) {
  asm volatile(
      "tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];" ::"r"(
          smem_u32(bar))
      : "memory");
}

// 16 consecutive 32-bit TMEM columns of this thread's lane, waited for in the
// same statement so no use of the values can be scheduled before the wait.
__device__ __forceinline__ void tmem_load16(uint32_t taddr, float (&v)[16]) {
  uint32_t r[16];
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x16.b32 "
      "{%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15}, [%16];\n\t"
      "tcgen05.wait::ld.sync.aligned;"
      : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]),
        "=r"(r[7]), "=r"(r[8]), "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]),
        "=r"(r[13]), "=r"(r[14]), "=r"(r[15])
      : "r"(taddr)
      : "memory");
#pragma unroll
  for (int i = 0; i < 16; ++i) v[i] = __uint_as_float(r[i]);
}

}  // namespace dsa
