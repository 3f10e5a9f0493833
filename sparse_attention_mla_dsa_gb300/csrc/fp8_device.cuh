// fp8_device.cuh -- E4M3 conversion, power-of-two block scales and the FP8
// tensor-core instruction, shared by the kernels of the 8-bit operators.
#pragma once

#include "dsa_device.cuh"

namespace dsa {
namespace fp8 {

constexpr int kBlock = 128;  // elements of k that share a scale

// Two floats to two E4M3 codes (round to nearest even, saturating, NaN to
// 0x7F): `lo` in the low byte.
__device__ __forceinline__ uint32_t e4m3x2(float lo, float hi) {
  uint16_t out;
  asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(out) : "f"(hi), "f"(lo));
  return out;
}
__device__ __forceinline__ uint32_t e4m3x4(float a, float b, float c, float d) {
  return e4m3x2(a, b) | (e4m3x2(c, d) << 16);
}

// Bits of the smallest power of two, 2^-126 at least, whose 448-fold is not
// below the finite float whose bits (without sign) are `top`: 448 is 1.75 * 2^8,
// so a mantissa above 1.75 (0x600000) carries into the exponent, which is then
// lowered by 8.  And its inverse's, exact: the exponent field is in 1 .. 247.
__device__ __forceinline__ uint32_t scale_bits(uint32_t top) {
  const uint32_t e = (top + 0x1FFFFFu) >> 23;
  return (e > 9u ? e - 8u : 1u) << 23;
}
__device__ __forceinline__ float inverse_scale(uint32_t scale) {
  return __uint_as_float((254u << 23) - scale);
}

// Instruction descriptor, kind::f8f6f4 with E4M3 A and B (format code 0), FP32
// accumulate, both operands K-major, M x N tile.
__host__ __device__ constexpr uint32_t idesc_e4m3(int m, int n) {
  return (1u << 4) | (static_cast<uint32_t>(n >> 3) << 17) | (static_cast<uint32_t>(m >> 4) << 24);
}
// High word of umma_desc_sw128_kmajor.
constexpr uint32_t kDescHigh = (1024u >> 4) | (1u << 14) | (2u << 29);
// D[tmem] (+)= A[smem] * B[smem]^T over 32 of k, issued by one thread; operands by
// the low words of their descriptors, which alone differ between MMAs: an add for
// each, nothing else.
template <uint32_t kHigh>
__device__ __forceinline__ void umma_low(uint32_t d_tmem, uint32_t a, uint32_t b, uint32_t idesc, uint32_t accumulate) {
  asm volatile(
      "{\n\t.reg .pred p;\n\t.reg .b64 a, b;\n\t"
      "setp.ne.b32 p, %4, 0;\n\t"
      "mov.b64 a, {%1, %5};\n\tmov.b64 b, {%2, %5};\n\t"
      "tcgen05.mma.cta_group::1.kind::f8f6f4 [%0], a, b, %3, p;\n\t}" ::"r"(d_tmem),
      "r"(a), "r"(b), "r"(idesc), "r"(accumulate), "n"(kHigh)
      : "memory");
}

// One lane of the whole warp.  A branch on it leaves the operands of MMAs and copies
// in uniform registers, which the warp shares; one on lane == 0 does not.  So where
// the lane waits inside, the others must stand still before those are set: its first
// wait is one that cannot be over yet (for copies that have only begun), and what
// follows the branch is a barrier of the CTA, no operation of the warp.  Otherwise
// the warp waits as a whole and the branch holds the instructions alone.
__device__ __forceinline__ bool elect_one() {
  uint32_t one;
  asm volatile("{\n\t.reg .pred p;\n\telect.sync _|p, 0xFFFFFFFF;\n\tselp.u32 %0, 1, 0, p;\n\t}" : "=r"(one));
  return one != 0;
}

// Which of two phases are complete (bits 0-1): two looks in a row, and not one after
// the other's answer, for which a thread waits long beside an epilogue's warps.
__device__ __forceinline__ uint32_t look2(uint64_t* b0, uint32_t p0, uint64_t* b1, uint32_t p1) {
  uint32_t r;
  asm volatile(
      "{\n\t.reg .pred p, q;\n\t.reg .b32 x, y;\n\t"
      "mbarrier.test_wait.parity.shared::cta.b64 p, [%1], %2;\n\t"
      "mbarrier.test_wait.parity.shared::cta.b64 q, [%3], %4;\n\t"
      "selp.b32 x, 1, 0, p;\n\tselp.b32 y, 2, 0, q;\n\tor.b32 %0, x, y;\n\t}"
      : "=r"(r)
      : "r"(smem_u32(b0)), "r"(p0), "r"(smem_u32(b1)), "r"(p1)
      : "memory");
  return r;
}

// (a.x * b.x + c.x, a.y * b.y + c.y), each rounded once.
__device__ __forceinline__ float2 fma2(float2 a, float2 b, float2 c) {
  float2 d;
  asm("{\n\t.reg .b64 a, b, c, d;\n\t"
      "mov.b64 a, {%2, %3};\n\tmov.b64 b, {%4, %5};\n\tmov.b64 c, {%6, %7};\n\t"
      "fma.rn.f32x2 d, a, b, c;\n\t"
      "mov.b64 {%0, %1}, d;\n\t}"
      : "=f"(d.x), "=f"(d.y)
      : "f"(a.x), "f"(a.y), "f"(b.x), "f"(b.y), "f"(c.x), "f"(c.y));
  return d;
}

// 32 consecutive 32-bit TMEM columns of this thread's lane, one wait for all.
__device__ __forceinline__ void tmem_load32(uint32_t taddr, float (&v)[32]) {
  uint32_t r[32];
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x32.b32 "
      "{%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,"
      "%16,%17,%18,%19,%20,%21,%22,%23,%24,%25,%26,%27,%28,%29,%30,%31}, [%32];\n\t"
      "tcgen05.wait::ld.sync.aligned;"
      : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]),
        "=r"(r[7]), "=r"(r[8]), "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]),
        "=r"(r[14]), "=r"(r[15]), "=r"(r[16]), "=r"(r[17]), "=r"(r[18]), "=r"(r[19]),
        "=r"(r[20]), "=r"(r[21]), "=r"(r[22]), "=r"(r[23]), "=r"(r[24]), "=r"(r[25]),
        "=r"(r[26]), "=r"(r[27]), "=r"(r[28]), "=r"(r[29]), "=r"(r[30]), "=r"(r[31])
      : "r"(taddr)
      : "memory");
#pragma unroll
  for (int i = 0; i < 32; ++i) v[i] = __uint_as_float(r[i]);
}

// The same in two steps: the registers hold the columns once tmem_wait32 of them
// is past (which waits for every load of the thread).
#define DSA_REGS32(c, r)                                                                                       \
  c(r[0]), c(r[1]), c(r[2]), c(r[3]), c(r[4]), c(r[5]), c(r[6]), c(r[7]), c(r[8]), c(r[9]), c(r[10]),          \
      c(r[11]), c(r[12]), c(r[13]), c(r[14]), c(r[15]), c(r[16]), c(r[17]), c(r[18]), c(r[19]), c(r[20]),      \
      c(r[21]), c(r[22]), c(r[23]), c(r[24]), c(r[25]), c(r[26]), c(r[27]), c(r[28]), c(r[29]), c(r[30]), c(r[31])
#define DSA_OUT(x) "=r"(x)
#define DSA_INOUT(x) "+r"(x)
__device__ __forceinline__ void tmem_issue32(uint32_t taddr, uint32_t (&r)[32]) {
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x32.b32 "
      "{%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,"
      "%16,%17,%18,%19,%20,%21,%22,%23,%24,%25,%26,%27,%28,%29,%30,%31}, [%32];"
      : DSA_REGS32(DSA_OUT, r)
      : "r"(taddr)
      : "memory");
}
__device__ __forceinline__ void tmem_wait32(uint32_t (&r)[32]) {
  asm volatile("tcgen05.wait::ld.sync.aligned;" : DSA_REGS32(DSA_INOUT, r) : : "memory");
}

// ------------------------------------------------------------------ clusters
// Address of `p` in the shared memory of CTA `rank` of the cluster.
__device__ __forceinline__ uint32_t map_to(const void* p, uint32_t rank) {
  uint32_t a;
  asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(a) : "r"(smem_u32(p)), "r"(rank));
  return a;
}
__device__ __forceinline__ uint32_t cluster_rank() {
  uint32_t r;
  asm volatile("mov.u32 %0, %%cluster_ctarank;" : "=r"(r));
  return r;
}
// Every thread of every CTA of the cluster; writes to shared memory before it
// are seen by all after it.
__device__ __forceinline__ void cluster_sync() {
  __syncwarp();
  asm volatile("barrier.cluster.arrive.release.aligned;\n\tbarrier.cluster.wait.acquire.aligned;" ::: "memory");
}
// Four floats at `p` in the CTA of rank `rank`.
__device__ __forceinline__ float4 ld_cluster_f4(const void* p, uint32_t rank) {
  float4 v;
  asm volatile("ld.shared::cluster.v4.f32 {%0, %1, %2, %3}, [%4];"
               : "=f"(v.x), "=f"(v.y), "=f"(v.z), "=f"(v.w)
               : "r"(map_to(p, rank))
               : "memory");
  return v;
}

}  // namespace fp8
}  // namespace dsa
