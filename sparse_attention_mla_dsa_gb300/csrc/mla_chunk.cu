// mla_chunk.cu -- dense causal attention of each request's new tokens over its
// paged FP8 latent cache.
//
// "glm5next_dsa/layer.rs", module header trap 4 (Q arrives absorbed into the
// 512-wide latent space) and decode_k (K and V are the same latent pool, slot =
// block * block_size + pos % block_size).  Per row, head and visible token j:
//   z_j = sm_scale * kv_scale * (q . e4m3(latent_j)),  p = softmax(z),
//   out = kv_scale * sum_j p_j e4m3(latent_j),  lse = log sum_j exp(z_j).
//
// One warp a (row, head): 16 dims a lane in registers, one pass over the tokens
// with the running maximum and sum of the softmax.
#include "dsa_device.cuh"
#include "dsa_internal.h"

namespace dsa {
namespace {

constexpr int kHeadsPerCta = 16;
constexpr int kThreads = 32 * kHeadsPerCta;

__device__ __forceinline__ void decode16(uint4 w, float (&x)[16]) {
  const uint32_t u[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    uint32_t h2;
    const uint16_t c = static_cast<uint16_t>(u[i >> 1] >> (16 * (i & 1)));
    asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(h2) : "h"(c));
    const float2 f = __half22float2(*reinterpret_cast<const __half2*>(&h2));
    x[2 * i] = f.x;
    x[2 * i + 1] = f.y;
  }
}

__global__ void __launch_bounds__(kThreads) mla_chunk_kernel(const ChunkParams p) {
  const int r = blockIdx.x, lane = threadIdx.x & 31;
  const int h = blockIdx.y * kHeadsPerCta + (threadIdx.x >> 5);
  grid_dep_launch();
  grid_dep_wait();
  const int32_t* start = p.seqs.row_start;
  int lo = 0, hi = p.seqs.seqs;  // the last request whose first row is <= r
  while (lo < hi) {
    const int mid = (lo + hi + 1) >> 1;
    if (mid < p.seqs.seqs && start[mid] <= r) lo = mid; else hi = mid - 1;
  }
  const int s = lo, r0 = start[s], r1 = start[s + 1], len = p.seqs.seq_lens[s];
  if (r < r0 || r >= r1) return;  // a row of no request
  const bool report = r == r0 && h == 0 && lane == 0;
  if (r0 < 0 || r1 > p.rows) {
    if (report) record_error(p.err, DSA_DEVERR_ROWS, s);
    return;
  }
  if (len < r1 - r0 || static_cast<int64_t>(len) > static_cast<int64_t>(p.seqs.max_blocks_per_seq) * p.seqs.block_size) {
    if (report) record_error(p.err, DSA_DEVERR_SEQ_LEN, s);
    return;
  }
  const int visible = len - (r1 - 1 - r);
  const int64_t line = static_cast<int64_t>(r) * p.heads + h;
  float q[16], o[16];
  const uint4* src = reinterpret_cast<const uint4*>(p.q + line * 512 + lane * 16);
  const uint4 qa = src[0], qb = src[1];
  const uint32_t w[8] = {qa.x, qa.y, qa.z, qa.w, qb.x, qb.y, qb.z, qb.w};
  const float scale = p.sm_scale * p.kv_scale * 1.4426950408889634f;
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    q[2 * i] = __uint_as_float(w[i] << 16) * scale;
    q[2 * i + 1] = __uint_as_float(w[i] & 0xFFFF0000u) * scale;
  }
#pragma unroll
  for (int i = 0; i < 16; ++i) o[i] = 0.0f;
  float m = -INFINITY, l = 0.0f, lc = 0.0f;  // lc: what l's additions have dropped
  const int32_t* bt = p.seqs.block_table + static_cast<int64_t>(s) * p.seqs.bt_stride;
  for (int b = 0; b * static_cast<int64_t>(p.seqs.block_size) < visible; ++b) {
    const int64_t slot0 = static_cast<int64_t>(bt[b]) * p.seqs.block_size;
    const int n = min(p.seqs.block_size, visible - b * p.seqs.block_size);
    for (int i = 0; i < n; ++i) {
      const int64_t slot = slot0 + i;
      if (slot < 0 || slot >= p.nslots) {
        if (lane == 0 && h == 0 && r == r1 - 1) record_error(p.err, DSA_DEVERR_BLOCK, s);
        continue;
      }
      float k[16];
      decode16(reinterpret_cast<const uint4*>(p.pool + slot * 512)[lane], k);
      float z = 0.0f;
#pragma unroll
      for (int d = 0; d < 16; ++d) z = fmaf(q[d], k[d], z);
#pragma unroll
      for (int d = 16; d > 0; d >>= 1) z += __shfl_xor_sync(0xFFFFFFFFu, z, d);
      if (z > m) {
        const float a = exp2f(m - z);
        l *= a;
        lc *= a;
#pragma unroll
        for (int d = 0; d < 16; ++d) o[d] *= a;
        m = z;
      }
      const float e = exp2f(z - m);
      const float y = e - lc, t = l + y;
      lc = (t - l) - y;
      l = t;
#pragma unroll
      for (int d = 0; d < 16; ++d) o[d] = fmaf(e, k[d], o[d]);
    }
  }
  const float inv = l != 0.0f ? p.kv_scale / l : 0.0f;
  uint32_t packed[8];
#pragma unroll
  for (int i = 0; i < 8; ++i)
    asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(packed[i]) : "f"(o[2 * i + 1] * inv), "f"(o[2 * i] * inv));
  uint4* dst = reinterpret_cast<uint4*>(p.out + line * 512 + lane * 16);
  dst[0] = make_uint4(packed[0], packed[1], packed[2], packed[3]);
  dst[1] = make_uint4(packed[4], packed[5], packed[6], packed[7]);
  if (p.lse != nullptr && lane == 0)
    p.lse[line] = l != 0.0f ? (m + log2f(l)) * 0.69314718055994531f : -INFINITY;
}

}  // namespace

cudaError_t launch_mla_chunk(const ChunkParams& p, cudaStream_t stream) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(p.rows, p.heads / kHeadsPerCta, 1);
  cfg.blockDim = dim3(kThreads, 1, 1);
  cfg.stream = stream;
  cudaLaunchAttribute attr[1] = {dependent_launch_attr()};
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, mla_chunk_kernel, p);
}

}  // namespace dsa
