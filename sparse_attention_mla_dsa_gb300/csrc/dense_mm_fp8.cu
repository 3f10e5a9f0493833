// dense_mm_fp8.cu -- matrix product of E4M3 operands with an FP32 scale for each
// block of 128 of k (of one activation row, of 128 weight rows).
//
//   c[m][n] = sum_j sa[m][j] sb[n / 128][j] * sum_{k in block j} a[m][k] b[n][k]
//
// The scales are any FP32 values, so a block's sum leaves the tensor core before
// its scale is applied: every block of k is an accumulator of its own in TMEM
// (four MMAs of 32 of k), which the epilogue warps read, scale and add in
// registers while the MMAs of the next blocks run into the other accumulators.
//
// Weight rows are M ("swap AB"):
//   A = 128 weight rows x 128 of k (TMA, 128-byte swizzle, K-major): one scale
//   B = kRows activation rows x 128 of k; rows >= m arrive as zeros
//   D = 128 x kRows FP32 (lane = weight row, column = activation row)
// A CTA takes one tile over one range of k.  Where the tiles alone leave SMs
// idle, up to eight CTAs, a cluster, share a tile's blocks of k, and add their
// sums through distributed shared memory in the order of the ranges: one launch,
// no workspace.
//
// Bound by the weight's bytes (32 x 4,096 x 32,768: 22.2 us, 6.1 TB/s); one token by
// the launch and the first loads (1 x 2,048 x 4,096: 4.4 us).
//
// Times in this file are of captured calls, up to eight weights in turn (those above
// 16 MB then come from HBM); two for one shape were measured on one box in turn.
//
// CTA roles (192 threads): warp 0 issues TMA, warp 1 owns TMEM and issues the
// MMAs (one thread), warps 2-5 are the epilogue (one TMEM lane quarter each).
#include <mutex>

#include "dsa_internal.h"
#include "fp8_device.cuh"

namespace dsa {
namespace {

using fp8::kBlock;

constexpr int kTileN = 128;                  // weight rows per tile (MMA M): one row of weight scales
constexpr int kThreads = 192;
constexpr int kEpiThreads = 128;
constexpr int kMaxSplits = 8;                // portable cluster size
constexpr int kGroup = 4;                    // blocks of k whose scales are fetched together
constexpr uint32_t kWBytes = kTileN * kBlock;

template <int kRows>
struct Shape {
  static constexpr int kStages = kRows <= 32 ? 5 : 4;
  static constexpr uint32_t kStageBytes = kWBytes + kRows * kBlock;
  static constexpr int kSlots = 4;                    // accumulators in TMEM
  static constexpr uint32_t kTmemCols = kRows * kSlots;
  static_assert(kStageBytes % 1024 == 0 && kTmemCols >= 32 && kTmemCols <= 256, "two CTAs an SM");
};

template <int kRows>
struct __align__(16) Ctl {
  float factor[2][kGroup][kRows];  // products of the scales, of two groups of blocks
  uint64_t full[Shape<kRows>::kStages];
  uint64_t empty[Shape<kRows>::kStages];
  uint64_t tfull[Shape<kRows>::kSlots];
  uint64_t tempty[Shape<kRows>::kSlots];
  uint64_t drain;
  uint32_t tmem_base;
  int abort_flag;
};
template <int kRows>
constexpr uint32_t smem_bytes() {
  return Shape<kRows>::kStages * Shape<kRows>::kStageBytes + sizeof(Ctl<kRows>) + 1024;  // + alignment slack
}

__device__ __forceinline__ void set_abort(int* flag, int* err, int tile) {
  record_error(err, DSA_DEVERR_TIMEOUT, tile);
  *reinterpret_cast<volatile int*>(flag) = 1;
}
__device__ __forceinline__ bool aborted(int* flag) { return *reinterpret_cast<volatile int*>(flag) != 0; }
__device__ __forceinline__ void epi_sync() { asm volatile("bar.sync 1, %0;" ::"n"(kEpiThreads) : "memory"); }

__device__ __forceinline__ void store_c(const Fp8MmParams& p, int64_t m, int n, float v) {
  if (p.c_fp32)
    static_cast<float*>(p.c)[m * p.n + n] = v;
  else
    static_cast<uint16_t*>(p.c)[m * p.n + n] = __bfloat16_as_ushort(__float2bfloat16_rn(v));
}

__device__ __forceinline__ uint32_t bf16x2(float lo, float hi) {
  uint32_t out;
  asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(out) : "f"(hi), "f"(lo));
  return out;
}
// Columns n .. n + 3 (n a multiple of 4), those that there are.
__device__ __forceinline__ void store_c4(const Fp8MmParams& p, int64_t m, int n, float4 v) {
  if ((p.n & 3) == 0) {
    if (p.c_fp32)
      *reinterpret_cast<float4*>(static_cast<float*>(p.c) + m * p.n + n) = v;
    else
      *reinterpret_cast<uint2*>(static_cast<uint16_t*>(p.c) + m * p.n + n) = make_uint2(bf16x2(v.x, v.y), bf16x2(v.z, v.w));
    return;
  }
  store_c(p, m, n, v.x);
  if (n + 1 < p.n) store_c(p, m, n + 1, v.y);
  if (n + 2 < p.n) store_c(p, m, n + 2, v.z);
  if (n + 3 < p.n) store_c(p, m, n + 3, v.w);
}

template <int kRows>
__global__ void __launch_bounds__(kThreads, 2)
    fp8_mm_rows_kernel(const __grid_constant__ CUtensorMap wmap, const __grid_constant__ CUtensorMap amap,
                       const Fp8MmParams p) {
  using S = Shape<kRows>;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = smem_raw + ((1024u - (smem_u32(smem_raw) & 1023u)) & 1023u);
  Ctl<kRows>* ctl = reinterpret_cast<Ctl<kRows>*>(smem + S::kStages * S::kStageBytes);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int split = blockIdx.x, tile = blockIdx.z;
  const int kb_begin = split * p.kb_per_split;
  const int nkb = min(p.kb_per_split, p.kblocks - kb_begin);  // >= 1 by the plan
  const int n0 = tile * kTileN, m0 = blockIdx.y * kRows;

  if (threadIdx.x == 0) {
    for (int s = 0; s < S::kStages; ++s) {
      mbar_init(&ctl->full[s], 1);
      mbar_init(&ctl->empty[s], 1);
    }
    for (int s = 0; s < S::kSlots; ++s) {
      mbar_init(&ctl->tfull[s], 1);
      mbar_init(&ctl->tempty[s], kEpiThreads / 32);
    }
    mbar_init(&ctl->drain, 1);
    ctl->abort_flag = 0;
    fence_mbar_init();
    tma_prefetch_map(&wmap);
    tma_prefetch_map(&amap);
  }
  if (warp == 1) tmem_alloc_then_launch(&ctl->tmem_base, S::kTmemCols);
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = ctl->tmem_base;

  if (warp == 0) {
    // Any operand may come from the kernel before (a weight just quantised), so
    // nothing is loaded before the dependency wait; the first tiles of the weight
    // are on their way to L2 meanwhile, where a write of that kernel lands too.
    if (lane == 0)
      for (int i = 0; i < min(nkb, S::kStages); ++i) tma_prefetch_l2_2d(&wmap, (kb_begin + i) * kBlock, n0);
    __syncwarp();
    grid_dep_wait();
    if (lane == 0) {
      const uint64_t w_policy = l2_policy_evict_first();
      uint64_t a_policy;
      asm volatile("createpolicy.fractional.L2::evict_normal.b64 %0, 1.0;" : "=l"(a_policy));
      int issued = 0;
      for (; issued < nkb; ++issued) {
        if (aborted(&ctl->abort_flag)) break;
        const int s = issued % S::kStages;
        if (issued >= S::kStages && !mbar_wait(&ctl->empty[s], ((issued / S::kStages) - 1) & 1, p.wait_ns)) {
          set_abort(&ctl->abort_flag, p.err, tile);
          break;
        }
        uint8_t* dst = smem + s * S::kStageBytes;
        const int32_t x = (kb_begin + issued) * kBlock;
        mbar_arrive_expect_tx(&ctl->full[s], S::kStageBytes);
        tma_load_2d(dst, &wmap, &ctl->full[s], x, n0, w_policy);
        tma_load_2d(dst + kWBytes, &amap, &ctl->full[s], x, m0, a_policy);
      }
      // Never leave with a copy in flight: wait (bounded) for the last loads.
      for (int i = max(0, issued - S::kStages); i < issued; ++i)
        mbar_wait(&ctl->full[i % S::kStages], (i / S::kStages) & 1, kDrainWaitNs);
    }
  } else if (warp == 1) {
    grid_dep_wait();  // no wait's clock starts before (the copies do not)
    if (fp8::elect_one()) {
      constexpr uint32_t idesc = fp8::idesc_e4m3(kTileN, kRows);
      const uint32_t desc0 = static_cast<uint32_t>(umma_desc_sw128_kmajor(smem_u32(smem)));
      uint32_t s = 0, round = 0;  // block i's stage, and how often that was filled before
      for (int i = 0; i < nkb; ++i) {
        const uint32_t t = i % S::kSlots;
        const uint32_t empty_at = (i / S::kSlots - 1) & 1;  // (the first ones: the phase before the first)
        const uint32_t there = fp8::look2(&ctl->full[s], round & 1, &ctl->tempty[t], empty_at);
        if (((there & 1) == 0 && !mbar_wait(&ctl->full[s], round & 1, p.wait_ns)) ||
            ((there & 2) == 0 && !mbar_wait(&ctl->tempty[t], empty_at, p.wait_ns))) {
          set_abort(&ctl->abort_flag, p.err, tile);
          break;
        }
        tc_fence_after();
        const uint32_t w = desc0 + s * (S::kStageBytes >> 4);
#pragma unroll
        for (int kk = 0; kk < kBlock / 32; ++kk)
          fp8::umma_low<fp8::kDescHigh>(tmem + t * kRows, w + kk * 2, w + (kWBytes >> 4) + kk * 2, idesc, kk != 0);
        umma_commit(&ctl->empty[s]);
        umma_commit(&ctl->tfull[t]);
        if (++s == S::kStages) {
          s = 0;
          ++round;
        }
      }
      umma_commit(&ctl->drain);
      mbar_wait(&ctl->drain, 0, kDrainWaitNs);
    }
  }

  float2 acc[kRows / 2];
#pragma unroll
  for (int i = 0; i < kRows / 2; ++i) acc[i] = make_float2(0.0f, 0.0f);
  const int quarter = warp & 3, et = threadIdx.x - 64;
  const int row_n = quarter * 32 + lane;  // this thread's weight row in the tile
  if (warp >= 2) {
    // Thread et fetches activation row et's scales, four blocks at a time, two
    // groups ahead of their use.
    grid_dep_wait();
    const bool fetches = et < kRows && m0 + et < p.m;
    const float* sa = p.a_scale + static_cast<int64_t>(fetches ? m0 + et : 0) * p.kblocks + kb_begin;
    const float* sb = p.b_scale + static_cast<int64_t>(tile) * p.kblocks + kb_begin;
    float next[kGroup];
    auto fetch = [&](int i0) {
#pragma unroll
      for (int j = 0; j < kGroup; ++j) next[j] = fetches && i0 + j < nkb ? sa[i0 + j] * sb[i0 + j] : 0.0f;
    };
    auto put = [&](int g) {
      if (et < kRows)
#pragma unroll
        for (int j = 0; j < kGroup; ++j) ctl->factor[g & 1][j][et] = next[j];
    };
    fetch(0);
    put(0);
    fetch(kGroup);
    bool ok = true;
    for (int i0 = 0; i0 < nkb; i0 += kGroup) {
      const int g = i0 / kGroup;
      epi_sync();  // group g is in place, and nobody reads the group before any more
      put(g + 1);
      fetch(i0 + 2 * kGroup);
      for (int i = i0; i < min(i0 + kGroup, nkb) && ok; ++i) {
        const int t = i % S::kSlots;
        int w = 1;
        if (lane == 0) w = mbar_wait(&ctl->tfull[t], (i / S::kSlots) & 1, p.wait_ns) ? 1 : 0;
        ok = __shfl_sync(0xFFFFFFFFu, w, 0) != 0;
        if (!ok) {
          if (lane == 0) set_abort(&ctl->abort_flag, p.err, tile);
          break;
        }
        tc_fence_after();
        const uint32_t src = tmem + (static_cast<uint32_t>(quarter * 32) << 16) + t * kRows;
        const float* f = ctl->factor[g & 1][i - i0];
        if constexpr (kRows == 16) {
          float v[16];
          tmem_load16(src, v);
#pragma unroll
          for (int c = 0; c < 16; c += 4) {
            const float4 f4 = *reinterpret_cast<const float4*>(f + c);
            acc[c / 2] = fp8::fma2(make_float2(v[c], v[c + 1]), make_float2(f4.x, f4.y), acc[c / 2]);
            acc[c / 2 + 1] = fp8::fma2(make_float2(v[c + 2], v[c + 3]), make_float2(f4.z, f4.w), acc[c / 2 + 1]);
          }
        } else {
#pragma unroll
          for (int c0 = 0; c0 < kRows; c0 += 32) {
            float v[32];
            fp8::tmem_load32(src + c0, v);
#pragma unroll
            for (int c = 0; c < 32; c += 4) {
              const float4 f4 = *reinterpret_cast<const float4*>(f + c0 + c);
              float2& x = acc[(c0 + c) / 2];
              float2& y = acc[(c0 + c) / 2 + 1];
              x = fp8::fma2(make_float2(v[c], v[c + 1]), make_float2(f4.x, f4.y), x);
              y = fp8::fma2(make_float2(v[c + 2], v[c + 3]), make_float2(f4.z, f4.w), y);
            }
          }
        }
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(&ctl->tempty[t]);
      }
    }
  }

  if (p.splits == 1) {
    if (warp >= 2 && n0 + row_n < p.n) {
#pragma unroll
      for (int c = 0; c < kRows; ++c)
        if (m0 + c < p.m) store_c(p, m0 + c, n0 + row_n, c & 1 ? acc[c / 2].y : acc[c / 2].x);
    }
    tc_fence_before();
    __syncthreads();
  } else {
    // This range's sums into shared memory [activation row][weight row], over the
    // stages: their copies and MMAs are complete once every role is here.
    tc_fence_before();
    __syncthreads();
    float* part = reinterpret_cast<float*>(smem);
    if (warp >= 2) {
#pragma unroll
      for (int c = 0; c < kRows; ++c) part[c * kTileN + row_n] = c & 1 ? acc[c / 2].y : acc[c / 2].x;
    }
    fp8::cluster_sync();
    // The sums of the ranges, four columns and a row a thread, the rows shared out
    // among the cluster's warps.
    const int rows_here = min(kRows, p.m - m0), n = n0 + lane * 4;
    if (warp >= 2 && n < p.n) {
      for (int c = split * (kEpiThreads / 32) + warp - 2; c < rows_here; c += p.splits * (kEpiThreads / 32)) {
        float4 v[kMaxSplits];
#pragma unroll
        for (int r = 0; r < kMaxSplits; ++r)
          if (r < p.splits) v[r] = fp8::ld_cluster_f4(part + c * kTileN + lane * 4, r);
        float4 sum = v[0];
#pragma unroll
        for (int r = 1; r < kMaxSplits; ++r)
          if (r < p.splits) {
            sum.x += v[r].x;
            sum.y += v[r].y;
            sum.z += v[r].z;
            sum.w += v[r].w;
          }
        store_c4(p, m0 + c, n, sum);
      }
    }
    fp8::cluster_sync();  // nobody reads this CTA's shared memory any more
  }
  if (warp == 1) {
    tc_fence_after();
    tmem_dealloc(tmem, S::kTmemCols);
  }
}

// ------------------------------------------------------------------ shared by the tiles below
constexpr uint32_t kOutBytes = 32 * 128;          // 32 rows x 128 bytes of the output
constexpr int kScaleBlocks = 16;                  // blocks of k whose scales are fetched together
constexpr int kScalePitch = 130;                  // floats between their rows

// Bounded waits; a timeout is recorded and marks the CTA, whose later waits are
// skipped.  (All of it inline: around a call the accumulators' registers could not
// stay where they are.)
struct Waits {
  int* flag;
  int* err;
  uint64_t limit_ns;
  __device__ __forceinline__ bool aborted() const { return *reinterpret_cast<volatile int*>(flag) != 0; }
  // Of one thread, without marking.
  __device__ __forceinline__ bool polled(uint64_t* bar, uint32_t parity) const {
    if (limit_ns >= kShortWaitNs && mbar_try_wait(bar, parity)) return true;
    const uint64_t t0 = global_ns();
    for (uint32_t i = 1; i < (1u << 30) && !aborted(); ++i) {
      if (mbar_try_wait_hint(bar, parity, limit_ns < kShortWaitNs ? 32 : kSuspendHintNs)) return true;
      if (((i & 15u) == 0 || limit_ns < kShortWaitNs) && global_ns() - t0 > limit_ns) break;
    }
    if (!aborted()) record_error(err, DSA_DEVERR_TIMEOUT, -1);
    return false;
  }
  __device__ __forceinline__ bool one(uint64_t* bar, uint32_t parity) const {
    if (polled(bar, parity)) return true;
    *reinterpret_cast<volatile int*>(flag) = 1;
    return false;
  }
  // Of a whole warp: every lane polls, one goes on where it is not there yet.
  __device__ __forceinline__ bool warp(uint64_t* bar, uint32_t parity, int lane) const {
    const bool done = limit_ns >= kShortWaitNs && mbar_try_wait(bar, parity);
    if (__all_sync(0xFFFFFFFFu, done)) return true;
    int ok = 1;
    if (lane == 0) ok = one(bar, parity) ? 1 : 0;
    return __shfl_sync(0xFFFFFFFFu, ok, 0) != 0;
  }
};

// Scales of 64 activation rows (half of 128, from row m0 on) in the kScaleBlocks
// blocks from kb0 on, turned to [block][row]: a warp takes two rows x 16 blocks a
// load, kAtOnce of them at once: a round's latency is a small tile's (300 x 4,096 x
// 4,096 13.1 us with 8, 10.9 with all 32).  Rows and blocks outside the tensor get
// scales of others.
template <int kAtOnce>
__device__ __forceinline__ void fetch_scales(const Fp8MmParams& p, float* sa, int m0, int half, int lane, int kb0) {
  const int kb_in = lane & (kScaleBlocks - 1), odd = lane >> 4;
  const int row0 = m0 + half * 64 + odd, kb = min(kb0 + kb_in, p.kblocks - 1);
  float* dst = sa + kb_in * kScalePitch + half * 64 + odd;
#pragma unroll 1
  for (int r = 0; r < 64; r += 2 * kAtOnce) {
    float v[kAtOnce];
#pragma unroll
    for (int u = 0; u < kAtOnce; ++u) v[u] = p.a_scale[static_cast<int64_t>(min(row0 + r + 2 * u, p.m - 1)) * p.kblocks + kb];
#pragma unroll
    for (int u = 0; u < kAtOnce; ++u) dst[r + 2 * u] = v[u];
  }
}

// A warp's 32 rows (a lane each) x kCols columns of the output, through kBufs buffers
// of kOutBytes; what lies outside the output is not stored.  The copies out may still
// run when it returns.
template <int kCols, int kBufs>
__device__ __forceinline__ void store_tile(const Fp8MmParams& p, const CUtensorMap& cmap, const float (&acc)[kCols],
                                           uint8_t* outs, int row0, int col0, int lane) {
  const bool by_tma = (static_cast<int64_t>(p.n) * (p.c_fp32 ? 4 : 2)) % 16 == 0;
#pragma unroll
  for (int c = 0; c < kCols; c += 32) {
    if (by_tma && !p.c_fp32 && (c & 32) != 0) continue;  // (64 columns at a time)
    uint8_t* out = outs + ((by_tma && !p.c_fp32 ? c / 64 : c / 32) % kBufs) * kOutBytes;
    if (lane == 0) asm volatile("cp.async.bulk.wait_group.read %0;" ::"n"(kBufs - 1) : "memory");
    __syncwarp();
    if (by_tma) {
      // 128 bytes of each row (64 bf16 columns or 32 FP32 ones), in the 128-byte swizzle.
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        uint4 w;
        if (p.c_fp32) {
          const int b = c + e * 4;
          w = make_uint4(__float_as_uint(acc[b]), __float_as_uint(acc[b + 1]), __float_as_uint(acc[b + 2]),
                         __float_as_uint(acc[b + 3]));
        } else {
          const int b = (c & ~63) + e * 8;
          w = make_uint4(bf16x2(acc[b], acc[b + 1]), bf16x2(acc[b + 2], acc[b + 3]),
                         bf16x2(acc[b + 4], acc[b + 5]), bf16x2(acc[b + 6], acc[b + 7]));
        }
        *reinterpret_cast<uint4*>(out + lane * 128 + ((e ^ (lane & 7)) * 16)) = w;
      }
      fence_proxy_async_smem();
      __syncwarp();
      if (lane == 0)
        asm volatile(
            "cp.async.bulk.tensor.2d.global.shared::cta.tile.bulk_group [%0, {%1, %2}], [%3];\n\t"
            "cp.async.bulk.commit_group;" ::"l"(reinterpret_cast<uint64_t>(&cmap)),
            "r"(col0 + c), "r"(row0), "r"(smem_u32(out))
            : "memory");
    } else {
      // Rows that are not multiples of 16 bytes: turned in shared memory, so that
      // neighbouring lanes store neighbouring columns.
      float* turn = reinterpret_cast<float*>(out);
#pragma unroll
      for (int e = 0; e < 32; ++e) turn[lane * 32 + (e ^ lane)] = acc[c + e];
      __syncwarp();
      if (col0 + c + lane < p.n)
        for (int r = 0; r < min(32, p.m - row0); ++r) store_c(p, row0 + r, col0 + c + lane, turn[r * 32 + (lane ^ r)]);
      __syncwarp();
    }
  }
}

// ------------------------------------------------------------------ some rows more
// Tiles of 128 activation rows x 128 weight rows, a CTA each, for what is too much for
// the row tiles above and too little for the pairs below.  Activation rows are M:
//   A = 128 activation rows x 128 of k,  B = 128 weight rows x 128 of k
//   D = 128 x 128 FP32 (lane = activation row, column = weight row), four in turn
// so a thread of the epilogue has one row and columns of one row of weight scales: one
// factor a block of k, where row tiles read one for every column from shared memory,
// whose bandwidth then bounds them (256 x 4,096 x 32,768: 40.6 us, by row tiles 69.4).  Up to
// four CTAs, a cluster, share a tile's blocks of k as above.
//
// Bound by 32 KB from L2 for each block and CTA and the epilogue's reads of TMEM (512 x
// 4,096 x 4,096: 11.9 us, 1.4 PFLOP/s).  Where k is not a multiple of 128 a block of a
// row lies in two lines of L2 (777 x 1,003 with k 4,112: 12.7 us, with 4,224 10.8).
//
// Roles (384 threads): warp 0 copies, warp 1 issues the MMAs, warps 2-3 fetch the
// activation scales and turn them in shared memory, warps 4-11 are the epilogue (a
// TMEM lane quarter and 64 columns each).
namespace block {

constexpr int kTile = 128;
constexpr int kThreads = 384;
constexpr int kFirstEpiWarp = 4;
constexpr int kEpiWarps = 8;
constexpr int kCols = 64;                         // columns of an epilogue warp
constexpr int kMaxSplits = 4;
constexpr int kStages = 6;
constexpr uint32_t kOperandBytes = 128 * kBlock;
constexpr uint32_t kStageBytes = 2 * kOperandBytes;
constexpr uint32_t kSlots = 4;
constexpr uint32_t kTmemCols = kSlots * kTile;
constexpr int kPartPitch = kTile + 4;             // floats between rows of a range's sums
constexpr int kAtOnce = 2;                        // rows of sums that a thread has on their way

struct __align__(8) Ctl {
  uint64_t full[kStages];
  uint64_t empty[kStages];
  uint64_t tfull[kSlots];
  uint64_t tempty[kSlots];
  uint64_t sfull[2];
  uint64_t sempty[2];
  uint64_t drain;
  uint32_t tmem_base;
  int abort_flag;
  float sb[2][kScaleBlocks];
  float sa[2][kScaleBlocks * kScalePitch];        // [block][row]
};
constexpr uint32_t kCtlOff = kStages * kStageBytes;
constexpr uint32_t kSmemBytes = kCtlOff + sizeof(Ctl) + 1024;  // + alignment slack
static_assert(kSmemBytes <= 227 * 1024 && kCtlOff % 8 == 0, "shared memory budget");
static_assert(128 * kPartPitch * 4 <= kCtlOff && kEpiWarps * kOutBytes <= kCtlOff, "sums and outputs take the place of the stages");

__global__ void __launch_bounds__(kThreads, 1)
    fp8_mm_block_kernel(const __grid_constant__ CUtensorMap wmap, const __grid_constant__ CUtensorMap amap,
                        const __grid_constant__ CUtensorMap cmap, const Fp8MmParams p) {
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = smem_raw + ((1024u - (smem_u32(smem_raw) & 1023u)) & 1023u);
  Ctl* ctl = reinterpret_cast<Ctl*>(smem + kCtlOff);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int split = blockIdx.x, m0 = blockIdx.y * kTile, n0 = blockIdx.z * kTile;
  const int kb_begin = split * p.kb_per_split;
  const int nkb = min(p.kb_per_split, p.kblocks - kb_begin);  // >= 1 by the plan
  const Waits waits{&ctl->abort_flag, p.err, p.wait_ns};

  if (threadIdx.x == 0) {
    for (int s = 0; s < kStages; ++s) {
      mbar_init(&ctl->full[s], 1);
      mbar_init(&ctl->empty[s], 1);
    }
    for (uint32_t s = 0; s < kSlots; ++s) {
      mbar_init(&ctl->tfull[s], 1);
      mbar_init(&ctl->tempty[s], kEpiWarps);
    }
    for (int s = 0; s < 2; ++s) {
      mbar_init(&ctl->sfull[s], 2);
      mbar_init(&ctl->sempty[s], kEpiWarps);
    }
    mbar_init(&ctl->drain, 1);
    ctl->abort_flag = 0;
    fence_mbar_init();
    tma_prefetch_map(&wmap);
    tma_prefetch_map(&amap);
    tma_prefetch_map(&cmap);
  }
  if (warp == 1) tmem_alloc_then_launch(&ctl->tmem_base, kTmemCols);
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = ctl->tmem_base;

  float acc[kCols];
#pragma unroll
  for (int c = 0; c < kCols; ++c) acc[c] = 0.0f;
  const int quarter = warp & 3, half = (warp - kFirstEpiWarp) >> 2;
  if (warp == 0) {
    // -------------------------------------------------------------- copies
    if (lane == 0)
      for (int i = 0; i < min(nkb, kStages); ++i) tma_prefetch_l2_2d(&wmap, (kb_begin + i) * kBlock, n0);  // (as above)
    __syncwarp();
    grid_dep_wait();
    if (fp8::elect_one()) {
      uint64_t policy;
      asm volatile("createpolicy.fractional.L2::evict_normal.b64 %0, 1.0;" : "=l"(policy));
      auto copy = [&](int i, const CUtensorMap* map, uint32_t at, int row) {
        const int s = i % kStages;
        tma_load_2d(smem + s * kStageBytes + at, map, &ctl->full[s], (kb_begin + i) * kBlock, row, policy);
      };
      int issued = 0;
      for (; issued < nkb; ++issued) {
        const int s = issued % kStages;
        if (issued >= kStages && !waits.one(&ctl->empty[s], (issued / kStages - 1) & 1)) break;
        mbar_arrive_expect_tx(&ctl->full[s], kStageBytes);
        copy(issued, &wmap, kOperandBytes, n0);
        copy(issued, &amap, 0, m0);
      }
      // Never leave with a copy in flight: wait (bounded) for the last loads.
      for (int i = max(0, issued - kStages); i < issued; ++i)
        mbar_wait(&ctl->full[i % kStages], (i / kStages) & 1, kDrainWaitNs);
    }
  } else if (warp == 1) {
    // -------------------------------------------------------------- MMAs
    grid_dep_wait();  // no wait's clock starts before (the copies do not)
    if (fp8::elect_one()) {
      constexpr uint32_t idesc = fp8::idesc_e4m3(kTile, kTile);
      const uint32_t desc0 = static_cast<uint32_t>(umma_desc_sw128_kmajor(smem_u32(smem)));
      uint32_t s = 0, round = 0;
      for (int i = 0; i < nkb; ++i) {
        const uint32_t d = i % kSlots, empty_at = (i / kSlots - 1) & 1;  // (the first ones: the phase before the first)
        const uint32_t there = fp8::look2(&ctl->full[s], round & 1, &ctl->tempty[d], empty_at);
        if (((there & 1) == 0 && !waits.one(&ctl->full[s], round & 1)) ||
            ((there & 2) == 0 && !waits.one(&ctl->tempty[d], empty_at)))
          break;
        tc_fence_after();
        const uint32_t a = desc0 + s * (kStageBytes >> 4);
#pragma unroll
        for (int kk = 0; kk < kBlock / 32; ++kk)
          fp8::umma_low<fp8::kDescHigh>(tmem + d * kTile, a + kk * 2, a + (kOperandBytes >> 4) + kk * 2, idesc, kk != 0);
        umma_commit(&ctl->empty[s]);
        umma_commit(&ctl->tfull[d]);
        if (++s == kStages) {
          s = 0;
          ++round;
        }
      }
      umma_commit(&ctl->drain);
      mbar_wait(&ctl->drain, 0, kDrainWaitNs);
    }
  } else if (warp < kFirstEpiWarp) {
    // -------------------------------------------------------------- scales
    grid_dep_wait();
    const float* sb = p.b_scale + static_cast<int64_t>(blockIdx.z) * p.kblocks;
    for (int kb0 = 0, g = 0; kb0 < nkb; kb0 += kScaleBlocks, ++g) {
      if (g >= 2 && !waits.warp(&ctl->sempty[g & 1], (g / 2 - 1) & 1, lane)) break;
      fetch_scales<32>(p, ctl->sa[g & 1], m0, warp - 2, lane, kb_begin + kb0);
      if (warp == 2 && lane < kScaleBlocks) ctl->sb[g & 1][lane] = sb[min(kb_begin + kb0 + lane, p.kblocks - 1)];
      __syncwarp();
      if (lane == 0) mbar_arrive(&ctl->sfull[g & 1]);
    }
  } else {
    // -------------------------------------------------------------- epilogue
    grid_dep_wait();  // as above, and the kernel before may still read the output
    const uint32_t src = tmem + (static_cast<uint32_t>(quarter * 32) << 16) + half * kCols;
    // (After a wait that gave up the warps go on, with waits that no longer wait.)
    for (int kb0 = 0, g = 0, i = 0; kb0 < nkb; kb0 += kScaleBlocks, ++g) {
      waits.warp(&ctl->sfull[g & 1], (g / 2) & 1, lane);
      const float* sa = ctl->sa[g & 1] + quarter * 32 + lane;
      const float* sb = ctl->sb[g & 1];
      const int n = min(kScaleBlocks, nkb - kb0);
#pragma unroll 1
      for (int j = 0; j < n; ++j, ++i) {
        const uint32_t d = i % kSlots;
        const float f = sa[j * kScalePitch] * sb[j];
        waits.warp(&ctl->tfull[d], (i / kSlots) & 1, lane);
        tc_fence_after();
#pragma unroll
        for (int c = 0; c < kCols; c += 32) {
          float v[32];
          fp8::tmem_load32(src + d * kTile + c, v);
          if (c + 32 == kCols) {  // read: the accumulator is free
            tc_fence_before();
            __syncwarp();
            if (lane == 0) mbar_arrive(&ctl->tempty[d]);
          }
#pragma unroll
          for (int e = 0; e < 32; ++e) acc[c + e] = fmaf(v[e], f, acc[c + e]);
        }
      }
      __syncwarp();
      if (lane == 0) mbar_arrive(&ctl->sempty[g & 1]);
    }
    const int row0 = m0 + quarter * 32, col0 = n0 + half * kCols;
    // The last accumulator has been read, so every copy and MMA is complete and the
    // stages are free.
    if (p.splits > 1) {
      float4* part = reinterpret_cast<float4*>(reinterpret_cast<float*>(smem) + (quarter * 32 + lane) * kPartPitch + half * kCols);
#pragma unroll
      for (int c = 0; c < kCols; c += 4) part[c / 4] = make_float4(acc[c], acc[c + 1], acc[c + 2], acc[c + 3]);
    } else if (row0 < p.m && col0 < p.n && !__any_sync(0xFFFFFFFFu, waits.aborted())) {
      store_tile<kCols, 1>(p, cmap, acc, smem + (warp - kFirstEpiWarp) * kOutBytes, row0, col0, lane);
      if (lane == 0) asm volatile("cp.async.bulk.wait_group 0;" ::: "memory");  // the stores are complete
    }
  }

  tc_fence_before();
  __syncthreads();
  if (p.splits > 1) {
    fp8::cluster_sync();
    // The sums of the ranges, four columns of a row a thread, the rows shared out among
    // the cluster's CTAs.
    const int e = threadIdx.x - kFirstEpiWarp * 32, n = n0 + (e & 31) * 4;
    const int rows = (kTile + p.splits - 1) / p.splits, r_end = min(min((split + 1) * rows, kTile), p.m - m0);
    if (warp >= kFirstEpiWarp && n < p.n)
      for (int r0 = split * rows + (e >> 5); r0 < r_end; r0 += 8 * kAtOnce) {
        float4 v[kAtOnce][kMaxSplits];
#pragma unroll
        for (int u = 0; u < kAtOnce; ++u)
#pragma unroll
          for (int q = 0; q < kMaxSplits; ++q)
            if (q < p.splits && r0 + 8 * u < r_end)
              v[u][q] = fp8::ld_cluster_f4(reinterpret_cast<float*>(smem) + (r0 + 8 * u) * kPartPitch + (e & 31) * 4, q);
#pragma unroll
        for (int u = 0; u < kAtOnce; ++u) {
          if (r0 + 8 * u >= r_end) break;
          float4 sum = v[u][0];
#pragma unroll
          for (int q = 1; q < kMaxSplits; ++q)
            if (q < p.splits) {
              sum.x += v[u][q].x;
              sum.y += v[u][q].y;
              sum.z += v[u][q].z;
              sum.w += v[u][q].w;
            }
          store_c4(p, m0 + r0 + 8 * u, n, sum);
        }
      }
    fp8::cluster_sync();  // nobody reads this CTA's shared memory any more
  }
  if (warp == 1) {
    tc_fence_after();
    tmem_dealloc(tmem, kTmemCols);
  }
}

}  // namespace block

// ------------------------------------------------------------------ many rows
// Tiles of 256 activation rows x 256 weight rows for a pair of CTAs (a cluster of
// two, cta_group::2): CTA r multiplies rows 128 r .. 128 r + 127 of the tile by all
// 256 weight rows, of which it copies half, so 32 KB a CTA and block of k feed the
// tensor core for 544 clocks; a CTA by itself would need 48.  Activation rows are M:
//   A = 128 rows of each CTA x 128 of k,  B = 2 x 64 weight rows of each CTA x 128 of k
//   D = 128 x 128 FP32 in each CTA's TMEM (lane = row, column = weight row) for either
//       half of the weight rows, two of each in turn
// so a thread of the epilogue has one row and columns of one row of weight scales:
// one factor a block of k.
//
// What bounds it is how soon an accumulator is read, scaled and free again (by
// halves the MMAs of three others, not of one, run meanwhile) and that the epilogue's
// reads of TMEM take turns with the MMAs.  Eight epilogue warps of 128 columns and
// not sixteen of 64 (1,024 x 4,096 x 32,768: 108 us, 111 with sixteen): beside
// their instructions the one thread that issues the MMAs has to find room, which is
// also why it looks at three barriers at once and adds to descriptors' low words only
// (one after the other 121 us for 108; a whole warp that waits, with a lane elected
// for the MMAs alone, 120.6 for 103.2, and 13.8 for 10.8 at 300 x 4,096 x 4,096).  The activation scales come through shared memory,
// turned there by two warps: a load by the epilogue would touch a line for each row.
// The outputs leave through shared memory by TMA, behind the next tile's MMAs.
//
// Persistent: one pair for every two SMs, tiles in turn.  (Two or four pairs that share
// a tile's blocks of k, their sums added through distributed shared memory: 512 x 4,096
// x 4,096 16.6 us for 17.3, 128 x 2,048 x 4,096 11.9 where row tiles take 8.0: not kept.)
//
// Roles (384 threads a CTA): warp 0 copies, warp 1 of the leader issues both CTAs'
// MMAs, warps 2-3 fetch the scales, warps 4-11 are the epilogue (a TMEM lane quarter
// and half of the columns each) and get the registers that the first four give up.
namespace pair {

constexpr int kTile = 256;
constexpr int kThreads = 384;
constexpr int kFirstEpiWarp = 4;
constexpr int kEpiWarps = 8;
constexpr int kCols = 128;                        // columns of an epilogue warp
constexpr int kFewRegs = 72, kManyRegs = 216;
static_assert(128 * kFewRegs + 256 * kManyRegs <= kThreads * 168, "register split");
constexpr int kStages = 4;
constexpr uint32_t kOperandBytes = 128 * kBlock;
constexpr uint32_t kStageBytes = 2 * kOperandBytes;
constexpr uint32_t kTmemCols = 512;
constexpr int kGroupTiles = 16;                   // row tiles that share a sweep of the weight

struct __align__(8) Ctl {
  uint64_t full[kStages];    // leader's: both CTAs' copies of a stage
  uint64_t empty[kStages];
  uint64_t tfull[4];         // [block of k % 2][half]
  uint64_t tempty[4];        // leader's
  uint64_t sfull[2];
  uint64_t sempty[2];
  uint64_t drain;
  uint64_t never;
  uint32_t tmem_base;
  int abort_flag;
  float sb[2][2][kScaleBlocks];                 // weight scales of the two halves
  float sa[2][kScaleBlocks * kScalePitch];      // this CTA's rows' scales, [block][row]
};
constexpr uint32_t kCtlOff = kStages * kStageBytes + kEpiWarps * 2 * kOutBytes;
constexpr uint32_t kSmemBytes = kCtlOff + sizeof(Ctl) + 1024;  // + alignment slack
static_assert(kSmemBytes <= 227 * 1024 && kCtlOff % 8 == 0, "shared memory budget");

// Waits that mark both CTAs of the pair.
struct PairWaits : Waits {
  __device__ __forceinline__ bool one(uint64_t* bar, uint32_t parity) const {
    if (polled(bar, parity)) return true;
    for (uint32_t r = 0; r < 2; ++r)
      asm volatile("st.volatile.shared::cluster.u32 [%0], %1;" ::"r"(fp8::map_to(flag, r)), "r"(1) : "memory");
    return false;
  }
  __device__ __forceinline__ bool warp(uint64_t* bar, uint32_t parity, int lane) const {
    const bool done = limit_ns >= kShortWaitNs && mbar_try_wait(bar, parity);
    if (__all_sync(0xFFFFFFFFu, done)) return true;
    int ok = 1;
    if (lane == 0) ok = one(bar, parity) ? 1 : 0;
    return __shfl_sync(0xFFFFFFFFu, ok, 0) != 0;
  }
};
// Which of three phases are complete (bits 0-2): three looks in a row, and not one
// after the other's answer, for which a thread waits long beside the epilogue's warps.
__device__ __forceinline__ uint32_t look3(uint64_t* b0, uint32_t p0, uint64_t* b1, uint64_t* b2, uint32_t p12) {
  uint32_t r;
  asm volatile(
      "{\n\t.reg .pred p, q, r;\n\t.reg .b32 x, y, z;\n\t"
      "mbarrier.test_wait.parity.shared::cta.b64 p, [%1], %2;\n\t"
      "mbarrier.test_wait.parity.shared::cta.b64 q, [%3], %5;\n\t"
      "mbarrier.test_wait.parity.shared::cta.b64 r, [%4], %5;\n\t"
      "selp.b32 x, 1, 0, p;\n\tselp.b32 y, 2, 0, q;\n\tselp.b32 z, 4, 0, r;\n\t"
      "or.b32 x, x, y;\n\tor.b32 %0, x, z;\n\t}"
      : "=r"(r)
      : "r"(smem_u32(b0)), "r"(p0), "r"(smem_u32(b1)), "r"(smem_u32(b2)), "r"(p12)
      : "memory");
  return r;
}
// A box into this CTA's shared memory, its bytes counted on the leader's barrier.
__device__ __forceinline__ void copy(uint32_t dst, const CUtensorMap* map, uint32_t bar, int32_t x, int32_t y) {
  asm volatile(
      "cp.async.bulk.tensor.2d.cta_group::2.shared::cluster.global.tile.mbarrier::complete_tx::bytes"
      " [%0], [%1, {%2, %3}], [%4];" ::"r"(dst),
      "l"(reinterpret_cast<uint64_t>(map)), "r"(x), "r"(y), "r"(bar)
      : "memory");
}
// Operands by the low words of their descriptors, which alone differ between MMAs
// (in 16-byte units): an add for each, nothing else.
__device__ __forceinline__ void mma(uint32_t d, uint32_t a, uint32_t b, uint32_t acc) {
  asm volatile(
      "{\n\t.reg .pred p;\n\t.reg .b64 a, b;\n\t"
      "setp.ne.b32 p, %3, 0;\n\t"
      "mov.b64 a, {%1, %4};\n\tmov.b64 b, {%2, %4};\n\t"
      "tcgen05.mma.cta_group::2.kind::f8f6f4 [%0], a, b, %5, p;\n\t}" ::"r"(d),
      "r"(a), "r"(b), "r"(acc), "n"(fp8::kDescHigh), "n"(fp8::idesc_e4m3(256, kTile / 2))
      : "memory");
}
// Arrives on `bar` of both CTAs once every MMA issued so far is complete.
__device__ __forceinline__ void commit(uint64_t* bar) {
  asm volatile(
      "tcgen05.commit.cta_group::2.mbarrier::arrive::one.shared::cluster.multicast::cluster.b64 [%0], %1;" ::"r"(
          smem_u32(bar)),
      "h"(static_cast<uint16_t>(3))
      : "memory");
}
// Tile `t`'s first row and column: groups of kGroupTiles row tiles sweep the
// weight together, so that both stay in L2 however many rows there are.
struct Place {
  int m, n;
};
__device__ __forceinline__ Place place(const Fp8MmParams& p, int t) {
  const int mt = (p.m + kTile - 1) / kTile, nt = (p.n + kTile - 1) / kTile;
  const int group = t / (kGroupTiles * nt), first = group * kGroupTiles;
  const int wide = min(kGroupTiles, mt - first), at = t - group * kGroupTiles * nt;
  return {(first + at % wide) * kTile, at / wide * kTile};
}

__global__ void __launch_bounds__(kThreads, 1) __cluster_dims__(2, 1, 1)
    fp8_mm_pair_kernel(const __grid_constant__ CUtensorMap wmap, const __grid_constant__ CUtensorMap amap,
                       const __grid_constant__ CUtensorMap cmap, const Fp8MmParams p) {
  extern __shared__ uint8_t smem_raw[];
  // (Both CTAs' shared memory starts at the same address, so that the leader's
  // descriptors are right in the other CTA too.)
  uint8_t* smem = smem_raw + ((1024u - (smem_u32(smem_raw) & 1023u)) & 1023u);
  Ctl* ctl = reinterpret_cast<Ctl*>(smem + kCtlOff);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const uint32_t rank = fp8::cluster_rank();
  const int tiles = ((p.m + kTile - 1) / kTile) * ((p.n + kTile - 1) / kTile);
  const int first = blockIdx.x >> 1, step = gridDim.x >> 1;
  const PairWaits waits{{&ctl->abort_flag, p.err, p.wait_ns}};

  if (threadIdx.x == 0) {
    for (int s = 0; s < kStages; ++s) {
      mbar_init(&ctl->full[s], 1);
      mbar_init(&ctl->empty[s], 1);
    }
    for (int s = 0; s < 4; ++s) {
      mbar_init(&ctl->tfull[s], 1);
      mbar_init(&ctl->tempty[s], kEpiWarps);  // half of the warps of both CTAs
    }
    for (int s = 0; s < 2; ++s) {
      mbar_init(&ctl->sfull[s], 2);
      mbar_init(&ctl->sempty[s], kEpiWarps);
    }
    mbar_init(&ctl->drain, 1);
    mbar_init(&ctl->never, 1);
    ctl->abort_flag = 0;
    fence_mbar_init();
    tma_prefetch_map(&wmap);
    tma_prefetch_map(&amap);
    tma_prefetch_map(&cmap);
  }
  if (warp == 1) tmem_alloc_pair_then_launch(&ctl->tmem_base, kTmemCols);
  tc_fence_before();
  fp8::cluster_sync();
  tc_fence_after();
  const uint32_t tmem = ctl->tmem_base;
  grid_dep_wait();

  if (warp < kFirstEpiWarp) {
    asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(kFewRegs));
    if (warp == 0) {
      // ------------------------------------------------------------ copies
      if (fp8::elect_one()) {
        uint32_t i = 0;
        bool ok = true;
        for (int t = first; t < tiles && ok; t += step) {
          const Place at = place(p, t);
          for (int kb = 0; kb < p.kblocks; ++kb, ++i) {
            const uint32_t s = i % kStages;
            if (i >= kStages && !(ok = waits.one(&ctl->empty[s], (i / kStages - 1) & 1))) break;
            const uint32_t dst = smem_u32(smem) + s * kStageBytes, bar = fp8::map_to(&ctl->full[s], 0);
            // (The phase ends with this arrival at the earliest, so the other CTA's
            // bytes may come before they are expected.)
            if (rank == 0) mbar_arrive_expect_tx(&ctl->full[s], 2 * kStageBytes);
            copy(dst, &amap, bar, kb * kBlock, at.m + static_cast<int>(rank) * 128);
            copy(dst + kOperandBytes, &wmap, bar, kb * kBlock, at.n + static_cast<int>(rank) * 64);
            copy(dst + kOperandBytes + kOperandBytes / 2, &wmap, bar, kb * kBlock,
                 at.n + 128 + static_cast<int>(rank) * 64);
          }
        }
      }
    } else if (warp == 1) {
      // ------------------------------------------------------------ MMAs
      if (rank == 0 && fp8::elect_one()) {
        const uint32_t desc0 = static_cast<uint32_t>(umma_desc_sw128_kmajor(smem_u32(smem)));
        uint32_t i = 0;
        bool ok = true;
        for (int t = first; t < tiles && ok; t += step) {
          for (int kb = 0; kb < p.kblocks; ++kb, ++i) {
            const uint32_t s = i % kStages;
            const uint32_t full_at = (i / kStages) & 1, empty_at = ((i >> 1) - 1) & 1;  // (i < 2: the phase before the first)
            const uint32_t there =
                look3(&ctl->full[s], full_at, &ctl->tempty[(i & 1) * 2], &ctl->tempty[(i & 1) * 2 + 1], empty_at);
            ok = (there & 1) != 0 || waits.one(&ctl->full[s], full_at);
            const uint32_t a = desc0 + s * (kStageBytes >> 4);
#pragma unroll
            for (uint32_t h = 0; h < 2; ++h) {
              const uint32_t d = (i & 1) * 2 + h;
              ok = ok && ((there >> (1 + h) & 1) != 0 || waits.one(&ctl->tempty[d], empty_at));
              if (!ok) break;
              tc_fence_after();
#pragma unroll
              for (int kk = 0; kk < kBlock / 32; ++kk)
                mma(tmem + d * 128, a + kk * 2, a + ((kOperandBytes + h * (kOperandBytes / 2)) >> 4) + kk * 2, kk != 0);
              if (h == 1) commit(&ctl->empty[s]);
              commit(&ctl->tfull[d]);
            }
            if (!ok) break;
          }
        }
        // Every MMA is complete before tensor memory is released.
        asm volatile(
            "tcgen05.commit.cta_group::2.mbarrier::arrive::one.shared::cluster.b64 [%0];" ::"r"(smem_u32(&ctl->drain))
            : "memory");
        mbar_wait(&ctl->drain, 0, kDrainWaitNs);
      }
    } else {
      // ------------------------------------------------------------ scales
      // 64 of the CTA's rows each, and the weight scales of half of the columns.
      const int half = warp - 2;
      uint32_t g = 0;
      bool ok = true;
      for (int t = first; t < tiles && ok; t += step) {
        const Place at = place(p, t);
        const float* sb = p.b_scale + static_cast<int64_t>(min(at.n / 128 + half, (p.n - 1) / 128)) * p.kblocks;
        for (int kb0 = 0; kb0 < p.kblocks; kb0 += kScaleBlocks, ++g) {
          if (g >= 2 && !(ok = waits.warp(&ctl->sempty[g & 1], (g / 2 - 1) & 1, lane))) break;
          fetch_scales<16>(p, ctl->sa[g & 1], at.m + static_cast<int>(rank) * 128, half, lane, kb0);
          if (lane < kScaleBlocks) ctl->sb[g & 1][half][lane] = sb[min(kb0 + lane, p.kblocks - 1)];
          __syncwarp();
          if (lane == 0) mbar_arrive(&ctl->sfull[g & 1]);
        }
      }
    }
  } else {
    // -------------------------------------------------------------- epilogue
    asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(kManyRegs));
    const int quarter = warp & 3, half = (warp - kFirstEpiWarp) >> 2;
    const uint32_t src0 = tmem + (static_cast<uint32_t>(quarter * 32) << 16) + half * kCols;
    uint8_t* outs = smem + kStages * kStageBytes + (warp - kFirstEpiWarp) * 2 * kOutBytes;
    const uint32_t tempty = fp8::map_to(&ctl->tempty[half], 0);  // and 16 bytes on
    uint32_t i = 0, g = 0;
    // (After a wait that gave up the warps go on, with waits that no longer wait, and
    // store nothing.)
    for (int t = first; t < tiles; t += step) {
      float acc[kCols];
#pragma unroll
      for (int c = 0; c < kCols; ++c) acc[c] = 0.0f;
      for (int kb0 = 0; kb0 < p.kblocks; kb0 += kScaleBlocks, ++g) {
        waits.warp(&ctl->sfull[g & 1], (g / 2) & 1, lane);
        const float* sa = ctl->sa[g & 1] + quarter * 32 + lane;
        const float* sb = ctl->sb[g & 1][half];
        const int n = min(kScaleBlocks, p.kblocks - kb0);
#pragma unroll 1
        for (int j = 0; j < n; ++j, ++i) {
          const uint32_t d = i & 1;
          const float f = sa[j * kScalePitch] * sb[j];
          waits.warp(&ctl->tfull[2 * d + half], (i >> 1) & 1, lane);
          tc_fence_after();
          const uint32_t src = src0 + d * kTile;
          uint32_t v[2][32];
          fp8::tmem_issue32(src, v[0]);
#pragma unroll
          for (int c = 0; c < 4; ++c) {
            fp8::tmem_wait32(v[c & 1]);
            if (c < 3) {
              fp8::tmem_issue32(src + (c + 1) * 32, v[(c + 1) & 1]);
            } else {  // read: the accumulator is free
              tc_fence_before();
              __syncwarp();
              if (lane == 0)
                asm volatile("mbarrier.arrive.shared::cluster.b64 _, [%0];" ::"r"(tempty + d * 16) : "memory");
            }
#pragma unroll
            for (int e = 0; e < 32; ++e) acc[c * 32 + e] = fmaf(__uint_as_float(v[c & 1][e]), f, acc[c * 32 + e]);
          }
        }
        __syncwarp();
        if (lane == 0) mbar_arrive(&ctl->sempty[g & 1]);
      }
      if (__any_sync(0xFFFFFFFFu, waits.aborted())) break;
      const Place at = place(p, t);
      const int row0 = at.m + static_cast<int>(rank) * 128 + quarter * 32, col0 = at.n + half * kCols;
      if (row0 < p.m && col0 < p.n) store_tile<kCols, 2>(p, cmap, acc, outs, row0, col0, lane);
    }
    if (lane == 0) asm volatile("cp.async.bulk.wait_group 0;" ::: "memory");  // the stores are complete
  }

  tc_fence_before();
  __syncthreads();
  // After a wait that gave up, copies of this CTA may be in flight that no barrier
  // accounts for: half a second is far more than they take.
  if (threadIdx.x == 0 && waits.aborted()) mbar_wait(&ctl->never, 0, kDrainWaitNs);
  fp8::cluster_sync();
  if (warp == 1) {
    tc_fence_after();
    asm volatile("tcgen05.dealloc.cta_group::2.sync.aligned.b32 %0, %1;" ::"r"(tmem), "r"(kTmemCols) : "memory");
  }
}

}  // namespace pair

cudaLaunchAttribute cluster_attr(int ctas) {
  cudaLaunchAttribute a{};
  a.id = cudaLaunchAttributeClusterDimension;
  a.val.clusterDim.x = static_cast<unsigned>(ctas);
  a.val.clusterDim.y = 1;
  a.val.clusterDim.z = 1;
  return a;
}

// How many clusters of 1 .. 4 CTAs that fill an SM each the current device holds at
// once: fewer than its SMs would, as the SMs of a cluster lie together (152, 76, 46, 36).
struct ClustersAtOnce {
  int of[block::kMaxSplits + 1];
};
const ClustersAtOnce& clusters_at_once(int num_sms) {
  constexpr int kDevices = 64;          // (device_info refuses more)
  static ClustersAtOnce counts[kDevices];
  static std::once_flag counted[kDevices];
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= kDevices) dev = 0;
  std::call_once(counted[dev], [&] {
    (void)cudaFuncSetAttribute(block::fp8_mm_block_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize,
                               static_cast<int>(block::kSmemBytes));
    for (int s = 1; s <= block::kMaxSplits; ++s) {
      cudaLaunchConfig_t cfg = {};
      cfg.gridDim = dim3(static_cast<unsigned>(s), 1, 1);
      cfg.blockDim = dim3(block::kThreads, 1, 1);
      cfg.dynamicSmemBytes = block::kSmemBytes;
      cudaLaunchAttribute attr[1] = {cluster_attr(s)};
      cfg.attrs = attr;
      cfg.numAttrs = 1;
      int& n = counts[dev].of[s];
      if (cudaOccupancyMaxActiveClusters(&n, block::fp8_mm_block_kernel, &cfg) != cudaSuccess) {
        (void)cudaGetLastError();
        n = num_sms / s;
      }
    }
  });
  return counts[dev];
}

cudaError_t launch_blocks(const Fp8MmParams& p, const CUtensorMap& wmap, const CUtensorMap& amap,
                          const CUtensorMap& cmap, cudaStream_t stream) {
  static std::atomic<uint64_t> allowed{0};
  cudaError_t e = allow_smem(reinterpret_cast<const void*>(block::fp8_mm_block_kernel),
                             static_cast<int>(block::kSmemBytes), allowed);
  if (e != cudaSuccess) return e;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(static_cast<unsigned>(p.splits), static_cast<unsigned>((p.m + block::kTile - 1) / block::kTile),
                     static_cast<unsigned>((p.n + block::kTile - 1) / block::kTile));
  cfg.blockDim = dim3(block::kThreads, 1, 1);
  cfg.dynamicSmemBytes = block::kSmemBytes;
  cfg.stream = stream;
  cudaLaunchAttribute attr[2] = {dependent_launch_attr(), cluster_attr(p.splits)};
  cfg.attrs = attr;
  cfg.numAttrs = 2;
  return cudaLaunchKernelEx(&cfg, block::fp8_mm_block_kernel, wmap, amap, cmap, p);
}

cudaError_t launch_pairs(const Fp8MmParams& p, const CUtensorMap& wmap, const CUtensorMap& amap,
                         const CUtensorMap& cmap, cudaStream_t stream) {
  static std::atomic<uint64_t> allowed{0};
  cudaError_t e = allow_smem(reinterpret_cast<const void*>(pair::fp8_mm_pair_kernel),
                             static_cast<int>(pair::kSmemBytes), allowed);
  if (e != cudaSuccess) return e;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(static_cast<unsigned>(2 * p.pairs), 1, 1);
  cfg.blockDim = dim3(pair::kThreads, 1, 1);
  cfg.dynamicSmemBytes = pair::kSmemBytes;
  cfg.stream = stream;
  cudaLaunchAttribute attr[1] = {dependent_launch_attr()};
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, pair::fp8_mm_pair_kernel, wmap, amap, cmap, p);
}

template <int kRows>
cudaError_t launch_rows(const Fp8MmParams& p, const CUtensorMap& wmap, const CUtensorMap& amap,
                        cudaStream_t stream) {
  const auto kernel = fp8_mm_rows_kernel<kRows>;
  constexpr uint32_t bytes = smem_bytes<kRows>();
  static_assert(bytes <= 227 * 1024 && kRows * kTileN * 4 <= Shape<kRows>::kStages * Shape<kRows>::kStageBytes, "");
  static std::atomic<uint64_t> allowed{0};
  cudaError_t e = allow_smem(reinterpret_cast<const void*>(kernel), static_cast<int>(bytes), allowed);
  if (e != cudaSuccess) return e;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(static_cast<unsigned>(p.splits), static_cast<unsigned>((p.m + kRows - 1) / kRows),
                     static_cast<unsigned>((p.n + kTileN - 1) / kTileN));
  cfg.blockDim = dim3(kThreads, 1, 1);
  cfg.dynamicSmemBytes = bytes;
  cfg.stream = stream;
  cudaLaunchAttribute attr[2] = {dependent_launch_attr(), cluster_attr(p.splits)};
  cfg.attrs = attr;
  cfg.numAttrs = 2;
  return cudaLaunchKernelEx(&cfg, kernel, wmap, amap, p);
}

}  // namespace

void plan_fp8_mm(Fp8MmParams& p, int num_sms) {
  p.kblocks = ceil_div(p.k, kBlock);
  // Up to 64 rows: row tiles.  More: pairs from more than one tile of 128 x 128 an SM
  // on (1,024 x 4,096 x 4,096: 18.0 us, by CTAs 22.4; 129 x 16,384 x 4,096 20.4 and 24.4;
  // 512 x 4,096 x 4,096, 128 tiles, 17.5 and 11.9), below that a CTA or some for each of
  // those tiles (777 x 1,024 x 2,048: 7.2 us, by row tiles 8.9; 1,000 x 2,048 x 512 4.2
  // and 5.6), unless they are fewer than eight, where k can be split further for row
  // tiles (65 x 128 x 16,384: 9.4 us, by 128 x 128 11.0; 100 x 512 x 2,048 5.1 and 5.5).
  // Up to 128 rows the second CTA of each pair has none: pairs are ahead there only
  // where k is short and the outputs count (100 x 65,536 x 512: 15.7 us, by CTAs 18.3;
  // 128 x 32,768 x 1,536 17.6 and 16.5, x 4,096 35.9 and 30.3; 100 x 20,000 x 4,096 33.4
  // and 26.6), which this rule does not see.
  const int64_t mt = (p.m + block::kTile - 1) / block::kTile, nt = (p.n + block::kTile - 1) / block::kTile;
  p.pairs = 0;
  p.row_tile = p.m <= 16 ? 16 : p.m <= 32 ? 32 : 64;
  if (p.m > 64 && mt * nt > num_sms) {
    const int64_t pair_tiles = (mt + 1) / 2 * ((nt + 1) / 2);
    p.row_tile = 128;
    p.splits = 1;
    p.kb_per_split = p.kblocks;
    p.pairs = static_cast<int32_t>(pair_tiles < num_sms / 2 ? pair_tiles : num_sms / 2);
    return;
  }
  if (p.m > 64 && mt * nt >= 8) p.row_tile = 128;
  // k is split as far as the launch's clusters run at once, with two blocks of k in each
  // range at least (32 x 4,096 x 32,768 in eight, four and two ranges: 22.2, 27.0, 45.8 us;
  // 1 x 2,048 x 4,096 4.4, 5.1, 6.9; 20 x 5,120 x 4,096 in clusters of 7 row tiles, which
  // take two turns, 11.1 us, of 6 7.0; 300 x 2,048 x 4,096 in clusters of 3 tiles of 128 x
  // 128 15.4, of 2 9.3).  Two CTAs of row tiles fit an SM.  Up to 64 rows the split must
  // not depend on m.
  const int64_t tiles = static_cast<int64_t>((p.n + kTileN - 1) / kTileN) * ((p.m + p.row_tile - 1) / p.row_tile);
  const ClustersAtOnce& at_once = clusters_at_once(num_sms);
  const bool rows = p.row_tile <= 64;
  int splits = rows ? kMaxSplits : block::kMaxSplits;
  while (splits > 1 && tiles > at_once.of[rows ? (splits + 1) / 2 : splits]) --splits;
  const int most = p.kblocks / 2 > 1 ? p.kblocks / 2 : 1;
  splits = splits < most ? splits : most;
  p.kb_per_split = (p.kblocks + splits - 1) / splits;
  p.splits = (p.kblocks + p.kb_per_split - 1) / p.kb_per_split;  // no empty range
}

cudaError_t launch_fp8_mm(const Fp8MmParams& p, const CUtensorMap& wmap, const CUtensorMap& amap,
                          const CUtensorMap& cmap, cudaStream_t stream) {
  if (p.pairs > 0) return launch_pairs(p, wmap, amap, cmap, stream);
  switch (p.row_tile) {
    case 16: return launch_rows<16>(p, wmap, amap, stream);
    case 32: return launch_rows<32>(p, wmap, amap, stream);
    case 64: return launch_rows<64>(p, wmap, amap, stream);
    default: return launch_blocks(p, wmap, amap, cmap, stream);
  }
}

}  // namespace dsa
