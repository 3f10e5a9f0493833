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
// CTA roles (192 threads): warp 0 issues TMA, warp 1 owns TMEM and issues the
// MMAs (one thread), warps 2-5 are the epilogue (one TMEM lane quarter each).
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
  static constexpr int kSlots = kRows <= 64 ? 4 : 2;  // accumulators in TMEM
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

template <int kRows>
__global__ void __launch_bounds__(kThreads, kRows <= 64 ? 2 : 1)
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
  grid_dep_launch();

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
  if (warp == 1) {
    tmem_alloc(&ctl->tmem_base, S::kTmemCols);
    tmem_relinquish();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = ctl->tmem_base;

  if (warp == 0) {
    if (lane == 0) {
      const uint64_t w_policy = l2_policy_evict_first();
      uint64_t a_policy;
      asm volatile("createpolicy.fractional.L2::evict_normal.b64 %0, 1.0;" : "=l"(a_policy));
      // The weight is an input that no kernel writes: its first tiles go out
      // before the dependency wait, the activations' after it.
      const int early = min(nkb, S::kStages);
      for (int i = 0; i < early; ++i) {
        mbar_arrive_expect_tx(&ctl->full[i], S::kStageBytes);
        tma_load_2d(smem + i * S::kStageBytes, &wmap, &ctl->full[i], (kb_begin + i) * kBlock, n0, w_policy);
      }
      grid_dep_wait();
      for (int i = 0; i < early; ++i)
        tma_load_2d(smem + i * S::kStageBytes + kWBytes, &amap, &ctl->full[i], (kb_begin + i) * kBlock, m0,
                    a_policy);
      int issued = early;
      for (; issued < nkb; ++issued) {
        if (aborted(&ctl->abort_flag)) break;
        const int s = issued % S::kStages;
        if (!mbar_wait(&ctl->empty[s], ((issued / S::kStages) - 1) & 1, p.wait_ns)) {
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
    if (lane == 0) {
      constexpr uint32_t idesc = fp8::idesc_e4m3(kTileN, kRows);
      const uint32_t base = smem_u32(smem);
      for (int i = 0; i < nkb; ++i) {
        const int s = i % S::kStages, t = i % S::kSlots;
        if (aborted(&ctl->abort_flag)) break;
        if (!mbar_wait(&ctl->full[s], (i / S::kStages) & 1, p.wait_ns) ||
            (i >= S::kSlots && !mbar_wait(&ctl->tempty[t], ((i / S::kSlots) - 1) & 1, p.wait_ns))) {
          set_abort(&ctl->abort_flag, p.err, tile);
          break;
        }
        tc_fence_after();
        const uint32_t w_addr = base + s * S::kStageBytes;
        const uint32_t a_addr = w_addr + kWBytes;
#pragma unroll
        for (int kk = 0; kk < kBlock / 32; ++kk)
          fp8::umma_e4m3(tmem + t * kRows, umma_desc_sw128_kmajor(w_addr + kk * 32),
                         umma_desc_sw128_kmajor(a_addr + kk * 32), idesc, kk != 0);
        umma_commit(&ctl->empty[s]);
        umma_commit(&ctl->tfull[t]);
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
    // Output (row, column) pairs shared out among the cluster's epilogue threads.
    const int rows_here = min(kRows, p.m - m0);
    if (warp >= 2 && n0 + et < p.n) {
      for (int c = split; c < rows_here; c += p.splits) {
        const uint32_t at = smem_u32(part + c * kTileN + et);
        float v[kMaxSplits];
#pragma unroll
        for (int r = 0; r < kMaxSplits; ++r) v[r] = r < p.splits ? fp8::ld_cluster_f32(at, r) : 0.0f;
        float sum = v[0];
#pragma unroll
        for (int r = 1; r < kMaxSplits; ++r)
          if (r < p.splits) sum += v[r];
        store_c(p, m0 + c, n0 + et, sum);
      }
    }
    fp8::cluster_sync();  // nobody reads this CTA's shared memory any more
  }
  if (warp == 1) {
    tc_fence_after();
    tmem_dealloc(tmem, S::kTmemCols);
  }
}

template <int kRows>
cudaError_t launch_rows(const Fp8MmParams& p, const CUtensorMap& wmap, const CUtensorMap& amap,
                        cudaStream_t stream) {
  const auto kernel = fp8_mm_rows_kernel<kRows>;
  constexpr uint32_t bytes = smem_bytes<kRows>();
  static_assert(bytes <= 227 * 1024 && kRows * kTileN * 4 <= Shape<kRows>::kStages * Shape<kRows>::kStageBytes, "");
  cudaError_t e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, bytes);
  if (e != cudaSuccess) return e;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(static_cast<unsigned>(p.splits), static_cast<unsigned>((p.m + kRows - 1) / kRows),
                     static_cast<unsigned>((p.n + kTileN - 1) / kTileN));
  cfg.blockDim = dim3(kThreads, 1, 1);
  cfg.dynamicSmemBytes = bytes;
  cfg.stream = stream;
  cudaLaunchAttribute attr[2] = {dependent_launch_attr(), {}};
  attr[1].id = cudaLaunchAttributeClusterDimension;
  attr[1].val.clusterDim.x = static_cast<unsigned>(p.splits);
  attr[1].val.clusterDim.y = 1;
  attr[1].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 2;
  return cudaLaunchKernelEx(&cfg, kernel, wmap, amap, p);
}

}  // namespace

void plan_fp8_mm(Fp8MmParams& p, int num_sms) {
  p.kblocks = (p.k + kBlock - 1) / kBlock;
  p.row_tile = p.m <= 16 ? 16 : p.m <= 32 ? 32 : p.m <= 64 ? 64 : 128;
  // k is split only where the tiles alone leave SMs idle, with two blocks of it
  // a CTA at least.  Up to 64 rows the split must not depend on m.
  const int64_t tiles = static_cast<int64_t>((p.n + kTileN - 1) / kTileN) * ((p.m + p.row_tile - 1) / p.row_tile);
  int splits = tiles < num_sms ? static_cast<int>((num_sms + tiles - 1) / tiles) : 1;
  splits = splits < kMaxSplits ? splits : kMaxSplits;
  const int most = p.kblocks / 2 > 1 ? p.kblocks / 2 : 1;
  splits = splits < most ? splits : most;
  p.kb_per_split = (p.kblocks + splits - 1) / splits;
  p.splits = (p.kblocks + p.kb_per_split - 1) / p.kb_per_split;  // no empty range
}

cudaError_t launch_fp8_mm(const Fp8MmParams& p, const CUtensorMap& wmap, const CUtensorMap& amap,
                          cudaStream_t stream) {
  switch (p.row_tile) {
    case 16: return launch_rows<16>(p, wmap, amap, stream);
    case 32: return launch_rows<32>(p, wmap, amap, stream);
    case 64: return launch_rows<64>(p, wmap, amap, stream);
    default: return launch_rows<128>(p, wmap, amap, stream);
  }
}

}  // namespace dsa
