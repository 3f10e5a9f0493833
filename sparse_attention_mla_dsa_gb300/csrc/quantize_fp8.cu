// quantize_fp8.cu -- bf16 or FP32 values to E4M3 codes with a power-of-two
// scale for each block of 128 along k, of one row (activations, queries) or of
// 128 rows (weights).
//
//   2^e = smallest power of two, 2^-126 at least, with max |x| <= 448 * 2^e
//   code = E4M3_RNE(x / 2^e)
// E4M3 keeps its three bits of mantissa whatever the scale, so a power of two
// costs no precision against max / 448, and x / 2^e is exact (where it falls
// below 2^-126 its code is 0 either way): the code is rounded once, and
// values that are quantised again stay what they are.
//
// Bound by memory: 3 bytes an element from bf16, 5 from FP32.  Rows of 1: a
// block is 16 bytes of each of 16 lanes (bf16) or of 32 (FP32), its largest
// element is found by shuffles and its values stay in registers in between (1,024 x
// 32,768 bf16: 15.1 us, 6.7 TB/s, with part of the codes still in L2; 17.8 where every
// byte comes from and goes to other buffers).  Maxima are of the bits without signs,
// two bf16 values at a time, and infinities and NaN are taken out only in a warp that
// has one: by a test of every value, 16.8 us.  Tiles of 128 rows: one CTA a tile, which
// it holds in registers (FP32: but for 8 bytes a thread), two an SM (5,003 x 4,112 FP32:
// 15.2 us, 6.8 TB/s, with part of the codes still in L2; 18.5 over other buffers).
#include "dsa_internal.h"
#include "fp8_device.cuh"

namespace dsa {
namespace {

using fp8::kBlock;

constexpr int kThreads = 128;
constexpr int kTileRows = 128;
constexpr int kTileThreads = 512;

// 16 bytes of x: 8 bf16 or 4 FP32 values.
template <bool kF32>
struct Vec {
  static constexpr int kElems = kF32 ? 4 : 8;
  static constexpr int kLanes = kBlock / kElems;  // lanes of one block of a row
  uint4 v;

  // The largest |x| so far as maxima() keeps it: bits without signs, of two bf16
  // values beside each other or of one float.
  __device__ __forceinline__ uint32_t maxima() const {
    constexpr uint32_t kMagnitude = kF32 ? 0x7FFFFFFFu : 0x7FFF7FFFu;
    return larger(larger(v.x & kMagnitude, v.y & kMagnitude), larger(v.z & kMagnitude, v.w & kMagnitude));
  }
  static __device__ __forceinline__ uint32_t larger(uint32_t a, uint32_t b) { return kF32 ? max(a, b) : __vmaxu2(a, b); }
  // The bits of that as a float; not below those of infinity if one of them is not finite.
  static __device__ __forceinline__ uint32_t as_float(uint32_t m) {
    return kF32 ? m : max(m & 0xFFFF0000u, m << 16);
  }
  // Without the infinities and NaN.
  __device__ __forceinline__ Vec finite() const {
    auto keep = [](uint32_t w) {
      if constexpr (kF32) return (w & 0x7FFFFFFFu) < 0x7F800000u ? w : 0u;
      return ((w & 0x7FFF0000u) < 0x7F800000u ? w & 0xFFFF0000u : 0u) | ((w & 0x7FFFu) < 0x7F80u ? w & 0xFFFFu : 0u);
    };
    return {make_uint4(keep(v.x), keep(v.y), keep(v.z), keep(v.w))};
  }

  __device__ __forceinline__ void store_codes(uint8_t* dst, float inv) const {
    const uint32_t w[4] = {v.x, v.y, v.z, v.w};
    if constexpr (kF32) {
      *reinterpret_cast<uint32_t*>(dst) =
          fp8::e4m3x4(__uint_as_float(w[0]) * inv, __uint_as_float(w[1]) * inv,
                      __uint_as_float(w[2]) * inv, __uint_as_float(w[3]) * inv);
    } else {
      uint32_t c[2];
#pragma unroll
      for (int i = 0; i < 2; ++i)
        c[i] = fp8::e4m3x4(__uint_as_float(w[2 * i] << 16) * inv, __uint_as_float(w[2 * i] & 0xFFFF0000u) * inv,
                           __uint_as_float(w[2 * i + 1] << 16) * inv,
                           __uint_as_float(w[2 * i + 1] & 0xFFFF0000u) * inv);
      *reinterpret_cast<uint2*>(dst) = make_uint2(c[0], c[1]);
    }
  }
};

__device__ __forceinline__ uint4 load16(const void* p) { return ld_dep_u4(static_cast<const uint4*>(p)); }

// kUnroll blocks a group of lanes, loaded together.
template <bool kF32, int kUnroll>
__global__ void __launch_bounds__(kThreads) quantize_rows_kernel(const QuantizeParams p) {
  using V = Vec<kF32>;
  constexpr int kGroups = kThreads / V::kLanes;  // blocks that a CTA works on at a time
  const int group = threadIdx.x / V::kLanes, lane = threadIdx.x % V::kLanes;
  const uint32_t kb = static_cast<uint32_t>(p.kblocks);
  const uint32_t total = static_cast<uint32_t>(p.rows) * kb;  // below 2^31
  const uint32_t b0 = blockIdx.x * (kGroups * kUnroll) + group;
  grid_dep_launch();
  grid_dep_wait();
  V v[kUnroll];
  int64_t at[kUnroll];  // -1: nothing of the tensor here
#pragma unroll
  for (int u = 0; u < kUnroll; ++u) {
    const uint32_t b = b0 + u * kGroups;
    const uint32_t row = b / kb;
    const int col = static_cast<int>(b - row * kb) * kBlock + lane * V::kElems;
    at[u] = b < total && col < p.k ? static_cast<int64_t>(row) * p.k + col : -1;
    v[u].v = make_uint4(0u, 0u, 0u, 0u);
    if (at[u] >= 0) v[u].v = load16(static_cast<const char*>(p.x) + at[u] * (kF32 ? 4 : 2));
  }
#pragma unroll
  for (int u = 0; u < kUnroll; ++u) {
    auto over_lanes = [](uint32_t m) {
#pragma unroll
      for (int o = V::kLanes / 2; o > 0; o >>= 1) m = V::larger(m, __shfl_xor_sync(0xFFFFFFFFu, m, o));
      return V::as_float(m);
    };
    uint32_t top = over_lanes(v[u].maxima());
    if (__any_sync(0xFFFFFFFFu, top >= 0x7F800000u)) top = over_lanes(v[u].finite().maxima());
    const uint32_t scale = fp8::scale_bits(top);
    if (at[u] >= 0) {
      v[u].store_codes(p.codes + at[u], fp8::inverse_scale(scale));
      if (lane == 0) p.scales[b0 + u * kGroups] = __uint_as_float(scale);
    }
  }
}

// One CTA a tile of 128 x 128.
template <bool kF32>
__global__ void __launch_bounds__(kTileThreads, 2) quantize_tiles_kernel(const QuantizeParams p) {
  using V = Vec<kF32>;
  constexpr int kRowsAtOnce = kTileThreads / V::kLanes;
  constexpr int kVecs = kTileRows / kRowsAtOnce;
  __shared__ uint32_t warp_top[kTileThreads / 32];
  const int64_t row0 = static_cast<int64_t>(blockIdx.y) * kTileRows + threadIdx.x / V::kLanes;
  const int col = static_cast<int>(blockIdx.x) * kBlock + (threadIdx.x % V::kLanes) * V::kElems;
  grid_dep_launch();
  grid_dep_wait();
  V v[kVecs];
#pragma unroll
  for (int i = 0; i < kVecs; ++i) {
    const int64_t row = row0 + i * kRowsAtOnce;
    v[i].v = make_uint4(0u, 0u, 0u, 0u);
    if (row < p.rows && col < p.k)
      v[i].v = load16(static_cast<const char*>(p.x) + (row * p.k + col) * (kF32 ? 4 : 2));
  }
  auto over_tile = [&](bool all) {
    uint32_t m = 0;
#pragma unroll
    for (int i = 0; i < kVecs; ++i) m = V::larger(m, all ? v[i].maxima() : v[i].finite().maxima());
    m = __reduce_max_sync(0xFFFFFFFFu, V::as_float(m));
    if ((threadIdx.x & 31) == 0) warp_top[threadIdx.x >> 5] = m;
    __syncthreads();
#pragma unroll
    for (int w = 0; w < kTileThreads / 32; ++w) m = max(m, warp_top[w]);
    return m;
  };
  uint32_t top = over_tile(true);
  if (top >= 0x7F800000u) {  // (of the whole CTA)
    __syncthreads();
    top = over_tile(false);
  }
  const uint32_t scale = fp8::scale_bits(top);
  const float inv = fp8::inverse_scale(scale);
#pragma unroll
  for (int i = 0; i < kVecs; ++i) {
    const int64_t row = row0 + i * kRowsAtOnce;
    if (row < p.rows && col < p.k) v[i].store_codes(p.codes + row * p.k + col, inv);
  }
  if (threadIdx.x == 0)
    p.scales[static_cast<int64_t>(blockIdx.y) * p.kblocks + blockIdx.x] = __uint_as_float(scale);
}

// Blocks that a group of lanes loads together: 1 while the CTAs then half fill
// the SMs (16 of 128 threads each), 2 while they fit them at once, else 4.
// Measured for k 4,096 of bf16, 1 / 2 / 4 blocks in us: 1 row 1.05 / 1.20 / 1.52,
// 256 rows 2.08 / 2.55 / 2.98, 512 rows 3.00 / 2.74 / 3.92, 1,024 rows
// 4.51 / 3.60 / 4.60, 4,096 rows 17.1 / 10.1 / 10.4; 1,024 rows of k 32,768
// 18.3 with 2 and 17.9 with 4; 5,003 x 4,112 FP32 21.4 and 19.0.
template <bool kF32>
cudaError_t launch_rows(const QuantizeParams& p, int num_sms, cudaLaunchConfig_t& cfg) {
  constexpr int64_t kGroups = kThreads / Vec<kF32>::kLanes;
  const int64_t total = static_cast<int64_t>(p.rows) * p.kblocks;
  const int64_t ctas = (total + kGroups - 1) / kGroups;
  const int unroll = ctas <= 8 * num_sms ? 1 : ctas <= 32 * num_sms ? 2 : 4;
  cfg.gridDim = dim3(static_cast<unsigned>((ctas + unroll - 1) / unroll), 1, 1);
  return cudaLaunchKernelEx(&cfg,
                            unroll == 1   ? quantize_rows_kernel<kF32, 1>
                            : unroll == 2 ? quantize_rows_kernel<kF32, 2>
                                          : quantize_rows_kernel<kF32, 4>,
                            p);
}

}  // namespace

cudaError_t launch_quantize_fp8(const QuantizeParams& p, int num_sms, cudaStream_t stream) {
  cudaLaunchConfig_t cfg = {};
  cfg.blockDim = dim3(kThreads, 1, 1);
  cfg.stream = stream;
  cudaLaunchAttribute attr[1] = {dependent_launch_attr()};
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  if (p.block_rows == kTileRows) {
    cfg.blockDim = dim3(kTileThreads, 1, 1);
    cfg.gridDim = dim3(static_cast<unsigned>(p.kblocks), static_cast<unsigned>((p.rows + kTileRows - 1) / kTileRows), 1);
    return p.x_fp32 ? cudaLaunchKernelEx(&cfg, quantize_tiles_kernel<true>, p)
                    : cudaLaunchKernelEx(&cfg, quantize_tiles_kernel<false>, p);
  }
  return p.x_fp32 ? launch_rows<true>(p, num_sms, cfg) : launch_rows<false>(p, num_sms, cfg);
}

}  // namespace dsa
