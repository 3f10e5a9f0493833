// indexer_write_fp8.cu -- the indexer's write side into an FP8 key cache: the
// k_norm LayerNorm (with a bias) of each row's wk projection, quantised to E4M3
// with one power-of-two scale a key as it is stored.
//
// "glm5next_dsa/layer.rs", module header trap 2 and indexer_forward, and
// decode_k for the lockstep with the KV cache, as in indexer_write.cu.  With
// mu and var the row's mean and (biased) variance,
//   y = (x - mu) / sqrt(var + eps) * w + b
//   2^e = smallest power of two, 2^-126 at least, with max |y| <= 448 * 2^e
//   idx_k[t] = E4M3_RNE(y / 2^e),   idx_scale[t] = 2^e,   t = idx_base + position
// y is taken in double and y / 2^e is exact, so the codes are its one rounding.
//
// One warp a row.  A row is written only if its whole sequence is in order, which
// every warp of the sequence finds for itself (a lane looks at each of its rows,
// 32 at most), so the warps need not wait for one another; a count that another
// warp has already raised leads to the same decision.
#include "dsa_internal.h"
#include "fp8_device.cuh"

namespace dsa {
namespace {

constexpr int kWarps = 4;

// v rounded to float with the last bit odd where it is not exact: rounding that
// to at most 22 bits of mantissa is rounding v (Boldo and Melquiond, IEEE Trans.
// Computers 57(4), 2008).
__device__ __forceinline__ float round_to_odd(double v) {
  float f = __double2float_rz(v);
  if (static_cast<double>(f) != v && !isnan(v) && !isinf(f)) f = __uint_as_float(__float_as_uint(f) | 1u);
  return f;
}

// Exponent of the scale of a row whose largest finite |y| is `top`, as
// fp8::scale_bits on a double (a mantissa above 1.75 carries).
__device__ __forceinline__ int scale_exponent(double top) {
  const int e = static_cast<int>((__double_as_longlong(top) + 0x3FFFFFFFFFFFFll) >> 52) - 1023 - 8;
  return max(-126, min(127, e));
}
__device__ __forceinline__ double power_of_two(int e) {
  return __longlong_as_double(static_cast<long long>(e + 1023) << 52);
}

template <int D>
__global__ void __launch_bounds__(kWarps * 32) indexer_write_fp8_kernel(const IndexerWriteFp8Params p) {
  constexpr int kPer = D / 32;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int r = blockIdx.x * kWarps + warp;
  grid_dep_launch();
  if (r >= p.rows) return;  // whole warps only
  // The norm's weight and bias are weights (no kernel of a chain writes them).
  double w[kPer], b[kPer];
#pragma unroll
  for (int i = 0; i < kPer; ++i) {
    w[i] = static_cast<double>(__uint_as_float(static_cast<uint32_t>(p.ln_w[lane * kPer + i]) << 16));
    b[i] = static_cast<double>(__uint_as_float(static_cast<uint32_t>(p.ln_b[lane * kPer + i]) << 16));
  }
  grid_dep_wait();
  double x[kPer];
#pragma unroll
  for (int i = 0; i < kPer; ++i)
    x[i] = static_cast<double>(
        __uint_as_float(static_cast<uint32_t>(p.k_raw[static_cast<int64_t>(r) * D + lane * kPer + i]) << 16));

  // ---- the sequence's rows, one a lane
  const int per = p.rows_per_seq, seq = r / per, r0 = seq * per, mine = r - r0;
  int64_t pos = 0, len = 0, at = 0;
  if (lane < per) {
    pos = p.positions[r0 + lane];
    len = p.seq_lens[r0 + lane];
    const int64_t base = p.idx_base[r0 + lane];
    at = base < 0 ? -1 : base + pos;
  }
  const int64_t written = p.idx_written != nullptr ? p.idx_written[seq] : -1;
  const int64_t p0 = __shfl_sync(0xFFFFFFFFu, pos, 0);
  const bool empty = lane < per && pos == 0 && len == 0;  // a row without a token
  const bool in_place = lane >= per || empty || (pos + 1 == len && pos == p0 + lane);
  const bool in_arena = lane >= per || empty || (at >= 0 && at < p.idx_tokens);
  const bool any_empty = __any_sync(0xFFFFFFFFu, empty);
  const bool all_empty = __all_sync(0xFFFFFFFFu, lane >= per || empty);
  if (all_empty) return;
  bool ok = __all_sync(0xFFFFFFFFu, in_place && in_arena) && !any_empty;
  if (!ok && lane == mine) {
    if (!in_place || empty) record_error(p.err, DSA_DEVERR_POSITION, r);
    else if (!in_arena) record_error(p.err, DSA_DEVERR_ARENA, r);
  }
  if (ok && p.idx_written != nullptr && written < p0) {  // rows [written, p0) were never written
    if (lane == 0 && mine == 0) record_error(p.err, DSA_DEVERR_BEHIND, r0);
    ok = false;
  }
  if (!ok) return;

  // ---- norm
  double s = 0.0;
#pragma unroll
  for (int i = 0; i < kPer; ++i) s += x[i];
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) s += __shfl_xor_sync(0xFFFFFFFFu, s, o);
  const double mu = s / D;
  double q = 0.0;
#pragma unroll
  for (int i = 0; i < kPer; ++i) q += (x[i] - mu) * (x[i] - mu);
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) q += __shfl_xor_sync(0xFFFFFFFFu, q, o);
  const double inv = 1.0 / sqrt(q / D + static_cast<double>(p.eps));
  double top = 0.0;
#pragma unroll
  for (int i = 0; i < kPer; ++i) {
    x[i] = (x[i] - mu) * inv * w[i] + b[i];
    if (isfinite(x[i])) top = fmax(top, fabs(x[i]));
  }
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) top = fmax(top, __shfl_xor_sync(0xFFFFFFFFu, top, o));

  // ---- codes
  const int e = scale_exponent(top);
  const double down = power_of_two(-e);
  float f[kPer];
#pragma unroll
  for (int i = 0; i < kPer; ++i) f[i] = round_to_odd(x[i] * down);
  const int64_t t = __shfl_sync(0xFFFFFFFFu, at, mine);
  uint8_t* dst = p.idx_k + t * D + lane * kPer;
  if constexpr (kPer == 4)
    *reinterpret_cast<uint32_t*>(dst) = fp8::e4m3x4(f[0], f[1], f[2], f[3]);
  else
    *reinterpret_cast<uint16_t*>(dst) = static_cast<uint16_t>(fp8::e4m3x2(f[0], f[1]));
  if (lane == 0) {
    p.idx_scale[t] = static_cast<float>(power_of_two(e));
    if (p.gate != nullptr) p.idx_gate[t] = p.gate[r];
    // the sequence now holds exactly the rows up to its last new one
    if (p.idx_written != nullptr && mine == 0) p.idx_written[seq] = static_cast<int32_t>(p0 + per);
  }
}

}  // namespace

cudaError_t launch_indexer_write_fp8(const IndexerWriteFp8Params& p, cudaStream_t stream) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(static_cast<unsigned>((p.rows + kWarps - 1) / kWarps), 1, 1);
  cfg.blockDim = dim3(kWarps * 32, 1, 1);
  cfg.stream = stream;
  cudaLaunchAttribute attr[1] = {dependent_launch_attr()};
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  if (p.dim == 64) return cudaLaunchKernelEx(&cfg, indexer_write_fp8_kernel<64>, p);
  return cudaLaunchKernelEx(&cfg, indexer_write_fp8_kernel<128>, p);
}

}  // namespace dsa
