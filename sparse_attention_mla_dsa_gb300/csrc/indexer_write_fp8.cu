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
// y / 2^e is exact, so the codes are y's one rounding.
//
// y has to be known only as far as the code goes (4 bits) and on which side of a
// border it lies.  It is taken in FP32 with a bound on its error; a row where that
// leaves a code or the scale open (0.6 % of rows of normal inputs), or that FP32
// does not hold, is taken again in double.  In double throughout, 4,001 rows took
// 34 us (7.4 now) and four rows 4.9 (1.7): the FP64 rate is a small part of the FP32 one.
//   mean      two FP32 words (sums that keep their rounding errors), so x - mean
//             is good to 2^-23 of itself however far the mean is from 0
//   variance  d^2 2^-22, nine additions of positive terms 9 * 2^-24: 2^-20.2
//   1/sqrt    half of that and 2^-22 of rsqrtf: 2^-20.5;  t = d / sqrt * w: 2^-20
//   y = t + b one rounding more: |error| < 2^-19 (|t| + |b|), taken as the bound
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

constexpr float kBound = 1.0f / (1 << 19);

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

// (s, e) = a + b as a float and its rounding error (Knuth's two-sum).
__device__ __forceinline__ void two_sum(float a, float b, float& s, float& e) {
  s = __fadd_rn(a, b);
  const float t = __fadd_rn(s, -a);
  e = __fadd_rn(__fadd_rn(a, -__fadd_rn(s, -t)), __fadd_rn(b, -t));
}
__device__ __forceinline__ float warp_max(float v) {  // v >= 0
  return __uint_as_float(__reduce_max_sync(0xFFFFFFFFu, __float_as_uint(v)));
}
// kPer consecutive bf16 values, in one load.
template <int kPer>
__device__ __forceinline__ void load_bf16(const uint16_t* src, float (&v)[kPer]) {
  uint32_t u[kPer / 2];
  if constexpr (kPer == 4)
    *reinterpret_cast<uint2*>(u) = *reinterpret_cast<const uint2*>(src);
  else
    u[0] = *reinterpret_cast<const uint32_t*>(src);
#pragma unroll
  for (int i = 0; i < kPer; ++i) v[i] = __uint_as_float(i & 1 ? u[i / 2] & 0xFFFF0000u : u[i / 2] << 16);
}

// This lane's codes and the row's scale, by FP32; false: not certain of them all.
template <int kPer>
__device__ __forceinline__ bool codes_fp32(const float (&x)[kPer], const float (&w)[kPer], const float (&b)[kPer],
                                           float eps, uint32_t& codes, float& scale) {
  constexpr float kInvD = 1.0f / (32 * kPer);
  float hi = x[0], lo = 0.0f;
#pragma unroll
  for (int i = 1; i < kPer; ++i) {
    float e;
    two_sum(hi, x[i], hi, e);
    lo += e;
  }
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) {
    const float h2 = __shfl_xor_sync(0xFFFFFFFFu, hi, o), l2 = __shfl_xor_sync(0xFFFFFFFFu, lo, o);
    float e;
    two_sum(hi, h2, hi, e);
    lo += l2 + e;
  }
  float mu, mu_lo;
  two_sum(hi * kInvD, lo * kInvD, mu, mu_lo);
  float d[kPer], q = 0.0f;
#pragma unroll
  for (int i = 0; i < kPer; ++i) {
    d[i] = __fadd_rn(__fadd_rn(x[i], -mu), -mu_lo);
    q = fmaf(d[i], d[i], q);
  }
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) q += __shfl_xor_sync(0xFFFFFFFFu, q, o);
  const float v = fmaf(q, kInvD, eps);
  const float inv = rsqrtf(v);
  float y[kPer], size = 0.0f, top = 0.0f;
#pragma unroll
  for (int i = 0; i < kPer; ++i) {
    const float t = d[i] * inv;
    y[i] = fmaf(t, w[i], b[i]);
    d[i] = fmaf(fabsf(t), fabsf(w[i]), fabsf(b[i]));
    size = fmaxf(size, d[i]);
    top = fmaxf(top, fabsf(y[i]));
  }
  size = warp_max(size);
  top = warp_max(top);
  const float most = kBound * size;  // error of any y
  const uint32_t bits = fp8::scale_bits(__float_as_uint(top + most));
  const float down = fp8::inverse_scale(bits);
  scale = __uint_as_float(bits);
  bool sure = v > 1e-25f && v < 1e30f && size < 1e30f && bits == fp8::scale_bits(__float_as_uint(fmaxf(top - most, 0.0f)));
  uint32_t c[kPer / 2];
#pragma unroll
  for (int i = 0; i < kPer; i += 2) {
    const float a0 = fabsf(y[i] * down), a1 = fabsf(y[i + 1] * down);
    const float e0 = fmaf(d[i] * down, kBound, 1e-6f), e1 = fmaf(d[i + 1] * down, kBound, 1e-6f);
    c[i / 2] = fp8::e4m3x2(y[i] * down, y[i + 1] * down);
    sure = sure && fp8::e4m3x2(fmaxf(a0 - e0, 0.0f), fmaxf(a1 - e1, 0.0f)) == fp8::e4m3x2(a0 + e0, a1 + e1);
  }
  codes = c[0];
  if constexpr (kPer == 4) codes |= c[1] << 16;
  return __all_sync(0xFFFFFFFFu, sure);  // (false too where something is NaN)
}

// The same in double.
template <int kPer>
__device__ __noinline__ void codes_double(const float (&xf)[kPer], const float (&w)[kPer], const float (&b)[kPer],
                                          float eps, uint32_t& codes, float& scale) {
  double x[kPer], s = 0.0;
#pragma unroll
  for (int i = 0; i < kPer; ++i) {
    x[i] = xf[i];
    s += x[i];
  }
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) s += __shfl_xor_sync(0xFFFFFFFFu, s, o);
  const double mu = s / (32 * kPer);
  double q = 0.0;
#pragma unroll
  for (int i = 0; i < kPer; ++i) q += (x[i] - mu) * (x[i] - mu);
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) q += __shfl_xor_sync(0xFFFFFFFFu, q, o);
  const double inv = 1.0 / sqrt(q / (32 * kPer) + static_cast<double>(eps));
  double top = 0.0;
#pragma unroll
  for (int i = 0; i < kPer; ++i) {
    x[i] = (x[i] - mu) * inv * w[i] + b[i];
    if (isfinite(x[i])) top = fmax(top, fabs(x[i]));
  }
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) top = fmax(top, __shfl_xor_sync(0xFFFFFFFFu, top, o));
  const int e = scale_exponent(top);
  const double down = power_of_two(-e);
  float f[kPer];
#pragma unroll
  for (int i = 0; i < kPer; ++i) f[i] = round_to_odd(x[i] * down);
  if constexpr (kPer == 4) codes = fp8::e4m3x4(f[0], f[1], f[2], f[3]);
  else codes = fp8::e4m3x2(f[0], f[1]);
  scale = static_cast<float>(power_of_two(e));
}

template <int D>
__global__ void __launch_bounds__(kWarps * 32) indexer_write_fp8_kernel(const IndexerWriteFp8Params p) {
  constexpr int kPer = D / 32;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int r = blockIdx.x * kWarps + warp;
  grid_dep_launch();
  if (r >= p.rows) return;  // whole warps only
  // Any input may come from the kernel before: only their lines are fetched before the
  // wait (the norm's by one warp: by each, 20,000 rows take 35 us for 13).
  if (lane < 2)
    prefetch_l2(p.k_raw + static_cast<int64_t>(r) * D + lane * (D / 2));
  else if (r == 0 && lane < 6)
    prefetch_l2((lane < 4 ? p.ln_w : p.ln_b) + (lane & 1) * (D / 2));
  grid_dep_wait();
  float w[kPer], b[kPer], x[kPer];
  load_bf16<kPer>(p.ln_w + lane * kPer, w);
  load_bf16<kPer>(p.ln_b + lane * kPer, b);
  load_bf16<kPer>(p.k_raw + static_cast<int64_t>(r) * D + lane * kPer, x);

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

  uint32_t codes;
  float scale;
  if (!codes_fp32<kPer>(x, w, b, p.eps, codes, scale)) codes_double<kPer>(x, w, b, p.eps, codes, scale);
  const int64_t t = __shfl_sync(0xFFFFFFFFu, at, mine);
  uint8_t* dst = p.idx_k + t * D + lane * kPer;
  if constexpr (kPer == 4)
    *reinterpret_cast<uint32_t*>(dst) = codes;
  else
    *reinterpret_cast<uint16_t*>(dst) = static_cast<uint16_t>(codes);
  if (lane == 0) {
    p.idx_scale[t] = scale;
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
