// plan_rows.cu -- block tables and row metadata of a batch of requests, made
// on the device from the requests' lengths.
//
// "glm5next_dsa/layer.rs", decode_k: the K-row attn_metadata (positions, slots,
// seq_lens, block tables at stable addresses) that every call of the path reads.
//
// With a_s = max(0, need_s - held_s) blocks wanted and r_s = max(0, held_s -
// need_s) given back, everything follows from three prefix sums over the
// requests (rows, a, r): the k-th block taken is element F + Rtot - 1 - k of the
// free stack with the given-back blocks on top, whichever request takes it, and
// a given-back block is found by a binary search of r's prefix sum.  So no CTA
// waits for another: each loads the three arrays (12 bytes a request, from L2),
// scans them in shared memory and writes its share of the rows, and a table
// entry that another CTA appends is computed, not read.  Only the state kept in
// place (held, the stack's count) has to change after every CTA has read it:
// the CTA that takes the last ticket writes it.
#include <algorithm>

#include "dsa_device.cuh"
#include "dsa_internal.h"

namespace dsa {
namespace {

constexpr int kThreads = 1024;
static_assert((kThreads & (kThreads - 1)) == 0, "the rows' threads are counted from the middle");
constexpr int kWarps = kThreads / 32;
// Row-table entries of a warp's turn, all loads in flight before the first
// store.
constexpr int kSpan = 512;
constexpr int kPer = kSpan / 32;

struct Shared {
  int warp_sum[3][32];
  int taken;  // blocks taken from the stack by the requests that are served
  int last;
};

// Exclusive scan over the CTA of three values at once; `total` their sums.
__device__ __forceinline__ void scan3(const int (&v)[3], int (&ex)[3], int (&total)[3], Shared* sh) {
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
#pragma unroll
  for (int k = 0; k < 3; ++k) {
    int x = v[k];
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int y = __shfl_up_sync(0xFFFFFFFFu, x, o);
      if (lane >= o) x += y;
    }
    if (lane == 31) sh->warp_sum[k][warp] = x;
    ex[k] = x - v[k];
  }
  __syncthreads();
#pragma unroll
  for (int k = 0; k < 3; ++k) {
    const int w = lane < kWarps ? sh->warp_sum[k][lane] : 0;
    int x = w;
#pragma unroll
    for (int o = 1; o < kWarps; o <<= 1) {
      const int y = __shfl_up_sync(0xFFFFFFFFu, x, o);
      if (lane >= o) x += y;
    }
    ex[k] += __shfl_sync(0xFFFFFFFFu, x - w, warp);
    total[k] = __shfl_sync(0xFFFFFFFFu, x, kWarps - 1);
  }
  __syncthreads();
}

// The requests' prefix sums in shared memory, [seqs + 1] each.
struct Scan {
  int* rows;   // first row
  int* want;   // blocks wanted by the requests before
  int* back;   // blocks given back by the requests before
  int* held;   // blocks held before the call
  int* need;   // blocks needed after it; -1: invalid request
};

constexpr size_t scan_bytes(int seqs) { return 5 * (static_cast<size_t>(seqs) + 1) * sizeof(int); }
static_assert(scan_bytes(DSA_PLAN_MAX_SEQS) + sizeof(Shared) <= kMaxSmemBytes, "shared memory budget");

// Index of the last entry of the exclusive prefix `a` [n + 1] that is <= x,
// among the requests (0 <= x < a[n]): the request that x falls into.
__device__ __forceinline__ int find(const int* a, int n, int x) {
  int lo = 0, hi = n;  // a[lo] <= x < a[hi]
  while (hi - lo > 1) {
    const int mid = (lo + hi) >> 1;
    if (a[mid] <= x) lo = mid; else hi = mid;
  }
  return lo;
}

__global__ void __launch_bounds__(kThreads) plan_rows_kernel(const PlanRowsParams kp) {
  extern __shared__ int smem[];
  __shared__ Shared sh;
  const dsa_plan& p = kp.p;
  const int n = p.seqs, tid = threadIdx.x, lane = tid & 31;
  Scan sc;
  sc.rows = smem;
  sc.want = sc.rows + n + 1;
  sc.back = sc.want + n + 1;
  sc.held = sc.back + n + 1;
  sc.need = sc.held + n + 1;
  const bool first = blockIdx.x == 0;
  grid_dep_launch();
  grid_dep_wait();  // the lengths and the state may come from the kernel before

  if (tid == 0) sh.taken = 0;
  int carry[3] = {0, 0, 0};
  for (int s0 = 0; s0 < n; s0 += kThreads) {
    const int s = s0 + tid;
    int v[3] = {0, 0, 0};
    int held = 0, need = -1;
    if (s < n) {
      const int len = p.seq_lens[s], fresh = p.new_tokens[s];
      held = p.held_in[s];
      const bool rows_ok = fresh >= 0 && fresh <= p.rows;
      // (32 bits hold the sum of a length of 0 or more and a block size; a length below
      // has no rows and is refused with them)
      const uint32_t blocks = (static_cast<uint32_t>(len) + (p.block_size - 1)) / static_cast<uint32_t>(p.block_size);
      if (rows_ok && fresh <= len && blocks <= static_cast<uint32_t>(p.max_blocks_per_seq) && held >= 0 &&
          held <= p.max_blocks_per_seq) {
        need = static_cast<int>(blocks);
        v[1] = max(0, need - held);
        v[2] = max(0, held - need);
      } else if (first) {
        record_error(kp.err, DSA_DEVERR_SEQ_LEN, s);
      }
      v[0] = rows_ok ? fresh : 0;
    }
    int ex[3], total[3];
    scan3(v, ex, total, &sh);
    if (s < n) {
      sc.rows[s] = carry[0] + ex[0];
      sc.want[s] = carry[1] + ex[1];
      sc.back[s] = carry[2] + ex[2];
      sc.held[s] = held;
      sc.need[s] = need;
    }
#pragma unroll
    for (int k = 0; k < 3; ++k) carry[k] += total[k];
  }
  const int nrows = carry[0], nback = carry[2];
  if (tid == 0) {
    sc.rows[n] = carry[0];
    sc.want[n] = carry[1];
    sc.back[n] = carry[2];
  }
  int stack = p.free_in[0];
  if (stack < 0 || stack > p.free_capacity) {
    if (first && tid == 0) record_error(kp.err, DSA_DEVERR_FREE, -1);
    stack = 0;
  }
  const int64_t avail = static_cast<int64_t>(stack) + nback;
  __syncthreads();
  // The largest amount wanted that the stack covers: what leaves it.
  for (int s = tid; s < n; s += kThreads) {
    const int upto = sc.want[s + 1];
    if (upto <= avail) {
      if (upto > sc.want[s]) atomicMax(&sh.taken, upto);
    } else if (first && upto > sc.want[s]) {
      record_error(kp.err, DSA_DEVERR_FREE, s);
    }
  }
  // Every thread of this CTA has read held_in and free_in; the last CTA to get
  // here writes their successors, at its end (the ticket's way to L2 and back is
  // nobody's wait until then).
  int ticket = 0;
  if (tid == 0) ticket = atomicAdd(&p.free_out[1], 1);
  __syncthreads();
  const int taken = sh.taken;
  const int kept = max(0, nback - taken);  // given-back blocks that stay on the stack
  auto refused = [&](int s) { return sc.want[s + 1] > avail && sc.want[s + 1] > sc.want[s]; };
  // The k-th block taken.
  auto pop = [&](int k) -> int {
    const int64_t at = avail - 1 - k;
    if (at < stack) return p.free_blocks[at];
    const int i = static_cast<int>(at - stack);
    const int s = find(sc.back, n, i);
    return p.block_table[static_cast<int64_t>(s) * p.bt_stride + sc.need[s] + (i - sc.back[s])];
  };
  // Entry b < need of request s's table after the call.
  auto entry = [&](int s, int b) -> int {
    if (b < sc.held[s]) return p.block_table[static_cast<int64_t>(s) * p.bt_stride + b];
    return pop(sc.want[s] + (b - sc.held[s]));
  };

  if (first) {
    for (int s = tid; s <= n; s += kThreads) p.row_start[s] = sc.rows[s];
    if (p.served_lens != nullptr)
      for (int s = tid; s < n; s += kThreads) p.served_lens[s] = sc.need[s] < 0 || refused(s) ? 0 : p.seq_lens[s];
    if (tid == 0 && nrows > p.rows) record_error(kp.err, DSA_DEVERR_ROWS, find(sc.rows, n, p.rows));
  }

  const int gwarp = blockIdx.x * kWarps + (tid >> 5), nwarps = gridDim.x * kWarps;
  // The requests' own tables and the stack, one warp a request.
  for (int s = gwarp; s < n; s += nwarps) {
    const int held = sc.held[s], need = sc.need[s];
    int32_t* row = p.block_table + static_cast<int64_t>(s) * p.bt_stride;
    if (need < 0) continue;  // an invalid request's `held` bounds nothing
    const bool no = refused(s);
    // (Loads of eight turns before their stores: a prompt takes, a request that
    // ends gives back, its blocks by the hundred.)
    constexpr int kTurns = 8;
    for (int b0 = held + lane; b0 < need; b0 += 32 * kTurns) {
      int v[kTurns];
#pragma unroll
      for (int k = 0; k < kTurns; ++k) v[k] = !no && b0 + 32 * k < need ? pop(sc.want[s] + (b0 + 32 * k - held)) : -1;
#pragma unroll
      for (int k = 0; k < kTurns; ++k)
        if (b0 + 32 * k < need) row[b0 + 32 * k] = v[k];
    }
    const int fits = static_cast<int>(min(static_cast<int64_t>(kept), static_cast<int64_t>(p.free_capacity) - stack));
    const int up = need + min(held - need, max(0, fits - sc.back[s]));  // entries below it go onto the stack
    for (int b0 = need + lane; b0 < up; b0 += 32 * kTurns) {
      int v[kTurns];
#pragma unroll
      for (int k = 0; k < kTurns; ++k)
        if (b0 + 32 * k < up) v[k] = row[b0 + 32 * k];
#pragma unroll
      for (int k = 0; k < kTurns; ++k)
        if (b0 + 32 * k < up) p.free_blocks[stack + sc.back[s] + (b0 + 32 * k - need)] = v[k];
    }
  }
  // The rows: the requests', and empty ones behind them where they are asked for.
  const int out_rows = (p.flags & DSA_PLAN_EMPTY_TAIL) != 0 ? p.rows : min(nrows, p.rows);
  // (Other warps begin with the requests' tables, and others with the rows'.)
  for (int r = blockIdx.x * kThreads + ((tid + kThreads / 2) & (kThreads - 1)); r < out_rows; r += gridDim.x * kThreads) {
    const int s = r < nrows ? find(sc.rows, n, r) : -1;
    const bool live = s >= 0 && sc.need[s] >= 0 && !refused(s);
    int pos = 0;
    int64_t slot = -1;
    if (live) {
      pos = p.seq_lens[s] - (sc.rows[s + 1] - r);
      slot = static_cast<int64_t>(entry(s, pos / p.block_size)) * p.block_size + pos % p.block_size;
    }
    p.positions[r] = static_cast<uint32_t>(pos);
    p.slots[r] = slot;
    p.row_lens[r] = live ? pos + 1 : 0;
    if (p.row_seq != nullptr) p.row_seq[r] = s;
  }
  // A warp's turn is kSpan entries of `run` consecutive rows, whose request's
  // entries are looked up and loaded once; single rows while there are warps to
  // spare (12,000 rows of 1,031 entries: 17.6 us by single rows, 12.9 by fours,
  // where a fill of the tables takes 7.4; 28 rows of 1,025: 4.7 by single rows, 6.2
  // by fours).
  const int width = p.max_blocks_per_seq, spans = (width + kSpan - 1) / kSpan;
  const int run = static_cast<int64_t>(out_rows) * spans >= 4ll * nwarps ? 4 : 1;
  const int turns = p.row_table != nullptr ? (out_rows + run - 1) / run * spans : 0;
  constexpr uint32_t kAll = (1u << kPer) - 1u;
  // Entries base + 32 k + lane of a span that are below x.
  auto below = [&](int base, int x) {
    const int m = (x - base - lane + 31) >> 5;          // k < m
    return m >= kPer ? kAll : m <= 0 ? 0u : (1u << m) - 1u;
  };
  for (int turn = nwarps - 1 - gwarp; turn < turns; turn += nwarps) {
    const int r0 = turn / spans * run, base = turn % spans * kSpan;
    const int r1 = min(r0 + run, out_rows);
    const uint32_t in = below(base, width);
    int s = find(sc.rows, n, r0), until = 0, need = 0, kept_blocks = 0, fresh = -1;
    int v[kPer];
    uint32_t put = 0;                                   // entries to be written from v
    for (int r = r0; r < r1; ++r) {
      if (r >= until) {                                 // the first row of s, or behind the requests' rows
        if (r < nrows)
          while ((until = sc.rows[s + 1]) <= r) ++s;
        else
          until = out_rows;
        need = r >= nrows || refused(s) ? 0 : max(0, sc.need[s]);
        kept_blocks = min(max(0, sc.held[s]), need);
        const int32_t* row = p.block_table + static_cast<int64_t>(s) * p.bt_stride + base + lane;
        const uint32_t old = below(base, kept_blocks);
        if (__all_sync(0xFFFFFFFFu, old == kAll)) {
#pragma unroll
          for (int k = 0; k < kPer; ++k) v[k] = row[32 * k];
        } else {
#pragma unroll
          for (int k = 0; k < kPer; ++k) v[k] = (old >> k) & 1u ? row[32 * k] : -1;
        }
        put = in & (old | ~below(base, need));
        if (kept_blocks + lane < need && kept_blocks < base + kSpan && base < need) fresh = pop(sc.want[s] + lane);
      }
      int32_t* row = p.row_table + static_cast<int64_t>(r) * p.row_bt_stride;
      int32_t* to = row + base + lane;
      if (__all_sync(0xFFFFFFFFu, put == kAll)) {
#pragma unroll
        for (int k = 0; k < kPer; ++k) to[32 * k] = v[k];
      } else {
#pragma unroll
        for (int k = 0; k < kPer; ++k)
          if ((put >> k) & 1u) to[32 * k] = v[k];
      }
      // The entries taken in this call: few, and in few of the spans.
      for (int b = kept_blocks + lane; b < min(need, base + kSpan); b += 32)
        if (b >= base) row[b] = b < kept_blocks + 32 ? fresh : pop(sc.want[s] + (b - kept_blocks));
    }
  }

  if (tid == 0) sh.last = ticket == static_cast<int>(gridDim.x) - 1;
  __syncthreads();
  if (sh.last) {
    for (int s = tid; s < n; s += kThreads)
      p.held_out[s] = sc.need[s] < 0 || refused(s) ? sc.held[s] : sc.need[s];
    if (tid == 0) {
      int64_t left = avail - taken;
      if (left > p.free_capacity) {
        record_error(kp.err, DSA_DEVERR_FREE, -1);
        left = p.free_capacity;
      }
      p.free_out[0] = static_cast<int>(left);
      p.free_out[1] = 0;
    }
  }
}

}  // namespace

cudaError_t launch_plan_rows(const PlanRowsParams& p, int num_sms, cudaStream_t stream) {
  const size_t smem = scan_bytes(p.p.seqs);
  // Above 48 KB a block in all, its static part included, a kernel has to ask; for the
  // most there can be (see kMaxSmemBytes).
  static_assert(sizeof(Shared) <= 1008, "47 KB leave room for it");
  if (smem > 47 * 1024) {
    const cudaError_t e = cudaFuncSetAttribute(
        plan_rows_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, static_cast<int>(scan_bytes(DSA_PLAN_MAX_SEQS)));
    if (e != cudaSuccess) return e;
  }
  // A CTA for every 32 warps' turns, 1,024 rows or 64 requests, up to one a SM: each scans
  // all requests.
  const int64_t spans = p.p.row_table != nullptr ? (p.p.max_blocks_per_seq + kSpan - 1) / kSpan : 0;
  int64_t ctas = std::max((p.p.rows * spans + kWarps - 1) / kWarps,
                          static_cast<int64_t>(std::max((p.p.rows + kThreads - 1) / kThreads, p.p.seqs / (2 * kWarps))));
  if (ctas > num_sms) ctas = num_sms;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(static_cast<unsigned>(ctas), 1, 1);
  cfg.blockDim = dim3(kThreads, 1, 1);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = stream;
  cudaLaunchAttribute attr[1] = {dependent_launch_attr()};
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, plan_rows_kernel, p);
}

}  // namespace dsa
