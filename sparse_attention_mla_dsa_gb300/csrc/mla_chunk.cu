// mla_chunk.cu -- dense causal attention of each request's new tokens over its
// paged FP8 latent cache, on the 5th-generation tensor cores.
//
// "glm5next_dsa/layer.rs", module header trap 4 (Q arrives absorbed into the
// 512-wide latent space) and decode_k (K and V are the same latent pool, slot =
// block * block_size + pos % block_size).  Per row, head and visible token j:
//   z_j = sm_scale * kv_scale * (q . e4m3(latent_j)),  p = softmax(z),
//   out = kv_scale * sum_j p_j e4m3(latent_j),  lse = log sum_j exp(z_j).
//
// Work.  A request's (row, head) pairs, in order, are its lines; 128 lines in a
// row are an item, 256 tokens a tile, and an item has as many tiles as its last
// line sees.  A pair of CTAs (a cluster on two SMs) works through a contiguous
// range of the tiles of all items, every pair the same number, whatever the
// lengths: an item that a range ends inside leaves its unnormalised output and
// its (maximum, sum) in the workspace, and a merge kernel adds such parts up in
// the order of the tiles.
//
// Why a pair.  The output of 128 lines is 128 x 512 FP32, the whole tensor
// memory of one SM.  A cta_group::2 MMA of M = 128 gives each SM 64 lines and
// puts the two halves of N on the two halves of its lanes, so a line's 512
// output columns take 256 of its 512 tensor memory columns and two tiles of
// logits fit beside them.  Each CTA stages half of every operand: for S = Q K^T
// its 64 lines of Q and its 128 tokens of the tile (all 512 dims), for O += P V
// its 64 lines of P and its 256 dims of V (all 256 tokens).
//
// Copies.  A block of 16 KB is 128 tokens x 128 dims, K-major for S and MN-major
// for O; a tile has four of K and four of V a CTA, taken again as soon as the
// MMAs have read them.  An SM takes in 32 bytes a clock from L2 (62 GB/s measured,
// on every SM), so these 128 KB cost the 4,100 clocks that the tile's MMAs take.
// Keeping the two K blocks that are also V (a CTA's tokens, its dims) and copying
// 96 KB measured slower but for gathered pages (prompt of 1,024 rows 731 -> 775
// us): a block then lives from its copy to the end of O, and two tiles' blocks
// fill the shared memory, so that load, S, softmax and O of a tile follow each
// other.
//
// Precision.  The latents stay E4M3.  q * 2^s = hi + lo, two E4M3 terms, holds
// a bf16 q exactly but for elements 2^10 below the head's largest; a softmax
// weight is an E4M3 term and the E5M2 term of its remainder: within 2^-7 of the
// weight, about 2^-9.6 rms, down to 2^-14 of the line's largest; then within 2^-21
// of the largest or a quarter of the weight, whichever is less, rounded up or down by
// the token's place, so that sums over a long tail of small weights are not off
// (split_weights).  Two FP8 terms cost what one 16-bit term would and need no
// conversion of the latents.
// Products, sums, maxima and the output are FP32.
//
// What bounds it.  A tile's 64 MMAs take 4,100 clocks and its copies as many, each
// waiting for blocks that the other holds: the tensor pipe is busy 87 % of the time
// (1,024 rows of 64 heads at 9,000 tokens, one launch of 592 us) and the card at its
// power limit in calls after each other: 687 us then, 1.66 PFLOP/s counting only
// visible tokens.  64 tokens of 128 heads at up to 128k: 364 us.  32 tokens of 64
// heads (half of every MMA is empty) at up to 64k: 138 us, 3.1 TB/s of latents.  An
// item costs ~10,000 clocks besides: Q through the same 32 bytes a clock (3,800),
// its conversion (2,400), the output's store (3,800), the warps' meetings; 2,049
// rows of 128 heads, an item each: 466 us.  One token of 16 heads: 12.5 us a call in
// calls after each other, most of it first times.  Where the maxima move (logits of a
// standard deviation of 1.1 instead of 0.07) long calls take 11 to 21 % more.
#include "dsa_device.cuh"
#include "dsa_internal.h"

namespace dsa {
namespace {

constexpr int kThreads = 640;        // warps 0, 2 copy K, V; 1, 3 issue S, O; 4-19 softmax
constexpr int kSoftmaxWarp0 = 4;
constexpr int kSoftmaxWarps = 16;
constexpr int kSoftmaxThreads = 32 * kSoftmaxWarps;
constexpr int kItem = 128;           // lines of an item (MMA M over the pair)
constexpr int kLines = 64;           // lines of a CTA
constexpr int kTile = 256;           // tokens of a tile
constexpr int kTok = 32;             // tokens of a softmax thread
constexpr int kBlocks = 8;           // of 128 tokens x 128 dims: four of K, four of V
constexpr uint32_t kBlockBytes = 16384;
constexpr uint32_t kQBytes = 65536;  // [term][128-dim block][64 lines][128 B]
constexpr uint32_t kPBytes = 32768;  // [term][128-token half][64 lines][128 B]
constexpr uint32_t kBlockOff = kQBytes + kPBytes;
constexpr uint32_t kCtlOff = kBlockOff + kBlocks * kBlockBytes;
constexpr uint32_t kTmemCols = 512;  // O: 0..255, S: 256 + 128 * buffer
constexpr uint32_t kSCol = 256;
constexpr int kMasks = 8;            // tiles whose token masks are kept (the copies are up to four ahead)
// An item costs what so many tiles cost, besides its tiles (2,049 rows of 128 heads:
// 558 us with 1, 473 with 2 or 3; a ragged batch of 24: 230, 200, 213).
constexpr int kItemCost = 2;
constexpr float kPMaxLog2 = 0.75f;   // a weight 2^(z - m) stays below 2^0.75 ...
constexpr float kPLog2 = 8.0f;       // ... and 2^8 times it, as it is summed too, below the E4M3 maximum 448
constexpr float kPUnit = 1.0f / 256.0f;
constexpr float kSmallLog2 = 10.0f;  // weights of a thread that are all below 2^-10 are dithered
constexpr int kMergeThreads = 256;
constexpr int kMaxPairs = 256;
static_assert(kMaxPairs == kMergeThreads, "a merge thread for every pair");

// What the softmax warps need of a segment, as the warp that copies K leaves it.
struct SegRecord {
  int64_t gline;                     // the item's first line in q and out
  int32_t lines;                     // of the request, from the item's first on
  int32_t ctx;                       // tokens that its new ones come after
  int32_t first;                     // the item's first line in the request
  int32_t begin, end;                // tiles; begin = end: the range is done
  int32_t whole;                     // the item is in this range alone
  int32_t parts;                     // else, where it begins here: ranges that share it
  int32_t pad;
};
constexpr int kSegs = 4;

// Barriers of tile t; where no phase is given, index t & 1 and phase t >> 1.
struct __align__(16) Ctl {
  uint64_t kfull[4], vfull[4];       // leader: copies have landed, in both CTAs (phase: t)
  uint64_t kread[4];                 // S has read the block (phase: t)
  uint64_t vread[4];                 // O has read V and P of the tokens 0..127, 128..255 (2 * (t & 1) + half)
  uint64_t sfull[2], sfree[2];
  uint64_t pready[2];                // P of the tile's first and second 128 tokens (index: half, phase: t)
  uint64_t qready, vseen, drain[2];
  uint32_t mask[kMasks][8];          // a bit for each token of a tile: there is a latent
  uint32_t tag[kMasks];              // 2 * (tile + 1), and 1 if every token before the item's end has one
  SegRecord seg[kSegs];
  uint32_t segs;                     // segments left in seg[], over all
  int more;                          // whether there is a next one: the softmax warps' common view
  uint16_t fills[kBlocks], peer_fills[kBlocks];  // copies begun of each block, see copy(); the other CTA's
  uint32_t tmem_base;
  int abort_flag;
  int begun;                         // the copies of the first tile's K are on their way
  float qexp[kLines];
  float red[8][kLines];
};
constexpr uint32_t kSmemBytes = kCtlOff + sizeof(Ctl);
static_assert(kSmemBytes <= 227 * 1024, "shared memory budget");

// ------------------------------------------------------------------ schedule
struct SeqInfo {
  int row0, rows, ctx, lines, items;
};

// Rows, lines and items of request s; no items where it has no rows or is
// refused (`why`: the error to record).  One of length 0 with rows (-ctx of them, of
// which none sees a token) has its items, of one tile with no tokens.
__device__ __forceinline__ SeqInfo seq_info(const ChunkParams& p, int s, int* why = nullptr) {
  SeqInfo q;
  q.row0 = p.seqs.row_start[s];
  const int64_t end = p.seqs.row_start[s + 1], len = p.seqs.seq_lens[s];
  const int64_t rows = end - q.row0;
  int bad = 0;
  if (rows > 0 && (q.row0 < 0 || end > p.rows)) bad = DSA_DEVERR_ROWS;
  else if (rows > 0 && len != 0 && (len < rows || len > static_cast<int64_t>(p.seqs.max_blocks_per_seq) * p.seqs.block_size))
    bad = DSA_DEVERR_SEQ_LEN;
  if (why != nullptr) *why = bad;
  q.rows = rows > 0 && bad == 0 ? static_cast<int>(rows) : 0;
  q.ctx = static_cast<int>(len) - q.rows;
  q.lines = q.rows * p.heads;
  q.items = (q.lines + kItem - 1) / kItem;
  return q;
}
// Tokens that the last line of item j sees, and its tiles.
__device__ __forceinline__ int item_end(const ChunkParams& p, const SeqInfo& q, int j) {
  return q.ctx + (min(kItem * (j + 1), q.lines) - 1) / p.heads + 1;
}
__device__ __forceinline__ int item_tiles(const ChunkParams& p, const SeqInfo& q, int j) {
  return max(1, (item_end(p, q, j) + kTile - 1) / kTile);
}
// The fewest tiles of an item of the request.
__device__ __forceinline__ int least_tiles(const SeqInfo& q) { return max(1, (q.ctx + kTile) / kTile); }
// How many of the request's items see at most x new tokens.
__device__ __forceinline__ int items_within(const ChunkParams& p, const SeqInfo& q, int x) {
  return x <= 0 ? 0 : x >= q.rows ? q.items : x * p.heads / kItem;  // (65,535 x 4,096 lines at most)
}
// The request's cost: items by their number of tiles v, those within v tiles
// less those within v - 1.
__device__ __forceinline__ int64_t seq_cost(const ChunkParams& p, const SeqInfo& q) {
  if (q.items == 0) return 0;
  int64_t sum = 0;
  int below = 0;
  for (int v = least_tiles(q); below < q.items; ++v) {
    const int upto = items_within(p, q, static_cast<int>(min(static_cast<int64_t>(v) * kTile - q.ctx, static_cast<int64_t>(q.rows))));
    sum += static_cast<int64_t>(upto - below) * (v + kItemCost);
    below = upto;
  }
  return sum;
}

// a / b and a % b, in 32 bits where they fit (a 64-bit division is a routine of
// its own, and every CTA of a call waits for these).
__device__ __forceinline__ int64_t div_small(int64_t a, uint32_t b, int64_t* rest = nullptr) {
  int64_t q;
  if ((a >> 32) == 0) q = static_cast<uint32_t>(a) / b;
  else q = a / static_cast<int64_t>(b);
  if (rest != nullptr) *rest = a - q * b;
  return q;
}

struct Place {
  int64_t total;   // cost of the call
  int64_t per;     // cost of a pair's range
  int seq, item;
  int64_t off;     // cost of the item before the place: its own first, then its tiles
};

// Finds place `target(per)` of the call: every thread sums a run of requests,
// the CTA scans the sums, and the thread whose run holds it walks to it.
// `scratch`: kN int64 and a Place of shared memory, free again after the caller's
// next barrier.  Returns seq -1 past the end.  (All threads read the answer from
// shared memory: values that a shuffle gave are not known to be the same in all
// lanes, and what is computed from them then costs long calls 2 to 10 %.)
template <int kN, typename Target>
__device__ __forceinline__ Place find_place(const ChunkParams& p, int pairs, Target target,
                                            int64_t* scratch, bool report) {
  Place& found = *reinterpret_cast<Place*>(scratch + kN);
  const int tid = threadIdx.x, n = p.seqs.seqs, run = (n + kN - 1) / kN;
  const int s0 = min(n, tid * run), s1 = min(n, s0 + run);
  int64_t sum = 0;
  for (int s = s0; s < s1; ++s) {
    int why = 0;
    const SeqInfo q = seq_info(p, s, &why);
    if (why != 0 && report) record_error(p.err, why, s);
    sum += seq_cost(p, q);
  }
  // A scan over the warp, then one of the warps' sums.
  const int lane = tid & 31, warp = tid >> 5;
  int64_t upto = sum;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int64_t y = __shfl_up_sync(0xFFFFFFFFu, upto, o);
    if (lane >= o) upto += y;
  }
  if (lane == 31) scratch[warp] = upto;
  if (tid == 0) found.seq = -1;
  __syncthreads();
  if (tid < 32) {
    const int64_t mine = tid < kN / 32 ? scratch[tid] : 0;
    int64_t x = mine;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int64_t y = __shfl_up_sync(0xFFFFFFFFu, x, o);
      if (tid >= o) x += y;
    }
    if (tid < kN / 32) scratch[tid] = x - mine;
    if (tid == 31) {
      found.total = x;
      found.per = max(static_cast<int64_t>(1), div_small(x + pairs - 1, static_cast<uint32_t>(pairs)));
    }
  }
  __syncthreads();
  const int64_t want = target(found.per);
  int64_t at = scratch[warp] + upto - sum;
  if (want < found.total && want >= at && want < at + sum) {
    for (int s = s0; s < s1; ++s) {
      const SeqInfo q = seq_info(p, s);
      const int64_t t = seq_cost(p, q);
      if (want >= at + t) {
        at += t;
        continue;
      }
      int64_t off = want - at;
      int below = 0;
      for (int v = least_tiles(q);; ++v) {
        const int within = items_within(p, q, static_cast<int>(min(static_cast<int64_t>(v) * kTile - q.ctx, static_cast<int64_t>(q.rows))));
        const int64_t here = static_cast<int64_t>(within - below) * (v + kItemCost);
        if (off < here) {
          found.seq = s;
          found.item = below + static_cast<int>(div_small(off, static_cast<uint32_t>(v + kItemCost), &found.off));
          break;
        }
        off -= here;
        below = within;
      }
      break;
    }
  }
  __syncthreads();
  return found;
}

// The part of one item in a pair's range, and the walk over the range.
struct Segment {
  SeqInfo q;
  int seq, item, tiles;   // tiles: of the item
  int begin, end;         // tiles of the segment
};
struct Walk {
  int seq, item;
  int64_t off;            // cost of the item before the range's place in it
  int64_t left;           // cost
};
__device__ __forceinline__ bool next_segment(const ChunkParams& p, Walk& w, Segment& g) {
  if (w.left <= 0) return false;
  g.q = seq_info(p, w.seq);
  while (w.item >= g.q.items) {
    w.item = 0;
    if (++w.seq >= p.seqs.seqs) return false;
    g.q = seq_info(p, w.seq);
  }
  g.seq = w.seq;
  g.item = w.item;
  g.tiles = item_tiles(p, g.q, w.item);
  const int64_t end = min(w.off + w.left, static_cast<int64_t>(g.tiles + kItemCost));
  g.begin = static_cast<int>(max(static_cast<int64_t>(0), w.off - kItemCost));
  g.end = static_cast<int>(end - kItemCost);
  w.left -= end - w.off;
  w.off = 0;
  ++w.item;
  // A range that ends in an item's own cost leaves it to the next.
  return g.end > g.begin;
}

// Lines of an item in each CTA of its pair, of `lines` that the request has from
// the item's first on: those of a half-empty item (one token at 64 heads) are
// shared by both, which then load, convert and store half of them each (one decode
// 23.6 -> 22.5 us, 32 decodes 137.5 -> 136.8).
__device__ __forceinline__ int cta_lines(int lines) { return lines > kLines ? kLines : kLines / 2; }

// ------------------------------------------------------------------ pair
__device__ __forceinline__ uint32_t cta_rank() {
  uint32_t r;
  asm volatile("mov.u32 %0, %%cluster_ctarank;" : "=r"(r));
  return r;
}
// One lane of the whole warp, always the same.  A branch on it leaves the operands
// of MMAs and copies in uniform registers, one on lane == 0 does not: first token
// 15.7 -> 15.0 us, a prompt of 2,049 rows 496 -> 489.
__device__ __forceinline__ bool elect_one() {
  uint32_t one;
  asm volatile("{\n\t.reg .pred p;\n\telect.sync _|p, 0xFFFFFFFF;\n\tselp.u32 %0, 1, 0, p;\n\t}" : "=r"(one));
  return one != 0;
}
__device__ __forceinline__ void cluster_sync() {
  asm volatile("barrier.cluster.arrive.release.aligned;\n\tbarrier.cluster.wait.acquire.aligned;" ::: "memory");
}
// Address of `p` in the shared memory of CTA `rank` of the cluster.
__device__ __forceinline__ uint32_t map_to(const void* p, uint32_t rank) {
  uint32_t a;
  asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(a) : "r"(smem_u32(p)), "r"(rank));
  return a;
}
// Arrival on a barrier of either CTA.  The data it announces is read by MMAs
// (written for them by fence.proxy.async) or is none, so the order within this
// CTA is enough; a release to the cluster costs ~1,700 clocks of the softmax's
// 4,200 a tile, and an acquire from it ~200 (it invalidates the L1).
__device__ __forceinline__ void arrive_at(uint32_t bar) {
  asm volatile("mbarrier.arrive.shared::cluster.b64 _, [%0];" ::"r"(bar) : "memory");
}
// Orders what the leader's MMAs thread announced (V has landed) before this
// thread's reads of it.
__device__ __forceinline__ void acquire_cluster() { asm volatile("fence.acq_rel.cluster;" ::: "memory"); }
__device__ __forceinline__ bool aborted(Ctl* c) {
  return *reinterpret_cast<volatile int*>(&c->abort_flag) != 0;
}
// Marks both CTAs of the pair: their later waits are skipped.
__device__ __forceinline__ void set_abort(Ctl* c) {
  for (uint32_t r = 0; r < 2; ++r)
    asm volatile("st.volatile.shared::cluster.u32 [%0], %1;" ::"r"(map_to(&c->abort_flag, r)), "r"(1) : "memory");
}
// Bounded wait of one thread; a timeout is recorded and marks the pair.
__device__ __noinline__ bool wait_polls(Ctl* c, uint64_t* bar, uint32_t parity, int* err, uint64_t limit_ns) {
  const uint64_t t0 = global_ns();
  for (uint32_t i = 1; i < (1u << 30); ++i) {
    if (mbar_try_wait_hint(bar, parity, limit_ns < kShortWaitNs ? 32 : kSuspendHintNs)) return true;
    if ((i & 15u) == 0 || limit_ns < kShortWaitNs) {
      if (aborted(c)) return false;
      if (global_ns() - t0 > limit_ns) break;
    }
  }
  record_error(err, DSA_DEVERR_TIMEOUT, -1);
  set_abort(c);
  return false;
}
__device__ __forceinline__ bool wait_one(Ctl* c, uint64_t* bar, uint32_t parity, const ChunkParams& p) {
  if (p.wait_ns >= kShortWaitNs && mbar_try_wait(bar, parity)) return true;
  return wait_polls(c, bar, parity, p.err, p.wait_ns);
}
// The same for a whole warp, every lane polling (no lane waits for another's
// answer unless there is none yet).
__device__ __forceinline__ bool wait_all(Ctl* c, uint64_t* bar, uint32_t parity, int lane, const ChunkParams& p) {
  const bool done = p.wait_ns >= kShortWaitNs && mbar_try_wait(bar, parity);
  if (__all_sync(0xFFFFFFFFu, done)) return true;
  int ok = 1;
  if (lane == 0) ok = wait_polls(c, bar, parity, p.err, p.wait_ns) ? 1 : 0;
  return __shfl_sync(0xFFFFFFFFu, ok, 0) != 0;
}
__device__ __forceinline__ bool warp_wait(Ctl* c, uint64_t* bar, uint32_t parity, int lane, const ChunkParams& p) {
  int ok = 1;
  if (lane == 0) ok = wait_one(c, bar, parity, p) ? 1 : 0;
  return __shfl_sync(0xFFFFFFFFu, ok, 0) != 0;
}

// Bounded wait of a warp until `there()`, a test of shared memory by lane 0.
template <typename There>
__device__ __forceinline__ bool wait_until(Ctl* c, int lane, const ChunkParams& p, There there) {
  int ok = 1;
  if (lane == 0) {
    const uint64_t t0 = global_ns();
    while (!there()) {
      if (aborted(c) || global_ns() - t0 > p.wait_ns) {
        if (!aborted(c)) record_error(p.err, DSA_DEVERR_TIMEOUT, -1);
        set_abort(c);
        ok = 0;
        break;
      }
    }
    __threadfence_block();
  }
  return __shfl_sync(0xFFFFFFFFu, ok, 0) != 0;
}
// More than `seg` segments have been left.
__device__ __forceinline__ bool wait_segment(Ctl* c, uint32_t seg, int lane, const ChunkParams& p) {
  return wait_until(c, lane, p, [&] { return *reinterpret_cast<volatile uint32_t*>(&c->segs) > seg; });
}

// ------------------------------------------------------------------ tensor core
// kind::f8f6f4, F32 accumulate, M = 128 over the pair, N = 256; A E4M3 or E5M2
// K-major, B E4M3.
__host__ __device__ constexpr uint32_t idesc_f8(bool a_e5m2, bool b_mn_major) {
  return (1u << 4) | (a_e5m2 ? (1u << 7) : 0u) | (b_mn_major ? (1u << 16) : 0u) | ((256u >> 3) << 17) |
         ((128u >> 4) << 24);
}
// Low words of the operands' descriptors (umma_desc_sw128_kmajor; the same
// serves V, 128 contiguous bytes of MN per K row with the next 8 rows 1024 B on),
// which alone differ between MMAs: by the offset in 16-byte units.
__device__ __forceinline__ uint32_t desc_low(uint32_t saddr) {
  return static_cast<uint32_t>(umma_desc_sw128_kmajor(saddr));
}
constexpr uint32_t kDescHigh = (1024u >> 4) | (1u << 14) | (2u << 29);
// An MMA takes 64 clocks, so the instructions that lead to it count: an add for
// each operand, nothing else.
template <uint32_t kIdesc>
__device__ __forceinline__ void mma_pair(uint32_t d, uint32_t a, uint32_t b, uint32_t acc) {
  asm volatile(
      "{\n\t.reg .pred p;\n\t.reg .b64 a, b;\n\t"
      "setp.ne.b32 p, %3, 0;\n\t"
      "mov.b64 a, {%1, %4};\n\tmov.b64 b, {%2, %4};\n\t"
      "tcgen05.mma.cta_group::2.kind::f8f6f4 [%0], a, b, %5, p;\n\t}" ::"r"(d),
      "r"(a), "r"(b), "r"(acc), "n"(kDescHigh), "n"(kIdesc)
      : "memory");
}
// Arrives on `bar` of both CTAs once every MMA issued so far is complete.
__device__ __forceinline__ void commit_pair(uint64_t* bar) {
  asm volatile(
      "tcgen05.commit.cta_group::2.mbarrier::arrive::one.shared::cluster.multicast::cluster.b64 [%0], %1;" ::"r"(
          smem_u32(bar)),
      "h"(static_cast<uint16_t>(3))
      : "memory");
}
#define DSA_R16(r, o) \
  "=r"(r[o]), "=r"(r[o + 1]), "=r"(r[o + 2]), "=r"(r[o + 3]), "=r"(r[o + 4]), "=r"(r[o + 5]), "=r"(r[o + 6]), \
  "=r"(r[o + 7]), "=r"(r[o + 8]), "=r"(r[o + 9]), "=r"(r[o + 10]), "=r"(r[o + 11]), "=r"(r[o + 12]), \
  "=r"(r[o + 13]), "=r"(r[o + 14]), "=r"(r[o + 15])
// 32 consecutive columns of this thread's lane, waited for in the same statement.
__device__ __forceinline__ void tmem_load32(uint32_t taddr, float* v) {
  uint32_t r[32];
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x32.b32 "
      "{%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16,%17,%18,%19,%20,%21,%22,%23,%24,%25,%26,%27,%28,"
      "%29,%30,%31}, [%32];\n\t"
      "tcgen05.wait::ld.sync.aligned;"
      : DSA_R16(r, 0), DSA_R16(r, 16)
      : "r"(taddr)
      : "memory");
#pragma unroll
  for (int i = 0; i < 32; ++i) v[i] = __uint_as_float(r[i]);
}
__device__ __forceinline__ void tmem_store16(uint32_t taddr, const float* v) {
  asm volatile(
      "tcgen05.st.sync.aligned.32x32b.x16.b32 [%0], "
      "{%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16};" ::"r"(taddr),
      "r"(__float_as_uint(v[0])), "r"(__float_as_uint(v[1])), "r"(__float_as_uint(v[2])),
      "r"(__float_as_uint(v[3])), "r"(__float_as_uint(v[4])), "r"(__float_as_uint(v[5])),
      "r"(__float_as_uint(v[6])), "r"(__float_as_uint(v[7])), "r"(__float_as_uint(v[8])),
      "r"(__float_as_uint(v[9])), "r"(__float_as_uint(v[10])), "r"(__float_as_uint(v[11])),
      "r"(__float_as_uint(v[12])), "r"(__float_as_uint(v[13])), "r"(__float_as_uint(v[14])),
      "r"(__float_as_uint(v[15]))
      : "memory");
}

// ------------------------------------------------------------------ copies
// A box of the latent pool, 128 bytes (column x) of the rows from y on, into
// this CTA's shared memory; its bytes count on the leader's barrier `bar`.
__device__ __forceinline__ void tma_box(uint32_t dst, const CUtensorMap* map, uint32_t bar, int32_t x, int32_t y) {
  asm volatile(
      "cp.async.bulk.tensor.2d.cta_group::2.shared::cluster.global.tile.mbarrier::complete_tx::bytes"
      " [%0], [%1, {%2, %3}], [%4];" ::"r"(dst),
      "l"(reinterpret_cast<uint64_t>(map)), "r"(x), "r"(y), "r"(bar)
      : "memory");
}
// Four rows of 128 bytes each.
__device__ __forceinline__ void tma_gather4(uint32_t dst, const CUtensorMap* map, uint32_t bar, int32_t x,
                                            const int32_t* y) {
  asm volatile(
      "cp.async.bulk.tensor.2d.cta_group::2.shared::cluster.global.tile::gather4.mbarrier::complete_tx::bytes"
      " [%0], [%1, {%2, %3, %4, %5, %6}], [%7];" ::"r"(dst),
      "l"(reinterpret_cast<uint64_t>(map)), "r"(x), "r"(y[0]), "r"(y[1]), "r"(y[2]), "r"(y[3]), "r"(bar)
      : "memory");
}

// 32 lines x 32 dims of the output, from this warp's 2 KB of shared memory.
__device__ __forceinline__ void tma_store(const CUtensorMap* map, uint32_t src, int32_t x, int32_t y) {
  asm volatile(
      "cp.async.bulk.tensor.2d.global.shared::cta.tile.bulk_group [%0, {%1, %2}], [%3];\n\t"
      "cp.async.bulk.commit_group;" ::"l"(reinterpret_cast<uint64_t>(map)), "r"(x), "r"(y), "r"(src)
      : "memory");
}
__device__ __forceinline__ void tma_store_read() { asm volatile("cp.async.bulk.wait_group.read 0;" ::: "memory"); }
__device__ __forceinline__ void tma_store_done() { asm volatile("cp.async.bulk.wait_group 0;" ::: "memory"); }

// Two fp16 values as E4M3 codes, and their remainders, which fp16 holds exactly.
__device__ __forceinline__ uint16_t split_e4m3(uint32_t h2, uint32_t& rest) {
  uint16_t hi;
  uint32_t d2;
  asm("cvt.rn.satfinite.e4m3x2.f16x2 %0, %1;" : "=h"(hi) : "r"(h2));
  asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(d2) : "h"(hi));
  asm("sub.rn.f16x2 %0, %1, %2;" : "=r"(rest) : "r"(h2), "r"(d2));
  return hi;
}
__device__ __forceinline__ uint32_t pack_f16(float lo, float hi) {
  uint32_t h2;
  asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(h2) : "f"(hi), "f"(lo));
  return h2;
}
// q, already scaled: two E4M3 terms.
__device__ __forceinline__ void split_q(uint32_t h2, uint16_t& hi, uint16_t& lo) {
  uint32_t r2;
  hi = split_e4m3(h2, r2);
  asm("cvt.rn.satfinite.e4m3x2.f16x2 %0, %1;" : "=h"(lo) : "r"(r2));
}
// Two softmax weights (already times 2^8): an E4M3 term, returned, and the E5M2 term
// of the remainder, left as the upper bytes of `lo`'s halves: E5M2 is fp16's upper
// byte, so `add` to the lower byte before it goes is the rounding (half a step: 0x80).
// Below 2^-14 of the line's largest, where E4M3 has no full precision, the two terms
// keep so few bits that a long tail of like weights would all be rounded the same way
// (131,072 weights of 1.125 x 2^-19 beside one of 1 were 11 % short).  A thread none
// of whose 32 weights reaches 2^-10 therefore adds a dither, another of 0 .. 255 for
// each of a tile's 256 tokens, so that as many are rounded up as their sum needs; a
// weight of 2^-14 or more is still within 2^-7.  Beside a weight of 2^-10 the small
// ones' errors, 31 of at most 2^-22, are under 2^-7 of it.  A weight of 0 stays 0.
__device__ __forceinline__ uint16_t split_weights(uint32_t h2, uint32_t add, uint32_t& lo) {
  uint32_t rest;
  const uint16_t hi = split_e4m3(h2, rest);
  lo = rest + add;
  return hi;
}
constexpr uint32_t reverse_bits(uint32_t x, int n) {
  uint32_t y = 0;
  for (int i = 0; i < n; ++i) y |= ((x >> i) & 1u) << (n - 1 - i);
  return y;
}
// The upper five bits of the dither of tokens k and k + 1 of a thread's 32: evenly
// spread over tokens that follow each other.
constexpr uint32_t dither_of(int k) { return (reverse_bits(k, 5) << 3) | (reverse_bits(k + 1, 5) << 19); }
__device__ __forceinline__ float ex2(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}
__device__ __forceinline__ float2 fma2(float2 a, float2 b, float2 c) {
  float2 d;
  asm("{\n\t.reg .b64 a, b, c, d;\n\t"
      "mov.b64 a, {%2, %3};\n\tmov.b64 b, {%4, %5};\n\tmov.b64 c, {%6, %7};\n\t"
      "fma.rn.f32x2 d, a, b, c;\n\tmov.b64 {%0, %1}, d;\n\t}"
      : "=f"(d.x), "=f"(d.y)
      : "f"(a.x), "f"(a.y), "f"(b.x), "f"(b.y), "f"(c.x), "f"(c.y));
  return d;
}
// The bytes of w that are E4M3 NaN codes, zeroed.
__device__ __forceinline__ uint32_t zero_nan4(uint32_t w) {
  const uint32_t nan = __vcmpeq4(w & 0x7F7F7F7Fu, 0x7F7F7F7Fu);
  return w & ~nan;
}

// Barriers of the eight softmax warps that have the same 32 lines (ids 1, 2).
__device__ __forceinline__ void line_sync(int group) {
  asm volatile("bar.sync %0, %1;" ::"r"(1 + group), "n"(kSoftmaxThreads / 2) : "memory");
}
__device__ __forceinline__ bool line_sync_or(int group, bool pred) {
  uint32_t out;
  asm volatile(
      "{\n\t.reg .pred p, q;\n\t"
      "setp.ne.u32 p, %1, 0;\n\t"
      "bar.red.or.pred q, %2, %3, p;\n\t"
      "selp.u32 %0, 1, 0, q;\n\t}"
      : "=r"(out)
      : "r"(pred ? 1u : 0u), "r"(1 + group), "n"(kSoftmaxThreads / 2)
      : "memory");
  return out != 0;
}
__device__ __forceinline__ void softmax_sync() {
  asm volatile("bar.sync 3, %0;" ::"n"(kSoftmaxThreads) : "memory");
}

// ------------------------------------------------------------------ roles
// Where a tile's token groups (a box of box_rows tokens inside one block, or
// four tokens gathered) are in the pool: a group is one lane's, which looks its
// block up and issues its copies.  Absent tokens are at row nslots, past the end.
struct Rows {
  int32_t at[8];   // [0]: the box's first row; gathers: tokens 4l.. and 128 + 4l..
  int how[2];      // gathers: 0 nothing (another lane's box has them), 4 a gather, 16 a box
  bool missing;    // this lane has a token without a latent before the item's end
};
// kMask: also the tile's token mask, and the error of a missing block.
template <bool kMask, bool kGather>
__device__ __forceinline__ Rows lookup(const ChunkParams& p, const Segment& g, int end, int t, int lane,
                                       uint32_t rank, uint32_t* mask_words) {
  const int bs = p.seqs.block_size, h = p.box_rows, t0 = t * kTile;
  const int32_t* bt = p.seqs.block_table + static_cast<int64_t>(g.seq) * p.seqs.bt_stride;
  uint8_t* mask = reinterpret_cast<uint8_t*>(mask_words);
  const int32_t none = static_cast<int32_t>(p.nslots);
  Rows r;
#pragma unroll
  for (int i = 0; i < 8; ++i) r.at[i] = none;
  bool missing = false;
  if constexpr (!kGather) {
    const int tok = t0 + lane * h;
    int there = 0;
    if (lane * h < kTile) {
      if (tok < end) {
        const int64_t first = static_cast<int64_t>(bt[tok / bs]) * bs + tok % bs;
        if (first >= 0 && first < p.nslots) {
          r.at[0] = static_cast<int32_t>(first);
          there = static_cast<int>(min(static_cast<int64_t>(h), p.nslots - first));
        }
        missing = there < min(h, end - tok);
      }
      if constexpr (kMask)
        for (int i = 0; i < h; i += 8)
          mask[(lane * h + i) >> 3] = there >= i + 8 ? 0xFF : there <= i ? 0 : static_cast<uint8_t>((1 << (there - i)) - 1);
    }
  } else {
#pragma unroll
    for (int k = 0; k < 2; ++k) {
      // The four tokens' blocks first (one division, then steps), so that their
      // loads are in flight together.
      const int tok = t0 + (k * 32 + lane) * 4;
      int blk[4], in[4], phys[4];
      blk[0] = tok / bs;
      in[0] = tok - blk[0] * bs;
#pragma unroll
      for (int i = 1; i < 4; ++i) {
        const bool over = in[i - 1] + 1 == bs;
        blk[i] = blk[i - 1] + (over ? 1 : 0);
        in[i] = over ? 0 : in[i - 1] + 1;
      }
#pragma unroll
      for (int i = 0; i < 4; ++i) phys[i] = tok + i < end ? bt[blk[i]] : -1;
      uint32_t bits = 0;
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const int64_t slot = static_cast<int64_t>(phys[i]) * bs + in[i];
        if (phys[i] >= 0 && slot < p.nslots) {
          r.at[k * 4 + i] = static_cast<int32_t>(slot);
          bits |= 1u << i;
        } else if (tok + i < end) {
          missing = true;
        }
      }
      if constexpr (kMask) {
        const uint32_t other = __shfl_down_sync(0xFFFFFFFFu, bits, 1);
        if ((lane & 1) == 0) mask[(k * 32 + lane) >> 1] = static_cast<uint8_t>(bits | (other << 4));
      }
      // Four lanes whose sixteen rows follow each other leave them to the first
      // of the four, counted from where their run begins: one copy for four (a
      // warp issues one in ~35 ns; pages of 20 tokens: 13 copies for 32).
      const int32_t* y = &r.at[k * 4];
      const bool run = y[0] < none && y[1] == y[0] + 1 && y[2] == y[0] + 2 && y[3] == y[0] + 3;
      const int32_t after = __shfl_down_sync(0xFFFFFFFFu, run ? y[0] : -1, 1);
      const uint32_t link = __ballot_sync(0xFFFFFFFFu, run && lane < 31 && after == y[0] + 4);
      const uint32_t breaks = ~link & ((1u << lane) - 1u);
      const int pos = lane - (32 - __clz(breaks)), more = __ffs(~(link >> lane)) - 1;
      r.how[k] = (pos & 3) + more >= 3 ? ((pos & 3) == 0 ? 16 : 0) : 4;
    }
  }
  if constexpr (kMask) __syncwarp();
  if (kMask && missing && rank == 0) record_error(p.err, DSA_DEVERR_BLOCK, g.seq);
  r.missing = missing;
  return r;
}

// Warp 0: this CTA's 128 tokens of every tile's K, a block for each 128 dims.
// Warp 2 (kV): the tile's V, all tokens and this CTA's 256 dims, a block for each
// 128 tokens x 128 dims.  The leader's warps expect the bytes of both CTAs.  Each
// has its own blocks: one warp alone fills a block, as a barrier's parity says
// nothing to a warp that may be two fills behind.
template <bool kV, bool kGather>
__device__ __forceinline__ void copy(const CUtensorMap& map, const CUtensorMap& map16, const ChunkParams& p, Ctl* ctl, uint8_t* blocks,
                                     int lane, uint32_t rank, int pair, int64_t per, Walk w) {
  const int from = rank ? 128 : 0;             // K: the tokens of this CTA
  uint32_t looked = 0, n = 0, segs = 0;
  const uint32_t dst0 = smem_u32(blocks + (kV ? 4 : 0) * kBlockBytes);
  const uint32_t bar0 = map_to(kV ? &ctl->vfull[0] : &ctl->kfull[0], 0);
  int64_t at = kV ? 0 : per * pair - w.off;    // cost of the call before the item
  // K: leaves the segment for the softmax warps (at most two ahead of them: the
  // copies before waited for an S of this segment's last or the one before that,
  // whose Q the softmax warps converted when they were done with what came before).
  auto publish = [&](const SegRecord& r) {
    if (lane == 0) {
      ctl->seg[segs % kSegs] = r;
      __threadfence_block();
      *reinterpret_cast<volatile uint32_t*>(&ctl->segs) = segs + 1;
    }
    ++segs;
  };
  // The copies begun of each block, for the kernel's end: those of tile n's first i
  // blocks too.  (As many as 3, or 4 .. 7 with the count's last two bits: a range may
  // have more tiles than 16 bits hold.)
  auto leave = [&](uint32_t n, int i) {
    const uint32_t begun = n + (lane < i ? 1 : 0);
    if (lane < 4) ctl->fills[(kV ? 4 : 0) + lane] = static_cast<uint16_t>(begun < 4 ? begun : 4 | (begun & 3));
  };
  Segment g;
  while (next_segment(p, w, g)) {
    const int end = item_end(p, g.q, g.item);
    if constexpr (!kV) {
      SegRecord r;
      r.first = g.item * kItem;
      r.gline = static_cast<int64_t>(g.q.row0) * p.heads + r.first;
      r.lines = g.q.lines - r.first;
      r.ctx = g.q.ctx;
      r.begin = g.begin;
      r.end = g.end;
      r.whole = g.begin == 0 && g.end == g.tiles ? 1 : 0;
      // the last range that has a tile of the item, from this one on
      r.parts = static_cast<int>((at + kItemCost + g.tiles - 1) / per - pair) + 1;
      r.pad = 0;
      at += g.tiles + kItemCost;
      publish(r);
    }
    // K: also leaves the tile's mask and brings the latents of a tile to come into
    // L2.
    auto look = [&](int t) {
      const Rows r = lookup<!kV, kGather>(p, g, end, t, lane, rank, kV ? nullptr : ctl->mask[looked % kMasks]);
      if constexpr (!kV) {
        const bool whole = !__any_sync(0xFFFFFFFFu, r.missing);
        if (lane == 0) {
          __threadfence_block();
          *reinterpret_cast<volatile uint32_t*>(&ctl->tag[looked % kMasks]) = 2 * (looked + 1) + (whole ? 1u : 0u);
        }
        ++looked;
        const int tok = lane * p.box_rows - from;
        if (!kGather && t > g.begin && tok >= 0 && tok < 128 && r.at[0] < p.nslots)
          for (int d = 0; d < 4; ++d) tma_prefetch_l2_2d(&map, d * 128, r.at[0]);
      }
      return r;
    };
    Rows next = look(g.begin);
    for (int t = g.begin; t < g.end; ++t, ++n) {
      const Rows r = next;
      // The call's first K before its first V: both would share the SM's way in.
      if (kV && n == 0 &&
          !wait_until(ctl, lane, p, [&] { return *reinterpret_cast<volatile int*>(&ctl->begun) != 0; }))
        return;
#pragma unroll 1
      for (int i = 0; i < 4; ++i) {
        uint64_t* const full = kV ? &ctl->vfull[i] : &ctl->kfull[i];
        if (n >= 1) {
          const uint32_t before = n - 1;
          bool go = true;
          if (!kV) go = wait_all(ctl, &ctl->kread[i], before & 1, lane, p);
          else if ((i & 1) == 0) go = wait_all(ctl, &ctl->vread[2 * (before & 1) + (i >> 1)], (before >> 1) & 1, lane, p);
          if (!go) {
            leave(n, i);
            return;
          }
        }
        const uint32_t dst = dst0 + i * kBlockBytes, bar = bar0 + i * 8;
        const int x = kV ? static_cast<int>(rank) * 256 + (i & 1) * 128 : i * 128;
        const int f = kV ? (i >> 1) * 128 : from;
        if constexpr (!kGather) {
          const int tok = lane * p.box_rows - f;
          if (tok >= 0 && tok < 128) tma_box(dst + tok * 128, &map, bar, x, r.at[0]);
        } else {
          int32_t y[4];
#pragma unroll
          for (int k = 0; k < 4; ++k) y[k] = f ? r.at[4 + k] : r.at[k];
          const int how = f ? r.how[1] : r.how[0];
          if (how == 16) tma_box(dst + lane * 512, &map16, bar, x, y[0]);
          else if (how == 4) tma_gather4(dst + lane * 512, &map, bar, x, y);
        }
        // (The barrier's phase ends with this arrival at the earliest, so the bytes may
        // come before they are expected.)
        if (rank == 0 && lane == 31) mbar_arrive_expect_tx(full, 2 * kBlockBytes);
        __syncwarp();
      }
      if (!kV && n == 0 && lane == 0) *const_cast<volatile int*>(&ctl->begun) = 1;
      if (!kV && t == g.begin) {
        // The segment's Q into L2 (a segment ahead of its conversion, but for the
        // first).
        const SegRecord& q = ctl->seg[(segs - 1) % kSegs];
        const int own = cta_lines(q.lines);
        for (int k = lane; k < kLines * 8; k += 32) {
          const int i = static_cast<int>(rank) * own + (k >> 3);
          if (i < q.lines && (k >> 3) < own) prefetch_l2(p.q + (q.gline + i) * 512 + (k & 7) * 64);
        }
      }
      if (t + 1 < g.end) next = look(t + 1);   // while this tile's copies are on their way
    }
  }
  if constexpr (!kV) publish(SegRecord{});
  leave(n, 0);
}

// Leader, one thread of warps 1 and 3: the MMAs of both CTAs.  kPv false: S = Q K^T
// of every tile; kPv true: O += P V.  A thread of its own for each, on its own
// scheduler: beside four softmax warps one alone issues an MMA in 94 to 128
// clocks, where the tensor cores take 64.
template <bool kPv>
__device__ __forceinline__ void issue_mmas(const ChunkParams& p, Ctl* ctl, uint32_t q0, uint32_t p0, uint32_t block0,
                                           uint32_t tmem, Walk w) {
  const uint32_t a0 = desc_low(kPv ? p0 : q0);
  uint32_t n = 0, nq = 0;            // tiles issued, segments
  bool ok = true;
  Segment g;
  while (ok && next_segment(p, w, g)) {
    if (!kPv) ok = wait_one(ctl, &ctl->qready, nq & 1, p);
    ++nq;
    for (int t = g.begin; t < g.end && ok; ++t, ++n) {
      const uint32_t par = n & 1, phase = (n >> 1) & 1;
      const uint32_t b0 = desc_low(block0) + (kPv ? 4096u : 0u);
      if (!kPv && n >= 2) ok = wait_one(ctl, &ctl->sfree[par], phase ^ 1, p);
      const uint32_t s = tmem + kSCol + par * 128;
      const uint32_t add = t == g.begin ? 0u : 1u;
      if constexpr (!kPv) {
#pragma unroll 1
        for (int i = 0; i < 4; ++i) {              // 128 dims
          ok = ok && wait_one(ctl, &ctl->kfull[i], par, p);
          if (!ok) break;
          tc_fence_after();
#pragma unroll
          for (int u = 0; u < 4; ++u)              // 32 dims
#pragma unroll
            for (int v = 0; v < 2; ++v)            // term
              mma_pair<idesc_f8(false, false)>(s, a0 + (v * 4 + i) * 512 + u * 2, b0 + i * 1024 + u * 2,
                                               (i | u | v) != 0 ? 1u : 0u);
          commit_pair(&ctl->kread[i]);
        }
        if (ok) commit_pair(&ctl->sfull[par]);
      } else {
        if (g.q.ctx + g.item * kItem / p.heads + 1 < (t + 1) * kTile) {
          // Softmax warps of either CTA may have to rewrite this V, see there.
          for (int v = 0; v < 4; ++v) ok = ok && wait_one(ctl, &ctl->vfull[v], par, p);
          if (!ok) break;
          commit_pair(&ctl->vseen);
        }
#pragma unroll 1
        for (int h = 0; h < 2; ++h) {              // 128 tokens
          ok = ok && wait_one(ctl, &ctl->vfull[2 * h], par, p) && wait_one(ctl, &ctl->vfull[2 * h + 1], par, p) &&
               wait_one(ctl, &ctl->pready[h], par, p);
          if (!ok) break;
          tc_fence_after();
#pragma unroll 1
          for (int u = 0; u < 4; ++u)              // 32 tokens
#pragma unroll
            for (int v = 0; v < 4; ++v) {          // term v / 2, 128 dims v % 2
              const uint32_t a = a0 + (v >> 1) * 1024 + h * 512 + u * 2;
              const uint32_t b = b0 + (2 * h + (v & 1)) * 1024 + u * 256;
              if (v < 2) mma_pair<idesc_f8(false, true)>(tmem + (v & 1) * 128, a, b, (h | u) == 0 ? add : 1u);
              else mma_pair<idesc_f8(true, true)>(tmem + (v & 1) * 128, a, b, 1u);
            }
          commit_pair(&ctl->vread[2 * par + h]);
        }
      }
    }
  }
  // Every MMA is complete before tensor memory is released.
  asm volatile(
      "tcgen05.commit.cta_group::2.mbarrier::arrive::one.shared::cluster.b64 [%0];" ::"r"(smem_u32(&ctl->drain[kPv]))
      : "memory");
  mbar_wait(&ctl->drain[kPv], 0, kDrainWaitNs);
}

// This warp's lines of Q in registers: lines w, w + 16, ... of warp w, dims 16l ..
// 16l + 15 in lane l.  Lines past the request's last are zero.
constexpr int kPer = kLines / kSoftmaxWarps;
__device__ __forceinline__ void load_q(const ChunkParams& p, int64_t gline, int lines, int sw, int lane, uint4 (&qa)[kPer],
                                       uint4 (&qb)[kPer]) {
#pragma unroll
  for (int j = 0; j < kPer; ++j) {
    const int i = sw + j * kSoftmaxWarps;
    qa[j] = qb[j] = make_uint4(0, 0, 0, 0);
    if (i < lines) {
      const uint4* src = reinterpret_cast<const uint4*>(p.q + (gline + i) * 512 + lane * 16);
      qa[j] = ld_dep_u4(src);
      qb[j] = ld_dep_u4(src + 1);
    }
  }
}
// Q of the segment's lines of this CTA: q * 2^s = hi + lo, s a power of two a line
// that puts its largest |q| in [128, 256), negated where the logits' scale is
// negative (so that it never is in the softmax).
__device__ __forceinline__ void convert_q(const ChunkParams& p, Ctl* ctl, uint8_t* qop, const uint4 (&qa)[kPer],
                                          const uint4 (&qb)[kPer], int sw, int lane) {
  const float sz = p.sm_scale * p.kv_scale * 1.4426950408889634f;
#pragma unroll
  for (int j = 0; j < kPer; ++j) {
    const int i = sw + j * kSoftmaxWarps;
    const uint32_t w[8] = {qa[j].x, qa[j].y, qa[j].z, qa[j].w, qb[j].x, qb[j].y, qb[j].z, qb[j].w};
    // |q| as an integer orders as |q| does, infinities and NaN on top.
    uint32_t top = w[0] & 0x7FFF7FFFu;
#pragma unroll
    for (int k = 1; k < 8; ++k) top = __vmaxu2(top, w[k] & 0x7FFF7FFFu);
    const uint32_t bits = __reduce_max_sync(0xFFFFFFFFu, max(top >> 16, top & 0xFFFFu)) << 16;
    const bool finite = bits < 0x7F800000u;
    // amax < 2^(field - 126); 2^sh puts it in [128, 256)
    const int sh = finite ? min(126, 134 - static_cast<int>(bits >> 23)) : 0;
    // A line with an infinity or a NaN gives NaN logits, as its formula does: by its
    // operand, so that one that sees no token has none.
    const float scale = finite ? copysignf(__uint_as_float(static_cast<uint32_t>(127 + sh) << 23), sz) : NAN;
    if (lane == 0) {
      // Never 0, which times a masked -inf would be NaN.
      float f = fabsf(sz) * __uint_as_float(static_cast<uint32_t>(127 - sh) << 23);
      if (f < 1e-37f) f = 1e-37f;
      ctl->qexp[i] = f;
    }
    uint32_t hw[4], lw[4];
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      uint16_t hc[2], lc[2];
#pragma unroll
      for (int u = 0; u < 2; ++u) {
        const uint32_t x = w[2 * k + u];
        const float2 f = fma2(make_float2(__uint_as_float(x << 16), __uint_as_float(x & 0xFFFF0000u)),
                              make_float2(scale, scale), make_float2(-0.0f, -0.0f));
        split_q(pack_f16(f.x, f.y), hc[u], lc[u]);
      }
      hw[k] = static_cast<uint32_t>(hc[0]) | (static_cast<uint32_t>(hc[1]) << 16);
      lw[k] = static_cast<uint32_t>(lc[0]) | (static_cast<uint32_t>(lc[1]) << 16);
    }
    uint8_t* row = qop + (lane >> 3) * 8192 + i * 128 + (((lane & 7) ^ (i & 7)) * 16);
    *reinterpret_cast<uint4*>(row) = make_uint4(hw[0], hw[1], hw[2], hw[3]);
    *reinterpret_cast<uint4*>(row + 32768) = make_uint4(lw[0], lw[1], lw[2], lw[3]);
  }
}

// Softmax, and everything else that is not a copy or an MMA.  A thread has one
// line: lane i and lane 64 + i of tensor memory hold its logits of the tile's
// first and second 128 tokens (its output's first and second 256 dims), and four
// warps share a quarter of the lanes, so eight threads have a line.
// The warps pass the same barriers in the same order whatever happens: after a
// wait that gave up they go on with what there is, without telling the MMAs.
__device__ __forceinline__ void softmax(const CUtensorMap& omap, const ChunkParams& p, Ctl* ctl, uint8_t* qop,
                                        uint8_t* pop, uint8_t* blocks, uint32_t tmem, int warp, int lane,
                                        uint32_t rank, int pair) {
  const int sw = warp - kSoftmaxWarp0, quarter = warp & 3, sub = sw >> 2;
  const int half = quarter >> 1, group = quarter & 1;
  const int i = group * 32 + lane;                      // line of this CTA
  const int part = half * 4 + sub;
  const uint32_t lane_base = static_cast<uint32_t>(quarter * 32) << 16;
  const uint32_t ocol = tmem + lane_base + sub * 64;    // this thread's 64 output columns
  const uint32_t scol = tmem + lane_base + kSCol + sub * kTok;
  const uint32_t sfree0 = map_to(&ctl->sfree[0], 0), sfree1 = map_to(&ctl->sfree[1], 0);
  const uint32_t pready = map_to(&ctl->pready[half], 0), qready = map_to(&ctl->qready, 0);
  uint8_t* const prow = pop + half * 8192 + i * 128;
  // O of tile n is complete.  A warp that waits for tile n has seen the first half
  // of n - 1 complete, so n - 2, the phase before on n's barrier, is.
  auto wait_o = [&](uint32_t n) { return wait_all(ctl, &ctl->vread[2 * (n & 1) + 1], (n >> 1) & 1, lane, p); };
  uint32_t ns = 0, nv = 0, seg = 0;                     // tiles, masked tiles, segments done
  bool ok = true;
  // The next segment's Q, loaded before the warps meet.  One warp's view of whether
  // there is one is everyone's.
  auto next_q = [&]() {
    const bool there = wait_segment(ctl, seg, lane, p);
    const SegRecord& r = ctl->seg[seg % kSegs];
    const bool some = there && r.end > r.begin;
    const int own = cta_lines(r.lines), before = static_cast<int>(rank) * own;
    uint4 qa[kPer], qb[kPer];
    load_q(p, r.gline + before, some ? min(own, r.lines - before) : 0, sw, lane, qa, qb);
    if (sw == 0 && lane == 0) ctl->more = some ? 1 : 0;
    softmax_sync();
    const bool go = *reinterpret_cast<volatile int*>(&ctl->more) != 0;
    if (go) {
      convert_q(p, ctl, qop, qa, qb, sw, lane);
      fence_proxy_async_smem();
      __syncwarp();
      if (lane == 0 && ok) arrive_at(qready);
    }
    return go;
  };
  bool more = next_q();
  softmax_sync();                                       // qexp
  while (more) {
    const SegRecord& g = ctl->seg[seg % kSegs];
    const float scale = ctl->qexp[i];
    const int first_tile = g.begin, tiles = g.end - g.begin;
    const int in = min(static_cast<int>(rank) * cta_lines(g.lines) + i, g.lines - 1);
    // tokens that this line sees of this thread's, and that every line of the item sees, from the tile on
    int visible = g.ctx + (g.first + in) / p.heads + 1 - (first_tile * kTile + half * 128 + sub * kTok);
    int all_see = g.ctx + g.first / p.heads + 1 - first_tile * kTile;
    float m = -INFINITY, l = 0.0f;
    for (int t = 0; t < tiles; ++t, ++ns, visible -= kTile, all_see -= kTile) {
      const uint32_t b = ns & 1;
      float z[kTok];
      ok = ok && wait_all(ctl, &ctl->sfull[b], (ns >> 1) & 1, lane, p);
      tc_fence_after();
      // This warp has none of the item's lines: it only keeps step, as P of the tile
      // before has to be complete before its part of this one is.
      if (group == 1 && g.lines <= kLines) {
        if (lane == 0 && ok) arrive_at(b ? sfree1 : sfree0);
        if (all_see < kTile) ++nv;
        if (ns > 0) ok = ok && wait_all(ctl, &ctl->vread[2 * ((ns - 1) & 1) + half], ((ns - 1) >> 1) & 1, lane, p);
        if (t == 0) {
          // Zeros, which take less power than what is there (32 decodes at 64 heads, at
          // the power limit: 141 -> 137 us).  The output that left through here first.
          if (lane == 0) tma_store_read();
          line_sync(group);
#pragma unroll
          for (int k = 0; k < 2; ++k) {
            const int at = ((sub * 2 + k) ^ (i & 7)) * 16;
            *reinterpret_cast<uint4*>(prow + at) = make_uint4(0, 0, 0, 0);
            *reinterpret_cast<uint4*>(prow + 16384 + at) = make_uint4(0, 0, 0, 0);
          }
          fence_proxy_async_smem();
          __syncwarp();
        }
        if (lane == 0 && ok) arrive_at(pready);
        continue;
      }
      tmem_load32(scol + b * 128, z);
      tc_fence_before();
      if (lane == 0 && ok) arrive_at(b ? sfree1 : sfree0);
      // Left before the tile's copies began, which S waited for.
      const uint32_t tag = *reinterpret_cast<volatile uint32_t*>(&ctl->tag[ns % kMasks]);
      uint32_t seen = visible >= kTok ? ~0u : visible <= 0 ? 0u : (1u << visible) - 1u;
      if (tag != 2 * (ns + 1) + 1) {
        __threadfence_block();
        seen &= ctl->mask[ns % kMasks][part];
      }
      const int from = max(0, all_see);                 // the tile's tokens from here on are hidden from some line
      bool nan = false;                                 // one of them has a NaN logit
      if (from < kTile || seen != ~0u) {
        const int hidden = from - (half * 128 + sub * kTok);
#pragma unroll
        for (int k = 0; k < kTok; ++k) {
          nan |= k >= hidden && z[k] != z[k];
          z[k] = (seen >> k) & 1u ? z[k] : -INFINITY;
        }
      }
      float mk[4] = {z[0], z[1], z[2], z[3]};
#pragma unroll
      for (int k = 4; k < kTok; k += 8)
#pragma unroll
        for (int u = 0; u < 4; ++u) mk[u] = fmaxf(fmaxf(mk[u], z[k + u]), k + 4 + u < kTok ? z[k + 4 + u] : -INFINITY);
      float mx = fmaxf(fmaxf(mk[0], mk[1]), fmaxf(mk[2], mk[3])) * scale;
      // The output that left through this warp's share of P has been read, before
      // any of its eight warps writes weights there.
      if (t == 0 && lane == 0) tma_store_read();
      if (line_sync_or(group, mx > m + kPMaxLog2)) {
        ctl->red[part][i] = mx;
        line_sync(group);
        float tm = ctl->red[0][i];
#pragma unroll
        for (int k = 1; k < 8; ++k) tm = fmaxf(tm, ctl->red[k][i]);
        float alpha = 1.0f;
        if (tm > m + kPMaxLog2) {
          alpha = ex2(m - tm);                          // 0 while nothing was added
          m = tm;
          l *= alpha;
        }
        if (t > 0 && __any_sync(0xFFFFFFFFu, alpha != 1.0f)) {
          ok = ok && wait_o(ns - 1);
          tc_fence_after();
#pragma unroll 1
          for (int k = 0; k < 64; k += 32) {
            float v[32];
            tmem_load32(ocol + k, v);
#pragma unroll
            for (int d = 0; d < 32; ++d) v[d] *= alpha;
            tmem_store16(ocol + k, v);
            tmem_store16(ocol + k + 16, v + 16);
          }
          asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory");
        }
        line_sync(group);                               // red[] has been read
      }
      const float base = m == -INFINITY ? 0.0f : kPLog2 - m;  // nothing seen yet: every weight is 0
      float2 sum[2] = {{0.0f, 0.0f}, {0.0f, 0.0f}};     // of the tile first: a long tail of small weights
      uint32_t hw[kTok / 4], lw[kTok / 4];              // would be rounded away against a large running sum
      auto weigh = [&](uint32_t vary, uint32_t same) {
#pragma unroll
        for (int k = 0; k < kTok / 4; ++k) {
          uint16_t hc[2];
          uint32_t lc[2];
#pragma unroll
          for (int u = 0; u < 2; ++u) {
            const float2 x = fma2(make_float2(z[4 * k + 2 * u], z[4 * k + 2 * u + 1]), make_float2(scale, scale),
                                  make_float2(base, base));
            const float2 e = make_float2(ex2(x.x), ex2(x.y));
            sum[u].x += e.x;
            sum[u].y += e.y;
            hc[u] = split_weights(pack_f16(e.x, e.y), (dither_of(4 * k + 2 * u) & vary) ^ same, lc[u]);
          }
          hw[k] = static_cast<uint32_t>(hc[0]) | (static_cast<uint32_t>(hc[1]) << 16);
          lw[k] = __byte_perm(lc[0], lc[1], 0x7531);
        }
      };
      // Half a step added in the rounding; or, of the dither, what a token's tile and
      // the eight threads of a line differ in.  (Two copies, as the dither's steps slow
      // the warps that gather beside these: a ragged batch in pages of 20 took 203 us
      // with them alone, 200 so, 196 without.)
      const bool small = mx < m - kSmallLog2;
      if (__any_sync(0xFFFFFFFFu, small))
        weigh(small ? 0x00FF00FFu : 0u,
              small ? ((static_cast<uint32_t>(all_see >> 8) * 0x9Du & 0xFFu) ^ static_cast<uint32_t>(part)) * 0x00010001u
                    : 0x00800080u);
      else
        weigh(0u, 0x00800080u);
      l += (sum[0].x + sum[0].y) + (sum[1].x + sum[1].y);
      // This half of P has been read: the MMAs take the tile's first 128 tokens
      // first, so it is written again while those of the second half run.
      if (ns > 0) ok = ok && wait_all(ctl, &ctl->vread[2 * ((ns - 1) & 1) + half], ((ns - 1) >> 1) & 1, lane, p);
#pragma unroll
      for (int k = 0; k < 2; ++k) {
        const int at = ((sub * 2 + k) ^ (i & 7)) * 16;
        *reinterpret_cast<uint4*>(prow + at) = make_uint4(hw[4 * k], hw[4 * k + 1], hw[4 * k + 2], hw[4 * k + 3]);
        *reinterpret_cast<uint4*>(prow + 16384 + at) =
            make_uint4(lw[4 * k], lw[4 * k + 1], lw[4 * k + 2], lw[4 * k + 3]);
      }
      // A token that some line of the item does not see has weight 0 there, which
      // a NaN latent would turn into NaN.  Such a latent shows as a NaN logit of
      // every line of both CTAs; its codes are then zeroed in V (a line that sees
      // it has a NaN weight, so its output is NaN all the same).  The thread that
      // issues the O of the tile, whose barriers say when V has landed in both CTAs,
      // tells both in every such tile.
      if (from < kTile) {
        const bool patch = line_sync_or(group, nan);
        if (patch) {
          ok = ok && warp_wait(ctl, &ctl->vseen, nv & 1, lane, p);
          acquire_cluster();
        }
        ++nv;
        if (patch) {
          for (int v = from / 128 * 2; v < 4; ++v) {    // block: 128 tokens x 128 dims
            const int r0 = max(0, from - (v >> 1) * 128), units = (128 - r0) * 8;
            uint4* rows = reinterpret_cast<uint4*>(blocks + (4 + v) * kBlockBytes) + r0 * 8;
            for (int u = part * 32 + lane; u < units; u += kSoftmaxThreads / 2) {
              const uint4 x = rows[u];
              const uint4 y = make_uint4(zero_nan4(x.x), zero_nan4(x.y), zero_nan4(x.z), zero_nan4(x.w));
              if (x.x != y.x || x.y != y.y || x.z != y.z || x.w != y.w) rows[u] = y;
            }
          }
          fence_proxy_async_smem();
          line_sync(group);                             // before the first half of P tells that V can be used
        }
      }
      fence_proxy_async_smem();
      tc_fence_before();
      __syncwarp();
      if (lane == 0 && ok) arrive_at(pready);
    }

    // Every S of the segment is complete: the next one's Q takes its place
    // while the last P V runs, and its first S runs beside the epilogue.
    const bool whole = g.whole != 0;
    const int own = cta_lines(g.lines), before = static_cast<int>(rank) * own;
    const int64_t gline0 = g.gline + before;
    const int lines = min(own, g.lines - before);       // of this CTA
    const bool idle = group * 32 >= lines;
    const int parts = g.parts, item_lines = min(kItem, g.lines);
    ctl->red[part][i] = l;
    ++seg;
    more = next_q();                                    // (and: l; qexp has been read)
    // The line's sum in a fixed order, then its output.
    float lt = ctl->red[0][i];
#pragma unroll
    for (int k = 1; k < 8; ++k) lt += ctl->red[k][i];
    softmax_sync();                                     // red[] has been read; the next qexp is there
    ok = ok && wait_o(ns - 1);
    tc_fence_after();
    const int d0 = half * 256 + sub * 64;
    if (idle) {                                         // (nothing to leave)
    } else if (whole) {
      const float inv = m != -INFINITY ? p.kv_scale / lt : (lt != lt ? lt : 0.0f);
      // Through 2 KB of this warp's share of P, 32 lines x 32 dims at a time:
      // rows of 64 bytes, swizzled, which a copy then writes in whole sectors.
      uint8_t* const stage = pop + (part >> 1) * 8192 + group * 4096 + (part & 1) * 2048;
      const bool box = ok && group * 32 + 31 < lines;
#pragma unroll 1
      for (int k = 0; k < 64; k += 32) {
        float v[32];
        tmem_load32(ocol + k, v);
        uint4 o[4];
        uint32_t* ow = reinterpret_cast<uint32_t*>(o);
#pragma unroll
        for (int d = 0; d < 16; ++d)
          asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(ow[d]) : "f"(v[2 * d + 1] * inv), "f"(v[2 * d] * inv));
        if (box) {
          if (k > 0) {
            if (lane == 0) tma_store_read();
            __syncwarp();
          }
#pragma unroll
          for (int d = 0; d < 4; ++d)
            *reinterpret_cast<uint4*>(stage + lane * 64 + ((d ^ ((lane >> 1) & 3)) * 16)) = o[d];
          fence_proxy_async_smem();
          __syncwarp();
          if (lane == 0) tma_store(&omap, smem_u32(stage), d0 + k, static_cast<int32_t>(gline0 + group * 32));
        } else if (ok && i < lines) {
          uint4* dst = reinterpret_cast<uint4*>(p.out + (gline0 + i) * 512 + d0 + k);
#pragma unroll
          for (int d = 0; d < 4; ++d) dst[d] = o[d];
        }
        __syncwarp();
      }
      if (ok && part == 0 && i < lines && p.lse != nullptr)
        p.lse[gline0 + i] = lt != 0.0f ? (m + log2f(lt * kPUnit)) * 0.69314718055994531f : -INFINITY;
    } else {
      // Slot 0: the item began in an earlier range, 1: it goes on in a later one.
      // [128 groups of 4 dims][128 lines][4]: a warp's lines side by side.
      const int slot = first_tile > 0 ? 0 : 1, pline = before + i;
      float4* dst = reinterpret_cast<float4*>(p.part_o) +
                    ((static_cast<int64_t>(pair) * 2 + slot) * 128 + d0 / 4) * kItem + pline;
#pragma unroll 1
      for (int k = 0; k < 64; k += 32) {
        float v[32];
        tmem_load32(ocol + k, v);
#pragma unroll
        for (int d = 0; d < 8; ++d)
          dst[(k / 4 + d) * kItem] = make_float4(v[4 * d], v[4 * d + 1], v[4 * d + 2], v[4 * d + 3]);
      }
      if (part == 0)
        reinterpret_cast<float2*>(p.part_ml)[(static_cast<int64_t>(pair) * 2 + slot) * kItem + pline] = make_float2(m, lt);
      if (slot == 1 && rank == 0 && sw == 0 && lane == 0) p.records[pair] = ChunkRecord{gline0, item_lines, parts};
    }
    tc_fence_before();
    __syncwarp();
  }
  if (lane == 0) tma_store_done();
}

// kGather: pages whose size no box of 8 tokens or more divides.  A kernel of its
// own, as what a copying warp runs between a block's release and its next copy
// counts, fetches of instructions included: as one kernel, a prompt of 1,024 rows
// took 702 us instead of 693, 32 decodes 146 instead of 142, a ragged batch in
// pages of 20 211 instead of 205.
template <bool kGather>
__global__ void __cluster_dims__(2, 1, 1) __launch_bounds__(kThreads, 1)
    mla_chunk_kernel(const __grid_constant__ CUtensorMap map, const __grid_constant__ CUtensorMap map16,
                     const __grid_constant__ CUtensorMap omap, const ChunkParams p) {
  extern __shared__ __align__(1024) uint8_t smem_raw[];
  uint8_t* smem = smem_raw;           // (no static shared memory: it begins on a 1024-byte boundary)
  uint8_t* qop = smem;
  uint8_t* pop = smem + kQBytes;
  uint8_t* blocks = smem + kBlockOff;
  Ctl* ctl = reinterpret_cast<Ctl*>(smem + kCtlOff);
  const int tid = threadIdx.x, warp = __shfl_sync(0xFFFFFFFFu, tid >> 5, 0), lane = tid & 31;
  const uint32_t rank = cta_rank();
  const int pair = blockIdx.x >> 1;

  if (tid == 0) {
    for (int k = 0; k < 4; ++k) {
      mbar_init(&ctl->kfull[k], 1);
      mbar_init(&ctl->vfull[k], 1);
      mbar_init(&ctl->kread[k], 1);
      mbar_init(&ctl->vread[k], 1);
    }
    for (int k = 0; k < kBlocks; ++k) ctl->fills[k] = 0;
    for (int k = 0; k < 2; ++k) {
      mbar_init(&ctl->sfull[k], 1);
      mbar_init(&ctl->sfree[k], 2 * kSoftmaxWarps);
      mbar_init(&ctl->pready[k], kSoftmaxWarps);
      mbar_init(&ctl->drain[k], 1);
    }
    mbar_init(&ctl->qready, 2 * kSoftmaxWarps);
    mbar_init(&ctl->vseen, 1);
    for (int k = 0; k < kMasks; ++k) ctl->tag[k] = 0;
    ctl->abort_flag = 0;
    ctl->begun = 0;
    ctl->segs = 0;
    fence_mbar_init();
    tma_prefetch_map(&map);
    tma_prefetch_map(&omap);
    if (kGather) tma_prefetch_map(&map16);
  }
  if (warp == 1) {
    asm volatile("tcgen05.alloc.cta_group::2.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(smem_u32(&ctl->tmem_base)),
                 "r"(kTmemCols)
                 : "memory");
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::2.sync.aligned;" ::: "memory");
  }
  grid_dep_launch();
  grid_dep_wait();    // lengths, tables, latents and q come from kernels before
  const Place at = find_place<kThreads>(p, p.pairs, [&](int64_t per) { return per * pair; },
                                        reinterpret_cast<int64_t*>(smem), blockIdx.x == 0);
  Walk w;
  if (rank == 0 && tid == 0) p.records[pair].parts = 0;  // until an item begins in this range and goes on
  w.seq = at.seq;
  w.item = at.item;
  w.off = at.off;
  w.left = at.seq < 0 ? 0 : min(at.per, at.total - at.per * pair);
  tc_fence_before();
  cluster_sync();     // barriers, tensor memory address; the scratch is free
  tc_fence_after();
  const uint32_t tmem = ctl->tmem_base;

  if (warp == 0) {
    copy<false, kGather>(map, map16, p, ctl, blocks, lane, rank, pair, at.per, w);
  } else if (warp == 1 || warp == 3) {
    if (rank == 0 && elect_one()) {
      if (warp == 1) issue_mmas<false>(p, ctl, smem_u32(qop), smem_u32(pop), smem_u32(blocks), tmem, w);
      else issue_mmas<true>(p, ctl, smem_u32(qop), smem_u32(pop), smem_u32(blocks), tmem, w);
    }
    __syncwarp();
  } else if (warp == 2) {
    copy<true, kGather>(map, map16, p, ctl, blocks, lane, rank, pair, at.per, w);
  } else if (warp >= kSoftmaxWarp0) {
    softmax(omap, p, ctl, qop, pop, blocks, tmem, warp, lane, rank, pair);
  }

  tc_fence_before();
  __syncthreads();
  if (rank == 1 && tid < kBlocks)
    asm volatile("st.shared::cluster.u16 [%0], %1;" ::"r"(map_to(&ctl->peer_fills[tid], 0)), "h"(ctl->fills[tid]) : "memory");
  cluster_sync();     // neither CTA leaves while the other may still signal it
  // Nor with a copy of either in flight.  All are complete unless a wait gave up
  // (which both know by now); then one CTA may have begun a block's copies that the
  // other has not, and the bytes that will not come are made up for.
  if (aborted(ctl)) {
    if (rank == 0 && tid < kBlocks) {
      uint64_t* const full = tid < 4 ? &ctl->kfull[tid] : &ctl->vfull[tid - 4];
      const uint16_t mine = ctl->fills[tid], other = ctl->peer_fills[tid];
      const int ahead = (mine - other) & 3;                   // 1, 0 or 3: one behind
      const uint32_t n = ahead == 3 ? other : mine;
      if (ahead == 1)
        asm volatile("mbarrier.complete_tx.relaxed.cluster.shared::cta.b64 [%0], %1;" ::"r"(smem_u32(full)), "r"(kBlockBytes) : "memory");
      else if (ahead == 3)
        mbar_arrive_expect_tx(full, kBlockBytes);
      if (n > 0) mbar_wait(full, (n - 1) & 1, kDrainWaitNs);
    }
    __syncthreads();
    cluster_sync();
  }
  if (warp == 1) {
    tc_fence_after();
    asm volatile("tcgen05.dealloc.cta_group::2.sync.aligned.b32 %0, %1;" ::"r"(tmem), "r"(kTmemCols) : "memory");
  }
}

// Adds up the parts of the items that several ranges share.  Few parts: a
// thread has a line and kDims groups of 4 dims, and adds the parts in order.
template <int kDims>
__device__ __forceinline__ void merge_few(const ChunkParams& p, const ChunkRecord& r, int first, int line, int d4) {
  if (line >= r.lines) return;
  // part 0 in slot 1 of its pair, the others in slot 0 of theirs
  auto slot = [&](int u) { return static_cast<int64_t>(first + u) * 2 + (u == 0 ? 1 : 0); };
  const float2* ml = reinterpret_cast<const float2*>(p.part_ml) + line;
  const float4* o = reinterpret_cast<const float4*>(p.part_o) + static_cast<int64_t>(d4) * kItem + line;
  float m = -INFINITY, l = 0.0f;
  float4 acc[kDims];
#pragma unroll
  for (int d = 0; d < kDims; ++d) acc[d] = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
  for (int u0 = 0; u0 < r.parts; u0 += 2) {             // two in flight
    float2 x[2];
    float4 v[2][kDims];
#pragma unroll
    for (int k = 0; k < 2; ++k) {
      const int u = min(u0 + k, r.parts - 1);
      x[k] = ld_dep_f2(ml + slot(u) * kItem);
      if (u0 + k >= r.parts) x[k] = make_float2(-INFINITY, 0.0f);
#pragma unroll
      for (int d = 0; d < kDims; ++d) v[k][d] = ld_dep_f4(o + (slot(u) * 128 + d) * kItem);
    }
    const float top = fmaxf(m, fmaxf(x[0].x, x[1].x));
    const float base = top == -INFINITY ? 0.0f : top;   // (no weight yet: 0 times a sum that may be NaN)
    const float a = ex2(m - base), w0 = ex2(x[0].x - base), w1 = ex2(x[1].x - base);
    m = top;
    l = l * a + w0 * x[0].y + w1 * x[1].y;
#pragma unroll
    for (int d = 0; d < kDims; ++d) {
      acc[d].x = acc[d].x * a + w0 * v[0][d].x + w1 * v[1][d].x;
      acc[d].y = acc[d].y * a + w0 * v[0][d].y + w1 * v[1][d].y;
      acc[d].z = acc[d].z * a + w0 * v[0][d].z + w1 * v[1][d].z;
      acc[d].w = acc[d].w * a + w0 * v[0][d].w + w1 * v[1][d].w;
    }
  }
  const float inv = l != l ? l : (m != -INFINITY ? p.kv_scale / l : 0.0f);
  const int64_t gline = r.line0 + line;
  uint4* out = reinterpret_cast<uint4*>(p.out + gline * 512 + d4 * 4);
#pragma unroll
  for (int d = 0; d < kDims; d += 2) {
    uint32_t w[4];
#pragma unroll
    for (int k = 0; k < 2; ++k) {
      asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(w[2 * k]) : "f"(acc[d + k].y * inv), "f"(acc[d + k].x * inv));
      asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(w[2 * k + 1]) : "f"(acc[d + k].w * inv), "f"(acc[d + k].z * inv));
    }
    out[d / 2] = make_uint4(w[0], w[1], w[2], w[3]);
  }
  if (d4 == 0 && p.lse != nullptr)
    p.lse[gline] = l != 0.0f ? (m + log2f(l * kPUnit)) * 0.69314718055994531f : -INFINITY;
}

// Many parts: four threads have a line and 4 dims and take every fourth part,
// sixteen in flight, then are added up in order.
__device__ __forceinline__ void merge_many(const ChunkParams& p, const ChunkRecord& r, int first, int half, int d4,
                                           float4 (&x_acc)[3][64], float2 (&x_ml)[3][64]) {
  constexpr int kBatch = 16;
  const int i = threadIdx.x & 63, set = threadIdx.x >> 6, line = half * 64 + i;
  auto slot = [&](int u) { return static_cast<int64_t>(first + u) * 2 + (u == 0 ? 1 : 0); };
  const float2* ml = reinterpret_cast<const float2*>(p.part_ml) + line;
  const float4* o = reinterpret_cast<const float4*>(p.part_o) + static_cast<int64_t>(d4) * kItem + line;
  float m = -INFINITY, l = 0.0f;
  float4 acc = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
  auto add = [&](float mk, float lk, float4 v, float base) {
    const float w = ex2(mk - base);
    l += w * lk;
    acc.x += w * v.x;
    acc.y += w * v.y;
    acc.z += w * v.z;
    acc.w += w * v.w;
  };
  auto scale_by = [&](float a) {
    l *= a;
    acc.x *= a;
    acc.y *= a;
    acc.z *= a;
    acc.w *= a;
  };
  for (int u0 = set; u0 < r.parts; u0 += 4 * kBatch) {
    float2 x[kBatch];
    float4 v[kBatch];
#pragma unroll
    for (int k = 0; k < kBatch; ++k) {
      x[k] = make_float2(-INFINITY, 0.0f);
      v[k] = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
      const int u = u0 + 4 * k;
      if (u < r.parts) {
        x[k] = ld_dep_f2(ml + slot(u) * kItem);
        v[k] = ld_dep_f4(o + slot(u) * 128 * kItem);
      }
    }
    float top = m;
#pragma unroll
    for (int k = 0; k < kBatch; ++k) top = fmaxf(top, x[k].x);
    const float base = top == -INFINITY ? 0.0f : top;   // (no weight yet: 0 times a sum that may be NaN)
    scale_by(ex2(m - base));
    m = top;
#pragma unroll
    for (int k = 0; k < kBatch; ++k) add(x[k].x, x[k].y, v[k], base);
  }
  __syncthreads();                                      // the unit before has been read
  if (set > 0) {
    x_ml[set - 1][i] = make_float2(m, l);
    x_acc[set - 1][i] = acc;
  }
  __syncthreads();
  if (set > 0 || line >= r.lines) return;
  float top = m;
#pragma unroll
  for (int k = 0; k < 3; ++k) top = fmaxf(top, x_ml[k][i].x);
  const float base = top == -INFINITY ? 0.0f : top;
  scale_by(ex2(m - base));
#pragma unroll
  for (int k = 0; k < 3; ++k) add(x_ml[k][i].x, x_ml[k][i].y, x_acc[k][i], base);
  const float inv = l != l ? l : (top != -INFINITY ? p.kv_scale / l : 0.0f);
  const int64_t gline = r.line0 + line;
  uint32_t w[2];
  asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(w[0]) : "f"(acc.y * inv), "f"(acc.x * inv));
  asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(w[1]) : "f"(acc.w * inv), "f"(acc.z * inv));
  *reinterpret_cast<uint2*>(p.out + gline * 512 + d4 * 4) = make_uint2(w[0], w[1]);
  if (d4 == 0 && p.lse != nullptr)
    p.lse[gline] = l != 0.0f ? (top + log2f(l * kPUnit)) * 0.69314718055994531f : -INFINITY;
}

// CTAs take units of 64 lines in turn: 64 dims of an item with few parts, 4 of
// one with many (few items then, which have to reach every SM).  All as few: one
// decode at 32k, 64 parts, 22.5 -> 41 us a call; all as many: a prompt of 1,024
// rows, whose items have two parts or three, 686 -> 724, a ragged batch 200 -> 255.
__global__ void __launch_bounds__(kMergeThreads) mla_chunk_merge_kernel(const ChunkParams p) {
  constexpr int kFew = 8;
  __shared__ ChunkRecord rec[kMaxPairs];
  __shared__ int begin[kMaxPairs + 1];                  // first unit of each pair's record
  __shared__ float4 x_acc[3][64];
  __shared__ float2 x_ml[3][64];
  const int tid = threadIdx.x, lane = tid & 31;
  grid_dep_launch();
  grid_dep_wait();
  int units = 0;
  if (tid < p.pairs) {
    const ChunkRecord r = p.records[tid];
    rec[tid] = r;
    if (r.parts > 1) units = (r.lines > 64 ? 2 : 1) * (r.parts > kFew ? 128 : 8);
  }
  if (!__syncthreads_or(units)) return;
  begin[tid] = units;
  __syncthreads();
  if (tid < 32) {                                       // exclusive sums
    constexpr int kPer = kMaxPairs / 32;
    int mine = 0;
    for (int k = 0; k < kPer; ++k) mine += begin[lane * kPer + k];
    int x = mine;
    for (int o = 1; o < 32; o <<= 1) {
      const int y = __shfl_up_sync(0xFFFFFFFFu, x, o);
      if (lane >= o) x += y;
    }
    int at = x - mine;
    for (int k = 0; k < kPer; ++k) {
      const int v = begin[lane * kPer + k];
      begin[lane * kPer + k] = at;
      at += v;
    }
    if (lane == 31) begin[kMaxPairs] = at;
  }
  __syncthreads();
  for (int unit = blockIdx.x; unit < begin[kMaxPairs]; unit += gridDim.x) {
    int lo = 0, hi = kMaxPairs;                         // begin[lo] <= unit < begin[hi]
    while (hi - lo > 1) {
      const int mid = (lo + hi) >> 1;
      if (begin[mid] <= unit) lo = mid; else hi = mid;
    }
    const ChunkRecord r = rec[lo];
    const int at = unit - begin[lo];
    const int half = r.lines > 64 ? at & 1 : 0, d = r.lines > 64 ? at >> 1 : at;
    if (r.parts > kFew) merge_many(p, r, lo, half, d, x_acc, x_ml);
    else merge_few<4>(p, r, lo, half * 64 + (tid & 63), d * 16 + (tid >> 6) * 4);
  }
}

}  // namespace

// Two slots a pair: the part of an item that began before its range, and of one
// that goes on after it; their (max, sum); a record of the latter.
size_t mla_chunk_workspace_bytes(int pairs) {
  const size_t lines = static_cast<size_t>(pairs) * 2 * kItem;
  return lines * 512 * sizeof(float) + lines * 2 * sizeof(float) + pairs * sizeof(ChunkRecord);
}

// Token rows of one copy: the largest power of two, 64 at most, that divides
// the block.  A warp has a copy for each lane, so 8 rows at least for the tile's
// 256 tokens; below that the rows are gathered four at a time, or sixteen where
// they run on (a ragged batch in pages of 20: 362 us by fours alone, 274 so).
int mla_chunk_box_rows(int block_size) {
  int h = 64;
  while (block_size % h != 0) h >>= 1;
  return h >= 8 ? h : 0;
}

// What the host knows of the work: a call that can only have one tile (a first
// token at few heads) is one pair, with nothing to merge: 15.9 us become 14.6.
int mla_chunk_pairs(const dsa_seqs* seqs, int rows, int heads, int num_sms) {
  const int64_t items = static_cast<int64_t>(rows) * heads / kItem + (seqs->seqs < rows ? seqs->seqs : rows);
  const int64_t tiles = (static_cast<int64_t>(seqs->block_size) * seqs->max_blocks_per_seq + kTile - 1) / kTile;
  const int64_t pairs = num_sms / 2;
  return static_cast<int>(items * tiles < pairs ? items * tiles : pairs);
}

cudaError_t launch_mla_chunk(ChunkParams p, const CUtensorMap& map, const CUtensorMap& map16,
                             const CUtensorMap& omap, void* workspace, int num_sms, cudaStream_t stream) {
  if (p.pairs < 1 || p.pairs > kMaxPairs) return cudaErrorInvalidValue;
  const size_t lines = static_cast<size_t>(p.pairs) * 2 * kItem;
  p.part_o = static_cast<float*>(workspace);
  p.part_ml = p.part_o + lines * 512;
  p.records = reinterpret_cast<ChunkRecord*>(p.part_ml + lines * 2);
  auto kernel = p.box_rows > 0 ? mla_chunk_kernel<false> : mla_chunk_kernel<true>;
  cudaError_t e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                       static_cast<int>(kSmemBytes));
  if (e != cudaSuccess) return e;
  cudaLaunchAttribute attr[1] = {dependent_launch_attr()};
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(static_cast<unsigned>(2 * p.pairs), 1, 1);
  cfg.blockDim = dim3(kThreads, 1, 1);
  cfg.dynamicSmemBytes = kSmemBytes;
  cfg.stream = stream;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  e = cudaLaunchKernelEx(&cfg, kernel, map, map16, omap, p);
  if (e != cudaSuccess || p.pairs == 1) return e;
  cudaLaunchConfig_t mcfg = {};
  mcfg.gridDim = dim3(static_cast<unsigned>(2 * num_sms), 1, 1);
  mcfg.blockDim = dim3(kMergeThreads, 1, 1);
  mcfg.stream = stream;
  mcfg.attrs = attr;
  mcfg.numAttrs = 1;
  return cudaLaunchKernelEx(&mcfg, mla_chunk_merge_kernel, p);
}

}  // namespace dsa
