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
// Precision.  The latents stay E4M3.  q * 2^s = hi + lo, two E4M3 terms, holds
// a bf16 q exactly but for elements 2^10 below the head's largest; a softmax
// weight is an E4M3 term and the E5M2 term of its remainder (2^-7 of the weight
// at most, about 2^-9.6 rms; the second term's range keeps weights down to 2^-25
// of the largest, so that a long tail of small weights is not lost).  Two FP8
// terms cost what one 16-bit term would and need no conversion of the latents.
// Products, sums, maxima and the output are FP32.
#include <mutex>

#include "dsa_device.cuh"
#include "dsa_internal.h"

namespace dsa {
namespace {

constexpr int kThreads = 320;        // warp 0 copies, warp 1 MMA or forwards, warps 2-9 softmax
constexpr int kSoftmaxThreads = 256;
constexpr int kSoftmaxWarps = 8;
constexpr int kItem = 128;           // lines of an item (MMA M over the pair)
constexpr int kLines = 64;           // lines of a CTA
constexpr int kTile = 256;           // tokens of a tile
constexpr int kChunks = 8;           // ring of 16 KB: a tile's K is four of them, its V four
constexpr uint32_t kChunkBytes = 16384;
constexpr uint32_t kQBytes = 65536;  // [term][128-dim block][64 lines][128 B]
constexpr uint32_t kPBytes = 32768;  // [term][128-token half][64 lines][128 B]
constexpr uint32_t kRingOff = kQBytes + kPBytes;
constexpr uint32_t kCtlOff = kRingOff + kChunks * kChunkBytes;
constexpr uint32_t kTmemCols = 512;  // O: 0..255, S: 256 + 128 * buffer
constexpr uint32_t kSCol = 256;
constexpr int kMasks = 4;            // tiles whose token masks are kept
constexpr float kPMaxLog2 = 8.75f;   // a weight 2^(z - m) stays below 2^8.75 < 448
constexpr float kPResetLog2 = 8.0f;  // a new maximum maps to 2^8
constexpr int kMergeThreads = 256;
constexpr int kMergeLines = 8;       // lines of a merge CTA, a warp each

struct __align__(16) Ctl {
  uint64_t full[kChunks], empty[kChunks];
  uint64_t peer_full[kChunks];       // leader: the other CTA's copies have landed
  uint64_t sfull[2], sfree[2], mask_ready[kMasks];
  uint64_t pready, odone, qready, drain;
  uint64_t mask[kMasks][4];          // a bit for each token of a tile: there is a latent
  uint32_t tmem_base;
  int abort_flag;
  float qexp[kLines];
  float red[4][kLines];
};
constexpr uint32_t kSmemBytes = kCtlOff + sizeof(Ctl) + 1024;  // + alignment slack
static_assert(kSmemBytes + 64 <= 227 * 1024, "shared memory budget (and find_place's own)");

// ------------------------------------------------------------------ schedule
struct SeqInfo {
  int row0, rows, ctx, lines, items;
};

// Rows, lines and items of request s; no items where it has no rows or is
// refused (`why`: the error to record).
__device__ __forceinline__ SeqInfo seq_info(const ChunkParams& p, int s, int* why = nullptr) {
  SeqInfo q;
  q.row0 = p.seqs.row_start[s];
  const int64_t end = p.seqs.row_start[s + 1], len = p.seqs.seq_lens[s];
  const int64_t rows = end - q.row0;
  int bad = 0;
  if (rows > 0 && (q.row0 < 0 || end > p.rows)) bad = DSA_DEVERR_ROWS;
  else if (rows > 0 && (len < rows || len > static_cast<int64_t>(p.seqs.max_blocks_per_seq) * p.seqs.block_size))
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
  return (item_end(p, q, j) + kTile - 1) / kTile;
}
// How many of the request's items see at most x new tokens.
__device__ __forceinline__ int items_within(const ChunkParams& p, const SeqInfo& q, int x) {
  return x <= 0 ? 0 : x >= q.rows ? q.items : static_cast<int>(static_cast<int64_t>(x) * p.heads / kItem);
}
// All its tiles: items by their number of tiles v, those within v tiles less
// those within v - 1.
__device__ __forceinline__ int64_t seq_tiles(const ChunkParams& p, const SeqInfo& q) {
  if (q.items == 0) return 0;
  int64_t sum = 0;
  int below = 0;
  for (int v = (q.ctx + kTile) / kTile; below < q.items; ++v) {
    const int upto = items_within(p, q, static_cast<int>(min(static_cast<int64_t>(v) * kTile - q.ctx, static_cast<int64_t>(q.rows))));
    sum += static_cast<int64_t>(upto - below) * v;
    below = upto;
  }
  return sum;
}

struct Place {
  int64_t total;   // tiles of the call
  int64_t per;     // tiles of a pair
  int seq, item, tile;
};

// Finds tile `target(total)` of the call: every thread sums a run of requests,
// the CTA scans the sums, and the thread whose run holds it walks to it.
// `scratch`: kN + 2 int64 of shared memory.  Returns seq -1 past the end.
template <int kN, typename Target>
__device__ __forceinline__ Place find_place(const ChunkParams& p, int pairs, Target target,
                                            int64_t* scratch, bool report) {
  __shared__ Place found;
  const int tid = threadIdx.x, n = p.seqs.seqs, run = (n + kN - 1) / kN;
  const int s0 = min(n, tid * run), s1 = min(n, s0 + run);
  int64_t sum = 0;
  for (int s = s0; s < s1; ++s) {
    int why = 0;
    const SeqInfo q = seq_info(p, s, &why);
    if (why != 0 && report) record_error(p.err, why, s);
    sum += seq_tiles(p, q);
  }
  scratch[tid] = sum;
  if (tid == 0) found.seq = -1;
  __syncthreads();
  if (tid < 32) {
    constexpr int kPer = (kN + 31) / 32;
    int64_t mine = 0;
    for (int i = 0; i < kPer; ++i)
      if (tid * kPer + i < kN) mine += scratch[tid * kPer + i];
    int64_t x = mine;
    for (int o = 1; o < 32; o <<= 1) {
      const int64_t y = __shfl_up_sync(0xFFFFFFFFu, x, o);
      if (tid >= o) x += y;
    }
    int64_t at = x - mine;
    for (int i = 0; i < kPer; ++i)
      if (tid * kPer + i < kN) {
        const int64_t v = scratch[tid * kPer + i];
        scratch[tid * kPer + i] = at;
        at += v;
      }
    if (tid == 31) {
      found.total = x;
      found.per = max(static_cast<int64_t>(1), (x + pairs - 1) / pairs);
    }
  }
  __syncthreads();
  const int64_t want = target(found.per);
  int64_t at = scratch[tid];
  if (want < found.total && want >= at && want < at + sum) {
    for (int s = s0; s < s1; ++s) {
      const SeqInfo q = seq_info(p, s);
      const int64_t t = seq_tiles(p, q);
      if (want >= at + t) {
        at += t;
        continue;
      }
      int64_t off = want - at;
      int below = 0;
      for (int v = (q.ctx + kTile) / kTile;; ++v) {
        const int upto = items_within(p, q, static_cast<int>(min(static_cast<int64_t>(v) * kTile - q.ctx, static_cast<int64_t>(q.rows))));
        const int64_t here = static_cast<int64_t>(upto - below) * v;
        if (off < here) {
          found.seq = s;
          found.item = below + static_cast<int>(off / v);
          found.tile = static_cast<int>(off % v);
          break;
        }
        off -= here;
        below = upto;
      }
      break;
    }
  }
  __syncthreads();
  const Place out = found;
  __syncthreads();
  return out;
}

// The part of one item in a pair's range, and the walk over the range.
struct Segment {
  SeqInfo q;
  int seq, item, tiles;   // tiles: of the item
  int begin, end;         // tiles of the segment
};
struct Walk {
  int seq, item, begin;
  int64_t left;           // tiles
};
__device__ __forceinline__ bool next_segment(const ChunkParams& p, Walk& w, Segment& g) {
  if (w.left <= 0) return false;
  g.q = seq_info(p, w.seq);
  while (w.item >= g.q.items) {
    w.item = 0;
    w.begin = 0;
    if (++w.seq >= p.seqs.seqs) return false;
    g.q = seq_info(p, w.seq);
  }
  g.seq = w.seq;
  g.item = w.item;
  g.tiles = item_tiles(p, g.q, w.item);
  g.begin = w.begin;
  g.end = static_cast<int>(min(static_cast<int64_t>(g.tiles), w.begin + w.left));
  w.left -= g.end - g.begin;
  w.begin = 0;
  ++w.item;
  return true;
}

// ------------------------------------------------------------------ pair
__device__ __forceinline__ uint32_t cta_rank() {
  uint32_t r;
  asm volatile("mov.u32 %0, %%cluster_ctarank;" : "=r"(r));
  return r;
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
__device__ __forceinline__ void arrive_at(uint32_t bar) {
  asm volatile("mbarrier.arrive.release.cluster.shared::cluster.b64 _, [%0];" ::"r"(bar) : "memory");
}
__device__ __forceinline__ bool try_wait_cluster(uint64_t* bar, uint32_t parity) {
  uint32_t ok;
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "mbarrier.try_wait.parity.acquire.cluster.shared::cta.b64 p, [%1], %2, %3;\n\t"
      "selp.u32 %0, 1, 0, p;\n\t}"
      : "=r"(ok)
      : "r"(smem_u32(bar)), "r"(parity), "r"(32u)
      : "memory");
  return ok != 0;
}
__device__ __forceinline__ bool aborted(Ctl* c) {
  return *reinterpret_cast<volatile int*>(&c->abort_flag) != 0;
}
// Marks both CTAs of the pair: their later waits are skipped.
__device__ __forceinline__ void set_abort(Ctl* c) {
  for (uint32_t r = 0; r < 2; ++r)
    asm volatile("st.volatile.shared::cluster.u32 [%0], %1;" ::"r"(map_to(&c->abort_flag, r)), "r"(1) : "memory");
}
// Bounded wait of one thread; a timeout is recorded and marks the pair.
__device__ __forceinline__ bool wait_one(Ctl* c, uint64_t* bar, uint32_t parity, const ChunkParams& p) {
  if (p.wait_ns >= kShortWaitNs && try_wait_cluster(bar, parity)) return true;
  const uint64_t t0 = global_ns();
  for (uint32_t i = 1; i < (1u << 30); ++i) {
    if (try_wait_cluster(bar, parity)) return true;
    if ((i & 15u) == 0 || p.wait_ns < kShortWaitNs) {
      if (aborted(c)) return false;
      if (global_ns() - t0 > p.wait_ns) break;
    }
  }
  record_error(p.err, DSA_DEVERR_TIMEOUT, -1);
  set_abort(c);
  return false;
}
__device__ __forceinline__ bool warp_wait(Ctl* c, uint64_t* bar, uint32_t parity, int lane, const ChunkParams& p) {
  int ok = 1;
  if (lane == 0) ok = wait_one(c, bar, parity, p) ? 1 : 0;
  return __shfl_sync(0xFFFFFFFFu, ok, 0) != 0;
}

// ------------------------------------------------------------------ tensor core
__device__ __forceinline__ uint64_t desc_mnmajor(uint32_t saddr) {
  // 128 contiguous bytes of MN per K row, K rows 128 B apart, the next 8 of
  // them 1024 B on; a CTA's share of MN is one 128-byte span.
  return umma_desc_sw128_kmajor(saddr);
}
// kind::f8f6f4, F32 accumulate, M = 128 over the pair, N = 256; A E4M3 or E5M2
// K-major, B E4M3.
__host__ __device__ constexpr uint32_t idesc_f8(bool a_e5m2, bool b_mn_major) {
  return (1u << 4) | (a_e5m2 ? (1u << 7) : 0u) | (b_mn_major ? (1u << 16) : 0u) | ((256u >> 3) << 17) |
         ((128u >> 4) << 24);
}
__device__ __forceinline__ void mma_pair(uint32_t d, uint64_t a, uint64_t b, uint32_t idesc, uint32_t acc) {
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "setp.ne.b32 p, %4, 0;\n\t"
      "tcgen05.mma.cta_group::2.kind::f8f6f4 [%0], %1, %2, %3, p;\n\t}" ::"r"(d),
      "l"(a), "l"(b), "r"(idesc), "r"(acc)
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
// A box of the latent pool: 128 bytes (column x) of the rows from y on.
__device__ __forceinline__ void tma_box(uint32_t dst, const CUtensorMap* map, uint64_t* bar, int32_t x, int32_t y) {
  asm volatile(
      "cp.async.bulk.tensor.2d.shared::cluster.global.tile.mbarrier::complete_tx::bytes [%0], [%1, {%2, %3}], [%4];" ::"r"(dst),
      "l"(reinterpret_cast<uint64_t>(map)), "r"(x), "r"(y), "r"(smem_u32(bar))
      : "memory");
}
// Four rows of 128 bytes each.
__device__ __forceinline__ void tma_gather4(uint32_t dst, const CUtensorMap* map, uint64_t* bar, int32_t x,
                                            int32_t y0, int32_t y1, int32_t y2, int32_t y3) {
  asm volatile(
      "cp.async.bulk.tensor.2d.shared::cluster.global.tile::gather4.mbarrier::complete_tx::bytes"
      " [%0], [%1, {%2, %3, %4, %5, %6}], [%7];" ::"r"(dst),
      "l"(reinterpret_cast<uint64_t>(map)), "r"(x), "r"(y0), "r"(y1), "r"(y2), "r"(y3), "r"(smem_u32(bar))
      : "memory");
}

__device__ __forceinline__ uint16_t e4m3x2(float lo, float hi) {
  uint16_t out;
  asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(out) : "f"(hi), "f"(lo));
  return out;
}
__device__ __forceinline__ uint16_t e5m2x2(float lo, float hi) {
  uint16_t out;
  asm("cvt.rn.satfinite.e5m2x2.f32 %0, %1, %2;" : "=h"(out) : "f"(hi), "f"(lo));
  return out;
}
__device__ __forceinline__ float2 e4m3x2_decode(uint16_t codes) {
  uint32_t h2;
  asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(h2) : "h"(codes));
  return __half22float2(*reinterpret_cast<const __half2*>(&h2));
}
// The bytes of w that are E4M3 NaN codes, zeroed.
__device__ __forceinline__ uint32_t zero_nan4(uint32_t w) {
  const uint32_t nan = __vcmpeq4(w & 0x7F7F7F7Fu, 0x7F7F7F7Fu);
  return w & ~nan;
}

__device__ __forceinline__ void softmax_sync() {
  asm volatile("bar.sync 1, %0;" ::"n"(kSoftmaxThreads) : "memory");
}
__device__ __forceinline__ bool softmax_sync_or(bool pred) {
  uint32_t out;
  asm volatile(
      "{\n\t.reg .pred p, q;\n\t"
      "setp.ne.u32 p, %1, 0;\n\t"
      "bar.red.or.pred q, 1, %2, p;\n\t"
      "selp.u32 %0, 1, 0, q;\n\t}"
      : "=r"(out)
      : "r"(pred ? 1u : 0u), "n"(kSoftmaxThreads)
      : "memory");
  return out != 0;
}

// ------------------------------------------------------------------ roles
// Copies of both operands of every tile of the range, in the order in which the
// MMAs take them: K(0), then K(t+1), V(t) of each segment.  A token group (a box
// of box_rows tokens inside one block, or four tokens gathered) belongs to one
// lane, which looks its block up and issues its copies.
__device__ __forceinline__ void produce(const CUtensorMap& map, const ChunkParams& p, Ctl* ctl, uint8_t* ring,
                                        int lane, uint32_t rank, Walk w) {
  const int bs = p.seqs.block_size;
  const int h = p.box_rows;             // 8..64, or 0: gathers
  uint32_t c = 0;                       // chunk counter
  uint32_t tiles = 0;
  bool ok = true;
  // Rows of this lane's token groups: [tile parity][...]
  int32_t at[2][8];
  // chunk c's slot is free, and its bytes are expected
  auto open = [&]() {
    if (c >= kChunks) ok = warp_wait(ctl, &ctl->empty[c % kChunks], (c / kChunks - 1) & 1, lane, p);
    if (ok && lane == 0) mbar_arrive_expect_tx(&ctl->full[c % kChunks], kChunkBytes);
    __syncwarp();
  };
  Segment g;
  while (ok && next_segment(p, w, g)) {
    const int32_t* bt = p.seqs.block_table + static_cast<int64_t>(g.seq) * p.seqs.bt_stride;
    const int end = item_end(p, g.q, g.item);
    auto lookup = [&](int t, int32_t (&rows)[8]) {
      const int t0 = t * kTile;
      uint8_t* mask = reinterpret_cast<uint8_t*>(ctl->mask[tiles % kMasks]);
      bool missing = false;
      if (h > 0) {
        const int tok = t0 + lane * h;
        int32_t row = -1;
        int there = 0;
        if (lane * h < kTile) {
          if (tok < end) {
            const int64_t first = static_cast<int64_t>(bt[tok / bs]) * bs + tok % bs;
            if (first >= 0 && first < p.nslots) {
              row = static_cast<int32_t>(first);
              there = static_cast<int>(min(static_cast<int64_t>(h), p.nslots - first));
            }
            missing = there < min(h, end - tok);
          }
          for (int i = 0; i < h; i += 8)
            mask[(lane * h + i) >> 3] = there >= i + 8 ? 0xFF : there <= i ? 0 : static_cast<uint8_t>((1 << (there - i)) - 1);
        }
        rows[0] = row >= 0 ? row : static_cast<int32_t>(p.nslots);
      } else {
#pragma unroll
        for (int k = 0; k < 2; ++k) {
          uint32_t bits = 0;
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            const int tok = t0 + (k * 32 + lane) * 4 + i;
            int32_t row = static_cast<int32_t>(p.nslots);
            if (tok < end) {
              const int64_t slot = static_cast<int64_t>(bt[tok / bs]) * bs + tok % bs;
              if (slot >= 0 && slot < p.nslots) {
                row = static_cast<int32_t>(slot);
                bits |= 1u << i;
              } else {
                missing = true;
              }
            }
            rows[k * 4 + i] = row;
          }
          const uint32_t other = __shfl_down_sync(0xFFFFFFFFu, bits, 1);
          if ((lane & 1) == 0) mask[(k * 32 + lane) >> 1] = static_cast<uint8_t>(bits | (other << 4));
        }
      }
      if (missing && rank == 0) record_error(p.err, DSA_DEVERR_BLOCK, g.seq);
      __syncwarp();
      if (lane == 0) mbar_arrive(&ctl->mask_ready[tiles % kMasks]);
      ++tiles;
    };
    auto load_k = [&](const int32_t (&rows)[8]) {
      for (int d = 0; d < 4 && ok; ++d) {
        open();
        if (!ok) return;
        const uint32_t dst = smem_u32(ring + (c % kChunks) * kChunkBytes);
        uint64_t* bar = &ctl->full[c % kChunks];
        if (h > 0) {
          const int tok = lane * h - static_cast<int>(rank) * 128;
          if (tok >= 0 && tok < 128) tma_box(dst + tok * 128, &map, bar, d * 128, rows[0]);
        } else {
          tma_gather4(dst + lane * 512, &map, bar, d * 128, rank ? rows[4] : rows[0], rank ? rows[5] : rows[1],
                      rank ? rows[6] : rows[2], rank ? rows[7] : rows[3]);
        }
        ++c;
      }
    };
    auto load_v = [&](const int32_t (&rows)[8]) {
      const int x0 = static_cast<int>(rank) * 256;
      for (int v = 0; v < 4 && ok; ++v) {
        open();
        if (!ok) return;
        const uint32_t dst = smem_u32(ring + (c % kChunks) * kChunkBytes);
        uint64_t* bar = &ctl->full[c % kChunks];
        if (h > 0) {
          const int tok = lane * h - v * 64;
          if (tok >= 0 && tok < 64)
            for (int n = 0; n < 2; ++n) tma_box(dst + n * 8192 + tok * 128, &map, bar, x0 + n * 128, rows[0]);
        } else if ((lane >> 4) == (v & 1)) {
          const bool up = v >= 2;
          for (int n = 0; n < 2; ++n)
            tma_gather4(dst + n * 8192 + (lane & 15) * 512, &map, bar, x0 + n * 128, up ? rows[4] : rows[0],
                        up ? rows[5] : rows[1], up ? rows[6] : rows[2], up ? rows[7] : rows[3]);
        }
        ++c;
      }
    };
    lookup(g.begin, at[0]);
    load_k(at[0]);
    for (int t = g.begin; t < g.end && ok; ++t) {
      if (t + 1 < g.end) {
        lookup(t + 1, at[1]);
        load_k(at[1]);
      }
      if (ok) load_v(at[0]);
#pragma unroll
      for (int i = 0; i < 8; ++i) at[0][i] = at[1][i];
    }
  }
  // Never leave with a copy in flight (already complete unless a wait gave up).
  if (lane == 0)
    for (uint32_t i = c > kChunks ? c - kChunks : 0; i < c; ++i)
      mbar_wait(&ctl->full[i % kChunks], (i / kChunks) & 1, kDrainWaitNs);
}

// Leader, one thread: the MMAs of both CTAs.
__device__ __forceinline__ void issue_mmas(const ChunkParams& p, Ctl* ctl, uint32_t q0, uint32_t p0, uint32_t ring0,
                                           uint32_t tmem, Walk w) {
  uint32_t c = 0, ns = 0, no = 0, nq = 0;   // chunks, S and O tiles issued, segments
  bool ok = true;
  auto chunk = [&]() {
    const uint32_t s = c % kChunks, par = (c / kChunks) & 1;
    ok = ok && wait_one(ctl, &ctl->full[s], par, p) && wait_one(ctl, &ctl->peer_full[s], par, p);
    tc_fence_after();
    return ring0 + s * kChunkBytes;
  };
  auto issue_s = [&]() {
    if (ns >= 2) ok = ok && wait_one(ctl, &ctl->sfree[ns & 1], ((ns - 2) >> 1) & 1, p);
    const uint32_t d = tmem + kSCol + (ns & 1) * 128;
    for (int b = 0; b < 4 && ok; ++b) {
      const uint32_t k0 = chunk();
      if (!ok) return;
#pragma unroll
      for (int kk = 0; kk < 4; ++kk)
#pragma unroll
        for (int term = 0; term < 2; ++term)
          mma_pair(d, umma_desc_sw128_kmajor(q0 + (term * 4 + b) * 8192 + kk * 32),
                   umma_desc_sw128_kmajor(k0 + kk * 32), idesc_f8(false, false), (b | kk | term) != 0 ? 1u : 0u);
      commit_pair(&ctl->empty[c % kChunks]);
      ++c;
    }
    commit_pair(&ctl->sfull[ns & 1]);
    ++ns;
  };
  auto issue_o = [&](bool first) {
    ok = ok && wait_one(ctl, &ctl->pready, no & 1, p);
    for (int v = 0; v < 4 && ok; ++v) {
      const uint32_t v0 = chunk();
      if (!ok) return;
#pragma unroll
      for (int kk = 0; kk < 2; ++kk)
#pragma unroll
        for (int term = 0; term < 2; ++term)
#pragma unroll
          for (int n = 0; n < 2; ++n)
            mma_pair(tmem + n * 128,
                     umma_desc_sw128_kmajor(p0 + term * 16384 + (v >> 1) * 8192 + (v & 1) * 64 + kk * 32),
                     desc_mnmajor(v0 + n * 8192 + kk * 4096), idesc_f8(term != 0, true),
                     first && (v | kk | term) == 0 ? 0u : 1u);
      commit_pair(&ctl->empty[c % kChunks]);
      ++c;
    }
    commit_pair(&ctl->odone);
    ++no;
  };
  Segment g;
  while (ok && next_segment(p, w, g)) {
    ok = wait_one(ctl, &ctl->qready, nq & 1, p);
    ++nq;
    if (ok) issue_s();
    for (int t = g.begin; t < g.end && ok; ++t) {
      if (t + 1 < g.end) issue_s();
      if (ok) issue_o(t == g.begin);
    }
  }
  // Every MMA is complete before tensor memory is released.
  asm volatile(
      "tcgen05.commit.cta_group::2.mbarrier::arrive::one.shared::cluster.b64 [%0];" ::"r"(smem_u32(&ctl->drain))
      : "memory");
  mbar_wait(&ctl->drain, 0, kDrainWaitNs);
}

// The other CTA, one thread: tells the leader that its copies have landed.
__device__ __forceinline__ void forward(const ChunkParams& p, Ctl* ctl, int64_t tiles) {
  const int64_t n = tiles * kChunks;
  for (int64_t c = 0; c < n; ++c) {
    if (!wait_one(ctl, &ctl->full[c % kChunks], (c / kChunks) & 1, p)) return;
    arrive_at(map_to(&ctl->peer_full[c % kChunks], 0));
  }
}

// Q of the segment's 64 lines of this CTA: q * 2^s = hi + lo, s a power of two a
// line that puts its largest |q| in [128, 256).  Warp w converts lines w, w+8,
// ...; lane l dims 16l..16l+15.  Lines past the request's last are zero.
__device__ __forceinline__ void convert_q(const ChunkParams& p, Ctl* ctl, uint8_t* qop, const Segment& g, int line0,
                                          int sw, int lane) {
  constexpr int kPer = kLines / kSoftmaxWarps;
  uint4 qa[kPer], qb[kPer];
#pragma unroll
  for (int j = 0; j < kPer; ++j) {
    const int i = sw + j * kSoftmaxWarps;
    qa[j] = qb[j] = make_uint4(0, 0, 0, 0);
    if (line0 + i < g.q.lines) {
      const uint4* src = reinterpret_cast<const uint4*>(
          p.q + (static_cast<int64_t>(g.q.row0) * p.heads + line0 + i) * 512 + lane * 16);
      qa[j] = ld_dep_u4(src);
      qb[j] = ld_dep_u4(src + 1);
    }
  }
#pragma unroll
  for (int j = 0; j < kPer; ++j) {
    const int i = sw + j * kSoftmaxWarps;
    const uint32_t w[8] = {qa[j].x, qa[j].y, qa[j].z, qa[j].w, qb[j].x, qb[j].y, qb[j].z, qb[j].w};
    float x[16];
    float amax = 0.0f;
    bool finite = true;
#pragma unroll
    for (int k = 0; k < 8; ++k) {
      x[2 * k] = __uint_as_float(w[k] << 16);
      x[2 * k + 1] = __uint_as_float(w[k] & 0xFFFF0000u);
    }
#pragma unroll
    for (int k = 0; k < 16; ++k) {
      finite &= fabsf(x[k]) < INFINITY;
      amax = fmaxf(amax, fabsf(x[k]));
    }
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) amax = fmaxf(amax, __shfl_xor_sync(0xFFFFFFFFu, amax, o));
    finite = __all_sync(0xFFFFFFFFu, finite);
    int e = 0;
    if (finite && amax > 0.0f) frexpf(amax, &e);  // amax < 2^e
    const int sh = max(-126, min(126, 8 - e));
    const float scale = ldexpf(1.0f, sh);
    // A line with an infinity or a NaN gives NaN logits, as its formula does.
    if (lane == 0)
      ctl->qexp[i] = finite ? p.sm_scale * p.kv_scale * 1.4426950408889634f * ldexpf(1.0f, -sh) : NAN;
    uint32_t hw[4], lw[4];
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      uint16_t hc[2], lc[2];
#pragma unroll
      for (int u = 0; u < 2; ++u) {
        const float a0 = x[4 * k + 2 * u] * scale, a1 = x[4 * k + 2 * u + 1] * scale;
        hc[u] = e4m3x2(a0, a1);
        const float2 hv = e4m3x2_decode(hc[u]);
        lc[u] = e4m3x2(a0 - hv.x, a1 - hv.y);
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
// first and second 128 tokens (its output's first and second 256 dims), and two
// warps share a quarter of the lanes, so four threads have a line.
__device__ __forceinline__ void softmax(const ChunkParams& p, Ctl* ctl, uint8_t* qop, uint8_t* pop, uint8_t* ring,
                                        uint32_t tmem, int warp, int lane, uint32_t rank, int pair, Walk w) {
  const int sw = warp - 2, quarter = warp & 3, ch = sw >> 2;
  const int half = quarter >> 1;
  const int i = (quarter & 1) * 32 + lane;              // line of this CTA
  const int part = half * 2 + ch;
  const uint32_t lane_base = static_cast<uint32_t>(quarter * 32) << 16;
  const uint32_t ocol = tmem + lane_base + ch * 128;    // this thread's output columns
  const uint32_t sfree0 = map_to(&ctl->sfree[0], 0), sfree1 = map_to(&ctl->sfree[1], 0);
  const uint32_t pready = map_to(&ctl->pready, 0), qready = map_to(&ctl->qready, 0);
  uint32_t ns = 0, c = 0;                               // tiles done, chunks before this tile's V
  bool ok = true;
  Segment g;
  while (next_segment(p, w, g)) {
    const int line0 = g.item * kItem + static_cast<int>(rank) * kLines;
    convert_q(p, ctl, qop, g, line0, sw, lane);
    fence_proxy_async_smem();
    softmax_sync();                                     // qexp
    if (lane == 0) arrive_at(qready);
    const float scale = ctl->qexp[i];
    const int last = g.q.lines - 1;
    const int sees = g.q.ctx + min(line0 + i, last) / p.heads + 1;                 // tokens of this line
    const int all_see = g.q.ctx + min(g.item * kItem, last) / p.heads + 1;        // of every line of the item
    float m = -INFINITY, l = 0.0f;
    for (int t = g.begin; t < g.end; ++t, ++ns) {
      const int b = ns & 1;
      const int tok0 = t * kTile + half * 128 + ch * 64;
      // chunks of this segment before V(t): K(begin) .. K(min(t + 1, end - 1)), V(begin) .. V(t - 1)
      const uint32_t vchunk = c + 4 * (min(t + 1, g.end - 1) - g.begin + 1) + 4 * (t - g.begin);
      float z[64];
      if (ok) ok = warp_wait(ctl, &ctl->sfull[b], (ns >> 1) & 1, lane, p);
      if (ok) ok = warp_wait(ctl, &ctl->mask_ready[ns % kMasks], (ns / kMasks) & 1, lane, p);
      bool exceed = false;
      float mx = -INFINITY;
      if (ok) {
        tc_fence_after();
        tmem_load32(tmem + lane_base + kSCol + b * 128 + ch * 64, z);
        tmem_load32(tmem + lane_base + kSCol + b * 128 + ch * 64 + 32, z + 32);
        const uint64_t there = ctl->mask[ns % kMasks][part];
        tc_fence_before();
        __syncwarp();
        if (lane == 0) arrive_at(b ? sfree1 : sfree0);
        const int visible = sees - tok0;                // of this thread's 64 tokens
        if (visible >= 64 && there == ~0ull) {
#pragma unroll
          for (int k = 0; k < 64; ++k) z[k] *= scale;
        } else {
#pragma unroll
          for (int k = 0; k < 64; ++k) z[k] = (k < visible && ((there >> k) & 1)) ? z[k] * scale : -INFINITY;
        }
        float mk[4] = {-INFINITY, -INFINITY, -INFINITY, -INFINITY};
#pragma unroll
        for (int k = 0; k < 64; ++k) mk[k & 3] = fmaxf(mk[k & 3], z[k]);
        mx = fmaxf(fmaxf(mk[0], mk[1]), fmaxf(mk[2], mk[3]));
        exceed = mx > m + kPMaxLog2;
      }
      bool o_idle = ns == 0;                            // the MMAs that read P and add to O are done
      if (softmax_sync_or(exceed)) {
        ctl->red[part][i] = mx;
        softmax_sync();
        const float tm = fmaxf(fmaxf(ctl->red[0][i], ctl->red[1][i]), fmaxf(ctl->red[2][i], ctl->red[3][i]));
        float alpha = 1.0f;
        if (tm > m + kPMaxLog2) {
          const float mn = tm - kPResetLog2;
          alpha = exp2f(m - mn);                        // 0 while nothing was added
          m = mn;
          l *= alpha;
        }
        if (ok && t > g.begin && __any_sync(0xFFFFFFFFu, alpha != 1.0f)) {
          ok = warp_wait(ctl, &ctl->odone, (ns - 1) & 1, lane, p);
          o_idle = true;
          if (ok) {
            tc_fence_after();
#pragma unroll 1
            for (int k = 0; k < 128; k += 32) {
              float v[32];
              tmem_load32(ocol + k, v);
#pragma unroll
              for (int d = 0; d < 32; ++d) v[d] *= alpha;
              tmem_store16(ocol + k, v);
              tmem_store16(ocol + k + 16, v + 16);
            }
            asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory");
          }
        }
        softmax_sync();                                 // red[] has been read
      }
      uint32_t hw[16], lw[16];
      if (ok) {
        const float base = m == -INFINITY ? 0.0f : m;   // nothing seen yet: every p is 0
        float sum[4] = {0.0f, 0.0f, 0.0f, 0.0f};        // of the tile first: a long tail of small weights
#pragma unroll                                          // would be rounded away against a large running sum
        for (int k = 0; k < 16; ++k) {
          uint16_t hc[2], lc[2];
#pragma unroll
          for (int u = 0; u < 2; ++u) {
            const float a0 = exp2f(z[4 * k + 2 * u] - base), a1 = exp2f(z[4 * k + 2 * u + 1] - base);
            hc[u] = e4m3x2(a0, a1);
            const float2 hv = e4m3x2_decode(hc[u]);
            lc[u] = e5m2x2(a0 - hv.x, a1 - hv.y);
            sum[2 * u] += a0;
            sum[2 * u + 1] += a1;
          }
          hw[k] = static_cast<uint32_t>(hc[0]) | (static_cast<uint32_t>(hc[1]) << 16);
          lw[k] = static_cast<uint32_t>(lc[0]) | (static_cast<uint32_t>(lc[1]) << 16);
        }
        l += (sum[0] + sum[1]) + (sum[2] + sum[3]);
        if (!o_idle) ok = warp_wait(ctl, &ctl->odone, (ns - 1) & 1, lane, p);
      }
      if (ok) {
        uint8_t* row = pop + half * 8192 + i * 128;
#pragma unroll
        for (int k = 0; k < 4; ++k) {
          const int at = ((ch * 4 + k) ^ (i & 7)) * 16;
          *reinterpret_cast<uint4*>(row + at) = make_uint4(hw[4 * k], hw[4 * k + 1], hw[4 * k + 2], hw[4 * k + 3]);
          *reinterpret_cast<uint4*>(row + 16384 + at) =
              make_uint4(lw[4 * k], lw[4 * k + 1], lw[4 * k + 2], lw[4 * k + 3]);
        }
        // Tokens that a line of the item does not see have weight 0 there, which
        // a NaN latent would turn into NaN: such codes are zeroed (a line that
        // sees one has a NaN weight, so its output is NaN all the same).
        const int from = all_see - t * kTile;
        if (from < kTile) {
          for (int v = max(0, from) / 64; v < 4 && ok; ++v) {
            const uint32_t slot = (vchunk + v) % kChunks;
            ok = warp_wait(ctl, &ctl->full[slot], ((vchunk + v) / kChunks) & 1, lane, p);
            if (!ok) break;
            const int r0 = max(0, from - v * 64), units = (64 - r0) * 16;  // rows r0..63 x 2 blocks x 8
            uint4* base = reinterpret_cast<uint4*>(ring + slot * kChunkBytes);
            for (int u = sw * 32 + lane; u < units; u += kSoftmaxThreads) {
              uint4* q4 = base + (u & 1) * 512 + r0 * 8 + (u >> 1);
              const uint4 x = *q4;
              const uint4 y = make_uint4(zero_nan4(x.x), zero_nan4(x.y), zero_nan4(x.z), zero_nan4(x.w));
              if (x.x != y.x || x.y != y.y || x.z != y.z || x.w != y.w) *q4 = y;
            }
          }
        }
      }
      if (ok) {
        fence_proxy_async_smem();
        tc_fence_before();
        __syncwarp();
        if (lane == 0) arrive_at(pready);
      }
    }
    c += 8 * (g.end - g.begin);

    // The line's sum in a fixed order, then its output.
    ctl->red[part][i] = l;
    softmax_sync();
    const float lt = (ctl->red[0][i] + ctl->red[1][i]) + (ctl->red[2][i] + ctl->red[3][i]);
    softmax_sync();
    if (ok) ok = warp_wait(ctl, &ctl->odone, (ns - 1) & 1, lane, p);
    if (!ok) continue;
    tc_fence_after();
    const bool whole = g.begin == 0 && g.end == g.tiles;
    const int line = line0 + i;
    const int64_t gline = static_cast<int64_t>(g.q.row0) * p.heads + line;
    const int d0 = half * 256 + ch * 128;
    // slot 0: the item began in an earlier range, 1: it goes on in a later one
    const int64_t pline = (static_cast<int64_t>(pair) * 2 + (g.begin > 0 ? 0 : 1)) * kItem + rank * kLines + i;
    const float inv = m != -INFINITY ? p.kv_scale / lt : (lt != lt ? lt : 0.0f);
#pragma unroll 1
    for (int k = 0; k < 128; k += 32) {
      float v[32];
      tmem_load32(ocol + k, v);
      if (line <= last) {
        if (whole) {
          uint32_t o[16];
#pragma unroll
          for (int d = 0; d < 16; ++d)
            asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(o[d]) : "f"(v[2 * d + 1] * inv), "f"(v[2 * d] * inv));
          uint4* dst = reinterpret_cast<uint4*>(p.out + gline * 512 + d0 + k);
#pragma unroll
          for (int d = 0; d < 4; ++d) dst[d] = make_uint4(o[4 * d], o[4 * d + 1], o[4 * d + 2], o[4 * d + 3]);
        } else {
          float4* dst = reinterpret_cast<float4*>(p.part_o + pline * 512 + d0 + k);
#pragma unroll
          for (int d = 0; d < 8; ++d) dst[d] = make_float4(v[4 * d], v[4 * d + 1], v[4 * d + 2], v[4 * d + 3]);
        }
      }
      __syncwarp();
    }
    if (part == 0 && line <= last) {
      if (whole) {
        if (p.lse != nullptr) p.lse[gline] = lt != 0.0f ? (m + log2f(lt)) * 0.69314718055994531f : -INFINITY;
      } else {
        reinterpret_cast<float2*>(p.part_ml)[pline] = make_float2(m, lt);
      }
    }
    tc_fence_before();
  }
}

__global__ void __cluster_dims__(2, 1, 1) __launch_bounds__(kThreads, 1)
    mla_chunk_kernel(const __grid_constant__ CUtensorMap map, const ChunkParams p) {
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = smem_raw + ((1024u - (smem_u32(smem_raw) & 1023u)) & 1023u);
  uint8_t* qop = smem;
  uint8_t* pop = smem + kQBytes;
  uint8_t* ring = smem + kRingOff;
  Ctl* ctl = reinterpret_cast<Ctl*>(smem + kCtlOff);
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const uint32_t rank = cta_rank();
  const int pair = blockIdx.x >> 1;

  if (tid == 0) {
    for (int k = 0; k < kChunks; ++k) {
      mbar_init(&ctl->full[k], 1);
      mbar_init(&ctl->empty[k], 1);
      mbar_init(&ctl->peer_full[k], 1);
    }
    for (int k = 0; k < 2; ++k) {
      mbar_init(&ctl->sfull[k], 1);
      mbar_init(&ctl->sfree[k], 2 * kSoftmaxWarps);
    }
    for (int k = 0; k < kMasks; ++k) mbar_init(&ctl->mask_ready[k], 1);
    mbar_init(&ctl->pready, 2 * kSoftmaxWarps);
    mbar_init(&ctl->qready, 2 * kSoftmaxWarps);
    mbar_init(&ctl->odone, 1);
    mbar_init(&ctl->drain, 1);
    ctl->abort_flag = 0;
    fence_mbar_init();
    tma_prefetch_map(&map);
  }
  if (warp == 1) {
    asm volatile("tcgen05.alloc.cta_group::2.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(smem_u32(&ctl->tmem_base)),
                 "r"(kTmemCols)
                 : "memory");
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::2.sync.aligned;" ::: "memory");
  }
  grid_dep_wait();    // lengths, tables, latents and q come from kernels before
  // The merge kernel reads the lengths before its own wait: released only now,
  // when the kernels that write them are complete.
  grid_dep_launch();
  const Place at = find_place<kThreads>(p, p.pairs, [&](int64_t per) { return per * pair; },
                                        reinterpret_cast<int64_t*>(smem), blockIdx.x == 0);
  Walk w;
  w.seq = at.seq;
  w.item = at.item;
  w.begin = at.tile;
  w.left = at.seq < 0 ? 0 : min(at.per, at.total - at.per * pair);
  tc_fence_before();
  cluster_sync();     // barriers, tensor memory address; the scratch is free
  tc_fence_after();
  const uint32_t tmem = ctl->tmem_base;

  if (warp == 0) {
    produce(map, p, ctl, ring, lane, rank, w);
  } else if (warp == 1) {
    if (lane == 0) {
      if (rank == 0) issue_mmas(p, ctl, smem_u32(qop), smem_u32(pop), smem_u32(ring), tmem, w);
      else forward(p, ctl, w.left);
    }
    __syncwarp();
  } else {
    softmax(p, ctl, qop, pop, ring, tmem, warp, lane, rank, pair, w);
  }

  tc_fence_before();
  __syncthreads();
  cluster_sync();     // neither CTA leaves while the other may still signal it or its MMAs run
  if (warp == 1) {
    tc_fence_after();
    asm volatile("tcgen05.dealloc.cta_group::2.sync.aligned.b32 %0, %1;" ::"r"(tmem), "r"(kTmemCols) : "memory");
  }
}

// Adds up the parts of the items that several ranges share.  Block x: the item
// that the boundary between ranges x and x + 1 falls into, if that is the
// item's first; block y: eight of its lines, a warp each.
__global__ void __launch_bounds__(kMergeThreads) mla_chunk_merge_kernel(const ChunkParams p) {
  __shared__ int64_t scratch[kMergeThreads];
  const int boundary = blockIdx.x + 1, warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  grid_dep_launch();
  const Place at = find_place<kMergeThreads>(p, p.pairs, [&](int64_t per) { return per * boundary; }, scratch, false);
  if (at.seq < 0 || at.tile == 0 || at.tile > at.per) return;  // (more than a range ago: not the first)
  const SeqInfo q = seq_info(p, at.seq);
  const int tiles = item_tiles(p, q, at.item);
  const int64_t start = at.per * boundary - at.tile;
  const int parts = static_cast<int>((start + tiles - 1) / at.per) - (boundary - 1) + 1;
  const int i = blockIdx.y * kMergeLines + warp, line = at.item * kItem + i;
  grid_dep_wait();
  if (line >= q.lines) return;
  // part 0 in slot 1 of its pair, the others in slot 0 of theirs
  auto pline = [&](int u) {
    return (static_cast<int64_t>(boundary - 1 + u) * 2 + (u == 0 ? 1 : 0)) * kItem + i;
  };
  const float2* ml = reinterpret_cast<const float2*>(p.part_ml);
  float m = -INFINITY;
  bool nan = false;
  for (int u = lane; u < parts; u += 32) {
    const float2 x = ld_dep_f2(ml + pline(u));
    m = fmaxf(m, x.x);
    nan |= x.y != x.y;
  }
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) m = fmaxf(m, __shfl_xor_sync(0xFFFFFFFFu, m, o));
  nan = __any_sync(0xFFFFFFFFu, nan);
  float l = 0.0f, acc[16];
#pragma unroll
  for (int d = 0; d < 16; ++d) acc[d] = 0.0f;
  if (m != -INFINITY) {
#pragma unroll 2
    for (int u = 0; u < parts; ++u) {
      const float2 x = ld_dep_f2(ml + pline(u));
      const float wgt = exp2f(x.x - m);
      const float4* src = reinterpret_cast<const float4*>(p.part_o + pline(u) * 512) + lane;
      l += wgt * x.y;
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        const float4 v = ld_dep_f4(src + k * 32);
        // (0 of a part without weight: it may hold anything)
        if (wgt != 0.0f) {
          acc[4 * k] += wgt * v.x;
          acc[4 * k + 1] += wgt * v.y;
          acc[4 * k + 2] += wgt * v.z;
          acc[4 * k + 3] += wgt * v.w;
        }
      }
    }
  }
  const float inv = nan ? NAN : (m != -INFINITY ? p.kv_scale / l : 0.0f);
  const int64_t gline = static_cast<int64_t>(q.row0) * p.heads + line;
#pragma unroll
  for (int k = 0; k < 4; ++k) {
    uint32_t o[2];
#pragma unroll
    for (int d = 0; d < 2; ++d)
      asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(o[d]) : "f"(acc[4 * k + 2 * d + 1] * inv), "f"(acc[4 * k + 2 * d] * inv));
    *reinterpret_cast<uint2*>(p.out + gline * 512 + k * 128 + lane * 4) = make_uint2(o[0], o[1]);
  }
  if (lane == 0 && p.lse != nullptr)
    p.lse[gline] = nan ? NAN : (m != -INFINITY ? (m + log2f(l)) * 0.69314718055994531f : -INFINITY);
}

}  // namespace

// Two slots a pair: the part of an item that began before its range, and of one
// that goes on after it.
size_t mla_chunk_workspace_bytes(int pairs) {
  const size_t lines = static_cast<size_t>(pairs) * 2 * kItem;
  return lines * 512 * sizeof(float) + lines * 2 * sizeof(float);
}

// Token rows of one copy: the largest power of two, 64 at most, that divides
// the block; under 8 the rows are gathered four at a time.
int mla_chunk_box_rows(int block_size) {
  int h = 64;
  while (block_size % h != 0) h >>= 1;
  return h >= 8 ? h : 0;
}

cudaError_t launch_mla_chunk(ChunkParams p, const CUtensorMap& map, void* workspace, cudaStream_t stream) {
  p.part_o = static_cast<float*>(workspace);
  p.part_ml = p.part_o + static_cast<size_t>(p.pairs) * 2 * kItem * 512;
  cudaError_t e = cudaFuncSetAttribute(mla_chunk_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                       static_cast<int>(kSmemBytes));
  if (e != cudaSuccess) return e;
  cudaLaunchAttribute attr[1] = {dependent_launch_attr()};
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(2 * p.pairs, 1, 1);
  cfg.blockDim = dim3(kThreads, 1, 1);
  cfg.dynamicSmemBytes = kSmemBytes;
  cfg.stream = stream;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  e = cudaLaunchKernelEx(&cfg, mla_chunk_kernel, map, p);
  if (e != cudaSuccess || p.pairs == 1) return e;
  cudaLaunchConfig_t mcfg = {};
  mcfg.gridDim = dim3(p.pairs - 1, kItem / kMergeLines, 1);
  mcfg.blockDim = dim3(kMergeThreads, 1, 1);
  mcfg.stream = stream;
  mcfg.attrs = attr;
  mcfg.numAttrs = 1;
  return cudaLaunchKernelEx(&mcfg, mla_chunk_merge_kernel, p);
}

}  // namespace dsa
