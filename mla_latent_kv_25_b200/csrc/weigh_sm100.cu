// Attention weight per cached token on tcgen05 tensor cores:
//   weight_out[b,t] = weight_in[b,t] + sum_{j,h} exp(scale q[j,h] . row_t - lse[j,h])
//
// Cached tokens are the M dimension, query rows (token j, head h) the N
// dimension, so a TMEM lane holds one token's scores and the sum over heads
// and queries is a sum along the lane: no shuffles, no atomics, one fixed
// order.  A pair of CTAs (cta_group::2) takes M = 256 tokens, 128 each; the
// query rows are split over the two CTAs' shared memory, so every row is
// fetched once per 256 tokens.
//
// Bound: with one query token per sequence the cache is read once and the
// kernel is bound by HBM (1152 bytes per token); with many query tokens by
// the tensor pipe (and L2, which has to deliver 32 bytes per clock and SM).
// Each pair takes a contiguous range of the concatenated block list
// (SegWalker).  One operand of a tile stays in shared memory while the other
// streams through a ring of 16 KB chunks [128 rows x 64 columns]:
//   a sequence with at most 128 query rows: the queries stay (64 rows per
//     CTA), the cache streams past them through nine slots;
//   more query rows: 128 tokens per CTA stay, the queries stream 256 rows at
//     a time through five slots.
//
// With few blocks and many queries a cluster has two or four pairs: they share
// its tokens, take the query tiles in turn and add their sums up from the last
// pair to the first over distributed shared memory, again in one fixed order.
//
// w0: TMA; w1: MMA (one thread of a pair's even CTA), TMEM; w2-5: epilogue,
// thread = token.
//
// Measured (H = 128): 64 sequences x 4096 tokens 65 us (0.75 of the measured
// copy bandwidth; 0.93 at 16384), 32 queries over 4 x 16384 228 us (0.82 of the
// measured bf16 peak; 261 us in a long run under the power cap).
#include <cuda.h>
#include <math.h>

#include <atomic>

#include "common.cuh"
#include "kernels.h"
#include "pair.cuh"
#include "schedule.cuh"
#include "sm100.cuh"

namespace mla {
namespace {

using namespace sm100;

constexpr int kThreads = 192;
constexpr int kTileBlocks = 4;                // blocks of a tile, two per CTA
constexpr int kStayRows = 128;                // queries stay up to this many rows
constexpr int kStreamRows = 256;              // else they stream in tiles of this many
constexpr int kChunks = kRow / 64;            // 64-column chunks of a row
constexpr uint32_t kChunk = 128 * 128;        // [128 rows x 64] bf16
constexpr uint32_t kHalf = kChunk / 2;        // [64 rows x 64]
constexpr int kRingMax = 9;                   // slots while the queries stay
constexpr int kRingMin = 5;                   // slots while the tokens stay
constexpr int kAcc = 2;                       // accumulators [128 x 256] fp32 in TMEM
constexpr uint32_t kTmemCols = 512;
constexpr float kLog2e = 1.4426950408889634f;

// Barriers live at the same offsets in all CTAs; "leader" ones are used in a
// pair's even CTA only and count both CTAs' bytes or arrivals.
struct Bars {
  uint64_t ring_full[kRingMax];   // leader
  uint64_t ring_empty[kRingMax];  // commit to both
  uint64_t res_full;              // leader
  uint64_t res_empty;             // commit to both
  uint64_t acc_full[kAcc];        // commit to both
  uint64_t acc_empty[kAcc];       // leader
  uint64_t lse_full[2];           // this CTA's epilogue warps wrote their shares
  uint64_t red_full;              // the next pair's sums landed here
  uint64_t red_empty;             // the previous pair has read this pair's sums
  uint32_t tmem_base;
  int abort;
};
constexpr uint32_t kRedOff = 512;               // float [128]: sums of the next pair
static_assert(sizeof(Bars) <= kRedOff, "barrier block too large");

constexpr uint32_t kLseOff = 1024;              // float [2][kStreamRows]: a query tile's lse, base 2
constexpr uint32_t kResOff = kLseOff + 2 * kStreamRows * 4;
// the resident operand: 64 query rows or 128 tokens; the ring behind it
__host__ __device__ constexpr uint32_t ring_off(bool queries_stay) {
  return kResOff + kChunks * (queries_stay ? kHalf : kChunk);
}
// the dynamic shared memory of a kernel without static shared memory starts
// at a multiple of 1024 here; the kernel checks it
constexpr uint32_t kSmem = ring_off(false) + kRingMin * kChunk;
static_assert(ring_off(true) + kRingMax * kChunk <= kSmem && kSmem <= 232448, "shared memory budget");

struct Queries {
  int n;        // query tokens of the sequence
  int row0;     // first row of q
  int rows;     // n * H
  bool stay;    // one tile of at most kStayRows rows, held in shared memory
  int tiles;
};

__device__ __forceinline__ Queries queries_of(const WeighParams& p, int b) {
  const int a = p.q_offsets[b], e = p.q_offsets[b + 1];
  Queries q;
  q.n = a >= 0 && e >= a && e <= p.T ? e - a : 0;
  q.row0 = a * p.H;
  q.rows = q.n * p.H;
  q.stay = q.rows <= kStayRows;
  q.tiles = q.stay ? (q.rows > 0 ? 1 : 0) : (q.rows + kStreamRows - 1) / kStreamRows;
  return q;
}

// Rows of query tile i: a multiple of 16.
__device__ __forceinline__ int tile_rows(const Queries& q, int i) {
  return q.stay ? q.rows : min(kStreamRows, q.rows - kStreamRows * i);
}
// Rows that its MMAs take, half of them from each CTA.  With cta_group::2 N is a
// multiple of 32: behind the tile up to 16 rows of other tokens (or zeros) are
// multiplied and not looked at.
__device__ __forceinline__ int mma_rows(const Queries& q, int i) { return (tile_rows(q, i) + 31) & ~31; }

struct Ctx {
  const WeighParams* p;
  uint32_t base;
  Bars* bars;
  uint32_t tmem;
  WaitCtx wc;
  int rank;        // in the pair
  uint32_t lead;   // cluster rank of the pair's even CTA
  uint16_t both;   // mask of the pair's CTAs
  int pair, pairs; // of the cluster
  int warp, lane;
};

__device__ __forceinline__ uint32_t bar_addr(const uint64_t& b) { return smem_u32(&b); }

// Pairs that work on a segment (the first ones of the cluster): one per query
// tile at most.  Pair k takes the query tiles k, k + active, ...
__device__ __forceinline__ int active_pairs(const Ctx& c, const Queries& q) {
  return q.tiles < c.pairs ? (q.tiles > 0 ? q.tiles : 1) : c.pairs;
}

// Position in the ring.  The slot count depends on the operand that stays, so
// every slot has a phase of its own; a segment with the other operand starts
// at slot 0 again (its first resident load waits for all earlier MMAs, so
// every slot is free then).
struct Ring {
  int slot = 0;
  uint32_t phases = 0;  // bit s: parity of slot s's next fill
  bool stay = false;
  __device__ __forceinline__ bool mode(bool queries_stay) {
    const bool switched = stay != queries_stay;
    if (switched) slot = 0;
    stay = queries_stay;
    return switched;
  }
  __device__ __forceinline__ uint32_t phase() const { return (phases >> slot) & 1u; }
  __device__ __forceinline__ void next() {
    phases ^= 1u << slot;
    slot = slot + 1 == (stay ? kRingMax : kRingMin) ? 0 : slot + 1;
  }
};

// A block of the tile that is safe to load; missing blocks load block 0 (both
// CTAs always load, so that neither runs ahead of the other).
__device__ __forceinline__ int safe_block(const WeighParams& p, const Segment& g, int j) {
  const int id = j < g.blk_hi ? p.block_table[size_t(g.b) * p.max_blocks + j] : 0;
  return id >= 0 && id < p.num_blocks ? id : 0;
}

// The producer's loop over one segment (one thread of each CTA); bytes are
// counted on the even CTA's barriers, announced there by it for both.
__device__ __forceinline__ bool produce(const Ctx& c, const CUtensorMap* qmap, const CUtensorMap* kmap,
                                        const Segment& g, const Queries& q, uint32_t& rit, Ring& ring) {
  const WeighParams& p = *c.p;
  Bars* bars = c.bars;
  const uint32_t res_bar = map_to_rank(bar_addr(bars->res_full), c.lead);
  const uint32_t full0 = map_to_rank(bar_addr(bars->ring_full[0]), c.lead);
  const uint32_t own_full0 = bar_addr(bars->ring_full[0]), empty0 = bar_addr(bars->ring_empty[0]);
  const CUtensorMap* stream = q.stay ? kmap : qmap;
  const bool switched = ring.mode(q.stay);
  const uint32_t ring0 = c.base + ring_off(q.stay);
  const int active = active_pairs(c, q);
  auto resident = [&](uint32_t bytes) {
    const bool ok = wait_phase(bar_addr(bars->res_empty), (rit & 1u) ^ 1u, c.wc);
    ++rit;
    if (ok && c.rank == 0) mbar_arrive_expect_tx(bar_addr(bars->res_full), 2 * bytes);
    return ok;
  };
  auto load_queries = [&]() {
    if (!resident(kChunks * kHalf)) return false;
    for (int ch = 0; ch < kChunks; ++ch)
      pair_tma_load_2d(c.base + kResOff + ch * kHalf, qmap, 64 * ch, q.row0 + c.rank * (mma_rows(q, 0) / 2), res_bar);
    return true;
  };
  // The next sequence's queries have to wait for all of the previous one's
  // MMAs; its first tile (as many chunks as slots) need not, unless the ring
  // is laid out anew.
  bool queries_due = q.stay;
  if (queries_due && switched) {
    if (!load_queries()) return false;
    queries_due = false;
  }
  for (int j = g.blk_lo; j < g.blk_hi; j += kTileBlocks) {
    const int y0 = safe_block(p, g, j + 2 * c.rank) * kBlock, y1 = safe_block(p, g, j + 2 * c.rank + 1) * kBlock;
    if (!q.stay) {
      if (!resident(kChunks * kChunk)) return false;
      for (int ch = 0; ch < kChunks; ++ch) {
        pair_tma_load_2d(c.base + kResOff + ch * kChunk, kmap, 64 * ch, y0, res_bar);
        pair_tma_load_2d(c.base + kResOff + ch * kChunk + kHalf, kmap, 64 * ch, y1, res_bar);
      }
    }
    for (int i = c.pair; i < q.tiles; i += active) {
      const int row = q.row0 + kStreamRows * i + c.rank * (mma_rows(q, i) / 2);
      const int r0 = q.stay ? y0 : row, r1 = q.stay ? y1 : row + 64;
#pragma unroll 1
      for (int x = 0; x < 64 * kChunks; x += 64) {
        const uint32_t at = 8 * ring.slot;
        if (!wait_phase(empty0 + at, ring.phase() ^ 1u, c.wc)) return false;
        if (c.rank == 0) mbar_arrive_expect_tx(own_full0 + at, 2 * kChunk);
        const uint32_t dst = ring0 + ring.slot * kChunk;
        pair_tma_load_2d(dst, stream, x, r0, full0 + at);
        pair_tma_load_2d(dst + kHalf, stream, x, r1, full0 + at);
        ring.next();
      }
      if (queries_due) {
        if (!load_queries()) return false;
        queries_due = false;
      }
    }
  }
  return true;
}

// The MMA warp's loop over one segment (the elected thread of the pair's even CTA); the
// next chunk's barrier is probed before the current chunk's MMAs are issued.
__device__ __forceinline__ bool multiply(const Ctx& c, int tiles, const Queries& q, uint32_t& rit, Ring& ring,
                                         uint32_t& ait) {
  Bars* bars = c.bars;
  ring.mode(q.stay);
  const uint32_t full0 = bar_addr(bars->ring_full[0]), empty0 = bar_addr(bars->ring_empty[0]);
  const uint64_t res0 = sw128_desc(c.base + kResOff, 16, 1024);
  const uint64_t ring0 = sw128_desc(c.base + ring_off(q.stay), 16, 1024);
  const uint32_t res_step = (q.stay ? kHalf : kChunk) >> 4;
  auto wait_resident = [&]() {
    const bool ok = wait_phase(bar_addr(bars->res_full), rit & 1u, c.wc);
    ++rit;
    return ok;
  };
  const int active = active_pairs(c, q);
  bool ready = false;
  if (q.stay && !wait_resident()) return false;
  for (int j = 0; j < tiles; ++j) {
    if (!q.stay && !wait_resident()) return false;
    for (int i = c.pair; i < q.tiles; i += active, ++ait) {
      const int buf = ait % kAcc;
      const uint32_t idesc = idesc_bf16(256, mma_rows(q, i), false, false);
      const uint32_t d = c.tmem + 256 * buf;
      if (!wait_phase(bar_addr(bars->acc_empty[buf]), ((ait / kAcc) & 1u) ^ 1u, c.wc)) return false;
      tc_fence_after();
#pragma unroll 1
      for (int ch = 0; ch < kChunks; ++ch) {
        if (!ready && !wait_phase(full0 + 8 * ring.slot, ring.phase(), c.wc)) return false;
        const uint32_t s = ring.slot;
        ring.next();
        ready = mbar_test_wait(full0 + 8 * ring.slot, ring.phase());
        const uint64_t res = res0 + static_cast<uint32_t>(ch) * res_step, str = ring0 + s * (kChunk >> 4);
        const uint64_t a = q.stay ? str : res, bq = q.stay ? res : str;
#pragma unroll
        for (int kk = 0; kk < 4; ++kk) pair_mma_ss(d, a + 2 * kk, bq + 2 * kk, idesc, (ch | kk) ? 1u : 0u);
        pair_commit(empty0 + 8 * s, c.both);
      }
      pair_commit(bar_addr(bars->acc_full[buf]), c.both);
    }
    if (!q.stay) pair_commit(bar_addr(bars->res_empty), c.both);
  }
  if (q.stay) pair_commit(bar_addr(bars->res_empty), c.both);
  return true;
}

// Writes a query tile's lse in base 2 (rows past the tile: +inf, whose
// exponential is 0) to its buffer, 64 rows per epilogue warp.
__device__ __forceinline__ void stage_lse(const Ctx& c, const Queries& q, int i, uint32_t lit, int quad) {
  float* dst = reinterpret_cast<float*>(reinterpret_cast<uint8_t*>(c.bars) + kLseOff) + (lit & 1u) * kStreamRows;
#pragma unroll
  for (int k = 0; k < 2; ++k) {
    const int at = 64 * quad + 32 * k + c.lane;
    const int r = kStreamRows * i + at;
    dst[at] = r < q.rows ? c.p->lse[static_cast<size_t>(q.row0) + r] * kLog2e : INFINITY;
  }
  __syncwarp();
  if (c.lane == 0) mbar_arrive(bar_addr(c.bars->lse_full[lit & 1u]));
}

__device__ __forceinline__ bool accumulate(const Ctx& c, const Segment& g, const Queries& q, uint32_t& ait,
                                           uint32_t& lit, uint32_t& sent, uint32_t& got) {
  const WeighParams& p = *c.p;
  Bars* bars = c.bars;
  const int quad = c.warp & 3;
  const int row = c.rank * 128 + quad * 32 + c.lane;  // token of the tile: TMEM lane of this CTA
  const uint32_t lane_off = static_cast<uint32_t>(quad * 32) << 16;
  const uint32_t empty0 = map_to_rank(bar_addr(bars->acc_empty[0]), c.lead);
  const float sl2 = p.softmax_scale * kLog2e;
  const size_t S = size_t(p.max_blocks) * kBlock;
  const int len_off = g.len - (q.n - 1);  // query token j sees the first len_off + j rows
  const int active = active_pairs(c, q);
  const int slot = quad * 32 + c.lane;
  const float* lse = nullptr;
  // A buffer is written again two tiles on: by then every warp has arrived
  // for the tile between, that is, has left this one.
  auto next_lse = [&](int i) {
    stage_lse(c, q, i, lit, quad);
    if (!warp_wait(bar_addr(bars->lse_full[lit & 1u]), (lit >> 1) & 1u, c.wc)) return false;
    lse = reinterpret_cast<const float*>(reinterpret_cast<const uint8_t*>(bars) + kLseOff) + (lit & 1u) * kStreamRows;
    ++lit;
    return true;
  };
  if (q.stay && q.tiles > 0 && !next_lse(0)) return false;
  for (int j = g.blk_lo; j < g.blk_hi; j += kTileBlocks) {
    const int tok = j * kBlock + row;
    const int last = min((j + kTileBlocks) * kBlock, g.len) - 1;
    float sum[4] = {0.f, 0.f, 0.f, 0.f};
    for (int i = c.pair; i < q.tiles; i += active, ++ait) {
      if (!q.stay && !next_lse(i)) return false;
      const int buf = ait % kAcc;
      if (!warp_wait(bar_addr(bars->acc_full[buf]), (ait / kAcc) & 1u, c.wc)) return false;
      tc_fence_after();
      const int cols = tile_rows(q, i);  // a multiple of 16
      const uint32_t taddr = c.tmem + lane_off + 256 * buf;
      // whether the tile's first row, which sees least, sees the tile's last token
      const bool seen = last < len_off + kStreamRows * i / p.H;
#pragma unroll
      for (int k = 0; k < kStreamRows / 32; ++k) {
        if (32 * k >= cols) break;
        uint32_t v[32];
        tmem_ld32(taddr + 32 * k, v);
        tmem_ld_wait();
        if (seen && 32 * k + 32 <= cols) {
#pragma unroll
          for (int e = 0; e < 32; e += 4) {
            const float4 l = *reinterpret_cast<const float4*>(lse + 32 * k + e);
            sum[0] += ex2_approx(fmaf(__uint_as_float(v[e]), sl2, -l.x));
            sum[1] += ex2_approx(fmaf(__uint_as_float(v[e + 1]), sl2, -l.y));
            sum[2] += ex2_approx(fmaf(__uint_as_float(v[e + 2]), sl2, -l.z));
            sum[3] += ex2_approx(fmaf(__uint_as_float(v[e + 3]), sl2, -l.w));
          }
        } else {
          // 16 columns at a time belong to one query token (H is a multiple of 16)
#pragma unroll
          for (int half = 0; half < 2; ++half) {
            const int c0 = 32 * k + 16 * half;
            const bool in = c0 < cols && tok < len_off + (kStreamRows * i + c0) / p.H;
#pragma unroll
            for (int e = 16 * half; e < 16 * half + 16; ++e) {
              const float x = ex2_approx(fmaf(__uint_as_float(v[e]), sl2, -lse[32 * k + e]));
              if (in) sum[e & 3] += x;
            }
          }
        }
      }
      tc_fence_before();
      __syncwarp();
      if (c.lane == 0) mbar_arrive_cluster_relaxed(empty0 + 8 * buf);  // the loads are in registers
    }
    float total = (sum[0] + sum[1]) + (sum[2] + sum[3]);
    if (c.pair + 1 < active) {  // the later pairs' sums
      if (!warp_wait(bar_addr(bars->red_full), got & 1u, c.wc)) return false;
      ++got;
      total += *reinterpret_cast<const volatile float*>(reinterpret_cast<const uint8_t*>(bars) + kRedOff + 4 * slot);
      __syncwarp();
      if (c.lane == 0) mbar_arrive_remote(bar_addr(bars->red_empty), c.lead + c.rank + 2);
    }
    if (c.pair > 0) {  // on to the pair before
      if (!warp_wait(bar_addr(bars->red_empty), (sent & 1u) ^ 1u, c.wc)) return false;
      ++sent;
      const uint32_t to = c.lead + c.rank - 2, full = map_to_rank(bar_addr(bars->red_full), to);
      if (c.lane == 0) mbar_arrive_expect_tx_cluster_relaxed(full, 32 * 4);
      st_async_b32(map_to_rank(c.base + kRedOff + 4 * slot, to), __float_as_uint(total), full);
      continue;
    }
    if (tok < g.len && j + (row >> 6) < g.blk_hi) {
      const int id = p.block_table[size_t(g.b) * p.max_blocks + tok / kBlock];
      const bool ok = id >= 0 && id < p.num_blocks;
      if (!ok && (row & 63) == 0) atomicOr(p.err, kErrBadBlock);
      const size_t at = g.b * S + tok;
      const float w = p.weight_in != nullptr ? p.weight_in[at] : 0.f;
      p.weight_out[at] = ok ? w + total : w;
    }
  }
  return true;
}

// clusters of 2 * pairs CTAs
__global__ void __launch_bounds__(kThreads, 1)
weigh_sm100_kernel(const __grid_constant__ CUtensorMap qmap, const __grid_constant__ CUtensorMap kmap,
                   const WeighParams p, int pairs) {
  extern __shared__ __align__(1024) uint8_t smem_raw[];
  const uint32_t base = smem_u32(smem_raw);
  Bars* bars = reinterpret_cast<Bars*>(smem_raw);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  if (threadIdx.x == 0) {
    for (int s = 0; s < kRingMax; ++s) {
      mbar_init(bar_addr(bars->ring_full[s]), 1);
      mbar_init(bar_addr(bars->ring_empty[s]), 1);
    }
    mbar_init(bar_addr(bars->res_full), 1);
    mbar_init(bar_addr(bars->res_empty), 1);
    for (int s = 0; s < kAcc; ++s) {
      mbar_init(bar_addr(bars->acc_full[s]), 1);
      mbar_init(bar_addr(bars->acc_empty[s]), 8);  // every epilogue warp of both CTAs
    }
    mbar_init(bar_addr(bars->lse_full[0]), 4);
    mbar_init(bar_addr(bars->lse_full[1]), 4);
    mbar_init(bar_addr(bars->red_full), 4);       // the next pair's epilogue warps
    mbar_init(bar_addr(bars->red_empty), 4);      // the previous pair's
    bars->abort = 0;
    fence_mbar_init();
    prefetch_tmap(&qmap);
    prefetch_tmap(&kmap);
  }
  if (warp == 1) {
    pair_tmem_alloc(smem_u32(&bars->tmem_base), kTmemCols);
    pair_tmem_relinquish();
  }
  tc_fence_before();
  cluster_sync();
  tc_fence_after();
  Ctx c;
  c.p = &p;
  c.base = base;
  c.bars = bars;
  c.tmem = bars->tmem_base;
  c.wc = WaitCtx{p.spin_limit, p.err, &bars->abort};
  const uint32_t in_cluster = cluster_ctarank();
  c.rank = static_cast<int>(in_cluster & 1u);
  c.lead = in_cluster & ~1u;
  c.both = static_cast<uint16_t>(0x3u << c.lead);
  c.pair = static_cast<int>(in_cluster >> 1);
  c.pairs = pairs;
  c.warp = warp;
  c.lane = lane;

  if (blockIdx.x == 0)  // bad lengths and offsets, once
    for (int b = threadIdx.x; b < p.B; b += kThreads) {
      checked_len(p.seq_lens, b, p.max_blocks, p.err);
      if (p.q_offsets[b] < 0 || p.q_offsets[b + 1] < p.q_offsets[b] || p.q_offsets[b + 1] > p.T)
        atomicOr(p.err, kErrSeqTooLong);
    }

  SegWalker w;
  w.init(p.seq_lens, p.B, p.max_blocks, gridDim.x / (2 * pairs), blockIdx.x / (2 * pairs));
  // swizzled tiles need 1024-byte aligned shared memory
  if ((base & 1023u) != 0) {
    if (threadIdx.x == 0) atomicOr(p.err, kErrTimeout);
    w.b = p.B;  // no segments
  }
  Segment gs;
  uint32_t rit = 0, ait = 0, lit = 0, sent = 0, got = 0;
  Ring ring;
  while (w.next(gs)) {
    const Segment g = gs;  // in registers, not behind the walker's reference
    const Queries q = queries_of(p, g.b);
    if (c.pair >= active_pairs(c, q)) continue;
    int ok = 1;
    if (warp == 0) {
      // counters live in the elected thread, the same one every time
      if (q.tiles > 0 && elect_one()) {
        if (!produce(c, &qmap, &kmap, g, q, rit, ring)) ok = 0;
      }
      ok = __all_sync(0xffffffffu, ok);
    } else if (warp == 1) {
      if (q.tiles > 0 && c.rank == 0 && elect_one()) {
        if (!multiply(c, (g.blk_hi - g.blk_lo + kTileBlocks - 1) / kTileBlocks, q, rit, ring, ait)) ok = 0;
      }
      ok = __all_sync(0xffffffffu, ok);
    } else {
      ok = accumulate(c, g, q, ait, lit, sent, got) ? 1 : 0;
    }
    if (!ok) break;
  }

  __syncthreads();
  if (bars->abort) {
    // let any asynchronous copy still in flight land before the CTA exits
    if (threadIdx.x == 0) {
      const long long t0 = clock64();
      while (clock64() - t0 < 20000000LL) __nanosleep(1000);
    }
    __syncthreads();
  }
  // no CTA leaves while another may still signal it or run MMAs on its memory
  cluster_sync();
  if (warp == 1) {
    tc_fence_after();
    pair_tmem_dealloc(c.tmem, kTmemCols);
  }
  cluster_sync();
}

}  // namespace

cudaError_t launch_weigh(const WeighParams& p, const CUtensorMap& qmap, const CUtensorMap& kmap,
                         cudaStream_t stream) {
  // clusters of 1, 2 and 4 pairs that fit on the device at once, 0 = not known yet
  static std::atomic<int> fit[64][3];
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= 64) return cudaErrorInvalidDevice;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim.x = 2;
  attr[0].val.clusterDim.y = attr[0].val.clusterDim.z = 1;
  cudaLaunchConfig_t cfg = {};
  cfg.blockDim = dim3(kThreads);
  cfg.dynamicSmemBytes = kSmem;
  cfg.stream = stream;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  if (fit[dev][2].load(std::memory_order_acquire) == 0) {
    cudaError_t e = cudaFuncSetAttribute(weigh_sm100_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, int(kSmem));
    if (e != cudaSuccess) return e;
    for (int k = 0; k < 3; ++k) {
      int n = 0;
      attr[0].val.clusterDim.x = 2u << k;
      cfg.gridDim = dim3(2u << k);
      if ((e = cudaOccupancyMaxActiveClusters(&n, weigh_sm100_kernel, &cfg)) != cudaSuccess) return e;
      fit[dev][k].store(n > 0 ? n : 1, std::memory_order_release);
    }
  }
  // Pairs per cluster by the steps of the longest one: tiles of its share of
  // the blocks (the table's width stands for the lengths, which are on the
  // device) times its share of the query tiles of an average sequence.  32
  // queries x 128 heads over 1024 tokens: 58 us with one pair, 27 with four.
  const long long blocks = static_cast<long long>(p.B) * p.max_blocks;
  const long long rows = static_cast<long long>(p.T) * p.H / p.B;
  const long long qtiles = rows <= kStayRows ? 1 : (rows + kStreamRows - 1) / kStreamRows;
  int best = 0;
  long long least = -1;
  for (int k = 0; k < 3; ++k) {
    const long long n = fit[dev][k].load(std::memory_order_acquire);
    const long long share = (blocks + n - 1) / n;
    const long long steps = (share + kTileBlocks - 1) / kTileBlocks * ((qtiles + (1 << k) - 1) >> k);
    if (least < 0 || steps < least) {
      least = steps;
      best = k;
    }
  }
  attr[0].val.clusterDim.x = 2u << best;
  // With one query tile a pair takes a tile of blocks as fast as one block: no
  // more pairs than such tiles (1 x 16 heads over 5000: 12.1 us with all, 10.2;
  // with more query tiles short ragged sequences lose 2-4 us by it).
  long long n = fit[dev][best].load(std::memory_order_acquire);
  const long long tiles = (blocks + kTileBlocks - 1) / kTileBlocks;
  if (qtiles <= 1 && tiles < n) n = tiles > 0 ? tiles : 1;
  cfg.gridDim = dim3((2u << best) * static_cast<unsigned>(n));
  return cudaLaunchKernelEx(&cfg, weigh_sm100_kernel, qmap, kmap, p, 1 << best);
}

}  // namespace mla
