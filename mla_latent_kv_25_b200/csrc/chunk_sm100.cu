// Attention of ragged chunks of new tokens over the paged latent cache on
// sm_100a tensor cores.
//
// A tile is 256 query rows: as many whole tokens of one sequence as fit (2 at
// H = 128).  One engine = a cluster of four CTAs, two pairs of SMs split by
// role, because the fp32 output of 256 rows x 512 latent columns fills the
// TMEM of two SMs:
//
//   score pair (ranks 0, 1)                     value pair (ranks 2, 3)
//   S[256 x 128] = Q K^T, cta_group::2:         O[256 x 512] += P V, cta_group::2:
//   each CTA holds 128 query rows (eight of     each CTA holds P of 128 rows and half
//   their nine chunks in TMEM) and one of the   of the latent columns of each block;
//   pass's two blocks; S is double-buffered     O fills TMEM
//   w0 feeds Q and K, w2 the last chunk of Q,   w0 feeds V, w1 MMA (rank 2), w2 zeroes
//   w1 MMA (rank 0); w4-7 and w8-11 softmax     V rows past the length, w3 relays P's
//   of every other pass, P by st.async to       arrival to rank 2, w4-11 rescale, output
//   CTA rank + 2
//
// Bound: the tensor pipe, 2 * rows * tokens * (576 + 512) FLOPs.  Why this
// shape: with 256 rows to a cached token a pair reads 576 bytes of K (512 of
// V) per SM and token while its MMAs take 18 (16) cycles, 32 bytes per clock
// and SM from L2; 128 rows on two SMs would need twice that.  Q in TMEM (M =
// 256, N = 128 runs at the pipe's full rate with A there) leaves 208 KB for K:
// a ring of 80 KB next to all of Q in shared memory, with S of N = 256, took 490
// us for the 16 tokens below.
//
// The tiles' blocks (and a charge per tile) are laid end to end and cut into P
// equal ranges, one per engine, so ragged batches balance and a few tokens over
// a long context still use every engine; cut tiles are merged by
// chunk_merge_kernel.  chunk_plan_kernel writes the tile list and the ranges.
//
// Softmax as in the decode: fp32, a row's running max moves only when a pass
// exceeds it by 2^8, P is rounded to bf16 (at most 2^-8 of the value, like any
// bf16 operand of a tensor-core product) while its sum is taken unrounded.
// Every wait is bounded (WaitCtx).
//
// Measured (B200, H = 128): 16 tokens over 131072 0.44 ms = 1320 TFLOP/s (0.90
// of what 132 SMs can reach at the measured bf16 peak); 512 tokens over 16384
// 1.49 ms = 1540 TFLOP/s in a short run (0.51 and 1.73 ms in a long one under
// the power cap, at 1.6 GHz).  What remains: 33 clusters of four use 132 of 148 SMs, the start and the
// end of a tile (about eight blocks' time), and the merge.
#include <cuda.h>
#include <math.h>

#include <atomic>

#include "common.cuh"
#include "kernels.h"
#include "pair.cuh"
#include "plan.h"
#include "sm100.cuh"

namespace mla {
namespace {

using namespace sm100;

constexpr int kThreads = 384;
constexpr int kTileRows = kChunkTileRows;     // 256
constexpr int kPassBlocks = 2;                // blocks per QK pass (N = 128), one from each score CTA
constexpr int kChunks = kRow / 64;            // 64-column chunks of a row
constexpr int kQTmem = kChunks - 1;           // chunks of Q kept in TMEM; the last stays in shared memory
constexpr int kKSlots = 13;                   // score: ring of two [64 tokens x 64] chunks of K, or one of Q
constexpr int kVSlots = 4;                    // value: ring of [64 tokens x 256] half blocks
constexpr int kNP = 4;                        // P records in flight (5 measured the same, 3 are 15 % slower)

constexpr uint32_t kQChunk = 128 * 128;       // [128 rows x 64] bf16
constexpr uint32_t kBlkChunk = 64 * 128;      // [64 tokens x 64] bf16
constexpr uint32_t kKSlot = 2 * kBlkChunk;
static_assert(kKSlot == kQChunk, "Q is staged in the ring");
constexpr uint32_t kVSlot = 4 * kBlkChunk;
constexpr uint32_t kPBytes = 128 * 64 * 2;    // P [128 rows x 64 tokens] bf16, 8 x 8 core matrices
constexpr uint32_t kPCoreK = 128 * 16;        // bytes per 8-token column of core matrices
constexpr uint32_t kMetaBytes = 128 * 16;     // per row: alpha, m, l, unused
constexpr uint32_t kFlagBytes = 64;           // per quadrant: rescale flag
constexpr uint32_t kRecBytes = 19 * 1024;
constexpr float kRescaleThreshold = 8.0f;     // log2 units
constexpr float kLog2e = 1.4426950408889634f;
static_assert(kPBytes + kMetaBytes + kFlagBytes <= kRecBytes, "record layout");
constexpr uint32_t kTmemCols = 512;
constexpr uint32_t kTmemQ = 256;              // score: S in columns 0-127 and 128-255, then 32 columns per chunk of Q
static_assert(kTmemQ + 32 * kQTmem == kTmemCols, "TMEM of the score pair");
constexpr uint16_t kScoreMask = 0x3, kValueMask = 0xc;

// Barriers live at the same offsets in all four CTAs; "leader" ones are used
// in rank 0 (score) or rank 2 (value) only.
struct Barriers {
  uint64_t k_full[kKSlots];                    // leader: both CTAs' chunks landed
  uint64_t k_empty[kKSlots];                   // commit to both
  uint64_t q_full;                             // leader: the last chunk of Q
  uint64_t q_empty;                            // commit to both
  uint64_t s_full[2];                          // commit to both
  uint64_t s_empty[2];                         // leader: the softmax warps of both that read this buffer
  uint64_t m_set[2][4];                        // a warp of this half published its rows' maxima
  uint64_t l_set[2][4];                        // and their sums, before a segment's last pass
  uint64_t p_empty[kNP];                       // score CTAs: record r of the value CTA is free
  uint64_t v_full[kVSlots];                    // this CTA's V landed
  uint64_t v_ready[kVSlots];                   // leader: both CTAs' V landed and cleaned
  uint64_t v_empty[kVSlots];                   // commit to both
  uint64_t p_full[kNP];                        // this CTA's P record landed
  uint64_t p_ready[kNP];                       // leader: both CTAs' records landed
  uint64_t epi_req;                            // both: request posted + MMAs done
  uint64_t corr_done, o_free;                  // leader: all epilogue warps of both
  uint64_t meta_done;                          // all epilogue warps read the final record
  alignas(8) uint32_t flag[kNP][2];            // leader: a row of each CTA's record asks for a rescale
  uint32_t sink;                               // words that only end a phase
  uint32_t req;
  uint32_t tmem_base;
  int abort;
};
static_assert(sizeof(Barriers) <= 1024, "barrier block too large");

constexpr uint32_t kMaxOff = 1024;             // score: float [2 halves][128] running maxima
constexpr uint32_t kSumOff = kMaxOff + 1024;   // score: float [2 halves][128] sums
constexpr uint32_t kQOff = kSumOff + 1024;     // score: the last chunk of Q
__host__ __device__ constexpr uint32_t k_slot_off(int s) { return kQOff + kQChunk + s * kKSlot; }
__host__ __device__ constexpr uint32_t v_slot_off(int s) { return 1024 + s * kVSlot; }
__host__ __device__ constexpr uint32_t rec_off(int r) { return 1024 + kVSlots * kVSlot + r * kRecBytes; }
// value: every epilogue warp's staging of 16 rows x 128 bytes of output
constexpr uint32_t kStageBytes = 16 * 128;
__host__ __device__ constexpr uint32_t stage_off(int w) { return rec_off(kNP) + w * kStageBytes; }
constexpr uint32_t kScoreSmem = k_slot_off(kKSlots);
constexpr uint32_t kValueSmem = stage_off(8);
// the dynamic shared memory of a kernel without static shared memory starts
// at a multiple of 1024 here; the kernel checks it
constexpr uint32_t kSmemBytes = kScoreSmem > kValueSmem ? kScoreSmem : kValueSmem;
static_assert(kSmemBytes <= 232448, "shared memory budget");

constexpr uint32_t kIdescQK = idesc_bf16(256, 128, false, false);
constexpr uint32_t kIdescPV = idesc_bf16(256, 256, false, true);

// ------------------------------------------------------------------ segments

// One piece of a tile: blocks [blk_lo, blk_hi) of its sequence.
struct Seg {
  int row0, rows;  // first row of q / out, number of rows
  int b;
  int len;         // cached tokens that the tile's last query token sees
  int blk_lo, blk_hi;
  int slot;        // partial slot, or -1 when the piece is the whole tile
};

// The axis that is cut: every tile that reads the cache takes kTileUnits units
// (what starting and finishing a tile costs next to a block) and one per block,
// its blocks last.  Without that charge an engine that gets many short tiles
// takes far longer than one with a single long tile.
constexpr int kTileUnits = 8;
// An engine gets at least this many units: shorter ranges cost more in the
// merge than they save.  With 8, 10 and 16 (captured runs, us): 5 x 16 heads over
// 261 (cut in two, two and one) 19.1, 19.1, 19.3; 1 x 16 over 1000 20.2, 20.1,
// 22.8; ragged 4 x 3 x 32 over 2000 24.8, 25.3, 29.0; 1 x 128 over 4096 26.2,
// 27.3, 29.7; over 16384 40.1, 39.0, 37.1; 1 x 16 over 65536 56.0, 55.7, 56.0.
constexpr int kMinUnits = 10;
// What a range may have above the even share for the tiles to stay whole.
constexpr int kWholeUnits = 16;
constexpr int kMaxEngines = 64;  // 148 SMs hold 37 clusters of four

__device__ __forceinline__ int engines_of(const ChunkParams& p, long long total) {
  const long long most = (total + kMinUnits - 1) / kMinUnits;
  return most < p.P ? static_cast<int>(most) : p.P;
}

// Tile holding unit x: the last t with pre[t] <= x that has units.
__device__ __forceinline__ int tile_of(const long long* pre, int nt, long long x) {
  int lo = 0, hi = nt;  // pre[lo] <= x < pre[hi]
  while (hi - lo > 1) {
    const int mid = (lo + hi) >> 1;
    if (pre[mid] <= x) lo = mid; else hi = mid;
  }
  return lo;
}

// Inlined, as are the roles: state passed by reference to a real call would
// live in local memory, whose cache next to 227 KB of shared memory holds a
// fraction of the threads' frames (measured: an L2 round trip per access, 6.5
// us instead of 4.9 us for a tile's output).
struct Walker {
  const ChunkParams* p;
  long long s, e, a0, z0;  // range; units of tile t0
  int4 tile0;
  int t, nt, t0, engine, count;

  __device__ __forceinline__ void init(const ChunkParams& pp, int engine_) {
    p = &pp;
    engine = engine_;
    count = 0;
    const ChunkEngine r = pp.engines[engine_];
    s = r.s;
    e = r.e;
    a0 = r.a;
    z0 = r.z;
    tile0 = r.tile;
    t = t0 = r.t;
    nt = r.nt;
  }

  __device__ __forceinline__ bool next(Seg& g) {
    for (; t < nt; ++t) {
      // the first tile came with the range: one load later saved
      const bool known = t == t0;
      const long long a = (known ? a0 : p->pre[t]) + kTileUnits, z = known ? z0 : p->pre[t + 1];
      const int4 info = known ? tile0 : p->tiles[t];
      if (a - kTileUnits >= e) return false;
      const long long lo = s > a ? s : a, hi = e < z ? e : z;
      if (lo >= hi) continue;  // no cached token, or none of its blocks in the range
      g.row0 = info.x;
      g.rows = info.y;
      g.b = info.z;
      g.len = info.w;
      g.blk_lo = static_cast<int>(lo - a);
      g.blk_hi = static_cast<int>(hi - a);
      g.slot = lo == a && hi == z ? -1 : 2 * engine + (count == 0 ? 0 : 1);
      ++count;
      ++t;
      return true;
    }
    return false;
  }
};

struct Ctx {
  const ChunkParams* p;
  uint32_t base;
  uint8_t* gbase;
  Barriers* bars;
  uint32_t tmem;
  WaitCtx wc;
  int engine, rank, warp, lane;
};

__device__ __forceinline__ uint32_t bar_addr(const uint64_t& b) { return smem_u32(&b); }

// An arrival (cluster address) that passes on what this thread has observed:
// bytes that other threads or copies have written or, for a slot that becomes
// free, have read.  It announces four bytes and sends them, so that the phase
// ends with the complete-tx of an st.async, which is a release at cluster scope
// issued behind this thread's own acquire.  An arrival with release semantics
// in its place costs about 0.5 us, as much as a block takes (512 tokens over
// 16384: 1.63 -> 2.1 ms); the four bytes do not show.  Hand-offs of TMEM are
// ordered by tcgen05.wait and the tcgen05 fences around a relaxed arrival.
__device__ __forceinline__ void arrive_with_word(uint32_t bar, uint32_t word, uint32_t v) {
  mbar_arrive_expect_tx_cluster_relaxed(bar, 4);
  st_async_b32(word, v, bar);
}

struct BlockCursor {
  const int32_t* row;
  int nblk, base, cached;
  // Fetches the segment's first ids at once, ahead of their use.
  __device__ __forceinline__ void reset(const ChunkParams& p, const Seg& g, int lane) {
    row = p.block_table + size_t(g.b) * p.max_blocks;
    nblk = nblocks_of(g.len);
    base = g.blk_lo;
    cached = (base + lane < nblk) ? row[base + lane] : -1;
  }
  __device__ __forceinline__ int id(int j, int lane) {
    if (j < base || j >= base + 32) {
      base = j;
      cached = (j + lane < nblk) ? row[j + lane] : -1;
    }
    return __shfl_sync(0xffffffffu, cached, j - base);
  }
};

// Valid rows of block j (0 for a bad id); *blk receives a block that is safe to load.
__device__ __forceinline__ int block_rows(const ChunkParams& p, const Seg& g, BlockCursor& cur, int j, int lane,
                                          int* blk) {
  const int id = cur.id(j, lane);
  const bool ok = id >= 0 && id < p.num_blocks;
  *blk = ok ? id : 0;
  const int nv = min(g.len - j * kBlock, kBlock);
  return ok ? nv : 0;
}

// ------------------------------------------------------------------ score pair

// The ring carries each segment's first eight chunks of Q, one per slot, then
// its passes' chunks of K, two per slot (a pass has nine, so a slot may hold
// the last of one pass and the first of the next).  One elected thread runs
// it: with whole-warp waits and loads issued by `lane == 0` a slot took 850
// cycles against the 512 of its MMAs, and this warp bound the whole kernel; with
// per-slot bookkeeping of passes and blocks in the one thread still 590 (of
// which the load is 40: it runs next to the softmax warps' code), so that the
// loops here are tight and a slot is one load of two chunks.
__device__ __forceinline__ void score_feed(const Ctx& c, const CUtensorMap* kmap, const CUtensorMap* kmap2, const CUtensorMap* qmap) {
  const ChunkParams& p = *c.p;
  Walker w;
  w.init(p, c.engine);
  Seg g;
  uint32_t slot = 0, parity = 1;
  const uint32_t full0 = map_to_rank(bar_addr(c.bars->k_full[0]), 0), empty0 = bar_addr(c.bars->k_empty[0]);
  prefetch_tmap(kmap);
  prefetch_tmap(kmap2);
  prefetch_tmap(qmap);
  // The slot is free; rank 0 announces the bytes of both CTAs (those of rank 1
  // may land first).
  auto open = [&](uint32_t bytes) {
    if (!spin_phase(empty0 + 8 * slot, parity, c.wc)) return false;
    if (c.rank == 0) mbar_arrive_expect_tx(bar_addr(c.bars->k_full[0]) + 8 * slot, 2 * bytes);
    return true;
  };
  auto advance = [&]() {
    if (++slot == kKSlots) {
      slot = 0;
      parity ^= 1u;
    }
  };
  // this CTA's block of the pass from j on: its own, or a masked copy of the
  // pass's only block, so that neither CTA's ring runs ahead; ids are read a
  // pair of passes early
  auto fetch = [&](const Seg& sg, int j) {
    if (j >= sg.blk_hi) return 0;
    return p.block_table[size_t(sg.b) * p.max_blocks + (j + c.rank < sg.blk_hi ? j + c.rank : j)];
  };
  auto row_of = [&](const Seg& sg, int id, int j) {
    const bool ok = id >= 0 && id < p.num_blocks;
    if (!ok && j + c.rank < sg.blk_hi) atomicOr(p.err, kErrBadBlock);
    return ok ? id * kBlock : 0;
  };
  // chunks ch, ch + 2, ch + 4 and ch + 6 of a pass with their successors
  auto four = [&](int row, int ch) {
#pragma unroll 1
    for (int end = ch + 8; ch < end; ch += 2) {
      if (!open(2 * kBlkChunk)) return false;
      pair_tma_load_3d(c.base + k_slot_off(0) + slot * kKSlot, kmap2, row, ch, full0 + 8 * slot);
      advance();
    }
    return true;
  };
  bool more = w.next(g);
  int id0 = 0, id1 = 0;
  if (more) {
    id0 = fetch(g, g.blk_lo);
    id1 = fetch(g, g.blk_lo + kPassBlocks);
  }
  while (more) {
#pragma unroll 1
    for (int ch = 0; ch < kQTmem; ++ch) {
      if (!open(kQChunk)) return;
      // rows past the tile belong to other tokens (or read as zeros): their
      // scores are masked
      pair_tma_load_2d(c.base + k_slot_off(0) + slot * kKSlot, qmap, 64 * ch, g.row0 + 128 * c.rank, full0 + 8 * slot);
      advance();
    }
    Seg gn = g;
    int n0 = 0, n1 = 0;
    // two passes fill nine slots, the middle one with a chunk of each
    for (int j = g.blk_lo; j < g.blk_hi; j += 2 * kPassBlocks) {
      const bool two = j + kPassBlocks < g.blk_hi;
      const int row0 = row_of(g, id0, j), row1 = two ? row_of(g, id1, j + kPassBlocks) : 0;
      id0 = fetch(g, j + 2 * kPassBlocks);
      id1 = fetch(g, j + 3 * kPassBlocks);
      if (!four(row0, 0)) return;
      if (!open(two ? 2 * kBlkChunk : kBlkChunk)) return;
      const uint32_t dst = c.base + k_slot_off(0) + slot * kKSlot;
      pair_tma_load_2d(dst, kmap, 64 * (kChunks - 1), row0, full0 + 8 * slot);
      if (two) pair_tma_load_2d(dst + kBlkChunk, kmap, 0, row1, full0 + 8 * slot);
      advance();
      if (two && !four(row1, 1)) return;
      if (j == g.blk_lo) {  // the next segment's records, while the ring is full
        more = w.next(gn);
        if (more) {
          n0 = fetch(gn, gn.blk_lo);
          n1 = fetch(gn, gn.blk_lo + kPassBlocks);
        }
      }
    }
    g = gn;
    id0 = n0;
    id1 = n1;
  }
}

// The last chunk of Q.
__device__ __forceinline__ void score_tma_q(const Ctx& c, const CUtensorMap* qmap) {
  const ChunkParams& p = *c.p;
  Walker w;
  w.init(p, c.engine);
  Seg g;
  uint32_t seg = 0;
  const uint32_t full = map_to_rank(bar_addr(c.bars->q_full), 0);
  while (w.next(g)) {
    if (!warp_wait(bar_addr(c.bars->q_empty), (seg & 1u) ^ 1u, c.wc)) return;
    if (c.lane == 0) {
      if (c.rank == 0) mbar_arrive_expect_tx(bar_addr(c.bars->q_full), 2 * kQChunk);
      pair_tma_load_2d(c.base + kQOff, qmap, 64 * kQTmem, g.row0 + 128 * c.rank, full);
    }
    __syncwarp();
    ++seg;
  }
}

// The elected thread of rank 0.  The barrier of the next slot is probed before
// the current slot's last MMAs are issued: a probe behind them would wait for
// their issue and leave the pipe idle meanwhile.
struct Feed {
  uint32_t full0, empty0;  // barriers of slot 0
  uint64_t k0;             // descriptor of slot 0
  uint32_t slot, phase;
  bool ready;

  __device__ __forceinline__ bool wait(const Ctx& c) {
    return ready || spin_phase(full0 + 8 * slot, phase, c.wc);
  }
  __device__ __forceinline__ void next() {
    if (++slot == kKSlots) {
      slot = 0;
      phase ^= 1u;
    }
    ready = mbar_test_wait(full0 + 8 * slot, phase);
  }
};

// One pass.  kOdd: its first chunk is the second one of a slot.
template <bool kOdd>
__device__ __forceinline__ bool score_mma_pass(const Ctx& c, Feed& f, uint32_t d, bool first, bool last, uint32_t seg) {
  const uint32_t q = c.tmem + kTmemQ;
  const uint64_t q8 = sw128_desc(c.base + kQOff, 16, 1024);
#pragma unroll
  for (int ch = 0; ch < kChunks; ++ch) {
    const bool second = ((ch + kOdd) & 1) != 0;
    if (!second && !f.wait(c)) return false;
    const uint32_t s = f.slot;
    const uint64_t kd = f.k0 + s * (kKSlot >> 4) + (second ? kBlkChunk >> 4 : 0);
    const bool done = second || (ch == kChunks - 1 && last);
    if (done) f.next();
    if (ch < kQTmem) {
#pragma unroll
      for (int kk = 0; kk < 4; ++kk)
        pair_mma_ts(d, q + 32 * ch + 8 * kk, kd + 2 * kk, kIdescQK, (ch | kk) ? 1u : 0u);
    } else {
      if (first && !spin_phase(bar_addr(c.bars->q_full), seg & 1u, c.wc)) return false;
#pragma unroll
      for (int kk = 0; kk < 4; ++kk) pair_mma_ss(d, q8 + 2 * kk, kd + 2 * kk, kIdescQK, 1u);
      if (last) pair_commit(bar_addr(c.bars->q_empty), kScoreMask);
    }
    if (done) pair_commit(f.empty0 + 8 * s, kScoreMask);
  }
  return true;
}

__device__ __forceinline__ bool score_mma_segment(const Ctx& c, const Seg& g, uint32_t seg, Feed& f, uint32_t& pit) {
  Barriers* bars = c.bars;
  // Q moves to TMEM once the MMAs that read the last segment's have finished
  if (pit > 0 && !spin_phase(bar_addr(bars->s_full[(pit - 1) & 1u]), ((pit - 1) >> 1) & 1u, c.wc)) return false;
  tc_fence_after();
#pragma unroll 1
  for (int ch = 0; ch < kQTmem; ++ch) {
    if (!f.wait(c)) return false;
    const uint64_t qd = f.k0 + f.slot * (kKSlot >> 4);
    const uint32_t s = f.slot, d = c.tmem + kTmemQ + 32 * ch;
    f.next();
#pragma unroll
    for (int kk = 0; kk < 4; ++kk) pair_cp_128x32b(d + 8 * kk, qd + 2 * kk);
    pair_commit(f.empty0 + 8 * s, kScoreMask);
  }
  bool odd = false;
  for (int j = g.blk_lo; j < g.blk_hi; j += kPassBlocks, ++pit, odd = !odd) {
    const bool first = j == g.blk_lo, last = j + kPassBlocks >= g.blk_hi;
    const uint32_t d = c.tmem + 128 * (pit & 1u);
    if (!spin_phase(bar_addr(bars->s_empty[pit & 1u]), ((pit >> 1) & 1u) ^ 1u, c.wc)) return false;
    tc_fence_after();
    if (!(odd ? score_mma_pass<true>(c, f, d, first, last, seg) : score_mma_pass<false>(c, f, d, first, last, seg)))
      return false;
    pair_commit(bar_addr(bars->s_full[pit & 1u]), kScoreMask);
  }
  return true;
}

__device__ __forceinline__ void score_mma(const Ctx& c) {
  if (elect_one()) {
    Walker w;
    w.init(*c.p, c.engine);
    Seg g;
    Feed f{bar_addr(c.bars->k_full[0]), bar_addr(c.bars->k_empty[0]), sw128_desc(c.base + k_slot_off(0), 16, 1024),
           0u, 0u, false};
    uint32_t pit = 0, seg = 0;
    while (w.next(g) && score_mma_segment(c, g, seg, f, pit)) ++seg;
  }
  __syncwarp();
}

// Publish one float per row to the other half's warp of the same rows.
__device__ __forceinline__ float ld_shared(uint32_t at) {
  float v;
  asm volatile("ld.shared.f32 %0, [%1];" : "=f"(v) : "r"(at) : "memory");
  return v;
}
__device__ __forceinline__ void publish(uint32_t bar, uint32_t at, float v, int lane) {
  asm volatile("st.shared.f32 [%0], %1;" ::"r"(at), "f"(v) : "memory");
  __syncwarp();
  if (lane == 0) mbar_arrive(bar);
}

// Thread = row; the four warps of a half take every other pass, so that one
// half's exponentials overlap the other's loads and waits.  The running
// maximum passes from pass to pass through shared memory; each half sums its
// own passes, and the segment's last pass joins the two sums.
__device__ __forceinline__ void score_softmax(const Ctx& c) {
  const ChunkParams& p = *c.p;
  const int q4 = c.warp & 3;                                  // TMEM lane quadrant
  const uint32_t half = static_cast<uint32_t>(c.warp - 4) >> 2;  // S buffer, parity of its passes
  const int h = q4 * 32 + c.lane;                             // row of this CTA
  const uint32_t s_addr = c.tmem + (static_cast<uint32_t>(q4 * 32) << 16) + 128 * half;
  // a zero scale (uniform attention) runs as a tiny one, so that a masked
  // score (-inf) still gives exactly 0
  const float sl2 = p.softmax_scale != 0.f ? p.softmax_scale * kLog2e : 1e-30f;
  const bool pos = sl2 >= 0.f;
  const float sg = pos ? 1.f : -1.f;
  const uint32_t to = static_cast<uint32_t>(c.rank) + 2;
  const uint32_t rec0 = map_to_rank(c.base + rec_off(0), to);
  const uint32_t pfull0 = map_to_rank(bar_addr(c.bars->p_full[0]), to);
  const uint32_t sempty = map_to_rank(bar_addr(c.bars->s_empty[half]), 0);
  // this half's published values and its barriers
  const uint32_t maxima = c.base + kMaxOff + 512 * half + 4 * h, sums = maxima + (kSumOff - kMaxOff);
  const uint32_t m_set = bar_addr(c.bars->m_set[half][q4]), l_set = bar_addr(c.bars->l_set[half][q4]);
  const uint32_t other = half ? 0u - 512u : 512u, other_bar = half ? 0u - 32u : 32u;
  Walker w;
  w.init(p, c.engine);
  Seg g;
  BlockCursor cur;
  uint32_t it = 0, pit = 0, joined = 0;
  while (w.next(g)) {
    cur.reset(p, g, c.lane);
    // this row's query token sees the tile's length without its last
    // tokens' rows; padding rows see nothing
    const int row = 128 * c.rank + h;
    const int row_len = row < g.rows ? g.len - (g.rows - 1 - row) / p.H : 0;
    float m_ref = -INFINITY, l = 0.f;
    for (int j0 = g.blk_lo; j0 < g.blk_hi; j0 += kPassBlocks, ++pit) {
      const int nb = min(kPassBlocks, g.blk_hi - j0);
      if ((pit & 1u) != half) {
        it += static_cast<uint32_t>(nb);
        continue;
      }
      const bool first_pass = j0 == g.blk_lo, last_pass = j0 + kPassBlocks >= g.blk_hi;
      int nvr[2];
#pragma unroll
      for (int k = 0; k < 2; ++k) {
        int blk;
        const int nv = block_rows(p, g, cur, k < nb ? j0 + k : j0, c.lane, &blk);
        nvr[k] = k < nb ? max(0, min(nv, row_len - (j0 + k) * kBlock)) : 0;
      }
      if (!warp_wait(bar_addr(c.bars->s_full[half]), (pit >> 1) & 1u, c.wc)) return;
      tc_fence_after();
      uint32_t sv[128];
#pragma unroll
      for (int q = 0; q < 4; ++q) tmem_ld32(s_addr + 32 * q, *reinterpret_cast<uint32_t(*)[32]>(&sv[32 * q]));
      tmem_ld_wait();
      tc_fence_before();
      __syncwarp();
      if (c.lane == 0) mbar_arrive_cluster_relaxed(sempty);  // the loads are in registers

      // masked columns take the score -sg * inf, which no max selects and
      // whose exponential is exactly 0
      if (!__all_sync(0xffffffffu, nvr[0] == kBlock && nvr[1] == kBlock)) {
        const uint32_t masked = __float_as_uint(-INFINITY * sg);
#pragma unroll
        for (int t = 0; t < 128; ++t)
          if ((t & 63) >= nvr[t >> 6]) sv[t] = masked;
      }
      float mr;
      if (pos) {
        float mv[4] = {-INFINITY, -INFINITY, -INFINITY, -INFINITY};
#pragma unroll
        for (int t = 0; t < 128; t += 8)
#pragma unroll
          for (int u = 0; u < 4; ++u)
            mv[u] = fmax3(mv[u], __uint_as_float(sv[t + 2 * u]), __uint_as_float(sv[t + 2 * u + 1]));
        mr = fmax3(fmaxf(mv[0], mv[1]), mv[2], mv[3]);
      } else {
        float mv[4] = {INFINITY, INFINITY, INFINITY, INFINITY};
#pragma unroll
        for (int t = 0; t < 128; t += 8)
#pragma unroll
          for (int u = 0; u < 4; ++u)
            mv[u] = fmin3(mv[u], __uint_as_float(sv[t + 2 * u]), __uint_as_float(sv[t + 2 * u + 1]));
        mr = -fmin3(fminf(mv[0], mv[1]), mv[2], mv[3]);
      }
      const float mx = (nvr[0] | nvr[1]) ? mr * sg * sl2 : -INFINITY;
      // the maximum after the pass before (another segment's is not used, but
      // every publication is waited for, so that none is two phases behind)
      float m_prev = -INFINITY;
      if (pit > 0) {
        if (!warp_wait(m_set + other_bar, ((pit - 1) >> 1) & 1u, c.wc)) return;
        if (!first_pass) m_prev = ld_shared(maxima + other);
      }
      const float m_sum = m_ref;  // l is relative to this one
      float alpha = 1.f;
      bool resc = false;
      if (first_pass) {
        m_ref = mx;
      } else if (mx > m_prev + kRescaleThreshold) {
        alpha = (m_prev == -INFINITY) ? 0.f : ex2_approx(m_prev - mx);
        m_ref = mx;
        resc = true;
      } else {
        m_ref = m_prev;
      }
      // a last pass's maximum serves nobody: it is published when the sums
      // have been read
      if (!last_pass) publish(m_set, maxima, m_ref, c.lane);
      if (m_sum != m_ref) l *= (m_sum == -INFINITY) ? 0.f : ex2_approx(m_sum - m_ref);
      const float neg_m = m_ref == -INFINITY ? 0.f : -m_ref;
      const unsigned any = __any_sync(0xffffffffu, resc);
#pragma unroll
      for (int k = 0; k < 2; ++k) {
        if (k >= nb) continue;
        const uint32_t ib = it + static_cast<uint32_t>(k);
        const int r = ib % kNP;
        if (!warp_wait(bar_addr(c.bars->p_empty[r]), ((ib / kNP) & 1u) ^ 1u, c.wc)) return;
        const uint32_t full = pfull0 + 8 * r;
        const uint32_t rec = rec0 + r * kRecBytes;
        // one arrival per warp announces its bytes: each lane's P row, for a
        // pass's first block and the segment's last its factors, a flag
        const bool meta = k == 0 || (last_pass && k == nb - 1);
        if (c.lane == 0) mbar_arrive_expect_tx_cluster_relaxed(full, 32 * (128 + (meta ? 16 : 0)) + 4);
        float sum0 = 0.f, sum1 = 0.f;
#pragma unroll
        for (int tp = 0; tp < 4; ++tp) {
          uint32_t pk[2][4];
#pragma unroll
          for (int u = 0; u < 2; ++u)
#pragma unroll
            for (int e = 0; e < 4; ++e) {
              const int t = 64 * k + 16 * tp + 8 * u + 2 * e;
              const float e0 = ex2_approx(fmaf(__uint_as_float(sv[t]), sl2, neg_m));
              const float e1 = ex2_approx(fmaf(__uint_as_float(sv[t + 1]), sl2, neg_m));
              sum0 += e0;
              sum1 += e1;
              __nv_bfloat162 b2 = __floats2bfloat162_rn(e0, e1);
              pk[u][e] = *reinterpret_cast<uint32_t*>(&b2);
            }
#pragma unroll
          for (int u = 0; u < 2; ++u)
            st_async_v4(rec + (2 * tp + u) * kPCoreK + h * 16, make_uint4(pk[u][0], pk[u][1], pk[u][2], pk[u][3]),
                        full);
        }
        l += sum0 + sum1;
        if (c.lane == 0) st_async_b32(rec + kPBytes + kMetaBytes + q4 * 4, (k == 0 && any) ? 1u : 0u, full);
        if (k == 0 && !(last_pass && nb == 1))
          st_async_v4(rec + kPBytes + h * 16, make_uint4(__float_as_uint(alpha), __float_as_uint(m_ref), 0u, 0u), full);
      }
      it += static_cast<uint32_t>(nb);
      if (!last_pass) {
        if (j0 + 2 * kPassBlocks >= g.blk_hi) publish(l_set, sums, l, c.lane);
        continue;
      }
      float ltot = l;
      if (!first_pass) {  // the other half's sum, relative to the maximum after its last pass
        if (!warp_wait(l_set + other_bar, joined & 1u, c.wc)) return;
        ++joined;
        const float lo = ld_shared(sums + other);
        ltot += m_prev == m_ref ? lo : lo * ((m_prev == -INFINITY) ? 0.f : ex2_approx(m_prev - m_ref));
      }
      publish(m_set, maxima, m_ref, c.lane);
      const int r = (it - 1) % kNP;
      st_async_v4(rec0 + r * kRecBytes + kPBytes + h * 16,
                  make_uint4(__float_as_uint(nb == 1 ? alpha : 1.f), __float_as_uint(m_ref), __float_as_uint(ltot), 0u),
                  pfull0 + 8 * r);
    }
  }
}

// ------------------------------------------------------------------ value pair

// One elected thread, as score_feed.
__device__ __forceinline__ void value_feed(const Ctx& c, const CUtensorMap* kmap4) {
  const ChunkParams& p = *c.p;
  Walker w;
  w.init(p, c.engine);
  Seg g;
  uint32_t slot = 0, parity = 1;
  const int chunk0 = 4 * (c.rank - 2);  // this CTA's half of the latent
  prefetch_tmap(kmap4);
  auto fetch = [&](const Seg& sg, int j) { return p.block_table[size_t(sg.b) * p.max_blocks + j]; };
  bool more = w.next(g);
  // ids are read two blocks early
  int id0 = more ? fetch(g, g.blk_lo) : 0, id1 = more && g.blk_lo + 1 < g.blk_hi ? fetch(g, g.blk_lo + 1) : 0;
  while (more) {
    Seg gn = g;
    int n0 = 0, n1 = 0;
    for (int j = g.blk_lo; j < g.blk_hi; ++j) {
      const int id = id0;
      id0 = id1;
      if (j + 2 < g.blk_hi) id1 = fetch(g, j + 2);
      if (j == g.blk_lo) {
        more = w.next(gn);
        if (more) {
          n0 = fetch(gn, gn.blk_lo);
          if (gn.blk_lo + 1 < gn.blk_hi) n1 = fetch(gn, gn.blk_lo + 1);
        }
      }
      const int row = id >= 0 && id < p.num_blocks ? id * kBlock : 0;
      if (!spin_phase(bar_addr(c.bars->v_empty[0]) + 8 * slot, parity, c.wc)) return;
      const uint32_t full = bar_addr(c.bars->v_full[0]) + 8 * slot;
      mbar_arrive_expect_tx(full, kVSlot);
      const uint32_t dst = c.base + v_slot_off(0) + slot * kVSlot;
      tma_load_chunks(dst, kmap4, row, chunk0, full);
      if (++slot == kVSlots) {
        slot = 0;
        parity ^= 1u;
      }
    }
    g = gn;
    id0 = n0;
    id1 = n1;
  }
}

__device__ __forceinline__ uint32_t finite_or_zero(uint32_t two) {
  if ((two & 0x7f80u) == 0x7f80u) two &= 0xffff0000u;
  if ((two & 0x7f800000u) == 0x7f800000u) two &= 0x0000ffffu;
  return two;
}

// Rows past the tile's length are zeroed, so that whatever the cache holds
// there (even NaN) contributes exactly 0 * 0.  Rows that the tile's last
// token sees and its first does not lose their infinities and NaN, because a
// token that does not see such a row (P = 0) must not meet 0 * NaN.  One that
// sees it loses nothing that counts: with a NaN or +inf score its probability
// is NaN, and so is all of its output; with a -inf score its probability is 0
// and the row drops out, except that in rows which every token sees, and which
// are not searched for infinities here, 0 * inf makes the infinite columns NaN.
__device__ __forceinline__ void value_fixup(const Ctx& c) {
  const ChunkParams& p = *c.p;
  Walker w;
  w.init(p, c.engine);
  Seg g;
  BlockCursor cur;
  uint32_t vit = 0;
  const uint32_t ready0 = map_to_rank(bar_addr(c.bars->v_ready[0]), 2), sink = map_to_rank(smem_u32(&c.bars->sink), 2);
  while (w.next(g)) {
    cur.reset(p, g, c.lane);
    const int all_see = g.len - (g.rows - 1) / p.H;  // tokens that every row of the tile sees
    for (int j = g.blk_lo; j < g.blk_hi; ++j, ++vit) {
      int blk;
      const int nv = block_rows(p, g, cur, j, c.lane, &blk);
      const int s = vit % kVSlots;
      if (!warp_wait(bar_addr(c.bars->v_full[s]), (vit / kVSlots) & 1u, c.wc)) return;
      const int from = max(0, min(nv, all_see - j * kBlock));
      if (from < kBlock) {
        // eight lanes per 128-byte row of a chunk
        uint8_t* st = c.gbase + v_slot_off(s) + (c.lane & 7) * 16;
        for (int row = from + (c.lane >> 3); row < kBlock; row += 4) {
#pragma unroll
          for (int ch = 0; ch < 4; ++ch) {
            uint4* at = reinterpret_cast<uint4*>(st + ch * kBlkChunk + row * 128);
            uint4 v = make_uint4(0, 0, 0, 0);
            if (row < nv) {
              v = *at;
              v = make_uint4(finite_or_zero(v.x), finite_or_zero(v.y), finite_or_zero(v.z), finite_or_zero(v.w));
            }
            *at = v;
          }
        }
        fence_proxy_async_smem();
      }
      __syncwarp();
      if (c.lane == 0) {
        // the zeros are this warp's own writes (from rank 2 to itself too: a plain
        // arrival there made the smallest call 0.4 us longer)
        if (from < kBlock)
          mbar_arrive_remote(bar_addr(c.bars->v_ready[s]), 2);
        else
          arrive_with_word(ready0 + 8 * s, sink, 0u);
      }
    }
  }
}

// Each value CTA tells rank 2's MMA thread that its P record landed, and
// whether a row of it asks for a rescale.  P was written by asynchronous
// stores of the score CTA: the proxy fence here makes it visible to the MMAs,
// off the issuing thread's path.
__device__ __forceinline__ void value_relay(const Ctx& c) {
  Walker w;
  w.init(*c.p, c.engine);
  Seg g;
  uint32_t it = 0;
  const uint32_t ready0 = map_to_rank(bar_addr(c.bars->p_ready[0]), 2);
  const uint32_t flag0 = map_to_rank(smem_u32(&c.bars->flag[0][c.rank - 2]), 2);
  while (w.next(g)) {
    int ok = 1;
    if (c.lane == 0) {
      for (int j = g.blk_lo; j < g.blk_hi; ++j, ++it) {
        const int r = it % kNP;
        if (!spin_phase(bar_addr(c.bars->p_full[r]), (it / kNP) & 1u, c.wc)) {
          ok = 0;
          break;
        }
        const uint4 f = *reinterpret_cast<const uint4*>(c.gbase + rec_off(r) + kPBytes + kMetaBytes);
        fence_proxy_async_smem();
        arrive_with_word(ready0 + 8 * r, flag0 + 8 * r, f.x | f.y | f.z | f.w);
      }
    }
    if (!__shfl_sync(0xffffffffu, ok, 0)) return;
  }
}

constexpr uint32_t kReqFinal = 0x80000000u;

// Posts a request to the epilogue warps of both CTAs: the word, an arrival,
// and a commit (the MMAs issued so far are done).
__device__ __forceinline__ void post_request(const Ctx& c, uint32_t req) {
  *reinterpret_cast<volatile uint32_t*>(&c.bars->req) = req;
  st_cluster_b32(map_to_rank(smem_u32(&c.bars->req), 3), req);
  mbar_arrive(bar_addr(c.bars->epi_req));
  mbar_arrive_remote(bar_addr(c.bars->epi_req), 3);
  pair_commit(bar_addr(c.bars->epi_req), kValueMask);
}

// The elected thread of rank 2; the next block's barriers are probed before
// the current block's MMAs are issued.
__device__ __forceinline__ bool value_mma_segment(const Ctx& c, const Seg& g, uint32_t seg, uint32_t& it, uint32_t& ncorr) {
  Barriers* bars = c.bars;
  const uint64_t p0 = plain_desc(c.base + rec_off(0), kPCoreK, 128);
  const uint64_t v0 = sw128_desc(c.base + v_slot_off(0), kBlkChunk, 1024);
  if (seg > 0) {
    if (!spin_phase(bar_addr(bars->o_free), (seg - 1) & 1u, c.wc)) return false;
    tc_fence_after();
  }
  bool p_ok = false, v_ok = false;
  for (int j = g.blk_lo; j < g.blk_hi; ++j, ++it) {
    const uint32_t r = it % kNP, s = it % kVSlots;
    const bool first = (j == g.blk_lo), last = (j == g.blk_hi - 1);
    if (!p_ok && !spin_phase(bar_addr(bars->p_ready[r]), (it / kNP) & 1u, c.wc)) return false;
    const uint32_t flags = *reinterpret_cast<volatile uint32_t*>(&bars->flag[r][0]) |
                           *reinterpret_cast<volatile uint32_t*>(&bars->flag[r][1]);
    if (flags && !first) {
      post_request(c, r);
      if (!wait_phase(bar_addr(bars->corr_done), ncorr & 1u, c.wc)) return false;
      ++ncorr;
      tc_fence_after();
    }
    if (!v_ok && !spin_phase(bar_addr(bars->v_ready[s]), (it / kVSlots) & 1u, c.wc)) return false;
    const uint32_t nx = it + 1;
    p_ok = mbar_test_wait(bar_addr(bars->p_ready[nx % kNP]), (nx / kNP) & 1u);
    v_ok = mbar_test_wait(bar_addr(bars->v_ready[nx % kVSlots]), (nx / kVSlots) & 1u);
    const uint64_t pd = p0 + r * (kRecBytes >> 4), vd = v0 + s * (kVSlot >> 4);
#pragma unroll
    for (int n = 0; n < 2; ++n)
#pragma unroll
      for (int k = 0; k < kBlock / 16; ++k)
        pair_mma_ss(c.tmem + 256 * n, pd + k * (2 * kPCoreK >> 4), vd + (2 * n * kBlkChunk >> 4) + k * (2048 >> 4),
                    kIdescPV, (k > 0 || !first) ? 1u : 0u);
    pair_commit(bar_addr(bars->v_empty[s]), kValueMask);
    if (last)
      post_request(c, kReqFinal | r);  // the epilogues release the record
    else
      pair_commit(bar_addr(bars->p_empty[r]), kScoreMask);
  }
  return true;
}

__device__ __forceinline__ void value_mma(const Ctx& c) {
  if (elect_one()) {
    Walker w;
    w.init(*c.p, c.engine);
    Seg g;
    uint32_t it = 0, seg = 0, ncorr = 0;
    while (w.next(g) && value_mma_segment(c, g, seg, it, ncorr)) ++seg;
  }
  __syncwarp();
}

// Latent column of TMEM column c: every MMA's N = 256 columns are 128 of each
// CTA's half.
__device__ __forceinline__ int latent_of(int c) { return 256 * ((c >> 7) & 1) + 128 * (c >> 8) + (c & 127); }

// A piece's output is kept by columns, four floats of one row next to those of
// the next row ([slot][512 / 4][256 rows][4]): a warp, whose lanes are rows,
// then stores 512 contiguous bytes at a time, and the merge reads so too.
__device__ __forceinline__ size_t piece_unit(int slot, int col4, int row) {
  return (size_t(slot) * (kDc / 4) + col4) * kTileRows + row;
}

// Writes 128 bytes of each of the warp's 32 rows (lane = row, v = its bytes):
// turned around in shared memory, 16 rows at a time, so that a store of the
// warp fills four whole lines.  The time of a store goes with the lines it
// touches (measured for a tile's output: 7 us when every lane stores its own
// row, 2.3-5 us with eight 64-byte pieces a store).  16-byte units are swizzled
// against bank conflicts.  `dst` is where lane l's 16 bytes of row l / 8 go;
// rows are kDc elements apart, and `rows` of them from that one on exist.
__device__ __forceinline__ void store_rows(uint8_t* stage, int lane, const uint4 (&a)[4], const uint4 (&b)[4], uint8_t* dst,
                                           int rows) {
  uint8_t* const to = stage + (lane & 15) * 128;
  const uint8_t* const from = stage + (lane >> 3) * 128;
#pragma unroll
  for (int half = 0; half < 2; ++half) {
    __syncwarp();
    if ((lane >> 4) == half) {
#pragma unroll
      for (int q = 0; q < 8; ++q) *reinterpret_cast<uint4*>(to + ((q ^ (lane & 7)) << 4)) = q < 4 ? a[q & 3] : b[q & 3];
    }
    __syncwarp();
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const int r = 16 * half + 4 * i;  // and lane / 8; swizzled by the row's place in its group of eight
      if (r < rows)
        *reinterpret_cast<uint4*>(dst + r * (kDc * 2)) = *reinterpret_cast<const uint4*>(
            from + 4 * i * 128 + (((lane & 7) ^ ((4 * i + (lane >> 3)) & 7)) << 4));
    }
  }
}

// Thread = (row, half of the TMEM columns).
__device__ __forceinline__ void value_epilogue(const Ctx& c) {
  const ChunkParams& p = *c.p;
  const int q4 = c.warp & 3;
  const int half = (c.warp - 4) >> 2;
  const int h = q4 * 32 + c.lane;
  const int row = 128 * (c.rank - 2) + h;
  const uint32_t lane_off = static_cast<uint32_t>(q4 * 32) << 16;
  const uint32_t ocol = 256 * half;
  const uint32_t corr_done = map_to_rank(bar_addr(c.bars->corr_done), 2);
  const uint32_t o_free = map_to_rank(bar_addr(c.bars->o_free), 2);
  const uint32_t pempty0 = map_to_rank(bar_addr(c.bars->p_empty[0]), c.rank - 2);
  const uint32_t sink = map_to_rank(smem_u32(&c.bars->sink), c.rank - 2);
  Walker w;
  w.init(p, c.engine);
  Seg g;
  uint32_t nreq = 0, nfinal = 0;
  while (w.next(g)) {
    for (;;) {
      if (!warp_wait(bar_addr(c.bars->epi_req), nreq & 1u, c.wc)) return;
      ++nreq;
      tc_fence_after();
      const uint32_t req = *reinterpret_cast<volatile uint32_t*>(&c.bars->req);
      const uint8_t* rec = c.gbase + rec_off(static_cast<int>(req & 0xffu));
      const float4 meta = *reinterpret_cast<const float4*>(rec + kPBytes + h * 16);
      if (!(req & kReqFinal)) {
        const float alpha = meta.x;
        if (__any_sync(0xffffffffu, alpha != 1.f)) {
#pragma unroll 1
          for (int ch = 0; ch < 8; ++ch) {
            uint32_t v[32];
            tmem_ld32(c.tmem + lane_off + ocol + 32 * ch, v);
            tmem_ld_wait();
#pragma unroll
            for (int t = 0; t < 32; ++t) v[t] = __float_as_uint(__uint_as_float(v[t]) * alpha);
            tmem_st32(c.tmem + lane_off + ocol + 32 * ch, v);
          }
          tmem_st_wait();
        }
        tc_fence_before();
        __syncwarp();
        if (c.lane == 0) mbar_arrive_cluster_relaxed(corr_done);
        continue;
      }
      const float m_fin = meta.y, l_fin = meta.z;
      __syncwarp();
      if (c.lane == 0) mbar_arrive(bar_addr(c.bars->meta_done));
      // the record goes back to the score CTA once all eight warps have read it
      auto release_record = [&]() {
        if (c.warp != 4) return true;
        if (!warp_wait(bar_addr(c.bars->meta_done), nfinal & 1u, c.wc)) return false;
        if (c.lane == 0) arrive_with_word(pempty0 + 8 * (req & 0xffu), sink, 0u);
        return true;
      };
      const bool live = row < g.rows;
      const float inv = l_fin > 0.f ? 1.f / l_fin : (l_fin == 0.f ? 0.f : l_fin);  // a NaN sum stays NaN
      const float lse = l_fin == 0.f ? -INFINITY : (m_fin + log2f(l_fin)) * 0.6931471805599453f;
      uint8_t* stage = c.gbase + stage_off(c.warp - 4);
      const int row0 = 128 * (c.rank - 2) + q4 * 32;  // the warp's first row
      if (!release_record()) return;
      const bool any_row = row0 < g.rows;  // padding warps only hand O back
      if (g.slot < 0) {
        // A loop: unrolled, with all of the row's half in registers before the
        // first store, a tile's output took 4.1 us against 3.2, most of it for
        // fetching instructions.  The next columns are read while these are
        // stored, so that O is free two steps before the end (512 tokens over
        // 512, eight short tiles an engine: 86.6 -> 81.0 us).
        uint32_t v[2][32];
        auto read = [&](int ch) {
          tmem_ld32(c.tmem + lane_off + ocol + 32 * ch, v[0]);
          tmem_ld32(c.tmem + lane_off + ocol + 32 * ch + 32, v[1]);
        };
        uint8_t* const out = reinterpret_cast<uint8_t*>(p.out + (size_t(g.row0) + row0 + (c.lane >> 3)) * kDc) + 16 * (c.lane & 7);
        const int rows = g.rows - row0 - (c.lane >> 3);
        if (any_row) {
          read(0);
          tmem_ld_wait();
        }
#pragma unroll 1
        for (int ch = 0; ch < 8; ch += 2) {
          uint4 o[2][4];
#pragma unroll
          for (int k = 0; k < 2; ++k) {
#pragma unroll
            for (int q = 0; q < 4; ++q) {
              uint32_t w4[4];
#pragma unroll
              for (int e = 0; e < 4; ++e) {
                __nv_bfloat162 b2 = __floats2bfloat162_rn(__uint_as_float(v[k][8 * q + 2 * e]) * inv,
                                                          __uint_as_float(v[k][8 * q + 2 * e + 1]) * inv);
                w4[e] = *reinterpret_cast<uint32_t*>(&b2);
              }
              o[k][q] = make_uint4(w4[0], w4[1], w4[2], w4[3]);
            }
          }
          if (ch < 6 && any_row) read(ch + 2);
          if (ch == 4 || !any_row) {  // the last columns are in registers
            tmem_ld_wait();
            tc_fence_before();
            __syncwarp();
            if (c.lane == 0) mbar_arrive_cluster_relaxed(o_free);
          }
          if (!any_row) break;
          store_rows(stage, c.lane, o[0], o[1], out + 2 * latent_of(ocol + 32 * ch), rows);
          if (ch < 4) tmem_ld_wait();
        }
      } else {
#pragma unroll 1
        for (int ch = 0; any_row && ch < 8; ++ch) {
          __syncwarp();
          uint32_t v[32];
          tmem_ld32(c.tmem + lane_off + ocol + 32 * ch, v);
          tmem_ld_wait();
          if (!live) continue;
          float4* dst = reinterpret_cast<float4*>(p.o_part) + piece_unit(g.slot, latent_of(ocol + 32 * ch) / 4, row);
#pragma unroll
          for (int q = 0; q < 8; ++q)
            dst[q * kTileRows] = make_float4(__uint_as_float(v[4 * q]) * inv, __uint_as_float(v[4 * q + 1]) * inv,
                                             __uint_as_float(v[4 * q + 2]) * inv, __uint_as_float(v[4 * q + 3]) * inv);
        }
        tc_fence_before();
        __syncwarp();
        if (c.lane == 0) mbar_arrive_cluster_relaxed(o_free);
      }
      ++nfinal;
      if (live && half == 0) {
        if (g.slot < 0)
          p.lse[size_t(g.row0) + row] = lse;
        else
          p.lse_part[size_t(g.slot) * kTileRows + row] = lse;
      }
      break;
    }
  }
}

// ------------------------------------------------------------------ kernels

__global__ void __cluster_dims__(4, 1, 1) __launch_bounds__(kThreads, 1)
chunk_sm100_kernel(const __grid_constant__ ChunkMaps maps,
                   const ChunkParams p) {
  extern __shared__ __align__(1024) uint8_t smem_raw[];
  const uint32_t base = smem_u32(smem_raw);
  Barriers* bars = reinterpret_cast<Barriers*>(smem_raw);
  const int rank = static_cast<int>(cluster_ctarank());
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;

  if (threadIdx.x == 0) {
    for (int s = 0; s < kKSlots; ++s) {
      mbar_init(bar_addr(bars->k_full[s]), 1);
      mbar_init(bar_addr(bars->k_empty[s]), 1);
    }
    mbar_init(bar_addr(bars->q_full), 1);
    mbar_init(bar_addr(bars->q_empty), 1);
    for (int s = 0; s < 2; ++s) {
      mbar_init(bar_addr(bars->s_full[s]), 1);
      mbar_init(bar_addr(bars->s_empty[s]), 8);    // four softmax warps of two CTAs
      for (int q = 0; q < 4; ++q) {
        mbar_init(bar_addr(bars->m_set[s][q]), 1);
        mbar_init(bar_addr(bars->l_set[s][q]), 1);
      }
    }
    for (int r = 0; r < kNP; ++r) {
      mbar_init(bar_addr(bars->p_empty[r]), 1);    // PV commit, or the epilogue (segment end)
      mbar_init(bar_addr(bars->p_full[r]), 4);     // the four softmax warps of one half
      mbar_init(bar_addr(bars->p_ready[r]), 2);    // the relays of two CTAs
    }
    for (int s = 0; s < kVSlots; ++s) {
      mbar_init(bar_addr(bars->v_full[s]), 1);
      mbar_init(bar_addr(bars->v_ready[s]), 2);    // the fixup warps of two CTAs
      mbar_init(bar_addr(bars->v_empty[s]), 1);
    }
    mbar_init(bar_addr(bars->epi_req), 2);         // request posted + commit
    mbar_init(bar_addr(bars->corr_done), 16);
    mbar_init(bar_addr(bars->o_free), 16);
    mbar_init(bar_addr(bars->meta_done), 8);
    bars->abort = 0;
    fence_mbar_init();
  }
  if (warp == 1) {
    pair_tmem_alloc(smem_u32(&bars->tmem_base), kTmemCols);
    pair_tmem_relinquish();
  }
  tc_fence_before();
  cluster_sync();
  tc_fence_after();
  // programmatic stream serialization: the set-up above overlaps the plan
  // kernel; the merge kernel may be scheduled now (it waits for this grid)
  asm volatile("griddepcontrol.wait;" ::: "memory");
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");

  Ctx c;
  c.p = &p;
  c.base = base;
  c.gbase = smem_raw;
  c.bars = bars;
  c.tmem = bars->tmem_base;
  c.wc = WaitCtx{p.spin_limit, p.err, &bars->abort, p.err + 1};
  c.engine = blockIdx.x >> 2;
  c.rank = rank;
  c.warp = warp;
  c.lane = lane;

  if ((base & 1023u) != 0) {
    // swizzled tiles need 1024-byte aligned shared memory: nothing was
    // issued, the call reads as one that gave up
    if (threadIdx.x == 0) atomicOr(p.err, kErrTimeout);
  } else if (rank < 2) {
    if (warp == 0) {
      if (elect_one()) score_feed(c, &maps.k, &maps.k2, &maps.q);
      __syncwarp();
    }
    if (warp == 1 && rank == 0) score_mma(c);
    else if (warp == 2) score_tma_q(c, &maps.q);
    else if (warp >= 4) score_softmax(c);
  } else {
    if (warp == 0) {
      if (elect_one()) value_feed(c, &maps.k4);
      __syncwarp();
    }
    if (warp == 1 && rank == 2) value_mma(c);
    else if (warp == 2) value_fixup(c);
    else if (warp == 3) value_relay(c);
    else if (warp >= 4) value_epilogue(c);
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
  // no CTA leaves (or frees TMEM) while another of its cluster may still
  // signal it or run MMAs on its memory
  cluster_sync();
  if (warp == 1) {
    tc_fence_after();
    pair_tmem_dealloc(c.tmem, kTmemCols);
  }
  cluster_sync();
}

// Threads of the plan: one CTA, fewer warps at its barriers for small calls.
constexpr int kPlanThreads = 1024;
constexpr int kPlanFew = 128;

// Inclusive scan of one value per thread over the block.
template <class T>
__device__ T block_scan(T v, T* warp_sums, T* total) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const T u = __shfl_up_sync(0xffffffffu, v, o);
    if (lane >= o) v += u;
  }
  __syncthreads();
  if (lane == 31) warp_sums[warp] = v;
  __syncthreads();
  T w = lane < static_cast<int>(blockDim.x >> 5) ? warp_sums[lane] : T(0);
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const T u = __shfl_up_sync(0xffffffffu, w, o);
    if (lane >= o) w += u;
  }
  *total = __shfl_sync(0xffffffffu, w, 31);
  return v + (warp > 0 ? __shfl_sync(0xffffffffu, w, warp - 1) : T(0));
}

// The tile list: tiles of up to 256 / H tokens of one sequence, and the
// running count of the cache blocks they read.
__global__ void __launch_bounds__(kPlanThreads) chunk_plan_kernel(const ChunkParams p) {
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  __shared__ long long sums[32];
  __shared__ int isums[32];
  __shared__ long long even[kMaxEngines + 1], whole[kMaxEngines + 1];
  __shared__ int uneven;
  if (threadIdx.x == 0) uneven = 0;
  const int per = kTileRows / p.H;
  int nt = 0;
  for (int b0 = 0; b0 < p.B; b0 += blockDim.x) {
    const int b = b0 + threadIdx.x;
    int tiles = 0;
    if (b < p.B) {
      const int a = p.q_offsets[b], e = p.q_offsets[b + 1];
      checked_len(p.seq_lens, b, p.max_blocks, p.err);
      if (a < 0 || e < a || e > p.T)
        atomicOr(p.err, kErrSeqTooLong);
      else
        tiles = (e - a + per - 1) / per;
    }
    int total;
    const int incl = block_scan(tiles, isums, &total);
    // only offsets that decrease somewhere can ask for more tiles than T
    // tokens fill: what is over is left out
    if (b < p.B) {
      p.tile_off[b] = min(p.max_tiles, nt + incl - tiles);
      if (nt + incl > p.max_tiles) atomicOr(p.err, kErrSeqTooLong);
    }
    nt = min(p.max_tiles, nt + total);
  }
  if (threadIdx.x == 0) {
    p.tile_off[p.B] = nt;
    *p.n_tiles = nt;
    p.pre[0] = 0;
  }
  __syncthreads();
  long long blocks = 0;
  for (int t0 = 0; t0 < nt; t0 += blockDim.x) {
    const int t = t0 + threadIdx.x;
    long long mine = 0;
    if (t < nt) {
      int lo = 0, hi = p.B;  // tile_off[lo] <= t < tile_off[hi]
      while (hi - lo > 1) {
        const int mid = (lo + hi) >> 1;
        if (p.tile_off[mid] <= t) lo = mid; else hi = mid;
      }
      const int a = p.q_offsets[lo], n = p.q_offsets[lo + 1] - a;
      const int j = (t - p.tile_off[lo]) * per;
      const int tok = min(per, n - j);
      // the tile's last token sees the sequence without the n - j - tok tokens behind it
      const int len = max(0, checked_len(p.seq_lens, lo, p.max_blocks, nullptr) - (n - j - tok));
      p.tiles[t] = make_int4((a + j) * p.H, tok * p.H, lo, len);
      mine = len > 0 ? nblocks_of(len) + kTileUnits : 0;
    }
    long long total;
    const long long incl = block_scan(mine, sums, &total);
    if (t < nt) p.pre[t + 1] = blocks + incl;
    blocks += total;
  }
  // Every engine's range and first tile (t = nt: none).  With few tiles to an
  // engine the even cut at x moves to the nearest end of its tile if that is
  // at most kTileUnits and a sixteenth of a range away (a piece costs as much),
  // or everywhere if no range then exceeds the even one by more than kWholeUnits
  // and half of it: no tile is cut, and there is nothing to merge.  (More than
  // kMaxEngines, which only a caller can ask for, keep the even cuts.)
  // No cut may reach the end of the last tile: the merge finds a cut's tile by
  // the cut, and there is none behind the last.  The even ones cannot (a range
  // is longer than a sixteenth of one).  With the others it takes a last tile of
  // two ranges at least, whose own range is then longer than one and a half: the
  // even cuts stay.  So `slack` must not exceed half a range.
  // Measured, even cuts first: 32 x 4 tokens x 128 heads over 256 44.2 us and
  // 34.7, 32 x 8 over 2048 142 and 131, 64 x 1 over 4096 127 and 121; a batch
  // that has to be cut anyway pays up to 1 us.
  __syncthreads();
  const int P = engines_of(p, blocks);
  const bool move = P > 1 && P <= kMaxEngines && nt > 1 && 2 * nt >= P;
  // 32-bit divisions where they do (64 * 2^26 = 2^32)
  const bool narrow = P <= kMaxEngines && blocks < (1LL << 26);
  const long long share = !move ? 0 : narrow ? static_cast<unsigned>(blocks) / static_cast<unsigned>(P) : blocks / P;
  const long long near = min(static_cast<long long>(kTileUnits), share / 16);
  const long long slack = min(static_cast<long long>(kWholeUnits), share / 2);
  auto start_of = [&](int e) -> long long {
    return narrow ? static_cast<unsigned>(e) * static_cast<unsigned>(blocks) / static_cast<unsigned>(P)
                  : range_start(e, blocks, P);
  };
  if (move) {
    for (int e = threadIdx.x; e <= P; e += blockDim.x) {
      long long x = start_of(e), w = x;
      if (e > 0 && e < P) {
        const int t = tile_of(p.pre, nt, x);
        const long long a = p.pre[t], z = p.pre[t + 1];
        w = x - a <= z - x ? a : z;
        if (llabs(w - x) <= near) x = w;
      }
      even[e] = x;
      whole[e] = w;
    }
    __syncthreads();
    if (threadIdx.x < kMaxEngines) {
      const int e = threadIdx.x;
      if (__any_sync(0xffffffffu, e < P && whole[e + 1] - whole[e] > share + slack) && (e & 31) == 0) uneven = 1;
    }
    __syncthreads();
  }
  const long long* cut = uneven != 0 ? even : whole;
  for (int e = threadIdx.x; e < p.P; e += blockDim.x) {
    ChunkEngine r = {};
    r.t = r.nt = nt;
    if (e < P) {
      r.s = move ? cut[e] : start_of(e);
      r.e = move ? cut[e + 1] : start_of(e + 1);
      r.t = tile_of(p.pre, nt, r.s);
      r.a = p.pre[r.t];
      r.z = p.pre[r.t + 1];
      r.tile = p.tiles[r.t];
    }
    p.engines[e] = r;
  }
}

constexpr int kMergeWarps = 8;
constexpr int kMergeThreads = 32 * kMergeWarps;
constexpr int kMergeCols = 16;                                              // columns of a thread
constexpr int kMergeGrid = (kTileRows / 32) * (kDc / kMergeCols) / kMergeWarps;  // CTAs per tile

__device__ __forceinline__ void fill_row(const ChunkParams& p, size_t row, float lse, int lane) {
  uint4* dst = reinterpret_cast<uint4*>(p.out + row * kDc + lane * 16);
  dst[0] = make_uint4(0u, 0u, 0u, 0u);
  dst[1] = make_uint4(0u, 0u, 0u, 0u);
  if (lane == 0) p.lse[row] = lse;
}

// grid (engines, kMergeGrid): the boundary at which a cut tile's first piece
// ends merges that tile; a warp takes 32 rows (lane = row) and 16 columns:
//   lse = M + log sum_i exp(lse_i - M),  out = sum_i exp(lse_i - lse) o_i.
// Rows of tokens that see no cached token are written here, and after a
// timeout every row of the call.
__global__ void __launch_bounds__(kMergeThreads) chunk_merge_kernel(const ChunkParams p) {
  asm volatile("griddepcontrol.wait;" ::: "memory");
  const int lane = threadIdx.x & 31;
  const int wid = blockIdx.y * kMergeWarps + (threadIdx.x >> 5);  // 0..255 within a tile
  const int nt = *p.n_tiles;
  if ((*reinterpret_cast<volatile uint32_t*>(p.err) & kErrTimeout) != 0) {
    for (int t = blockIdx.x; t < nt; t += gridDim.x)
      for (int r = wid; r < p.tiles[t].y; r += kMergeGrid * kMergeWarps) fill_row(p, size_t(p.tiles[t].x) + r, NAN, lane);
    return;
  }
  const int e1 = blockIdx.x + 1;  // the boundary between engines e1 - 1 and e1
  ChunkEngine r = {};
  if (e1 < p.P) r = p.engines[e1];
  const long long s0 = p.engines[blockIdx.x].s;
  for (int b = blockIdx.x; b < p.B; b += gridDim.x) {
    const int a = p.q_offsets[b], e = p.q_offsets[b + 1];
    if (a < 0 || e < a || e > p.T) continue;
    const int blind = e - a - checked_len(p.seq_lens, b, p.max_blocks, nullptr);  // tokens that see nothing
    for (long long r = wid; r < static_cast<long long>(blind) * p.H; r += kMergeGrid * kMergeWarps)
      fill_row(p, size_t(a) * p.H + r, -INFINITY, lane);
  }
  if (r.t >= r.nt) return;  // past the last engine
  const long long x = r.s, a = r.a, z = r.z;
  // merged at the boundary whose left engine holds the tile's first block
  if (x <= a + kTileUnits || s0 > a + kTileUnits) return;
  const int4 info = r.tile;
  // pieces: one per engine from the left one on whose range starts before the
  // tile ends (no range inside a tile is empty)
  int n = 1;
  for (int e0 = e1; e0 < p.P; e0 += 32) {
    const bool in = e0 + lane < p.P && p.engines[e0 + lane].t < r.nt && p.engines[e0 + lane].s < z;
    const unsigned m = __ballot_sync(0xffffffffu, in);
    n += __popc(m);
    if (m != 0xffffffffu) break;
  }
  const int row = (wid & 7) * 32 + lane, col4 = (wid >> 3) * (kMergeCols / 4);
  if (row >= info.y) return;
  // the first piece is its engine's second segment if the engine's range starts in an earlier tile
  auto slot_of = [&](int i) { return 2 * (e1 - 1 + i) + (i == 0 && s0 < a ? 1 : 0); };
  float M = -INFINITY, sum = 0.f;
  for (int i = 0; i < n; ++i) M = fmaxf(M, p.lse_part[size_t(slot_of(i)) * kTileRows + row]);
  const float base = M == -INFINITY ? 0.f : M;
  float acc[kMergeCols];
#pragma unroll
  for (int k = 0; k < kMergeCols; ++k) acc[k] = 0.f;
  // weights relative to M, divided by their sum at the end; an empty piece
  // holds zeros and weighs exp(-inf) = 0, a NaN piece makes the row NaN
#pragma unroll 2
  for (int i = 0; i < n; ++i) {
    const float wgt = expf(p.lse_part[size_t(slot_of(i)) * kTileRows + row] - base);
    const float4* src = reinterpret_cast<const float4*>(p.o_part) + piece_unit(slot_of(i), col4, row);
    sum += wgt;
#pragma unroll
    for (int q = 0; q < kMergeCols / 4; ++q) {
      const float4 v = src[q * kTileRows];
      acc[4 * q] += wgt * v.x;
      acc[4 * q + 1] += wgt * v.y;
      acc[4 * q + 2] += wgt * v.z;
      acc[4 * q + 3] += wgt * v.w;
    }
  }
  const float inv = sum == 0.f ? 0.f : 1.f / sum;
  uint32_t pk[kMergeCols / 2];
#pragma unroll
  for (int k = 0; k < kMergeCols / 2; ++k) {
    __nv_bfloat162 b2 = __floats2bfloat162_rn(acc[2 * k] * inv, acc[2 * k + 1] * inv);
    pk[k] = *reinterpret_cast<uint32_t*>(&b2);
  }
  uint4* dst = reinterpret_cast<uint4*>(p.out + (size_t(info.x) + row) * kDc + 4 * col4);
  dst[0] = make_uint4(pk[0], pk[1], pk[2], pk[3]);
  dst[1] = make_uint4(pk[4], pk[5], pk[6], pk[7]);
  if (col4 == 0) p.lse[size_t(info.x) + row] = sum == 0.f ? -INFINITY : M + logf(sum);
}

cudaError_t set_attributes() {
  return cudaFuncSetAttribute(chunk_sm100_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, int(kSmemBytes));
}

}  // namespace

int chunk_sm100_max_clusters() {
  if (set_attributes() != cudaSuccess) return 0;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(4);
  cfg.blockDim = dim3(kThreads);
  cfg.dynamicSmemBytes = kSmemBytes;
  int n = 0;
  if (cudaOccupancyMaxActiveClusters(&n, chunk_sm100_kernel, &cfg) != cudaSuccess) return 0;
  return n;
}

cudaError_t launch_chunk_sm100(const ChunkParams& given, const ChunkMaps& maps, cudaStream_t stream) {
  static std::atomic<bool> attr_set[64];
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= 64) return cudaErrorInvalidDevice;
  if (!attr_set[dev].load(std::memory_order_acquire)) {
    if (cudaError_t e = set_attributes(); e != cudaSuccess) return e;
    attr_set[dev].store(true, std::memory_order_release);
  }
  // no more engines than the table's width could fill with kMinUnits each
  const long long most = (static_cast<long long>(given.max_tiles) * (given.max_blocks + kTileUnits) + kMinUnits - 1) / kMinUnits;
  ChunkParams p = given;
  if (most < p.P) p.P = most > 0 ? static_cast<int>(most) : 1;
  const int threads = p.B <= kPlanFew && p.max_tiles <= kPlanFew ? kPlanFew : kPlanThreads;
  chunk_plan_kernel<<<1, threads, 0, stream>>>(p);
  if (cudaError_t e = cudaGetLastError(); e != cudaSuccess) return e;
  cudaLaunchConfig_t cfg = {};
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  cfg.stream = stream;
  cfg.gridDim = dim3(4 * p.P);
  cfg.blockDim = dim3(kThreads);
  cfg.dynamicSmemBytes = kSmemBytes;
  if (cudaError_t e = cudaLaunchKernelEx(&cfg, chunk_sm100_kernel, maps, p); e != cudaSuccess) return e;
  cfg.gridDim = dim3(p.P, kMergeGrid);
  cfg.blockDim = dim3(kMergeThreads);
  cfg.dynamicSmemBytes = 0;
  return cudaLaunchKernelEx(&cfg, chunk_merge_kernel, p);
}

}  // namespace mla
