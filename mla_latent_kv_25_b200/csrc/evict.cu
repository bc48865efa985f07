// Eviction from the paged cache by accumulated attention weight.
//
// Per sequence of L tokens and budget n: rank the slots by (protected, weight,
// lower slot), keep the first n, and move the kept rows behind slot n into the
// free slots before it (k-th to k-th).  Kept rows before slot n stay, sources
// lie at or past n and destinations before it, so no move reads what another
// writes and all moves can run at once.
//
// evict_select_kernel: one cluster of 1, 2, 4 or 8 CTAs per sequence, every
//   CTA and in it every warp owning a contiguous range of slots.  The n-th
//   largest weight is found by a radix select: three passes over an
//   order-preserving integer image of the weights, which is formed once and
//   stays in shared memory; the CTAs add up their histograms over distributed
//   shared memory.  Which slots stay is then one bit each; ties (only if some
//   of them go), free slots and movers are ranked by prefix sums of bit counts
//   over words, warps and CTAs, so the lists are ordered and the result is the
//   same every time.  Bound by latencies: 64 x 4096 slots (one CTA each) take
//   17,500 cycles, 3,600 of them the first loads and 4,300 the digits; 4 x
//   131072 (eight CTAs each) 56,000, with six cluster barriers and the
//   instructions of passes over 16 slots per thread.
// evict_move_kernel: bulk copies of whole rows through shared memory, 32 rows
//   in flight per warp, and behind each row its weight and position.  Bound: HBM,
//   2304 bytes per moved row.
// Whole call: 64 x 4096 -> 2048 39 us, 4 x 131072 -> 65536 87 us (rows alone at
// the measured copy bandwidth: 23.5 and 47).
#include <atomic>

#include "common.cuh"
#include "kernels.h"
#include "plan.h"
#include "sm100.cuh"

namespace mla {
namespace {

using namespace sm100;

constexpr int kSelThreads = 1024;
constexpr int kSelWarps = kSelThreads / 32;
// 16 (which needs an opt-in) measured the same for 4 x 131072 slots (87 us) and
// 21.3 us against 19.2 for 1 x 32768.
constexpr int kMaxCluster = 8;
// Digits of 11, 11 and 10 bits: the first holds sign, exponent and two bits of
// the mantissa.  With 8 bits, weights of a few exponents met in a few bins and
// their shared-memory atomics serialised (16,000 cycles for 16384 slots, of
// 93,000 of the whole kernel).
constexpr int kBins = 2048;
constexpr int kPasses = 3;
__device__ __forceinline__ constexpr int digit_shift(int pass) { return pass == 0 ? 21 : pass == 1 ? 10 : 0; }
__device__ __forceinline__ constexpr uint32_t digit_mask(int pass) { return pass == 2 ? 1023u : 2047u; }
// Slots of one CTA whose keys fit in shared memory (4 bytes and two bits each);
// of a longer range only the bits are kept and the weights read in every pass.
constexpr int kKeysInShared = 45056;

// Order-preserving image of a weight: larger weight, larger key; -0 equals +0,
// NaN ranks as -inf.
__device__ __forceinline__ uint32_t weight_key(float w) {
  if (w != w) w = -INFINITY;
  w += 0.f;  // -0 -> +0
  const uint32_t u = __float_as_uint(w);
  return (u & 0x80000000u) ? ~u : (u | 0x80000000u);
}

__device__ __forceinline__ int warp_sum(int v) { return __reduce_add_sync(0xffffffffu, v); }
__device__ __forceinline__ int warp_max(int v) { return __reduce_max_sync(0xffffffffu, v); }

__device__ __forceinline__ int ld_cluster(uint32_t local, uint32_t rank) {
  int v;
  asm volatile("ld.shared::cluster.b32 %0, [%1];" : "=r"(v) : "r"(map_to_rank(local, rank)) : "memory");
  return v;
}
__device__ __forceinline__ int2 ld_cluster2(uint32_t local, uint32_t rank) {
  int2 v;
  asm volatile("ld.shared::cluster.v2.b32 {%0, %1}, [%2];" : "=r"(v.x), "=r"(v.y) : "r"(map_to_rank(local, rank)) : "memory");
  return v;
}

__device__ __forceinline__ int scan_up(int v, int lane) {  // inclusive
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int u = __shfl_up_sync(0xffffffffu, v, o);
    if (lane >= o) v += u;
  }
  return v;
}

struct Shared {
  alignas(8) int hist[kPasses + 1][kBins];  // top digit of the unprotected and of the protected slots; the lower digits
  int group[2][kSelWarps];                  // sums of 64 bins each (of both classes, then of the lower digits)
  int warp_val[2][kSelWarps];
  int cta_val[6];        // published values: largest position, protected slots, ties, free slots, movers
  int pick[3];           // digit, rank within it, slots of that digit
};

// Exclusive prefixes of two values per warp over the block's warps, and their totals.
__device__ __forceinline__ int2 warps_before(Shared& sh, int warp, int lane, int2 mine, int2* total) {
  __syncthreads();
  if (lane == 0) {
    sh.warp_val[0][warp] = mine.x;
    sh.warp_val[1][warp] = mine.y;
  }
  __syncthreads();
  const int x = sh.warp_val[0][lane], y = sh.warp_val[1][lane];
  *total = make_int2(warp_sum(x), warp_sum(y));
  return make_int2(warp_sum(lane < warp ? x : 0), warp_sum(lane < warp ? y : 0));
}

template <bool kCluster>
__device__ __forceinline__ void everyone() {
  if (kCluster)
    cluster_sync();  // also releases and acquires the CTAs' global writes
  else
    __syncthreads();
}

// Publishes two values of this CTA (after the barrier others may read them)
// and returns the sums over the CTAs before it and over all.
template <bool kCluster>
__device__ __forceinline__ int2 ctas_before(Shared& sh, int what, int rank, int size, int2 mine, int2* total) {
  if (!kCluster) {
    *total = mine;
    return make_int2(0, 0);
  }
  if (threadIdx.x == 0) {
    sh.cta_val[what] = mine.x;
    sh.cta_val[what + 1] = mine.y;
  }
  cluster_sync();
  int2 before = make_int2(0, 0), all = make_int2(0, 0), v[kMaxCluster];
#pragma unroll
  for (int r = 0; r < kMaxCluster; ++r)  // all remote loads in flight at once
    v[r] = r < size ? make_int2(ld_cluster(smem_u32(&sh.cta_val[what]), r), ld_cluster(smem_u32(&sh.cta_val[what + 1]), r))
                    : make_int2(0, 0);
#pragma unroll
  for (int r = 0; r < kMaxCluster; ++r) {
    all.x += v[r].x;
    all.y += v[r].y;
    before.x += r < rank ? v[r].x : 0;
    before.y += r < rank ? v[r].y : 0;
  }
  *total = all;
  return before;
}

struct Digit {
  int digit, rank, count;
};

// Every warp adds up its 64 bins of a histogram that the block has completed.
__device__ __forceinline__ void sum_group(const int* hist, int* group, int warp, int lane) {
  const int2 v = *reinterpret_cast<const int2*>(hist + 64 * warp + 2 * lane);
  const int sum = warp_sum(v.x + v.y);
  if (lane == 0) group[warp] = sum;
}

// The digit, from the largest down, at which the histogram summed over the
// CTAs reaches `need`, the rank left within it and the slots that have it.
// One warp finds the group of 64 bins, then the bin: the other CTAs' shared
// memory is read twice 8 x 256 bytes, not whole histograms by every CTA.
template <bool kCluster>
__device__ __forceinline__ Digit find_digit(Shared& sh, const int* hist, const int* group, int size, int need, int warp,
                                            int lane) {
  static_assert(kBins == 64 * 32 && kSelWarps == 32, "groups of bins");
  if (warp == 0) {
    int c = 0;
    if (kCluster) {
      int v[kMaxCluster];
#pragma unroll
      for (int r = 0; r < kMaxCluster; ++r)  // all remote loads in flight at once
        v[r] = r < size ? ld_cluster(smem_u32(group + 31 - lane), r) : 0;
#pragma unroll
      for (int r = 0; r < kMaxCluster; ++r) c += v[r];
    } else {
      c = group[31 - lane];
    }
    int upto = scan_up(c, lane);
    const int at = __ffs(__ballot_sync(0xffffffffu, upto >= need)) - 1;  // the first group that reaches it
    need -= __shfl_sync(0xffffffffu, upto - c, at);
    const int top = 64 * (31 - at) + 63 - 2 * lane;  // this lane's bins: top, top - 1
    int2 f = make_int2(0, 0);
    if (kCluster) {
      int2 v[kMaxCluster];
#pragma unroll
      for (int r = 0; r < kMaxCluster; ++r)
        v[r] = r < size ? ld_cluster2(smem_u32(hist + top - 1), r) : make_int2(0, 0);
#pragma unroll
      for (int r = 0; r < kMaxCluster; ++r) {
        f.x += v[r].x;
        f.y += v[r].y;
      }
    } else {
      f = *reinterpret_cast<const int2*>(hist + top - 1);
    }
    upto = scan_up(f.x + f.y, lane);
    const int before = upto - f.x - f.y;
    if (before < need && need <= upto) {
      const bool low = need > before + f.y;
      sh.pick[0] = top - low;
      sh.pick[1] = need - before - (low ? f.y : 0);
      sh.pick[2] = low ? f.x : f.y;
    }
  }
  __syncthreads();
  return Digit{sh.pick[0], sh.pick[1], sh.pick[2]};
}

// Adds one to a bin per lane with bin >= 0; a warp whose lanes agree adds once.
__device__ __forceinline__ void count_bins(int* hist, int bin, int lane) {
  if (__all_sync(0xffffffffu, bin == __shfl_sync(0xffffffffu, bin, 0))) {
    if (lane == 0 && bin >= 0) atomicAdd(hist + bin, 32);
  } else if (bin >= 0) {
    atomicAdd(hist + bin, 1);
  }
}

// kStored: the keys live in shared memory.
template <bool kCluster, bool kStored>
__global__ void __launch_bounds__(kSelThreads, 1) evict_select_kernel(const EvictParams p, int size, int room) {
  __shared__ Shared sh;
  extern __shared__ uint32_t dyn[];
  uint32_t* gbits = dyn;                // [room / 32] protected slots, later ties
  uint32_t* kbits = gbits + room / 32;  // [room / 32] slots that stay
  uint32_t* keys = kbits + room / 32;   // [room] if kStored
  const int b = static_cast<int>(blockIdx.x) / size;
  const int rank = kCluster ? static_cast<int>(cluster_ctarank()) : 0;
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const size_t S = size_t(p.max_blocks) * kBlock;
  const float* w = p.weight + b * S;
  const int32_t* pos = p.slot_pos + b * S;
  float* nw = p.new_weight + b * S;
  int32_t* np = p.new_pos + b * S;
  const int L = checked_len(p.seq_lens, b, p.max_blocks, threadIdx.x == 0 && rank == 0 ? p.err : nullptr);
  const int n = min(max(p.keep[b], 0), L);
  const int tid = rank * kSelThreads + threadIdx.x, threads = size * kSelThreads;
  // the moving CTAs may take the free SMs now; they wait for this kernel's end
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  // values before slot n are copied as they are read; those of moved rows
  // follow with the rows, in the next kernel
  const bool copy = nw != w || np != pos;
  if (n == L) {  // nothing to evict (the same decision in every CTA of the cluster)
    everyone<kCluster>();  // new_lens may be seq_lens: all have read it
    if (copy)
      for (int s = tid; s < n; s += threads) {
        nw[s] = w[s];
        np[s] = pos[s];
      }
    if (threadIdx.x == 0 && rank == 0) {
      p.n_moves[b] = 0;
      p.new_lens[b] = n;
    }
    return;
  }
  // this CTA's slots [c0, c1) and this warp's [lo, hi)
  const int share = ((L + size - 1) / size + 31) / 32 * 32;  // <= room
  const int c0 = min(L, rank * share), c1 = min(L, c0 + share);
  const int per = ((c1 - c0 + kSelWarps - 1) / kSelWarps + 31) / 32 * 32;
  const int lo = min(c1, c0 + warp * per), hi = min(c1, lo + per);

  for (int i = threadIdx.x; i < (kPasses + 1) * kBins; i += kSelThreads) (&sh.hist[0][0])[i] = 0;

  // Keys and the newest position.  Four loads of each array are in flight
  // before the copies, which the compiler has to take for writes to them (16:
  // slower below 16384 slots a sequence, the same above; all of this kernel's
  // code runs once, and fetching unrolled loops costs more than they save).  Keys
  // are at least 0x7fffff; 0 stands for a slot that does not compete.
  int last = INT32_MIN;
  for (int s0 = lo; s0 < hi; s0 += 128) {
    int ps[4];
    float ws[4];
#pragma unroll
    for (int u = 0; u < 4; ++u) {
      const int s = s0 + 32 * u + lane;
      ps[u] = s < hi ? pos[s] : INT32_MIN;
      ws[u] = s < hi ? w[s] : 0.f;
    }
#pragma unroll
    for (int u = 0; u < 4; ++u) {
      const int s = s0 + 32 * u + lane;
      last = max(last, ps[u]);
      if (kStored && s0 + 32 * u < hi) keys[s - c0] = s < hi ? weight_key(ws[u]) : 0u;
      if (copy && s < n && s < hi) {
        nw[s] = ws[u];
        np[s] = ps[u];
      }
    }
  }
  last = warp_max(last);
  if (lane == 0) sh.warp_val[0][warp] = last;
  __syncthreads();
  last = warp_max(sh.warp_val[0][lane]);
  if (kCluster) {
    if (threadIdx.x == 0) sh.cta_val[0] = last;
    cluster_sync();
    for (int r = 0; r < size; ++r) last = max(last, ld_cluster(smem_u32(&sh.cta_val[0]), r));
  }
  const long long from = static_cast<long long>(last) - p.n_recent;  // protected: pos > from

  // protection bits, and the histogram of the top digit of each class
  int guarded_here = 0;
#pragma unroll 4
  for (int s0 = lo; s0 < hi; s0 += 32) {
    const int s = s0 + lane;
    const bool in = s < hi;
    const int ps = in ? pos[s] : 0;
    const uint32_t key = kStored ? keys[s - c0] : in ? weight_key(w[s]) : 0u;
    const bool g = in && (ps < p.n_first || ps > from);
    const unsigned gm = __ballot_sync(0xffffffffu, g);
    if (lane == 0) gbits[(s0 - c0) >> 5] = gm;
    if (kStored && g) keys[s - c0] = 0u;  // as long as it is the others that compete
    guarded_here += __popc(gm);
    count_bins(&sh.hist[0][0], in ? (g ? kBins : 0) + static_cast<int>(key >> digit_shift(0)) : -1, lane);
  }
  int2 here, all;
  warps_before(sh, warp, lane, make_int2(guarded_here, 0), &here);
  sum_group(sh.hist[0], sh.group[0], warp, lane);
  sum_group(sh.hist[1], sh.group[1], warp, lane);
  if (!kCluster) __syncthreads();
  ctas_before<kCluster>(sh, 1, rank, size, here, &all);
  const int n_guarded = all.x;
  // either some protected slots go too, or all stay and the others compete
  const bool among_guarded = n_guarded >= n;
  int need = among_guarded ? n : n - n_guarded;  // kept of the competing class

  if (kStored && among_guarded)
    for (int s = lo + lane; s < hi; s += 32)
      keys[s - c0] = (gbits[(s - c0) >> 5] >> lane) & 1u ? weight_key(w[s]) : 0u;
  // the key of this lane's slot of the 32 from s0 on, 0 if it does not compete
  auto key_of = [&](int s0) -> uint32_t {
    const int s = s0 + lane;
    if (kStored) return keys[s - c0];
    return s < hi && (((gbits[(s0 - c0) >> 5] >> lane) & 1u) != 0) == among_guarded ? weight_key(w[s]) : 0u;
  };

  // Radix select: the competing slots with key > thr are kept, and of those
  // with key == thr the first `need`, or all of them (`all_ties`).  need = 0
  // keeps none: no key reaches 0xffffffff.
  uint32_t thr = 0xffffffffu;
  bool all_ties = true;
  if (need > 0) {
    const int cls = among_guarded ? 1 : 0;
    Digit d = find_digit<kCluster>(sh, sh.hist[cls], sh.group[cls], size, need, warp, lane);
    thr = static_cast<uint32_t>(d.digit);
#pragma unroll
    for (int pass = 1; pass < kPasses; ++pass) {
      int* hist = sh.hist[1 + pass];
#pragma unroll 4
      for (int s0 = lo; s0 < hi; s0 += 32) {
        const uint32_t key = key_of(s0);
        if ((key >> digit_shift(pass - 1)) == thr) atomicAdd(&hist[(key >> digit_shift(pass)) & digit_mask(pass)], 1);
      }
      __syncthreads();
      // in turn: another CTA may still read the sums of the pass before
      int* group = sh.group[(cls + pass) & 1];
      sum_group(hist, group, warp, lane);
      everyone<kCluster>();
      d = find_digit<kCluster>(sh, hist, group, size, d.rank, warp, lane);
      thr = (thr << (digit_shift(pass - 1) - digit_shift(pass))) | static_cast<uint32_t>(d.digit);
    }
    need = d.rank;
    all_ties = d.rank == d.count;
  }

  // which slots stay, one bit each: the protected ones while the others
  // compete, and those whose key is large enough
  int2 before;
  int tie0 = 0;
  if (all_ties) {
#pragma unroll 4
    for (int s0 = lo; s0 < hi; s0 += 32) {
      const uint32_t over = __ballot_sync(0xffffffffu, key_of(s0) >= thr);
      if (lane == 0) kbits[(s0 - c0) >> 5] = among_guarded ? over : over | gbits[(s0 - c0) >> 5];
    }
  } else {
    // ties into gbits, all others that stay into kbits
    int ties = 0;
#pragma unroll 2
    for (int s0 = lo; s0 < hi; s0 += 32) {
      const uint32_t key = key_of(s0), g = gbits[(s0 - c0) >> 5];
      const uint32_t over = __ballot_sync(0xffffffffu, key > thr);
      const uint32_t tie = __ballot_sync(0xffffffffu, key == thr);
      __syncwarp();
      if (lane == 0) {
        kbits[(s0 - c0) >> 5] = among_guarded ? over : over | g;
        gbits[(s0 - c0) >> 5] = tie;
      }
      ties += __popc(tie);
    }
    before = warps_before(sh, warp, lane, make_int2(ties, 0), &here);
    tie0 = before.x + ctas_before<kCluster>(sh, 2, rank, size, here, &all).x;
  }
  __syncwarp();

  // one word of 32 slots per lane: the first `need` ties stay too; then the
  // free slots below n and the movers behind it
  int holes = 0, movers = 0;
  auto below_n = [&](int s0) -> uint32_t { return n - s0 >= 32 ? 0xffffffffu : n <= s0 ? 0u : (1u << (n - s0)) - 1u; };
  for (int s0 = lo; s0 < hi; s0 += 1024) {
    const int s = s0 + 32 * lane;
    const bool in = s < hi;
    uint32_t k = in ? kbits[(s - c0) >> 5] : 0u;
    if (!all_ties) {
      const uint32_t tie = in ? gbits[(s - c0) >> 5] : 0u;
      const int c = __popc(tie);
      const int incl = scan_up(c, lane);
      int room_left = need - (tie0 + incl - c);  // ties that still stay
      uint32_t take = room_left >= c ? tie : 0u;
      if (room_left > 0 && room_left < c)
        for (uint32_t t = tie; room_left > 0; --room_left) {
          take |= t & (0u - t);
          t &= t - 1;
        }
      k |= take;
      if (in) kbits[(s - c0) >> 5] = k;
      tie0 += __shfl_sync(0xffffffffu, incl, 31);
    }
    if (in) {
      // n < L: slots below n are cached ones
      const uint32_t low = below_n(s);
      holes += __popc(~k & low);
      movers += __popc(k & ~low);
    }
  }
  holes = warp_sum(holes);
  movers = warp_sum(movers);
  before = warps_before(sh, warp, lane, make_int2(holes, movers), &here);
  const int2 others = ctas_before<kCluster>(sh, 4, rank, size, here, &all);
  // the others' shared memory has been read: arrive before the lists' stores,
  // which an arrival behind them would wait for, and wait before the exit
  if (kCluster) asm volatile("barrier.cluster.arrive.release.aligned;" ::: "memory");
  int hole0 = before.x + others.x, mover0 = before.y + others.y;
  const int n_moves = all.y;
  int2* moves = p.moves + b * (S / 2);
  const uint32_t below_me = (1u << lane) - 1u;
#pragma unroll 4
  for (int s0 = lo; s0 < hi; s0 += 32) {
    const uint32_t k = kbits[(s0 - c0) >> 5], low = below_n(s0);
    const uint32_t mh = ~k & low, mm = k & ~low;
    const int s = s0 + lane;
    if (low != 0) {
      if ((mh >> lane) & 1u) moves[hole0 + __popc(mh & below_me)].y = s;
      hole0 += __popc(mh);
    }
    if (low != 0xffffffffu) {
      if ((mm >> lane) & 1u) {
        moves[mover0 + __popc(mm & below_me)].x = s;
      } else if (s >= n && s < hi) {  // freed; a moved row's own slot is cleared with the move
        nw[s] = 0.f;
        np[s] = -1;
      }
      mover0 += __popc(mm);
    }
  }
  if (threadIdx.x == 0 && rank == 0) {
    p.n_moves[b] = n_moves;
    p.new_lens[b] = n;
  }
  if (kCluster) asm volatile("barrier.cluster.wait.acquire.aligned;" ::: "memory");
}

constexpr int kMoveRows = 16;                        // rows of a stage, one per lane of half the warp
constexpr int kMoveStages = 2;
constexpr uint32_t kRowBytes = kRow * 2;
constexpr long long kMovePerSm = 6;                  // CTAs that fit on an SM
constexpr uint32_t kMoveSmem = kMoveStages * kMoveRows * kRowBytes;

__device__ __forceinline__ void bulk_load(uint32_t dst, const void* src, uint32_t bytes, uint32_t bar) {
  asm volatile("cp.async.bulk.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1], %2, [%3];" ::"r"(dst),
               "l"(reinterpret_cast<uint64_t>(src)), "r"(bytes), "r"(bar)
               : "memory");
}
__device__ __forceinline__ void bulk_store(void* dst, uint32_t src, uint32_t bytes) {
  asm volatile("cp.async.bulk.global.shared::cta.bulk_group [%0], [%1], %2;" ::"l"(reinterpret_cast<uint64_t>(dst)),
               "r"(src), "r"(bytes)
               : "memory");
}

// grid (groups, B), one warp per CTA: lane l < 16 of a step moves row 16 * step
// + l; the loads of one stage fly while the other's rows are stored.  (32 rows a
// stage and three CTAs per SM: 39.8 us against 38.5 for 64 x 4096, 27.8 against
// 26.3 for 4 x 32768, 84.5 against 86.5 for 4 x 131072.)
__global__ void __launch_bounds__(32) evict_move_kernel(const EvictParams p) {
  extern __shared__ __align__(128) uint8_t rows[];
  __shared__ __align__(8) uint64_t full[kMoveStages];
  asm volatile("griddepcontrol.wait;" ::: "memory");
  const int b = blockIdx.y, lane = threadIdx.x;
  const int n = p.n_moves[b];
  const int steps = (n + kMoveRows - 1) / kMoveRows;
  if (static_cast<int>(blockIdx.x) >= steps) return;
  if (lane < kMoveStages) mbar_init(smem_u32(&full[lane]), 1);
  asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
  __syncwarp();
  const int2* moves = p.moves + size_t(b) * p.max_blocks * (kBlock / 2);
  const int32_t* table = p.block_table + size_t(b) * p.max_blocks;
  int abort = 0;
  const WaitCtx wc{p.spin_limit, p.err, &abort};
  const size_t at = size_t(b) * p.max_blocks * kBlock;
  const float* w = p.weight + at;
  const int32_t* pos = p.slot_pos + at;
  float* nw = p.new_weight + at;
  int32_t* np = p.new_pos + at;
  // this lane's move of a step: its slots (x < 0: none), their values, and
  // where the row goes (null: a block id is bad)
  struct Move {
    int2 m;
    float w;
    int pos;
    void* dst;
  };
  auto read = [&](int step, const __nv_bfloat16** src) {
    const int k = lane < kMoveRows ? step * kMoveRows + lane : n;
    Move v = {make_int2(-1, -1), 0.f, 0, nullptr};
    *src = nullptr;
    if (k >= n) return v;
    v.m = moves[k];
    v.w = w[v.m.x];
    v.pos = pos[v.m.x];
    const int sb = table[v.m.x / kBlock], db = table[v.m.y / kBlock];
    if (sb < 0 || sb >= p.num_blocks || db < 0 || db >= p.num_blocks) {
      atomicOr(p.err, kErrBadBlock);
    } else {
      *src = p.cache + (size_t(sb) * kBlock + v.m.x % kBlock) * kRow;
      v.dst = p.cache + (size_t(db) * kBlock + v.m.y % kBlock) * kRow;
    }
    return v;
  };
  auto load = [&](int step, int st) {
    const __nv_bfloat16* src;
    const Move v = read(step, &src);
    const uint32_t bar = smem_u32(&full[st]);
    const int rows_in = __popc(__ballot_sync(0xffffffffu, src != nullptr));
    if (lane == 0) mbar_arrive_expect_tx(bar, rows_in * kRowBytes);
    __syncwarp();
    if (src != nullptr) bulk_load(smem_u32(rows) + (st * kMoveRows + lane) * kRowBytes, src, kRowBytes, bar);
    return v;
  };
  // The values follow a row once it has landed; a token whose row does not
  // move stays in its slot with them, and the slot that waited for it is
  // marked empty.  No other move reads or writes these slots: in place is safe.
  auto publish = [&](const Move& v, bool moved) {
    if (v.m.x < 0) return;
    nw[v.m.y] = moved ? v.w : 0.f;
    np[v.m.y] = moved ? v.pos : -1;
    nw[v.m.x] = moved ? 0.f : v.w;
    np[v.m.x] = moved ? -1 : v.pos;
  };
  const int stride = gridDim.x;
  Move now = load(blockIdx.x, 0);
  uint32_t it = 0;
  for (int step = blockIdx.x; step < steps; step += stride, ++it) {
    const int st = it & 1;
    Move next = {make_int2(-1, -1), 0.f, 0, nullptr};
    if (step + stride < steps) {
      // the other stage's stores have read their rows
      asm volatile("cp.async.bulk.wait_group.read 0;" ::: "memory");
      __syncwarp();
      next = load(step + stride, st ^ 1);
    }
    if (!warp_wait(smem_u32(&full[st]), (it >> 1) & 1u, wc)) {
      publish(now, false);
      publish(next, false);
      const __nv_bfloat16* src;
      for (int s = step + 2 * stride; s < steps; s += stride) publish(read(s, &src), false);
      // loads still in flight land before the CTA exits
      const long long t0 = clock64();
      while (clock64() - t0 < 20000000LL) __nanosleep(1000);
      return;
    }
    if (now.dst != nullptr) bulk_store(now.dst, smem_u32(rows) + (st * kMoveRows + lane) * kRowBytes, kRowBytes);
    publish(now, now.dst != nullptr);
    asm volatile("cp.async.bulk.commit_group;" ::: "memory");
    now = next;
  }
  asm volatile("cp.async.bulk.wait_group 0;" ::: "memory");
}

// Dynamic shared memory above 48 KB, allowed once per device.
template <class Kernel>
cudaError_t allow_shared(Kernel kernel, int bytes, std::atomic<bool> (&done)[64]) {
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= 64) return cudaErrorInvalidDevice;
  if (done[dev].load(std::memory_order_acquire)) return cudaSuccess;
  const cudaError_t e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, bytes);
  if (e == cudaSuccess) done[dev].store(true, std::memory_order_release);
  return e;
}

constexpr int kMaxDyn = kKeysInShared * 4 + kKeysInShared / 4;
static_assert(sizeof(Shared) + kMaxDyn <= 232448 - 1024, "shared memory budget");
static_assert(kMaxCluster * (kMaxDyn * 4LL - 1024) >= kMaxEvictBlocks * static_cast<long long>(kBlock), "bits of the longest sequence");

template <bool kCluster, bool kStored>
cudaError_t launch_select(const EvictParams& p, int size, int room, cudaStream_t stream) {
  const int smem = room / 4 + (kStored ? room * 4 : 0);
  auto kernel = evict_select_kernel<kCluster, kStored>;
  static std::atomic<bool> attr_set[64];
  if (cudaError_t e = allow_shared(kernel, kMaxDyn, attr_set); e != cudaSuccess) return e;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(p.B * size);
  cfg.blockDim = dim3(kSelThreads);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = stream;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim.x = size;
  attr[0].val.clusterDim.y = attr[0].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = kCluster ? 1 : 0;
  return cudaLaunchKernelEx(&cfg, kernel, p, size, room);
}

}  // namespace

cudaError_t launch_evict(const EvictParams& p, int num_sms, cudaStream_t stream) {
  const int sms = num_sms > 0 ? num_sms : 148;
  const long long S = static_cast<long long>(p.max_blocks) * kBlock;
  // More CTAs per sequence while each keeps 4096 slots and all sequences'
  // clusters fit on the device at once; one below 16384 slots, where the
  // cluster barriers cost more than the passes gain (measured, whole call: 4 x
  // 8192 slots 15.5 us with one CTA, 18.4 with two; 1 x 4096 11.7 and 15.6; 16 x
  // 16384 43.5 with four, 55.8 with eight, whose clusters do not all fit).
  int size = 1;
  while (size < kMaxCluster && S >= 16384 && S / (2 * size) >= 4096 && 2LL * size * p.B <= sms) size *= 2;
  // two bits per slot have to fit in any case (evict_layout bounds S)
  while (size < kMaxCluster && (S + size - 1) / size > kMaxDyn * 4 - 1024) size *= 2;
  const int room = static_cast<int>(((S + size - 1) / size + 31) / 32 * 32);
  const bool stored = room <= kKeysInShared;
  cudaError_t e;
  if (size > 1)
    e = stored ? launch_select<true, true>(p, size, room, stream) : launch_select<true, false>(p, size, room, stream);
  else
    e = stored ? launch_select<false, true>(p, size, room, stream) : launch_select<false, false>(p, size, room, stream);
  if (e != cudaSuccess) return e;
  static std::atomic<bool> attr_set[64];
  if ((e = allow_shared(evict_move_kernel, int(kMoveSmem), attr_set)) != cudaSuccess) return e;
  // at most half the slots of a sequence move
  const long long most = (S / 2 + kMoveRows - 1) / kMoveRows;
  const long long even = kMovePerSm * sms / p.B > 1 ? kMovePerSm * sms / p.B : 1;  // no second wave of a few CTAs
  cudaLaunchConfig_t cfg = {};
  cfg.blockDim = dim3(32);
  cfg.dynamicSmemBytes = kMoveSmem;
  cfg.stream = stream;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  // grid.y holds 65535 sequences at most
  for (int b0 = 0; b0 < p.B; b0 += 65535) {
    EvictParams q = p;
    q.n_moves += b0;
    q.moves += size_t(b0) * p.max_blocks * (kBlock / 2);
    q.block_table += size_t(b0) * p.max_blocks;
    q.weight += size_t(b0) * p.max_blocks * kBlock;
    q.slot_pos += size_t(b0) * p.max_blocks * kBlock;
    q.new_weight += size_t(b0) * p.max_blocks * kBlock;
    q.new_pos += size_t(b0) * p.max_blocks * kBlock;
    cfg.gridDim = dim3(static_cast<unsigned>(most < even ? most : even), p.B - b0 < 65535 ? p.B - b0 : 65535);
    if ((e = cudaLaunchKernelEx(&cfg, evict_move_kernel, q)) != cudaSuccess) return e;
  }
  return cudaSuccess;
}

}  // namespace mla
