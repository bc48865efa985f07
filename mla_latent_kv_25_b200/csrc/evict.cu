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
//   largest weight is found by a radix select: four passes of 8 bits over an
//   order-preserving integer image of the weights, which is formed once and
//   stays in shared memory; the CTAs add up their histograms over distributed
//   shared memory.  Ties, free slots and movers are ranked by ballots and
//   prefix sums over warps and CTAs, so the lists are ordered and the result
//   is the same every time.  Bound by the latency of its passes and barriers:
//   16 bytes per slot are read and written.
// evict_move_kernel: bulk copies of whole rows through shared memory, 64 rows
//   in flight per warp.  Bound: HBM, 2304 bytes per moved row.
#include <atomic>

#include "common.cuh"
#include "kernels.h"
#include "sm100.cuh"

namespace mla {
namespace {

using namespace sm100;

constexpr int kSelThreads = 1024;
constexpr int kSelWarps = kSelThreads / 32;
constexpr int kMaxCluster = 8;
// Slots of one CTA whose keys fit in shared memory (4 bytes and one bit each).
constexpr int kKeysInShared = 49152;

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

struct Shared {
  int hist[4][2][256];   // per pass; the first pass has one histogram per class
  int warp_val[kSelWarps];
  int cta_val[6];        // published values: largest position, protected slots, ties, holes, movers
  int pick[2];           // digit, rank within it
};

// Exclusive prefix of `mine` (one value per warp) over the block's warps.
__device__ __forceinline__ int warps_before(Shared& sh, int warp, int lane, int mine, int* total) {
  __syncthreads();
  if (lane == 0) sh.warp_val[warp] = mine;
  __syncthreads();
  const int v = sh.warp_val[lane];
  *total = warp_sum(v);
  return warp_sum(lane < warp ? v : 0);
}

// Publishes a value of this CTA and returns the sum over the CTAs before it
// and over all.
template <bool kCluster>
__device__ __forceinline__ int ctas_before(Shared& sh, int what, int rank, int size, int mine, int* total) {
  if (!kCluster) {
    *total = mine;
    return 0;
  }
  if (threadIdx.x == 0) sh.cta_val[what] = mine;
  cluster_sync();
  int before = 0, all = 0;
  for (int r = 0; r < size; ++r) {
    const int v = ld_cluster(smem_u32(&sh.cta_val[what]), r);
    all += v;
    before += r < rank ? v : 0;
  }
  *total = all;
  return before;
}

// kStored: the keys and the protection bits live in shared memory.
template <bool kCluster, bool kStored>
__global__ void __launch_bounds__(kSelThreads, 1) evict_select_kernel(const EvictParams p, int size, int room) {
  __shared__ Shared sh;
  extern __shared__ uint32_t dyn[];
  uint32_t* keys = dyn;            // [room]
  uint32_t* bits = dyn + room;     // [room / 32] protected slots
  const int b = static_cast<int>(blockIdx.x) / size;
  const int rank = kCluster ? static_cast<int>(cluster_ctarank()) : 0;
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const size_t S = size_t(p.max_blocks) * kBlock;
  const float* w = p.weight + b * S;
  const int32_t* pos = p.slot_pos + b * S;
  const int L = checked_len(p.seq_lens, b, p.max_blocks, threadIdx.x == 0 && rank == 0 ? p.err : nullptr);
  const int n = min(max(p.keep[b], 0), L);
  // this CTA's slots [c0, c1) and this warp's [lo, hi)
  const int share = ((L + size - 1) / size + 31) / 32 * 32;  // <= room
  const int c0 = min(L, rank * share), c1 = min(L, c0 + share);
  const int per = ((c1 - c0 + kSelWarps - 1) / kSelWarps + 31) / 32 * 32;
  const int lo = min(c1, c0 + warp * per), hi = min(c1, lo + per);

  for (int i = threadIdx.x; i < 4 * 2 * 256; i += kSelThreads) (&sh.hist[0][0][0])[i] = 0;

  // the newest position
  int last = INT32_MIN;
#pragma unroll 4
  for (int s = lo + lane; s < hi; s += 32) last = max(last, pos[s]);
  last = warp_max(last);
  if (lane == 0) sh.warp_val[warp] = last;
  __syncthreads();
  last = warp_max(sh.warp_val[lane]);
  if (kCluster) {
    if (threadIdx.x == 0) sh.cta_val[0] = last;
    cluster_sync();
    for (int r = 0; r < size; ++r) last = max(last, ld_cluster(smem_u32(&sh.cta_val[0]), r));
  }
  const long long from = static_cast<long long>(last) - p.n_recent;  // protected: pos > from

  // keys, protection bits, and the histogram of the top digit of each class
  int guarded_here = 0;
#pragma unroll 2
  for (int s0 = lo; s0 < hi; s0 += 32) {
    const int s = s0 + lane;
    const bool in = s < hi;
    const int ps = in ? pos[s] : 0;
    const uint32_t key = in ? weight_key(w[s]) : 0u;
    const bool g = in && (ps < p.n_first || ps > from);
    const unsigned gm = __ballot_sync(0xffffffffu, g);
    if (kStored) {
      if (in) keys[s - c0] = key;
      if (lane == 0) bits[(s0 - c0) >> 5] = gm;
    }
    guarded_here += __popc(gm);
    const int bin = in ? static_cast<int>((g ? 256u : 0u) | (key >> 24)) : -1;
    const unsigned same = __match_any_sync(0xffffffffu, bin);  // weights share few exponents
    if (in && lane == __ffs(same) - 1) atomicAdd(&sh.hist[0][0][0] + bin, __popc(same));
  }
  int total, n_guarded;
  warps_before(sh, warp, lane, guarded_here, &total);
  ctas_before<kCluster>(sh, 1, rank, size, total, &n_guarded);
  // either some protected slots go too, or all stay and the others compete
  const bool among_guarded = n_guarded >= n;
  int need = among_guarded ? n : n - n_guarded;  // kept of the competing class

  auto guarded = [&](int s) -> bool {
    if (kStored) return (bits[(s - c0) >> 5] >> ((s - c0) & 31)) & 1u;
    return pos[s] < p.n_first || pos[s] > from;
  };
  auto key_of = [&](int s) -> uint32_t { return kStored ? keys[s - c0] : weight_key(w[s]); };

  // radix select: the competing slots with key > thr are kept, and of those
  // with key == thr the first `need`.  need = 0 keeps none (thr = the largest key).
  uint32_t thr = 0;
  if (need == 0) {
    thr = 0xffffffffu;
  } else {
    for (int pass = 0; pass < 4; ++pass) {
      const int shift = 24 - 8 * pass;
      int* hist = sh.hist[pass][pass == 0 && among_guarded ? 1 : 0];
      if (pass > 0) {
        for (int s0 = lo; s0 < hi; s0 += 32) {
          const int s = s0 + lane;
          if (s < hi) {
            const uint32_t key = key_of(s);
            if ((key >> (shift + 8)) == (thr >> (shift + 8)) && guarded(s) == among_guarded)
              atomicAdd(&hist[(key >> shift) & 255u], 1);
          }
        }
        if (kCluster)
          cluster_sync();
        else
          __syncthreads();
      }
      if (warp == 0) {
        // lane l holds digits 255-8l .. 248-8l, from the largest down
        int c[8], sum = 0;
#pragma unroll
        for (int k = 0; k < 8; ++k) {
          const int digit = 255 - 8 * lane - k;
          c[k] = 0;
          if (kCluster) {
            for (int r = 0; r < size; ++r) c[k] += ld_cluster(smem_u32(&hist[digit]), r);
          } else {
            c[k] = hist[digit];
          }
          sum += c[k];
        }
        int incl = sum;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
          const int v = __shfl_up_sync(0xffffffffu, incl, o);
          if (lane >= o) incl += v;
        }
        int before = incl - sum;
        if (before < need && need <= incl) {
#pragma unroll
          for (int k = 0; k < 8; ++k) {
            if (before < need && need <= before + c[k]) {
              sh.pick[0] = 255 - 8 * lane - k;
              sh.pick[1] = need - before;
            }
            before += c[k];
          }
        }
      }
      __syncthreads();
      thr |= static_cast<uint32_t>(sh.pick[0]) << shift;
      need = sh.pick[1];
      __syncthreads();
    }
  }

  auto above = [&](int s, bool* tie) -> bool {
    const bool g = guarded(s);
    if (g != among_guarded) {
      *tie = false;
      return g;  // a protected slot while the others compete stays
    }
    const uint32_t key = key_of(s);
    *tie = key == thr;
    return key > thr;
  };
  int count = 0;
  for (int s0 = lo; s0 < hi; s0 += 32) {
    bool tie = false;
    if (s0 + lane < hi) above(s0 + lane, &tie);
    count += tie ? 1 : 0;
  }
  int ties0 = warps_before(sh, warp, lane, warp_sum(count), &total);
  int all;
  ties0 += ctas_before<kCluster>(sh, 2, rank, size, total, &all);
  // kept flags, 32 slots at a time, in slot order
  auto walk = [&](auto&& visit) {
    int ties = ties0;
    for (int s0 = lo; s0 < hi; s0 += 32) {
      const int s = s0 + lane;
      bool tie = false, kept = false;
      if (s < hi) kept = above(s, &tie);
      const unsigned m = __ballot_sync(0xffffffffu, tie);
      if (tie) kept = ties + __popc(m & ((1u << lane) - 1u)) < need;
      ties += __popc(m);
      visit(s, s < hi, kept);
    }
  };
  int holes = 0, movers = 0;
  walk([&](int s, bool in, bool kept) {
    holes += (in && !kept && s < n) ? 1 : 0;
    movers += (in && kept && s >= n) ? 1 : 0;
  });
  int n_moves;
  int hole0 = warps_before(sh, warp, lane, warp_sum(holes), &total);
  hole0 += ctas_before<kCluster>(sh, 3, rank, size, total, &all);
  int mover0 = warps_before(sh, warp, lane, warp_sum(movers), &total);
  mover0 += ctas_before<kCluster>(sh, 4, rank, size, total, &n_moves);
  int2* moves = p.moves + b * (S / 2);
  walk([&](int s, bool in, bool kept) {
    const bool hole = in && !kept && s < n, mover = in && kept && s >= n;
    const unsigned mh = __ballot_sync(0xffffffffu, hole), mm = __ballot_sync(0xffffffffu, mover);
    const unsigned below = (1u << lane) - 1u;
    if (hole) moves[hole0 + __popc(mh & below)].y = s;
    if (mover) moves[mover0 + __popc(mm & below)].x = s;
    hole0 += __popc(mh);
    mover0 += __popc(mm);
  });
  if (threadIdx.x == 0 && rank == 0) p.n_moves[b] = n_moves;

  // the small arrays: the slots that stay, the moved values (read before any
  // freed slot is cleared: they may live in the same arrays), the freed tail
  float* nw = p.new_weight + b * S;
  int32_t* np = p.new_pos + b * S;
  const int tid = rank * kSelThreads + threadIdx.x, threads = size * kSelThreads;
  if (nw != w || np != pos)
    for (int s = tid; s < n; s += threads) {
      nw[s] = w[s];
      np[s] = pos[s];
    }
  // a cluster barrier releases and acquires global writes of its CTAs too
  if (kCluster)
    cluster_sync();
  else
    __syncthreads();
  for (int k = tid; k < n_moves; k += threads) {
    const int2 m = moves[k];
    nw[m.y] = w[m.x];
    np[m.y] = pos[m.x];
  }
  if (kCluster)
    cluster_sync();
  else
    __syncthreads();
  for (int s = n + tid; s < L; s += threads) {
    nw[s] = 0.f;
    np[s] = -1;
  }
  if (threadIdx.x == 0 && rank == 0) p.new_lens[b] = n;
}

constexpr int kMoveRows = 32;                        // rows of a stage, one per lane
constexpr int kMoveStages = 2;
constexpr uint32_t kRowBytes = kRow * 2;
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

// grid (groups, B), one warp per CTA (three fit on an SM): lane l of a step
// moves row 32 * step + l; the loads of one stage fly while the other's rows
// are stored.
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
  void* dst[kMoveStages] = {nullptr, nullptr};
  auto load = [&](int step, int st) {
    const int k = step * kMoveRows + lane;
    const __nv_bfloat16* src = nullptr;
    dst[st] = nullptr;
    if (k < n) {
      const int2 m = moves[k];
      const int sb = table[m.x / kBlock], db = table[m.y / kBlock];
      if (sb < 0 || sb >= p.num_blocks || db < 0 || db >= p.num_blocks) {
        atomicOr(p.err, kErrBadBlock);
      } else {
        src = p.cache + (size_t(sb) * kBlock + m.x % kBlock) * kRow;
        dst[st] = p.cache + (size_t(db) * kBlock + m.y % kBlock) * kRow;
      }
    }
    const uint32_t bar = smem_u32(&full[st]);
    const int rows_in = __popc(__ballot_sync(0xffffffffu, src != nullptr));
    if (lane == 0) mbar_arrive_expect_tx(bar, rows_in * kRowBytes);
    __syncwarp();
    if (src != nullptr) bulk_load(smem_u32(rows) + (st * kMoveRows + lane) * kRowBytes, src, kRowBytes, bar);
  };
  load(blockIdx.x, 0);
  uint32_t it = 0;
  for (int step = blockIdx.x; step < steps; step += gridDim.x, ++it) {
    const int st = it & 1;
    if (step + static_cast<int>(gridDim.x) < steps) {
      // the other stage's stores have read their rows
      asm volatile("cp.async.bulk.wait_group.read 0;" ::: "memory");
      __syncwarp();
      load(step + gridDim.x, st ^ 1);
    }
    if (!warp_wait(smem_u32(&full[st]), (it >> 1) & 1u, wc)) {
      // loads still in flight land before the CTA exits
      const long long t0 = clock64();
      while (clock64() - t0 < 20000000LL) __nanosleep(1000);
      return;
    }
    if (dst[st] != nullptr) bulk_store(dst[st], smem_u32(rows) + (st * kMoveRows + lane) * kRowBytes, kRowBytes);
    asm volatile("cp.async.bulk.commit_group;" ::: "memory");
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

template <bool kCluster, bool kStored>
cudaError_t launch_select(const EvictParams& p, int size, int room, cudaStream_t stream) {
  const int smem = kStored ? room * 4 + room / 8 : 0;
  auto kernel = evict_select_kernel<kCluster, kStored>;
  static std::atomic<bool> attr_set[64];
  if (cudaError_t e = allow_shared(kernel, kKeysInShared * 4 + kKeysInShared / 8, attr_set); e != cudaSuccess) return e;
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
  return cudaLaunchKernelEx(&cfg, kernel, p, size, kStored ? room : 0);
}

}  // namespace

cudaError_t launch_evict(const EvictParams& p, int num_sms, cudaStream_t stream) {
  const int sms = num_sms > 0 ? num_sms : 148;
  const long long S = static_cast<long long>(p.max_blocks) * kBlock;
  // More CTAs per sequence while each keeps 4096 slots and all sequences'
  // clusters fit on the device at once; one below 16384 slots, where the
  // cluster barriers cost more than the passes gain (measured, whole call: 4 x
  // 8192 slots 24 us with one CTA, 33 with two; 16 x 16384 72 with two, 64 with
  // four; 4 x 32768 81 with one, 48 with eight).
  int size = 1;
  while (size < kMaxCluster && S >= 16384 && S / (2 * size) >= 4096 && 2LL * size * p.B <= sms) size *= 2;
  const long long room = ((S + size - 1) / size + 31) / 32 * 32;
  const bool stored = room <= kKeysInShared;
  cudaError_t e;
  if (size > 1)
    e = stored ? launch_select<true, true>(p, size, static_cast<int>(room), stream)
               : launch_select<true, false>(p, size, 0, stream);
  else
    e = stored ? launch_select<false, true>(p, size, static_cast<int>(room), stream)
               : launch_select<false, false>(p, size, 0, stream);
  if (e != cudaSuccess) return e;
  static std::atomic<bool> attr_set[64];
  if ((e = allow_shared(evict_move_kernel, int(kMoveSmem), attr_set)) != cudaSuccess) return e;
  // at most half the slots of a sequence move; three CTAs per SM in all
  const long long most = (S / 2 + kMoveRows - 1) / kMoveRows;
  const long long even = (3LL * sms + p.B - 1) / p.B;
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
    cfg.gridDim = dim3(static_cast<unsigned>(most < even ? most : even), p.B - b0 < 65535 ? p.B - b0 : 65535);
    if ((e = cudaLaunchKernelEx(&cfg, evict_move_kernel, q)) != cudaSuccess) return e;
  }
  return cudaSuccess;
}

}  // namespace mla
