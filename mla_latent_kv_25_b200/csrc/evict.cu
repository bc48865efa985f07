// Eviction from the paged cache by accumulated attention weight.
//
// Per sequence of L tokens and budget n: rank the slots by (protected, weight,
// lower slot), keep the first n, and move the kept rows behind slot n into the
// free slots before it (k-th to k-th).  Kept rows before slot n stay, sources
// lie at or past n and destinations before it, so no move reads what another
// writes and all moves can run at once.
//
// evict_select_kernel: one CTA per sequence.  The n-th largest weight is found
//   by a radix select (four passes of 8 bits over an order-preserving integer
//   image of the weights); then every warp owns a contiguous range of slots
//   and ranks its ties, free slots and movers by ballots and a scan over the
//   warps, which makes the lists ordered and the result the same every time.
// evict_move_kernel: 16-byte units of the moved rows, spread over the device.
//
// Bound: HBM, 16 bytes per slot of weights and positions and 2304 bytes per
// moved row; the select is bound by the passes over one sequence's weights
// (L2 resident) of one SM.
#include "common.cuh"
#include "kernels.h"

namespace mla {
namespace {

constexpr int kSelThreads = 1024;
constexpr int kSelWarps = kSelThreads / 32;

// Order-preserving image of a weight: larger weight, larger key; -0 equals +0,
// NaN ranks as -inf.
__device__ __forceinline__ uint32_t weight_key(float w) {
  if (w != w) w = -INFINITY;
  w += 0.f;  // -0 -> +0
  const uint32_t u = __float_as_uint(w);
  return (u & 0x80000000u) ? ~u : (u | 0x80000000u);
}

__device__ __forceinline__ int warp_sum(int v) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
  return v;
}

__device__ __forceinline__ int warp_max(int v) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) v = max(v, __shfl_xor_sync(0xffffffffu, v, o));
  return v;
}

// Exclusive prefix over the warps' values (every thread of the block calls it).
__device__ __forceinline__ int warps_before(int* buf, int warp, int lane, int mine, int* total) {
  __syncthreads();
  if (lane == 0) buf[warp] = mine;
  __syncthreads();
  const int v = buf[lane];
  const int before = warp_sum(lane < warp ? v : 0);
  if (total) *total = warp_sum(v);
  return before;
}

__global__ void __launch_bounds__(kSelThreads) evict_select_kernel(const EvictParams p) {
  __shared__ int hist[256];
  __shared__ int buf[kSelWarps];
  __shared__ int pick[2];  // digit, rank within it
  const int b = blockIdx.x;
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const size_t S = size_t(p.max_blocks) * kBlock;
  const float* w = p.weight + b * S;
  const int32_t* pos = p.slot_pos + b * S;
  const int L = checked_len(p.seq_lens, b, p.max_blocks, threadIdx.x == 0 ? p.err : nullptr);
  const int n = min(max(p.keep[b], 0), L);

  // the newest position, and how many slots are protected
  int last = INT32_MIN;
  for (int s = threadIdx.x; s < L; s += kSelThreads) last = max(last, pos[s]);
  last = warp_max(last);
  if (lane == 0) buf[warp] = last;
  __syncthreads();
  last = warp_max(buf[lane]);
  const long long from = static_cast<long long>(last) - p.n_recent;  // protected: pos > from
  auto guarded = [&](int s) { return pos[s] < p.n_first || pos[s] > from; };
  int count = 0;
  for (int s = threadIdx.x; s < L; s += kSelThreads) count += guarded(s) ? 1 : 0;
  int n_guarded;
  warps_before(buf, warp, lane, warp_sum(count), &n_guarded);
  // either some protected slots go too, or all stay and the others compete
  const bool among_guarded = n_guarded >= n;
  int need = among_guarded ? n : n - n_guarded;  // kept of the competing class

  // radix select: the competing slots with key > thr are kept, and of those
  // with key == thr the first `need`.  need = 0 keeps none (thr = the largest key).
  uint32_t thr = 0;
  if (need == 0) {
    thr = 0xffffffffu;
  } else {
    for (int shift = 24; shift >= 0; shift -= 8) {
      for (int i = threadIdx.x; i < 256; i += kSelThreads) hist[i] = 0;
      __syncthreads();
      for (int s0 = warp * 32; s0 < L; s0 += kSelThreads) {
        const int s = s0 + lane;
        bool in = s < L && guarded(s) == among_guarded;
        uint32_t key = 0;
        if (in) {
          key = weight_key(w[s]);
          in = shift == 24 || (key >> (shift + 8)) == (thr >> (shift + 8));
        }
        const int digit = in ? static_cast<int>((key >> shift) & 255u) : -1;
        const unsigned same = __match_any_sync(0xffffffffu, digit);
        if (in && lane == __ffs(same) - 1) atomicAdd(&hist[digit], __popc(same));
      }
      __syncthreads();
      if (warp == 0) {
        // lane l holds digits 255-8l .. 248-8l, from the largest down
        int c[8], sum = 0;
#pragma unroll
        for (int k = 0; k < 8; ++k) sum += c[k] = hist[255 - 8 * lane - k];
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
              pick[0] = 255 - 8 * lane - k;
              pick[1] = need - before;
            }
            before += c[k];
          }
        }
      }
      __syncthreads();
      thr |= static_cast<uint32_t>(pick[0]) << shift;
      need = pick[1];
    }
  }

  // every warp owns the slots [lo, hi)
  const int per = ((L + kSelWarps - 1) / kSelWarps + 31) / 32 * 32;
  const int lo = min(L, warp * per), hi = min(L, lo + per);
  auto above = [&](int s, bool* tie) {
    const bool g = guarded(s);
    if (g != among_guarded) {
      *tie = false;
      return g;  // a protected slot while the others compete stays
    }
    const uint32_t key = weight_key(w[s]);
    *tie = key == thr;
    return key > thr;
  };
  count = 0;
  for (int s0 = lo; s0 < hi; s0 += 32) {
    bool tie = false;
    if (s0 + lane < hi) above(s0 + lane, &tie);
    count += tie ? 1 : 0;
  }
  const int ties0 = warps_before(buf, warp, lane, warp_sum(count), nullptr);
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
  int hole0 = warps_before(buf, warp, lane, warp_sum(holes), nullptr);
  int mover0 = warps_before(buf, warp, lane, warp_sum(movers), &n_moves);
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
  if (threadIdx.x == 0) p.n_moves[b] = n_moves;
  __syncthreads();

  // the small arrays: moved values first (they may live in the same arrays),
  // the slots that stay, then the freed tail
  float* nw = p.new_weight + b * S;
  int32_t* np = p.new_pos + b * S;
  if (nw != w || np != pos) {
    for (int s = threadIdx.x; s < n; s += kSelThreads) {
      nw[s] = w[s];
      np[s] = pos[s];
    }
    __syncthreads();
  }
  for (int k = threadIdx.x; k < n_moves; k += kSelThreads) {
    const int2 m = moves[k];
    nw[m.y] = w[m.x];
    np[m.y] = pos[m.x];
  }
  __syncthreads();
  for (int s = n + threadIdx.x; s < L; s += kSelThreads) {
    nw[s] = 0.f;
    np[s] = -1;
  }
  if (threadIdx.x == 0) p.new_lens[b] = n;
}

constexpr int kMoveThreads = 256;
constexpr int kRowUnits = kRow / 8;  // 16-byte units of a row

__global__ void __launch_bounds__(kMoveThreads) evict_move_kernel(const EvictParams p) {
  const int b = blockIdx.y;
  const long long total = static_cast<long long>(p.n_moves[b]) * kRowUnits;
  const int2* moves = p.moves + size_t(b) * p.max_blocks * (kBlock / 2);
  const int32_t* table = p.block_table + size_t(b) * p.max_blocks;
  uint4* cache = reinterpret_cast<uint4*>(p.cache);
  const long long step = static_cast<long long>(gridDim.x) * kMoveThreads;
  for (long long u0 = static_cast<long long>(blockIdx.x) * kMoveThreads + threadIdx.x; u0 < total; u0 += 4 * step) {
    uint4 v[4];
    long long to[4];
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      const long long u = u0 + k * step;
      to[k] = -1;
      if (u >= total) continue;
      const int2 m = moves[u / kRowUnits];
      const int c = static_cast<int>(u % kRowUnits);
      const int sb = table[m.x / kBlock], db = table[m.y / kBlock];
      if (sb < 0 || sb >= p.num_blocks || db < 0 || db >= p.num_blocks) {
        atomicOr(p.err, kErrBadBlock);
        continue;
      }
      v[k] = cache[(static_cast<long long>(sb) * kBlock + m.x % kBlock) * kRowUnits + c];
      to[k] = (static_cast<long long>(db) * kBlock + m.y % kBlock) * kRowUnits + c;
    }
#pragma unroll
    for (int k = 0; k < 4; ++k)
      if (to[k] >= 0) cache[to[k]] = v[k];
  }
}

}  // namespace

cudaError_t launch_evict(const EvictParams& p, int num_sms, cudaStream_t stream) {
  evict_select_kernel<<<p.B, kSelThreads, 0, stream>>>(p);
  if (cudaError_t e = cudaGetLastError(); e != cudaSuccess) return e;
  // at most half the slots of a sequence move; about eight CTAs per SM in all
  const long long most = (static_cast<long long>(p.max_blocks) * (kBlock / 2) * kRowUnits + 4 * kMoveThreads - 1) /
                         (4 * kMoveThreads);
  const long long share = (8LL * (num_sms > 0 ? num_sms : 148) + p.B - 1) / p.B;
  const int gx = static_cast<int>(most < share ? most : share);
  // grid.y holds 65535 sequences at most
  for (int b0 = 0; b0 < p.B; b0 += 65535) {
    EvictParams q = p;
    q.n_moves += b0;
    q.moves += size_t(b0) * p.max_blocks * (kBlock / 2);
    q.block_table += size_t(b0) * p.max_blocks;
    evict_move_kernel<<<dim3(gx, p.B - b0 < 65535 ? p.B - b0 : 65535), kMoveThreads, 0, stream>>>(q);
    if (cudaError_t e = cudaGetLastError(); e != cudaSuccess) return e;
  }
  return cudaSuccess;
}

}  // namespace mla
