// Attention weight per cached token on tcgen05 tensor cores:
//   weight_out[b,t] = weight_in[b,t] + sum_{j,h} exp(scale q[j,h] . row_t - lse[j,h])
//
// Cached tokens are the M = 128 dimension (two 64-token blocks), query rows
// (token j, head h) the N dimension, so a TMEM lane holds one token's scores
// and the sum over heads and queries is a sum along the lane: no shuffles, no
// atomics, one fixed order.
//
// Bound: with one query token per sequence the cache is read once and the
// kernel is bound by HBM (1152 bytes per token); with many query tokens by
// the tensor pipe.  A persistent CTA per SM takes a contiguous range of the
// concatenated block list (SegWalker).  Both operands of a tile are 128 rows
// of 576 bf16 in nine 128-byte-swizzled chunks, so one may stay in shared
// memory while the other streams through a ring of 16 KB chunks:
//   a sequence with one query tile (<= 128 rows): the queries stay, the cache
//     streams past them (every cached row is fetched once);
//   more query tiles: a tile of 128 tokens stays, the queries stream (from L2).
//
// w0: TMA; w1: MMA (one thread), TMEM; w2-5: epilogue, thread = token.
#include <cuda.h>
#include <math.h>

#include <atomic>

#include "common.cuh"
#include "kernels.h"
#include "pair.cuh"
#include "schedule.cuh"
#include "sm100.cuh"

namespace mla {

// Error word of mla_cache_weigh (the call has no workspace); read and cleared
// by mla_cache_get_error.
__device__ uint32_t g_weigh_err;

namespace {

using namespace sm100;

constexpr int kThreads = 192;
constexpr int kTileTok = 128;                 // tokens per tile (two blocks)
constexpr int kChunks = kRow / 64;            // 64-column chunks of a row
constexpr uint32_t kChunk = 128 * 128;        // [128 rows x 64] bf16
constexpr int kRing = 5;
constexpr int kAcc = 2;                       // accumulators [128 x 128] fp32 in TMEM
constexpr uint32_t kTmemCols = 256;
constexpr float kLog2e = 1.4426950408889634f;

struct Bars {
  uint64_t ring_full[kRing], ring_empty[kRing];
  uint64_t res_full, res_empty;
  uint64_t acc_full[kAcc], acc_empty[kAcc];
  uint32_t tmem_base;
  int abort;
};
static_assert(sizeof(Bars) <= 1024, "barrier block too large");

constexpr uint32_t kResOff = 1024;
constexpr uint32_t kRingOff = kResOff + kChunks * kChunk;
constexpr uint32_t kSmem = kRingOff + kRing * kChunk + 1024;
static_assert(kSmem <= 232448, "shared memory budget");

struct Queries {
  int n;        // query tokens of the sequence
  int row0;     // first row of q
  int rows;     // n * H
  int tiles;    // of 128 rows
};

__device__ __forceinline__ Queries queries_of(const WeighParams& p, int b) {
  const int a = p.q_offsets[b], e = p.q_offsets[b + 1];
  Queries q;
  q.n = a >= 0 && e >= a && e <= p.T ? e - a : 0;
  q.row0 = a * p.H;
  q.rows = q.n * p.H;
  q.tiles = (q.rows + 127) / 128;
  return q;
}

struct Ctx {
  const WeighParams* p;
  uint32_t base;
  Bars* bars;
  uint32_t tmem;
  WaitCtx wc;
  int warp, lane;
};

__device__ __forceinline__ uint32_t bar_addr(const uint64_t& b) { return smem_u32(&b); }

__device__ __forceinline__ int safe_block(const WeighParams& p, const Segment& g, int j) {
  const int id = j < g.blk_hi ? p.block_table[size_t(g.b) * p.max_blocks + j] : 0;
  return id >= 0 && id < p.num_blocks ? id : 0;
}

// One 128-row operand chunk: query rows from `row`, or the two blocks of a tile.
__device__ __forceinline__ void load_q_chunk(const CUtensorMap* qmap, uint32_t dst, int ch, int row, uint32_t bar) {
  tma_load_2d(dst, qmap, 64 * ch, row, bar);
}
__device__ __forceinline__ void load_k_chunk(const CUtensorMap* kmap, uint32_t dst, int ch, int blk0, int blk1,
                                             uint32_t bar) {
  tma_load_2d(dst, kmap, 64 * ch, blk0 * kBlock, bar);
  tma_load_2d(dst + kChunk / 2, kmap, 64 * ch, blk1 * kBlock, bar);
}

// The producer's loop over one segment (one thread).
__device__ __forceinline__ bool produce(const Ctx& c, const CUtensorMap* qmap, const CUtensorMap* kmap, const Segment& g,
                        const Queries& q, uint32_t& rit, uint32_t& fit) {
  const WeighParams& p = *c.p;
  Bars* bars = c.bars;
  const bool queries_stay = q.tiles == 1;
  auto resident = [&]() {
    const bool ok = wait_phase(bar_addr(bars->res_empty), (rit & 1u) ^ 1u, c.wc);
    ++rit;
    if (ok) mbar_arrive_expect_tx(bar_addr(bars->res_full), kChunks * kChunk);
    return ok;
  };
  const uint32_t res_bar = bar_addr(bars->res_full);
  if (queries_stay) {
    if (!resident()) return false;
    for (int ch = 0; ch < kChunks; ++ch) load_q_chunk(qmap, c.base + kResOff + ch * kChunk, ch, q.row0, res_bar);
  }
  for (int j = g.blk_lo; j < g.blk_hi; j += 2) {
    const int b0 = safe_block(p, g, j), b1 = safe_block(p, g, j + 1);
    if (!queries_stay) {
      if (!resident()) return false;
      for (int ch = 0; ch < kChunks; ++ch) load_k_chunk(kmap, c.base + kResOff + ch * kChunk, ch, b0, b1, res_bar);
    }
    const int streams = queries_stay ? 1 : q.tiles;
    for (int i = 0; i < streams; ++i)
      for (int ch = 0; ch < kChunks; ++ch, ++fit) {
        const int s = fit % kRing;
        if (!wait_phase(bar_addr(bars->ring_empty[s]), ((fit / kRing) & 1u) ^ 1u, c.wc)) return false;
        const uint32_t full = bar_addr(bars->ring_full[s]);
        const uint32_t dst = c.base + kRingOff + s * kChunk;
        mbar_arrive_expect_tx(full, kChunk);
        if (queries_stay)
          load_k_chunk(kmap, dst, ch, b0, b1, full);
        else
          load_q_chunk(qmap, dst, ch, q.row0 + 128 * i, full);
      }
  }
  return true;
}

// The MMA warp's loop over one segment (its elected thread); the next chunk's
// barrier is probed before the current chunk's MMAs are issued.
__device__ __forceinline__ bool multiply(const Ctx& c, int tiles, const Queries& q, uint32_t& rit, uint32_t& slot,
                                         uint32_t& phase, uint32_t& ait) {
  Bars* bars = c.bars;
  const bool queries_stay = q.tiles == 1;
  const uint32_t full0 = bar_addr(bars->ring_full[0]), empty0 = bar_addr(bars->ring_empty[0]);
  const uint64_t res0 = sw128_desc(c.base + kResOff, 16, 1024), ring0 = sw128_desc(c.base + kRingOff, 16, 1024);
  auto wait_resident = [&]() {
    const bool ok = wait_phase(bar_addr(bars->res_full), rit & 1u, c.wc);
    ++rit;
    return ok;
  };
  bool ready = false;
  if (queries_stay && !wait_resident()) return false;
  for (int j = 0; j < tiles; ++j) {
    if (!queries_stay && !wait_resident()) return false;
    const int streams = queries_stay ? 1 : q.tiles;
    for (int i = 0; i < streams; ++i, ++ait) {
      const int buf = ait % kAcc;
      // the last tile of a sequence may have fewer rows (a multiple of 16)
      const uint32_t idesc = idesc_bf16(128, min(128, q.rows - 128 * i), false, false);
      const uint32_t d = c.tmem + 128 * buf;
      if (!wait_phase(bar_addr(bars->acc_empty[buf]), ((ait / kAcc) & 1u) ^ 1u, c.wc)) return false;
      tc_fence_after();
#pragma unroll 1
      for (int ch = 0; ch < kChunks; ++ch) {
        if (!ready && !wait_phase(full0 + 8 * slot, phase, c.wc)) return false;
        const uint32_t s = slot;
        if (++slot == kRing) {
          slot = 0;
          phase ^= 1u;
        }
        ready = mbar_test_wait(full0 + 8 * slot, phase);
        const uint64_t res = res0 + static_cast<uint32_t>(ch) * (kChunk >> 4), str = ring0 + s * (kChunk >> 4);
        const uint64_t a = queries_stay ? str : res, bq = queries_stay ? res : str;
#pragma unroll
        for (int kk = 0; kk < 4; ++kk) mma_ss(d, a + 2 * kk, bq + 2 * kk, idesc, (ch | kk) ? 1u : 0u);
        mma_commit(empty0 + 8 * s);
      }
      mma_commit(bar_addr(bars->acc_full[buf]));
    }
    if (!queries_stay) mma_commit(bar_addr(bars->res_empty));
  }
  if (queries_stay) mma_commit(bar_addr(bars->res_empty));
  return true;
}

// lse of the 128 rows of a query tile in base 2: lane l holds rows l, l + 32, l + 64, l + 96.
__device__ __forceinline__ void load_lse(const WeighParams& p, const Queries& q, int i, int lane, float (&l)[4]) {
#pragma unroll
  for (int k = 0; k < 4; ++k) {
    const int r = 128 * i + 32 * k + lane;
    l[k] = r < q.rows ? p.lse[static_cast<size_t>(q.row0) + r] * kLog2e : INFINITY;
  }
}

__device__ __forceinline__ bool accumulate(const Ctx& c, const Segment& g, const Queries& q, uint32_t& ait) {
  const WeighParams& p = *c.p;
  Bars* bars = c.bars;
  const int quad = c.warp & 3;
  const int row = quad * 32 + c.lane;  // TMEM lane: token of the tile
  const uint32_t lane_off = static_cast<uint32_t>(quad * 32) << 16;
  const float sl2 = p.softmax_scale * kLog2e;
  const size_t S = size_t(p.max_blocks) * kBlock;
  const int len_off = g.len - (q.n - 1);  // query token j sees the first len_off + j rows
  float l[4];
  if (q.tiles == 1) load_lse(p, q, 0, c.lane, l);
  for (int j = g.blk_lo; j < g.blk_hi; j += 2) {
    const int tok = j * kBlock + row;
    const int last = min(j * kBlock + kTileTok, g.len) - 1;
    float sum[4] = {0.f, 0.f, 0.f, 0.f};
    for (int i = 0; i < q.tiles; ++i, ++ait) {
      if (q.tiles > 1) load_lse(p, q, i, c.lane, l);
      const int buf = ait % kAcc;
      if (!warp_wait(bar_addr(bars->acc_full[buf]), (ait / kAcc) & 1u, c.wc)) return false;
      tc_fence_after();
      const int cols = min(128, q.rows - 128 * i);  // a multiple of 16
      const uint32_t taddr = c.tmem + lane_off + 128 * buf;
      // whether the tile's first row, which sees least, sees the tile's last token
      const bool seen = last < len_off + 128 * i / p.H;
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        if (32 * k >= cols) break;
        uint32_t v[32];
        tmem_ld32(taddr + 32 * k, v);
        tmem_ld_wait();
        if (seen && 32 * k + 32 <= cols) {
#pragma unroll
          for (int e = 0; e < 32; ++e)
            sum[e & 3] += ex2_approx(fmaf(__uint_as_float(v[e]), sl2, -__shfl_sync(0xffffffffu, l[k], e)));
        } else {
          // 16 columns at a time belong to one query token (H is a multiple of 16)
#pragma unroll
          for (int half = 0; half < 2; ++half) {
            const int c0 = 32 * k + 16 * half;
            const bool in = c0 < cols && tok < len_off + (128 * i + c0) / p.H;
#pragma unroll
            for (int e = 16 * half; e < 16 * half + 16; ++e) {
              const float x = ex2_approx(fmaf(__uint_as_float(v[e]), sl2, -__shfl_sync(0xffffffffu, l[k], e)));
              if (in) sum[e & 3] += x;
            }
          }
        }
      }
      tc_fence_before();
      __syncwarp();
      if (c.lane == 0) mbar_arrive(bar_addr(bars->acc_empty[buf]));
    }
    if (tok < g.len && j + (row >> 6) < g.blk_hi) {
      const int id = p.block_table[size_t(g.b) * p.max_blocks + tok / kBlock];
      const bool ok = id >= 0 && id < p.num_blocks;
      if (!ok && (row & 63) == 0) atomicOr(&g_weigh_err, kErrBadBlock);
      const size_t at = g.b * S + tok;
      const float w = p.weight_in != nullptr ? p.weight_in[at] : 0.f;
      p.weight_out[at] = ok ? w + ((sum[0] + sum[1]) + (sum[2] + sum[3])) : w;
    }
  }
  return true;
}

__global__ void __launch_bounds__(kThreads, 1)
weigh_sm100_kernel(const __grid_constant__ CUtensorMap qmap, const __grid_constant__ CUtensorMap kmap,
                   const WeighParams p) {
  extern __shared__ __align__(1024) uint8_t smem_raw[];
  const uint32_t raw = smem_u32(smem_raw);
  const uint32_t base = (raw + 1023u) & ~1023u;
  Bars* bars = reinterpret_cast<Bars*>(smem_raw + (base - raw));
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  if (threadIdx.x == 0) {
    for (int s = 0; s < kRing; ++s) {
      mbar_init(bar_addr(bars->ring_full[s]), 1);
      mbar_init(bar_addr(bars->ring_empty[s]), 1);
    }
    mbar_init(bar_addr(bars->res_full), 1);
    mbar_init(bar_addr(bars->res_empty), 1);
    for (int s = 0; s < kAcc; ++s) {
      mbar_init(bar_addr(bars->acc_full[s]), 1);
      mbar_init(bar_addr(bars->acc_empty[s]), 4);  // lane 0 of every epilogue warp
    }
    bars->abort = 0;
    fence_mbar_init();
    prefetch_tmap(&qmap);
    prefetch_tmap(&kmap);
  }
  if (warp == 1) {
    tmem_alloc(smem_u32(&bars->tmem_base), kTmemCols);
    tmem_relinquish();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  Ctx c;
  c.p = &p;
  c.base = base;
  c.bars = bars;
  c.tmem = bars->tmem_base;
  c.wc = WaitCtx{p.spin_limit, &g_weigh_err, &bars->abort};
  c.warp = warp;
  c.lane = lane;

  if (blockIdx.x == 0)  // bad lengths and offsets, once
    for (int b = threadIdx.x; b < p.B; b += kThreads) {
      checked_len(p.seq_lens, b, p.max_blocks, &g_weigh_err);
      if (p.q_offsets[b] < 0 || p.q_offsets[b + 1] < p.q_offsets[b] || p.q_offsets[b + 1] > p.T)
        atomicOr(&g_weigh_err, kErrSeqTooLong);
    }

  SegWalker w;
  w.init(p.seq_lens, p.B, p.max_blocks, gridDim.x, blockIdx.x);
  Segment gs;
  uint32_t rit = 0, fit = 0, ait = 0, slot = 0, phase = 0;
  while (w.next(gs)) {
    const Segment g = gs;  // in registers, not behind the walker's reference
    const Queries q = queries_of(p, g.b);
    int ok = 1;
    if (warp == 0) {
      if (q.tiles > 0 && lane == 0) ok = produce(c, &qmap, &kmap, g, q, rit, fit) ? 1 : 0;
      ok = __shfl_sync(0xffffffffu, ok, 0);
    } else if (warp == 1) {
      // counters live in the elected thread, the same one every time
      if (q.tiles > 0 && elect_one()) {
        if (!multiply(c, (g.blk_hi - g.blk_lo + 1) / 2, q, rit, slot, phase, ait)) ok = 0;
      }
      ok = __all_sync(0xffffffffu, ok);
    } else {
      ok = accumulate(c, g, q, ait) ? 1 : 0;
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
  if (warp == 1) {
    tc_fence_after();
    tmem_dealloc(c.tmem, kTmemCols);
  }
}

}  // namespace

cudaError_t launch_weigh(const WeighParams& p, const CUtensorMap& qmap, const CUtensorMap& kmap, int num_sms,
                         cudaStream_t stream) {
  static std::atomic<bool> attr_set[64];
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= 64) return cudaErrorInvalidDevice;
  if (!attr_set[dev].load(std::memory_order_acquire)) {
    cudaError_t e = cudaFuncSetAttribute(weigh_sm100_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, int(kSmem));
    if (e != cudaSuccess) return e;
    attr_set[dev].store(true, std::memory_order_release);
  }
  weigh_sm100_kernel<<<num_sms, kThreads, kSmem, stream>>>(qmap, kmap, p);
  return cudaGetLastError();
}

cudaError_t weigh_take_error(uint32_t* bits, cudaStream_t stream) {
  uint32_t* dev = nullptr;
  cudaError_t e = cudaGetSymbolAddress(reinterpret_cast<void**>(&dev), g_weigh_err);
  if (e != cudaSuccess) return e;
  if ((e = cudaMemcpyAsync(bits, dev, sizeof(uint32_t), cudaMemcpyDeviceToHost, stream)) != cudaSuccess) return e;
  if ((e = cudaMemsetAsync(dev, 0, sizeof(uint32_t), stream)) != cudaSuccess) return e;
  return cudaStreamSynchronize(stream);
}

}  // namespace mla
