// Chunk attention on CUDA cores: the plain loops over
// the definition, fp32 throughout.
#include <math.h>

#include "common.cuh"
#include "kernels.h"

namespace mla {

namespace {

constexpr int kThreads = 256;
constexpr int kRows = 16;  // query rows of one token per CTA (H is a multiple of 16)
constexpr int kTile = 32;  // cached tokens staged at a time

struct Where {
  int b, n, j, len;  // sequence, its tokens, this token among them, clamped length
};

// The sequence of token t: binary search of the last offset <= t.
__device__ bool find_token(const int32_t* offs, const int32_t* seq_lens, int T, int B, int max_blocks, int t,
                           uint32_t* err, Where* w) {
  int lo = 0, hi = B;
  while (hi - lo > 1) {
    const int mid = (lo + hi) / 2;
    if (offs[mid] <= t) lo = mid; else hi = mid;
  }
  const int a = offs[lo], e = offs[lo + 1];
  if (t < a || t >= e) return false;
  if (a < 0 || e > T) return false;
  w->b = lo;
  w->n = e - a;
  w->j = t - a;
  w->len = checked_len(seq_lens, lo, max_blocks, err);
  return true;
}

// Stage cached rows [t0, t0 + kTile) below `len`; bad blocks and rows past len read as zeros, valid[] = 0.
__device__ void stage(const __nv_bfloat16* cache, const int32_t* table, int num_blocks, int t0, int len,
                      __nv_bfloat16 (*k)[kRow + 8], int* valid, uint32_t* err) {
  for (int u = threadIdx.x; u < kTile * (kRow / 8); u += kThreads) {
    const int r = u / (kRow / 8), c = u % (kRow / 8);
    uint4 v = make_uint4(0, 0, 0, 0);
    bool ok = false;
    if (t0 + r < len) {
      const int blk = table[(t0 + r) / kBlock];
      ok = blk >= 0 && blk < num_blocks;
      if (ok)
        v = *reinterpret_cast<const uint4*>(cache + (size_t(blk) * kBlock + (t0 + r) % kBlock) * kRow + c * 8);
      else if (c == 0)
        atomicOr(err, kErrBadBlock);
    }
    *reinterpret_cast<uint4*>(&k[r][c * 8]) = v;
    if (c == 0) valid[r] = ok ? 1 : 0;
  }
}

// grid (T, H / 16)
__global__ void __launch_bounds__(kThreads) chunk_simple_kernel(const ChunkParams p) {
  extern __shared__ __align__(16) uint8_t raw[];
  auto* k = reinterpret_cast<__nv_bfloat16(*)[kRow + 8]>(raw);
  auto* q = reinterpret_cast<__nv_bfloat16(*)[kRow + 8]>(raw + kTile * (kRow + 8) * 2);
  __shared__ int valid[kTile];
  __shared__ float pr[kRows][kTile], alpha[kRows], mx[kRows], sum[kRows];
  const int t = blockIdx.x, h0 = blockIdx.y * kRows;
  if (t == 0 && blockIdx.y == 0)
    for (int b = threadIdx.x; b < p.B; b += kThreads)
      if (p.q_offsets[b] < 0 || p.q_offsets[b + 1] < p.q_offsets[b] || p.q_offsets[b + 1] > p.T)
        atomicOr(p.err, kErrSeqTooLong);
  Where w;
  if (!find_token(p.q_offsets, p.seq_lens, p.T, p.B, p.max_blocks, t, p.err, &w)) return;
  const int sees = max(0, w.len - (w.n - 1 - w.j));
  const __nv_bfloat16* qs = p.q + (size_t(t) * p.H + h0) * kRow;
  for (int u = threadIdx.x; u < kRows * (kRow / 8); u += kThreads)
    *reinterpret_cast<uint4*>(&q[u / (kRow / 8)][u % (kRow / 8) * 8]) = reinterpret_cast<const uint4*>(qs)[u];
  if (threadIdx.x < kRows) {
    mx[threadIdx.x] = -INFINITY;
    sum[threadIdx.x] = 0.f;
  }
  float o[kRows][2] = {};
  for (int t0 = 0; t0 < sees; t0 += kTile) {
    __syncthreads();
    stage(p.cache, p.block_table + size_t(w.b) * p.max_blocks, p.num_blocks, t0, sees, k, valid, p.err);
    __syncthreads();
    for (int i = threadIdx.x; i < kRows * kTile; i += kThreads) {
      const int r = i / kTile, c = i % kTile;
      float s = 0.f;
      for (int d = 0; d < kRow; ++d) s += __bfloat162float(q[r][d]) * __bfloat162float(k[c][d]);
      pr[r][c] = valid[c] ? s * p.softmax_scale : -INFINITY;
    }
    __syncthreads();
    if (threadIdx.x < kRows) {
      const int r = threadIdx.x;
      float m = mx[r];
      for (int c = 0; c < kTile; ++c) m = fmaxf(m, pr[r][c]);
      const float a = m == -INFINITY ? 1.f : expf(mx[r] - m);
      float z = sum[r] * a;
      for (int c = 0; c < kTile; ++c) {
        const float e = m == -INFINITY ? 0.f : expf(pr[r][c] - m);
        pr[r][c] = e;
        z += e;
      }
      alpha[r] = a;
      mx[r] = m;
      sum[r] = z;
    }
    __syncthreads();
    for (int r = 0; r < kRows; ++r)
      for (int e = 0; e < 2; ++e) {
        float acc = o[r][e] * alpha[r];
        for (int c = 0; c < kTile; ++c) acc += pr[r][c] * __bfloat162float(k[c][2 * threadIdx.x + e]);
        o[r][e] = acc;
      }
  }
  __syncthreads();
  for (int r = 0; r < kRows; ++r) {
    const float inv = sum[r] > 0.f ? 1.f / sum[r] : 0.f;
    const size_t row = size_t(t) * p.H + h0 + r;
    reinterpret_cast<__nv_bfloat162*>(p.out + row * kDc)[threadIdx.x] =
        __floats2bfloat162_rn(o[r][0] * inv, o[r][1] * inv);
    if (threadIdx.x == 0) p.lse[row] = sum[r] > 0.f ? mx[r] + logf(sum[r]) : -INFINITY;
  }
}

}  // namespace

cudaError_t launch_chunk_simple(const ChunkParams& p, cudaStream_t stream) {
  const int smem = (kTile + kRows) * (kRow + 8) * 2;
  if (cudaError_t e = cudaFuncSetAttribute(chunk_simple_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
      e != cudaSuccess)
    return e;
  chunk_simple_kernel<<<dim3(p.T, p.H / kRows), kThreads, smem, stream>>>(p);
  return cudaGetLastError();
}

}  // namespace mla
