// Rotary positions of queries (or keys): y[t,h] = R(pos[t]) x[t,h] on the rot
// rotated elements of every head.
//
// Bound: HBM, 4 bytes per rotated element (read and written once).  The
// angles of a token are shared by its heads, so a CTA takes one token: its
// first rot/2 threads form the cosines and sines once (double reduction, the
// expensive part) and leave them in shared memory, while every thread has its
// elements' loads already in flight.
//
// rope_vec_kernel: 16-byte vectors v (elements 8v..8v+7 of a row).  A thread
//   takes vectors v and v + rot/16: in the half layout these hold the two
//   members of eight pairs, in the interleaved layout four whole pairs each,
//   so both layouts read and write the same addresses.
// rope_scalar_kernel: rows that are not 16-byte aligned or whose rot is not a
//   multiple of 16; one pair per thread and step.
#include "kernels.h"
#include "rope.cuh"

namespace mla {
namespace {

// 128 threads with eight 16-byte loads each in flight: 45.4 us for 8192 tokens
// x 128 heads (0.91 of the measured copy bandwidth); with four loads 46.7, with
// 256 threads 50.8, 512 threads 69.
constexpr int kRopeThreads = 128;
constexpr int kRopeUnits = 4;

__device__ __forceinline__ void unpack8(const uint4& v, float (&f)[8]) {
  const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    f[2 * i] = __uint_as_float(w[i] << 16);
    f[2 * i + 1] = __uint_as_float(w[i] & 0xffff0000u);
  }
}

__device__ __forceinline__ uint4 pack8(const float (&f)[8]) {
  uint32_t w[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const __nv_bfloat162 b = __floats2bfloat162_rn(f[2 * i], f[2 * i + 1]);
    w[i] = *reinterpret_cast<const uint32_t*>(&b);
  }
  return make_uint4(w[0], w[1], w[2], w[3]);
}

// grid (T, head groups of `group`); units of one row: rot / 16.
__global__ void __launch_bounds__(kRopeThreads)
rope_vec_kernel(const RopeParams p, int group) {
  __shared__ float2 cs[kMaxRot / 2];
  const int t = blockIdx.x;
  const int h0 = blockIdx.y * group;
  const int units = p.rot / 16;
  const int n = min(group, p.H - h0) * units;
  const __nv_bfloat16* x = p.x + t * p.x_ldt + h0 * p.x_ldh;
  __nv_bfloat16* y = p.y + t * p.y_ldt + h0 * p.y_ldh;
  const bool half = (p.flags & kRopeHalf) != 0;
  for (int u0 = threadIdx.x; u0 - static_cast<int>(threadIdx.x) < n; u0 += kRopeUnits * kRopeThreads) {
    uint4 a[kRopeUnits], b[kRopeUnits];
#pragma unroll
    for (int k = 0; k < kRopeUnits; ++k) {
      const int u = u0 + k * kRopeThreads;
      if (u < n) {
        const uint4* row = reinterpret_cast<const uint4*>(x + (u / units) * p.x_ldh);
        a[k] = row[u % units];
        b[k] = row[u % units + units];
      }
    }
    if (u0 == static_cast<int>(threadIdx.x)) {
      if (threadIdx.x < p.rot / 2)
        cs[threadIdx.x] = rope_factors(p.pos[t], p.freqs[threadIdx.x], p.mscale, (p.flags & kRopeInverse) != 0);
      __syncthreads();
    }
#pragma unroll
    for (int k = 0; k < kRopeUnits; ++k) {
      const int u = u0 + k * kRopeThreads;
      if (u >= n) continue;
      const int v = u % units;
      float fa[8], fb[8];
      unpack8(a[k], fa);
      unpack8(b[k], fb);
      if (half) {
#pragma unroll
        for (int e = 0; e < 8; ++e) rope_pair(fa[e], fb[e], cs[8 * v + e]);
      } else {
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          rope_pair(fa[2 * e], fa[2 * e + 1], cs[4 * v + e]);
          rope_pair(fb[2 * e], fb[2 * e + 1], cs[4 * (v + units) + e]);
        }
      }
      uint4* row = reinterpret_cast<uint4*>(y + (u / units) * p.y_ldh);
      row[v] = pack8(fa);
      row[v + units] = pack8(fb);
    }
  }
}

__global__ void __launch_bounds__(kRopeThreads)
rope_scalar_kernel(const RopeParams p, int group) {
  __shared__ float2 cs[kMaxRot / 2];
  const int t = blockIdx.x;
  const int h0 = blockIdx.y * group;
  const int pairs = p.rot / 2;
  if (threadIdx.x < pairs)
    cs[threadIdx.x] = rope_factors(p.pos[t], p.freqs[threadIdx.x], p.mscale, (p.flags & kRopeInverse) != 0);
  __syncthreads();
  const bool half = (p.flags & kRopeHalf) != 0;
  const int n = min(group, p.H - h0) * pairs;
  for (int u = threadIdx.x; u < n; u += kRopeThreads) {
    const int h = h0 + u / pairs, i = u % pairs;
    const int ia = half ? i : 2 * i, ib = half ? i + pairs : 2 * i + 1;
    const __nv_bfloat16* x = p.x + t * p.x_ldt + h * p.x_ldh;
    __nv_bfloat16* y = p.y + t * p.y_ldt + h * p.y_ldh;
    float a = __bfloat162float(x[ia]), b = __bfloat162float(x[ib]);
    rope_pair(a, b, cs[i]);
    y[ia] = __float2bfloat16_rn(a);
    y[ib] = __float2bfloat16_rn(b);
  }
}

}  // namespace

cudaError_t launch_rope(const RopeParams& p, int num_sms, cudaStream_t stream) {
  static_assert(kMaxRot / 2 <= kRopeThreads, "one thread per pair forms the factors");
  // whole tokens per CTA once there are enough tokens to fill the device
  // several times; few tokens are split into groups of heads
  int group = p.H;
  const int sms = num_sms > 0 ? num_sms : 148;
  while (group > 16 && static_cast<long long>(p.T) * ((p.H + group - 1) / group) < 8LL * sms) group = (group + 1) / 2;
  const dim3 grid(p.T, (p.H + group - 1) / group);
  const uintptr_t bits = reinterpret_cast<uintptr_t>(p.x) | reinterpret_cast<uintptr_t>(p.y) |
                         static_cast<uintptr_t>((p.x_ldt | p.x_ldh | p.y_ldt | p.y_ldh) * 2);
  if ((bits & 15u) == 0 && p.rot % 16 == 0)
    rope_vec_kernel<<<grid, kRopeThreads, 0, stream>>>(p, group);
  else
    rope_scalar_kernel<<<grid, kRopeThreads, 0, stream>>>(p, group);
  return cudaGetLastError();
}

}  // namespace mla
