// The rotation shared by mla_rope and the rotating cache writer.
#pragma once

#include <cuda_bf16.h>
#include <math.h>
#include <stdint.h>

namespace mla {

// Layout flags (MLA_ROPE_* of include/mla.h).
constexpr unsigned kRopeHalf = 0x1u;
constexpr unsigned kRopeInverse = 0x2u;
constexpr int kMaxRot = 256;

// (cos, sin) of pos * freq times mscale.  The angle is taken in turns and
// reduced in double.  Its three roundings are off by at most 2.5 * 2^-53 of the
// turns: below 2^-30 turns up to position 2^24 and so lost in the rounding of the
// fp32 argument (2^-26 turns), at most 2^-23 turns (7e-7 rad) at position 2^31,
// where a bf16 result keeps 2^-9.
__device__ __forceinline__ float2 rope_factors(int pos, double freq, float mscale, bool inverse) {
  const double turns = static_cast<double>(pos) * (freq * 0.15915494309189533576888);  // 1 / (2 pi)
  const float r = static_cast<float>(turns - rint(turns));                               // [-1/2, 1/2]
  float s, c;
  sincospif(2.f * r, &s, &c);
  return make_float2(c * mscale, (inverse ? -s : s) * mscale);
}

__device__ __forceinline__ void rope_pair(float& a, float& b, float2 cs) {
  const float u = a * cs.x - b * cs.y;
  b = a * cs.y + b * cs.x;
  a = u;
}

}  // namespace mla
