// pow2_scale.cuh — the calibrated FP8 block scale: a power of two that just covers a
// row (append.cu, tree_commit.cu).
#pragma once

namespace pkv {

// The smallest power of two p with amax <= 448 p (1 for amax = 0).
__device__ __forceinline__ float pow2_scale(float amax) {
  if (!(amax > 0.f)) return 1.f;
  int e;
  const float m = frexpf(amax, &e);  // amax = m * 2^e, 0.5 <= m < 1
  return ldexpf(1.f, m <= 0.875f ? e - 9 : e - 8);  // amax <= 448 * 2^k = 0.875 * 2^(9 + k)
}

}  // namespace pkv
