// saw_norm.cuh -- the root and the reciprocal of an RMS norm, correctly rounded.
#pragma once

#include <math.h>

namespace saw {

// An approximation, its exact remainder by a fused step, and one correction each (P.
// Markstein, "Computation of elementary functions on the IBM RISC System/6000
// processor", 1990).  The built-in ones' results for every binary32 from 2^-100 on
// (tests/test_gpu_norm_factor.py); those, with their checks for the rest of binary32,
// cost 22 us of 592 at 131072 tokens.
__device__ __forceinline__ float norm_root(float t) {
  float y;
  asm("rsqrt.approx.f32 %0, %1;" : "=f"(y) : "f"(t));
  const float root = __fmul_rn(t, y);
  return __fmaf_rn(__fmaf_rn(-root, root, t), __fmul_rn(0.5f, y), root);
}

// 1 / root of t >= 2^-100.
__device__ __forceinline__ float norm_factor(float t) {
  const float root = norm_root(t);
  float y;
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(root));
  y = __fmaf_rn(y, __fmaf_rn(-root, y, 1.0f), y);
  return t == INFINITY ? 0.0f : y;                   // (squares beyond binary32)
}

}  // namespace saw
