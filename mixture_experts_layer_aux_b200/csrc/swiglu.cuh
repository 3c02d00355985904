// swiglu.cuh -- the gate of the feed-forward block, silu(z) u, and its
// derivative, in fp32 with one reciprocal instruction (1 ulp) in place of a
// division: the epilogues of short products spend most of their time here.
// z -> -inf: exp(-z) overflows to infinity, its reciprocal is 0, silu is -0.
#pragma once

#include "common.cuh"

namespace swiglu {

MOE_DEV float sigmoid(float z) {
  float r;
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(1.0f + __expf(-z)));
  return r;
}
MOE_DEV float act(float z, float u) { return z * sigmoid(z) * u; }

// v = d(silu(z) u) -> dz, du.
MOE_DEV void grad(float v, float z, float u, float& dz, float& du) {
  const float s = sigmoid(z);
  dz = v * u * s * (1.f + z * (1.f - s));
  du = v * z * s;
}

}  // namespace swiglu
