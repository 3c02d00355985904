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

// Saved pre-activations: the first 24 bits of an fp32 value (16 of significand), as a bf16 plane and a byte plane.
// Kept as bf16 they were the largest error of the gradients (0.0030 of dX and the weight gradients in 2-norm, where
// the bf16 rounding of an output alone is 0.0017; with 24 bits 0.0023); the third byte costs 1 % of a training step.
// Cut, not rounded: a NaN stays a NaN.
MOE_DEV uint32_t hi2(float a, float b) {  // bf16 plane of two values
  return __byte_perm(__float_as_uint(a), __float_as_uint(b), 0x7632);
}
MOE_DEV uint32_t lo4(float a, float b, float c, float d) {  // byte plane of four
  const uint32_t x = __byte_perm(__float_as_uint(a), __float_as_uint(b), 0x0051);
  const uint32_t y = __byte_perm(__float_as_uint(c), __float_as_uint(d), 0x0051);
  return __byte_perm(x, y, 0x5410);
}
MOE_DEV void join4(uint32_t h01, uint32_t h23, uint32_t lo, float (&v)[4]) {
  v[0] = __uint_as_float(__byte_perm(h01, lo, 0x1044) & 0xffffff00u);
  v[1] = __uint_as_float(__byte_perm(h01, lo, 0x3255) & 0xffffff00u);
  v[2] = __uint_as_float(__byte_perm(h23, lo, 0x1066) & 0xffffff00u);
  v[3] = __uint_as_float(__byte_perm(h23, lo, 0x3277) & 0xffffff00u);
}

}  // namespace swiglu
