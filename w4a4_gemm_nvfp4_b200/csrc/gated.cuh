// gated.cuh -- what the gated feed-forward kernels share: the activation and
// its derivative, and the 8-bit checkpoint format of the two products.
#pragma once

#include <cuda_runtime.h>
#include <stdint.h>

#include "common.cuh"

namespace nvfp4 {

// Both activations are act(g) = g * sigma(z(g)), sigma(z) = 1 / (1 + exp(-z)):
//   SiLU  z = g
//   GELU  z = 2c (g + 0.044715 g^3), c = sqrt(2 / pi): the tanh form, since
//         (1 + tanh(a)) / 2 = sigma(2a)
// and act'(g) = sigma + g sigma (1 - sigma) z'(g).
//
// sigma takes the hardware's exponential and reciprocal: relative to sigma the
// exponential is off by 2^-22 and |z| 2^-22 (the roundings of -z log2(e)), the
// reciprocal by 2^-23.  Where |z| is large and z negative that is |z| 2^-22 of a
// vanishing sigma, elsewhere below 2^-20 together.  The reciprocal flushes a
// subnormal result, so sigma below 2^-126 (z below -87.34) counts as 0: act(g) is
// then 0 and off by less than |g| 2^-126, act'(g) by less than (1 + |g| z') 2^-126.
constexpr float kGelu2C = 1.5957691216057308f;  // 2c
constexpr float kGeluCubic = 0.044715f;
constexpr float kLog2e = 1.4426950408889634f;
constexpr float kGeluT1 = -kGelu2C * kLog2e, kGeluT3 = kGeluT1 * kGeluCubic;

__device__ __forceinline__ float ex2_approx(float x) {
  float r;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(x));
  return r;
}
__device__ __forceinline__ float rcp_approx(float x) {
  float r;
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(x));
  return r;
}

// sigma(z(g))
__device__ __forceinline__ float gate_sigma(float g, int act) {
  const float t = act == NVFP4_ACT_SILU ? g * -kLog2e : g * fmaf(g * g, kGeluT3, kGeluT1);  // -z log2(e)
  return rcp_approx(1.0f + ex2_approx(t));
}

// act(g) * u; g sigma first, which a product g u past the range does not spoil.
__device__ __forceinline__ float act_mul(float g, float u, int act) { return g * gate_sigma(g, act) * u; }

// Columns of a row that share one scale in a checkpoint, and the smallest
// scale: 2^-100 keeps 1/s finite and makes an all-zero block no special case.
constexpr int kCkptBlock = 32;
constexpr float kCkptTiny = 7.888609052210118e-31f;  // 2^-100

// The scale of a block whose largest |v| is amax: amax / 127 rounded up to
// bf16, so that |v| / s never exceeds 127; NaN when a value was not finite.
__device__ __forceinline__ float ckpt_scale(float amax) {
  const float t = __fdiv_rn(amax, 127.0f);
  if (!(t < __int_as_float(0x7f800000))) return __int_as_float(0x7fffffff);
  return __uint_as_float((__float_as_uint(fmaxf(t, kCkptTiny)) + 0xFFFFu) & 0xFFFF0000u);
}

// Adding 1.5 * 2^23 to a number below 2^22 rounds it to the nearest whole one,
// ties to even, and leaves that in the low byte; in an FMA the number is an exact
// product.
constexpr float kCkptRound = 12582912.0f;

}  // namespace nvfp4
