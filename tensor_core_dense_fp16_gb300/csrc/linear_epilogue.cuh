// linear_epilogue.cuh — the arithmetic of the feed-forward block's operators
// on FP32 values: activations with their derivatives, and the 8-bit form.
#pragma once

#include <cuda_fp16.h>

#include "hgemm.h"
#include "internal.h"

namespace hg {

__device__ __forceinline__ float ex2_approx(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}
__device__ __forceinline__ float rcp_approx(float x) {
  float y;
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}

constexpr float kLog2e = 1.4426950408889634f;
constexpr float kGeluZ = 0.7978845608028654f;    // √(2/π)
constexpr float kGeluC = 0.044715f;
constexpr float kInvSqrt2 = 0.7071067811865476f;
constexpr float kInvSqrt2Pi = 0.3989422804014327f;

// σ(x) = 1 / (1 + e^-x), from the approximate 2^x and reciprocal (two
// special-function instructions, relative error ~2^-22: an FP16 output's
// rounding is 2^-11). x = ±∞ gives 1 and 0.
__device__ __forceinline__ float sigmoid_f(float x) { return rcp_approx(1.f + ex2_approx(-kLog2e * x)); }

// f(u), and f'(u) when GRAD. The tanh form of GELU is u·σ(2z),
// z = √(2/π)·(u + 0.044715·u³), with derivative
// σ + u·σ·(1 − σ)·2z'. Beyond |u| = 16 σ is 0 or 1 in FP32, so z is taken
// at u clamped to ±16, where no power of u overflows.
template <bool GRAD>
__device__ __forceinline__ void activate(float u, int act, float& f, float& df) {
  switch (act) {
    case HGEMM_ACT_RELU:
      f = u < 0.f ? 0.f : u;
      if (GRAD) df = u > 0.f ? 1.f : (u <= 0.f ? 0.f : u);  // NaN stays NaN
      return;
    case HGEMM_ACT_GELU: {
      const float c = fminf(fmaxf(u, -16.f), 16.f);
      const float c2 = c * c;
      const float s = sigmoid_f(2.f * kGeluZ * c * fmaf(kGeluC, c2, 1.f));
      f = u * s;
      // (a NaN u leaves f NaN; the clamp drops it from s)
      if (GRAD) df = fmaf(f * (1.f - s), 2.f * kGeluZ * fmaf(3.f * kGeluC, c2, 1.f), s);
      return;
    }
    case HGEMM_ACT_SILU: {
      const float s = sigmoid_f(u);
      f = u * s;
      if (GRAD) df = fmaf(f, 1.f - s, s);
      return;
    }
    case HGEMM_ACT_GELU_ERF: {
      const float phi = fmaf(0.5f, erff(u * kInvSqrt2), 0.5f);  // Φ(u)
      f = u * phi;
      if (GRAD) df = fmaf(u * kInvSqrt2Pi, ex2_approx(-0.5f * kLog2e * u * u), phi);
      return;
    }
    default:
      f = u;
      if (GRAD) df = 1.f;
  }
}

__device__ __forceinline__ float activate(float u, int act) {
  float f, df;
  activate<false>(u, act, f, df);
  return f;
}

// ------------------------------------------------------------ 8-bit form

constexpr int kCkptGroup = HGEMM_CKPT8_GROUP;

// max|u| as ordered bits: an infinity or a NaN compares above every finite
// magnitude, so one integer maximum finds both the top and the exceptions.
__device__ __forceinline__ uint32_t magnitude_bits(float u) { return __float_as_uint(u) & 0x7FFFFFFFu; }

// A group's scale and the factor its values are multiplied by, from the
// largest magnitude_bits.
__device__ __forceinline__ void ckpt_scale(uint32_t top_bits, float& scale, float& inv) {
  const float top = __uint_as_float(top_bits);
  if (top_bits >= 0x7F800000u) {  // an infinity or a NaN: codes 0, scale NaN
    scale = __uint_as_float(0x7FFFFFFFu);
    inv = 0.f;
  } else if (top < 7.888609e-31f) {  // 2^-100
    scale = 0.f;
    inv = 0.f;
  } else {
    scale = __fdiv_rn(top, 127.f);
    inv = __fdiv_rn(127.f, top);
  }
}

// rint(u·inv) as the low byte: adding 1.5·2^23 leaves the rounded whole
// number in the mantissa's low bits (|u·inv| < 128). inv = 0 gives 0 also for
// an infinity or a NaN.
__device__ __forceinline__ uint32_t ckpt_code(float u, float inv) {
  const float t = __fadd_rn(__fmul_rn(u, inv), 12582912.f);
  return inv == 0.f ? 0u : __float_as_uint(t) & 0xFFu;
}

// The FP32 value of the signed byte at position `i` of `word`: the byte,
// offset by 128, placed in the mantissa of 2^23.
__device__ __forceinline__ float ckpt_byte(uint32_t word, int i) {
  const uint32_t biased = __byte_perm(word ^ 0x80808080u, 0x4B000000u, 0x7440u + static_cast<uint32_t>(i));
  return __uint_as_float(biased) - 8388736.f;  // 2^23 + 128
}

}  // namespace hg
