// linear_epilogue.cuh — the arithmetic of the feed-forward block's operators
// on FP32 values: activations with their derivatives, and the 8-bit form.
#pragma once

#include <type_traits>

#include <cuda_fp16.h>

#include "hgemm.h"
#include "internal.h"
#include "kernel_common.cuh"

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

// f(u), and f'(u) when GRAD, f the activation ACT. The tanh form of GELU is u·σ(2z),
// z = √(2/π)·(u + 0.044715·u³), with derivative
// σ + u·σ·(1 − σ)·2z'. Beyond |u| = 16 σ is 0 or 1 in FP32, so z is taken
// at u clamped to ±16, where no power of u overflows.
template <int ACT, bool GRAD>
__device__ __forceinline__ void activate(float u, float& f, float& df) {
  if constexpr (ACT == HGEMM_ACT_RELU) {
    f = u < 0.f ? 0.f : u;
    if (GRAD) df = u > 0.f ? 1.f : (u <= 0.f ? 0.f : u);  // NaN stays NaN
  } else if constexpr (ACT == HGEMM_ACT_GELU) {
    const float c = fminf(fmaxf(u, -16.f), 16.f);  // (a NaN is dropped from s, not from f)
    const float c2 = c * c;
    const float s = sigmoid_f(2.f * kGeluZ * c * fmaf(kGeluC, c2, 1.f));
    f = u * s;
    if (GRAD) df = fmaf(f * (1.f - s), 2.f * kGeluZ * fmaf(3.f * kGeluC, c2, 1.f), s);
  } else if constexpr (ACT == HGEMM_ACT_SILU) {
    const float s = sigmoid_f(u);
    f = u * s;
    if (GRAD) df = fmaf(f, 1.f - s, s);
  } else if constexpr (ACT == HGEMM_ACT_GELU_ERF) {
    const float phi = fmaf(0.5f, erff(u * kInvSqrt2), 0.5f);  // Φ(u)
    f = u * phi;
    if (GRAD) df = fmaf(u * kInvSqrt2Pi, ex2_approx(-0.5f * kLog2e * u * u), phi);
  } else {
    f = u;
    if (GRAD) df = 1.f;
  }
}

// Calls body with the activation as a compile-time constant, so that a loop
// inside it branches once and not for each value.
template <typename Body>
__device__ __forceinline__ void with_activation(int act, Body body) {
  switch (act) {
    case HGEMM_ACT_RELU:
      body(std::integral_constant<int, HGEMM_ACT_RELU>{});
      return;
    case HGEMM_ACT_GELU:
      body(std::integral_constant<int, HGEMM_ACT_GELU>{});
      return;
    case HGEMM_ACT_SILU:
      body(std::integral_constant<int, HGEMM_ACT_SILU>{});
      return;
    case HGEMM_ACT_GELU_ERF:
      body(std::integral_constant<int, HGEMM_ACT_GELU_ERF>{});
      return;
    default:
      body(std::integral_constant<int, HGEMM_ACT_NONE>{});
  }
}

template <bool GRAD>
__device__ __forceinline__ void activate(float u, int act, float& f, float& df) {
  with_activation(act, [&](auto a) { activate<decltype(a)::value, GRAD>(u, f, df); });
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
// number in the mantissa's low bits (|u·inv| < 128). The caller takes 0 in
// place of all codes of a group whose inv is 0.
__device__ __forceinline__ uint32_t ckpt_code(float u, float inv) {
  return __float_as_uint(__fadd_rn(__fmul_rn(u, inv), 12582912.f));
}

// Four codes packed (the first in the low byte); all 0 where inv is 0.
__device__ __forceinline__ uint32_t ckpt_word(float a, float b, float c, float d, float inv) {
  const uint32_t w = __byte_perm(__byte_perm(ckpt_code(a, inv), ckpt_code(b, inv), 0x0040u),
                                 __byte_perm(ckpt_code(c, inv), ckpt_code(d, inv), 0x0040u), 0x5410u);
  return inv == 0.f ? 0u : w;
}

// The FP32 value of the signed byte at position `i` of `word`: the byte,
// offset by 128, placed in the mantissa of 2^23.
__device__ __forceinline__ float ckpt_byte(uint32_t word, int i) {
  const uint32_t biased = __byte_perm(word ^ 0x80808080u, 0x4B000000u, 0x7440u + static_cast<uint32_t>(i));
  return __uint_as_float(biased) - 8388736.f;  // 2^23 + 128
}

// The largest of three magnitudes; a NaN wins.
__device__ __forceinline__ float max_abs3(float a, float b, float c) {
  float d;
  asm("max.NaN.abs.f32 %0, %1, %2, %3;" : "=f"(d) : "f"(a), "f"(b), "f"(c));
  return d;
}

// ------------------------------------------- epilogue of a tile of 64 columns

// One output, its row m and column n inside the matrix: the scalar form of
// the epilogue, for columns that cannot be read eight at a time. scale (and
// inv, forward) are those of the row's group.
template <bool BACKWARD>
__device__ __forceinline__ void lin_scalar(const LinEpi& e, float acc, int64_t m, int64_t n, float scale, float inv,
                                           uint16_t* out) {
  float y;
  if constexpr (BACKWARD) {
    y = acc;
    if (e.codes) {
      float f, df;
      activate<true>(static_cast<float>(e.codes[m * e.ldq + n]) * scale, e.act, f, df);
      y *= df;
      if (e.h) e.h[m * e.ldh + n] = __half_as_ushort(__float2half_rn(f));
    }
  } else {
    // acc already holds the bias
    if (e.codes) e.codes[m * e.ldq + n] = static_cast<int8_t>(inv == 0.f ? 0u : ckpt_code(acc, inv));
    y = activate(acc, e.act);
    if (e.res) y += __half2float(__ushort_as_half(e.res[m * e.ldr + n]));
  }
  *out = __half_as_ushort(__float2half_rn(y));
}

__device__ __forceinline__ void prefetch_l2(const void* p) { asm volatile("prefetch.global.L2 [%0];" ::"l"(p)); }

// Asks L2 for what the epilogue of row `grow`, columns [x0, x0 + ncols), will
// read, while the tile's MMAs still run.
template <int EPI>
__device__ __forceinline__ void lin_prefetch_row(const LinEpi& e, int64_t M, int64_t N, int64_t grow, int64_t x0,
                                                 int ncols) {
  if (grow >= M) return;
  if constexpr (EPI == kEpiLinear) {
    if (e.res)
      for (int c = 0; c < ncols; c += 32)
        if (x0 + c < N) prefetch_l2(e.res + grow * e.ldr + x0 + c);
  } else {
    if (e.codes)
      for (int c = 0; c < ncols; c += 64)
        if (x0 + c < N) {
          prefetch_l2(e.codes + grow * e.ldq + x0 + c);
          prefetch_l2(e.scales + (x0 + c) / kCkptGroup * e.lds + grow);
        }
  }
}

// Eight FP32 values (bits), rounded and packed, into chunk j of the
// 128-byte-swizzled staging row of `lane`.
__device__ __forceinline__ uint4 pack8(const uint32_t* v) {
  return make_uint4(pack_half2(v[0], v[1]), pack_half2(v[2], v[3]), pack_half2(v[4], v[5]), pack_half2(v[6], v[7]));
}

// Row `lane` of a staged 32×64 box, columns x0 .. x0+63 (one 8-bit group):
// the 64 accumulators of row `grow` (v0: the first 32) through the epilogue
// into the staging row, as stage_row64 does. N, the pitches and x0 are
// multiples of 8, so eight columns are inside the matrix or none.
template <int EPI>
__device__ __forceinline__ void lin_stage_row64(uint8_t* row, int lane, uint32_t (&v0)[32], uint32_t (&v1)[32],
                                                const LinEpi& e, int64_t M, int64_t N, int64_t grow, int64_t x0) {
  const bool in_m = grow < M;
  auto half_of = [&](int j) -> uint32_t* { return j < 4 ? v0 + 8 * j : v1 + 8 * (j - 4); };
  if constexpr (EPI == kEpiLinear) {
    if (e.bias) {
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        const uint4 b8 = load_bias8(e.bias, x0 + 8 * j, N);
        const __half* b = reinterpret_cast<const __half*>(&b8);
        uint32_t* v = half_of(j);
#pragma unroll
        for (int i = 0; i < 8; ++i) v[i] = __float_as_uint(__uint_as_float(v[i]) + __half2float(b[i]));
      }
    }
    if (e.codes) {
      // columns past N hold 0: zero-filled operands and no bias
      float t0 = 0.f, t1 = 0.f;
#pragma unroll
      for (int i = 0; i < 32; i += 2) {
        t0 = max_abs3(t0, __uint_as_float(v0[i]), __uint_as_float(v0[i + 1]));
        t1 = max_abs3(t1, __uint_as_float(v1[i]), __uint_as_float(v1[i + 1]));
      }
      float scale, inv;
      ckpt_scale(magnitude_bits(max_abs3(t0, t1, 0.f)), scale, inv);
      uint32_t w[16];
#pragma unroll
      for (int j = 0; j < 16; ++j) {
        const uint32_t* v = j < 8 ? v0 + 4 * j : v1 + 4 * (j - 8);
        w[j] = ckpt_word(__uint_as_float(v[0]), __uint_as_float(v[1]), __uint_as_float(v[2]), __uint_as_float(v[3]),
                         inv);
      }
      if (in_m) {
        int8_t* q = e.codes + grow * e.ldq + x0;
        if (x0 + 64 <= N && (reinterpret_cast<uintptr_t>(q) & 15u) == 0) {
#pragma unroll
          for (int j = 0; j < 4; ++j)
            reinterpret_cast<uint4*>(q)[j] = make_uint4(w[4 * j], w[4 * j + 1], w[4 * j + 2], w[4 * j + 3]);
        } else {
#pragma unroll
          for (int j = 0; j < 8; ++j)
            if (x0 + 8 * j < N) reinterpret_cast<uint2*>(q)[j] = make_uint2(w[2 * j], w[2 * j + 1]);
        }
        e.scales[x0 / kCkptGroup * e.lds + grow] = scale;
      }
    }
    with_activation(e.act, [&](auto a) {
      if constexpr (decltype(a)::value != HGEMM_ACT_NONE) {
#pragma unroll
        for (int i = 0; i < 32; ++i) {
          float f, df;
          activate<decltype(a)::value, false>(__uint_as_float(v0[i]), f, df);
          v0[i] = __float_as_uint(f);
          activate<decltype(a)::value, false>(__uint_as_float(v1[i]), f, df);
          v1[i] = __float_as_uint(f);
        }
      }
    });
    if (e.res && in_m) {
      const uint16_t* r = e.res + grow * e.ldr + x0;
      uint4 r8[8];
#pragma unroll
      for (int j = 0; j < 8; ++j)
        r8[j] = x0 + 8 * j < N ? *reinterpret_cast<const uint4*>(r + 8 * j) : make_uint4(0u, 0u, 0u, 0u);
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        const __half* h = reinterpret_cast<const __half*>(&r8[j]);
        uint32_t* v = half_of(j);
#pragma unroll
        for (int i = 0; i < 8; ++i) v[i] = __float_as_uint(__uint_as_float(v[i]) + __half2float(h[i]));
      }
    }
  } else if (e.codes) {
    uint32_t w[16];
    float scale = 0.f;
#pragma unroll
    for (int j = 0; j < 16; ++j) w[j] = 0u;
    if (in_m) {
      const int8_t* q = e.codes + grow * e.ldq + x0;
      if (x0 + 64 <= N && (reinterpret_cast<uintptr_t>(q) & 15u) == 0) {
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          const uint4 t = reinterpret_cast<const uint4*>(q)[j];
          w[4 * j] = t.x, w[4 * j + 1] = t.y, w[4 * j + 2] = t.z, w[4 * j + 3] = t.w;
        }
      } else {
#pragma unroll
        for (int j = 0; j < 8; ++j)
          if (x0 + 8 * j < N) {
            const uint2 t = reinterpret_cast<const uint2*>(q)[j];
            w[2 * j] = t.x, w[2 * j + 1] = t.y;
          }
      }
      scale = e.scales[x0 / kCkptGroup * e.lds + grow];
    }
    uint32_t hid[32];
    with_activation(e.act, [&](auto a) {
#pragma unroll
      for (int i = 0; i < 64; i += 2) {
        float f[2], df;
#pragma unroll
        for (int k = 0; k < 2; ++k) {
          uint32_t& v = i < 32 ? v0[i + k] : v1[i - 32 + k];
          activate<decltype(a)::value, true>(ckpt_byte(w[i / 4], (i + k) & 3) * scale, f[k], df);
          v = __float_as_uint(__uint_as_float(v) * df);
        }
        hid[i / 2] = pack_half2(__float_as_uint(f[0]), __float_as_uint(f[1]));
      }
    });
    if (e.h && in_m) {
      uint16_t* h = e.h + grow * e.ldh + x0;
#pragma unroll
      for (int j = 0; j < 8; ++j)
        if (x0 + 8 * j < N)
          reinterpret_cast<uint4*>(h)[j] = make_uint4(hid[4 * j], hid[4 * j + 1], hid[4 * j + 2], hid[4 * j + 3]);
    }
  }
#pragma unroll
  for (int j = 0; j < 8; ++j) *reinterpret_cast<uint4*>(row + ((j ^ (lane & 7)) << 4)) = pack8(half_of(j));
}

}  // namespace hg
