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
constexpr float kInvSqrt2Pi = 0.3989422804014327f;

// The approximate 2^x and reciprocal, one special-function instruction each,
// have a relative error of ~2^-22 (an FP16 output's rounding is 2^-11); at
// ±∞ they give the limits 0, ∞ and 0.

// Φ(u), the normal distribution function, with a relative error below 2^-18 for
// |u| ≤ 6 (u·Φ(u) is 0 in FP16 below that): Φ(−|u|) = e^(−u²/2)·P(t), t = 1/(1 +
// 0.3475·|u|), and Φ(|u|) is the rest of 1. P, of degree 7, is within 2^-21.7 of
// e^(u²/2)·Φ(−|u|) relative to it for |u| ≤ 13.5, where the exponential has
// become 0 (least maximum of the relative error, fitted in 64 bits). ½ + ½·erf
// loses the digits of a negative u's small Φ, and erfc keeps them at twice the
// price (8192×8192 read back and activated: 138 us with erfc, 91 with erf, 65
// this way; the training product that keeps its pre-activations 263, 203, 171).
__device__ __forceinline__ f32x2 normal_cdf(f32x2 u, f32x2& e) {
  float a, b, ta, tb;
  unpair(u, a, b);
  unpair(fma2(pair_of(fabsf(a), fabsf(b)), pair_of(0.3475f), pair_of(1.f)), ta, tb);
  const f32x2 t = pair_of(rcp_approx(ta), rcp_approx(tb));
  unpair(mul2(mul2(u, u), pair_of(-0.5f * kLog2e)), ta, tb);
  e = pair_of(ex2_approx(ta), ex2_approx(tb));
  f32x2 p = fma2(t, pair_of(0.0486292429f), pair_of(-0.204973117f));
  p = fma2(p, t, pair_of(0.252273709f));
  p = fma2(p, t, pair_of(-0.0260401648f));
  p = fma2(p, t, pair_of(0.159388065f));
  p = fma2(p, t, pair_of(0.131353244f));
  p = fma2(p, t, pair_of(0.139403224f));
  p = mul2(fma2(p, t, pair_of(-3.4190627e-05f)), e);
  float qa, qb;
  unpair(p, qa, qb);
  return pair_of(a < 0.f ? qa : 1.f - qa, b < 0.f ? qb : 1.f - qb);
}

// A pair of f(u), and of f'(u) when GRAD, f the activation ACT. The tanh form
// of GELU is u·σ(2z), z = √(2/π)·(u + 0.044715·u³), with derivative
// σ + u·σ·(1 − σ)·2z'. Where σ has become 0 or 1 its factor u·σ·(1 − σ) is 0,
// and no power of u overflows below |u| = 2^62: products of FP16 values stay
// far below.
template <int ACT, bool GRAD>
__device__ __forceinline__ void activate(f32x2 u, f32x2& f, f32x2& df) {
  if constexpr (ACT == HGEMM_ACT_RELU) {
    float a, b;
    unpair(u, a, b);
    float fa, fb;  // max(u, 0); a NaN stays one, in f and in f'
    asm("max.NaN.f32 %0, %1, 0f00000000;" : "=f"(fa) : "f"(a));
    asm("max.NaN.f32 %0, %1, 0f00000000;" : "=f"(fb) : "f"(b));
    f = pair_of(fa, fb);
    if (GRAD) df = pair_of(a > 0.f ? 1.f : fa, b > 0.f ? 1.f : fb);
  } else if constexpr (ACT == HGEMM_ACT_GELU || ACT == HGEMM_ACT_SILU) {
    // σ(x) = 1 / (1 + 2^(-x·log2 e))
    f32x2 x, u2 = 0;
    if constexpr (ACT == HGEMM_ACT_GELU) {
      u2 = mul2(u, u);
      x = mul2(u, fma2(u2, pair_of(-2.f * kLog2e * kGeluZ * kGeluC), pair_of(-2.f * kLog2e * kGeluZ)));
    } else {
      x = mul2(u, pair_of(-kLog2e));
    }
    float a, b;
    unpair(x, a, b);
    unpair(add2(pair_of(ex2_approx(a), ex2_approx(b)), pair_of(1.f)), a, b);
    const f32x2 s = pair_of(rcp_approx(a), rcp_approx(b));
    f = mul2(u, s);
    if constexpr (GRAD) {
      const f32x2 w = fma2(f, mul2(s, pair_of(-1.f)), f);  // u·σ·(1 − σ)
      if constexpr (ACT == HGEMM_ACT_GELU)
        df = fma2(w, fma2(u2, pair_of(6.f * kGeluZ * kGeluC), pair_of(2.f * kGeluZ)), s);
      else
        df = add2(w, s);
    }
  } else if constexpr (ACT == HGEMM_ACT_GELU_ERF) {
    f32x2 e;  // e^(−u²/2)
    const f32x2 phi = normal_cdf(u, e);
    f = mul2(u, phi);
    if constexpr (GRAD) df = fma2(mul2(u, pair_of(kInvSqrt2Pi)), e, phi);
  } else {
    f = u;
    if (GRAD) df = pair_of(1.f);
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

// One value at a time.
template <bool GRAD>
__device__ __forceinline__ void activate(float u, int act, float& f, float& df) {
  with_activation(act, [&](auto a) {
    f32x2 f2, df2 = 0;
    activate<decltype(a)::value, GRAD>(pair_of(u), f2, df2);
    float other;
    unpair(f2, f, other);
    if (GRAD) unpair(df2, df, other);
  });
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
__device__ __forceinline__ uint32_t ckpt_word(f32x2 u01, f32x2 u23, float inv) {
  // (scalar products: a packed product and sum are contracted into one
  // rounding, which the form's definition does not have)
  float c[4];
  unpair(u01, c[0], c[1]);
  unpair(u23, c[2], c[3]);
  const f32x2 magic = pair_of(12582912.f);
  unpair(add2(pair_of(__fmul_rn(c[0], inv), __fmul_rn(c[1], inv)), magic), c[0], c[1]);
  unpair(add2(pair_of(__fmul_rn(c[2], inv), __fmul_rn(c[3], inv)), magic), c[2], c[3]);
  const uint32_t w = __byte_perm(__byte_perm(__float_as_uint(c[0]), __float_as_uint(c[1]), 0x0040u),
                                 __byte_perm(__float_as_uint(c[2]), __float_as_uint(c[3]), 0x0040u), 0x5410u);
  return inv == 0.f ? 0u : w;
}

// The FP32 values of the signed bytes 2·i and 2·i + 1 of a word: a byte,
// offset by 128 (`flipped`: the word with every top bit inverted), placed in
// the mantissa of 2^23.
__device__ __forceinline__ f32x2 ckpt_pair(uint32_t flipped, int i) {
  const uint32_t a = __byte_perm(flipped, 0x4B000000u, 0x7440u + static_cast<uint32_t>(2 * i));
  const uint32_t b = __byte_perm(flipped, 0x4B000000u, 0x7441u + static_cast<uint32_t>(2 * i));
  return add2(pair_of(__uint_as_float(a), __uint_as_float(b)), pair_of(-8388736.f));  // 2^23 + 128
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

__device__ __forceinline__ uint32_t pack_half2(f32x2 v) {
  float a, b;
  unpair(v, a, b);
  return pack_half2(__float_as_uint(a), __float_as_uint(b));
}
__device__ __forceinline__ f32x2 unpack_half2(uint32_t h) {
  const float2 f = __half22float2(*reinterpret_cast<const __half2*>(&h));
  return pair_of(f.x, f.y);
}
// Eight FP32 values, rounded and packed.
__device__ __forceinline__ uint4 pack8(const f32x2* v) {
  return make_uint4(pack_half2(v[0]), pack_half2(v[1]), pack_half2(v[2]), pack_half2(v[3]));
}
// v[0..3] += eight FP16 values.
__device__ __forceinline__ void add8(f32x2* v, uint4 h) {
  v[0] = add2(v[0], unpack_half2(h.x));
  v[1] = add2(v[1], unpack_half2(h.y));
  v[2] = add2(v[2], unpack_half2(h.z));
  v[3] = add2(v[3], unpack_half2(h.w));
}

// The 64 accumulators of a TMEM row as pairs.
__device__ __forceinline__ void tmem_row64(uint32_t taddr, f32x2 (&v)[32]) {
  uint32_t a[32], b[32];
  tmem_ld_32x32b_x32(taddr, a);
  tmem_ld_32x32b_x32(taddr + 32, b);
  tmem_ld_wait(a);
  tmem_ld_wait(b);
#pragma unroll
  for (int i = 0; i < 16; ++i) {
    v[i] = pair_of(__uint_as_float(a[2 * i]), __uint_as_float(a[2 * i + 1]));
    v[16 + i] = pair_of(__uint_as_float(b[2 * i]), __uint_as_float(b[2 * i + 1]));
  }
}

// A lane computes a row of 64 columns, but a warp whose lanes each access a
// row of their own touches 32 lines per instruction. So residual, codes and
// f(û) are read and written four or eight rows at a time, neighbouring lanes
// taking neighbouring 16 bytes, and pass through the warp's staging box on the
// way to or from the row's lane. (8192×8192 outputs of a contraction of
// 2048, GELU's gradient with f(û): 185 us with a row per lane, 173 this way,
// 150 without codes and f(û).)
//
// The 16-byte chunk j of row r of a box of 128-byte rows and of one of 64-byte
// rows, permuted so that neither way of access meets bank conflicts.
__device__ __forceinline__ uint4* box_chunk128(uint8_t* box, int r, int j) {
  return reinterpret_cast<uint4*>(box + r * 128 + ((j ^ (r & 7)) << 4));
}
__device__ __forceinline__ uint4* box_chunk64(uint8_t* box, int r, int j) {
  return reinterpret_cast<uint4*>(box + r * 64 + ((j ^ ((r >> 1) & 3)) << 4));
}

// What the epilogue of 32 rows' 64 columns reads besides the accumulator:
// fetched ahead of it, so that the reads wait while the product does.
template <int EPI>
struct LinSide {
  uint4 bias[EPI == kEpiLinear ? 8 : 1];
  uint4 side[EPI == kEpiLinear ? 8 : 4];  // residual: rows 4·j + lane/8; codes: rows 8·j + lane/4
  float scale;                            // of row `lane`
};

// Codes are accessed 16 bytes at a time where the matrix allows that.
__device__ __forceinline__ bool codes16(const LinEpi& e, int64_t N, int64_t x0) {
  return x0 + 64 <= N && (reinterpret_cast<uintptr_t>(e.codes) & 15u) == 0 && e.ldq % 16 == 0;
}

// grow: row `lane` of the box.
template <int EPI>
__device__ __forceinline__ void lin_fetch(LinSide<EPI>& s, const LinEpi& e, int lane, int64_t M, int64_t N,
                                          int64_t grow, int64_t x0) {
  const int64_t row0 = grow - lane;
  if constexpr (EPI == kEpiLinear) {
    if (e.bias) {
#pragma unroll
      for (int j = 0; j < 8; ++j) s.bias[j] = load_bias8(e.bias, x0 + 8 * j, N);
    }
    if (e.res) {
      const int64_t m = row0 + (lane >> 3), n = x0 + 8 * (lane & 7);
      const uint16_t* r = e.res + m * e.ldr + n;
#pragma unroll
      for (int j = 0; j < 8; ++j)
        s.side[j] = m + 4 * j < M && n < N && dbg_row(r + 4 * j * e.ldr, n, 8, N, 16)
                        ? *reinterpret_cast<const uint4*>(r + 4 * j * e.ldr)
                        : make_uint4(0u, 0u, 0u, 0u);
    }
  } else if (e.codes) {
    const int64_t m = row0 + (lane >> 2), n = x0 + 16 * (lane & 3);
    const int8_t* q = e.codes + m * e.ldq + n;
    const bool wide = codes16(e, N, x0);
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      s.side[j] = make_uint4(0u, 0u, 0u, 0u);
      const int8_t* at = q + 8 * j * e.ldq;
      if (m + 8 * j < M) {
        if (wide) {
          if (dbg_row(at, n, 16, N, 16)) s.side[j] = *reinterpret_cast<const uint4*>(at);
        } else {
          uint2 a = make_uint2(0u, 0u), b = a;
          if (n < N && dbg_row(at, n, 8, N, 8)) a = reinterpret_cast<const uint2*>(at)[0];
          if (n + 8 < N && dbg_row(at, n + 8, 8, N, 8)) b = reinterpret_cast<const uint2*>(at)[1];
          s.side[j] = make_uint4(a.x, a.y, b.x, b.y);
        }
      }
    }
    s.scale = grow < M && x0 < N && HG_DBG_INDEX(grow, e.lds) ? e.scales[x0 / kCkptGroup * e.lds + grow] : 0.f;
  }
}

// Row `lane` of a staging box of 32 rows of 64 columns x0 .. x0+63 (one 8-bit
// group), row `grow` of the output: its 64 accumulators v through the epilogue
// into the box, 128-byte swizzled as stage_row64 does. The whole warp calls;
// the box is free. N, the pitches and x0 are multiples of 8, so eight columns
// are inside the matrix or none.
template <int EPI>
__device__ __forceinline__ void lin_row64(uint8_t* box, int lane, f32x2 (&v)[32], const LinSide<EPI>& s,
                                          const LinEpi& e, int64_t M, int64_t N, int64_t grow, int64_t x0) {
  const int64_t row0 = grow - lane;
  if constexpr (EPI == kEpiLinear) {
    if (e.bias) {
#pragma unroll
      for (int j = 0; j < 8; ++j) add8(v + 4 * j, s.bias[j]);
    }
    if (e.codes) {
      // (columns past N hold 0: zero-filled operands and no bias)
      float top = 0.f;
#pragma unroll
      for (int i = 0; i < 32; ++i) {
        float a, b;
        unpair(v[i], a, b);
        top = max_abs3(top, a, b);
      }
      float scale, inv;
      ckpt_scale(magnitude_bits(top), scale, inv);
      if (grow < M && HG_DBG_INDEX(x0, N) && HG_DBG_INDEX(grow, e.lds))
        e.scales[x0 / kCkptGroup * e.lds + grow] = scale;
#pragma unroll
      for (int j = 0; j < 4; ++j)
        *box_chunk64(box, lane, j) =
            make_uint4(ckpt_word(v[8 * j], v[8 * j + 1], inv), ckpt_word(v[8 * j + 2], v[8 * j + 3], inv),
                       ckpt_word(v[8 * j + 4], v[8 * j + 5], inv), ckpt_word(v[8 * j + 6], v[8 * j + 7], inv));
      __syncwarp();
      const int64_t m = row0 + (lane >> 2), n = x0 + 16 * (lane & 3);
      int8_t* q = e.codes + m * e.ldq + n;
      const bool wide = codes16(e, N, x0);
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const uint4 w = *box_chunk64(box, 8 * j + (lane >> 2), lane & 3);
        int8_t* at = q + 8 * j * e.ldq;
        if (m + 8 * j < M) {
          if (wide) {
            if (dbg_row(at, n, 16, N, 16)) *reinterpret_cast<uint4*>(at) = w;
          } else {
            if (n < N && dbg_row(at, n, 8, N, 8)) reinterpret_cast<uint2*>(at)[0] = make_uint2(w.x, w.y);
            if (n + 8 < N && dbg_row(at, n + 8, 8, N, 8)) reinterpret_cast<uint2*>(at)[1] = make_uint2(w.z, w.w);
          }
        }
      }
      __syncwarp();
    }
    if (e.res) {
#pragma unroll
      for (int j = 0; j < 8; ++j) *box_chunk128(box, 4 * j + (lane >> 3), lane & 7) = s.side[j];
    }
    with_activation(e.act, [&](auto a) {
#pragma unroll
      for (int i = 0; i < 32; ++i) {
        f32x2 f, df;
        activate<decltype(a)::value, false>(v[i], f, df);
        v[i] = f;
      }
    });
    if (e.res) {
      __syncwarp();
#pragma unroll
      for (int j = 0; j < 8; ++j) add8(v + 4 * j, *box_chunk128(box, lane, j));
      // (a lane overwrites below what it alone has read)
    }
  } else if (e.codes) {
#pragma unroll
    for (int j = 0; j < 4; ++j) *box_chunk64(box, 8 * j + (lane >> 2), lane & 3) = s.side[j];
    __syncwarp();
    uint4 codes[4];
#pragma unroll
    for (int j = 0; j < 4; ++j) codes[j] = *box_chunk64(box, lane, j);
    __syncwarp();
    with_activation(e.act, [&](auto a) {
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        const uint32_t w[2] = {j & 1 ? codes[j / 2].z : codes[j / 2].x, j & 1 ? codes[j / 2].w : codes[j / 2].y};
        f32x2 f[4], df;
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const f32x2 u = mul2(ckpt_pair(w[i / 2] ^ 0x80808080u, i & 1), pair_of(s.scale));
          activate<decltype(a)::value, true>(u, f[i], df);
          v[4 * j + i] = mul2(v[4 * j + i], df);
        }
        if (e.h) *box_chunk128(box, lane, j) = pack8(f);
      }
    });
    if (e.h) {
      __syncwarp();
      const int64_t m = row0 + (lane >> 3), n = x0 + 8 * (lane & 7);
      uint16_t* h = e.h + m * e.ldh + n;
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        const uint4 w = *box_chunk128(box, 4 * j + (lane >> 3), lane & 7);
        if (m + 4 * j < M && n < N && dbg_row(h + 4 * j * e.ldh, n, 8, N, 16))
          *reinterpret_cast<uint4*>(h + 4 * j * e.ldh) = w;
      }
      __syncwarp();
    }
  }
#pragma unroll
  for (int j = 0; j < 8; ++j) *box_chunk128(box, lane, j) = pack8(v + 4 * j);
}

}  // namespace hg
