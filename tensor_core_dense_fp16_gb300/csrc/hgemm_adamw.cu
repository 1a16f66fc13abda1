// hgemm_adamw.cu — an AdamW step over many tensors in one launch, and 8-bit
// states read back (hgemm_adamw, hgemm_adamw_load; the formulas and the 8-bit
// forms are in hgemm.h). Bound by memory: with FP32 states, a master copy, an
// FP16 gradient and weight 28 bytes per value, with 8-bit states and no master
// 10.25. Measured: 33.6 M values with FP32 states and master 139 us (6.8 TB/s, a
// copy's rate); 100.8 M with 8-bit states 183 us (5.6 TB/s, issue slots 71%),
// rounded at random 192, read back 153 us (6.7 TB/s).
#include <cuda_fp16.h>

#include "debug.cuh"
#include "internal.h"
#include "linear_epilogue.cuh"
#include "ptx.cuh"
#include "row_sums.cuh"

namespace hg {
namespace {

constexpr int kThreads = 256;
constexpr int kChunk = 2048;  // values that a block moves at once: 8 per thread, whole groups
static_assert(kChunk == kThreads * 8 && kChunk % kCkptGroup == 0, "a group lies in one warp's values");

// The tensors travel as the launch's parameters: nothing has to be copied
// before it, and a captured graph holds them.
template <int MAX>
struct AdamwTable {
  AdamwStep step;
  int count;
  int per;          // chunks of a block's step
  uint32_t chunks;  // steps
  AdamwEntry t[MAX];
};

__device__ __forceinline__ float sqrt_approx(float x) {
  float y;
  asm("sqrt.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}

// ------------------------------------------------------ the 8-bit form of v

constexpr uint32_t kOneBits = 0x3F800000u;

// A group's scale and the factor its values are multiplied by, from the
// largest magnitude_bits.
__device__ __forceinline__ void second_scale(uint32_t top_bits, float& scale, float& inv) {
  const float top = __uint_as_float(top_bits);
  scale = inv = 0.f;
  if (top_bits >= 0x7F800000u) {
    scale = __uint_as_float(0x7FFFFFFFu);
  } else if (top >= 7.888609e-31f) {  // 2^-100
    scale = top;
    inv = __fdiv_rn(1.f, top);
  }
}

// The upper 12 bits of an FP32 number r in (0, 1] (8 of exponent, 3 of fraction
// and the leading 0) rounded at the 20th, counted from 1's; at least 1 where r
// is not 0. `add` goes to the 20 bits that are cut off: half of them rounds to
// nearest, a random number below 2^20 up with the probability of the rest (r is
// linear in its bits between two codes). r = v·(1/top) is at most 1 + 2^-23,
// whose code is 255. The caller takes 0 in place of all codes of a group whose
// inv is 0.
template <bool RANDOM>
__device__ __forceinline__ uint32_t second_code(float v_over_top, uint32_t add) {
  const uint32_t r = __float_as_uint(v_over_top);
  int c = static_cast<int>(r + add + ((255u << 20) - kOneBits)) >> 20;
  if (RANDOM) c = min(c, 255);
  return static_cast<uint32_t>(max(c, static_cast<int>(min(r, 1u))));
}
constexpr uint32_t kHalfCode = 0x80000u;

// What a code stands for, in units of the group's largest.
__device__ __forceinline__ float second_unit(uint32_t code) {
  return code ? __uint_as_float((code << 20) + (kOneBits - (255u << 20))) : 0.f;
}

__device__ __forceinline__ float second_value(uint32_t code, float scale) { return __fmul_rn(second_unit(code), scale); }

// ----------------------------------------------------------- random rounding

// 32 bits from 32, a bijection: shifts and products with odd numbers (the first
// bits of √2's and √3's fractions), after which a bit that changes changes each
// other with probability 0.497 to 0.503.
__device__ __forceinline__ uint32_t mixed(uint32_t x) {
  x = (x ^ (x >> 16)) * 0x6A09E667u;
  x = (x ^ (x >> 15)) * 0xBB67AE85u;
  return x ^ (x >> 16);
}

// The random bits of value i of a tensor in the step whose number gave `key`:
// one mixed number for eight values, times a power of an odd number (the golden
// section's bits) each. The upper 20 round v, the lower 12 m: over steps and
// over values both are even, and neighbours' are independent of one another
// within 1%.
constexpr uint32_t kGolden = 0x9E3779B1u;
__device__ __forceinline__ uint32_t eight_bits(uint32_t key, int64_t i) {
  return mixed(static_cast<uint32_t>(i >> 3) + key);
}

// A number in (1, 2) from the lower 12 bits, in the middle of its 4096th part.
__device__ __forceinline__ float one_and(uint32_t bits) {
  return __uint_as_float(0x3F800400u | ((bits & 0xFFFu) << 11));
}

// floor(m·inv + u) as the low byte, from 1 + u: adding 1.5·2^23 − 1 and rounding
// down leaves the whole number in the low bits. |m·inv| is at most 127 + 2^-15
// and u lies 2^-13 from 0 and 1, so that no code passes 127.
constexpr float kFloorMagic = 12582911.f;
__device__ __forceinline__ uint32_t random_code(float m, float inv, float one_and_u) {
  return __float_as_uint(__fadd_rd(__fmaf_rn(m, inv, one_and_u), kFloorMagic));
}

// ------------------------------------------------------------------ the step

struct Scalars {
  float gscale, a, b, lr;
  bool dynamic;
  uint32_t key;  // of random rounding
};

// One value: the states (each product and sum rounded, so that the kept codes
// do not depend on how a compiler contracts them) and the parameter.
__device__ __forceinline__ void adamw_value(const AdamwStep& s, const Scalars& c, float keep, float g, float& m,
                                            float& v, float& p) {
  g = __fmul_rn(g, c.gscale);
  m = __fadd_rn(__fmul_rn(m, s.beta1), __fmul_rn(g, s.rest1));
  v = __fadd_rn(__fmul_rn(v, s.beta2), __fmul_rn(__fmul_rn(g, g), s.rest2));
  // (the approximate root and reciprocal are within 2^-22)
  p = fmaf(p, keep, -(m * c.a) * rcp_approx(fmaf(sqrt_approx(v), c.b, s.eps)));
}

// Eight values of a thread; VEC: neighbours, moved 16 bytes at a time; else
// every 32nd of a warp's 256. `first` is the first value, `n` the tensor's.
template <bool VEC>
__device__ __forceinline__ int64_t value_at(int64_t first, int i) {
  return VEC ? first + i : first + 32 * i;
}

template <bool VEC>
__device__ __forceinline__ void load_f32(const float* p, int64_t first, int64_t n, float (&f)[8]) {
  if constexpr (VEC) {
    const uint4 a = load16(p + first), b = load16(p + first + 4);
    f[0] = __uint_as_float(a.x), f[1] = __uint_as_float(a.y), f[2] = __uint_as_float(a.z), f[3] = __uint_as_float(a.w);
    f[4] = __uint_as_float(b.x), f[5] = __uint_as_float(b.y), f[6] = __uint_as_float(b.z), f[7] = __uint_as_float(b.w);
  } else {
#pragma unroll
    for (int i = 0; i < 8; ++i) f[i] = value_at<VEC>(first, i) < n ? p[value_at<VEC>(first, i)] : 0.f;
  }
}

template <bool VEC>
__device__ __forceinline__ void store_f32(float* p, int64_t first, int64_t n, const float (&f)[8]) {
  if constexpr (VEC) {
    *reinterpret_cast<float4*>(p + first) = make_float4(f[0], f[1], f[2], f[3]);
    *reinterpret_cast<float4*>(p + first + 4) = make_float4(f[4], f[5], f[6], f[7]);
  } else {
#pragma unroll
    for (int i = 0; i < 8; ++i)
      if (value_at<VEC>(first, i) < n) p[value_at<VEC>(first, i)] = f[i];
  }
}

template <bool VEC>
__device__ __forceinline__ void load_f16(const uint16_t* p, int64_t first, int64_t n, float (&f)[8]) {
  if constexpr (VEC) {
    unpack8(load16(p + first), f);
  } else {
#pragma unroll
    for (int i = 0; i < 8; ++i) f[i] = value_at<VEC>(first, i) < n ? half_at(p, value_at<VEC>(first, i)) : 0.f;
  }
}

template <bool VEC>
__device__ __forceinline__ void store_f16(uint16_t* p, int64_t first, int64_t n, const float (&f)[8]) {
  if constexpr (VEC) {
    *reinterpret_cast<uint4*>(p + first) = pack8f(f);
  } else {
#pragma unroll
    for (int i = 0; i < 8; ++i)
      if (value_at<VEC>(first, i) < n) p[value_at<VEC>(first, i)] = __half_as_ushort(__float2half_rn(f[i]));
  }
}

template <bool VEC>
__device__ __forceinline__ void load_codes(const uint8_t* p, int64_t first, int64_t n, uint32_t (&c)[8]) {
  if constexpr (VEC) {
    const uint2 w = load8(p + first);
#pragma unroll
    for (int i = 0; i < 8; ++i) c[i] = ((i < 4 ? w.x : w.y) >> (8 * (i & 3))) & 0xFFu;
  } else {
#pragma unroll
    for (int i = 0; i < 8; ++i) c[i] = value_at<VEC>(first, i) < n ? p[value_at<VEC>(first, i)] : 0u;
  }
}

template <bool VEC>
__device__ __forceinline__ void store_codes(uint8_t* p, int64_t first, int64_t n, const uint32_t (&c)[8]) {
  if constexpr (VEC) {
    uint32_t w[2] = {};
#pragma unroll
    for (int i = 0; i < 8; ++i) w[i >> 2] |= (c[i] & 0xFFu) << (8 * (i & 3));
    *reinterpret_cast<uint2*>(p + first) = make_uint2(w[0], w[1]);
  } else {
#pragma unroll
    for (int i = 0; i < 8; ++i)
      if (value_at<VEC>(first, i) < n) p[value_at<VEC>(first, i)] = static_cast<uint8_t>(c[i]);
  }
}

// The group of a thread's value i: VEC, eight threads share one; else a warp's
// values 2j and 2j + 1 are group j.
template <bool VEC>
__device__ __forceinline__ int64_t group_at(int64_t first, int i) {
  return value_at<VEC>(first, i) / kCkptGroup;
}

// The largest magnitude of the group of value i, i even.
template <bool VEC>
__device__ __forceinline__ uint32_t group_top(const float (&f)[8], int i) {
  if constexpr (VEC) {
    uint32_t top = 0;
#pragma unroll
    for (int k = 0; k < 8; ++k) top = max(top, magnitude_bits(f[k]));
#pragma unroll
    for (int o = 4; o > 0; o >>= 1) top = max(top, __shfl_xor_sync(0xffffffffu, top, o));
    return top;
  } else {
    return __reduce_max_sync(0xffffffffu, max(magnitude_bits(f[i]), magnitude_bits(f[i + 1])));
  }
}

// Eight values of a tensor. All lanes of a warp come here together.
template <bool VEC, bool RANDOM>
__device__ __forceinline__ void adamw_eight(const AdamwEntry& t, const AdamwStep& s, const Scalars& c, float keep,
                                            int64_t first) {
  const int64_t n = t.n;
  const bool in = first < n;  // VEC: all eight, the chunks hold whole eights
  const bool eight = !VEC && t.ms != nullptr;  // (VEC: adamw_bytes)
  float g[8] = {}, m[8] = {}, v[8] = {}, p[8] = {};
  if (in && HG_DBG_INDEX(VEC ? first + 7 : first, n)) {
    if (t.grad_type == 0)
      load_f16<VEC>(static_cast<const uint16_t*>(t.grad), first, n, g);
    else
      load_f32<VEC>(static_cast<const float*>(t.grad), first, n, g);
    if (t.master)
      load_f32<VEC>(t.master, first, n, p);
    else
      load_f16<VEC>(t.weight, first, n, p);
    if (eight) {
      uint32_t q[8];
      load_codes<VEC>(static_cast<const uint8_t*>(t.m), first, n, q);
#pragma unroll
      for (int i = 0; i < 8; ++i)
        if (value_at<VEC>(first, i) < n)
          m[i] = __fmul_rn(static_cast<float>(static_cast<int8_t>(q[i])), t.ms[group_at<VEC>(first, i)]);
      load_codes<VEC>(static_cast<const uint8_t*>(t.v), first, n, q);
#pragma unroll
      for (int i = 0; i < 8; ++i)
        if (value_at<VEC>(first, i) < n) v[i] = second_value(q[i], t.vs[group_at<VEC>(first, i)]);
    } else {
      load_f32<VEC>(static_cast<const float*>(t.m), first, n, m);
      load_f32<VEC>(static_cast<const float*>(t.v), first, n, v);
    }
#pragma unroll
    for (int i = 0; i < 8; ++i)
      if (VEC || value_at<VEC>(first, i) < n) adamw_value(s, c, keep, g[i], m[i], v[i], p[i]);
  }
  if (eight) {
    __syncwarp();  // the group's scales have been read
    uint32_t qm[8], qv[8];
    uint32_t power = 1u;  // (a thread's values have the same place in their eights)
    if (RANDOM)
      for (int i = static_cast<int>(first & 7); i > 0; --i) power *= kGolden;
#pragma unroll
    for (int i = 0; i < 8; i += 2) {
      float scale_m, inv_m, scale_v, inv_v;
      ckpt_scale(group_top<VEC>(m, i), scale_m, inv_m);
      second_scale(group_top<VEC>(v, i), scale_v, inv_v);
#pragma unroll
      for (int j = i; j < (VEC ? 8 : i + 2); ++j) {
        const uint32_t bits = RANDOM ? eight_bits(c.key, value_at<VEC>(first, j)) * power : 0u;
        qm[j] = inv_m == 0.f ? 0u : RANDOM ? random_code(m[j], inv_m, one_and(bits)) : ckpt_code(m[j], inv_m);
        qv[j] = inv_v == 0.f ? 0u : second_code<RANDOM>(__fmul_rn(v[j], inv_v), RANDOM ? bits >> 12 : kHalfCode);
      }
      const int lane = threadIdx.x & 31;
      const int64_t at = VEC ? first : first - lane + 32 * i;  // a value of the group
      if (at < n && (VEC ? (lane & 7) == 0 : lane == 0)) {
        t.ms[at / kCkptGroup] = scale_m;
        t.vs[at / kCkptGroup] = scale_v;
      }
      if (VEC) break;
    }
    if (in) {
      store_codes<VEC>(static_cast<uint8_t*>(t.m), first, n, qm);
      store_codes<VEC>(static_cast<uint8_t*>(t.v), first, n, qv);
    }
  } else if (in) {
    store_f32<VEC>(static_cast<float*>(t.m), first, n, m);
    store_f32<VEC>(static_cast<float*>(t.v), first, n, v);
  }
  if (in) {
    if (t.master) store_f32<VEC>(t.master, first, n, p);
    if (t.weight) store_f16<VEC>(t.weight, first, n, p);
  }
}

// The same for 8-bit states moved eight at a time, the path of large tensors:
// `count` chunks from `first` on, the next one's loads under way while one is
// computed. The form's conversions cost as many instructions as its bytes
// save: the three quotients of a group are one division, each in a lane of its
// own.
template <bool G32, bool MASTER>
struct Packed {
  uint2 m, v;
  float sm, sv;
  uint4 g[G32 ? 2 : 1], p[MASTER ? 2 : 1];
};

template <bool WIDE>
__device__ __forceinline__ void unpack_wide(const uint4 (&w)[WIDE ? 2 : 1], f32x2 (&f)[4]) {
  if constexpr (WIDE) {
    f[0] = pair_of(__uint_as_float(w[0].x), __uint_as_float(w[0].y));
    f[1] = pair_of(__uint_as_float(w[0].z), __uint_as_float(w[0].w));
    f[2] = pair_of(__uint_as_float(w[1].x), __uint_as_float(w[1].y));
    f[3] = pair_of(__uint_as_float(w[1].z), __uint_as_float(w[1].w));
  } else {
    unpack8(w[0], f);
  }
}

template <bool RANDOM, bool G32, bool MASTER>
__device__ __forceinline__ void adamw_bytes(const AdamwEntry& t, const AdamwStep& s, const Scalars& c, float keep,
                                            int64_t first, int count) {
  const int64_t n = t.n;  // a multiple of 8, or past all these chunks
  uint8_t *tm = static_cast<uint8_t*>(t.m), *tv = static_cast<uint8_t*>(t.v);
  auto load = [&](int64_t i) {
    const int64_t at = i < n ? i : 0;  // (past the end: anything, not stored)
    Packed<G32, MASTER> r{};
    if (!HG_DBG_INDEX(at + 7, n)) return r;
    r.m = load8(tm + at);
    r.v = load8(tv + at);
    r.sm = t.ms[at / kCkptGroup];
    r.sv = t.vs[at / kCkptGroup];
    const uint8_t* g = static_cast<const uint8_t*>(t.grad) + at * (G32 ? 4 : 2);
    const uint8_t* p = MASTER ? reinterpret_cast<const uint8_t*>(t.master) + at * 4
                              : reinterpret_cast<const uint8_t*>(t.weight) + at * 2;
    r.g[0] = load16(g);
    if (G32) r.g[G32 ? 1 : 0] = load16(g + 16);
    r.p[0] = load16(p);
    if (MASTER) r.p[MASTER ? 1 : 0] = load16(p + 16);
    return r;
  };
  const int lane = threadIdx.x & 31, role = lane & 7;
  Packed<G32, MASTER> next = load(first);
  for (int i = 0; i < count; ++i, first += kChunk) {
    const Packed<G32, MASTER> r = next;
    if (i + 1 < count) next = load(first + kChunk);
    const bool in = first < n;  // all eight
    // Two values at a time. product2 is a product rounded by itself: a packed
    // product and sum would be contracted into one rounding.
    const f32x2 none = pair_of(s.minus_zero);
    auto product2 = [&](f32x2 x, f32x2 y) { return fma2(x, y, none); };
    f32x2 g[4], p[4], m[4], v[4];
    unpack_wide<G32>(r.g, g);
    unpack_wide<MASTER>(r.p, p);
    float top_m = 0.f, top_v = 0.f;
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      const uint32_t code = k < 2 ? r.v.x : r.v.y;
      m[k] = mul2(ckpt_pair((k < 2 ? r.m.x : r.m.y) ^ 0x80808080u, k & 1), pair_of(r.sm));
      v[k] = mul2(pair_of(second_unit(__byte_perm(code, 0u, 0x4440u + 2 * (k & 1))),
                          second_unit(__byte_perm(code, 0u, 0x4441u + 2 * (k & 1)))),
                  pair_of(r.sv));
      g[k] = mul2(g[k], pair_of(c.gscale));
      m[k] = add2(product2(m[k], pair_of(s.beta1)), product2(g[k], pair_of(s.rest1)));
      v[k] = add2(product2(v[k], pair_of(s.beta2)), product2(product2(g[k], g[k]), pair_of(s.rest2)));
      float a, b;
      unpair(v[k], a, b);
      top_v = max_abs3(top_v, a, b);
      unpair(fma2(pair_of(sqrt_approx(a), sqrt_approx(b)), pair_of(c.b), pair_of(s.eps)), a, b);
      p[k] = fma2(p[k], pair_of(keep), mul2(mul2(m[k], pair_of(-c.a)), pair_of(rcp_approx(a), rcp_approx(b))));
      unpair(m[k], a, b);
      top_m = max_abs3(top_m, a, b);
    }
    if (in) {
      if (MASTER) {
        *reinterpret_cast<ulonglong2*>(t.master + first) = make_ulonglong2(p[0], p[1]);
        *reinterpret_cast<ulonglong2*>(t.master + first + 4) = make_ulonglong2(p[2], p[3]);
      }
      if (!MASTER || t.weight) *reinterpret_cast<uint4*>(t.weight + first) = pack8(p);
    }
    // (a group lies whole in or past the tensor's last eight; what is past is not counted)
    uint32_t bits_m = in ? magnitude_bits(top_m) : 0u, bits_v = in ? magnitude_bits(top_v) : 0u;
#pragma unroll
    for (int o = 4; o > 0; o >>= 1) {
      bits_m = max(bits_m, __shfl_xor_sync(0xffffffffu, bits_m, o));
      bits_v = max(bits_v, __shfl_xor_sync(0xffffffffu, bits_v, o));
    }
    // lane 0 of a group's eight: max|m|/127, lane 1: 127/max|m|, lane 2: 1/max v
    top_m = __uint_as_float(bits_m);
    top_v = __uint_as_float(bits_v);
    const float q =
        __fdiv_rn(role == 0 ? top_m : role == 1 ? 127.f : 1.f, role == 0 ? 127.f : role == 1 ? top_m : top_v);
    const float inv_m = __shfl_sync(0xffffffffu, q, (lane & 24) | 1);
    const float inv_v = __shfl_sync(0xffffffffu, q, (lane & 24) | 2);
    // (no infinity or NaN, and not below 2^-100)
    const bool keep_m = bits_m < 0x7F800000u && top_m >= 7.888609e-31f;
    const bool keep_v = bits_v < 0x7F800000u && top_v >= 7.888609e-31f;
    uint32_t wm[2], wv[2];
    uint32_t bits = RANDOM ? eight_bits(c.key, first) : 0u;
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      uint32_t cm[4], cv[4];
#pragma unroll
      for (int k = 0; k < 2; ++k) {
        float a, b;
        const uint32_t other = bits * kGolden;
        if constexpr (RANDOM)  // (random_code)
          unpair(add2_down(fma2(m[2 * h + k], pair_of(inv_m), pair_of(one_and(bits), one_and(other))),
                           pair_of(kFloorMagic)),
                 a, b);
        else  // (ckpt_code)
          unpair(add2(product2(m[2 * h + k], pair_of(inv_m)), pair_of(12582912.f)), a, b);
        cm[2 * k] = __float_as_uint(a);
        cm[2 * k + 1] = __float_as_uint(b);
        unpair(product2(v[2 * h + k], pair_of(inv_v)), a, b);
        cv[2 * k] = second_code<RANDOM>(a, RANDOM ? bits >> 12 : kHalfCode);
        cv[2 * k + 1] = second_code<RANDOM>(b, RANDOM ? other >> 12 : kHalfCode);
        bits = other * kGolden;
      }
      wm[h] = __byte_perm(__byte_perm(cm[0], cm[1], 0x0040u), __byte_perm(cm[2], cm[3], 0x0040u), 0x5410u);
      wv[h] = __byte_perm(__byte_perm(cv[0], cv[1], 0x0040u), __byte_perm(cv[2], cv[3], 0x0040u), 0x5410u);
    }
    if (in) {
      *reinterpret_cast<uint2*>(tm + first) = keep_m ? make_uint2(wm[0], wm[1]) : make_uint2(0u, 0u);
      *reinterpret_cast<uint2*>(tv + first) = keep_v ? make_uint2(wv[0], wv[1]) : make_uint2(0u, 0u);
      if (role == 0) {
        const float nan = __uint_as_float(0x7FFFFFFFu);
        t.ms[first / kCkptGroup] = keep_m ? q : bits_m >= 0x7F800000u ? nan : 0.f;
        t.vs[first / kCkptGroup] = keep_v ? top_v : bits_v >= 0x7F800000u ? nan : 0.f;
      }
    }
  }
}

template <int MAX, bool RANDOM>
__global__ void __launch_bounds__(kThreads, 3) adamw_kernel(const __grid_constant__ AdamwTable<MAX> table) {
  grid_dependency_wait();
  grid_launch_dependents();
  const AdamwStep& s = table.step;
  Scalars c{s.gscale, s.a, s.b, s.lr, s.dynamic != nullptr, s.number};
  if (c.dynamic) {
    const hgemm_adamw_dynamic d = *s.dynamic;
    if (d.skip) return;
    const float step = static_cast<float>(max(d.step, 1));
    c.gscale = d.grad_scale;
    c.lr = d.lr;
    c.a = d.lr / -expm1f(step * s.ln1);
    c.b = rsqrtf(-expm1f(step * s.ln2));
    c.key = static_cast<uint32_t>(max(d.step, 1));
  }
  if (RANDOM) c.key = mixed(c.key);
  for (uint32_t chunk = blockIdx.x; chunk < table.chunks; chunk += gridDim.x) {
    int lo = 0, hi = table.count - 1;  // the last tensor that begins at or before the chunk
    while (lo < hi) {
      const int mid = (lo + hi + 1) >> 1;
      if (table.t[mid].chunk0 <= chunk)
        lo = mid;
      else
        hi = mid - 1;
    }
    const AdamwEntry& t = table.t[lo];
    int64_t first = static_cast<int64_t>(chunk - t.chunk0) * kChunk * table.per;
    const float keep = c.dynamic ? fmaf(-c.lr, t.decay, 1.f) : t.keep;
    // Chunks of whole eights where the pointers allow it; a tensor whose size is
    // no multiple of eight ends in a chunk moved value by value.
    const int64_t whole = !t.vec ? 0 : t.n % 8 == 0 ? t.n : t.n / kChunk * kChunk;
    int done = 0;
    if (first < whole) {
      const int64_t left = (whole - first + kChunk - 1) / kChunk;
      done = left < table.per ? static_cast<int>(left) : table.per;
      const int64_t at = first + 8 * static_cast<int>(threadIdx.x);
      if (!t.ms) {
        for (int i = 0; i < done; ++i) adamw_eight<true, RANDOM>(t, s, c, keep, at + i * kChunk);
      } else if (t.grad_type == 0) {
        t.master ? adamw_bytes<RANDOM, false, true>(t, s, c, keep, at, done)
                 : adamw_bytes<RANDOM, false, false>(t, s, c, keep, at, done);
      } else {
        t.master ? adamw_bytes<RANDOM, true, true>(t, s, c, keep, at, done)
                 : adamw_bytes<RANDOM, true, false>(t, s, c, keep, at, done);
      }
    }
    first += static_cast<int64_t>(done) * kChunk;
    for (int i = done; i < table.per && first < t.n; ++i, first += kChunk)
      adamw_eight<false, RANDOM>(t, s, c, keep, first + (threadIdx.x >> 5) * 256 + (threadIdx.x & 31));
  }
}

template <int MAX>
cudaError_t adamw_with(const AdamwEntry* t, int count, const AdamwStep& step, bool random, int num_sms,
                       cudaStream_t stream) {
  AdamwTable<MAX> table;
  table.step = step;
  table.count = count;
  auto steps_of = [](const AdamwEntry& x, int64_t values) { return static_cast<uint32_t>((x.n + values - 1) / values); };
  uint32_t chunks = 0;  // (384 tensors of 2^31 values are 2^29 of them)
  for (int i = 0; i < count; ++i) chunks += steps_of(t[i], kChunk);
  // A step of several chunks pays once for the search for the tensor and for
  // its addresses, and 8-bit states load the next chunk while one is computed;
  // too few steps leave blocks without one. 8-bit states, microseconds with 1, 2,
  // 4 and 8: 2.6 M values 8.9, 7.9, 8.2, 10.3; 5.2 M 15.9, 13.0, 12.6, 14.0;
  // 10.4 M 30, 23.2, 21.0, 21.8; 21 M 65, 50, 44, 42; 100 M 274, 213, 191, 182.
  // FP32 states and master: 2.6 M 11.1, 12.8, 13.5, 15.6; 10.4 M 47.9, 46.3, 46.5,
  // 52.4; 100 M 422, 413, 413, 419.
  bool eight = false;
  for (int i = 0; i < count; ++i) eight = eight || t[i].ms;
  const uint32_t each = chunks / static_cast<uint32_t>(num_sms);
  if (eight)
    table.per = each >= 64 ? 8 : each >= 16 ? 4 : each >= 3 ? 2 : 1;
  else
    table.per = each >= 16 ? 2 : 1;
  table.chunks = 0;
  for (int i = 0; i < count; ++i) {
    table.t[i] = t[i];
    table.t[i].chunk0 = table.chunks;
    table.chunks += steps_of(t[i], static_cast<int64_t>(kChunk) * table.per);
  }
  // More blocks than fit at once balance better than few waves of them (100 M
  // values with 8-bit states: 189 us with 16 an SM, 183 with 32 or 64).
  const uint32_t most = static_cast<uint32_t>(num_sms) * 64u;
  PdlLaunch l(dim3(table.chunks < most ? table.chunks : most), dim3(kThreads), 0, stream);
  return cudaLaunchKernelEx(&l.cfg, random && eight ? adamw_kernel<MAX, true> : adamw_kernel<MAX, false>, table);
}

// Four neighbouring values per thread and step where VEC, else one.
template <bool VEC>
__global__ void __launch_bounds__(kThreads)
    adamw_load_kernel(const int8_t* m, const float* ms, const uint8_t* v, const float* vs, float* m_out, float* v_out,
                      int64_t n) {
  constexpr int EACH = VEC ? 4 : 1, AHEAD = VEC ? 4 : 1;
  grid_dependency_wait();
  grid_launch_dependents();
  const int64_t step = static_cast<int64_t>(gridDim.x) * kThreads * EACH;
  const int64_t begin = (static_cast<int64_t>(blockIdx.x) * kThreads + threadIdx.x) * EACH;
  for (int64_t i0 = begin; i0 < n; i0 += AHEAD * step) {
    uint32_t cm[AHEAD], cv[AHEAD];
    float sm[AHEAD], sv[AHEAD];
#pragma unroll
    for (int j = 0; j < AHEAD; ++j) {
      const int64_t i = i0 + j * step;
      if (i >= n || !HG_DBG_INDEX(i + EACH - 1, n)) break;
      if (m) {
        cm[j] = VEC ? *reinterpret_cast<const uint32_t*>(m + i) : static_cast<uint8_t>(m[i]);
        sm[j] = ms[i / kCkptGroup];
      }
      if (v) {
        cv[j] = VEC ? *reinterpret_cast<const uint32_t*>(v + i) : v[i];
        sv[j] = vs[i / kCkptGroup];
      }
    }
#pragma unroll
    for (int j = 0; j < AHEAD; ++j) {
      const int64_t i = i0 + j * step;
      if (i >= n) break;
      float f[4];
      if (m) {
#pragma unroll
        for (int k = 0; k < EACH; ++k) f[k] = __fmul_rn(static_cast<float>(static_cast<int8_t>(cm[j] >> (8 * k))), sm[j]);
        if constexpr (VEC)
          *reinterpret_cast<float4*>(m_out + i) = make_float4(f[0], f[1], f[2], f[3]);
        else
          m_out[i] = f[0];
      }
      if (v) {
#pragma unroll
        for (int k = 0; k < EACH; ++k) f[k] = second_value((cv[j] >> (8 * k)) & 0xFFu, sv[j]);
        if constexpr (VEC)
          *reinterpret_cast<float4*>(v_out + i) = make_float4(f[0], f[1], f[2], f[3]);
        else
          v_out[i] = f[0];
      }
    }
  }
}

}  // namespace

cudaError_t launch_adamw(const AdamwEntry* t, int count, const AdamwStep& step, bool random, int num_sms,
                         cudaStream_t stream) {
  // (the parameters' bytes cost a launch time: 72 tensors of 4096, 6.8 us in the
  // largest table, 6.1 in the middle one)
  if (count <= 16) return adamw_with<16>(t, count, step, random, num_sms, stream);
  if (count <= 96) return adamw_with<96>(t, count, step, random, num_sms, stream);
  return adamw_with<kAdamwTensors>(t, count, step, random, num_sms, stream);
}

cudaError_t launch_adamw_load(const int8_t* m, const float* ms, const uint8_t* v, const float* vs, float* m_out,
                              float* v_out, int64_t n, int num_sms, cudaStream_t stream) {
  auto aligned = [](const void* p, uintptr_t bytes) { return (reinterpret_cast<uintptr_t>(p) & (bytes - 1)) == 0; };
  const bool vec = n % 4 == 0 && aligned(m, 4) && aligned(v, 4) && aligned(m_out, 16) && aligned(v_out, 16);
  const int64_t per = kThreads * (vec ? 16 : 1);
  // (four pieces a thread, and blocks that balance: 100.8 M values 168 us with 8
  // an SM, 155 with 32, 153 with 64; a block to every piece costs 6.2 M values 2.5 us)
  const int64_t want = (n + per - 1) / per, most = static_cast<int64_t>(num_sms) * 64;
  PdlLaunch l(dim3(static_cast<unsigned>(want < most ? want : most)), dim3(kThreads), 0, stream);
  return cudaLaunchKernelEx(&l.cfg, vec ? adamw_load_kernel<true> : adamw_load_kernel<false>, m, ms, v, vs, m_out, v_out,
                            n);
}

// The -DHGEMM_DEBUG build's check word of this file (null otherwise).
HG_DEBUG_WORD_ACCESSOR(adamw)

}  // namespace hg
