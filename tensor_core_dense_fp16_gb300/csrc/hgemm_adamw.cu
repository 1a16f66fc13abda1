// hgemm_adamw.cu — an AdamW step over many tensors in one launch, and 8-bit
// states read back (hgemm_adamw, hgemm_adamw_load; the formulas and the 8-bit
// forms are in hgemm.h). Bound by memory: with FP32 states, a master copy, an
// FP16 gradient and weight 28 bytes per value, with 8-bit states and no master
// 10.25.
#include <cuda_fp16.h>

#include "debug.cuh"
#include "internal.h"
#include "linear_epilogue.cuh"
#include "ptx.cuh"
#include "row_sums.cuh"

namespace hg {
namespace {

constexpr int kThreads = 256;
constexpr int kChunk = kAdamwChunk;  // values of a block's step: 8 per thread, whole groups
static_assert(kChunk == kThreads * 8 && kChunk % kCkptGroup == 0, "a group lies in one warp's values");

// The tensors travel as the launch's parameters: nothing has to be copied
// before it, and a captured graph holds them.
template <int MAX>
struct AdamwTable {
  AdamwStep step;
  int count;
  uint32_t chunks;
  AdamwEntry t[MAX];
};

__device__ __forceinline__ float sqrt_approx(float x) {
  float y;
  asm("sqrt.approx.f32 %0, %1;" : "=f"(y) : "f"(x));
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

// The upper 12 bits of an FP32 number in (0, 1] (8 of exponent, 3 of fraction)
// rounded at the 20th, counted from 1's.
__device__ __forceinline__ uint32_t second_code(float v, float inv) {
  const float r = __fmul_rn(v, inv);
  const int c = 255 + (static_cast<int>(__float_as_uint(r) - kOneBits + 0x80000u) >> 20);
  return r > 0.f ? static_cast<uint32_t>(min(max(c, 1), 255)) : 0u;
}

__device__ __forceinline__ float second_value(uint32_t code, float scale) {
  const float r = code ? __uint_as_float(kOneBits - ((255u - code) << 20)) : 0.f;
  return __fmul_rn(r, scale);
}

// ------------------------------------------------------------------ the step

struct Scalars {
  float gscale, a, b, lr;
  bool dynamic;
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
template <bool VEC>
__device__ __forceinline__ void adamw_eight(const AdamwEntry& t, const AdamwStep& s, const Scalars& c, float keep,
                                            int64_t first) {
  const int64_t n = t.n;
  const bool in = first < n;  // VEC: all eight, n is a multiple of 8
  const bool eight = t.ms != nullptr;
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
#pragma unroll
    for (int i = 0; i < 8; i += 2) {
      float scale_m, inv_m, scale_v, inv_v;
      ckpt_scale(group_top<VEC>(m, i), scale_m, inv_m);
      second_scale(group_top<VEC>(v, i), scale_v, inv_v);
#pragma unroll
      for (int j = i; j < (VEC ? 8 : i + 2); ++j) {
        qm[j] = inv_m == 0.f ? 0u : ckpt_code(m[j], inv_m);
        qv[j] = inv_v == 0.f ? 0u : second_code(v[j], inv_v);
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

template <int MAX>
__global__ void __launch_bounds__(kThreads) adamw_kernel(const __grid_constant__ AdamwTable<MAX> table) {
  grid_dependency_wait();
  grid_launch_dependents();
  const AdamwStep& s = table.step;
  Scalars c{s.gscale, s.a, s.b, s.lr, s.dynamic != nullptr};
  if (c.dynamic) {
    const hgemm_adamw_dynamic d = *s.dynamic;
    if (d.skip) return;
    const float step = static_cast<float>(max(d.step, 1));
    c.gscale = d.grad_scale;
    c.lr = d.lr;
    c.a = d.lr / -expm1f(step * s.ln1);
    c.b = rsqrtf(-expm1f(step * s.ln2));
  }
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
    const int64_t base = static_cast<int64_t>(chunk - t.chunk0) * kChunk;
    const float keep = c.dynamic ? fmaf(-c.lr, t.decay, 1.f) : t.keep;
    if (t.vec)
      adamw_eight<true>(t, s, c, keep, base + 8 * static_cast<int>(threadIdx.x));
    else
      adamw_eight<false>(t, s, c, keep, base + (threadIdx.x >> 5) * 256 + (threadIdx.x & 31));
  }
}

template <int MAX>
cudaError_t adamw_with(const AdamwEntry* t, int count, uint32_t chunks, const AdamwStep& step, int num_sms,
                       cudaStream_t stream) {
  AdamwTable<MAX> table;
  table.step = step;
  table.count = count;
  table.chunks = chunks;
  for (int i = 0; i < count; ++i) table.t[i] = t[i];
  const uint32_t most = static_cast<uint32_t>(num_sms) * 8u;
  PdlLaunch l(dim3(chunks < most ? chunks : most), dim3(kThreads), 0, stream);
  return cudaLaunchKernelEx(&l.cfg, adamw_kernel<MAX>, table);
}

// One value per thread.
__global__ void __launch_bounds__(kThreads)
    adamw_load_kernel(const int8_t* m, const float* ms, const uint8_t* v, const float* vs, float* m_out, float* v_out,
                      int64_t n) {
  grid_dependency_wait();
  grid_launch_dependents();
  const int64_t step = static_cast<int64_t>(gridDim.x) * kThreads;
  for (int64_t i = static_cast<int64_t>(blockIdx.x) * kThreads + threadIdx.x; i < n; i += step) {
    if (!HG_DBG_INDEX(i, n)) return;
    if (m) m_out[i] = __fmul_rn(static_cast<float>(m[i]), ms[i / kCkptGroup]);
    if (v) v_out[i] = second_value(v[i], vs[i / kCkptGroup]);
  }
}

}  // namespace

cudaError_t launch_adamw(const AdamwEntry* t, int count, uint32_t chunks, const AdamwStep& step, int num_sms,
                         cudaStream_t stream) {
  if (count <= 16) return adamw_with<16>(t, count, chunks, step, num_sms, stream);
  return adamw_with<kAdamwTensors>(t, count, chunks, step, num_sms, stream);
}

cudaError_t launch_adamw_load(const int8_t* m, const float* ms, const uint8_t* v, const float* vs, float* m_out,
                              float* v_out, int64_t n, int num_sms, cudaStream_t stream) {
  const int64_t want = (n + kThreads - 1) / kThreads, most = static_cast<int64_t>(num_sms) * 8;
  PdlLaunch l(dim3(static_cast<unsigned>(want < most ? want : most)), dim3(kThreads), 0, stream);
  return cudaLaunchKernelEx(&l.cfg, adamw_load_kernel, m, ms, v, vs, m_out, v_out, n);
}

// The -DHGEMM_DEBUG build's check word of this file (null otherwise).
HG_DEBUG_WORD_ACCESSOR(adamw)

}  // namespace hg
