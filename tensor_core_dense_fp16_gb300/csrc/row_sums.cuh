// row_sums.cuh — what the kernels over rows (the norms) share: FP16 values in
// and out, and sums over the threads that share a row.
#pragma once

#include <cuda_fp16.h>

#include "kernel_common.cuh"
#include "linear_epilogue.cuh"
#include "ptx.cuh"

namespace hg {

__device__ __forceinline__ float half_at(const uint16_t* p, int64_t i) {
  return __half2float(__ushort_as_half(p[i]));
}

__device__ __forceinline__ void unpack8(uint4 v, float (&f)[8]) {
  const __half2* h = reinterpret_cast<const __half2*>(&v);
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const float2 t = __half22float2(h[i]);
    f[2 * i] = t.x;
    f[2 * i + 1] = t.y;
  }
}

__device__ __forceinline__ void unpack8(uint4 v, f32x2 (&f)[4]) {
  f[0] = unpack_half2(v.x);
  f[1] = unpack_half2(v.y);
  f[2] = unpack_half2(v.z);
  f[3] = unpack_half2(v.w);
}

__device__ __forceinline__ uint4 pack8f(const float (&f)[8]) {
  uint32_t w[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) w[i] = pack_half2(__float_as_uint(f[2 * i]), __float_as_uint(f[2 * i + 1]));
  return make_uint4(w[0], w[1], w[2], w[3]);
}

__device__ __forceinline__ float warp_sum(float a) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) a += __shfl_xor_sync(0xffffffffu, a, o);
  return a;
}

// Both sums over a warp, in every lane, in 6 shuffles instead of 10: after the
// first the lower lanes go on with a and the upper with b.
__device__ __forceinline__ void warp_sum2(float& a, float& b) {
  const bool upper = (threadIdx.x & 16) != 0;
  const float other = __shfl_xor_sync(0xffffffffu, upper ? a : b, 16);
  float v = (upper ? b : a) + other;
#pragma unroll
  for (int o = 8; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
  const float w = __shfl_xor_sync(0xffffffffu, v, 16);
  a = upper ? w : v;
  b = upper ? v : w;
}

// A sum over the G threads that share a row, in each of them. `s` holds one
// value per warp of the block; the group's warps are neighbours.
template <int G>
__device__ __forceinline__ float group_sum(float a, float* s) {
  a = warp_sum(a);
  if constexpr (G > 32) {
    static_assert(G % 32 == 0, "whole warps");
    __syncthreads();  // (one group per block) the previous sum has been read
    if ((threadIdx.x & 31) == 0) s[threadIdx.x >> 5] = a;
    __syncthreads();
    a = 0.f;
#pragma unroll
    for (int i = 0; i < G / 32; ++i) a += s[i];
  }
  return a;
}

// One block per row, at most 65536.
inline unsigned rows_grid(int64_t M) { return static_cast<unsigned>(M < 1 ? 1 : (M > 65536 ? 65536 : M)); }

inline bool rows16(const void* p, int64_t ld) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0 && ld % 8 == 0; }

}  // namespace hg
