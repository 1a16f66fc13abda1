// hgemm_norm.cu — layer norm over rows, forward and backward (the formulas
// are in hgemm.h).
#include <cuda_fp16.h>

#include "debug.cuh"
#include "internal.h"
#include "ptx.cuh"

namespace hg {
namespace {

constexpr int kThreads = 256;

__device__ __forceinline__ float half_at(const uint16_t* p, int64_t i) {
  return __half2float(__ushort_as_half(p[i]));
}

// The block's sums of a and b, in every thread (a fixed order).
__device__ __forceinline__ void block_sum2(float& a, float& b, float (&s)[2][kThreads / 32]) {
  for (int o = 16; o > 0; o >>= 1) {
    a += __shfl_xor_sync(0xffffffffu, a, o);
    b += __shfl_xor_sync(0xffffffffu, b, o);
  }
  __syncthreads();
  if ((threadIdx.x & 31) == 0) {
    s[0][threadIdx.x >> 5] = a;
    s[1][threadIdx.x >> 5] = b;
  }
  __syncthreads();
  a = b = 0.f;
  for (int i = 0; i < kThreads / 32; ++i) {
    a += s[0][i];
    b += s[1][i];
  }
}

// One block per row: the mean, the variance around it, the output.
__global__ void __launch_bounds__(kThreads) layernorm_forward_kernel(const NormArgs a) {
  __shared__ float s[2][kThreads / 32];
  grid_dependency_wait();
  grid_launch_dependents();
  for (int64_t m = blockIdx.x; m < a.M; m += gridDim.x) {
    const uint16_t* x = a.x + m * a.ldx;
    float sum = 0.f, none = 0.f;
    for (int64_t d = threadIdx.x; d < a.D; d += kThreads) sum += half_at(x, d);
    block_sum2(sum, none, s);
    const float mu = sum / static_cast<float>(a.D);
    float sq = 0.f;
    for (int64_t d = threadIdx.x; d < a.D; d += kThreads) {
      const float v = half_at(x, d) - mu;
      sq = fmaf(v, v, sq);
    }
    block_sum2(sq, none, s);
    const float rs = rsqrtf(sq / static_cast<float>(a.D) + a.eps);
    for (int64_t d = threadIdx.x; d < a.D; d += kThreads)
      a.y[m * a.ldy + d] = __half_as_ushort(
          __float2half_rn(fmaf((half_at(x, d) - mu) * rs, half_at(a.gamma, d), half_at(a.beta, d))));
    if (threadIdx.x == 0 && a.mean) {
      a.mean[m] = mu;
      a.rstd[m] = rs;
    }
  }
}

// Partial sums of dgamma and dbeta: 32 columns per block, the rows of
// blockIdx.y's share; work holds [slice][2][D].
constexpr int kSlices = 32;
__global__ void __launch_bounds__(kThreads) layernorm_partials_kernel(const NormArgs a) {
  __shared__ float s[2][8][33];
  grid_dependency_wait();
  grid_launch_dependents();
  const int c = threadIdx.x & 31, r = threadIdx.x >> 5;
  const int64_t d = static_cast<int64_t>(blockIdx.x) * 32 + c;
  float dg = 0.f, db = 0.f;
  if (d < a.D)
    for (int64_t m = blockIdx.y * 8 + r; m < a.M; m += 8 * kSlices) {
      const float g = half_at(a.dy, m * a.lddy + d);
      dg = fmaf(g, (half_at(a.x, m * a.ldx + d) - a.mean[m]) * a.rstd[m], dg);
      db += g;
    }
  s[0][r][c] = dg;
  s[1][r][c] = db;
  __syncthreads();
  if (r == 0 && d < a.D) {
    for (int i = 1; i < 8; ++i) {
      dg += s[0][i][c];
      db += s[1][i][c];
    }
    a.work[(static_cast<int64_t>(blockIdx.y) * 2) * a.D + d] = dg;
    a.work[(static_cast<int64_t>(blockIdx.y) * 2 + 1) * a.D + d] = db;
  }
}

// One block per row of dX (after the partial sums, which read dY: dX may be
// dY itself); the first blocks also add up the partial sums.
__global__ void __launch_bounds__(kThreads) layernorm_backward_kernel(const NormArgs a) {
  __shared__ float s[2][kThreads / 32];
  grid_dependency_wait();
  grid_launch_dependents();
  for (int64_t d = static_cast<int64_t>(blockIdx.x) * kThreads + threadIdx.x; d < a.D;
       d += static_cast<int64_t>(gridDim.x) * kThreads) {
    float dg = 0.f, db = 0.f;
    for (int i = 0; i < kSlices; ++i) {
      dg += a.work[static_cast<int64_t>(i) * 2 * a.D + d];
      db += a.work[(static_cast<int64_t>(i) * 2 + 1) * a.D + d];
    }
    a.dgamma[d] = dg;
    a.dbeta[d] = db;
  }
  for (int64_t m = blockIdx.x; m < a.M; m += gridDim.x) {
    const float mu = a.mean[m], rs = a.rstd[m];
    float s1 = 0.f, s2 = 0.f;
    for (int64_t d = threadIdx.x; d < a.D; d += kThreads) {
      const float g = half_at(a.dy, m * a.lddy + d) * half_at(a.gamma, d);
      s1 += g;
      s2 = fmaf(g, (half_at(a.x, m * a.ldx + d) - mu) * rs, s2);
    }
    block_sum2(s1, s2, s);
    s1 /= static_cast<float>(a.D);
    s2 /= static_cast<float>(a.D);
    for (int64_t d = threadIdx.x; d < a.D; d += kThreads) {
      const float g = half_at(a.dy, m * a.lddy + d) * half_at(a.gamma, d);
      const float xh = (half_at(a.x, m * a.ldx + d) - mu) * rs;
      float v = rs * (g - s1 - xh * s2);
      if (a.res) v += half_at(a.res, m * a.ldr + d);
      a.y[m * a.ldy + d] = __half_as_ushort(__float2half_rn(v));
    }
  }
}

unsigned rows_grid(int64_t M) { return static_cast<unsigned>(M < 1 ? 1 : (M > 65536 ? 65536 : M)); }

}  // namespace

cudaError_t launch_layernorm_forward(const NormArgs& a, int, cudaStream_t stream) {
  PdlLaunch l(dim3(rows_grid(a.M)), dim3(kThreads), 0, stream);
  return cudaLaunchKernelEx(&l.cfg, layernorm_forward_kernel, a);
}

size_t layernorm_backward_workspace(int64_t, int64_t D) { return sizeof(float) * 2 * kSlices * static_cast<size_t>(D); }

cudaError_t launch_layernorm_backward(const NormArgs& a, int, cudaStream_t stream) {
  PdlLaunch p(dim3(static_cast<unsigned>((a.D + 31) / 32), kSlices), dim3(kThreads), 0, stream);
  const cudaError_t e = cudaLaunchKernelEx(&p.cfg, layernorm_partials_kernel, a);
  if (e != cudaSuccess) return e;
  PdlLaunch l(dim3(rows_grid(a.M)), dim3(kThreads), 0, stream);
  return cudaLaunchKernelEx(&l.cfg, layernorm_backward_kernel, a);
}

// The -DHGEMM_DEBUG build's check word of this file (null otherwise).
HG_DEBUG_WORD_ACCESSOR(norm)

}  // namespace hg
