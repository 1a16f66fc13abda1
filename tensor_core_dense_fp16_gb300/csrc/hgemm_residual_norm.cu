// hgemm_residual_norm.cu — the norms around a block with its gate and the
// residual's scale, forward and backward (the formulas are in hgemm.h). Both
// are bound by memory: forward reads 4 bytes per value and writes 4, backward
// reads 8 and writes 4.
#include <cuda_fp16.h>

#include "debug.cuh"
#include "hgemm.h"
#include "internal.h"
#include "kernel_common.cuh"
#include "ptx.cuh"
#include "row_sums.cuh"

namespace hg {
namespace {

constexpr int kThreads = 256;

__device__ __forceinline__ float half_or(const uint16_t* p, int64_t i, float otherwise) {
  return p ? half_at(p, i) : otherwise;
}

// μ and ρ of a row's values v(d), d = threadIdx.x, + kThreads, ...
template <typename Value>
__device__ __forceinline__ void row_moments(int kind, int64_t D, float eps, float* s, Value v, float& mu, float& rho) {
  const float n = static_cast<float>(D);
  mu = 0.f;
  if (kind == HGEMM_NORM_LAYER) {
    float sum = 0.f;
    for (int64_t d = threadIdx.x; d < D; d += kThreads) sum += v(d);
    mu = group_sum<kThreads>(sum, s) / n;
  }
  float sq = 0.f;
  for (int64_t d = threadIdx.x; d < D; d += kThreads) {
    const float c = v(d) - mu;
    sq = fmaf(c, c, sq);
  }
  rho = rsqrtf(group_sum<kThreads>(sq, s) / n + eps);
}

// Any length, pitch and alignment: a block per row, which it reads once per
// sum (from L1 or L2 after the first).
__global__ void __launch_bounds__(kThreads) residual_norm_forward_kernel(const ResidualNormArgs a) {
  __shared__ float s[kThreads / 32];
  grid_dependency_wait();
  grid_launch_dependents();
  for (int64_t m = blockIdx.x; m < a.M; m += gridDim.x) {
    if (!HG_DBG_INDEX(m, a.M)) return;
    const uint16_t *x = a.x + m * a.ldx, *y = a.y + m * a.ldy;
    float my = 0.f, ry = 1.f, mz = 0.f, rz = 1.f;
    if (a.post) row_moments(a.post, a.D, a.eps, s, [&](int64_t d) { return half_at(y, d); }, my, ry);
    auto z = [&](int64_t d) {
      float n = half_at(y, d);
      if (a.post) n = fmaf((n - my) * ry, half_at(a.post_gamma, d), half_or(a.post_beta, d, 0.f));
      return fmaf(a.alpha, half_at(x, d), n * half_or(a.gate, d, 1.f));
    };
    if (a.pre) row_moments(a.pre, a.D, a.eps, s, z, mz, rz);
    __syncthreads();  // (Z may be X and H may be Y) the row has been read
    for (int64_t d = threadIdx.x; d < a.D; d += kThreads) {
      const float v = z(d);
      a.z[m * a.ldz + d] = __half_as_ushort(__float2half_rn(v));
      if (a.pre)
        a.h[m * a.ldh + d] = __half_as_ushort(
            __float2half_rn(fmaf((v - mz) * rz, half_at(a.pre_gamma, d), half_or(a.pre_beta, d, 0.f))));
    }
    if (threadIdx.x == 0 && a.stats) {
      if (a.post) a.stats[m] = my, a.stats[a.M + m] = ry;
      if (a.pre) a.stats[2 * a.M + m] = mz, a.stats[3 * a.M + m] = rz;
    }
  }
}

// ----------------------------------------------------------------- backward

// What the gradients of a value need of its row: the statistics and the four
// means a1 = mean(g), a2 = mean(g·ẑ) (g = dH·γ), b1 = mean(w·dz),
// b2 = mean(w·dz·ŷ) (w = gate·γ'), a layer norm's a1 and b1 0 for an RMS norm.
struct BackRow {
  float my, ry, mz, rz, a1, a2, b1, b2;
};

__device__ __forceinline__ BackRow back_row(const ResidualNormBackArgs& a, int64_t m) {
  BackRow r{0.f, 1.f, 0.f, 1.f, 0.f, 0.f, 0.f, 0.f};
  if (a.post) r.my = a.stats[m], r.ry = a.stats[a.M + m];
  if (a.pre) r.mz = a.stats[2 * a.M + m], r.rz = a.stats[3 * a.M + m];
  return r;
}

// dz of one value.
__device__ __forceinline__ float back_dz(const ResidualNormBackArgs& a, const BackRow& r, int64_t m, int64_t d) {
  float v = a.dz ? half_at(a.dz, m * a.lddz + d) : 0.f;
  if (a.pre) {
    const float g = half_at(a.dh, m * a.lddh + d) * half_at(a.pre_gamma, d);
    const float zh = (half_at(a.z, m * a.ldz + d) - r.mz) * r.rz;
    v = fmaf(r.rz, g - r.a1 - zh * r.a2, v);
  }
  return v;
}

__device__ __forceinline__ float back_yh(const ResidualNormBackArgs& a, const BackRow& r, int64_t m, int64_t d) {
  return (half_at(a.y, m * a.ldy + d) - r.my) * r.ry;
}

// Any length, pitch and alignment, for the rows m0 .. m1-1 whose means the
// workspace holds. First the four means of every row ...
__global__ void __launch_bounds__(kThreads) residual_norm_means_kernel(const ResidualNormBackArgs a) {
  __shared__ float s[kThreads / 32];
  grid_dependency_wait();
  grid_launch_dependents();
  const float n = static_cast<float>(a.D);
  for (int64_t m = a.m0 + blockIdx.x; m < a.m1; m += gridDim.x) {
    if (!HG_DBG_INDEX(m, a.M)) return;
    BackRow r = back_row(a, m);
    float s1 = 0.f, s2 = 0.f;
    if (a.pre) {
      for (int64_t d = threadIdx.x; d < a.D; d += kThreads) {
        const float g = half_at(a.dh, m * a.lddh + d) * half_at(a.pre_gamma, d);
        s1 += g;
        s2 = fmaf(g, (half_at(a.z, m * a.ldz + d) - r.mz) * r.rz, s2);
      }
      if (a.pre == HGEMM_NORM_LAYER) r.a1 = group_sum<kThreads>(s1, s) / n;
      r.a2 = group_sum<kThreads>(s2, s) / n;
    }
    if (a.post) {
      s1 = s2 = 0.f;
      for (int64_t d = threadIdx.x; d < a.D; d += kThreads) {
        const float w = half_or(a.gate, d, 1.f) * half_at(a.post_gamma, d) * back_dz(a, r, m, d);
        s1 += w;
        s2 = fmaf(w, back_yh(a, r, m, d), s2);
      }
      if (a.post == HGEMM_NORM_LAYER) r.b1 = group_sum<kThreads>(s1, s) / n;
      r.b2 = group_sum<kThreads>(s2, s) / n;
    }
    if (threadIdx.x == 0) reinterpret_cast<float4*>(a.means)[m - a.m0] = make_float4(r.a1, r.a2, r.b1, r.b2);
  }
}

__device__ __forceinline__ BackRow back_row_means(const ResidualNormBackArgs& a, int64_t m) {
  BackRow r = back_row(a, m);
  const float4 v = reinterpret_cast<const float4*>(a.means)[m - a.m0];
  r.a1 = v.x, r.a2 = v.y, r.b1 = v.z, r.b2 = v.w;
  return r;
}

// ... then partial sums down the columns (dX may be dZ and dY may be dH):
// S1 = Σ dz·ŷ, S0 = Σ dz, T1 = Σ dH·ẑ, T0 = Σ dH ...
constexpr int kSlices = 32;
__global__ void __launch_bounds__(kThreads) residual_norm_partials_kernel(const ResidualNormBackArgs a) {
  __shared__ float s[4][8][33];
  grid_dependency_wait();
  grid_launch_dependents();
  const int c = threadIdx.x & 31, row = threadIdx.x >> 5;
  const int64_t d = static_cast<int64_t>(blockIdx.x) * 32 + c;
  float v[4] = {};
  if (d < a.D) {
    for (int64_t m = a.m0 + blockIdx.y * 8 + row; m < a.m1; m += 8 * kSlices) {
      const BackRow r = back_row_means(a, m);
      const float dz = back_dz(a, r, m, d);
      v[0] = fmaf(dz, back_yh(a, r, m, d), v[0]);
      v[1] += dz;
      if (a.pre) {
        const float dh = half_at(a.dh, m * a.lddh + d);
        v[2] = fmaf(dh, (half_at(a.z, m * a.ldz + d) - r.mz) * r.rz, v[2]);
        v[3] += dh;
      }
    }
  }
#pragma unroll
  for (int i = 0; i < 4; ++i) s[i][row][c] = v[i];
  __syncthreads();
  if (row == 0 && d < a.D && HG_DBG_INDEX(blockIdx.y, kResidualNormPartials)) {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      for (int j = 1; j < 8; ++j) v[i] += s[i][j][c];
      float* out = a.partials + (static_cast<int64_t>(blockIdx.y) * 4 + i) * a.D + d;
      *out = a.m0 > 0 ? *out + v[i] : v[i];
    }
  }
}

// ... then dX and dY.
__global__ void __launch_bounds__(kThreads) residual_norm_backward_kernel(const ResidualNormBackArgs a) {
  grid_dependency_wait();
  grid_launch_dependents();
  for (int64_t m = a.m0 + blockIdx.x; m < a.m1; m += gridDim.x) {
    if (!HG_DBG_INDEX(m, a.M)) return;
    const BackRow r = back_row_means(a, m);
    for (int64_t d = threadIdx.x; d < a.D; d += kThreads) {
      const float dz = back_dz(a, r, m, d), gate = half_or(a.gate, d, 1.f);
      float dy = gate * dz;
      if (a.post) dy = r.ry * (dy * half_at(a.post_gamma, d) - r.b1 - back_yh(a, r, m, d) * r.b2);
      a.dx[m * a.lddx + d] = __half_as_ushort(__float2half_rn(a.alpha * dz));
      a.dy[m * a.lddy + d] = __half_as_ushort(__float2half_rn(dy));
    }
  }
}

// The vectors' gradients from `count` partial sums, in a fixed order: 32
// columns per block, 8 threads down each.
__global__ void __launch_bounds__(kThreads) residual_norm_sums_kernel(const ResidualNormBackArgs a, int count) {
  __shared__ float s[4][8][33];
  grid_dependency_wait();
  grid_launch_dependents();
  const int c = threadIdx.x & 31, r = threadIdx.x >> 5;
  const int64_t d = static_cast<int64_t>(blockIdx.x) * 32 + c;
  float v[4] = {};
  if (d < a.D)
    for (int i = r; i < count; i += 8)
#pragma unroll
      for (int j = 0; j < 4; ++j) v[j] += a.partials[(static_cast<int64_t>(i) * 4 + j) * a.D + d];
#pragma unroll
  for (int j = 0; j < 4; ++j) s[j][r][c] = v[j];
  __syncthreads();
  if (r != 0 || d >= a.D || !HG_DBG_INDEX(d, a.D)) return;
#pragma unroll
  for (int j = 0; j < 4; ++j)
    for (int i = 1; i < 8; ++i) v[j] += s[j][i][c];
  const float gate = half_or(a.gate, d, 1.f);
  if (a.dgate)
    a.dgate[d] = a.post ? fmaf(half_at(a.post_gamma, d), v[0], half_or(a.post_beta, d, 0.f) * v[1]) : v[0];
  if (a.dpost_gamma) a.dpost_gamma[d] = gate * v[0];
  if (a.dpost_beta) a.dpost_beta[d] = gate * v[1];
  if (a.dpre_gamma) a.dpre_gamma[d] = v[2];
  if (a.dpre_beta) a.dpre_beta[d] = v[3];
}

}  // namespace

cudaError_t launch_residual_norm_forward(const ResidualNormArgs& a, int num_sms, cudaStream_t stream) {
  PdlLaunch l(dim3(rows_grid(a.M)), dim3(kThreads), 0, stream);
  return cudaLaunchKernelEx(&l.cfg, residual_norm_forward_kernel, a);
}

// Partial sums; the kernels for any row keep theirs in the first kSlices, and
// the rows' means in the rest.
size_t residual_norm_backward_workspace(int64_t, int64_t D) {
  return sizeof(float) * 4 * kResidualNormPartials * static_cast<size_t>((D + 3) / 4 * 4);
}

cudaError_t launch_residual_norm_backward(ResidualNormBackArgs a, int num_sms, cudaStream_t stream) {
  cudaError_t e = cudaSuccess;
  const int64_t pitch = (a.D + 3) / 4 * 4, most = (kResidualNormPartials - kSlices) * pitch;
  a.means = a.partials + 4 * kSlices * pitch;
  int partials = 0;
  for (a.m0 = 0; a.m0 < a.M; a.m0 = a.m1) {
    a.m1 = a.m0 + most < a.M ? a.m0 + most : a.M;
    PdlLaunch r(dim3(rows_grid(a.m1 - a.m0)), dim3(kThreads), 0, stream);
    if ((e = cudaLaunchKernelEx(&r.cfg, residual_norm_means_kernel, a)) != cudaSuccess) return e;
    PdlLaunch p(dim3(static_cast<unsigned>((a.D + 31) / 32), kSlices), dim3(kThreads), 0, stream);
    if ((e = cudaLaunchKernelEx(&p.cfg, residual_norm_partials_kernel, a)) != cudaSuccess) return e;
    if ((e = cudaLaunchKernelEx(&r.cfg, residual_norm_backward_kernel, a)) != cudaSuccess) return e;
    partials = kSlices;
  }
  if (!a.dgate && !a.dpost_gamma && !a.dpost_beta && !a.dpre_gamma && !a.dpre_beta) return e;
  PdlLaunch l(dim3(static_cast<unsigned>((a.D + 31) / 32)), dim3(kThreads), 0, stream);
  return cudaLaunchKernelEx(&l.cfg, residual_norm_sums_kernel, a, partials);
}

// The -DHGEMM_DEBUG build's check word of this file (null otherwise).
HG_DEBUG_WORD_ACCESSOR(residual_norm)

}  // namespace hg
