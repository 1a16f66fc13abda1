// hgemm_linear.cu — linear layers (hgemm_linear, its input's and its weight's
// gradient) in a form that is right for every shape, pitch and alignment.
#include "debug.cuh"
#include "linear_epilogue.cuh"
#include "ptx.cuh"

namespace hg {
namespace {

constexpr int kTile = 64;  // output rows and columns per block: one 8-bit group wide
constexpr int kStep = 16;  // K per stage

// C = epilogue(A·B), 64×64 outputs per block of 256 threads (4×4 each),
// FP32 multiply-adds on operands staged in shared memory.
__global__ void __launch_bounds__(256) linear_simple_kernel(const SimpleProduct p) {
  __shared__ float sa[kStep][kTile + 1], sb[kStep][kTile + 1];
  __shared__ float sc[kTile][kTile + 1];
  grid_dependency_wait();
  grid_launch_dependents();
  const int64_t tiles_n = (p.N + kTile - 1) / kTile;
  const int64_t m0 = blockIdx.x / tiles_n * kTile, n0 = blockIdx.x % tiles_n * kTile;
  const int tx = threadIdx.x & 15, ty = threadIdx.x >> 4;
  float acc[4][4] = {};
  for (int64_t k0 = 0; k0 < p.K; k0 += kStep) {
    for (int i = threadIdx.x; i < kTile * kStep; i += 256) {
      const int r = i / kStep, k = i % kStep;
      const bool in_k = k0 + k < p.K;
      sa[k][r] = in_k && m0 + r < p.M
                     ? __half2float(__ushort_as_half(p.A[(m0 + r) * p.sai + (k0 + k) * p.sak])) : 0.f;
      sb[k][r] = in_k && n0 + r < p.N
                     ? __half2float(__ushort_as_half(p.B[(k0 + k) * p.sbk + (n0 + r) * p.sbj])) : 0.f;
    }
    __syncthreads();
#pragma unroll
    for (int k = 0; k < kStep; ++k)
#pragma unroll
      for (int i = 0; i < 4; ++i)
#pragma unroll
        for (int j = 0; j < 4; ++j) acc[i][j] = fmaf(sa[k][ty * 4 + i], sb[k][tx * 4 + j], acc[i][j]);
    __syncthreads();
  }
  for (int i = 0; i < 4; ++i)
    for (int j = 0; j < 4; ++j) sc[ty * 4 + i][tx * 4 + j] = acc[i][j];
  __syncthreads();
  // one row per warp at a time, two columns per lane
  const LinEpi& e = p.epi;
  const int lane = threadIdx.x & 31;
  for (int r = threadIdx.x >> 5; r < kTile; r += 8) {
    const int64_t m = m0 + r;
    if (m >= p.M) break;
    float u[2], scale = 1.f, inv = 0.f;
    if (e.backward) {
      if (e.codes) scale = e.scales[n0 / kCkptGroup * e.lds + m];
    } else {
      uint32_t top = 0;
      for (int i = 0; i < 2; ++i) {
        const int64_t n = n0 + lane + 32 * i;
        u[i] = sc[r][lane + 32 * i];
        if (e.bias && n < p.N) u[i] += __half2float(__ushort_as_half(e.bias[n]));
        top = max(top, magnitude_bits(u[i]));
      }
      if (e.codes) {
        ckpt_scale(__reduce_max_sync(0xffffffffu, top), scale, inv);
        if (lane == 0) e.scales[n0 / kCkptGroup * e.lds + m] = scale;
      }
    }
    for (int i = 0; i < 2; ++i) {
      const int64_t n = n0 + lane + 32 * i;
      if (n >= p.N) continue;
      float y;
      if (e.backward) {
        y = sc[r][lane + 32 * i];
        if (e.codes) {
          float f, df;
          activate<true>(static_cast<float>(e.codes[m * e.ldq + n]) * scale, e.act, f, df);
          y *= df;
          if (e.h) e.h[m * e.ldh + n] = __half_as_ushort(__float2half_rn(f));
        }
      } else {
        if (e.codes) e.codes[m * e.ldq + n] = static_cast<int8_t>(ckpt_code(u[i], inv));
        y = activate(u[i], e.act);
        if (e.res) y += __half2float(__ushort_as_half(e.res[m * e.ldr + n]));
      }
      p.C[m * p.ldc + n] = __half_as_ushort(__float2half_rn(y));
    }
  }
}

// Column sums: 32 columns per block, 8 threads down each, rows in a fixed order.
__global__ void __launch_bounds__(256)
    column_sums_kernel(const uint16_t* __restrict__ dy, int64_t ld, int64_t M, int64_t N, float* __restrict__ out,
                       int accumulate) {
  __shared__ float s[8][33];
  grid_dependency_wait();
  grid_launch_dependents();
  const int c = threadIdx.x & 31, r = threadIdx.x >> 5;
  const int64_t n = static_cast<int64_t>(blockIdx.x) * 32 + c;
  float sum = 0.f;
  if (n < N)
    for (int64_t m = r; m < M; m += 8) sum += __half2float(__ushort_as_half(dy[m * ld + n]));
  s[r][c] = sum;
  __syncthreads();
  if (r == 0 && n < N) {
    for (int i = 1; i < 8; ++i) sum += s[i][c];
    out[n] = accumulate ? out[n] + sum : sum;
  }
}

}  // namespace

cudaError_t launch_linear_simple(const SimpleProduct& p, cudaStream_t stream) {
  const int64_t blocks = ((p.M + kTile - 1) / kTile) * ((p.N + kTile - 1) / kTile);
  if (blocks > 0x7FFFFFFF) return cudaErrorInvalidValue;
  PdlLaunch l(dim3(static_cast<unsigned>(blocks)), dim3(256), 0, stream);
  return cudaLaunchKernelEx(&l.cfg, linear_simple_kernel, p);
}

cudaError_t launch_column_sums(const uint16_t* dy, int64_t ld, int64_t M, int64_t N, float* out, bool accumulate,
                               cudaStream_t stream) {
  PdlLaunch l(dim3(static_cast<unsigned>((N + 31) / 32)), dim3(256), 0, stream);
  return cudaLaunchKernelEx(&l.cfg, column_sums_kernel, dy, ld, M, N, out, accumulate ? 1 : 0);
}

// The -DHGEMM_DEBUG build's check word of this file (null otherwise).
HG_DEBUG_WORD_ACCESSOR(linear)

}  // namespace hg
