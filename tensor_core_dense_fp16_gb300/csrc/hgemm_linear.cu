// hgemm_linear.cu — the parts of linear layers (hgemm_linear and its
// gradients) that are no large products: these run on the product kernels
// with the epilogues of linear_epilogue.cuh.
#include "debug.cuh"
#include "linear_epilogue.cuh"
#include "ptx.cuh"

namespace hg {
namespace {

// The epilogue of empty sums: one warp per row and group of 64 columns, two
// columns per lane.
template <bool BACKWARD>
__global__ void __launch_bounds__(256)
    linear_empty_kernel(uint16_t* __restrict__ C, int64_t ldc, int64_t M, int64_t N, const LinEpi e) {
  grid_dependency_wait();
  grid_launch_dependents();
  const int lane = threadIdx.x & 31;
  const int64_t groups = (N + kCkptGroup - 1) / kCkptGroup;
  const int64_t warps = static_cast<int64_t>(gridDim.x) * 8;
  for (int64_t t = static_cast<int64_t>(blockIdx.x) * 8 + (threadIdx.x >> 5); t < M * groups; t += warps) {
    const int64_t m = t / groups, g = t - m * groups;
    float u[2], scale = 0.f, inv = 0.f;
    for (int i = 0; i < 2; ++i) {
      const int64_t n = g * kCkptGroup + lane + 32 * i;
      u[i] = !BACKWARD && e.bias && n < N ? __half2float(__ushort_as_half(e.bias[n])) : 0.f;
    }
    if (e.codes) {
      if (BACKWARD) {
        scale = e.scales[g * e.lds + m];
      } else {
        ckpt_scale(__reduce_max_sync(0xffffffffu, max(magnitude_bits(u[0]), magnitude_bits(u[1]))), scale, inv);
        if (lane == 0) e.scales[g * e.lds + m] = scale;
      }
    }
    for (int i = 0; i < 2; ++i) {
      const int64_t n = g * kCkptGroup + lane + 32 * i;
      if (n < N) lin_scalar<BACKWARD>(e, u[i], m, n, scale, inv, C + m * ldc + n);
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

cudaError_t launch_linear_empty(uint16_t* C, int64_t ldc, int64_t M, int64_t N, const LinEpi& epi,
                                cudaStream_t stream) {
  const int64_t blocks = (M * ((N + kCkptGroup - 1) / kCkptGroup) + 7) / 8;
  PdlLaunch l(dim3(static_cast<unsigned>(blocks < 4096 ? blocks : 4096)), dim3(256), 0, stream);
  return cudaLaunchKernelEx(&l.cfg, epi.backward ? linear_empty_kernel<true> : linear_empty_kernel<false>, C, ldc, M,
                            N, epi);
}

cudaError_t launch_column_sums(const uint16_t* dy, int64_t ld, int64_t M, int64_t N, float* out, bool accumulate,
                               cudaStream_t stream) {
  PdlLaunch l(dim3(static_cast<unsigned>((N + 31) / 32)), dim3(256), 0, stream);
  return cudaLaunchKernelEx(&l.cfg, column_sums_kernel, dy, ld, M, N, out, accumulate ? 1 : 0);
}

// The -DHGEMM_DEBUG build's check word of this file (null otherwise).
HG_DEBUG_WORD_ACCESSOR(linear)

}  // namespace hg
