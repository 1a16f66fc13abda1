// hgemm_ckpt8.cu — a matrix into its 8-bit form and back (hgemm_ckpt8_save,
// hgemm_ckpt8_load; the form is defined in hgemm.h).
#include "debug.cuh"
#include "linear_epilogue.cuh"
#include "ptx.cuh"

namespace hg {
namespace {

// One warp per group of 64 columns of a row, two columns per lane.
__global__ void __launch_bounds__(256)
    ckpt8_save_kernel(const uint16_t* __restrict__ x, int64_t ldx, int8_t* __restrict__ codes, int64_t ldq,
                      float* __restrict__ scales, int64_t lds, int64_t M, int64_t N) {
  grid_dependency_wait();
  grid_launch_dependents();
  const int lane = threadIdx.x & 31;
  const int64_t groups = (N + kCkptGroup - 1) / kCkptGroup;
  const int64_t warps = static_cast<int64_t>(gridDim.x) * (blockDim.x >> 5);
  for (int64_t t = static_cast<int64_t>(blockIdx.x) * (blockDim.x >> 5) + (threadIdx.x >> 5); t < M * groups;
       t += warps) {
    const int64_t m = t / groups, g = t - m * groups;
    float u[2];
    uint32_t top = 0;
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      const int64_t n = g * kCkptGroup + lane + 32 * i;
      u[i] = n < N ? __half2float(__ushort_as_half(x[m * ldx + n])) : 0.f;
      top = max(top, magnitude_bits(u[i]));
    }
    top = __reduce_max_sync(0xffffffffu, top);
    float scale, inv;
    ckpt_scale(top, scale, inv);
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      const int64_t n = g * kCkptGroup + lane + 32 * i;
      if (n < N) codes[m * ldq + n] = static_cast<int8_t>(inv == 0.f ? 0u : ckpt_code(u[i], inv));
    }
    if (lane == 0) scales[g * lds + m] = scale;
  }
}

__global__ void __launch_bounds__(256)
    ckpt8_load_kernel(const int8_t* __restrict__ codes, int64_t ldq, const float* __restrict__ scales, int64_t lds,
                      int act, uint16_t* __restrict__ y, int64_t ldy, int64_t M, int64_t N) {
  grid_dependency_wait();
  grid_launch_dependents();
  const int64_t stride = static_cast<int64_t>(gridDim.x) * blockDim.x;
  for (int64_t i = static_cast<int64_t>(blockIdx.x) * blockDim.x + threadIdx.x; i < M * N; i += stride) {
    const int64_t m = i / N, n = i - m * N;
    const float u = static_cast<float>(codes[m * ldq + n]) * scales[n / kCkptGroup * lds + m];
    y[m * ldy + n] = __half_as_ushort(__float2half_rn(activate(u, act)));
  }
}

unsigned blocks_for(int64_t items, int64_t per_block) {
  const int64_t b = (items + per_block - 1) / per_block;
  return static_cast<unsigned>(b < 1 ? 1 : (b > 65536 ? 65536 : b));
}

}  // namespace

cudaError_t launch_ckpt8_save(const uint16_t* x, int64_t ldx, int8_t* codes, int64_t ldq, float* scales,
                              int64_t lds, int64_t M, int64_t N, cudaStream_t stream) {
  const int64_t groups = (N + kCkptGroup - 1) / kCkptGroup;
  PdlLaunch l(dim3(blocks_for(M * groups, 8)), dim3(256), 0, stream);
  return cudaLaunchKernelEx(&l.cfg, ckpt8_save_kernel, x, ldx, codes, ldq, scales, lds, M, N);
}

cudaError_t launch_ckpt8_load(const int8_t* codes, int64_t ldq, const float* scales, int64_t lds, int act,
                              uint16_t* y, int64_t ldy, int64_t M, int64_t N, cudaStream_t stream) {
  PdlLaunch l(dim3(blocks_for(M * N, 256)), dim3(256), 0, stream);
  return cudaLaunchKernelEx(&l.cfg, ckpt8_load_kernel, codes, ldq, scales, lds, act, y, ldy, M, N);
}

// The -DHGEMM_DEBUG build's check word of this file (null otherwise).
HG_DEBUG_WORD_ACCESSOR(ckpt8)

}  // namespace hg
