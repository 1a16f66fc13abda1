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

// Column sums, in a fixed order. A cluster of CTAs takes 64 columns (128
// bytes of a row, so that every row's piece is whole sectors), each CTA a run
// of rows; within a CTA a thread takes VEC neighbouring columns of every
// 256·VEC/64-th row, kUnroll rows in flight, then the threads of a column are
// added in order through shared memory, and the CTAs in rank order through
// distributed shared memory by rank 0. Bound by reading dY once.
constexpr int kSumCols = 64;
constexpr int kUnroll = 8;
template <int VEC>
__global__ void __launch_bounds__(256)
    column_sums_kernel(const uint16_t* __restrict__ dy, int64_t ld, int64_t M, int64_t N, float* __restrict__ out,
                       int accumulate, int cluster) {
  constexpr int ACROSS = kSumCols / VEC;  // threads across the columns
  constexpr int DOWN = 256 / ACROSS;      // threads down the rows
  __shared__ float s[DOWN][kSumCols + 1];
  __shared__ float part[kSumCols + 2];
  grid_dependency_wait();
  grid_launch_dependents();
  const int rank = static_cast<int>(blockIdx.x) % cluster;
  const int c = threadIdx.x % ACROSS * VEC, r = threadIdx.x / ACROSS;
  const int64_t n = static_cast<int64_t>(blockIdx.x) / cluster * kSumCols + c;
  const int64_t m0 = M * rank / cluster, m1 = M * (rank + 1) / cluster;
  float sum[VEC] = {};
  if (n < N) {
    for (int64_t m = m0 + r; m < m1; m += DOWN * kUnroll) {
      uint16_t v[kUnroll][VEC];
#pragma unroll
      for (int k = 0; k < kUnroll; ++k) {
        const int64_t row = m + k * DOWN;
        if constexpr (VEC == 8)
          *reinterpret_cast<uint4*>(v[k]) =
              row < m1 ? __ldg(reinterpret_cast<const uint4*>(dy + row * ld + n)) : make_uint4(0u, 0u, 0u, 0u);
        else
          v[k][0] = row < m1 ? __ldg(dy + row * ld + n) : static_cast<uint16_t>(0);
      }
#pragma unroll
      for (int k = 0; k < kUnroll; ++k)
#pragma unroll
        for (int i = 0; i < VEC; ++i) sum[i] += __half2float(__ushort_as_half(v[k][i]));
    }
  }
#pragma unroll
  for (int i = 0; i < VEC; ++i) s[r][c + i] = sum[i];
  __syncthreads();
  float total = 0.f;
  if (threadIdx.x < kSumCols) {
#pragma unroll
    for (int i = 0; i < DOWN; ++i) total += s[i][threadIdx.x];
    part[threadIdx.x] = total;
  }
  if (cluster > 1) {
    cluster_sync();
    if (rank == 0 && threadIdx.x < kSumCols)
      for (int i = 1; i < cluster; ++i)
        total += ld_cluster_f32(mapa_shared(smem_u32(&part[threadIdx.x]), static_cast<uint32_t>(i)));
    cluster_sync();  // the other ranks' shared memory stays until rank 0 has read it
  }
  const int64_t col = static_cast<int64_t>(blockIdx.x) / cluster * kSumCols + threadIdx.x;
  if (rank == 0 && threadIdx.x < kSumCols && col < N) out[col] = accumulate ? out[col] + total : total;
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
  const bool vec = N % 8 == 0 && ld % 8 == 0 && (reinterpret_cast<uintptr_t>(dy) & 15u) == 0;
  // up to 8 CTAs (the portable cluster size) per 64 columns, 256 rows or more each
  int cluster = 1;
  while (cluster < 8 && M >= 512 * cluster) cluster *= 2;
  const int64_t blocks = (N + kSumCols - 1) / kSumCols * cluster;
  if (blocks > 0x7FFFFFFF) return cudaErrorInvalidValue;
  PdlLaunch l(dim3(static_cast<unsigned>(blocks)), dim3(256), 0, stream);
  l.cluster(static_cast<unsigned>(cluster));
  return cudaLaunchKernelEx(&l.cfg, vec ? column_sums_kernel<8> : column_sums_kernel<1>, dy, ld, M, N, out,
                            accumulate ? 1 : 0, cluster);
}

// The -DHGEMM_DEBUG build's check word of this file (null otherwise).
HG_DEBUG_WORD_ACCESSOR(linear)

}  // namespace hg
