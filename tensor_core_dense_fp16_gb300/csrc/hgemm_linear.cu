// hgemm_linear.cu — the parts of linear layers (hgemm_linear and its
// gradients) that are no large products: these run on the product kernels
// with the epilogues of linear_epilogue.cuh.
#include "debug.cuh"
#include "linear_epilogue.cuh"
#include "linear_rows.h"
#include "ptx.cuh"

namespace hg {
namespace {

// The epilogue of empty sums: one warp per row and group of 64 columns, two
// columns per lane.
template <bool BACKWARD>
__global__ void __launch_bounds__(256)
    linear_empty_kernel(uint16_t* C, int64_t ldc, int64_t M, int64_t N, const LinEpi e) {
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
      if (n < N && HG_DBG_INDEX(m, M)) lin_scalar<BACKWARD>(e, u[i], m, n, scale, inv, C + m * ldc + n);
    }
  }
}

// ------------------------------------------------------------ few rows of X

// D (16×8, FP32) += A (16×16) · B (16×8).
__device__ __forceinline__ void mma_16816(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3,
                                          uint32_t b0, uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, "
      "{%0, %1, %2, %3};"
      : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

// Y for at most 8·MT rows of X (a step of token generation), bound by reading
// W once. A block takes 16 features, its warps interleaved 32-wide pieces of
// K. Weights go from memory straight into the fragments of a 16×8×16 matrix
// instruction with the features as its rows and the rows of X as its columns:
// a sum does not depend on which k stands in which slot, so lane 4g + t takes
// the 16 contiguous bytes at k = 8t of a piece (of features g and g + 8, and
// of row g of X), which are its slots of two instructions, and nothing passes
// through shared memory. One row of X costs as much as eight. The warps'
// partial sums are added in order through shared memory. One row, us and the
// rate at which weights arrive: 8192×8192 22.2, 6.0 TB/s, 89% of a copy's;
// 8192×2048 7.3, 4.6 TB/s, the rest launch, first read and sums; one launch
// after another. VEC: pitches and
// bases allow the 16-byte loads; otherwise the slots are filled by 2-byte
// loads.
struct RowsArgs {
  const uint16_t* X;
  int64_t ldx;
  const uint16_t* W;
  int64_t ldw;
  uint16_t* Y;
  int64_t ldy;
  int M, N, K;
  LinEpi epi;
};

template <int MT, int WARPS, bool VEC>
__global__ void __launch_bounds__(WARPS * 32) linear_rows_kernel(const RowsArgs p) {
  constexpr int AHEAD = MT == 1 ? kRowsAhead : 2;  // pieces in flight per warp, 64 bytes of each feature
  static_assert(WARPS <= kRowsWarps, "the walk along K fits");
  constexpr int PITCH = kRowsFeatures + 1;
  __shared__ float part[WARPS][8 * MT][PITCH];
  // The first weights, four lines per thread, into L2 while the previous launch
  // on the stream ends (only asked for: whatever it still writes there is read
  // after the wait). A token through 2048→8192→2048, two launches: 16.4 us
  // without, 14.4 with.
  const int lines = rows_lines(p.K);
  for (int i = threadIdx.x; i < kRowsFeatures * lines && i < 4 * WARPS * 32; i += WARPS * 32) {
    const int f = static_cast<int>(blockIdx.x) * kRowsFeatures + i / lines;
    if (f < p.N) prefetch_l2(p.W + f * p.ldw + static_cast<int64_t>(i % lines) * 64);
  }
  grid_dependency_wait();
  grid_launch_dependents();
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int g = lane >> 2, t = lane & 3;
  const int n0 = static_cast<int>(blockIdx.x) * kRowsFeatures;
  // features past N are computed as copies of the last one and not stored
  const uint16_t* w0 = p.W + static_cast<int64_t>(min(n0 + g, p.N - 1)) * p.ldw;
  const uint16_t* w1 = p.W + static_cast<int64_t>(min(n0 + g + 8, p.N - 1)) * p.ldw;
  auto load = [&](const uint16_t* row, RowsK k, bool weights) {
    if constexpr (VEC) {
      if (!rows_inside(k, p.K) || !dbg_row(row + k, k, 8, p.K, 16)) return make_uint4(0u, 0u, 0u, 0u);
      return weights ? load16_once(row + k) : load16(row + k);  // (L1 keeps X)
    } else {
      uint32_t v[4];
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const uint32_t lo = rows_inside(k + 2 * i, p.K) ? row[k + 2 * i] : 0u;
        const uint32_t hi = rows_inside(k + 2 * i + 1, p.K) ? row[k + 2 * i + 1] : 0u;
        v[i] = lo | hi << 16;
      }
      return make_uint4(v[0], v[1], v[2], v[3]);
    }
  };
  float acc[MT][4] = {};
  // AHEAD pieces in turn: as soon as one has been multiplied, its registers
  // take the piece AHEAD further on
  uint4 a0[AHEAD], a1[AHEAD], b[AHEAD][MT];
  auto fetch = [&](int u, RowsK k) {
    a0[u] = load(w0, k, true);
    a1[u] = load(w1, k, true);
#pragma unroll
    for (int i = 0; i < MT; ++i) {
      const int m = 8 * i + g;
      b[u][i] = m < p.M ? load(p.X + m * p.ldx, k, false) : make_uint4(0u, 0u, 0u, 0u);
    }
  };
  RowsK k0 = rows_begin(warp, t);
#pragma unroll
  for (int u = 0; u < AHEAD; ++u) fetch(u, rows_on(k0, u, WARPS));
  for (; rows_inside(k0 - 8 * t, p.K); k0 = rows_on(k0, AHEAD, WARPS)) {
#pragma unroll
    for (int u = 0; u < AHEAD; ++u) {
#pragma unroll
      for (int i = 0; i < MT; ++i) {
        mma_16816(acc[i], a0[u].x, a1[u].x, a0[u].y, a1[u].y, b[u][i].x, b[u][i].y);
        mma_16816(acc[i], a0[u].z, a1[u].z, a0[u].w, a1[u].w, b[u][i].z, b[u][i].w);
      }
      fetch(u, rows_on(k0, AHEAD + u, WARPS));
    }
  }
#pragma unroll
  for (int i = 0; i < MT; ++i) {
    part[warp][8 * i + 2 * t][g] = acc[i][0];
    part[warp][8 * i + 2 * t + 1][g] = acc[i][1];
    part[warp][8 * i + 2 * t][g + 8] = acc[i][2];
    part[warp][8 * i + 2 * t + 1][g + 8] = acc[i][3];
  }
  __syncthreads();
  for (int i = threadIdx.x; i < p.M * kRowsFeatures; i += WARPS * 32) {
    const int m = i / kRowsFeatures, f = i % kRowsFeatures;
    if (n0 + f >= p.N) continue;
    float u = part[0][m][f];
#pragma unroll
    for (int w = 1; w < WARPS; ++w) u += part[w][m][f];
    if (p.epi.bias) u += __half2float(__ushort_as_half(p.epi.bias[n0 + f]));
    if (HG_DBG_INDEX(n0 + f, p.N) && HG_DBG_INDEX(m, p.M))
      lin_scalar<false>(p.epi, u, m, n0 + f, 0.f, 0.f, p.Y + m * p.ldy + n0 + f);
  }
}

template <int MT, int WARPS>
cudaError_t rows_with(const RowsArgs& p, bool vec, cudaStream_t stream) {
  PdlLaunch l(dim3(static_cast<unsigned>(rows_blocks(p.N))), dim3(WARPS * 32), 0, stream);
  return cudaLaunchKernelEx(&l.cfg, vec ? linear_rows_kernel<MT, WARPS, true> : linear_rows_kernel<MT, WARPS, false>,
                            p);
}

template <int MT>
cudaError_t rows_tiles(const RowsArgs& p, bool vec, cudaStream_t stream) {
  // About 2048 warps in all, 13 per SM: enough loads under way, and all
  // blocks resident at once; four pieces or more per warp. One row, us with 4,
  // 8 and 16 warps: 8192×2048 7.3, 7.7, 11.3; 4096×4096 9.5, 6.6, 8.5; 2048×8192
  // 14.9, 9.9, 7.4; 1024×1024 2.4, 2.1, 2.3.
  const int64_t blocks = rows_blocks(p.N), pieces = rows_pieces(p.K);
  if (blocks >= 384 || pieces < 32) return rows_with<MT, 4>(p, vec, stream);
  if (blocks >= 192 || pieces < 64) return rows_with<MT, 8>(p, vec, stream);
  return rows_with<MT, 16>(p, vec, stream);
}

// Column sums, in a fixed order. A cluster of CTAs takes a strip of columns,
// each CTA a run of rows; within a CTA `across` threads lie along a row, VEC
// neighbouring columns each, the others down the rows, kUnroll rows in
// flight per thread. The threads of a column are added in order through
// shared memory, and the CTAs in rank order through distributed shared memory
// by rank 0. Bound by reading dY once (8192×8192 26.0 us, 5.2 TB/s; 8192×1001,
// two bytes at a time, 16.1); a strip is as wide as leaves enough CTAs, because
// the longer a row's piece the better memory delivers it.
//
// beside: the launch before this one on the stream is the product with the
// same dY, and the two may run at the same time, the sums on SMs that the
// product leaves idle. Nothing here depends on that product, and what it
// waited for is complete (it lets this launch start only after its own
// wait), so the sums need not wait, and read dY and the old sums from L2
// behind a fence; but the first block ends only after the product has, so
// that whoever waits for this launch waits for both.
constexpr int kSumThreads = 512;
constexpr int kUnroll = 8;
template <int VEC>
__global__ void __launch_bounds__(kSumThreads)
    column_sums_kernel(const uint16_t* dy, int64_t ld, int64_t M, int64_t N, float* out,
                       int accumulate, int across, int cluster, int beside) {
  __shared__ float s[kSumThreads * VEC];  // [down][columns]
  if (beside) {
    fence_gpu();
  } else {
    grid_dependency_wait();
    grid_launch_dependents();
  }
  const int columns = across * VEC, down = kSumThreads / across;
  const int rank = static_cast<int>(blockIdx.x) % cluster;
  const int c = threadIdx.x % across * VEC, r = threadIdx.x / across;
  const int64_t n0 = static_cast<int64_t>(blockIdx.x) / cluster * columns;
  const int64_t m1 = M * (rank + 1) / cluster;
  float sum[VEC] = {};
  if (n0 + c < N) {
    for (int64_t m = M * rank / cluster + r; m < m1; m += down * kUnroll) {
      uint16_t v[kUnroll][VEC];
#pragma unroll
      for (int k = 0; k < kUnroll; ++k) {
        const int64_t row = m + k * down;
        if constexpr (VEC == 8)
          *reinterpret_cast<uint4*>(v[k]) = row < m1 && dbg_row(dy + row * ld + n0 + c, n0 + c, 8, N, 16)
                                                ? ld_gpu_16(dy + row * ld + n0 + c)
                                                : make_uint4(0u, 0u, 0u, 0u);
        else
          v[k][0] = row < m1 && dbg_row(dy, n0 + c, 1, N, 2) ? ld_gpu_u16(dy + row * ld + n0 + c) : static_cast<uint16_t>(0);
      }
#pragma unroll
      for (int k = 0; k < kUnroll; ++k)
#pragma unroll
        for (int i = 0; i < VEC; ++i) sum[i] += __half2float(__ushort_as_half(v[k][i]));
    }
  }
#pragma unroll
  for (int i = 0; i < VEC; ++i) s[r * columns + c + i] = sum[i];
  __syncthreads();
  float total = 0.f;
  const bool mine = static_cast<int>(threadIdx.x) < columns;
  if (mine) {
    for (int i = 0; i < down; ++i) total += s[i * columns + threadIdx.x];
    s[threadIdx.x] = total;  // (only this thread reads its column)
  }
  if (cluster > 1) {
    cluster_sync();
    if (rank == 0 && mine)
      for (int i = 1; i < cluster; ++i)
        total += ld_cluster_f32(mapa_shared(smem_u32(&s[threadIdx.x]), static_cast<uint32_t>(i)));
    cluster_sync();  // the other ranks' shared memory stays until rank 0 has read it
  }
  const int64_t n = n0 + threadIdx.x;
  if (rank == 0 && mine && n < N) out[n] = accumulate ? ld_gpu_f32(out + n) + total : total;
  if (beside && blockIdx.x == 0) grid_dependency_wait();
}

// The same beside a product that fills every SM: blocks small enough for what
// the pair and wide kernels leave of an SM (1.8 KB of shared memory with the
// block's own 1 KB, registers for 256 threads of 64), so they read dY while
// the product, bound by the matrix instructions, runs. A block takes 64 columns
// (8 lanes along a row, 16 bytes each, 32 rows at a time) of a run of rows; its
// cluster adds the runs in rank order. With the product, which alone takes the
// first time, us, and with the wide blocks above: dY 8192×8192, X 8192×2048
// 155, 160, 180; 4096×8192, 8192×2048 87, 89, 93; 2048 all 14.6, 16.1, 20.3;
// but 8192×2048, 8192×8192 163, 166, 164.
constexpr int kThinColumns = 64;
constexpr int kThinThreads = 256;
__global__ void __launch_bounds__(kThinThreads)
    column_sums_thin_kernel(const uint16_t* dy, int64_t ld, int64_t M, int64_t N, float* out, int accumulate,
                            int cluster) {
  fence_gpu();
  __shared__ float s[3][kThinColumns];
  constexpr int WARPS = kThinThreads / 32, STEP = 4 * WARPS;  // rows per step
  const int rank = static_cast<int>(blockIdx.x) % cluster;
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int64_t n0 = static_cast<int64_t>(blockIdx.x) / cluster * kThinColumns, n = n0 + 8 * (lane & 7);
  const int64_t m1 = M * (rank + 1) / cluster;
  f32x2 sum[4] = {};
  if (n < N) {
    const uint16_t* p = dy + n;
    for (int64_t m = M * rank / cluster + warp * 4 + (lane >> 3); m < m1; m += STEP * kUnroll) {
      uint4 v[kUnroll];
#pragma unroll
      for (int k = 0; k < kUnroll; ++k)
        v[k] = m + k * STEP < m1 && dbg_row(p + (m + k * STEP) * ld, n, 8, N, 16) ? ld_gpu_16(p + (m + k * STEP) * ld)
                                                                                  : make_uint4(0u, 0u, 0u, 0u);
#pragma unroll
      for (int k = 0; k < kUnroll; ++k) add8(sum, v[k]);
    }
  }
  float v[8];
#pragma unroll
  for (int i = 0; i < 4; ++i) unpair(sum[i], v[2 * i], v[2 * i + 1]);
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    v[i] += __shfl_xor_sync(0xffffffffu, v[i], 8);
    v[i] += __shfl_xor_sync(0xffffffffu, v[i], 16);
  }
  // warp 0 adds the others' in order, three at a time
#pragma unroll
  for (int w0 = 1; w0 < WARPS; w0 += 3) {
    if (w0 > 1) __syncthreads();
#pragma unroll
    for (int i = 0; i < 8; ++i)
      if (warp >= w0 && warp < w0 + 3 && lane < 8) s[warp - w0][8 * lane + i] = v[i];
    __syncthreads();
#pragma unroll
    for (int w = w0; w < w0 + 3 && w < WARPS; ++w)
#pragma unroll
      for (int i = 0; i < 8; ++i)
        if (warp == 0 && lane < 8) v[i] += s[w - w0][8 * lane + i];
  }
  if (warp == 0 && lane < 8) {
#pragma unroll
    for (int i = 0; i < 8; ++i) s[0][8 * lane + i] = v[i];
  }
  cluster_sync();
  if (rank == 0 && threadIdx.x < kThinColumns && n0 + threadIdx.x < N) {
    float total = s[0][threadIdx.x];
    for (int i = 1; i < cluster; ++i)
      total += ld_cluster_f32(mapa_shared(smem_u32(&s[0][threadIdx.x]), static_cast<uint32_t>(i)));
    float* o = out + n0 + threadIdx.x;
    *o = accumulate ? ld_gpu_f32(o) + total : total;
  }
  cluster_sync();  // the other ranks' shared memory stays until rank 0 has read it
  if (blockIdx.x == 0) grid_dependency_wait();
}

}  // namespace

bool linear_rows_suits(const LinearProduct& p) {
  return p.M <= kLinearRows && p.K > 0 && !p.b_mn && !p.epi.backward && !p.epi.codes;
}

cudaError_t launch_linear_rows(const LinearProduct& q, cudaStream_t stream) {
  const RowsArgs p{q.A, q.lda, q.B, q.ldb, q.C, q.ldc, static_cast<int>(q.M), static_cast<int>(q.N),
                   static_cast<int>(q.K), q.epi};
  auto rows16 = [](const void* b, int64_t ld) { return (reinterpret_cast<uintptr_t>(b) & 15u) == 0 && ld % 8 == 0; };
  const bool vec = q.K % 8 == 0 && rows16(q.A, q.lda) && rows16(q.B, q.ldb);
  switch ((q.M + 7) / 8) {
    case 1:
      return rows_tiles<1>(p, vec, stream);
    case 2:
      return rows_tiles<2>(p, vec, stream);
    case 3:
      return rows_tiles<3>(p, vec, stream);
    default:
      return rows_tiles<4>(p, vec, stream);
  }
}

cudaError_t launch_linear_empty(uint16_t* C, int64_t ldc, int64_t M, int64_t N, const LinEpi& epi,
                                cudaStream_t stream) {
  const int64_t blocks = (M * ((N + kCkptGroup - 1) / kCkptGroup) + 7) / 8;
  PdlLaunch l(dim3(static_cast<unsigned>(blocks < 4096 ? blocks : 4096)), dim3(256), 0, stream);
  return cudaLaunchKernelEx(&l.cfg, epi.backward ? linear_empty_kernel<true> : linear_empty_kernel<false>, C, ldc, M,
                            N, epi);
}

cudaError_t launch_column_sums(const uint16_t* dy, int64_t ld, int64_t M, int64_t N, float* out, bool accumulate,
                               bool beside, bool thin, cudaStream_t stream) {
  const bool vec = N % 8 == 0 && ld % 8 == 0 && (reinterpret_cast<uintptr_t>(dy) & 15u) == 0;
  if (beside && vec && thin) {
    int runs = 1;
    while (runs < 8 && M >= 256 * runs) runs *= 2;
    const int64_t grid = (N + kThinColumns - 1) / kThinColumns * runs;
    if (grid > 0x7FFFFFFF) return cudaErrorInvalidValue;
    PdlLaunch l(dim3(static_cast<unsigned>(grid)), dim3(kThinThreads), 0, stream);
    l.cluster(static_cast<unsigned>(runs));
    return cudaLaunchKernelEx(&l.cfg, column_sums_thin_kernel, dy, ld, M, N, out, accumulate ? 1 : 0, runs);
  }
  const int vec_cols = vec ? 8 : 1;
  // up to 8 CTAs (the portable cluster size) per strip, 128 rows or more each
  int cluster = 1;
  while (cluster < 8 && M >= 256 * cluster) cluster *= 2;
  // from 512 bytes of a row down to 64, while a strip's CTAs are fewer than
  // would fill most of the GPU
  int across = vec ? 32 : 256;
  auto blocks = [&] { return (N + across * vec_cols - 1) / (across * vec_cols) * cluster; };
  while (across > (vec ? 4 : 32) && blocks() < 128) across /= 2;
  if (blocks() > 0x7FFFFFFF) return cudaErrorInvalidValue;
  PdlLaunch l(dim3(static_cast<unsigned>(blocks())), dim3(kSumThreads), 0, stream);
  l.cluster(static_cast<unsigned>(cluster));
  return cudaLaunchKernelEx(&l.cfg, vec ? column_sums_kernel<8> : column_sums_kernel<1>, dy, ld, M, N, out,
                            accumulate ? 1 : 0, across, cluster, beside ? 1 : 0);
}

// The -DHGEMM_DEBUG build's check word of this file (null otherwise).
HG_DEBUG_WORD_ACCESSOR(linear)

}  // namespace hg
