// hgemm_ckpt8.cu — a matrix into its 8-bit form and back (hgemm_ckpt8_save,
// hgemm_ckpt8_load; the form is defined in hgemm.h).
//
// Both are bound by memory: 2 bytes read and 1.06 written per value, or the
// other way round (16384×8192: saved in 73 us, 5.7 TB/s, loaded in 60, 6.8 TB/s, and
// with GELU in 63; a copy moves 6.8 TB/s; 16384×8191, one or two bytes at a time,
// 175 and 109). A warp takes 8 rows of a few groups at once, so that it has
// eight independent loads in flight per lane and so that the scales of 8 rows,
// neighbours in memory, form one 32-byte sector per group.
#include "debug.cuh"
#include "linear_epilogue.cuh"
#include "ptx.cuh"

namespace hg {
namespace {

constexpr int kRows = 8;      // rows of a warp's piece
constexpr int kVecCols = 256;  // its columns, eight per lane: four groups of eight lanes

// A warp's piece: rows [m0, m0 + 8), columns from n0.
struct Piece {
  int64_t m0, n0;
};

// Pieces are numbered along the columns first, so that neighbouring warps
// read neighbouring memory.
__device__ __forceinline__ bool piece_of(int64_t M, int64_t N, int cols, Piece& p) {
  const int64_t per_row = (N + cols - 1) / cols;
  const int64_t t = static_cast<int64_t>(blockIdx.x) * (blockDim.x >> 5) + (threadIdx.x >> 5);
  p.m0 = t / per_row * kRows;
  p.n0 = t % per_row * cols;
  return p.m0 < M;
}

// N, the pitches and the bases let eight columns be moved at once.
__global__ void __launch_bounds__(256)
    ckpt8_save_vec_kernel(const uint16_t* x, int64_t ldx, int8_t* codes, int64_t ldq,
                          float* scales, int64_t lds, int64_t M, int64_t N) {
  grid_dependency_wait();
  grid_launch_dependents();
  Piece p;
  if (!piece_of(M, N, kVecCols, p)) return;
  const int lane = threadIdx.x & 31;
  const int64_t n = p.n0 + 8 * lane;
  const bool in_n = n < N;
  uint4 v[kRows];
#pragma unroll
  for (int r = 0; r < kRows; ++r)
    v[r] = in_n && p.m0 + r < M && dbg_row(x + (p.m0 + r) * ldx + n, n, 8, N, 16) ? load16(x + (p.m0 + r) * ldx + n)
                                                                                  : make_uint4(0u, 0u, 0u, 0u);
  float mine = 0.f;  // lane 8g + r keeps the scale of group g, row r
#pragma unroll
  for (int r = 0; r < kRows; ++r) {
    const f32x2 u[4] = {unpack_half2(v[r].x), unpack_half2(v[r].y), unpack_half2(v[r].z), unpack_half2(v[r].w)};
    float top = 0.f;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      float a, b;
      unpair(u[i], a, b);
      top = max_abs3(top, a, b);
    }
    uint32_t bits = magnitude_bits(top);
#pragma unroll
    for (int o = 4; o > 0; o >>= 1) bits = max(bits, __shfl_xor_sync(0xffffffffu, bits, o));
    float scale, inv;
    ckpt_scale(bits, scale, inv);
    if ((lane & 7) == r) mine = scale;
    if (in_n && p.m0 + r < M && dbg_row(codes + (p.m0 + r) * ldq + n, n, 8, N, 8))
      *reinterpret_cast<uint2*>(codes + (p.m0 + r) * ldq + n) =
          make_uint2(ckpt_word(u[0], u[1], inv), ckpt_word(u[2], u[3], inv));
  }
  const int64_t m = p.m0 + (lane & 7);
  const int64_t g = n / kCkptGroup;  // (its last lanes may be past N)
  if (g * kCkptGroup < N && m < M && HG_DBG_INDEX(m, lds)) scales[g * lds + m] = mine;
}

// Any pitch and alignment: one group per warp, two columns per lane.
__global__ void __launch_bounds__(256)
    ckpt8_save_kernel(const uint16_t* x, int64_t ldx, int8_t* codes, int64_t ldq,
                      float* scales, int64_t lds, int64_t M, int64_t N) {
  grid_dependency_wait();
  grid_launch_dependents();
  Piece p;
  if (!piece_of(M, N, kCkptGroup, p)) return;
  const int lane = threadIdx.x & 31;
  float u[kRows][2];
#pragma unroll
  for (int r = 0; r < kRows; ++r)
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      const int64_t n = p.n0 + lane + 32 * i;
      u[r][i] = n < N && p.m0 + r < M ? __half2float(__ushort_as_half(x[(p.m0 + r) * ldx + n])) : 0.f;
    }
  float mine = 0.f;
#pragma unroll
  for (int r = 0; r < kRows; ++r) {
    float scale, inv;
    ckpt_scale(__reduce_max_sync(0xffffffffu, max(magnitude_bits(u[r][0]), magnitude_bits(u[r][1]))), scale, inv);
    if (lane == r) mine = scale;
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      const int64_t n = p.n0 + lane + 32 * i;
      if (n < N && p.m0 + r < M)
        codes[(p.m0 + r) * ldq + n] = static_cast<int8_t>(inv == 0.f ? 0u : ckpt_code(u[r][i], inv));
    }
  }
  if (lane < kRows && p.m0 + lane < M && HG_DBG_INDEX(p.n0, N) && HG_DBG_INDEX(p.m0 + lane, lds))
    scales[p.n0 / kCkptGroup * lds + p.m0 + lane] = mine;
}

__global__ void __launch_bounds__(256)
    ckpt8_load_vec_kernel(const int8_t* codes, int64_t ldq, const float* scales,
                          int64_t lds, int act, uint16_t* __restrict__ y, int64_t ldy, int64_t M, int64_t N) {
  grid_dependency_wait();
  grid_launch_dependents();
  Piece p;
  if (!piece_of(M, N, kVecCols, p)) return;
  const int lane = threadIdx.x & 31;
  const int64_t n = p.n0 + 8 * lane;
  const bool in_n = n < N;
  uint2 w[kRows];
#pragma unroll
  for (int r = 0; r < kRows; ++r)
    w[r] = in_n && p.m0 + r < M && dbg_row(codes + (p.m0 + r) * ldq + n, n, 8, N, 8)
               ? load8(codes + (p.m0 + r) * ldq + n)
               : make_uint2(0u, 0u);
  const int64_t m = p.m0 + (lane & 7);
  const int64_t g = n / kCkptGroup;  // (its last lanes may be past N)
  const float mine = g * kCkptGroup < N && m < M && HG_DBG_INDEX(m, lds) ? scales[g * lds + m] : 0.f;
  with_activation(act, [&](auto a) {
#pragma unroll
    for (int r = 0; r < kRows; ++r) {
      const float scale = __shfl_sync(0xffffffffu, mine, (lane & 24) | r);
      f32x2 f[4], df;
#pragma unroll
      for (int i = 0; i < 4; ++i)
        activate<decltype(a)::value, false>(
            mul2(ckpt_pair((i < 2 ? w[r].x : w[r].y) ^ 0x80808080u, i & 1), pair_of(scale)), f[i], df);
      if (in_n && p.m0 + r < M && dbg_row(y + (p.m0 + r) * ldy + n, n, 8, N, 16))
        *reinterpret_cast<uint4*>(y + (p.m0 + r) * ldy + n) = pack8(f);
    }
  });
}

__global__ void __launch_bounds__(256)
    ckpt8_load_kernel(const int8_t* codes, int64_t ldq, const float* scales, int64_t lds,
                      int act, uint16_t* y, int64_t ldy, int64_t M, int64_t N) {
  grid_dependency_wait();
  grid_launch_dependents();
  Piece p;
  if (!piece_of(M, N, kCkptGroup, p)) return;
  const int lane = threadIdx.x & 31;
  int8_t c[kRows][2];
#pragma unroll
  for (int r = 0; r < kRows; ++r)
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      const int64_t n = p.n0 + lane + 32 * i;
      c[r][i] = n < N && p.m0 + r < M ? codes[(p.m0 + r) * ldq + n] : static_cast<int8_t>(0);
    }
  const int64_t m = p.m0 + (lane & 7);
  const float mine = m < M && HG_DBG_INDEX(p.n0, N) && HG_DBG_INDEX(m, lds) ? scales[p.n0 / kCkptGroup * lds + m] : 0.f;
#pragma unroll
  for (int r = 0; r < kRows; ++r) {
    const float scale = __shfl_sync(0xffffffffu, mine, r);
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      const int64_t n = p.n0 + lane + 32 * i;
      if (n < N && p.m0 + r < M)
        y[(p.m0 + r) * ldy + n] =
            __half_as_ushort(__float2half_rn(activate(static_cast<float>(c[r][i]) * scale, act)));
    }
  }
}

bool aligned(const void* p, int64_t ld, uintptr_t bytes) {
  return (reinterpret_cast<uintptr_t>(p) & (bytes - 1)) == 0 && ld % 8 == 0;
}

// Blocks of eight warps over the pieces; 0: more than a grid holds.
unsigned pieces_grid(int64_t M, int64_t N, int cols) {
  const int64_t pieces = ((M + kRows - 1) / kRows) * ((N + cols - 1) / cols);
  const int64_t blocks = (pieces + 7) / 8;
  return blocks > 0x7FFFFFFF ? 0u : static_cast<unsigned>(blocks);
}

}  // namespace

cudaError_t launch_ckpt8_save(const uint16_t* x, int64_t ldx, int8_t* codes, int64_t ldq, float* scales,
                              int64_t lds, int64_t M, int64_t N, cudaStream_t stream) {
  const bool vec = N % 8 == 0 && aligned(x, ldx, 16) && aligned(codes, ldq, 8);
  const unsigned grid = pieces_grid(M, N, vec ? kVecCols : kCkptGroup);
  if (grid == 0) return cudaErrorInvalidValue;
  PdlLaunch l(dim3(grid), dim3(256), 0, stream);
  return cudaLaunchKernelEx(&l.cfg, vec ? ckpt8_save_vec_kernel : ckpt8_save_kernel, x, ldx, codes, ldq, scales, lds,
                            M, N);
}

cudaError_t launch_ckpt8_load(const int8_t* codes, int64_t ldq, const float* scales, int64_t lds, int act,
                              uint16_t* y, int64_t ldy, int64_t M, int64_t N, cudaStream_t stream) {
  const bool vec = N % 8 == 0 && aligned(y, ldy, 16) && aligned(codes, ldq, 8);
  const unsigned grid = pieces_grid(M, N, vec ? kVecCols : kCkptGroup);
  if (grid == 0) return cudaErrorInvalidValue;
  PdlLaunch l(dim3(grid), dim3(256), 0, stream);
  return cudaLaunchKernelEx(&l.cfg, vec ? ckpt8_load_vec_kernel : ckpt8_load_kernel, codes, ldq, scales, lds, act, y,
                            ldy, M, N);
}

// The -DHGEMM_DEBUG build's check word of this file (null otherwise).
HG_DEBUG_WORD_ACCESSOR(ckpt8)

}  // namespace hg
