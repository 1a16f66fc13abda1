// hgemm_norm.cu — layer norm over rows, forward and backward (the formulas
// are in hgemm.h). Both are bound by memory: forward reads and writes 2
// bytes per value, backward reads 4 (6 with the residual branch) and writes 2.
// 16384 rows of 8192: forward 85 us, 6.3 TB/s, backward with the residual
// branch 174 us, 6.2 TB/s, 93 and 91% of a copy's rate; of 4096 43 and 83; of
// 1024 (32768 rows) 23 and 47, 85%. Rows that 16-byte accesses cannot describe
// (16384 of 5001: 216 and 455 us) move two bytes at a time and are bound by the
// number of those accesses.
#include <atomic>

#include <cuda_fp16.h>

#include "debug.cuh"
#include "internal.h"
#include "kernel_common.cuh"
#include "linear_epilogue.cuh"
#include "ptx.cuh"

namespace hg {
namespace {

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

// ------------------------------------------------------------------ forward

// G threads per row, which they hold in registers (8·NV values each): the
// mean, the variance around it, the output; one read and one write. VEC: the
// row in 16-byte pieces; otherwise value by value, neighbouring threads on
// neighbouring values. Blocks of max(G, 128) threads.
template <int G, int NV, bool VEC>
__global__ void __launch_bounds__(G < 128 ? 128 : G) layernorm_forward_kernel(const NormArgs a) {
  constexpr int THREADS = G < 128 ? 128 : G;
  __shared__ float s[THREADS / 32];
  const int t = threadIdx.x % G;
  const int64_t m = static_cast<int64_t>(blockIdx.x) * (THREADS / G) + threadIdx.x / G;
  const int D = static_cast<int>(a.D);
  // the column of value k of piece i
  auto col = [&](int i, int k) { return VEC ? (t + i * G) * 8 + k : (i * 8 + k) * G + t; };
  auto load = [&](const uint16_t* p, int i, float (&f)[8]) {
    if constexpr (VEC) {
      unpack8(col(i, 0) < D && dbg_row(p + col(i, 0), col(i, 0), 8, D, 16)
                  ? *reinterpret_cast<const uint4*>(p + col(i, 0))
                  : make_uint4(0u, 0u, 0u, 0u),
              f);
    } else {
#pragma unroll
      for (int k = 0; k < 8; ++k) f[k] = col(i, k) < D ? half_at(p, col(i, k)) : 0.f;
    }
  };
  grid_dependency_wait();
  grid_launch_dependents();
  if (G < 128 && m >= a.M) return;  // whole warps; larger groups have a block of their own
  float x[NV][8];
  float sum = 0.f;
#pragma unroll
  for (int i = 0; i < NV; ++i) load(a.x + m * a.ldx, i, x[i]);
#pragma unroll
  for (int i = 0; i < NV; ++i)
#pragma unroll
    for (int k = 0; k < 8; ++k) sum += x[i][k];
  const float mu = group_sum<G>(sum, s) / static_cast<float>(D);
  float sq = 0.f;
#pragma unroll
  for (int i = 0; i < NV; ++i)
#pragma unroll
    for (int k = 0; k < 8; ++k) {
      const float v = x[i][k] - mu;
      if (col(i, k) < D) sq = fmaf(v, v, sq);
    }
  const float rs = rsqrtf(group_sum<G>(sq, s) / static_cast<float>(D) + a.eps);
#pragma unroll
  for (int i = 0; i < NV; ++i) {
    float g[8], b[8];
    load(a.gamma, i, g);
    load(a.beta, i, b);
#pragma unroll
    for (int k = 0; k < 8; ++k) g[k] = fmaf((x[i][k] - mu) * rs, g[k], b[k]);
    uint16_t* y = a.y + m * a.ldy;
    if constexpr (VEC) {
      if (col(i, 0) < D && dbg_row(y + col(i, 0), col(i, 0), 8, D, 16))
        *reinterpret_cast<uint4*>(y + col(i, 0)) = pack8f(g);
    } else {
#pragma unroll
      for (int k = 0; k < 8; ++k)
        if (col(i, k) < D) y[col(i, k)] = __half_as_ushort(__float2half_rn(g[k]));
    }
  }
  if (t == 0 && a.mean && HG_DBG_INDEX(m, a.M)) {
    a.mean[m] = mu;
    a.rstd[m] = rs;
  }
}

constexpr int kThreads = 256;

// Rows too long for registers: a block per row, which it reads three times
// (from L1 or L2 after the first).
__global__ void __launch_bounds__(kThreads) layernorm_forward_long_kernel(const NormArgs a) {
  __shared__ float s[kThreads / 32];
  grid_dependency_wait();
  grid_launch_dependents();
  for (int64_t m = blockIdx.x; m < a.M; m += gridDim.x) {
    const uint16_t* x = a.x + m * a.ldx;
    float sum = 0.f;
    for (int64_t d = threadIdx.x; d < a.D; d += kThreads) sum += half_at(x, d);
    const float mu = group_sum<kThreads>(sum, s) / static_cast<float>(a.D);
    float sq = 0.f;
    for (int64_t d = threadIdx.x; d < a.D; d += kThreads) {
      const float v = half_at(x, d) - mu;
      sq = fmaf(v, v, sq);
    }
    const float rs = rsqrtf(group_sum<kThreads>(sq, s) / static_cast<float>(a.D) + a.eps);
    for (int64_t d = threadIdx.x; d < a.D; d += kThreads)
      a.y[m * a.ldy + d] = __half_as_ushort(
          __float2half_rn(fmaf((half_at(x, d) - mu) * rs, half_at(a.gamma, d), half_at(a.beta, d))));
    if (threadIdx.x == 0 && a.mean) {
      a.mean[m] = mu;
      a.rstd[m] = rs;
    }
  }
}

// ----------------------------------------------------------------- backward

// At most this many partial sums of dgamma and dbeta, one pair per CTA, in
// the workspace as [partial][2][D].
constexpr int kMaxPartials = 160;

// Persistent CTAs of 512 threads, one per SM, in groups of G threads; group
// j of a CTA owns a row at a time. Rows arrive by bulk copies, several ahead,
// in a ring per group: x, dY and (RES) the residual branch. A thread owns the
// same 8·NV columns of every row, so dgamma and dbeta add up in its
// registers; at the end the groups of a CTA are added in order through shared
// memory and the CTA writes one partial sum.
//
// Per row: pass 1 over x and dY gives the two means and the gradients'
// terms, one exchange between the group's warps, pass 2 over x, dY and the
// residual gives dX. Both passes read shared memory, which keeps the
// registers for the 16·NV sums. The exchange is also what frees the stage of
// the row before: every thread of the group has finished its pass 2 by then,
// and the group's first thread copies the next row into it.
template <int G_, int NV_>
struct RingCfg {
  static constexpr int G = G_, NV = NV_;
  static constexpr int THREADS = 512;
  static constexpr int GROUPS = THREADS / G;
  static constexpr int WARPS = G / 32;  // per group
  static constexpr int MAX_STAGES = 8;
  static constexpr int RING_BYTES = 200 * 1024;  // of the CTA
  static constexpr int OFF_BAR = RING_BYTES;
  static constexpr int OFF_EXCHANGE = OFF_BAR + GROUPS * MAX_STAGES * 8;
  static constexpr int OFF_MISC = OFF_EXCHANGE + 2 * (THREADS / 32) * 8;  // two buffers of one float2 per warp
  static constexpr int SMEM_BYTES = OFF_MISC + 16;
  static_assert(SMEM_BYTES <= 232448 - 1024, "fits an SM");
  static_assert(GROUPS == 1 || THREADS * 8 * 4 * NV * 2 <= RING_BYTES, "the groups' sums fit the ring");
};

template <int G, int NV, bool RES>
__global__ void __launch_bounds__(512, 1) layernorm_backward_ring_kernel(const NormArgs a, int stages) {
  using Cfg = RingCfg<G, NV>;
  extern __shared__ __align__(128) uint8_t ring_smem[];
  const int group = threadIdx.x / G, t = threadIdx.x % G;
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int D = static_cast<int>(a.D);
  const uint32_t row_bytes = static_cast<uint32_t>(D) * 2u;
  const uint32_t stage_bytes = row_bytes * (RES ? 3u : 2u);
  uint8_t* ring = ring_smem + static_cast<uint32_t>(group * stages) * stage_bytes;
  const uint32_t ring_addr = smem_u32(ring);
  const uint32_t bar0 = smem_u32(ring_smem + Cfg::OFF_BAR) + static_cast<uint32_t>(group * Cfg::MAX_STAGES * 8);
  float2* exchange = reinterpret_cast<float2*>(ring_smem + Cfg::OFF_EXCHANGE);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(ring_smem + Cfg::OFF_MISC);
  const Watchdog wd{abort_flag, a.status, a.timeout_ns};

  if (threadIdx.x == 0) *abort_flag = 0;
  if (t == 0) {
    for (int i = 0; i < stages; ++i) mbar_init(bar0 + 8u * i, 1);
    fence_barrier_init();
  }
  __syncthreads();
  grid_dependency_wait();
  grid_launch_dependents();

  const int64_t first = static_cast<int64_t>(blockIdx.x) * Cfg::GROUPS + group;
  const int64_t step = static_cast<int64_t>(gridDim.x) * Cfg::GROUPS;
  int copied = 0;  // rows the group's first thread has issued
  auto copy_row = [&](int64_t m, int stage) {
    ++copied;
    const uint32_t bar = bar0 + 8u * stage, dst = ring_addr + static_cast<uint32_t>(stage) * stage_bytes;
    if (!(a.inject == 1 && copied == 1))  // testing aid: withhold one arrival
      mbar_arrive_expect_tx(bar, stage_bytes);
    bulk_load(dst, a.x + m * a.ldx, row_bytes, bar);
    bulk_load(dst + row_bytes, a.dy + m * a.lddy, row_bytes, bar);
    if (RES) bulk_load(dst + 2 * row_bytes, a.res + m * a.ldr, row_bytes, bar);
  };
  if (t == 0)
    for (int i = 0; i < stages - 1; ++i)
      if (first + i * step < a.M) copy_row(first + i * step, i);

  uint4 gamma[NV];
  f32x2 dgamma[NV][4], dbeta[NV][4];
#pragma unroll
  for (int i = 0; i < NV; ++i) {
    const int c = (t + i * G) * 8;
    gamma[i] = make_uint4(0u, 0u, 0u, 0u);
    if (c < D && dbg_row(a.gamma + c, c, 8, D, 16)) gamma[i] = *reinterpret_cast<const uint4*>(a.gamma + c);
#pragma unroll
    for (int k = 0; k < 4; ++k) dgamma[i][k] = dbeta[i][k] = 0;  // a pair of +0
  }

  const float inv_d = 1.f / static_cast<float>(D);
  int stage = 0, flip = 0;
  uint32_t phase = 0;
  float mu = 0.f, rs = 0.f;
  if (first < a.M) {
    mu = a.mean[first];
    rs = a.rstd[first];
  }
  for (int64_t m = first; m < a.M; m += step) {
    float next_mu = 0.f, next_rs = 0.f;
    if (m + step < a.M) {
      next_mu = a.mean[m + step];
      next_rs = a.rstd[m + step];
    }
    // A wait that gives up has raised the abort flag: no more copies are
    // issued, later waits give up at once, and the loop runs out on what the
    // ring holds, so that every thread still reaches every barrier.
    (void)wait_phase(bar0 + 8u * stage, phase, wd, kWdRows);
    const uint4* sx = reinterpret_cast<const uint4*>(ring + static_cast<uint32_t>(stage) * stage_bytes);
    const uint4* sdy = reinterpret_cast<const uint4*>(ring + static_cast<uint32_t>(stage) * stage_bytes + row_bytes);
    const uint4* sres =
        reinterpret_cast<const uint4*>(ring + static_cast<uint32_t>(stage) * stage_bytes + 2 * row_bytes);
    // (x̂ from the difference: x·rstd − mean·rstd loses its digits in a row far
    // from zero)
    const f32x2 scale = pair_of(rs), shift = pair_of(-mu);
    f32x2 p1 = 0, p2 = 0;
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      const int v = t + i * G;
      if (v * 8 < D) {
        f32x2 x[4], dy[4], g[4];
        unpack8(sx[v], x);
        unpack8(sdy[v], dy);
        unpack8(gamma[i], g);
#pragma unroll
        for (int k = 0; k < 4; ++k) {
          const f32x2 xh = mul2(add2(x[k], shift), scale), gy = mul2(dy[k], g[k]);
          p1 = add2(p1, gy);
          p2 = fma2(gy, xh, p2);
          dgamma[i][k] = fma2(dy[k], xh, dgamma[i][k]);
          dbeta[i][k] = add2(dbeta[i][k], dy[k]);
        }
      }
    }
    float s1, s2;
    {
      float lo, hi;
      unpair(p1, lo, hi);
      s1 = lo + hi;
      unpair(p2, lo, hi);
      s2 = lo + hi;
    }
    warp_sum2(s1, s2);
    if constexpr (Cfg::WARPS > 1) {
      float2* ex = exchange + flip * (Cfg::THREADS / 32) + group * Cfg::WARPS;
      if (lane == 0) ex[warp - group * Cfg::WARPS] = make_float2(s1, s2);
      named_bar_sync(1 + group, G);
      s1 = s2 = 0.f;
#pragma unroll
      for (int i = 0; i < Cfg::WARPS; ++i) {
        const float2 e = ex[i];
        s1 += e.x;
        s2 += e.y;
      }
      flip ^= 1;  // the other buffer next: nobody writes this one before everybody has read it
    } else {
      __syncwarp();
    }
    if (t == 0) {
      // the stage before this one is free: the group is past that row
      const int64_t ahead = m + (stages - 1) * step;
      if (ahead < a.M && !*abort_flag) copy_row(ahead, stage == 0 ? stages - 1 : stage - 1);
    }
    const f32x2 k1 = pair_of(-rs * (s1 * inv_d)), k2 = pair_of(-rs * (s2 * inv_d) * rs);
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      const int v = t + i * G;
      if (v * 8 < D) {
        f32x2 x[4], dy[4], g[4];
        unpack8(sx[v], x);
        unpack8(sdy[v], dy);
        unpack8(gamma[i], g);
#pragma unroll
        for (int k = 0; k < 4; ++k)
          x[k] = fma2(mul2(dy[k], g[k]), scale, fma2(add2(x[k], shift), k2, k1));
        if (RES) {
          unpack8(sres[v], dy);
#pragma unroll
          for (int k = 0; k < 4; ++k) x[k] = add2(x[k], dy[k]);
        }
        if (dbg_row(a.y + m * a.ldy + v * 8, v * 8, 8, D, 16))
          *reinterpret_cast<uint4*>(a.y + m * a.ldy + v * 8) = pack8(x);
      }
    }
    mu = next_mu;
    rs = next_rs;
    if (++stage == stages) {
      stage = 0;
      phase ^= 1u;
    }
  }

  // Every copy has landed, each waited for before its row, unless a wait gave
  // up: the last copy into each stage lands before the CTA leaves.
  __syncthreads();
  if (*abort_flag) {
    if (t == 0)
      for (int i = copied > stages ? copied - stages : 0; i < copied; ++i)
        wait_drain(bar0 + 8u * (i % stages), static_cast<uint32_t>(i / stages) & 1u, wd);
    __syncthreads();
    return;
  }
  // The CTA's partial sums: the groups in order.
  if (!HG_DBG_INDEX(blockIdx.x, kMaxPartials) || !HG_DBG_ALIGN(a.work, 16)) return;
  float* out = a.work + static_cast<int64_t>(blockIdx.x) * 2 * D;
  if constexpr (Cfg::GROUPS > 1) {
    // [group][2][NV·8·G] in the ring
    float* mine = reinterpret_cast<float*>(ring_smem) + static_cast<uint32_t>(group) * (2 * NV * 8 * G);
#pragma unroll
    for (int i = 0; i < NV; ++i)
#pragma unroll
      for (int k = 0; k < 2; ++k) {
        const int c = (t + i * G) * 8 + 4 * k;
        *reinterpret_cast<ulonglong2*>(mine + c) = make_ulonglong2(dgamma[i][2 * k], dgamma[i][2 * k + 1]);
        *reinterpret_cast<ulonglong2*>(mine + NV * 8 * G + c) = make_ulonglong2(dbeta[i][2 * k], dbeta[i][2 * k + 1]);
      }
    __syncthreads();
    for (int i = threadIdx.x; i < 2 * NV * 8 * G; i += Cfg::THREADS) {
      const int which = i / (NV * 8 * G), c = i - which * (NV * 8 * G);
      if (c >= D) continue;
      float v = 0.f;
#pragma unroll
      for (int j = 0; j < Cfg::GROUPS; ++j) v += reinterpret_cast<float*>(ring_smem)[j * (2 * NV * 8 * G) + i];
      out[static_cast<int64_t>(which) * D + c] = v;
    }
  } else {
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      const int c = (t + i * G) * 8;
      if (c < D) {
#pragma unroll
        for (int k = 0; k < 2; ++k) {
          *reinterpret_cast<ulonglong2*>(out + c + 4 * k) = make_ulonglong2(dgamma[i][2 * k], dgamma[i][2 * k + 1]);
          *reinterpret_cast<ulonglong2*>(out + D + c + 4 * k) = make_ulonglong2(dbeta[i][2 * k], dbeta[i][2 * k + 1]);
        }
      }
    }
  }
}

// dgamma and dbeta from `count` partial sums, in a fixed order: 32 of the 2D
// values per block, 8 threads down each.
__global__ void __launch_bounds__(kThreads) layernorm_sums_kernel(const NormArgs a, int count) {
  __shared__ float s[8][33];
  grid_dependency_wait();
  grid_launch_dependents();
  const int c = threadIdx.x & 31, r = threadIdx.x >> 5;
  const int64_t d = static_cast<int64_t>(blockIdx.x) * 32 + c;
  float v = 0.f;
  if (d < 2 * a.D) {
#pragma unroll 4
    for (int i = r; i < count; i += 8) v += a.work[i * 2 * a.D + d];
  }
  s[r][c] = v;
  __syncthreads();
  if (r == 0 && d < 2 * a.D) {
#pragma unroll
    for (int i = 1; i < 8; ++i) v += s[i][c];
    if (d < a.D)
      a.dgamma[d] = v;
    else
      a.dbeta[d - a.D] = v;
  }
}

// Rows that bulk copies or 16-byte reads cannot describe, or longer than the
// ring: partial sums down the columns first (dX may be dY itself) ...
constexpr int kSlices = 32;
__global__ void __launch_bounds__(kThreads) layernorm_partials_kernel(const NormArgs a) {
  __shared__ float s[2][8][33];
  grid_dependency_wait();
  grid_launch_dependents();
  const int c = threadIdx.x & 31, r = threadIdx.x >> 5;
  const int64_t d = static_cast<int64_t>(blockIdx.x) * 32 + c;
  float dg = 0.f, db = 0.f;
  if (d < a.D) {
#pragma unroll 4
    for (int64_t m = blockIdx.y * 8 + r; m < a.M; m += 8 * kSlices) {
      const float g = half_at(a.dy, m * a.lddy + d);
      dg = fmaf(g, (half_at(a.x, m * a.ldx + d) - a.mean[m]) * a.rstd[m], dg);
      db += g;
    }
  }
  s[0][r][c] = dg;
  s[1][r][c] = db;
  __syncthreads();
  if (r == 0 && d < a.D && HG_DBG_INDEX(blockIdx.y, kMaxPartials)) {
    for (int i = 1; i < 8; ++i) {
      dg += s[0][i][c];
      db += s[1][i][c];
    }
    a.work[(static_cast<int64_t>(blockIdx.y) * 2) * a.D + d] = dg;
    a.work[(static_cast<int64_t>(blockIdx.y) * 2 + 1) * a.D + d] = db;
  }
}

// ... then a block per row of dX.
__global__ void __launch_bounds__(kThreads) layernorm_backward_kernel(const NormArgs a) {
  __shared__ float s[kThreads / 32];
  grid_dependency_wait();
  grid_launch_dependents();
  for (int64_t m = blockIdx.x; m < a.M; m += gridDim.x) {
    const float mu = a.mean[m], rs = a.rstd[m];
    float s1 = 0.f, s2 = 0.f;
#pragma unroll 4
    for (int64_t d = threadIdx.x; d < a.D; d += kThreads) {
      const float g = half_at(a.dy, m * a.lddy + d) * half_at(a.gamma, d);
      s1 += g;
      s2 = fmaf(g, (half_at(a.x, m * a.ldx + d) - mu) * rs, s2);
    }
    s1 = group_sum<kThreads>(s1, s) / static_cast<float>(a.D);
    s2 = group_sum<kThreads>(s2, s) / static_cast<float>(a.D);
#pragma unroll 4
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

bool rows16(const void* p, int64_t ld) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0 && ld % 8 == 0; }

template <int G, int NV>
cudaError_t forward_with(const NormArgs& a, bool vec, cudaStream_t stream) {
  constexpr int THREADS = G < 128 ? 128 : G;
  const int64_t blocks = (a.M + THREADS / G - 1) / (THREADS / G);
  if (blocks > 0x7FFFFFFF) return cudaErrorInvalidValue;
  PdlLaunch l(dim3(static_cast<unsigned>(blocks)), dim3(THREADS), 0, stream);
  return cudaLaunchKernelEx(&l.cfg, vec ? layernorm_forward_kernel<G, NV, true> : layernorm_forward_kernel<G, NV, false>,
                            a);
}

template <int G>
cudaError_t forward_group(const NormArgs& a, bool vec, cudaStream_t stream) {
  const int64_t nv = (a.D + 8 * G - 1) / (8 * G);
  if (nv <= 1) return forward_with<G, 1>(a, vec, stream);
  if (nv <= 2) return forward_with<G, 2>(a, vec, stream);
  return forward_with<G, 4>(a, vec, stream);
}

template <int G, int NV, bool RES>
cudaError_t ring_with(const NormArgs& a, int grid, int stages, cudaStream_t stream) {
  using Cfg = RingCfg<G, NV>;
  static std::atomic<bool> attr_done[64];
  auto kern = layernorm_backward_ring_kernel<G, NV, RES>;
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  if (dev < 0 || dev >= 64 || !attr_done[dev]) {
    e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, Cfg::SMEM_BYTES);
    if (e != cudaSuccess) return e;
    if (dev >= 0 && dev < 64) attr_done[dev] = true;
  }
  PdlLaunch l(dim3(static_cast<unsigned>(grid)), dim3(Cfg::THREADS), Cfg::SMEM_BYTES, stream);
  return cudaLaunchKernelEx(&l.cfg, kern, a, stages);
}

// The ring kernel with G threads per row; *partials: how many it leaves.
template <int G, int NV>
cudaError_t ring_group(const NormArgs& a, int num_sms, int* partials, cudaStream_t stream) {
  using Cfg = RingCfg<G, NV>;
  const int64_t want = (a.M + Cfg::GROUPS - 1) / Cfg::GROUPS;
  const int most = num_sms < kMaxPartials ? num_sms : kMaxPartials;
  const int grid = static_cast<int>(want < most ? want : most);
  const int64_t per_stage = a.D * 2 * (a.res ? 3 : 2) * Cfg::GROUPS;
  int64_t stages = Cfg::RING_BYTES / per_stage;
  stages = stages > Cfg::MAX_STAGES ? Cfg::MAX_STAGES : stages;
  *partials = grid;
  return a.res ? ring_with<G, NV, true>(a, grid, static_cast<int>(stages), stream)
               : ring_with<G, NV, false>(a, grid, static_cast<int>(stages), stream);
}

}  // namespace

cudaError_t launch_layernorm_forward(const NormArgs& a, int num_sms, cudaStream_t stream) {
  const bool vec = a.D % 8 == 0 && rows16(a.x, a.ldx) && rows16(a.y, a.ldy) && rows16(a.gamma, 8) && rows16(a.beta, 8);
  // Enough threads per row to hold it, 32 values each at most; when the rows
  // do not fill the GPU, as many as have a piece of it, which is faster for
  // a single row.
  const int64_t each = a.M > 4 * static_cast<int64_t>(num_sms) ? 32 : 8;
  if (a.D <= 32 * each) return forward_group<32>(a, vec, stream);
  if (a.D <= 128 * each) return forward_group<128>(a, vec, stream);
  if (a.D <= 256 * each) return forward_group<256>(a, vec, stream);
  if (a.D <= 512 * 32) return forward_group<512>(a, vec, stream);
  PdlLaunch l(dim3(rows_grid(a.M)), dim3(kThreads), 0, stream);
  return cudaLaunchKernelEx(&l.cfg, layernorm_forward_long_kernel, a);
}

size_t layernorm_backward_workspace(int64_t, int64_t D) {
  return sizeof(float) * 2 * kMaxPartials * static_cast<size_t>(D);
}

cudaError_t launch_layernorm_backward(const NormArgs& a, int num_sms, cudaStream_t stream) {
  // (the partial sums are written 16 bytes at a time: D is a multiple of 8)
  const bool ring = a.D % 8 == 0 && a.D <= 16384 && rows16(a.x, a.ldx) && rows16(a.dy, a.lddy) && rows16(a.y, a.ldy) &&
                    rows16(a.gamma, 8) && (!a.res || rows16(a.res, a.ldr));
  int partials = 0;
  cudaError_t e = cudaSuccess;
  if (a.M == 0) {
    // no rows: the sums of nothing
  } else if (ring) {
    // 16 columns per thread, and 32 where a row would otherwise take the whole
    // CTA: the fewer threads a row needs, the more rows a CTA has under way,
    // each waiting for its own copies and exchanges. With residual, 16384
    // rows: 8192 columns on 512 threads (one row at a time) 207 us, on 256
    // (two rows) 171; 4096 columns on 256 threads 83 us, on 128 88.
    e = a.D <= 512    ? ring_group<32, 2>(a, num_sms, &partials, stream)
        : a.D <= 1024 ? ring_group<64, 2>(a, num_sms, &partials, stream)
        : a.D <= 2048 ? ring_group<128, 2>(a, num_sms, &partials, stream)
        : a.D <= 4096 ? ring_group<256, 2>(a, num_sms, &partials, stream)
        : a.D <= 8192 ? ring_group<256, 4>(a, num_sms, &partials, stream)
                      : ring_group<512, 4>(a, num_sms, &partials, stream);
  } else {
    PdlLaunch p(dim3(static_cast<unsigned>((a.D + 31) / 32), kSlices), dim3(kThreads), 0, stream);
    if ((e = cudaLaunchKernelEx(&p.cfg, layernorm_partials_kernel, a)) != cudaSuccess) return e;
    partials = kSlices;
    PdlLaunch l(dim3(rows_grid(a.M)), dim3(kThreads), 0, stream);
    e = cudaLaunchKernelEx(&l.cfg, layernorm_backward_kernel, a);
  }
  if (e != cudaSuccess) return e;
  PdlLaunch l(dim3(static_cast<unsigned>((2 * a.D + 31) / 32)), dim3(kThreads), 0, stream);
  return cudaLaunchKernelEx(&l.cfg, layernorm_sums_kernel, a, partials);
}

// The -DHGEMM_DEBUG build's check word of this file (null otherwise).
HG_DEBUG_WORD_ACCESSOR(norm)

}  // namespace hg
