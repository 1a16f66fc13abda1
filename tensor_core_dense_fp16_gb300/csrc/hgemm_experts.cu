// hgemm_experts.cu — a mixture-of-experts feed-forward layer for few tokens
// (hgemm_experts; the formulas are in hgemm.h). Bound by reading the chosen
// experts' weights once. Four launches, each started while the one before it
// ends: the router, the experts' first products, their second products, and
// the weighted sums.
//
// The products are those of the few-row linear layers: 16 rows of a weight go
// from memory straight into the fragments of a 16×8×16 matrix instruction,
// whose 8 columns are tokens, lane 4g + t taking the 16 contiguous bytes at k =
// 8t of a 32-wide piece of rows g and g + 8; the warps of a block take
// interleaved pieces of K and their sums are added in order through shared
// memory. Work is numbered over the experts that some token chose, so that
// only their weights are read, each by one block.
#include <cuda_fp16.h>

#include "debug.cuh"
#include "hgemm.h"
#include "internal.h"
#include "linear_epilogue.cuh"
#include "ptx.cuh"
#include "row_sums.cuh"

namespace hg {
namespace {

constexpr int kThreads = 256;
constexpr int kWarps = kThreads / 32;
constexpr int kTokens = HGEMM_EXPERTS_MAX_TOKENS;
constexpr int kMost = HGEMM_EXPERTS_MAX;
constexpr int kPiece = 32;  // of K, per warp and step

// D (16×8, FP32) += A (16×16) · B (16×8).
__device__ __forceinline__ void mma_16816(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3,
                                          uint32_t b0, uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, "
      "{%0, %1, %2, %3};"
      : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

// -------------------------------------------------------------------- router

// An order of FP32 logits as whole numbers: larger logit, larger number; a NaN
// below every number (0), and ties, by the lower half, to the lowest index.
__device__ __forceinline__ unsigned long long order_key(float l, int e) {
  const uint32_t b = __float_as_uint(l == 0.f ? 0.f : l);  // (−0 is +0)
  const uint32_t up = (b & 0x80000000u) ? ~b : (b | 0x80000000u);
  return (static_cast<unsigned long long>(l != l ? 0u : up) << 32) | static_cast<uint32_t>(~e);
}

__device__ __forceinline__ unsigned long long warp_max(unsigned long long v) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) {
    const unsigned long long w = __shfl_xor_sync(0xffffffffu, v, o);
    v = w > v ? w : v;
  }
  return v;
}

// The k largest of the E logits in shared memory, by one warp: lane j < k
// leaves with choice j and its share.
__device__ __forceinline__ void choose(const float* logits, int E, int k, bool normalize, int& mine, float& share) {
  const int lane = threadIdx.x & 31;
  unsigned long long last = ~0ull;
  float chosen = 0.f, top = 0.f;
  mine = 0;
  for (int j = 0; j < k; ++j) {
    unsigned long long best = 0;
    for (int e = lane; e < E; e += 32) {
      const unsigned long long key = order_key(logits[e], e);
      if (key < last && key > best) best = key;
    }
    last = best = warp_max(best);
    const int e = static_cast<int>(~static_cast<uint32_t>(best));
    if (j == 0) top = logits[e];
    if (lane == j) {
      mine = e;
      chosen = logits[e];
    }
  }
  float sum = 0.f;
  share = lane < k ? expf(chosen - top) : 0.f;
  if (normalize) {
    sum = share;
  } else {
    for (int e = lane; e < E; e += 32) sum += expf(logits[e] - top);
  }
  share = __fdiv_rn(share, warp_sum(sum));
}

// A block per token: a warp per logit, then the choice.
template <bool VEC>
__global__ void __launch_bounds__(kThreads) experts_router_kernel(const ExpertsArgs a) {
  __shared__ float logits[kMost];
  grid_dependency_wait();
  grid_launch_dependents();
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, m = blockIdx.x;
  if (!HG_DBG_INDEX(m, a.M)) return;
  const uint16_t* x = a.X + m * a.ldx;
  for (int e = warp; e < a.E; e += kWarps) {
    const uint16_t* w = a.Wr + e * a.ldwr;
    float sum = 0.f;
    if constexpr (VEC) {
      for (int64_t d = 8 * lane; d < a.D; d += 256) {
        float p[8], q[8];
        unpack8(load16(x + d), p);
        unpack8(load16(w + d), q);
#pragma unroll
        for (int i = 0; i < 8; ++i) sum = fmaf(p[i], q[i], sum);
      }
    } else {
      for (int64_t d = lane; d < a.D; d += 32) sum = fmaf(half_at(x, d), half_at(w, d), sum);
    }
    sum = warp_sum(sum);
    if (lane == 0) logits[e] = sum;
  }
  __syncthreads();
  if (warp > 0) return;
  int e;
  float share;
  choose(logits, a.E, a.k, a.normalize, e, share);
  if (lane < a.k) {
    const int at = m * a.k + lane;
    a.ws_chosen[at] = e;
    a.ws_share[at] = share;
    if (a.chosen) a.chosen[at] = e;
    if (a.share) a.share[at] = share;
  }
}

// ------------------------------------------------------------------ products

// Which experts some token chose, and who chose the one at hand. A slot is a
// choice, m·k + j.
struct Routing {
  int chosen[kTokens * HGEMM_EXPERTS_MAX_CHOICES];
  int active[kMost];  // the chosen experts, in order
  int count;
  int slots[kTokens];  // the slots that chose the expert at hand, in order
  int rows;
};

__device__ __forceinline__ void find_active(Routing& r, const ExpertsArgs& a) {
  for (int e = threadIdx.x; e < a.E; e += kThreads) r.active[e] = 0;
  __syncthreads();
  for (int i = threadIdx.x; i < a.M * a.k; i += kThreads) {
    r.chosen[i] = a.ws_chosen[i];
    r.active[r.chosen[i]] = 1;
  }
  __syncthreads();
  if (threadIdx.x < 32) {  // in place: what is written lies before what is read
    int n = 0;
    for (int e0 = 0; e0 < a.E; e0 += 32) {
      const int e = e0 + static_cast<int>(threadIdx.x);
      const bool is = e < a.E && r.active[e];
      const uint32_t all = __ballot_sync(0xffffffffu, is);
      if (is) r.active[n + __popc(all & ((1u << threadIdx.x) - 1u))] = e;
      n += __popc(all);
      __syncwarp();
    }
    if (threadIdx.x == 0) r.count = n;
  }
  __syncthreads();
}

__device__ __forceinline__ void find_slots(Routing& r, const ExpertsArgs& a, int expert) {
  __syncthreads();
  if (threadIdx.x < 32) {
    int n = 0;
    for (int i0 = 0; i0 < a.M * a.k; i0 += 32) {
      const int i = i0 + static_cast<int>(threadIdx.x);
      const bool is = i < a.M * a.k && r.chosen[i] == expert;
      const uint32_t all = __ballot_sync(0xffffffffu, is);
      if (is) r.slots[n + __popc(all & ((1u << threadIdx.x) - 1u))] = i;
      n += __popc(all);
    }
    if (threadIdx.x == 0) r.rows = n;
  }
  __syncthreads();
}

template <bool VEC>
__device__ __forceinline__ uint4 load_piece(const uint16_t* row, int k, int K, bool once) {
  if constexpr (VEC) {
    if (k >= K || !dbg_row(row + k, k, 8, K, 16)) return make_uint4(0u, 0u, 0u, 0u);
    return once ? load16_once(row + k) : load16(row + k);
  } else {
    uint32_t v[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const uint32_t lo = k + 2 * i < K ? row[k + 2 * i] : 0u;
      const uint32_t hi = k + 2 * i + 1 < K ? row[k + 2 * i + 1] : 0u;
      v[i] = lo | hi << 16;
    }
    return make_uint4(v[0], v[1], v[2], v[3]);
  }
}

// FIRST: unit u of an expert is features 8u .. 8u+7 and their gates (gated) or
// 16u .. 16u+15, and H is written; else outputs 16u .. 16u+15 and the slots'
// FP32 outputs are. MT tiles of 8 tokens.
template <int MT, bool FIRST, bool VEC>
__global__ void __launch_bounds__(kThreads) experts_product_kernel(const ExpertsArgs a) {
  __shared__ Routing r;
  __shared__ float part[kWarps][8 * MT][17];
  grid_dependency_wait();
  grid_launch_dependents();
  find_active(r, a);
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int g = lane >> 2, t = lane & 3;
  const int K = FIRST ? a.D : a.F;
  const bool gated = FIRST && a.gated;
  const int per = gated ? 8 : 16;  // outputs of a unit
  const int rows = FIRST ? a.F : a.D;
  const int units = (rows + per - 1) / per;
  const int total = r.count * units;
  const uint16_t* W = FIRST ? a.W1 : a.W2;
  const int64_t ldw = FIRST ? a.ldw1 : a.ldw2;
  const int64_t expert_rows = FIRST && gated ? 2 * static_cast<int64_t>(a.F) : rows;
  int held = -1;
  for (int u = blockIdx.x; u < total; u += gridDim.x) {
    const int at = u / units, n0 = (u - at * units) * per;
    if (at != held) {
      find_slots(r, a, r.active[at]);
      held = at;
    }
    const int expert = r.active[at], count = r.rows;
    // rows past the end are computed as copies of the last one and not stored
    const uint16_t* base = W + expert * expert_rows * ldw;
    const int64_t row0 = min(n0 + g, rows - 1);
    const int64_t row1 = gated ? row0 + a.F : min(n0 + g + 8, rows - 1);
    const uint16_t *w0 = base + row0 * ldw, *w1 = base + row1 * ldw;
    const uint16_t* x[MT];
#pragma unroll
    for (int i = 0; i < MT; ++i) {
      const int slot = 8 * i + g < count ? r.slots[8 * i + g] : -1;
      x[i] = slot < 0 ? nullptr : FIRST ? a.X + slot / a.k * a.ldx : a.ws_h + slot * a.ldh;
    }
    float acc[MT][4] = {};
    for (int k = warp * kPiece + 8 * t; k - 8 * t < K; k += kWarps * kPiece) {
      const uint4 a0 = load_piece<VEC>(w0, k, K, true), a1 = load_piece<VEC>(w1, k, K, true);
#pragma unroll
      for (int i = 0; i < MT; ++i) {
        if (8 * i >= count) break;
        const uint4 b = x[i] ? load_piece<VEC>(x[i], k, K, false) : make_uint4(0u, 0u, 0u, 0u);
        mma_16816(acc[i], a0.x, a1.x, a0.y, a1.y, b.x, b.y);
        mma_16816(acc[i], a0.z, a1.z, a0.w, a1.w, b.z, b.w);
      }
    }
    __syncthreads();  // the unit before has been added up
#pragma unroll
    for (int i = 0; i < MT; ++i) {
      part[warp][8 * i + 2 * t][g] = acc[i][0];
      part[warp][8 * i + 2 * t + 1][g] = acc[i][1];
      part[warp][8 * i + 2 * t][g + 8] = acc[i][2];
      part[warp][8 * i + 2 * t + 1][g + 8] = acc[i][3];
    }
    __syncthreads();
    for (int i = threadIdx.x; i < count * per; i += kThreads) {
      const int row = i / per, f = i - row * per, n = n0 + f;
      if (n >= rows) continue;
      const int slot = r.slots[row];
      float v = part[0][row][f];
#pragma unroll
      for (int w = 1; w < kWarps; ++w) v += part[w][row][f];
      if constexpr (FIRST) {
        const uint16_t* b = a.b1 ? a.b1 + expert * expert_rows : nullptr;
        if (b) v += half_at(b, n);
        v = activate(v, a.act);
        if (gated) {
          float up = part[0][row][f + 8];
#pragma unroll
          for (int w = 1; w < kWarps; ++w) up += part[w][row][f + 8];
          if (b) up += half_at(b, a.F + n);
          v *= up;
        }
        if (HG_DBG_INDEX(n, a.F)) a.ws_h[slot * a.ldh + n] = __half_as_ushort(__float2half_rn(v));
      } else {
        if (HG_DBG_INDEX(n, a.D)) a.ws_out[slot * a.ldo + n] = v;
      }
    }
  }
}

// Y = Σ s·(output + b2) + R, the choices in order.
__global__ void __launch_bounds__(kThreads) experts_sum_kernel(const ExpertsArgs a) {
  grid_dependency_wait();
  grid_launch_dependents();
  const int m = blockIdx.y;
  const int64_t d = static_cast<int64_t>(blockIdx.x) * kThreads + threadIdx.x;
  if (d >= a.D || !HG_DBG_INDEX(m, a.M)) return;
  float y = a.R ? half_at(a.R, m * a.ldr + d) : 0.f;
  for (int j = 0; j < a.k; ++j) {
    const int slot = m * a.k + j;
    float v = a.F > 0 ? a.ws_out[slot * a.ldo + d] : 0.f;
    if (a.b2) v += half_at(a.b2, static_cast<int64_t>(a.ws_chosen[slot]) * a.D + d);
    y = fmaf(a.ws_share[slot], v, y);
  }
  a.Y[m * a.ldy + d] = __half_as_ushort(__float2half_rn(y));
}

template <int MT, bool FIRST>
cudaError_t product_with(const ExpertsArgs& a, bool vec, int num_sms, cudaStream_t stream) {
  PdlLaunch l(dim3(static_cast<unsigned>(num_sms * 3)), dim3(kThreads), 0, stream);
  return cudaLaunchKernelEx(&l.cfg, vec ? experts_product_kernel<MT, FIRST, true> : experts_product_kernel<MT, FIRST, false>,
                            a);
}

template <bool FIRST>
cudaError_t product(const ExpertsArgs& a, bool vec, int num_sms, cudaStream_t stream) {
  if (a.M <= 8) return product_with<1, FIRST>(a, vec, num_sms, stream);
  if (a.M <= 16) return product_with<2, FIRST>(a, vec, num_sms, stream);
  if (a.M <= 32) return product_with<4, FIRST>(a, vec, num_sms, stream);
  return product_with<8, FIRST>(a, vec, num_sms, stream);
}

int64_t align16(int64_t bytes) { return (bytes + 15) / 16 * 16; }

}  // namespace

// The choice, its shares, H (rows of whole 16 bytes) and the slots' outputs.
size_t experts_workspace(int64_t M, int64_t D, int64_t F, int64_t k) {
  return static_cast<size_t>(2 * align16(4 * M * k) + M * k * align16(2 * F) + M * k * align16(4 * D));
}

cudaError_t launch_experts(ExpertsArgs a, void* workspace, int num_sms, cudaStream_t stream) {
  const int64_t slots = static_cast<int64_t>(a.M) * a.k;
  uint8_t* ws = static_cast<uint8_t*>(workspace);
  a.ws_chosen = reinterpret_cast<int*>(ws);
  a.ws_share = reinterpret_cast<float*>(ws += align16(4 * slots));
  a.ws_h = reinterpret_cast<uint16_t*>(ws += align16(4 * slots));
  a.ldh = align16(2 * static_cast<int64_t>(a.F)) / 2;
  a.ws_out = reinterpret_cast<float*>(ws += slots * a.ldh * 2);
  a.ldo = align16(4 * static_cast<int64_t>(a.D)) / 4;
  const bool vec_x = a.D % 8 == 0 && rows16(a.X, a.ldx);
  const bool vec_r = vec_x && rows16(a.Wr, a.ldwr), vec1 = vec_x && rows16(a.W1, a.ldw1);
  const bool vec2 = a.F % 8 == 0 && rows16(a.W2, a.ldw2);
  cudaError_t e;
  {
    PdlLaunch l(dim3(static_cast<unsigned>(a.M)), dim3(kThreads), 0, stream);
    e = cudaLaunchKernelEx(&l.cfg, vec_r ? experts_router_kernel<true> : experts_router_kernel<false>, a);
    if (e != cudaSuccess) return e;
  }
  if (a.F > 0) {
    if ((e = product<true>(a, vec1, num_sms, stream)) != cudaSuccess) return e;
    if ((e = product<false>(a, vec2, num_sms, stream)) != cudaSuccess) return e;
  }
  if (a.D == 0) return cudaSuccess;
  PdlLaunch l(dim3(static_cast<unsigned>((a.D + kThreads - 1) / kThreads), static_cast<unsigned>(a.M)), dim3(kThreads),
              0, stream);
  return cudaLaunchKernelEx(&l.cfg, experts_sum_kernel, a);
}

// The -DHGEMM_DEBUG build's check word of this file (null otherwise).
HG_DEBUG_WORD_ACCESSOR(experts)

}  // namespace hg
