// hgemm_linear_small.cu — products of linear layers with few rows or a small
// output: the forward product and the input gradient of at most 128 rows (a
// batch of generated tokens, a short prompt), bound by reading the weights
// once, and the gradient of a small weight over many rows.
//
// The product is computed turned around: the columns of the output (features)
// are the rows of the matrix instruction (M = 128) and the output's rows its
// columns (N = 16 to 128, as many as there are), so that no part of the
// instruction is spent on rows that do not exist, and a CTA's ring of stages
// is almost all weights: 5 to 12 stages, about 200 KB under way per SM. A
// cluster of CTAs shares an output tile, each a run of K. Each output row has
// one of them as its owner: the others store their FP32 partial sums into the
// owner's shared memory, beside its ring, and the owner adds them and its own
// in rank order, so the result does not depend on timing. (Read by the owner
// instead, between two barriers of the cluster, they took 3.7 us of 10: 24 rows
// 2048×8192.) In the accumulator a thread owns a
// feature: bias, residual, 8-bit codes and outputs are read and written along
// the features, whatever their pitch and alignment.
//
// Measured (us, weights from memory, bias and GELU, one launch after another): 24
// rows 8192×2048 8.7, 4096×4096 9.0, 2048×8192 10.0, each 4.9 at a copy's rate; 100
// rows 8192×8192 29.2, 4.6 TB/s. The weights of 2048×8192 arrive in 5.0; before
// them come the previous launch's end and the first read, after them the sums'
// exchange and the output, 1.5 to 2.
#include <atomic>

#include "internal.h"
#include "kernel_common.cuh"
#include "linear_epilogue.cuh"
#include "linear_rows.h"
#include "ptx.cuh"

namespace hg {
namespace {

template <int NT_>
struct SmallCfg {
  static constexpr int NT = NT_;   // output rows per CTA: columns of the instruction
  static constexpr int BM = 128;   // features
  static constexpr int BK = kTcBK, UMMA_K = 16;
  static constexpr int W_BYTES = BM * BK * 2;
  static constexpr int X_BYTES = NT * BK * 2;
  static constexpr int STAGE_BYTES = W_BYTES + X_BYTES;
  // four rows of 128 features' partial sums are a unit; the units that a CTA
  // receives take the end of the ring's space
  static constexpr int UNITS = NT / 4;
  static constexpr int UNIT_BYTES = BM * 4 * 4;
  static constexpr int OFF_BAR = 224 * 1024;
  static constexpr int STAGES = OFF_BAR / STAGE_BYTES;  // the most, without a cluster
  static constexpr int NUM_BARS = 2 * STAGES + 3;  // full, empty, accumulator full, drain, received
  static constexpr int OFF_MISC = OFF_BAR + NUM_BARS * 8;
  static constexpr int SMEM_BYTES = OFF_MISC + 16 + 1024;
  static constexpr int THREADS = 192;
  static constexpr int TMEM_COLS = NT < 32 ? 32 : NT;
  static constexpr uint32_t IDESC = idesc_f16_f32acc(BM, NT);
  static_assert(STAGE_BYTES % 1024 == 0, "swizzled tiles are 1024-byte aligned");
  static_assert(SMEM_BYTES <= 232448, "exceeds 227 KB of shared memory per CTA");
};

// What the outputs of feature f and rows m .. m + R - 1, the first `count` of
// them inside, read besides the sums.
template <int R>
struct RowSide {
  uint32_t side[R];  // residual, or codes
  float scale[R];
};
template <bool BACKWARD, int R>
__device__ __forceinline__ RowSide<R> fetch_rows(const SmallArgs& p, int64_t m, int f, int count) {
  const LinEpi& e = p.epi;
  RowSide<R> s;
#pragma unroll
  for (int i = 0; i < R; ++i) {
    s.side[i] = 0u;
    s.scale[i] = 0.f;
  }
  if (count > 0 && !(HG_DBG_INDEX(f, p.N) && HG_DBG_INDEX(m + (count < R ? count : R) - 1, p.M))) count = 0;
  if (BACKWARD && e.codes) {
    const int8_t* q = e.codes + m * e.ldq + f;
    const float* scale = e.scales + f / kCkptGroup * e.lds + m;
#pragma unroll
    for (int i = 0; i < R; ++i, q += e.ldq)
      if (i < count) {
        s.side[i] = static_cast<uint8_t>(*q);
        s.scale[i] = scale[i];
      }
  } else if (!BACKWARD && e.res) {
    const uint16_t* r = e.res + m * e.ldr + f;
#pragma unroll
    for (int i = 0; i < R; ++i, r += e.ldr)
      if (i < count) s.side[i] = *r;
  }
  return s;
}

// The outputs themselves.
template <bool BACKWARD, int R>
__device__ __forceinline__ void put_rows(const SmallArgs& p, const float (&sum)[R], const RowSide<R>& s, float bias,
                                         int64_t m, int f, int count) {
  const LinEpi& e = p.epi;
  const uint32_t(&side)[R] = s.side;
  const float(&scale)[R] = s.scale;
  if (count > 0 && !(HG_DBG_INDEX(f, p.N) && HG_DBG_INDEX(m + (count < R ? count : R) - 1, p.M))) count = 0;
  uint16_t* y = p.Y + m * p.ldy + f;
  uint16_t* h = e.h + m * e.ldh + f;
  with_activation(!BACKWARD || e.codes ? e.act : HGEMM_ACT_NONE, [&](auto a) {
#pragma unroll
    for (int i = 0; i < R; i += 2) {
      f32x2 v = pair_of(sum[i], sum[i + 1]), df;
      if constexpr (BACKWARD) {
        if (e.codes) {
          f32x2 hid;
          activate<decltype(a)::value, true>(pair_of(static_cast<float>(static_cast<int8_t>(side[i])) * scale[i],
                                                     static_cast<float>(static_cast<int8_t>(side[i + 1])) * scale[i + 1]),
                                             hid, df);
          v = mul2(v, df);
          if (e.h) {
            const uint32_t w = pack_half2(hid);
            if (i < count) h[0] = static_cast<uint16_t>(w);
            if (i + 1 < count) h[e.ldh] = static_cast<uint16_t>(w >> 16);
            h += 2 * e.ldh;
          }
        }
      } else {
        f32x2 f2;
        activate<decltype(a)::value, false>(add2(v, pair_of(bias)), f2, df);
        v = add2(f2, unpack_half2(side[i] | side[i + 1] << 16));
      }
      const uint32_t w = pack_half2(v);
      if (i < count) y[0] = static_cast<uint16_t>(w);
      if (i + 1 < count) y[p.ldy] = static_cast<uint16_t>(w >> 16);
      y += 2 * p.ldy;
    }
  });
}

// W_MN, X_MN: the operand whose rows are features, or output rows, is stored
// with those contiguous (K×features, K×rows) and read as MN-major tiles.
template <int NT, bool W_MN, bool X_MN, bool BACKWARD>
__global__ void __launch_bounds__(192, 1)
    linear_small_kernel(const __grid_constant__ CUtensorMap tmW, const __grid_constant__ CUtensorMap tmX,
                        const SmallArgs p) {
  using Cfg = SmallCfg<NT>;
  extern __shared__ uint8_t smem_raw[];
  const uint32_t raw_addr = smem_u32(smem_raw);
  uint8_t* smem = smem_raw + ((1024u - (raw_addr & 1023u)) & 1023u);
  const uint32_t sbase = smem_u32(smem);
  const uint32_t bar0 = sbase + Cfg::OFF_BAR;
  const uint32_t accf_bar = bar0 + 8u * (2 * Cfg::STAGES), drain_bar = accf_bar + 8u;
  const uint32_t recv_bar = drain_bar + 8u;
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(smem + Cfg::OFF_MISC);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(smem + Cfg::OFF_MISC + 4);
  auto full_bar = [&](int s) { return bar0 + 8u * s; };
  auto empty_bar = [&](int s) { return bar0 + 8u * (Cfg::STAGES + s); };
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int rank = p.split > 1 ? static_cast<int>(cluster_ctarank()) : 0;
  const int tile = static_cast<int>(blockIdx.x) / p.split;
  const int f0 = tile / p.row_tiles * Cfg::BM;  // first feature
  const int r0 = tile % p.row_tiles * NT;       // first output row
  const int rows = p.M - r0 < NT ? p.M - r0 : NT;
  const int kb0 = static_cast<int>(static_cast<long long>(p.num_kb) * rank / p.split);
  const int kb1 = static_cast<int>(static_cast<long long>(p.num_kb) * (rank + 1) / p.split);
  // units with rows inside; this CTA owns [u0, u1), and its buffer, at the end
  // of the space, has room for `per` of each other rank
  const int units = (rows + 3) / 4;
  const int u0 = units * rank / p.split, u1 = units * (rank + 1) / p.split;
  const int per = (units + p.split - 1) / p.split;
  const int off_part = Cfg::OFF_BAR - (p.split - 1) * per * Cfg::UNIT_BYTES;
  const int stages = off_part / Cfg::STAGE_BYTES;
  const Watchdog wd{abort_flag, p.status, p.timeout_ns};

  if (threadIdx.x == 0) {
    for (int s = 0; s < Cfg::STAGES; ++s) {
      mbar_init(full_bar(s), 1);
      mbar_init(empty_bar(s), 1);
    }
    mbar_init(accf_bar, 1);
    mbar_init(drain_bar, 1);
    mbar_init(recv_bar, 4 * (p.split > 1 ? p.split - 1 : 1));  // the other ranks' epilogue warps
    *abort_flag = 0;
    fence_barrier_init();
    prefetch_tensormap(&tmW);
    prefetch_tensormap(&tmX);
  }
  if (warp == 1) {
    tmem_alloc(smem_u32(tmem_slot), Cfg::TMEM_COLS);
    tmem_relinquish_alloc_permit();
  }
  tc_fence_before_sync();
  __syncthreads();
  if (p.split > 1) cluster_sync_after_init();  // partial sums reach the other CTAs' barriers
  tc_fence_after_sync();
  const uint32_t tmem_base = *tmem_slot;
  // As much of the weights as the ring holds, into L2 while the previous
  // launch on the stream ends (only asked for: whatever it still writes there
  // is read after the wait). 24 rows 8192×2048 9.6 to 9.1 us, one after another.
  if (warp == 0 && elect_one())
    for (int kb = kb0; kb < kb1 && kb < kb0 + stages; ++kb) {
      if constexpr (W_MN) {
        tma_prefetch_2d(&tmW, f0, kb * Cfg::BK);
        tma_prefetch_2d(&tmW, f0 + kMnBox, kb * Cfg::BK);
      } else {
        tma_prefetch_2d(&tmW, kb * Cfg::BK, f0);
      }
    }
  grid_dependency_wait();
  grid_launch_dependents();

  const int q = warp & 3;
  const int f = f0 + q * 32 + lane;  // this epilogue thread's feature
  const bool in_f = f < p.N;
  const float bias =
      !BACKWARD && warp >= 2 && p.epi.bias && in_f ? __half2float(__ushort_as_half(p.epi.bias[f])) : 0.f;

  if (warp == 0) {
    if (elect_one()) {
      int stage = 0;
      uint32_t phase = 0;
      int issued = 0;
      for (int kb = kb0; kb < kb1; ++kb) {
        if (!wait_phase(empty_bar(stage), phase ^ 1u, wd, kWdProducerEmpty)) break;
        if (!(p.inject == 1 && issued == 0))  // testing aid: withhold one arrival
          mbar_arrive_expect_tx(full_bar(stage), Cfg::STAGE_BYTES);
        const uint32_t dst = sbase + stage * Cfg::STAGE_BYTES;
        if constexpr (W_MN) {
          tma_load_2d(dst, &tmW, full_bar(stage), f0, kb * Cfg::BK);
          tma_load_2d(dst + kMnBoxBytes, &tmW, full_bar(stage), f0 + kMnBox, kb * Cfg::BK);
        } else {
          tma_load_2d(dst, &tmW, full_bar(stage), kb * Cfg::BK, f0);
        }
        if constexpr (X_MN) {
#pragma unroll
          for (int b = 0; b < NT / kMnBox; ++b)
            tma_load_2d(dst + Cfg::W_BYTES + b * kMnBoxBytes, &tmX, full_bar(stage), r0 + b * kMnBox, kb * Cfg::BK);
        } else {
          tma_load_2d(dst + Cfg::W_BYTES, &tmX, full_bar(stage), kb * Cfg::BK, r0);
        }
        ++issued;
        if (++stage == stages) {
          stage = 0;
          phase ^= 1u;
        }
      }
      // the last loads must have landed before the ring is reused or left
      int s = stage;
      uint32_t ph = phase;
      for (int i = 0; i < issued && i < stages; ++i) {
        if (s == 0) {
          s = stages - 1;
          ph ^= 1u;
        } else {
          --s;
        }
        wait_drain(full_bar(s), ph, wd);
      }
    }
    __syncwarp();
  } else if (warp == 1) {
    if (elect_one()) {
      int stage = 0;
      uint32_t phase = 0;
      bool ok = true;
      for (int kb = kb0; kb < kb1; ++kb) {
        if (!wait_phase(full_bar(stage), phase, wd, kWdMmaFull)) {
          ok = false;
          break;
        }
        tc_fence_after_sync();
        const uint32_t sw = sbase + stage * Cfg::STAGE_BYTES, sx = sw + Cfg::W_BYTES;
        const uint64_t w_desc = W_MN ? sdesc_mnmajor_sw128(sw) : sdesc_kmajor_sw128(sw);
        const uint64_t x_desc = X_MN ? sdesc_mnmajor_sw128(sx) : sdesc_kmajor_sw128(sx);
#pragma unroll
        for (int k = 0; k < Cfg::BK / Cfg::UMMA_K; ++k)
          mma_f16_ss(tmem_base, w_desc + (W_MN ? 128u : 2u) * k, x_desc + (X_MN ? 128u : 2u) * k,
                     Cfg::IDESC | idesc_major_bits(W_MN, X_MN), (kb > kb0 || k > 0) ? 1u : 0u);
        mma_commit(empty_bar(stage));
        if (++stage == stages) {
          stage = 0;
          phase ^= 1u;
        }
      }
      if (ok) mma_commit(accf_bar);
      mma_commit(drain_bar);
      wait_drain(drain_bar, 0, wd);
    }
    __syncwarp();
  } else {
    int ok = 1;
    if (lane == 0) ok = wait_phase(accf_bar, 0, wd, kWdEpiAccFull) ? 1 : 0;
    ok = __shfl_sync(0xffffffffu, ok, 0);
    if (ok) {
      tc_fence_after_sync();
      const uint32_t t_row = tmem_base + (static_cast<uint32_t>(q * 32) << 16);
      if (p.split == 1) {
#pragma unroll 1
        for (int c = 0; c < rows; c += 16) {
          float v[16];
          tmem_ld_32x32b_x16(t_row + c, v);
          const int count = in_f ? rows - c : 0;
          put_rows<BACKWARD, 16>(p, v, fetch_rows<BACKWARD, 16>(p, r0 + c, f, count), bias, r0 + c, f, count);
        }
      } else {
        const uint32_t column = static_cast<uint32_t>(q * 32 + lane) * 16u;
        int owner = 0, first = 0, end = units / p.split;  // the owner's units
#pragma unroll 1
        for (int c = 0; c < rows; c += 16) {
          float v[16];
          tmem_ld_32x32b_x16(t_row + c, v);
#pragma unroll
          for (int i = 0; i < 16; i += 4) {
            const int u = (c + i) / 4;
            while (u >= end && owner + 1 < p.split) {
              first = end;
              end = units * (++owner + 1) / p.split;
            }
            if (u < units && owner != rank) {
              const int slot = (rank < owner ? rank : rank - 1) * per + u - first;
              st_cluster_v4(mapa_shared(sbase + static_cast<uint32_t>(off_part + slot * Cfg::UNIT_BYTES) + column, owner),
                            __float_as_uint(v[i]), __float_as_uint(v[i + 1]), __float_as_uint(v[i + 2]),
                            __float_as_uint(v[i + 3]));
            }
          }
        }
        __syncwarp();
        if (lane < p.split && lane != rank) mbar_arrive_cluster(mapa_shared(recv_bar, static_cast<uint32_t>(lane)));
      }
    }
    if (p.split > 1) {
      // (read while the other ranks' sums are on their way)
      auto inside = [&](int u) { return in_f ? min(rows, 4 * u1) - 4 * u : 0; };
      RowSide<8> side = fetch_rows<BACKWARD, 8>(p, r0 + 4 * u0, f, inside(u0));
      // Nothing is left under way to this CTA's shared memory once the other
      // ranks have all arrived (after a wait that gave up they are awaited too).
      if (lane == 0)
        ok = (ok ? wait_phase_cluster(recv_bar, 0, wd, kWdReduce) : wait_drain_cluster(recv_bar, 0, wd)) ? ok : 0;
      ok = __shfl_sync(0xffffffffu, ok, 0);
      const uint8_t* part = smem + off_part + (q * 32 + lane) * 16;
      const uint32_t t_row = tmem_base + (static_cast<uint32_t>(q * 32) << 16);
#pragma unroll 1
      for (int u = u0; ok && u < u1; u += 2) {
        float own[2][4] = {}, sum[8];
        tmem_ld_32x32b_x4(t_row + 4 * u, own[0]);
        if (u + 1 < u1) tmem_ld_32x32b_x4(t_row + 4 * u + 4, own[1]);
#pragma unroll
        for (int i = 0; i < 8; ++i) sum[i] = 0.f;
#pragma unroll 1
        for (int r = 0; r < p.split; ++r) {
          const uint8_t* from = part + ((r < rank ? r : r - 1) * per + u - u0) * Cfg::UNIT_BYTES;
#pragma unroll
          for (int j = 0; j < 2; ++j) {
            float4 w = make_float4(own[j][0], own[j][1], own[j][2], own[j][3]);
            if (r != rank && u + j < u1) w = *reinterpret_cast<const float4*>(from + j * Cfg::UNIT_BYTES);
            sum[4 * j] += w.x;
            sum[4 * j + 1] += w.y;
            sum[4 * j + 2] += w.z;
            sum[4 * j + 3] += w.w;
          }
        }
        put_rows<BACKWARD, 8>(p, sum, side, bias, r0 + 4 * u, f, inside(u));
        if (u + 2 < u1) side = fetch_rows<BACKWARD, 8>(p, r0 + 4 * (u + 2), f, inside(u + 2));
      }
    }
  }
  tc_fence_before_sync();
  __syncthreads();
  tc_fence_after_sync();
  if (warp == 1) tmem_dealloc(tmem_base, Cfg::TMEM_COLS);
}

template <int NT, bool W_MN, bool X_MN, bool BACKWARD>
cudaError_t launch_with(const CUtensorMap& w, const CUtensorMap& x, const SmallArgs& a, cudaStream_t stream) {
  using Cfg = SmallCfg<NT>;
  static std::atomic<bool> attr_done[64];
  auto kern = linear_small_kernel<NT, W_MN, X_MN, BACKWARD>;
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  if (dev < 0 || dev >= 64 || !attr_done[dev]) {
    e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, Cfg::SMEM_BYTES);
    if (e != cudaSuccess) return e;
    if (dev >= 0 && dev < 64) attr_done[dev] = true;
  }
  const unsigned tiles = static_cast<unsigned>(tiles_of(a.N, Cfg::BM) * a.row_tiles);
  PdlLaunch l(dim3(tiles * static_cast<unsigned>(a.split)), dim3(Cfg::THREADS), Cfg::SMEM_BYTES, stream);
  l.cluster(static_cast<unsigned>(a.split));
  return cudaLaunchKernelEx(&l.cfg, kern, w, x, a);
}

template <int NT>
cudaError_t launch_rows(const CUtensorMap& w, const CUtensorMap& x, const SmallArgs& a, cudaStream_t stream) {
  if (a.epi.backward) return launch_with<NT, true, false, true>(w, x, a, stream);
  if (!a.w_mn) return launch_with<NT, false, false, false>(w, x, a, stream);
  if constexpr (NT % kMnBox == 0)
    return launch_with<NT, true, true, false>(w, x, a, stream);
  else
    return cudaErrorInvalidValue;
}

}  // namespace

int linear_small_clusters(int split, int num_sms) {
  static std::atomic<int> cached[64][9];
  int dev = 0;
  if (split < 1 || split > 8 || cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= 64) return 0;
  if (cached[dev][split] > 0) return cached[dev][split];
  using Cfg = SmallCfg<16>;  // (the others differ by a few KB of shared memory)
  auto kern = linear_small_kernel<16, false, false, false>;
  int n = 0;
  if (cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, Cfg::SMEM_BYTES) == cudaSuccess) {
    PdlLaunch l(dim3(static_cast<unsigned>(num_sms / split * split)), dim3(Cfg::THREADS), Cfg::SMEM_BYTES, nullptr);
    l.cluster(static_cast<unsigned>(split));
    if (cudaOccupancyMaxActiveClusters(&n, kern, &l.cfg) != cudaSuccess) n = 0;
  }
  (void)cudaGetLastError();
  if (n <= 0) n = 1;
  cached[dev][split] = n;
  return n;
}

cudaError_t launch_linear_small(const CUtensorMap& w, const CUtensorMap& x, const SmallArgs& a, cudaStream_t stream) {
  switch (a.tile_rows) {
    case 16:
      return launch_rows<16>(w, x, a, stream);
    case 32:
      return launch_rows<32>(w, x, a, stream);
    case 64:
      return launch_rows<64>(w, x, a, stream);
    case 128:
      return launch_rows<128>(w, x, a, stream);
    default:
      return cudaErrorInvalidValue;
  }
}

// The -DHGEMM_DEBUG build's check word of this file (null otherwise).
HG_DEBUG_WORD_ACCESSOR(linear_small)

}  // namespace hg
