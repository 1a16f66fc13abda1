// hgemm_linear_wave.cu — linear layers and their gradients whose output is a
// single wave of 128×64 tiles (about a thousand rows and columns): a CTA per
// tile, which loads its own operands, and the bias gradient summed from the
// weight gradient's staged tiles.
//
// Bound by what one SM can ask of L2: about one 128-byte line per cycle, 192 to
// a block of 64 of the contraction, twice that where rows begin inside lines
// (an odd multiple of 16 bytes). The operand order is a template parameter: a
// branch on it between the copies took 0.155 us per block where there was none
// 0.115.
//
// Measured (us, in a graph, operands in L2): 1024×1024 outputs of a contraction
// of 1024 4.7, with bias, SiLU and residual 5.5, the input gradient with
// SiLU's and f(û) 5.9, the weight gradient 4.9, with the bias's 5.5; 1000^3, whose rows
// begin inside lines, 7.4, 8.2, 9.0, 8.5 and 8.4 (a kernel of column sums beside the
// product instead of the sums here takes 10.8). Of the 5.5 us, about 3 are
// launch and set-up, and 1 the epilogue: its two special-function instructions
// per SiLU occupy their unit for 1,024 cycles.
#include <atomic>

#include "internal.h"
#include "kernel_common.cuh"
#include "linear_epilogue.cuh"
#include "ptx.cuh"

namespace hg {
namespace {

struct WaveCfg {
  static constexpr int BM = kTcBM, BN = kNarrowBN, BK = kTcBK, UMMA_K = 16;
  static constexpr int STAGES = 8;
  static constexpr int A_BYTES = BM * BK * 2;
  static constexpr int B_BYTES = BN * BK * 2;
  static constexpr int STAGE_BYTES = A_BYTES + B_BYTES;
  static constexpr int EPI_WARPS = 4;
  static constexpr int C_BOX_BYTES = kEpiRows * kEpiCols * 2;
  static constexpr int OFF_A = 0;
  static constexpr int OFF_B = OFF_A + STAGES * A_BYTES;
  static constexpr int OFF_C = OFF_B + STAGES * B_BYTES;
  static constexpr int OFF_SUM = OFF_C + EPI_WARPS * C_BOX_BYTES;  // partial row sums of A
  static constexpr int OFF_BAR = OFF_SUM + EPI_WARPS * kMnBox * 4;
  static constexpr int NUM_BARS = 2 * STAGES + 2;  // full, empty, accumulator full, drain
  static constexpr int OFF_MISC = OFF_BAR + NUM_BARS * 8;
  static constexpr int SMEM_BYTES = OFF_MISC + 16 + 1024;
  static constexpr int THREADS = 192;
  static constexpr int TMEM_COLS = BN;
  static constexpr uint32_t IDESC = idesc_f16_f32acc(BM, BN);
  static_assert(A_BYTES % 1024 == 0 && B_BYTES % 1024 == 0, "swizzled tiles are 1024-byte aligned");
  static_assert(BM == 2 * kMnBox && BN == kMnBox, "an MN-major A tile is two boxes, a B tile one");
  static_assert(SMEM_BYTES <= 232448, "exceeds 227 KB of shared memory per CTA");
};

// The sums over K of 64 rows of the A tile, by the epilogue warps while the
// product runs: the bias gradient beside the weight's, from the stages in
// shared memory (an MN-major box: 64 K rows of 128 bytes). The four warps take
// K blocks in turn, so that none of them delays the ring. A thread adds the
// eight rows of A of one 16-byte chunk in every fourth K row of its warp's
// blocks, and the 16 partial sums of a row are added in a fixed order.
__device__ __forceinline__ void sum_rows(const TcArgs& p, uint8_t* smem, uint32_t full0, uint32_t empty0, int box,
                                         int first, const Watchdog& wd) {
  using Cfg = WaveCfg;
  const int t = static_cast<int>(threadIdx.x) - 64, lane = t & 31;
  const int chunk = t & 7, k0 = lane >> 3;
  const uint8_t* tile = smem + Cfg::OFF_A + box * kMnBoxBytes;
  f32x2 sum[4] = {};
  for (int kb = t >> 5; kb < p.num_kb; kb += Cfg::EPI_WARPS) {
    const int stage = kb % Cfg::STAGES;
    int ok = 1;
    if (lane == 0) ok = wait_phase(full0 + 8u * stage, kb / Cfg::STAGES & 1, wd, kWdRows) ? 1 : 0;
    ok = __shfl_sync(0xffffffffu, ok, 0);
    if (!ok) break;
    const uint8_t* src = tile + stage * Cfg::A_BYTES;
#pragma unroll
    for (int i = 0; i < Cfg::BK / 4; ++i)
      add8(sum, *reinterpret_cast<const uint4*>(src + (k0 + 4 * i) * 128 + ((chunk ^ (k0 + 4 * (i & 1))) << 4)));
    __syncwarp();
    if (lane == 0) mbar_arrive(empty0 + 8u * stage);
  }
  float v[8];
#pragma unroll
  for (int i = 0; i < 4; ++i) unpair(sum[i], v[2 * i], v[2 * i + 1]);
  float* part = reinterpret_cast<float*>(smem + Cfg::OFF_SUM);  // [warp][row]
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    v[i] += __shfl_xor_sync(0xffffffffu, v[i], 8);
    v[i] += __shfl_xor_sync(0xffffffffu, v[i], 16);
    if (lane < 8) part[(t >> 5) * kMnBox + chunk * 8 + i] = v[i];
  }
  named_bar_sync(1, 32 * Cfg::EPI_WARPS);
  if (t < kMnBox && first + t < p.M && HG_DBG_INDEX(box, 2)) {
    float total = 0.f;
#pragma unroll
    for (int w = 0; w < Cfg::EPI_WARPS; ++w) total += part[w * kMnBox + t];
    float* out = p.row_sums + first + t;
    *out = p.row_sums_add ? *out + total : total;
  }
}

// A_MN, B_MN: the operand is stored with its rows contiguous (K×M, K×N).
template <int EPI, bool A_MN, bool B_MN>
__global__ void __launch_bounds__(WaveCfg::THREADS, 1)
    linear_wave_kernel(const __grid_constant__ CUtensorMap tmA, const __grid_constant__ CUtensorMap tmB,
                          const __grid_constant__ CUtensorMap tmC, const TcArgs p) {
  using Cfg = WaveCfg;
  extern __shared__ uint8_t smem_raw[];
  const uint32_t raw_addr = smem_u32(smem_raw);
  uint8_t* smem = smem_raw + ((1024u - (raw_addr & 1023u)) & 1023u);
  const uint32_t sbase = smem_u32(smem);
  const uint32_t sA = sbase + Cfg::OFF_A, sB = sbase + Cfg::OFF_B;
  const uint32_t bar0 = sbase + Cfg::OFF_BAR;
  const uint32_t accf_bar = bar0 + 8u * (2 * Cfg::STAGES), drain_bar = accf_bar + 8u;
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(smem + Cfg::OFF_MISC);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(smem + Cfg::OFF_MISC + 4);
  auto full_bar = [&](int s) { return bar0 + 8u * s; };
  auto empty_bar = [&](int s) { return bar0 + 8u * (Cfg::STAGES + s); };

  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int m0 = static_cast<int>(blockIdx.x) % p.num_m * Cfg::BM;
  const int nb = static_cast<int>(blockIdx.x) / p.num_m, n0 = nb * Cfg::BN;
  // sums of A's rows over K: a box of 64 rows each in the first two columns of
  // tiles (args.grid has both)
  const bool summed = A_MN && p.row_sums && nb < 2;
  const Watchdog wd{abort_flag, p.status, p.timeout_ns};

  if (threadIdx.x == 0) {
    for (int s = 0; s < Cfg::STAGES; ++s) {
      mbar_init(full_bar(s), 1);                // the producer's arrive.expect_tx (+ bytes)
      mbar_init(empty_bar(s), summed ? 2 : 1);  // tcgen05.commit, and the block's summing warp
    }
    mbar_init(accf_bar, 1);
    mbar_init(drain_bar, 1);
    *abort_flag = 0;
    fence_barrier_init();
    prefetch_tensormap(&tmA);
    prefetch_tensormap(&tmB);
    prefetch_tensormap(&tmC);
  }
  if (warp == 1) {
    tmem_alloc(smem_u32(tmem_slot), Cfg::TMEM_COLS);
    tmem_relinquish_alloc_permit();
  }
  tc_fence_before_sync();
  __syncthreads();
  tc_fence_after_sync();
  const uint32_t tmem_base = *tmem_slot;
  // operands and the epilogue's inputs may come from the previous launch
  grid_dependency_wait();
  grid_launch_dependents();

  if (warp == 0) {
    // ------------------------------------------------------ TMA producer
    if (elect_one()) {
      int stage = 0;
      uint32_t phase = 0;
      int issued = 0;
      for (int kb = 0; kb < p.num_kb; ++kb) {
        if (!wait_phase(empty_bar(stage), phase ^ 1u, wd, kWdProducerEmpty)) break;
        if (!(p.inject == 1 && issued == 0))  // testing aid: withhold one arrival
          mbar_arrive_expect_tx(full_bar(stage), Cfg::STAGE_BYTES);
        const int kx = kb * Cfg::BK;
        const uint32_t a_dst = sA + stage * Cfg::A_BYTES, b_dst = sB + stage * Cfg::B_BYTES;
        if constexpr (A_MN) {
          tma_load_2d(a_dst, &tmA, full_bar(stage), m0, kx);
          tma_load_2d(a_dst + kMnBoxBytes, &tmA, full_bar(stage), m0 + kMnBox, kx);
        } else {
          tma_load_2d(a_dst, &tmA, full_bar(stage), kx, m0);
        }
        if constexpr (B_MN)
          tma_load_2d(b_dst, &tmB, full_bar(stage), n0, kx);
        else
          tma_load_2d(b_dst, &tmB, full_bar(stage), kx, n0);
        ++issued;
        if (++stage == Cfg::STAGES) {
          stage = 0;
          phase ^= 1u;
        }
      }
      // the last loads must have landed before the CTA's memory goes away
      int s = stage;
      uint32_t ph = phase;
      for (int i = 0; i < issued && i < Cfg::STAGES; ++i) {
        if (s == 0) {
          s = Cfg::STAGES - 1;
          ph ^= 1u;
        } else {
          --s;
        }
        wait_drain(full_bar(s), ph, wd);
      }
    }
    __syncwarp();
  } else if (warp == 1) {
    // ------------------------------------------------------- MMA issuer
    if (elect_one()) {
      const uint64_t a_base = A_MN ? sdesc_mnmajor_sw128(sA) : sdesc_kmajor_sw128(sA);
      const uint64_t b_base = B_MN ? sdesc_mnmajor_sw128(sB) : sdesc_kmajor_sw128(sB);
      const uint32_t a_step = A_MN ? 128u : 2u, b_step = B_MN ? 128u : 2u;
      constexpr uint32_t idesc = Cfg::IDESC | idesc_major_bits(A_MN, B_MN);
      int stage = 0;
      uint32_t phase = 0;
      bool ok = true;
      for (int kb = 0; kb < p.num_kb; ++kb) {
        if (!wait_phase(full_bar(stage), phase, wd, kWdMmaFull)) {
          ok = false;
          break;
        }
        tc_fence_after_sync();
        const uint64_t a_desc = a_base + static_cast<uint32_t>(stage * (Cfg::A_BYTES >> 4));
        const uint64_t b_desc = b_base + static_cast<uint32_t>(stage * (Cfg::B_BYTES >> 4));
#pragma unroll
        for (int k = 0; k < Cfg::BK / Cfg::UMMA_K; ++k)
          mma_f16_ss(tmem_base, a_desc + a_step * k, b_desc + b_step * k, idesc, (kb > 0 || k > 0) ? 1u : 0u);
        mma_commit(empty_bar(stage));
        if (++stage == Cfg::STAGES) {
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
    // --------------------------------------------------------- epilogue
    const int q = warp & 3;  // TMEM lanes and tile rows 32q .. 32q+31
    uint8_t* box = smem + Cfg::OFF_C + q * Cfg::C_BOX_BYTES;
    const int y0 = m0 + q * kEpiRows;
    const bool inside = n0 < p.N && y0 < p.M;
    LinSide<EPI> side;
    if (inside) lin_fetch<EPI>(side, p.lin, lane, p.M, p.N, static_cast<int64_t>(y0) + lane, n0);
    if constexpr (A_MN) {
      if (summed) sum_rows(p, smem, full_bar(0), empty_bar(0), nb, m0 + nb * kMnBox, wd);
    }
    int ok = 1;
    if (lane == 0) ok = wait_phase(accf_bar, 0, wd, kWdEpiAccFull) ? 1 : 0;
    ok = __shfl_sync(0xffffffffu, ok, 0);
    if (ok && inside) {
      tc_fence_after_sync();
      f32x2 v[32];
      tmem_row64(tmem_base + (static_cast<uint32_t>(q * 32) << 16), v);
      lin_row64<EPI>(box, lane, v, side, p.lin, p.M, p.N, static_cast<int64_t>(y0) + lane, n0);
      fence_proxy_async_smem();
      __syncwarp();
      if (lane == 0) {
        tma_store_2d(&tmC, smem_u32(box), n0, y0);
        bulk_commit_group();
        bulk_wait_group_read<0>();  // staging read; the writes finish with the grid
      }
      __syncwarp();
    }
  }

  tc_fence_before_sync();
  __syncthreads();
  tc_fence_after_sync();
  if (warp == 1) tmem_dealloc(tmem_base, Cfg::TMEM_COLS);
}

cudaError_t prepare(const void* kern) {
  return cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, WaveCfg::SMEM_BYTES);
}

}  // namespace

cudaError_t launch_linear_wave(const CUtensorMap& a, const CUtensorMap& b, const CUtensorMap& c, const TcArgs& args,
                                  Epilogue kind, cudaStream_t stream) {
  static std::atomic<bool> attr_done[3][64];
  // the forward product, the input gradient, the weight gradient
  const int which = kind == kEpiLinearGrad ? 1 : args.a_mn ? 2 : 0;
  if (args.a_mn != (which == 2) || args.b_mn != (which != 0)) return cudaErrorInvalidValue;
  auto kern = which == 0   ? linear_wave_kernel<kEpiLinear, false, false>
              : which == 1 ? linear_wave_kernel<kEpiLinearGrad, false, true>
                           : linear_wave_kernel<kEpiLinear, true, true>;
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  if (dev < 0 || dev >= 64 || !attr_done[which][dev]) {
    if ((e = prepare(reinterpret_cast<const void*>(kern))) != cudaSuccess) return e;
    if (dev >= 0 && dev < 64) attr_done[which][dev] = true;
  }
  PdlLaunch l(dim3(static_cast<unsigned>(args.grid)), dim3(WaveCfg::THREADS), WaveCfg::SMEM_BYTES, stream);
  return cudaLaunchKernelEx(&l.cfg, kern, a, b, c, args);
}

// The -DHGEMM_DEBUG build's check word of this file (null otherwise).
HG_DEBUG_WORD_ACCESSOR(linear_wave)

}  // namespace hg
