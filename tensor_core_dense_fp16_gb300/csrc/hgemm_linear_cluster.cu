// hgemm_linear_cluster.cu — linear layers and their gradients whose output is
// a single wave of 128×64 tiles (about a thousand rows and columns), in
// clusters of four CTAs that share their operands.
//
// Such a product reads each operand many times from L2 (1000^3: 50 MB for 6 MB
// of operands and output), and rows that start on odd multiples of 16 bytes
// cost L2 almost twice. Here the CTAs of a cluster compute 2×2 neighbouring
// tiles. Each loads half of its A tile and half of its B tile and multicasts
// them to the CTA beside it in its row and in its column, so that half the
// bytes leave L2. A stage is free for the next loads once the MMAs of all three
// CTAs that receive them have read it (their commits arrive on the loader's
// empty barrier). The operand order is a template parameter: a branch on it
// between the copies took them out of uniform registers (a block of 64 of the
// contraction: 0.155 us, 0.115 without).
//
// Measured (us, in a graph, operands in L2), against the kernels of larger
// outputs: 1000^3 with bias, SiLU and residual 8.8 to 6.6, its input gradient
// with SiLU's and f(û) 9.6 to 7.0, its weight gradient 7.8 to 5.9 (with bias
// 11.1 to 7.1); 1024^3 without epilogue 5.1 to 4.8; 1024×1024, contraction 4096,
// 13.1 to 11.7; the one loss found is 1000×1000 with rows of 4000, 13.1 to 13.9.
// Of the 6.6 us, about 3 are launch and set-up, 2.2 the copies of 16 blocks, and
// 1.2 the epilogue: its two special-function instructions per SiLU occupy their
// unit for 1,024 cycles.
#include <atomic>

#include "internal.h"
#include "kernel_common.cuh"
#include "linear_epilogue.cuh"
#include "ptx.cuh"

namespace hg {
namespace {

struct ClCfg {
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
  static constexpr int OFF_BAR = OFF_SUM + EPI_WARPS * (BM / 2) * 4;
  static constexpr int NUM_BARS = 2 * STAGES + 2;  // full, empty, accumulator full, drain
  static constexpr int OFF_MISC = OFF_BAR + NUM_BARS * 8;
  static constexpr int SMEM_BYTES = OFF_MISC + 16 + 1024;
  static constexpr int THREADS = 192;
  static constexpr int TMEM_COLS = BN;
  static constexpr uint32_t IDESC = idesc_f16_f32acc(BM, BN);
  static_assert(A_BYTES % 2048 == 0 && B_BYTES % 2048 == 0, "halves of tiles are 1024-byte aligned");
  static_assert(BM == 2 * kMnBox && BN == kMnBox, "half an A tile is one MN-major box");
  static_assert(SMEM_BYTES <= 232448, "exceeds 227 KB of shared memory per CTA");
};

// The sums over K of the half of the A tile that this CTA loads (64 rows), by
// the epilogue warps while the product runs: the bias gradient beside the
// weight's, from the stages in shared memory (MN-major: 64 K rows of 128
// bytes). The four warps take K blocks in turn, so that none of them delays the
// ring. A thread adds the eight rows of A of one 16-byte chunk in every fourth K
// row of its warp's blocks, and the 16 partial sums of a row are added in a
// fixed order. (A CTA's own half, because then only its own loads wait for the
// sums. A kernel of column sums beside the product took 5 us more: 1000^3,
// 6.0 us without.)
__device__ __forceinline__ void sum_rows(const TcArgs& p, uint8_t* smem, uint32_t full0, uint32_t empty0, int half,
                                         int first, const Watchdog& wd) {
  using Cfg = ClCfg;
  const int t = static_cast<int>(threadIdx.x) - 64, lane = t & 31;
  const int chunk = t & 7, k0 = lane >> 3;
  const uint8_t* tile = smem + Cfg::OFF_A + half * kMnBoxBytes;
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
  if (t < kMnBox && first + t < p.M) {
    float total = 0.f;
#pragma unroll
    for (int w = 0; w < Cfg::EPI_WARPS; ++w) total += part[w * kMnBox + t];
    float* out = p.row_sums + first + t;
    *out = p.row_sums_add ? *out + total : total;
  }
}

// A_MN, B_MN: the operand is stored with its rows contiguous (K×M, K×N).
template <int EPI, bool A_MN, bool B_MN>
__global__ void __cluster_dims__(4, 1, 1) __launch_bounds__(ClCfg::THREADS, 1)
    linear_cluster_kernel(const __grid_constant__ CUtensorMap tmA, const __grid_constant__ CUtensorMap tmB,
                          const __grid_constant__ CUtensorMap tmC, const TcArgs p) {
  using Cfg = ClCfg;
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
  const int rank = static_cast<int>(cluster_ctarank());
  const int cluster = static_cast<int>(blockIdx.x) >> 2;
  const int clusters_m = (p.num_m + 1) >> 1;
  const int rm = rank & 1, rn = rank >> 1;  // this CTA's tile of the 2×2
  const int m0 = (2 * (cluster % clusters_m) + rm) * Cfg::BM;
  const int n0 = (2 * (cluster / clusters_m) + rn) * Cfg::BN;
  const uint16_t same_m = static_cast<uint16_t>(0x5u << rm);       // the two CTAs of these rows
  const uint16_t same_n = static_cast<uint16_t>(0x3u << (2 * rn));  // the two CTAs of these columns
  // sums of A's rows over K: computed in the first column of tiles
  const bool summed = A_MN && p.row_sums && cluster / clusters_m == 0;
  const Watchdog wd{abort_flag, p.status, p.timeout_ns};

  if (threadIdx.x == 0) {
    for (int s = 0; s < Cfg::STAGES; ++s) {
      mbar_init(full_bar(s), 1);   // the producer's arrive.expect_tx (+ the bytes of three CTAs)
      // commits of the CTAs that received this CTA's halves, and its own
      // summing warp
      mbar_init(empty_bar(s), summed ? 4 : 3);
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
  cluster_sync_after_init();  // copies and commits reach the other CTAs' barriers
  tc_fence_after_sync();
  const uint32_t tmem_base = *tmem_slot;
  // operands and the epilogue's inputs may come from the previous launch
  grid_dependency_wait();
  grid_launch_dependents();

  if (warp == 0) {
    // ------------------------------------------------------ TMA producer
    if (elect_one()) {
      // this CTA's halves: rows 64·rn.. of the A tile, rows 32·rm.. of the B
      // tile. K-major they are rows of 128 bytes; MN-major a tile is boxes of
      // 64 M or N by 64 K rows of 128 bytes, A's two halves being the two boxes
      // and B's the K rows 32·rm.. of its box.
      const uint32_t a_dst = sA + static_cast<uint32_t>(rn) * (Cfg::A_BYTES / 2);
      const uint32_t b_dst = sB + static_cast<uint32_t>(rm) * (Cfg::B_BYTES / 2);
      const int ya = m0 + rn * (Cfg::BM / 2), yb = n0 + rm * (Cfg::BN / 2);
      int stage = 0;
      uint32_t phase = 0;
      int issued = 0;
      for (int kb = 0; kb < p.num_kb; ++kb) {
        if (!wait_phase(empty_bar(stage), phase ^ 1u, wd, kWdProducerEmpty)) break;
        if (!(p.inject == 1 && issued == 0))  // testing aid: withhold one arrival
          mbar_arrive_expect_tx(full_bar(stage), Cfg::STAGE_BYTES);
        const int kx = kb * Cfg::BK;
        if constexpr (A_MN)
          tma_load_2d_multicast(a_dst + stage * Cfg::A_BYTES, &tmA, full_bar(stage), ya, kx, same_m);
        else
          tma_load_2d_multicast(a_dst + stage * Cfg::A_BYTES, &tmA, full_bar(stage), kx, ya, same_m);
        if constexpr (B_MN)
          tma_load_2d_multicast(b_dst + stage * Cfg::B_BYTES, &tmB, full_bar(stage), n0, kx + rm * (Cfg::BK / 2), same_n);
        else
          tma_load_2d_multicast(b_dst + stage * Cfg::B_BYTES, &tmB, full_bar(stage), kx, yb, same_n);
        ++issued;
        if (++stage == Cfg::STAGES) {
          stage = 0;
          phase ^= 1u;
        }
      }
      // Drain: once the last stages are free again, all that this CTA sent has
      // been read, and nothing more arrives here, bytes or commits.
      int s = stage;
      uint32_t ph = phase;
      for (int i = 0; i < issued && i < Cfg::STAGES; ++i) {
        if (s == 0) {
          s = Cfg::STAGES - 1;
          ph ^= 1u;
        } else {
          --s;
        }
        if (!wait_drain(empty_bar(s), ph, wd)) break;
      }
      // After a wait that gave up: the other CTAs' last copies and commits to
      // this one are under way or will never be issued.
      if (*abort_flag) {
        const uint64_t t0 = globaltimer_ns();
        while (globaltimer_ns() - t0 < 100000u) {
        }
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
      const uint16_t readers = same_m | same_n;  // the CTAs whose loads this stage held
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
        mma_commit_multicast(empty_bar(stage), readers);
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
      if (summed) sum_rows(p, smem, full_bar(0), empty_bar(0), rn, m0 + rn * kMnBox, wd);
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
  return cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, ClCfg::SMEM_BYTES);
}

}  // namespace

int linear_cluster_max(int num_sms) {
  static std::atomic<int> cached[64];
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= 64) return 0;
  if (cached[dev] > 0) return cached[dev];
  auto kern = linear_cluster_kernel<kEpiLinear, false, false>;
  int n = 0;
  if (prepare(reinterpret_cast<const void*>(kern)) == cudaSuccess) {
    PdlLaunch l(dim3(static_cast<unsigned>(num_sms / 4 * 4)), dim3(ClCfg::THREADS), ClCfg::SMEM_BYTES, nullptr);
    if (cudaOccupancyMaxActiveClusters(&n, kern, &l.cfg) != cudaSuccess) n = 0;
  }
  (void)cudaGetLastError();
  if (n <= 0) n = 1;
  cached[dev] = n;
  return n;
}

cudaError_t launch_linear_cluster(const CUtensorMap& a, const CUtensorMap& b, const CUtensorMap& c, const TcArgs& args,
                                  Epilogue kind, cudaStream_t stream) {
  static std::atomic<bool> attr_done[3][64];
  // the forward product, the input gradient, the weight gradient
  const int which = kind == kEpiLinearGrad ? 1 : args.a_mn ? 2 : 0;
  if (args.a_mn != (which == 2) || args.b_mn != (which != 0)) return cudaErrorInvalidValue;
  auto kern = which == 0   ? linear_cluster_kernel<kEpiLinear, false, false>
              : which == 1 ? linear_cluster_kernel<kEpiLinearGrad, false, true>
                           : linear_cluster_kernel<kEpiLinear, true, true>;
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  if (dev < 0 || dev >= 64 || !attr_done[which][dev]) {
    if ((e = prepare(reinterpret_cast<const void*>(kern))) != cudaSuccess) return e;
    if (dev >= 0 && dev < 64) attr_done[which][dev] = true;
  }
  PdlLaunch l(dim3(static_cast<unsigned>(args.grid)), dim3(ClCfg::THREADS), ClCfg::SMEM_BYTES, stream);
  return cudaLaunchKernelEx(&l.cfg, kern, a, b, c, args);
}

// The -DHGEMM_DEBUG build's check word of this file (null otherwise).
HG_DEBUG_WORD_ACCESSOR(linear_cluster)

}  // namespace hg
