// hgemm_linear_any.cu — products with a linear layer's epilogue (forward,
// input gradient, weight gradient) for operands and outputs that TMA cannot
// describe: odd feature counts, pitches that are not multiples of 8, bases
// that are not 16-byte aligned.
//
// The tensor-core pipeline is the usual one: a ring of 64-wide K blocks in
// 128-byte-swizzled shared memory, tcgen05.mma into one of two FP32
// accumulators, an epilogue that drains the other. What differs is who fills
// the ring. An operand's tile of a K block is 128 segments of 128 bytes: rows
// of 64 k, or (an M- or N-contiguous operand) for each of 64 k two runs of 64
// rows, which is TMA's MN-major layout. A loader warp copies the nine aligned
// 16-byte pieces that each of its segments touches into a buffer of its own,
// two K blocks ahead (asynchronous copies: what is under way occupies no
// registers), then shifts them into the tile, eight lanes to a segment. How far
// is the same in every K block (a block is 128 bytes on, or 64 pitches), so a
// lane keeps its pointers and its shifts for a whole output tile. Bound by
// the loaders' instructions: a K block takes them 1.3 us (8192×2049 outputs of
// a contraction of 2047, GELU and residual: 371 us, where 8192×2048 of 2048 takes
// the aligned kernels 49; 1001^3 41). Where only the outputs are odd, one thread
// loads the tiles by TMA instead and four of the loader warps join the epilogue
// (2000×2001, contraction 2000: 38 us, by the loader warps 102).
// Nothing past a matrix's last element is read, and before its first one at
// most the rest of the same aligned 16 bytes; what a tile has outside the
// matrix is zeros.
#include <atomic>

#include <cuda_fp16.h>

#include "internal.h"
#include "kernel_common.cuh"
#include "linear_epilogue.cuh"
#include "ptx.cuh"

namespace hg {
namespace {

struct AnyCfg {
  static constexpr int BM = 128, BN = 128, BK = 64, STAGES = 3, UMMA_K = 16;
  static constexpr int TILE_BYTES = 128 * BK * 2;  // of either operand
  static constexpr int STAGE_BYTES = 2 * TILE_BYTES;
  static constexpr int LOADERS = 16;                // warps 0 .. 15
  static constexpr int SEGMENTS = 128 / LOADERS;    // of each operand, per loader warp
  static constexpr int EPI_WARPS = 4;               // warps 16 .. 19: TMEM lanes 32·(w % 4)
  static constexpr int MMA_WARP = LOADERS + EPI_WARPS;
  static constexpr int THREADS = (MMA_WARP + 1) * 32;
  static constexpr int TMEM_COLS = 2 * BN;
  // the epilogue turns 32 rows × 16 columns around per warp (rows of 17
  // words), beside the rows' scales
  static constexpr int TURN_COLS = 16;
  static constexpr int TURN_WORDS = 32 * (TURN_COLS + 1) + 2 * 32;
  // ... or, where the outputs are aligned, stages 32 rows × 64 columns
  static constexpr int BOX_BYTES = 32 * 128;
  static_assert(BOX_BYTES >= TURN_WORDS * 4, "either fits");
  // the pieces of a loader warp's segments of either operand
  static constexpr int PIECES = 2 * SEGMENTS * 9;
  static constexpr int RAW_STAGES = 3;
  static constexpr int RAW_BYTES = PIECES * 16;  // of a warp and K block
  static constexpr int OFF_RAW = STAGES * STAGE_BYTES;
  // with tensor maps the buffers are ring as well, and staging of four more
  // epilogue warps, which are otherwise loaders
  static constexpr int TMA_STAGES = 5;
  static constexpr int OFF_TURN = OFF_RAW + LOADERS * RAW_STAGES * RAW_BYTES;
  static constexpr int OFF_BAR = OFF_TURN + EPI_WARPS * BOX_BYTES;
  // A cluster that splits K: the first CTA receives the others' accumulators
  // where its ring and buffers were.
  static constexpr int MOST_SPLIT = 3;
  static constexpr int PART_BYTES = BM * BN * 4;
  static_assert((MOST_SPLIT - 1) * PART_BYTES <= TMA_STAGES * STAGE_BYTES, "before the staging boxes");
  // full, empty, accumulator full ×2 and empty ×2, drain, ready to receive, received
  static constexpr int NUM_BARS = 2 * TMA_STAGES + 7;
  static constexpr int OFF_MISC = OFF_BAR + NUM_BARS * 8;
  static constexpr int SMEM_BYTES = OFF_MISC + 16 + 1024;
  static constexpr uint32_t IDESC = idesc_f16_f32acc(BM, BN);
  static_assert(TMA_STAGES * STAGE_BYTES + EPI_WARPS * BOX_BYTES <= OFF_TURN, "the ring of tensor-map loads fits");
  static_assert(OFF_BAR % 8 == 0, "aligned barriers");
  static_assert(SMEM_BYTES <= 232448, "exceeds 227 KB of shared memory per CTA");
};

struct AnyArgs {
  LinearProduct p;
  int64_t num_m, num_n, units;
  int num_kb;
  int wide;  // the epilogue can read and write eight columns at a time
  int tma;   // tensor maps describe the operands
  int split;  // CTAs of a cluster per unit, each a run of K blocks
  int* status;
  unsigned long long timeout_ns;
  int inject;  // HGEMM_INJECT_* (testing the watchdog)
};

// One operand: element (i, k) at p[i·ld + k], or p[k·ld + i] when mn.
struct AnyOperand {
  const uint16_t* p;
  const uint16_t* end;  // past its last element
  int64_t ld, rows, K;
  bool mn;
  bool aligned;  // every segment begins on 16 bytes
};

constexpr int kAnyGroups = AnyCfg::SEGMENTS / 4;  // of four segments, eight lanes each
constexpr int kAnyCopies = (AnyCfg::PIECES + 31) / 32;

__device__ __forceinline__ int any_clamp(int64_t v, int most) {
  return v < 0 ? 0 : (v < most ? static_cast<int>(v) : most);
}

// A loader warp's segments of an operand's block: segment j starts at
// src + j·ld.
struct AnySegments {
  const uint16_t* src;
  int64_t left;  // K that remains: of the segments' elements, or (mn) of the segments
  int fixed;     // rows that are inside: segments, or (mn) elements
};
__device__ __forceinline__ AnySegments any_start(const AnyOperand& o, int warp, int64_t i0) {
  const int s = warp * AnyCfg::SEGMENTS;
  const int64_t i = o.mn ? i0 + (s & 64) : i0 + s, k = o.mn ? s & 63 : 0;
  return AnySegments{o.p + (o.mn ? k * o.ld + i : i * o.ld), o.K - k,
                     any_clamp(o.rows - i, o.mn ? 64 : AnyCfg::SEGMENTS)};
}
// How many elements into its first aligned piece a segment begins.
__device__ __forceinline__ int any_shift(const uint16_t* segment) {
  return static_cast<int>(reinterpret_cast<uintptr_t>(segment) >> 1) & 7;
}

// The checking build: a piece lies between the 16 bytes in which the matrix
// begins and its end.
__device__ __forceinline__ bool any_inside([[maybe_unused]] const AnyOperand& o, [[maybe_unused]] const uint16_t* at,
                                           [[maybe_unused]] int elements) {
  [[maybe_unused]] const uint16_t* begin = o.p - any_shift(o.p);
  return HG_DBG_ALIGN(at, 16) && HG_DBG_INDEX(at - begin, o.end - begin) &&
         HG_DBG_INDEX(at + elements - 1 - begin, o.end - begin);
}

// One aligned piece at an edge on its way into the warp's buffer: what is past
// the matrix's last element is not read and becomes zeros.
__device__ __forceinline__ void any_copy_edge(const AnyOperand& o, const uint16_t* at, uint32_t dst) {
  const int elements = any_clamp(o.end - at, 8);
  if (elements > 0 && !any_inside(o, at, elements)) return;
  cp_async_16(dst, elements > 0 ? at : o.p - any_shift(o.p), 2 * elements);
}

// The pieces of an operand's segments from the buffer into its tile. count,
// valid: the elements of a segment and the segments that are inside.
__device__ __forceinline__ void any_shift_in(const uint8_t* raw, const int (&shift)[kAnyGroups], bool aligned, int count, int valid,
                                             uint8_t* tile, int warp, int lane) {
  using Cfg = AnyCfg;
  // (a warp's first segment is a multiple of 8: segment j's swizzle is j % 8)
  static_assert(Cfg::SEGMENTS % 8 == 0, "the swizzle of a warp's segments");
#pragma unroll
  for (int g = 0; g < kAnyGroups; ++g) {
    const int j = 4 * g + (lane >> 3);
    const uint4* from = reinterpret_cast<const uint4*>(raw) + j * 9 + (lane & 7);
    uint32_t v[4];
    const uint4 lo = from[0];
    if (aligned) {
      v[0] = lo.x, v[1] = lo.y, v[2] = lo.z, v[3] = lo.w;
    } else {
      const uint4 hi = from[1];
      // words shift / 2 .. of the eight, half a word on for an odd shift
      const uint32_t w[8] = {lo.x, lo.y, lo.z, lo.w, hi.x, hi.y, hi.z, hi.w};
      const bool two = (shift[g] & 4) != 0, one = (shift[g] & 2) != 0;
      uint32_t x[6], y[5];
#pragma unroll
      for (int i = 0; i < 6; ++i) x[i] = two ? w[i + 2] : w[i];
#pragma unroll
      for (int i = 0; i < 5; ++i) y[i] = one ? x[i + 1] : x[i];
      const uint32_t bits = static_cast<uint32_t>(shift[g] & 1) << 4;
#pragma unroll
      for (int i = 0; i < 4; ++i) v[i] = __funnelshift_r(y[i], y[i + 1], bits);
    }
    if (count < 64 || valid < Cfg::SEGMENTS) {
      const int left = j < valid ? count - 8 * (lane & 7) : 0;
#pragma unroll
      for (int i = 0; i < 4; ++i) v[i] = 2 * i + 1 < left ? v[i] : 2 * i < left ? v[i] & 0xFFFFu : 0u;
    }
    *reinterpret_cast<uint4*>(tile + (warp * Cfg::SEGMENTS + j) * 128 + (((lane & 7) ^ (j & 7)) << 4)) =
        make_uint4(v[0], v[1], v[2], v[3]);
  }
}

// The first row and column of unit t.
struct AnyUnit {
  int64_t m0, n0;
};
__device__ __forceinline__ AnyUnit any_unit(const AnyArgs& a, int64_t t) {
  int mb, nb;
  tile_coords(static_cast<int>(t), static_cast<int>(a.num_m), static_cast<int>(a.num_n), 12, mb, nb);
  return AnyUnit{static_cast<int64_t>(mb) * AnyCfg::BM, static_cast<int64_t>(nb) * AnyCfg::BN};
}

// The epilogue of 32 rows from m0 and 16 columns, turned around in shared
// memory: this lane's column n, rows m0 + (lane / 16) + 2i.
template <bool BACKWARD>
__device__ __noinline__ void any_columns(const LinearProduct& p, const float* turn, const float* row_scale,
                                         const float* row_inv, int64_t m0, int64_t n, float bias, int lane) {
  constexpr int PITCH = AnyCfg::TURN_COLS + 1;
  const LinEpi& e = p.epi;
  const int r0 = lane >> 4;
  const int64_t m = m0 + r0;
  // rows of this lane that are inside: i < count
  int count = n < p.N ? any_clamp((p.M - m + 1) / 2, 16) : 0;
  if (count > 0 && !(HG_DBG_INDEX(n, p.N) && HG_DBG_INDEX(m + 2 * (count - 1), p.M))) count = 0;
  turn += r0 * PITCH + (lane & 15);
  row_scale += r0;
  row_inv += r0;
  uint32_t side[16];  // residual, or codes
#pragma unroll
  for (int i = 0; i < 16; ++i) side[i] = 0u;
  if (BACKWARD && e.codes) {
    const int8_t* q = e.codes + m * e.ldq + n;
#pragma unroll
    for (int i = 0; i < 16; ++i, q += 2 * e.ldq)
      if (i < count) side[i] = static_cast<uint8_t>(*q);
  } else if (!BACKWARD && e.res) {
    const uint16_t* r = e.res + m * e.ldr + n;
#pragma unroll
    for (int i = 0; i < 16; ++i, r += 2 * e.ldr)
      if (i < count) side[i] = *r;
  }
  uint16_t* c = p.C + m * p.ldc + n;
  int8_t* q = e.codes + m * e.ldq + n;
  uint16_t* h = e.h + m * e.ldh + n;
  with_activation(!BACKWARD || e.codes ? e.act : HGEMM_ACT_NONE, [&](auto a) {
#pragma unroll
    for (int i = 0; i < 16; i += 2) {
      const f32x2 x = pair_of(turn[2 * i * PITCH], turn[(2 * i + 2) * PITCH]);
      f32x2 y, f = 0;
      if constexpr (BACKWARD) {
        y = x;
        if (e.codes) {
          f32x2 df;
          activate<decltype(a)::value, true>(
              pair_of(static_cast<float>(static_cast<int8_t>(side[i])) * row_scale[2 * i],
                      static_cast<float>(static_cast<int8_t>(side[i + 1])) * row_scale[2 * i + 2]), f, df);
          y = mul2(y, df);
        }
      } else {
        const f32x2 u = add2(x, pair_of(bias));
        if (e.codes) {
          float ua, ub;
          unpair(u, ua, ub);
          const float ia = row_inv[2 * i], ib = row_inv[2 * i + 2];
          if (i < count) q[0] = static_cast<int8_t>(ia == 0.f ? 0u : ckpt_code(ua, ia));
          if (i + 1 < count) q[2 * e.ldq] = static_cast<int8_t>(ib == 0.f ? 0u : ckpt_code(ub, ib));
          q += 4 * e.ldq;
        }
        f32x2 df;
        activate<decltype(a)::value, false>(u, y, df);
        y = add2(y, unpack_half2(side[i] | side[i + 1] << 16));
      }
      const uint32_t packed = pack_half2(y);
      if (i < count) c[0] = static_cast<uint16_t>(packed);
      if (i + 1 < count) c[2 * p.ldc] = static_cast<uint16_t>(packed >> 16);
      c += 4 * p.ldc;
      if (BACKWARD && e.h) {
        const uint32_t hid = pack_half2(f);
        if (i < count) h[0] = static_cast<uint16_t>(hid);
        if (i + 1 < count) h[2 * e.ldh] = static_cast<uint16_t>(hid >> 16);
        h += 4 * e.ldh;
      }
    }
  });
}

// SHARED: the CTAs of a cluster share the K of a unit.
template <bool BACKWARD, bool SHARED>
__global__ void __launch_bounds__(AnyCfg::THREADS, 1)
    linear_any_kernel(const __grid_constant__ CUtensorMap tmA, const __grid_constant__ CUtensorMap tmB, const AnyArgs a) {
  using Cfg = AnyCfg;
  extern __shared__ uint8_t smem_raw[];
  const uint32_t raw_addr = smem_u32(smem_raw);
  uint8_t* smem = smem_raw + ((1024u - (raw_addr & 1023u)) & 1023u);
  const uint32_t sbase = smem_u32(smem);
  const uint32_t bar0 = sbase + Cfg::OFF_BAR;
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(smem + Cfg::OFF_MISC);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(smem + Cfg::OFF_MISC + 4);
  auto full_bar = [&](int s) { return bar0 + 8u * s; };
  auto empty_bar = [&](int s) { return bar0 + 8u * (Cfg::TMA_STAGES + s); };
  auto accf_bar = [&](int b) { return bar0 + 8u * (2 * Cfg::TMA_STAGES + b); };
  auto acce_bar = [&](int b) { return bar0 + 8u * (2 * Cfg::TMA_STAGES + 2 + b); };
  const uint32_t drain_bar = bar0 + 8u * (2 * Cfg::TMA_STAGES + 4);
  const uint32_t ready_bar = drain_bar + 8u, recv_bar = drain_bar + 16u;
  const int split = SHARED ? a.split : 1, rank = SHARED ? static_cast<int>(cluster_ctarank()) : 0;
  const int64_t unit0 = blockIdx.x / split, unit_step = gridDim.x / split;
  const int kb0 = static_cast<int>(static_cast<int64_t>(a.num_kb) * rank / split);
  const int kb1 = static_cast<int>(static_cast<int64_t>(a.num_kb) * (rank + 1) / split);
  const int stages = a.tma ? Cfg::TMA_STAGES : Cfg::STAGES;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const Watchdog wd{abort_flag, a.status, a.timeout_ns};
  const LinearProduct& p = a.p;

  if (threadIdx.x == 0) {
    for (int s = 0; s < stages; ++s) {
      mbar_init(full_bar(s), a.tma ? 1 : Cfg::LOADERS);  // the producer, or one arrival per loader warp
      mbar_init(empty_bar(s), 1);            // tcgen05.commit
    }
    for (int b = 0; b < 2; ++b) {
      mbar_init(accf_bar(b), 1);               // tcgen05.commit
      mbar_init(acce_bar(b), a.tma ? 2 * Cfg::EPI_WARPS : Cfg::EPI_WARPS);  // one arrival per epilogue warp
    }
    mbar_init(drain_bar, 1);
    mbar_init(ready_bar, 1);
    mbar_init(recv_bar, SHARED ? (split - 1) * Cfg::EPI_WARPS : 1);
    *abort_flag = 0;
    fence_barrier_init();
  }
  if (warp == Cfg::MMA_WARP) {
    tmem_alloc(smem_u32(tmem_slot), Cfg::TMEM_COLS);
    tmem_relinquish_alloc_permit();
  }
  tc_fence_before_sync();
  __syncthreads();
  if (SHARED) cluster_sync_after_init();
  tc_fence_after_sync();
  const uint32_t tmem_base = *tmem_slot;
  grid_dependency_wait();
  grid_launch_dependents();

  if (a.tma && warp < Cfg::LOADERS - Cfg::EPI_WARPS) {
    // ------------------------------- TMA producer (only the outputs are odd)
    if (warp == 0 && elect_one()) {
      int stage = 0;
      uint32_t phase = 0;
      long long issued = 0;
      bool ok = true;
      for (int64_t t = unit0; ok && t < a.units; t += unit_step) {
        const AnyUnit u = any_unit(a, t);
        const int m0 = static_cast<int>(u.m0), n0 = static_cast<int>(u.n0);
        for (int kb = kb0; kb < kb1; ++kb) {
          ok = wait_phase(empty_bar(stage), phase ^ 1u, wd, kWdProducerEmpty);
          if (!ok) break;
          if (!(a.inject == 1 && issued == 0))  // testing aid: withhold one arrival
            mbar_arrive_expect_tx(full_bar(stage), Cfg::STAGE_BYTES);
          const uint32_t sa = sbase + stage * Cfg::STAGE_BYTES, sb = sa + Cfg::TILE_BYTES;
          const int kx = kb * Cfg::BK;
          if (p.a_mn) {
            tma_load_2d(sa, &tmA, full_bar(stage), m0, kx);
            tma_load_2d(sa + kMnBoxBytes, &tmA, full_bar(stage), m0 + kMnBox, kx);
          } else {
            tma_load_2d(sa, &tmA, full_bar(stage), kx, m0);
          }
          if (p.b_mn) {
            tma_load_2d(sb, &tmB, full_bar(stage), n0, kx);
            tma_load_2d(sb + kMnBoxBytes, &tmB, full_bar(stage), n0 + kMnBox, kx);
          } else {
            tma_load_2d(sb, &tmB, full_bar(stage), kx, n0);
          }
          ++issued;
          if (++stage == stages) {
            stage = 0;
            phase ^= 1u;
          }
        }
      }
      // the last loads must have landed before the CTA's memory goes away
      int s = stage;
      uint32_t ph = phase;
      for (long long i = 0; i < issued && i < stages; ++i) {
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
  } else if (!a.tma && warp < Cfg::LOADERS) {
    // ------------------------------------------------------------ loaders
    auto operand = [&](const uint16_t* q, int64_t ld, int64_t rows, bool mn) {
      const uint16_t* end = q + (mn ? (p.K - 1) * ld + rows : (rows - 1) * ld + p.K);
      return AnyOperand{q, end, ld, rows, p.K, mn, (reinterpret_cast<uintptr_t>(q) & 15u) == 0 && ld % 8 == 0};
    };
    const AnyOperand oa = operand(p.A, p.lda, p.M, p.a_mn), ob = operand(p.B, p.ldb, p.N, p.b_mn);
    const int64_t step_a = oa.mn ? Cfg::BK * oa.ld : Cfg::BK, step_b = ob.mn ? Cfg::BK * ob.ld : Cfg::BK;
    uint8_t* raw = smem + Cfg::OFF_RAW + warp * Cfg::RAW_STAGES * Cfg::RAW_BYTES;
    int stage = 0;
    uint32_t phase = 0;
    bool ok = true;
    for (int64_t t = unit0; ok && t < a.units; t += unit_step) {
      const AnyUnit u = any_unit(a, t);
      const AnySegments ca = any_start(oa, warp, u.m0), cb = any_start(ob, warp, u.n0);
      // this lane's pieces: piece i % 9 of segment i / 9, A's segments first
      const uint16_t* at[kAnyCopies];
      int shift_a[kAnyGroups], shift_b[kAnyGroups];
#pragma unroll
      for (int c = 0; c < kAnyCopies; ++c) {
        const int i = lane + 32 * c, j = i / 9;
        const uint16_t* seg = j < Cfg::SEGMENTS ? ca.src + j * oa.ld : cb.src + (j - Cfg::SEGMENTS) * ob.ld;
        at[c] = seg - any_shift(seg) + i % 9 * 8 + kb0 * (j < Cfg::SEGMENTS ? step_a : step_b);
      }
#pragma unroll
      for (int g = 0; g < kAnyGroups; ++g) {
        shift_a[g] = any_shift(ca.src + (4 * g + (lane >> 3)) * oa.ld);
        shift_b[g] = any_shift(cb.src + (4 * g + (lane >> 3)) * ob.ld);
      }
      int filled = 0;  // buffer of the next block to copy
      const uint16_t *src_a = ca.src + kb0 * step_a, *src_b = cb.src + kb0 * step_b;  // of the next block to copy
      auto inside = [&](const AnyOperand& o, const uint16_t* src) {  // every piece
        return src + (Cfg::SEGMENTS - 1) * o.ld + 72 <= o.end;
      };
      auto copy = [&](bool some) {
        if (some) {
          const bool whole = inside(oa, src_a) && inside(ob, src_b);
          uint8_t* dst = raw + filled * Cfg::RAW_BYTES + lane * 16;
#pragma unroll
          for (int c = 0; c < kAnyCopies; ++c) {
            const int i = lane + 32 * c;
            const bool of_a = i < Cfg::PIECES / 2;
            if (i < Cfg::PIECES) {
              if (whole) {
                if (any_inside(of_a ? oa : ob, at[c], 8)) cp_async_16(smem_u32(dst + 32 * 16 * c), at[c], 16);
              } else
                any_copy_edge(of_a ? oa : ob, at[c], smem_u32(dst + 32 * 16 * c));
            }
            at[c] += of_a ? step_a : step_b;
          }
          src_a += step_a;
          src_b += step_b;
        }
        cp_async_commit();
        if (++filled == Cfg::RAW_STAGES) filled = 0;
      };
      copy(true);
      copy(kb1 - kb0 > 1);
      int used = 0;
      for (int kb = kb0; kb < kb1; ++kb) {
        // (every lane has read the buffer that this overwrites)
        __syncwarp();
        copy(kb + 2 < kb1);
        int good = 1;
        if (lane == 0) good = wait_phase(empty_bar(stage), phase ^ 1u, wd, kWdProducerEmpty) ? 1 : 0;
        ok = __shfl_sync(0xffffffffu, good, 0) != 0;
        if (!ok) break;
        cp_async_wait<2>();
        __syncwarp();
        uint8_t* tile = smem + stage * Cfg::STAGE_BYTES;
        const uint8_t* from = raw + used * Cfg::RAW_BYTES;
        const int64_t la = ca.left - static_cast<int64_t>(kb) * Cfg::BK, lb = cb.left - static_cast<int64_t>(kb) * Cfg::BK;
        any_shift_in(from, shift_a, oa.aligned, oa.mn ? ca.fixed : any_clamp(la, 64),
                     oa.mn ? any_clamp(la, Cfg::SEGMENTS) : ca.fixed, tile, warp, lane);
        any_shift_in(from + Cfg::RAW_BYTES / 2, shift_b, ob.aligned, ob.mn ? cb.fixed : any_clamp(lb, 64),
                     ob.mn ? any_clamp(lb, Cfg::SEGMENTS) : cb.fixed, tile + Cfg::TILE_BYTES, warp, lane);
        fence_proxy_async_smem();
        __syncwarp();
        // (testing aid: one warp withholds one arrival)
        if (lane == 0 && !(a.inject == 1 && warp == 0 && kb == kb0 && t == unit0)) mbar_arrive(full_bar(stage));
        if (++stage == stages) {
          stage = 0;
          phase ^= 1u;
        }
        if (++used == Cfg::RAW_STAGES) used = 0;
      }
      cp_async_wait<0>();
      __syncwarp();
    }
  } else if (warp == Cfg::MMA_WARP) {
    // -------------------------------------------------------- MMA issuer
    if (elect_one()) {
      const uint32_t idesc = Cfg::IDESC | idesc_major_bits(p.a_mn, p.b_mn);
      const uint32_t a_step = p.a_mn ? 128u : 2u, b_step = p.b_mn ? 128u : 2u;
      int stage = 0;
      uint32_t phase = 0;
      int acc = 0;
      uint32_t acc_phase = 0;
      bool ok = true;
      for (int64_t t = unit0; ok && t < a.units; t += unit_step) {
        if (!wait_phase(acce_bar(acc), acc_phase ^ 1u, wd, kWdMmaAccEmpty)) break;
        tc_fence_after_sync();
        const uint32_t d_tmem = tmem_base + static_cast<uint32_t>(acc * Cfg::BN);
        for (int kb = kb0; kb < kb1; ++kb) {
          if (!wait_phase(full_bar(stage), phase, wd, kWdMmaFull)) {
            ok = false;
            break;
          }
          tc_fence_after_sync();
          const uint32_t sa = sbase + stage * Cfg::STAGE_BYTES, sb = sa + Cfg::TILE_BYTES;
          const uint64_t a_desc = p.a_mn ? sdesc_mnmajor_sw128(sa) : sdesc_kmajor_sw128(sa);
          const uint64_t b_desc = p.b_mn ? sdesc_mnmajor_sw128(sb) : sdesc_kmajor_sw128(sb);
#pragma unroll
          for (int k = 0; k < Cfg::BK / Cfg::UMMA_K; ++k)
            mma_f16_ss(d_tmem, a_desc + a_step * k, b_desc + b_step * k, idesc, (kb > kb0 || k > 0) ? 1u : 0u);
          mma_commit(empty_bar(stage));
          if (++stage == stages) {
            stage = 0;
            phase ^= 1u;
          }
        }
        if (!ok) break;
        mma_commit(accf_bar(acc));
        acc ^= 1;
        if (acc == 0) acc_phase ^= 1u;
      }
      mma_commit(drain_bar);
      wait_drain(drain_bar, 0, wd);
    }
    __syncwarp();
  } else {
    // ----------------------------------------------------------- epilogue
    // A lane holds a row of the accumulator, but unaligned rows are best read
    // and written along the columns: 16 columns at a time go through shared
    // memory, so that a lane has 16 rows of one column, and a warp's accesses
    // are two runs of 16 neighbours. All 16 reads are under way at once.
    const LinEpi& e = p.epi;
    const int q = warp & 3;
    // with tensor maps, warps 12 .. 15 take the second 64 columns of a tile
    const bool more = warp < Cfg::LOADERS;
    const int first = more ? kCkptGroup : 0, step = a.tma ? Cfg::BN : kCkptGroup;
    uint8_t* box = smem + (more ? Cfg::TMA_STAGES * Cfg::STAGE_BYTES : Cfg::OFF_TURN) + q * Cfg::BOX_BYTES;
    float* turn = reinterpret_cast<float*>(box);
    float* row_scale = turn + 32 * (Cfg::TURN_COLS + 1);
    float* row_inv = row_scale + 32;
    auto bias_at = [&](int64_t n) {
      return !BACKWARD && e.bias && n < p.N ? __half2float(__ushort_as_half(e.bias[n])) : 0.f;
    };
    int acc = 0;
    uint32_t acc_phase = 0;
    for (int64_t t = unit0; t < a.units; t += unit_step) {
      const AnyUnit u = any_unit(a, t);
      lin_prefetch_row<BACKWARD ? kEpiLinearGrad : kEpiLinear>(e, p.M, p.N, u.m0 + q * 32 + lane, u.n0, Cfg::BN);
      int ok = 1;
      if (lane == 0) ok = wait_phase(accf_bar(acc), acc_phase, wd, kWdEpiAccFull) ? 1 : 0;
      ok = __shfl_sync(0xffffffffu, ok, 0);
      if (!ok) {
        // (the first CTA's signal may still be under way)
        if (SHARED && rank != 0 && warp == Cfg::LOADERS && lane == 0) wait_drain_cluster(ready_bar, 0, wd);
        break;
      }
      tc_fence_after_sync();
      if constexpr (SHARED) {
        const uint32_t t_row = tmem_base + (static_cast<uint32_t>(q * 32) << 16);
        // [other rank][quarter][four columns][row]
        const uint32_t part = static_cast<uint32_t>(q * (Cfg::PART_BYTES / 4) + lane * 16);
        if (rank != 0) {
          if (more) break;
          if (lane == 0) ok = wait_phase_cluster(ready_bar, 0, wd, kWdReduce) ? 1 : 0;
          ok = __shfl_sync(0xffffffffu, ok, 0);
          if (!ok) break;
          const uint32_t to = mapa_shared(sbase + static_cast<uint32_t>((rank - 1) * Cfg::PART_BYTES) + part, 0);
#pragma unroll 1
          for (int c = 0; c < Cfg::BN; c += 16) {
            float v[16];
            tmem_ld_32x32b_x16(t_row + c, v);
#pragma unroll
            for (int i = 0; i < 16; i += 4)
              st_cluster_v4(to + static_cast<uint32_t>((c + i) * 128), __float_as_uint(v[i]), __float_as_uint(v[i + 1]),
                            __float_as_uint(v[i + 2]), __float_as_uint(v[i + 3]));
          }
          __syncwarp();
          if (lane == 0) mbar_arrive_cluster(mapa_shared(recv_bar, 0));
          break;
        }
        // the ring and the buffers have been read: the accumulator is complete
        if (warp == Cfg::LOADERS && lane > 0 && lane < split)
          mbar_arrive_cluster_relaxed(mapa_shared(ready_bar, static_cast<uint32_t>(lane)));
        if (lane == 0) {
          ok = wait_phase_cluster(recv_bar, 0, wd, kWdReduce) ? 1 : 0;
          if (!ok) wait_drain_cluster(recv_bar, 0, wd);
        }
        ok = __shfl_sync(0xffffffffu, ok, 0);
        if (!ok) break;
        // the columns that this warp goes on with, summed in rank order in TMEM
        const int c1 = a.tma ? first + kCkptGroup : Cfg::BN;
#pragma unroll 1
        for (int c = first; c < c1; c += 16) {
          float v[16];
          tmem_ld_32x32b_x16(t_row + c, v);
          for (int r = 1; r < split; ++r) {
            const uint8_t* from = smem + (r - 1) * Cfg::PART_BYTES + part + c * 128;
#pragma unroll
            for (int i = 0; i < 16; i += 4) {
              const float4 w = *reinterpret_cast<const float4*>(from + i * 128);
              v[i] += w.x;
              v[i + 1] += w.y;
              v[i + 2] += w.z;
              v[i + 3] += w.w;
            }
          }
          tmem_st_32x32b_x16(t_row + c, v);
        }
      }
      const int64_t gi = u.m0 + q * 32 + lane;
      for (int64_t col0 = u.n0 + first; col0 < u.n0 + Cfg::BN && col0 < p.N; col0 += step) {
        const uint32_t t_group = tmem_base + (static_cast<uint32_t>(q * 32) << 16) +
                                 static_cast<uint32_t>(acc * Cfg::BN + static_cast<int>(col0 - u.n0));
        if (a.wide) {
          // aligned rows: the tensor-map kernels' epilogue, eight lanes
          // writing a row of the box
          constexpr int EPI = BACKWARD ? kEpiLinearGrad : kEpiLinear;
          f32x2 v[32];
          tmem_row64(t_group, v);
          __syncwarp();
          LinSide<EPI> side;
          lin_fetch<EPI>(side, e, lane, p.M, p.N, gi, col0);
          lin_row64<EPI>(box, lane, v, side, e, p.M, p.N, gi, col0);
          __syncwarp();
          const int64_t n = col0 + 8 * (lane & 7);
#pragma unroll
          for (int r = lane >> 3; r < 32; r += 4) {
            const int64_t m = u.m0 + q * 32 + r;
            if (m < p.M && n < p.N && dbg_row(p.C + m * p.ldc + n, n, 8, p.N, 16))
              *reinterpret_cast<uint4*>(p.C + m * p.ldc + n) =
                  *reinterpret_cast<const uint4*>(box + r * 128 + (((lane & 7) ^ (r & 7)) << 4));
          }
          continue;
        }
        float scale = 0.f, inv = 0.f;
        if (e.codes) {
          float* s = e.scales + col0 / kCkptGroup * e.lds + gi;
          if constexpr (BACKWARD) {
            if (gi < p.M && HG_DBG_INDEX(gi, e.lds)) scale = *s;
          } else {
            // (columns past N hold 0: zeros in the tile and no bias)
            float top = 0.f;
#pragma unroll 1
            for (int c = 0; c < kCkptGroup; c += Cfg::TURN_COLS) {
              float v[16];
              tmem_ld_32x32b_x16(t_group + c, v);
#pragma unroll
              for (int j = 0; j < 16; j += 2)
                top = max_abs3(top, v[j] + bias_at(col0 + c + j), v[j + 1] + bias_at(col0 + c + j + 1));
            }
            ckpt_scale(magnitude_bits(top), scale, inv);
            if (gi < p.M && HG_DBG_INDEX(gi, e.lds)) *s = scale;
          }
        }
        row_scale[lane] = scale;
        row_inv[lane] = inv;
#pragma unroll 1
        for (int c = 0; c < kCkptGroup; c += Cfg::TURN_COLS) {
          float v[16];
          tmem_ld_32x32b_x16(t_group + c, v);
          __syncwarp();
#pragma unroll
          for (int j = 0; j < Cfg::TURN_COLS; ++j) turn[lane * (Cfg::TURN_COLS + 1) + j] = v[j];
          __syncwarp();
          const int64_t n = col0 + c + (lane & (Cfg::TURN_COLS - 1));
          const float bias = bias_at(n);
          any_columns<BACKWARD>(p, turn, row_scale, row_inv, u.m0 + q * 32, n, bias, lane);
        }
        __syncwarp();
      }
      // this accumulator may be overwritten by the unit after next
      tc_fence_before_sync();
      __syncwarp();
      if (lane == 0) mbar_arrive(acce_bar(acc));
      acc ^= 1;
      if (acc == 0) acc_phase ^= 1u;
    }
  }

  tc_fence_before_sync();
  __syncthreads();
  tc_fence_after_sync();
  if (warp == Cfg::MMA_WARP) tmem_dealloc(tmem_base, Cfg::TMEM_COLS);
}

}  // namespace

cudaError_t launch_linear_any(const LinearProduct& p, const CUtensorMap* ma, const CUtensorMap* mb,
                              const CallDevice& dev, cudaStream_t stream) {
  using Cfg = AnyCfg;
  static std::atomic<bool> attr_done[4][64];
  AnyArgs a{};
  a.p = p;
  a.num_m = (p.M + Cfg::BM - 1) / Cfg::BM;
  a.num_n = (p.N + Cfg::BN - 1) / Cfg::BN;
  a.units = a.num_m * a.num_n;
  if (a.units > 0x7FFFFFFF - 0xFFFF) return cudaErrorInvalidValue;
  a.num_kb = static_cast<int>((p.K + Cfg::BK - 1) / Cfg::BK);
  auto rows = [](const void* q, int64_t ld, uintptr_t bytes) {
    return !q || ((reinterpret_cast<uintptr_t>(q) & (bytes - 1)) == 0 && ld % 8 == 0);
  };
  a.wide = p.N % 8 == 0 && rows(p.C, p.ldc, 16) && rows(p.epi.res, p.epi.ldr, 16) && rows(p.epi.h, p.epi.ldh, 16) &&
           rows(p.epi.codes, p.epi.ldq, 8);
  a.tma = ma ? 1 : 0;
  a.status = dev.status;
  a.timeout_ns = dev.timeout_ns;
  a.inject = dev.inject;
  // Few tiles and a long K: clusters of two or three share it, eight K blocks or
  // more each (us, without and with: 200×201×8001 217, 91; 300×1001×4097 121, 61;
  // input gradient 1000^2 over 1001 38, 31), as long as all clusters run at once:
  // those of three leave a few SMs over.
  a.split = 1;
  for (int s = Cfg::MOST_SPLIT; s > 1 && a.split == 1; --s)
    if (a.units * s <= dev.num_sms - 16 && a.num_kb >= 8 * s) a.split = s;
  const int which = (p.epi.backward ? 1 : 0) + (a.split > 1 ? 2 : 0);
  auto kern = which == 0   ? linear_any_kernel<false, false>
              : which == 1 ? linear_any_kernel<true, false>
              : which == 2 ? linear_any_kernel<false, true>
                           : linear_any_kernel<true, true>;
  int id = 0;
  cudaError_t e = cudaGetDevice(&id);
  if (e != cudaSuccess) return e;
  if (id < 0 || id >= 64 || !attr_done[which][id]) {
    e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, Cfg::SMEM_BYTES);
    if (e != cudaSuccess) return e;
    if (id >= 0 && id < 64) attr_done[which][id] = true;
  }
  PdlLaunch l(dim3(static_cast<unsigned>(a.split > 1               ? a.units * a.split
                                         : a.units < dev.num_sms ? a.units
                                                                 : dev.num_sms)),
              dim3(Cfg::THREADS), Cfg::SMEM_BYTES, stream);
  l.cluster(static_cast<unsigned>(a.split));
  const CUtensorMap none{};
  return cudaLaunchKernelEx(&l.cfg, kern, ma ? *ma : none, mb ? *mb : none, a);
}

// The -DHGEMM_DEBUG build's check word of this file (null otherwise).
HG_DEBUG_WORD_ACCESSOR(linear_any)

}  // namespace hg
