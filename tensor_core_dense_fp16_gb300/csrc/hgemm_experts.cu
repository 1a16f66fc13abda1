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
#include <atomic>

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

// An order of FP32 logits as whole numbers: larger logit, larger number, and a
// NaN below every number. 0 is left for what has been chosen.
__device__ __forceinline__ uint32_t order_key(float l) {
  const uint32_t b = __float_as_uint(l == 0.f ? 0.f : l);  // (−0 is +0)
  return l != l ? 1u : (b & 0x80000000u) ? ~b : (b | 0x80000000u);
}

// The k largest of the E logits in shared memory, by one warp: lane j < k
// leaves with choice j and its share. A lane holds every 32nd logit; a round is
// two reductions, the largest and the lowest index that has it.
__device__ __forceinline__ void choose(const float* logits, int E, int k, bool normalize, int& mine, float& share) {
  const int lane = threadIdx.x & 31;
  uint32_t key[kMost / 32];
#pragma unroll
  for (int i = 0; i < kMost / 32; ++i) key[i] = lane + 32 * i < E ? order_key(logits[lane + 32 * i]) : 0u;
  float chosen = 0.f, top = 0.f;
  mine = 0;
  for (int j = 0; j < k; ++j) {
    uint32_t best = 0u;
    int at = 0;
#pragma unroll
    for (int i = 0; i < kMost / 32; ++i)
      if (key[i] > best) {
        best = key[i];
        at = lane + 32 * i;
      }
    const uint32_t most = __reduce_max_sync(0xffffffffu, best);
    const int e = __reduce_min_sync(0xffffffffu, best == most ? at : kMost);
#pragma unroll
    for (int i = 0; i < kMost / 32; ++i)
      if (e == lane + 32 * i) key[i] = 0u;
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

// A cluster of CTAs per token: a warp per logit, the logits gathered in the
// first CTA, which chooses. The launch is bound by its latencies: a lane asks
// for eight pieces of a row at once.
template <bool VEC>
__global__ void __launch_bounds__(kThreads) experts_router_kernel(const ExpertsArgs a) {
  __shared__ float logits[kMost];
  if (a.router_ctas > 1) cluster_sync();  // the first CTA is there
  grid_dependency_wait();
  grid_launch_dependents();
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int ctas = a.router_ctas, rank = blockIdx.x % ctas, m = blockIdx.x / ctas;
  const uint32_t gather = mapa_shared(smem_u32(logits), 0);
  const uint16_t* x = a.X + m * a.ldx;
  for (int e = rank * kWarps + warp; e < a.E; e += ctas * kWarps) {
    const uint16_t* w = a.Wr + e * a.ldwr;
    float sum = 0.f;
    if constexpr (VEC) {
      constexpr int AHEAD = 8;
      for (int d0 = 8 * lane; d0 < a.D; d0 += 256 * AHEAD) {
        uint4 p[AHEAD], q[AHEAD];
        // (unconditional, or the compiler waits for one pair before it asks for
        // the next; in place of pieces past the end the row's first, not summed)
#pragma unroll
        for (int j = 0; j < AHEAD; ++j) {
          const int d = d0 + 256 * j < a.D ? d0 + 256 * j : 0;
          if (!dbg_row(w + d, d, 8, a.D, 16)) return;
          p[j] = load16(x + d);
          q[j] = load16(w + d);
        }
#pragma unroll
        for (int j = 0; j < AHEAD; ++j) {
          if (d0 + 256 * j >= a.D) break;
          float f[8], h[8];
          unpack8(p[j], f);
          unpack8(q[j], h);
#pragma unroll
          for (int i = 0; i < 8; ++i) sum = fmaf(f[i], h[i], sum);
        }
      }
    } else {
#pragma unroll 8
      for (int d = lane; d < a.D; d += 32) sum = fmaf(half_at(x, d), half_at(w, d), sum);
    }
    sum = warp_sum(sum);
    if (lane == 0 && HG_DBG_INDEX(e, kMost)) {
      if (ctas == 1)
        logits[e] = sum;
      else
        st_cluster_f32(gather + 4u * static_cast<uint32_t>(e), sum);
    }
  }
  if (ctas == 1)
    __syncthreads();
  else
    cluster_sync();
  if (rank > 0 || warp > 0) return;
  int e;
  float share;
  choose(logits, a.E, a.k, a.normalize, e, share);
  if (lane < a.k && HG_DBG_INDEX(m, a.M)) {
    const int at = m * a.k + lane;
    a.ws_chosen[at] = e;
    a.ws_share[at] = share;
    if (a.chosen) a.chosen[at] = e;
    if (a.share) a.share[at] = share;
  }
}

// ------------------------------------------------------------------ products

// Who chose which expert. A slot is a choice, m·k + j; an entry a run of at
// most 8·MT slots that chose the same expert, whose weights are read once for
// it. Experts come in order, and within one the tokens.
constexpr int kSlots = kTokens * HGEMM_EXPERTS_MAX_CHOICES;
constexpr int kEntries = kMost + kSlots / 8;  // a partly filled one per expert, and full ones
struct Entry {
  uint32_t expert : 16, first : 10, count : 6;
};
static_assert(kMost <= 1 << 16 && kSlots <= 1 << 10, "an entry's parts");
template <bool FIRST>
struct Routing {
  uint16_t list[kSlots];               // the slots, by entry
  uint16_t token[FIRST ? kSlots : 1];  // and their tokens
  Entry entry[kEntries];
  int entries;
};
// What only finding them needs, in the room of the partial sums.
struct RoutingScratch {
  unsigned long long tokens[kMost];  // a bit per token that chose the expert
  uint16_t first[kMost];             // where an expert's slots begin in the list
};

template <int MT, bool FIRST>
__device__ __forceinline__ void find_entries(Routing<FIRST>& r, RoutingScratch& s, const ExpertsArgs& a) {
  for (int e = threadIdx.x; e < a.E; e += blockDim.x) s.tokens[e] = 0;
  const int slots = a.M * a.k;
  int chosen[kSlots / kThreads];
#pragma unroll
  for (int j = 0; j < kSlots / kThreads; ++j) {
    const int i = static_cast<int>(threadIdx.x) + j * kThreads;
    chosen[j] = threadIdx.x < kThreads && i < slots ? ld_gpu_s32(a.ws_chosen + i) : -1;
  }
  __syncthreads();
#pragma unroll
  for (int j = 0; j < kSlots / kThreads; ++j)
    if (chosen[j] >= 0) atomicOr(&s.tokens[chosen[j]], 1ull << ((static_cast<int>(threadIdx.x) + j * kThreads) / a.k));
  __syncthreads();
  if (threadIdx.x < 32) {
    const int lane = threadIdx.x;
    int at = 0, n = 0;  // slots and entries of the experts before
    for (int e0 = 0; e0 < a.E; e0 += 32) {
      const int e = e0 + lane;
      const int count = e < a.E ? __popcll(s.tokens[e]) : 0;
      const int runs = (count + 8 * MT - 1) / (8 * MT);
      int both = count | runs << 16, sum = both;  // (1024 slots, 640 entries at most)
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const int v = __shfl_up_sync(0xffffffffu, sum, o);
        if (lane >= o) sum += v;
      }
      const int all = __shfl_sync(0xffffffffu, sum, 31);
      const int first = at + ((sum - both) & 0xFFFF), entry = n + ((sum - both) >> 16);
      if (count > 0) {
        s.first[e] = static_cast<uint16_t>(first);
        for (int j = 0; j < runs; ++j)
          r.entry[entry + j] = Entry{static_cast<uint32_t>(e), static_cast<uint32_t>(first + 8 * MT * j),
                                     static_cast<uint32_t>(min(count - 8 * MT * j, 8 * MT))};
      }
      at += all & 0xFFFF;
      n += all >> 16;
    }
    if (lane == 0) r.entries = n;
  }
  __syncthreads();
#pragma unroll
  for (int j = 0; j < kSlots / kThreads; ++j) {
    const int i = static_cast<int>(threadIdx.x) + j * kThreads, e = chosen[j];
    if (e < 0) continue;
    const int token = i / a.k, at = s.first[e] + __popcll(s.tokens[e] & ((1ull << token) - 1));
    r.list[at] = static_cast<uint16_t>(i);
    if (FIRST) r.token[at] = static_cast<uint16_t>(token);
  }
  __syncthreads();
}

// What becomes of the sums of one unit: outputs n0 .. n0+per-1 of an entry's
// slots, `sum(row, column)` over the block's warps. By the threads t of T.
template <bool FIRST, typename Sum>
__device__ __forceinline__ void put_unit(const ExpertsArgs& a, const Routing<FIRST>& r, const Entry& e, int split, int n0,
                                         int per, int rows, int t, int T, Sum sum) {
  for (int i = t; i < e.count * per; i += T) {
    const int row = i / per, f = i - row * per, n = n0 + f;
    if (n >= rows) continue;
    const int slot = r.list[e.first + row];
    float v = sum(row, f);
    if constexpr (FIRST) {
      const uint16_t* bias = a.b1 ? a.b1 + e.expert * (a.gated ? 2 : 1) * static_cast<int64_t>(rows) : nullptr;
      if (bias) v += half_at(bias, n);
      v = activate(v, a.act);
      if (a.gated) {
        float up = sum(row, f + 8);
        if (bias) up += half_at(bias, rows + n);
        v *= up;
      }
      // In two parts, v's FP16 value and that of what it leaves out: within 2^-23
      // of v or 2^-25; from 65520 on infinite, with no rest.
      const __half upper = __float2half_rn(v);
      const float rest = __hisinf(upper) ? 0.f : v - __half2float(upper);
      if (HG_DBG_INDEX(n, a.F)) {
        a.ws_h[2 * slot * a.ldh + n] = __half_as_ushort(upper);
        a.ws_h[(2 * slot + 1) * a.ldh + n] = __half_as_ushort(__float2half_rn(rest));
      }
    } else {
      if (HG_DBG_INDEX(n, a.D)) a.ws_out[(static_cast<int64_t>(split) * a.M * a.k + slot) * a.ldo + n] = v;
    }
  }
}

// FIRST: a unit of work is features 8u .. 8u+7 and their gates (gated) or
// 16u .. 16u+15 of an entry's expert, and H is written; else outputs 16u ..
// 16u+15 over one of `splits` runs of F, and the slots' FP32 partial outputs
// are. Units are dealt to the blocks in turn.
//
// Eight warps multiply and a ninth adds their sums up, so that none of the
// eight waits for the others at a unit's end. A lane's pieces pass through a
// queue of its own in shared memory, filled by asynchronous copies: registers
// hold four pieces at most before a warp's scoreboards, six, make it wait for
// the youngest load instead of the oldest (24 tokens, 8 of 64 experts: 176 us
// that way, 136 with the queue; 347 with bulk copies of 1 KB, of which an SM
// starts one in some 125 cycles). A step is two pieces, 64 values of K per warp
// and 128 bytes of a row. A warp's steps of all its units form one sequence, so
// that the next unit's weights are on their way while one is added up. The
// second product starts on its weights before the first has ended: who chose
// what is known since the router, and only the tokens' values have to be waited
// for. Tokens are copied through L1: every block wants the same few rows, and
// the L2 lines of one token's row, asked for by all of them, held the first
// product to 4.4 TB/s (5.3 through L1, launched by itself).
//
// ANY: rows that begin at any even address. The copies are of the aligned 16
// bytes that a piece lies in, its row's last ones cut at the end (the rest is
// zeros), and a ninth to a row's eight; a lane takes its piece out of its own
// and its neighbour's by the row's distance from alignment. (The first copy of
// a row may begin up to 14 bytes before it, within the 16 that hold its first
// value and so within the same allocation.)
//
// The second product's tokens are pairs of rows, H's upper parts and what they
// leave out, both multiplied by the weights that are there anyway and summed by
// themselves. A tile of eight columns takes the pairs of up to four tokens, so
// that an entry of so few needs no second one, and its sums are the same (24
// tokens 2048 -> 1025, rows at any address: 203 us with two tiles, 197 with one;
// aligned rows within 1%).
template <int MT, bool FIRST, bool ANY>
struct QueueCfg {
  static constexpr int TILES = FIRST ? MT : 2 * MT;  // of eight rows, a step's tokens
  static constexpr int CTAS = TILES < 4 ? 2 : 1;     // per SM
  static constexpr int DEPTH = TILES < 4 ? 2 : 3;
  static constexpr int BUFFERS = 2;                  // of partial sums
  static constexpr int ROWS = 1024 + (ANY ? 128 : 0);  // of a warp: a step of eight rows
  static constexpr int SLOT = (2 + TILES) * ROWS;      // 16 rows of weights, and the tokens
  static constexpr int PART = kWarps * 8 * MT * 17;  // floats of one buffer
  static constexpr int OFF_ROUTING = BUFFERS * PART * 4;
  static constexpr int OFF_BAR = (OFF_ROUTING + static_cast<int>(sizeof(Routing<FIRST>)) + 15) / 16 * 16;
  static constexpr int OFF_MISC = OFF_BAR + 2 * 8 * BUFFERS;
  static constexpr int OFF_QUEUE = (OFF_MISC + 4 + 15) / 16 * 16;
  static_assert(sizeof(RoutingScratch) <= OFF_ROUTING, "fits the partial sums' room");
  // Enough that no further CTA fits: units are dealt out to CTAS on each SM, and
  // an SM that takes one more leaves another idle (one token 52 us in place of
  // 46.5). And no more than it takes: what is left of an SM's memory is L1, where
  // the tokens are, and both products' launches divide it alike, or an SM has to
  // run dry between them. (With four buffers of partial sums and the scratch of
  // the routing beside them one token took 48.7 us, 24 tokens 142.5.)
  static constexpr int NEEDED = OFF_QUEUE + kWarps * DEPTH * SLOT, LEAST = 233472 / (CTAS + 1) - 1024 + 16;
  static constexpr int SMEM_BYTES = NEEDED > LEAST ? NEEDED : LEAST;
  static_assert(CTAS * (SMEM_BYTES + 1024) <= 233472, "the CTAs fit an SM");
};

// The 16 bytes that begin s bytes (even) into two times 16.
__device__ __forceinline__ uint4 shifted(uint4 lo, uint4 hi, uint32_t s) {
  uint32_t w[8] = {lo.x, lo.y, lo.z, lo.w, hi.x, hi.y, hi.z, hi.w};
#pragma unroll
  for (int j = 0; j < 6; ++j) w[j] = s & 8u ? w[j + 2] : w[j];
#pragma unroll
  for (int j = 0; j < 5; ++j) w[j] = s & 4u ? w[j + 1] : w[j];
  const uint32_t bits = (s & 2u) * 8u;
  return make_uint4(__funnelshift_r(w[0], w[1], bits), __funnelshift_r(w[1], w[2], bits),
                    __funnelshift_r(w[2], w[3], bits), __funnelshift_r(w[3], w[4], bits));
}

template <int MT, bool FIRST, bool ANY>
__global__ void __launch_bounds__(kThreads + 32, QueueCfg<MT, FIRST, ANY>::CTAS) experts_queue_kernel(const ExpertsArgs a) {
  using Cfg = QueueCfg<MT, FIRST, ANY>;
  constexpr int DEPTH = Cfg::DEPTH, STEP = kWarps * 2 * kPiece;  // values of K per step
  extern __shared__ __align__(128) uint8_t experts_smem[];
  float* parts = reinterpret_cast<float*>(experts_smem);
  Routing<FIRST>& r = *reinterpret_cast<Routing<FIRST>*>(experts_smem + Cfg::OFF_ROUTING);
  const uint32_t full0 = smem_u32(experts_smem + Cfg::OFF_BAR), empty0 = full0 + 8u * Cfg::BUFFERS;
  volatile int* abort_flag = reinterpret_cast<volatile int*>(experts_smem + Cfg::OFF_MISC);
  const Watchdog wd{abort_flag, a.status, a.timeout_ns};
  if (threadIdx.x == 0) {
    *abort_flag = 0;
    for (int i = 0; i < Cfg::BUFFERS; ++i) {
      mbar_init(full0 + 8u * i, kWarps);
      mbar_init(empty0 + 8u * i, 1);
    }
  }
  if constexpr (FIRST) {
    grid_dependency_wait();
    grid_launch_dependents();
  } else {
    fence_gpu();
  }
  find_entries<MT>(r, *reinterpret_cast<RoutingScratch*>(experts_smem), a);  // (its barriers publish these)
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int K = FIRST ? a.D : a.F, rows = FIRST ? a.F : a.D;
  const bool gated = FIRST && a.gated;
  const int per = gated ? 8 : 16;  // outputs of a unit
  const int blocks = (rows + per - 1) / per, splits = FIRST ? 1 : a.splits;
  const int run = FIRST ? K : a.run;  // of K, of one split
  // The block's units, every gridDim.x-th of blocks × splits × entries, without
  // a division from one to the next: a warp that does not multiply does not
  // refill its queue either.
  const int entries = r.entries;
  const int block_step = static_cast<int>(gridDim.x) % blocks, rest = static_cast<int>(gridDim.x) / blocks;
  const int split_step = rest % splits, entry_step = rest / splits;
  struct Unit {
    int block, split, entry;
  };
  const Unit first{static_cast<int>(blockIdx.x) % blocks, static_cast<int>(blockIdx.x) / blocks % splits,
                   static_cast<int>(blockIdx.x) / blocks / splits};
  auto advance = [&](Unit& u) {
    u.block += block_step;
    u.split += split_step;
    u.entry += entry_step;
    if (u.block >= blocks) u.block -= blocks, ++u.split;
    if (u.split >= splits) u.split -= splits, ++u.entry;
  };
  // (of K: at least one value)
  auto k_end = [&](const Unit& u) { return min(u.split * run + run, K); };
  auto steps_of = [&](const Unit& u) { return (k_end(u) - u.split * run + STEP - 1) / STEP; };
  int buffer = 0;
  uint32_t phase = 0;
  auto next_buffer = [&]() {
    if (++buffer == Cfg::BUFFERS) {
      buffer = 0;
      phase ^= 1u;
    }
  };

  if (warp == kWarps) {
    // ---- the warp that adds up. (A wait that gives up has raised the abort
    // flag: later waits give up at once, and the loops run out.)
    if constexpr (!FIRST) {
      grid_dependency_wait();
      grid_launch_dependents();
    }
    for (Unit u = first; u.entry < entries; advance(u)) {
      (void)wait_phase(full0 + 8u * buffer, phase, wd, kWdReduce);
      const float* part = parts + buffer * Cfg::PART;
      put_unit<FIRST>(a, r, r.entry[u.entry], u.split, u.block * per, per, rows, lane, 32, [&](int row, int column) {
        float v = part[row * 17 + column];
#pragma unroll
        for (int w = 1; w < kWarps; ++w) v += part[w * (8 * MT * 17) + row * 17 + column];
        return v;
      });
      __syncwarp();
      if (lane == 0) mbar_arrive(empty0 + 8u * buffer);
      next_buffer();
    }
    return;
  }

  // ---- the eight warps that multiply
  const int g = lane >> 2, t = lane & 3;
  const uint16_t* W = FIRST ? a.W1 : a.W2;
  const int64_t ldw = FIRST ? a.ldw1 : a.ldw2;
  const int64_t expert_rows = gated ? 2 * static_cast<int64_t>(rows) : rows;
  uint8_t* queue = experts_smem + Cfg::OFF_QUEUE + warp * (DEPTH * Cfg::SLOT) + 16 * lane;
  const uint32_t queue_addr = smem_u32(queue);
  // What is copied next: unit fu, fsteps steps of it left, the next at fk of
  // these rows.
  Unit fu = first;
  int fsteps = 0, fk = 0, fend = 0;
  bool fpaired = false;
  const uint16_t *w0 = nullptr, *w1 = nullptr, *x[MT];
  // Whether an entry's upper parts and rests share a tile, in columns 0-3 and 4-7.
  auto paired = [](int count) { return !FIRST && MT == 1 && count <= 4; };
  auto begin_unit = [&]() {
    if (fu.entry >= entries) return;
    const auto& e = r.entry[fu.entry];
    fpaired = paired(e.count);
    const int n0 = fu.block * per;
    fk = fu.split * run + warp * 2 * kPiece + 8 * t;
    fend = k_end(fu);
    fsteps = steps_of(fu);
    // rows past the end are computed as copies of the last one and not stored
    const uint16_t* base = W + e.expert * expert_rows * ldw + fk;
    const int row0 = min(n0 + g, rows - 1), row1 = min(n0 + g + 8, rows - 1);
    w0 = base + row0 * ldw;
    w1 = base + (gated ? row0 + static_cast<int64_t>(rows) : row1) * ldw;
#pragma unroll
    for (int i = 0; i < MT; ++i) {
      const int token = fpaired ? g & 3 : 8 * i + g, row = e.first + token, rest = fpaired ? g >> 2 : 0;
      x[i] = token >= e.count ? nullptr
                              : (FIRST ? a.X + r.token[row] * a.ldx : a.ws_h + (2 * r.list[row] + rest) * a.ldh) + fk;
    }
  };
  // (past the end zeros; where there is no token nothing: a column of its own)
  auto copy_16 = [&](uint32_t to, const void* p, int bytes, bool weights) {
    if (weights)
      cp_async_16(to, p, bytes);
    else
      cp_async_16_shared(to, p, bytes);
  };
  auto copy = [&](uint32_t to, const uint16_t* p, bool weights) {
    if constexpr (ANY) {
      const uintptr_t at = reinterpret_cast<uintptr_t>(p) & ~static_cast<uintptr_t>(15);
      // bytes from here to the end of the row's part
      const int left = static_cast<int>(reinterpret_cast<uintptr_t>(p + (fend - fk)) - at);
#pragma unroll
      for (int i = 0; i < 3; ++i) {
        if (i == 2 && t != 3) continue;  // the ninth
        const int from = i == 2 ? 80 : 64 * i, bytes = min(max(left - from, 0), 16);
        // (its first value's index in the row: at most seven before it, of the row's first 16 bytes)
        if (bytes > 0 && !HG_DBG_INDEX(fk + static_cast<int>(static_cast<int64_t>(at + from) -
                                                             reinterpret_cast<int64_t>(p)) / 2 + 7,
                                       fend + 7))
          continue;
        copy_16(to + (i == 2 ? 1024u + 16u * g - 16u * lane : 512u * i),
                bytes > 0 ? reinterpret_cast<const void*>(at + from) : a.ws_h, bytes, weights);
      }
    } else {
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        const bool in = fk + kPiece * i < fend && dbg_row(p + kPiece * i, fk + kPiece * i, 8, fend, 16);
        copy_16(to + 512u * i, in ? p + kPiece * i : a.ws_h, in ? 16 : 0, weights);
      }
    }
  };
  auto copy_weights = [&](int into) {
    const uint32_t to = queue_addr + static_cast<uint32_t>(into * Cfg::SLOT);
    copy(to, w0, true);
    copy(to + Cfg::ROWS, w1, true);
  };
  auto copy_tokens = [&](int into) {
    const uint32_t to = queue_addr + static_cast<uint32_t>(into * Cfg::SLOT + 2 * Cfg::ROWS);
#pragma unroll
    for (int i = 0; i < MT; ++i)
      if (x[i]) {
        copy(to + static_cast<uint32_t>(Cfg::ROWS) * i, x[i], false);
        if (!FIRST && !fpaired) copy(to + static_cast<uint32_t>(Cfg::ROWS) * (MT + i), x[i] + a.ldh, false);
      }
  };
  // Piece i of the rows at `at`, their distance from alignment `off`.
  auto piece_of = [&](const uint8_t* at, int i, uint32_t off) {
    const uint4 lo = *reinterpret_cast<const uint4*>(at + 512 * i);
    if constexpr (!ANY) return lo;
    const int next = t < 3 ? 512 * i + 16 : i == 0 ? 512 - 48 : 1024 + 16 * g - 16 * lane;
    return shifted(lo, *reinterpret_cast<const uint4*>(at + next), off);
  };
  auto next_step = [&]() {
    if (--fsteps > 0) {
      fk += STEP;
      w0 += STEP;
      w1 += STEP;
#pragma unroll
      for (int i = 0; i < MT; ++i)
        if (x[i]) x[i] += STEP;
    } else {
      advance(fu);
      begin_unit();
    }
  };
  begin_unit();
  if constexpr (!FIRST) {
    // the first steps' weights, before the tokens' values are there
    for (int j = 0; j < DEPTH && fu.entry < entries; ++j) {
      copy_weights(j);
      next_step();
    }
    grid_dependency_wait();
    grid_launch_dependents();
    fu = first;
    begin_unit();
  }
  for (int j = 0; j < DEPTH; ++j) {
    if (fu.entry < entries) {
      if (FIRST) copy_weights(j);
      copy_tokens(j);
      next_step();
    }
    cp_async_commit();
  }

  int slot = 0, done = 0;
  for (Unit u = first; u.entry < entries; advance(u)) {
    const int steps = steps_of(u);
    const auto& e = r.entry[u.entry];
    const int count = e.count;
    uint32_t off0 = 0, off1 = 0, off[MT] = {};
    if constexpr (ANY) {
      // (whole steps further on a row's distance is the same)
      auto distance = [](const uint16_t* p) { return static_cast<uint32_t>(reinterpret_cast<uintptr_t>(p)) & 15u; };
      const int n0 = u.block * per, row0 = min(n0 + g, rows - 1), row1 = min(n0 + g + 8, rows - 1);
      const uint16_t* base = W + e.expert * expert_rows * ldw;
      off0 = distance(base + row0 * ldw);
      off1 = distance(base + (gated ? row0 + static_cast<int64_t>(rows) : row1) * ldw);
      if constexpr (FIRST) {  // (H's rows are aligned)
#pragma unroll
        for (int i = 0; i < MT; ++i)
          if (8 * i + g < count) off[i] = distance(a.X + r.token[e.first + 8 * i + g] * a.ldx);
      }
    }
    const bool pair = paired(count);
    float acc[Cfg::TILES][4] = {};
    for (int s = 0; s < steps; ++s) {
      cp_async_wait<DEPTH - 1>();
      if (ANY) __syncwarp();
      const uint8_t* at = queue + slot * Cfg::SLOT;
      uint4 p[2][2];
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        p[i][0] = piece_of(at, i, off0);
        p[i][1] = piece_of(at + Cfg::ROWS, i, off1);
      }
#pragma unroll
      for (int j = 0; j < Cfg::TILES; ++j) {
        if (8 * (j % MT) >= count || (j >= MT && pair)) continue;
#pragma unroll
        for (int i = 0; i < 2; ++i) {
          const uint4 b = piece_of(at + (2 + j) * Cfg::ROWS, i, off[j % MT]);
          mma_16816(acc[j], p[i][0].x, p[i][1].x, p[i][0].y, p[i][1].y, b.x, b.y);
          mma_16816(acc[j], p[i][0].z, p[i][1].z, p[i][0].w, p[i][1].w, b.z, b.w);
        }
      }
      if (ANY) __syncwarp();  // the neighbours have read theirs
      if (fu.entry < entries) {
        copy_weights(slot);
        copy_tokens(slot);
        next_step();
      }
      cp_async_commit();
      if (++slot == DEPTH) slot = 0;
    }
    if constexpr (!FIRST) {
#pragma unroll
      for (int i = 0; i < MT; ++i)
#pragma unroll
        for (int k = 0; k < 4; ++k) {
          // (columns 2t, 2t + 1 of a fragment's lane t; those four further are lane t + 2's)
          const float rest = pair ? __shfl_down_sync(0xffffffffu, acc[i][k], 2) : acc[MT + i][k];
          acc[i][k] += rest;
        }
    }
    if (done++ >= Cfg::BUFFERS) (void)wait_phase(empty0 + 8u * buffer, phase ^ 1u, wd, kWdReduce);
    float* part = parts + buffer * Cfg::PART + warp * (8 * MT * 17);
#pragma unroll
    for (int i = 0; i < MT; ++i) {
      float* q = part + (8 * i + 2 * t) * 17 + g;
      q[0] = acc[i][0];
      q[17] = acc[i][1];
      q[8] = acc[i][2];
      q[17 + 8] = acc[i][3];
    }
    __syncwarp();
    if (lane == 0 && !(a.inject == 1 && done == 1 && warp == 0))  // testing aid: withhold one arrival
      mbar_arrive(full0 + 8u * buffer);
    next_buffer();
  }
  cp_async_wait<0>();  // (nothing is under way any more but empty groups)
}

// Y = Σ s·(output + b2) + R, the choices in order, a choice's runs of F in
// order. A thread asks for four choices' values at once.
__global__ void __launch_bounds__(kThreads) experts_sum_kernel(const ExpertsArgs a) {
  grid_dependency_wait();
  grid_launch_dependents();
  const int m = blockIdx.y;
  const int64_t d = static_cast<int64_t>(blockIdx.x) * kThreads + threadIdx.x;
  if (d >= a.D || !HG_DBG_INDEX(m, a.M)) return;
  const float residual = a.R ? half_at(a.R, m * a.ldr + d) : 0.f;
  const float* out = a.ws_out + static_cast<int64_t>(m) * a.k * a.ldo + d;
  const int64_t split = static_cast<int64_t>(a.M) * a.k * a.ldo;
  float y = 0.f;
  for (int j0 = 0; j0 < a.k; j0 += 4) {
    float v[4], s[4], bias[4];
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      v[j] = s[j] = bias[j] = 0.f;
      if (j0 + j >= a.k) continue;
      const int slot = m * a.k + j0 + j;
      s[j] = a.ws_share[slot];
      if (a.b2) bias[j] = half_at(a.b2, static_cast<int64_t>(a.ws_chosen[slot]) * a.D + d);
    }
#pragma unroll 4
    for (int i = 0; i < a.splits; ++i)
#pragma unroll
      for (int j = 0; j < 4; ++j)
        if (j0 + j < a.k) v[j] += out[i * split + (j0 + j) * a.ldo];
#pragma unroll
    for (int j = 0; j < 4; ++j)
      if (j0 + j < a.k) y = fmaf(s[j], v[j] + bias[j], y);
  }
  a.Y[m * a.ldy + d] = __half_as_ushort(__float2half_rn(y + residual));
}

template <typename Kernel>
cudaError_t allow_smem(Kernel kern, int bytes, std::atomic<bool> (&done)[64]) {
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  if (dev < 0 || dev >= 64 || !done[dev]) {
    e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, bytes);
    if (e == cudaSuccess && dev >= 0 && dev < 64) done[dev] = true;
  }
  return e;
}

template <int MT, bool FIRST, bool ANY>
cudaError_t product_with(const ExpertsArgs& a, int num_sms, cudaStream_t stream) {
  using Cfg = QueueCfg<MT, FIRST, ANY>;
  static std::atomic<bool> done[64];
  auto kern = experts_queue_kernel<MT, FIRST, ANY>;
  const cudaError_t e = allow_smem(kern, Cfg::SMEM_BYTES, done);
  if (e != cudaSuccess) return e;
  PdlLaunch l(dim3(static_cast<unsigned>(num_sms * Cfg::CTAS)), dim3(kThreads + 32), Cfg::SMEM_BYTES, stream);
  return cudaLaunchKernelEx(&l.cfg, kern, a);
}

// Tiles of eight tokens that share a read of an expert's weights: as many as an
// expert is likely to have. More tokens than that read them again, from L2.
int token_tiles(const ExpertsArgs& a) {
  if (a.M <= 8 || a.M * a.k <= 8 * a.E) return 1;
  return a.M * a.k > 16 * a.E ? 4 : 2;
}

template <bool FIRST, bool ANY>
cudaError_t product_tiles(const ExpertsArgs& a, int num_sms, cudaStream_t stream) {
  const int tiles = token_tiles(a);
  if constexpr (FIRST) {
    if (tiles == 4) return product_with<4, FIRST, ANY>(a, num_sms, stream);
    if (tiles == 2) return product_with<2, FIRST, ANY>(a, num_sms, stream);
  } else {
    // Half as many: its tokens are pairs of rows, and tiles for all of them leave
    // an SM one block (40 tokens, 5 of 16 experts, 2048 -> 2048: 134 us with as
    // many as in the first product, 110 with half; 64 tokens, 4 of 8: 82 and 77.5).
    if (tiles == 4) return product_with<2, FIRST, ANY>(a, num_sms, stream);
  }
  return product_with<1, FIRST, ANY>(a, num_sms, stream);
}

template <bool FIRST>
cudaError_t product(const ExpertsArgs& a, bool vec, int num_sms, cudaStream_t stream) {
  return vec ? product_tiles<FIRST, false>(a, num_sms, stream) : product_tiles<FIRST, true>(a, num_sms, stream);
}

int64_t align16(int64_t bytes) { return (bytes + 15) / 16 * 16; }

// The second product's runs of F: enough units to keep every block busy for a
// few of them, and a step of the warps each at least.
constexpr int kUnits = 1024;
constexpr int kMaxSplits = 16;
constexpr int kStep = kWarps * 2 * kPiece;
int run_of(int64_t M, int64_t D, int64_t F, int64_t E, int64_t k, int* splits) {
  const int64_t experts = M * k < E ? M * k : E, blocks = (D + 15) / 16;
  int64_t want = experts * blocks > 0 ? (kUnits + experts * blocks - 1) / (experts * blocks) : 1;
  const int64_t most = F / kStep;
  want = want > kMaxSplits ? kMaxSplits : want;
  want = want > most ? most : want;
  want = want < 1 ? 1 : want;
  const int64_t run = ((F + want - 1) / want + kStep - 1) / kStep * kStep;
  *splits = static_cast<int>(run > 0 ? (F + run - 1) / run : 0);
  return static_cast<int>(run);
}

}  // namespace

// The choice, its shares, H (two rows of whole 16 bytes a slot) and the slots'
// outputs.
size_t experts_workspace(int64_t M, int64_t D, int64_t F, int64_t E, int64_t k) {
  int splits;
  run_of(M, D, F, E, k, &splits);
  return static_cast<size_t>(2 * align16(4 * M * k) + 2 * M * k * align16(2 * F) + splits * M * k * align16(4 * D));
}

cudaError_t launch_experts(ExpertsArgs a, void* workspace, int num_sms, cudaStream_t stream) {
  const int64_t slots = static_cast<int64_t>(a.M) * a.k;
  uint8_t* ws = static_cast<uint8_t*>(workspace);
  a.ws_chosen = reinterpret_cast<int*>(ws);
  a.ws_share = reinterpret_cast<float*>(ws += align16(4 * slots));
  a.ws_h = reinterpret_cast<uint16_t*>(ws += align16(4 * slots));
  a.ldh = align16(2 * static_cast<int64_t>(a.F)) / 2;
  a.ws_out = reinterpret_cast<float*>(ws += slots * a.ldh * 4);
  a.ldo = align16(4 * static_cast<int64_t>(a.D)) / 4;
  a.run = run_of(a.M, a.D, a.F, a.E, a.k, &a.splits);
  const bool vec_x = a.D % 8 == 0 && rows16(a.X, a.ldx);
  const bool vec_r = vec_x && rows16(a.Wr, a.ldwr), vec1 = vec_x && rows16(a.W1, a.ldw1);
  const bool vec2 = a.F % 8 == 0 && rows16(a.W2, a.ldw2);
  cudaError_t e;
  {
    // a warp per logit, up to eight CTAs of eight
    a.router_ctas = a.E <= kWarps ? 1 : a.E <= 2 * kWarps ? 2 : a.E <= 4 * kWarps ? 4 : 8;
    PdlLaunch l(dim3(static_cast<unsigned>(a.M * a.router_ctas)), dim3(kThreads), 0, stream);
    if (a.router_ctas > 1) l.cluster(static_cast<unsigned>(a.router_ctas));
    e = cudaLaunchKernelEx(&l.cfg, vec_r ? experts_router_kernel<true> : experts_router_kernel<false>, a);
    if (e != cudaSuccess) return e;
  }
  if (a.F > 0 && a.D > 0) {
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
