// internal.h — host-side interface between the C-ABI layer (hgemm_api.cu)
// and the kernel translation units. Not part of the public ABI.
#pragma once

#include <cstdint>

#include <cuda.h>
#include <cuda_runtime.h>

#include "hgemm.h"

namespace hg {

// Watchdog codes written to the device status word by a wait that gave up.
enum WatchdogCode : int {
  kWdNone = 0,
  kWdProducerEmpty = 1,   // TMA producer waiting for a free smem stage
  kWdMmaFull = 2,         // MMA issuer waiting for a loaded smem stage
  kWdMmaAccEmpty = 3,     // MMA issuer waiting for the epilogue to free TMEM
  kWdEpiAccFull = 4,      // epilogue waiting for a finished accumulator
  kWdDrain = 5,           // end-of-kernel drain of in-flight copies or MMAs
  kWdReduce = 6,          // split-K owner waiting for the other slices' partials
  kWdGridBarrier = 7,     // a CTA of a cooperative launch waiting for all others at a phase boundary
  kWdRowGroup = 8,        // an epilogue waiting for the CTAs that read the rows it overwrites
  kWdRows = 9,            // the layer norm's backward pass waiting for a row
};

// The fused epilogue ("GPU架构与CUDA", 核函数融合): each FP32 accumulator
// becomes alpha·acc + beta·C_old + bias[col], then max(·, 0) when relu is
// set, before the single rounding to FP16. mode 0: plain product (the
// accumulator is stored as is); 1: fused, C not read; 2: fused, C read.
struct EpiArgs {
  float alpha, beta;
  const uint16_t* bias;  // N FP16 values (one per column of C), or null
  int relu;
  int mode;
};

// Which epilogue a product kernel is instantiated with: the accumulator
// stored as it is, EpiArgs, or LinEpi forward or backward.
enum Epilogue : int { kEpiPlain = 0, kEpiFused = 1, kEpiLinear = 2, kEpiLinearGrad = 3 };

// The epilogue of a linear layer's product (forward) or of its input's
// gradient (backward); the definitions are in linear_epilogue.cuh.
struct LinEpi {
  int backward;              // 0: y = f(acc + bias) + res, u kept in 8 bits; 1: acc·f'(û), h = f(û)
  int act;                   // HGEMM_ACT_*
  const uint16_t* bias;      // forward: N values, or null
  const uint16_t* res;       // forward: M×N, or null
  int64_t ldr;
  int8_t* codes;             // forward: written; backward: read; null: none
  int64_t ldq;
  float* scales;             // scales[g·lds + m]
  int64_t lds;
  uint16_t* h;               // backward: f(û), or null
  int64_t ldh;
};

// The operands' order in memory, a template parameter of the pair, wide and
// split-K kernels: a branch on it between the copies and between the matrix
// instructions costs time in both (the wave kernel's copies 0.155 us a block
// with it, 0.115 without).
enum Layout {
  kLayoutK,    // both K-contiguous
  kLayoutBn,   // A K-contiguous, B N-contiguous: a linear layer's input gradient
  kLayoutMn,   // A M-contiguous, B N-contiguous: its weight's gradient
  kLayoutAny,  // by TcArgs::a_mn and b_mn
};
constexpr bool layout_a_mn(Layout l, int a_mn) { return l == kLayoutMn || (l == kLayoutAny && a_mn != 0); }
constexpr bool layout_b_mn(Layout l, int b_mn) {
  return l == kLayoutBn || l == kLayoutMn || (l == kLayoutAny && b_mn != 0);
}

// Everything a tensor-core launch needs besides the tensor maps.
struct TcArgs {
  int M, N, K;
  int num_m, num_n, num_kb;  // tiles along M and N, 64-wide K blocks
  int num_tiles;             // work units: whole tiles, then tile parts
  int full_tiles;            // units below this index are whole tiles; the rest are
                             // parts of part_cols columns of the last tiles (pair kernel)
  int part_cols;             // 128 or 64
  int stages, stage_bytes;   // operand ring geometry (pair kernel)
  int group_m;               // rasterisation group height (in M tiles)
  int grid;                  // persistent CTAs
  int* status;               // device watchdog word
  unsigned long long timeout_ns;
  int inject;                // HGEMM_INJECT_* (testing the watchdog)
  EpiArgs epi;
  const uint16_t* C;         // C itself, read in epilogue mode 2
  int64_t ldc;               // C's row pitch in elements
  int a_mn, b_mn;            // pair kernel: A stored M-contiguous (K×M), B stored
                             // N-contiguous (K×N); else K-contiguous
  LinEpi lin;                // kEpiLinear and kEpiLinearGrad
  float* row_sums;           // one wave of 128×64 tiles, kLayoutMn: A's sums over K, or null
  int row_sums_add;          // added to, instead of written
  int batch_tiles;           // pair kernel: whole tiles per product of a batch of
                             // equal products in one launch (0: a single product)
  int batch_shift;           // product j of the batch is the first one with A's K,
                             // B's N and K, and C's N coordinates shifted by j·batch_shift
};

// Plain-pointer launch arguments for the kernels that do not use TMA.
struct PlainArgs {
  const uint16_t* A;
  const uint16_t* B;
  uint16_t* C;
  int64_t M, N, K;
  int64_t lda, ldb, ldc;     // row pitches in elements
  int* status;
  unsigned long long timeout_ns;
  EpiArgs epi;
  int a_mn = 0, b_mn = 0;    // A(i,k) at A[k*lda + i]; B(k,j) at B[k*ldb + j]
};

// The diagonal blocks ("leaves") of a triangular product, for one batched
// launch of masked products.
constexpr int kMaxLeaves = 128;
struct TriLeaves {
  int count;
  int64_t off[kMaxLeaves];   // first row (and column) of each block in the triangle
  int64_t size[kMaxLeaves];  // its order
};

// Every kernel here is launched with programmatic stream serialization: it
// may start while the previous kernel on the stream is still running, and
// waits for it (griddepcontrol.wait) before touching memory that kernel may
// write, so its launch and prologue overlap the previous kernel's tail.
struct PdlLaunch {
  cudaLaunchAttribute attr[2];
  cudaLaunchConfig_t cfg;
  PdlLaunch(dim3 grid, dim3 block, size_t smem, cudaStream_t stream) : attr{}, cfg{} {
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.gridDim = grid;
    cfg.blockDim = block;
    cfg.dynamicSmemBytes = smem;
    cfg.stream = stream;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
  }
  // clusters of x CTAs set at launch time
  void cluster(unsigned x) {
    attr[1].id = cudaLaunchAttributeClusterDimension;
    attr[1].val.clusterDim.x = x;
    attr[1].val.clusterDim.y = 1;
    attr[1].val.clusterDim.z = 1;
    cfg.numAttrs = 2;
  }
};

// Launchers (each enqueues one kernel on `stream` and returns the launch
// error, if any). Shared-memory attributes are set on first use per device.
cudaError_t launch_tc_128x256(const CUtensorMap& a, const CUtensorMap& b, const CUtensorMap& c,
                              const TcArgs& args, Epilogue kind, cudaStream_t stream);
cudaError_t launch_tc_128x64(const CUtensorMap& a, const CUtensorMap& b, const CUtensorMap& c,
                             const TcArgs& args, Epilogue kind, cudaStream_t stream);
// b_part: the B map with part_cols / 2-row boxes, for the tile parts of the last wave.
cudaError_t launch_tc_pair(const CUtensorMap& a, const CUtensorMap& b, const CUtensorMap& b_part,
                           const CUtensorMap& c, const TcArgs& args, Epilogue kind, cudaStream_t stream);
// Largest number of co-resident 2-CTA clusters of the pair kernel.
int pair_max_clusters(int num_sms);
// Wide pair kernel: 256×512 tiles per CTA pair.
cudaError_t launch_tc_wide(const CUtensorMap& a, const CUtensorMap& b, const CUtensorMap& c,
                           const TcArgs& args, cudaStream_t stream);
int wide_max_clusters(int num_sms);
// Split-K cluster kernel for few output tiles: `split` K-slices, one cluster
// of 2*split CTAs per 256×tile_n tile (args.num_tiles of them); tile_n 256
// with 2, 3 or 4 slices, or tile_n 128 with 2.
cudaError_t launch_skinny(int split, int tile_n, const CUtensorMap& a, const CUtensorMap& b,
                          const CUtensorMap& c, const TcArgs& args, Epilogue kind, cudaStream_t stream);
// Largest number of co-resident clusters of the split-K kernel.
int skinny_max_clusters(int split, int tile_n, int num_sms);
// K = 0: C := f(beta·C_old + bias) elementwise (plain mode: +0).
cudaError_t launch_empty_sum(uint16_t* C, int64_t M, int64_t N, int64_t ldc, const EpiArgs& epi,
                             cudaStream_t stream);
cudaError_t launch_generic(const PlainArgs& args, int num_sms, cudaStream_t stream);
// A kernel that does nothing: one CTA of one warp, or (pair_config) one CTA
// per SM in clusters of two with `smem_bytes` of dynamic shared memory each.
cudaError_t launch_floor(int pair_config, int num_sms, int smem_bytes, cudaStream_t stream);
// Dynamic shared memory of one pair-kernel CTA.
int pair_smem_bytes();
// Every leaf b: C + off = (A operand + off) · lower(B operand at (off, off)),
// M × size (see hgemm_generic.cu).
cudaError_t launch_tri_leaves(const PlainArgs& args, const TriLeaves& leaves, int num_sms,
                              cudaStream_t stream);
// The same on the tensor cores for leaves whose orders are multiples of 64
// (see hgemm_trileaf.cu): x maps Bᵀ (m × n, 128×64 boxes), l maps the rows
// of the triangle (column i of A as row i, n × n, 64×64 boxes), c maps Cᵀ
// (m × n, 32×64 boxes); args.num_m row tiles of 128 per leaf.
// ext[b]: K columns past leaf b's own block that its product also covers,
// [off_b + s_b, off_b + s_b + ext[b]) (whole rows of the second operand:
// the off-diagonal updates of the blocks whose first half holds leaf b), a
// multiple of 64, or 0.
struct TriLeafExt {
  int32_t ext[kMaxLeaves];
};
cudaError_t launch_tri_leaves_tc(const CUtensorMap& x, const CUtensorMap& l, const CUtensorMap& c,
                                 const TcArgs& args, const TriLeaves& leaves, const TriLeafExt& ext,
                                 cudaStream_t stream);

// Triangular solve Aᵀ·X = alpha·B (see hgemm_trsm.cu): the largest diagonal
// block solved by substitution; X(:, j) = alpha·B(:, j) over n × m
// column-major operands (X == B allowed); the solve of the diagonal block of
// order s at (off, off) for all m right-hand sides, in place in X.
constexpr int kTrsmLeaf = 256;
cudaError_t launch_scale_copy(const uint16_t* B, int64_t ldb, uint16_t* X, int64_t ldx, int64_t n,
                              int64_t m, float alpha, int num_sms, cudaStream_t stream);
// chained: an earlier launch of the same solve precedes this one on the
// stream (the kernel may then read A before waiting for it).
// The inverses of every diagonal block (leaf b of order s_b ≤ kTrsmInverseLeaf
// at (off_b, off_b)) in one launch: W + b·kTrsmInverseLeaf² receives,
// column-major with pitch kTrsmInverseLeaf, the transpose of the block's
// inverse (row k of the inverse is contiguous), FP16.
constexpr int kTrsmInverseLeaf = 512;
// Bytes of the workspace's synchronisation words of the one-launch solve.
constexpr int kChainSyncBytes = 4096;
// sync (may be null): kChainSyncBytes that the launch zeroes (after waiting
// for the previous launch on the stream) for a chain launch that follows.
cudaError_t launch_trsm_inverse(const uint16_t* A, int64_t lda, uint16_t* W, const TriLeaves& leaves,
                                uint32_t* sync, cudaStream_t stream);
// fwd: the literal orientation A·X = alpha·B (forward substitution).
cudaError_t launch_trsm_leaf(const uint16_t* A, int64_t lda, uint16_t* X, int64_t ldx, int64_t off,
                             int s, int64_t m, int num_sms, bool chained, bool fwd, cudaStream_t stream);


// ------------------------------------------- feed-forward block operators

// Σ over the rows of dY (M×N): out[n], or out[n] + the sum. beside: the launch
// before it on the stream is the product that reads the same dY, which the
// sums may run beside; thin: on the same SMs (see the kernels).
cudaError_t launch_column_sums(const uint16_t* dy, int64_t ld, int64_t M, int64_t N, float* out,
                               bool accumulate, bool beside, bool thin, cudaStream_t stream);
// K = 0: C = the epilogue of zeros.
cudaError_t launch_linear_empty(uint16_t* C, int64_t ldc, int64_t M, int64_t N, const LinEpi& epi,
                                cudaStream_t stream);

// What an entry point outside hgemm_api.cu needs of a call: the current
// device checked (HGEMM_OK or an error status), and a CUDA error as a status.
struct CallDevice {
  int num_sms;
  int* status;
  unsigned long long timeout_ns;
  int inject;
};
int call_device(CallDevice* out);
int cuda_status(cudaError_t e);

// One wave of 128×64 tiles, a CTA each (args.grid).
cudaError_t launch_linear_wave(const CUtensorMap& a, const CUtensorMap& b, const CUtensorMap& c, const TcArgs& args,
                                  Epilogue kind, cudaStream_t stream);

// One product with a linear layer's epilogue, C (M×N) = epilogue(A·B) with A
// M×K, or K×M when a_mn, and B N×K, or K×N when b_mn.
struct LinearProduct {
  const uint16_t* A;
  int64_t lda;
  bool a_mn;
  const uint16_t* B;
  int64_t ldb;
  bool b_mn;
  uint16_t* C;
  int64_t ldc, M, N, K;
  LinEpi epi;
};
int run_linear(const LinearProduct& p, cudaStream_t stream);
// The kernel for at most kLinearRows rows of A, and whether it computes p.
constexpr int kLinearRows = 32;
constexpr int kLinearFragmentRows = 8;  // always that kernel: one column fragment
bool linear_rows_suits(const LinearProduct& p);
cudaError_t launch_linear_rows(const LinearProduct& p, cudaStream_t stream);
// The kernel for few rows or small outputs, fed by TMA: w maps the operand
// whose rows are the output's N columns, x the one whose rows are its M rows,
// in boxes of 128 × 64 and tile_rows × 64, or (stored with those contiguous)
// of 64 × 64. Forward: both K-major, or both contiguous (w_mn: a weight's
// gradient, tile_rows 64 or 128); backward: w contiguous, x K-major.
constexpr int kLinearSmall = 128;
struct SmallArgs {
  uint16_t* Y;
  int64_t ldy;
  int M, N, num_kb;
  int tile_rows, row_tiles;  // 16, 32, 64 or 128 output rows per CTA
  int split;  // CTAs of a cluster, each a run of the K blocks: 1 to 8
  int w_mn;
  int* status;
  unsigned long long timeout_ns;
  int inject;
  LinEpi epi;
};
cudaError_t launch_linear_small(const CUtensorMap& w, const CUtensorMap& x, const SmallArgs& a, cudaStream_t stream);
// How many clusters of `split` CTAs the device holds at once.
int linear_small_clusters(int split, int num_sms);
// The kernel for operands and outputs of any pitch and alignment; K > 0.
// ma, mb: tensor maps of the operands (boxes of 128 rows, MN-major 64 by 64),
// or null where there can be none.
cudaError_t launch_linear_any(const LinearProduct& p, const CUtensorMap* ma, const CUtensorMap* mb,
                              const CallDevice& dev, cudaStream_t stream);
// The gradient of a weight: C = A·B, or C + A·B, with an epilogue that says
// so; and, unless dbias is null, the sums of A's rows over K, beside the
// product or within it.
int run_wgrad(const LinearProduct& p, float* dbias, bool accumulate, cudaStream_t stream);

struct NormArgs {
  const uint16_t* x;
  int64_t ldx;
  const uint16_t* gamma;
  const uint16_t* beta;      // forward
  float eps;                 // forward
  uint16_t* y;               // forward: y; backward: dx
  int64_t ldy;
  float* mean;               // forward: written, or null; backward: read
  float* rstd;
  const uint16_t* dy;        // backward
  int64_t lddy;
  const uint16_t* res;       // backward, or null
  int64_t ldr;
  float* dgamma;             // backward
  float* dbeta;
  float* work;               // backward: partial sums
  int64_t M, D;
  int* status;               // device watchdog word
  unsigned long long timeout_ns;
  int inject;                // HGEMM_INJECT_* (testing the watchdog)
};
cudaError_t launch_layernorm_forward(const NormArgs& a, int num_sms, cudaStream_t stream);
cudaError_t launch_layernorm_backward(const NormArgs& a, int num_sms, cudaStream_t stream);
size_t layernorm_backward_workspace(int64_t M, int64_t D);

cudaError_t launch_ckpt8_save(const uint16_t* x, int64_t ldx, int8_t* codes, int64_t ldq, float* scales,
                              int64_t lds, int64_t M, int64_t N, cudaStream_t stream);
cudaError_t launch_ckpt8_load(const int8_t* codes, int64_t ldq, const float* scales, int64_t lds, int act,
                              uint16_t* y, int64_t ldy, int64_t M, int64_t N, cudaStream_t stream);

// The norms around a block; kinds are HGEMM_NORM_*, absent vectors null.
struct ResidualNormArgs {
  const uint16_t* x;
  int64_t ldx;
  float alpha;
  const uint16_t* y;
  int64_t ldy;
  const uint16_t* gate;
  int post;
  const uint16_t *post_gamma, *post_beta;
  int pre;
  const uint16_t *pre_gamma, *pre_beta;
  float eps;
  uint16_t* z;
  int64_t ldz;
  uint16_t* h;
  int64_t ldh;
  float* stats;  // [4][M], or null
  int64_t M, D;
};
cudaError_t launch_residual_norm_forward(const ResidualNormArgs& a, int num_sms, cudaStream_t stream);

// At most this many partial sums of the vectors' gradients.
constexpr int kResidualNormPartials = 160;
struct ResidualNormBackArgs {
  const uint16_t* dz;  // or null
  int64_t lddz;
  const uint16_t* dh;
  int64_t lddh;
  const uint16_t* z;
  int64_t ldz;
  const uint16_t* y;
  int64_t ldy;
  float alpha;
  const uint16_t* gate;
  int post;
  const uint16_t *post_gamma, *post_beta;
  int pre;
  const uint16_t* pre_gamma;
  const float* stats;
  uint16_t* dx;
  int64_t lddx;
  uint16_t* dy;
  int64_t lddy;
  float *dgate, *dpost_gamma, *dpost_beta, *dpre_gamma, *dpre_beta;  // each or null
  float* partials;  // the workspace: [partial][4][D], or fewer partials and
  float* means;     // four means for each of the rows m0 .. m1-1
  int64_t M, D, m0, m1;
  int* status;  // device watchdog word
  unsigned long long timeout_ns;
  int inject;   // HGEMM_INJECT_* (testing the watchdog)
};
cudaError_t launch_residual_norm_backward(ResidualNormBackArgs a, int num_sms, cudaStream_t stream);
size_t residual_norm_backward_workspace(int64_t M, int64_t D);

// One tensor of an AdamW step (hgemm_adamw_tensor), and where it begins in the
// launch's numbering of work (set by the launch).
constexpr int kAdamwTensors = 384;  // of one launch, its parameters at most 32764 bytes
struct AdamwEntry {
  uint16_t* weight;
  float* master;
  const void* grad;
  void *m, *v;
  float *ms, *vs;
  int64_t n;
  float decay, keep;  // weight_decay and 1 − lr·weight_decay
  uint32_t chunk0;
  int16_t grad_type;
  int16_t vec;        // the pointers let eight values be moved at once
};
struct AdamwStep {
  float beta1, rest1, beta2, rest2, eps;  // rest: 1 − β
  float gscale, lr, a, b;                 // a = lr/(1 − β1^step), b = 1/√(1 − β2^step)
  float ln1, ln2;                         // ln β, for a step number that the device holds
  float minus_zero;                       // −0, which no compiler folds into what it is added to
  const hgemm_adamw_dynamic* dynamic;     // or null
  uint32_t number;                        // the step's, for random rounding
};
// random: 8-bit states are rounded at random (HGEMM_ROUND_RANDOM).
cudaError_t launch_adamw(const AdamwEntry* t, int count, const AdamwStep& step, bool random, int num_sms,
                         cudaStream_t stream);
cudaError_t launch_adamw_load(const int8_t* m, const float* ms, const uint8_t* v, const float* vs, float* m_out,
                              float* v_out, int64_t n, int num_sms, cudaStream_t stream);

struct ExpertsArgs {
  const uint16_t* X;
  int64_t ldx;
  const uint16_t* Wr;
  int64_t ldwr;
  const uint16_t* W1;
  int64_t ldw1;
  const uint16_t* b1;
  const uint16_t* W2;
  int64_t ldw2;
  const uint16_t* b2;
  int act;
  bool gated, normalize;
  const uint16_t* R;
  int64_t ldr;
  uint16_t* Y;
  int64_t ldy;
  int* chosen;   // M×k, or null
  float* share;
  int M, D, F, E, k;
  // the workspace's parts
  int* ws_chosen;
  float* ws_share;
  uint16_t* ws_h;  // M·k pairs of rows, upper parts and what they leave out
  int64_t ldh;
  float* ws_out;   // [splits][M·k] rows
  int64_t ldo;
  int splits, run;  // the second product's runs of F, and their length
  int router_ctas;  // a cluster of the router
  int* status;      // device watchdog word
  unsigned long long timeout_ns;
  int inject;       // HGEMM_INJECT_* (testing the watchdog)
};
cudaError_t launch_experts(ExpertsArgs a, void* workspace, int num_sms, cudaStream_t stream);
size_t experts_workspace(int64_t M, int64_t D, int64_t F, int64_t E, int64_t k);

// Address of the device watchdog word on the current device.
cudaError_t status_word_address(int** addr);

// The -DHGEMM_DEBUG build's check words, one per kernel file (each sets
// *out to null in the release build).
cudaError_t debug_word_tc(int** out);
cudaError_t debug_word_tc2(int** out);
cudaError_t debug_word_tc2w(int** out);
cudaError_t debug_word_skinny(int** out);
cudaError_t debug_word_generic(int** out);
cudaError_t debug_word_trsm(int** out);
cudaError_t debug_word_trileaf(int** out);
cudaError_t debug_word_chain(int** out);
cudaError_t debug_word_linear(int** out);
cudaError_t debug_word_norm(int** out);
cudaError_t debug_word_ckpt8(int** out);
cudaError_t debug_word_linear_any(int** out);
cudaError_t debug_word_linear_small(int** out);
cudaError_t debug_word_linear_wave(int** out);
cudaError_t debug_word_residual_norm(int** out);
cudaError_t debug_word_adamw(int** out);
cudaError_t debug_word_experts(int** out);
constexpr int kDebugWords = 17;

// Co-residency limits of the cluster kernels on one device, measured once
// (or nominal GB300 figures when no device has been queried).
struct DeviceProfile {
  int num_sms;
  int pair_clusters;    // co-resident 2-CTA clusters of the pair kernel
  int split2_clusters;  // co-resident 4-CTA clusters of the split-K kernel
  int split3_clusters;  // co-resident 6-CTA clusters
  int split4_clusters;  // co-resident 8-CTA clusters
  int split2n_clusters;  // co-resident 4-CTA clusters of the 128-column split-K kernel
};

// Kernel choice for a TMA-able product. Returns an HGEMM_PATH_* value and,
// for the split-K path, the number of K-slices in *split and the tile width
// in *tile_n. forced: a forced HGEMM_PATH_* or -1; forced_split and
// forced_tile_n: a forced split-K configuration or 0; fused: the product
// has a fused epilogue (hgemm_ex other than the plain product).
int choose_tma_path(int64_t M, int64_t N, int64_t K, const DeviceProfile& dev, int forced,
                    int forced_split, int forced_tile_n, bool fused, int* split, int* tile_n);

// Tile geometry of the tensor-core path, for the host-side tensor maps.
constexpr int kTcBM = 128;
constexpr int kTcBN = 256;
constexpr int kNarrowBN = 64;  // single-CTA kernel for outputs of one wave of 128×64 tiles
constexpr int kTcBK = 64;
constexpr int kPairBN = 256;   // pair kernel: 256×256 tiles, 128 B rows per CTA
constexpr int kPairRingBytes = 6 * 32768;  // pair kernel: six whole-tile stages of A and B
constexpr int kEpiRows = 32;   // rows of one staged C box (one epilogue warp)
constexpr int kEpiCols = 64;   // columns of one staged C box (128 bytes)

}  // namespace hg
