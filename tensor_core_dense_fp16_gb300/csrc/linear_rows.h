// linear_rows.h — index arithmetic of the few-row linear kernels, host-testable:
// sizes reach 2^31 - 1, and the walk along K looks a few thousand past its end.
#pragma once

#include <cstdint>

#if defined(__CUDACC__)
#define HG_ROWS_FN __host__ __device__ constexpr
#else
#define HG_ROWS_FN constexpr
#endif

namespace hg {

constexpr int kRowsFeatures = 16;  // per block
constexpr int kRowsPiece = 32;     // of K, per warp and step
constexpr int kRowsAhead = 4;      // pieces in flight per warp, at most
constexpr int kRowsWarps = 16;     // at most

// A position along K: unsigned, so that K ≤ 2^31 - 1 leaves room for every
// position that the walk looks at.
using RowsK = uint32_t;
static_assert(0x7FFFFFFFu + 24u + 2u * kRowsAhead * kRowsWarps * kRowsPiece > 0x7FFFFFFFu, "no wrap-around");

// Where lane slot t (of 4) of a warp begins, and its position `pieces` pieces
// of all the warps further on.
HG_ROWS_FN RowsK rows_begin(int warp, int t) { return static_cast<RowsK>(warp * kRowsPiece + 8 * t); }
HG_ROWS_FN RowsK rows_on(RowsK k, int pieces, int warps) {
  return k + static_cast<RowsK>(pieces * warps * kRowsPiece);
}
HG_ROWS_FN bool rows_inside(RowsK k, int K) { return k < static_cast<RowsK>(K); }

HG_ROWS_FN int64_t rows_blocks(int N) { return (static_cast<int64_t>(N) + kRowsFeatures - 1) / kRowsFeatures; }
HG_ROWS_FN int64_t rows_pieces(int K) { return (static_cast<int64_t>(K) + kRowsPiece - 1) / kRowsPiece; }
// 128-byte lines of a feature's weights.
HG_ROWS_FN int rows_lines(int K) { return static_cast<int>((static_cast<int64_t>(K) + 63) / 64); }

// Tiles of `size` over a dimension.
HG_ROWS_FN int64_t tiles_of(int n, int size) { return (static_cast<int64_t>(n) + size - 1) / size; }

}  // namespace hg
