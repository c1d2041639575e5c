// Calls with more rows than one launch can hold (internal to libnmsparse).
//
// The work-items of a launch in one dimension have to stay below 2^32: the runtime takes a larger grid
// modulo 2^32, without an error.  Calls over tokens or rows are made in pieces that stay below it.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

namespace nms {

// A power of two, so that a piece's rows keep their alignment; with 64 work-items or fewer a row, as every
// kernel called by pieces of this many rows has, 2^30 work-items.
constexpr int64_t kPieceRows = int64_t(1) << 24;
// The same where a row takes 256 work-items.
constexpr int64_t kPieceRows256 = int64_t(1) << 22;

// launch(first row, rows) for every piece, until one fails.
template <typename F>
inline hipError_t in_pieces(int64_t rows, int64_t piece, F launch) {
  for (int64_t r0 = 0; r0 < rows; r0 += piece) {
    const hipError_t e = launch(r0, rows - r0 < piece ? rows - r0 : piece);
    if (e != hipSuccess) return e;
  }
  return hipSuccess;
}

inline bool grid_ok(int64_t workgroups, int threads) { return workgroups <= (int64_t)UINT32_MAX / threads; }

}  // namespace nms
