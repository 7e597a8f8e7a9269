// rlscan_sums.hpp -- rows of partial sums, added up by columns in a fixed order.
#ifndef RLSCAN_SUMS_HPP
#define RLSCAN_SUMS_HPP

#include <hip/hip_runtime.h>

#include <cstdint>

namespace rlscan {
namespace sums {

// Many rows are added up in two steps: blocks of kRows or more first, their sums (float64) into `more`.
constexpr int64_t kRows = 512, kMostBlocks = 65535;
inline int64_t rows_of(int64_t rows) { return rows > kRows * kMostBlocks ? (rows + kMostBlocks - 1) / kMostBlocks : kRows; }
inline int64_t blocks_of(int64_t rows) { return (rows + rows_of(rows) - 1) / rows_of(rows); }
// Floats of `more`; 0: one step.
inline int64_t more_floats(int64_t rows, int64_t n) { return rows > 2 * kRows ? (2 * blocks_of(rows) * n + 3) / 4 * 4 : 0; }

// out0[c] = sum over r of part[r, c] for c < n0, and out1[c - n0] for the n1 columns behind
// them; part [rows, n0 + n1], more [more_floats(rows, n0 + n1)], 8-byte aligned, or NULL for one step
// however many rows there are.  Summed in float64, rounded once.  Either output may be NULL: not written.
hipError_t launch_columns(const float* part, int64_t rows, float* more, float* out0, int64_t n0, float* out1,
                          int64_t n1, hipStream_t st);

}  // namespace sums
}  // namespace rlscan

#endif
