// rlscan_sums.hpp -- rows of partial sums, added up by columns in a fixed order.
#ifndef RLSCAN_SUMS_HPP
#define RLSCAN_SUMS_HPP

#include <hip/hip_runtime.h>

#include <cstdint>

namespace rlscan {
namespace sums {

// out0[c] = sum over r of part[r, c] for c < n0, and out1[c - n0] for the n1 columns behind
// them; part [rows, n0 + n1].  Summed in float64, rounded once.  Either output may be NULL: not written.
hipError_t launch_columns(const float* part, int64_t rows, float* out0, int64_t n0, float* out1, int64_t n1,
                          hipStream_t st);

}  // namespace sums
}  // namespace rlscan

#endif
