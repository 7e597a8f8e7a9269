// Rows of partial sums added up by columns (the learned rates and weights of the gated
// recurrence and of the normalised heads).  16 columns a block, 64 threads to a
// column with every 64th row each, then a tree: few rows and few columns make this a matter of
// latency, so the loads are spread over as many threads as there are rows.  Measured: 768 rows of 256
// columns 4.6 us, 1025 of 512 5.6, 2049 of 256 6.1; in two steps, blocks of 512 rows first, 8.8 and 9.4.
// Its callers make a few thousand rows at most.
#include "rlscan_sums.hpp"

namespace rlscan {
namespace sums {

__global__ void __launch_bounds__(1024) columns_kernel(const float* part, int64_t rows, float* out0, int64_t n0,
                                                       float* out1, int64_t n1) {
  __shared__ double s[64][17];
  const int c = threadIdx.x & 15, r = threadIdx.x >> 4;
  const int64_t n = n0 + n1, col = (int64_t)blockIdx.x * 16 + c;
  double sum = 0.0;
  if (col < n) {
#pragma unroll 8
    for (int64_t i = r; i < rows; i += 64) sum += (double)part[i * n + col];
  }
  s[r][c] = sum;
  for (int half = 32; half > 0; half /= 2) {
    __syncthreads();
    if (r < half) s[r][c] += s[r + half][c];
  }
  if (r != 0 || col >= n) return;
  float* out = col < n0 ? out0 : out1;
  if (out) out[col < n0 ? col : col - n0] = (float)s[0][c];
}

hipError_t launch_columns(const float* part, int64_t rows, float* out0, int64_t n0, float* out1, int64_t n1,
                          hipStream_t st) {
  columns_kernel<<<dim3((unsigned)((n0 + n1 + 15) / 16)), 1024, 0, st>>>(part, rows, out0, n0, out1, n1);
  return hipGetLastError();
}

}  // namespace sums
}  // namespace rlscan
