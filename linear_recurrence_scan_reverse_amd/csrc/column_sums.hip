// Rows of partial sums added up by columns (the learned rates and weights of the gated
// recurrence and of the normalised heads).  16 columns a block, 64 threads to a
// column with every 64th row each, then a tree: few rows and few columns make this a matter of
// latency, so the loads are spread over as many threads as there are rows.
#include "rlscan_sums.hpp"

namespace rlscan {
namespace sums {

template <class In>
__global__ void __launch_bounds__(1024) columns_kernel(const In* part, int64_t rows, int64_t per, double* more,
                                                       float* out0, int64_t n0, float* out1, int64_t n1) {
  __shared__ double s[64][17];
  const int c = threadIdx.x & 15, r = threadIdx.x >> 4;
  const int64_t n = n0 + n1, col = (int64_t)blockIdx.x * 16 + c;
  const int64_t from = blockIdx.y * per, to = from + per < rows ? from + per : rows;
  double sum = 0.0;
  if (col < n) {
#pragma unroll 8
    for (int64_t i = from + r; i < to; i += 64) sum += (double)part[i * n + col];
  }
  s[r][c] = sum;
  for (int half = 32; half > 0; half /= 2) {
    __syncthreads();
    if (r < half) s[r][c] += s[r + half][c];
  }
  if (r != 0 || col >= n) return;
  if (more) {
    more[blockIdx.y * n + col] = s[0][c];
    return;
  }
  float* out = col < n0 ? out0 : out1;
  if (out) out[col < n0 ? col : col - n0] = (float)s[0][c];
}

hipError_t launch_columns(const float* part, int64_t rows, float* more, float* out0, int64_t n0, float* out1,
                          int64_t n1, hipStream_t st) {
  const unsigned tiles = (unsigned)((n0 + n1 + 15) / 16);
  if (!more || more_floats(rows, n0 + n1) == 0) {
    columns_kernel<float><<<dim3(tiles), 1024, 0, st>>>(part, rows, rows, nullptr, out0, n0, out1, n1);
    return hipGetLastError();
  }
  double* const sums = reinterpret_cast<double*>(more);
  columns_kernel<float><<<dim3(tiles, (unsigned)blocks_of(rows)), 1024, 0, st>>>(part, rows, rows_of(rows), sums, out0, n0, out1, n1);
  const hipError_t e = hipGetLastError();
  if (e != hipSuccess) return e;
  columns_kernel<double><<<dim3(tiles), 1024, 0, st>>>(sums, blocks_of(rows), blocks_of(rows), nullptr, out0, n0, out1, n1);
  return hipGetLastError();
}

}  // namespace sums
}  // namespace rlscan
