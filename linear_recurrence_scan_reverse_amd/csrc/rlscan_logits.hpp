// rlscan_logits.hpp -- rows of logits: arguments, launchers and element access
// shared by the sampling and the log-probability kernels.
#ifndef RLSCAN_LOGITS_HPP
#define RLSCAN_LOGITS_HPP

#include <hip/hip_runtime.h>

#include <cstdint>

#include "rlscan.h"

namespace rlscan {
namespace logits {

typedef uint32_t u32x4 __attribute__((ext_vector_type(4)));

constexpr float kNegInf = -__builtin_inff();

// Largest row of logits: sums of weights in units of 2^-43 stay below 2^63.
constexpr int64_t kMaxActions = (int64_t)1 << 20;
constexpr int64_t kMaxSampleRows = ((int64_t)1 << 22) - 1;  // blocks of 1024 threads: below 2^32 work-items

struct SampleArgs {
  const void* x;          // [R, N], rows `stride` elements apart
  int64_t stride;
  const uint8_t* mask;    // [R, N], rows N apart, or NULL
  const float* u;         // [R]
  const float* temperature;  // [R] or NULL: the value below
  const int32_t* top_k;
  const float* top_p;
  const float* min_p;
  float temperature1, top_p1, min_p1;
  int32_t top_k1;
  int64_t* action;        // [R]
  float* log_prob;        // [R] or NULL
  int64_t R, N;
  void* shared;           // workspace where blocks share a row, or NULL
  int64_t shared_words;   // of 8 bytes, for one row
  int slices, tiles, slice_tiles;
};
int64_t sample_workspace(int64_t R, int64_t N);  // bytes; 0: rows are not shared
hipError_t launch_sample(rlscan_format f, const SampleArgs& a, hipStream_t st);

struct LogProbArgs {
  const void* x;
  int64_t stride;
  const uint8_t* mask;
  const int64_t* action;  // [R]
  double inv_t;           // 1 / temperature
  float* log_prob;        // [R]
  float* entropy;         // [R]
  double* lse;            // [R]
  float* part;            // workspace [R, split, 4] where split > 1
  int64_t R, N, split;
  // backward
  const float* d_log_prob;  // [R] or NULL
  const float* d_entropy;   // [R] or NULL
  void* dx;                 // [R, N], rows dx_stride apart
  int64_t dx_stride;
};
hipError_t launch_log_probs(rlscan_format f, const LogProbArgs& a, hipStream_t st);
hipError_t launch_log_probs_backward(rlscan_format f, const LogProbArgs& a, hipStream_t st);

// Blocks that share one row of logits: enough rows fill the card by themselves,
// few long rows are split (at least 8192 logits a block).
inline int64_t log_probs_split(int64_t R, int64_t N) {
  int64_t s = R > 0 ? (512 + R - 1) / R : 1;
  const int64_t most = N / 8192;
  if (s > most) s = most;
  return s < 1 ? 1 : s;
}

struct LF32 {
  using E = float;
  static constexpr int W = 4;     // elements in 16 bytes
  static constexpr int kLow = 0;  // low bits that are zero in every value, as a float32
  static __device__ __forceinline__ float get(E v) { return v; }
  static __device__ __forceinline__ E put(float v) { return v; }
};
struct LBf16 {
  using E = uint16_t;
  static constexpr int W = 8;
  static constexpr int kLow = 16;
  static __device__ __forceinline__ float get(E v) { return __builtin_bit_cast(float, (uint32_t)v << 16); }
  static __device__ __forceinline__ E put(float v) { return __builtin_bit_cast(uint16_t, (__bf16)v); }
};
struct LF16 {
  using E = uint16_t;
  static constexpr int W = 8;
  static constexpr int kLow = 13;
  static __device__ __forceinline__ float get(E v) { return (float)__builtin_bit_cast(_Float16, v); }
  static __device__ __forceinline__ E put(float v) { return __builtin_bit_cast(uint16_t, (_Float16)v); }
};

// The W elements of one 16-byte load.
template <class F>
union Vec {
  u32x4 w;
  typename F::E e[F::W];
};

}  // namespace logits
}  // namespace rlscan

#endif
