// rlscan_embed.hpp -- rows of a table by token: arguments, workspace and launchers.
#ifndef RLSCAN_EMBED_HPP
#define RLSCAN_EMBED_HPP

#include <hip/hip_runtime.h>

#include <cstdint>

#include "rlscan_logits.hpp"

namespace rlscan {
namespace embed {

constexpr int64_t kMaxKinds = (int64_t)1 << 20;   // two digits of at most ten bits
constexpr int64_t kMaxTokens = (int64_t)1 << 26;

struct LookupArgs {
  const void* table;       // [N, D], rows t_stride apart
  int64_t t_stride;
  const int64_t* tokens;   // [R]
  void* out;               // [R, D], rows o_stride apart
  int64_t o_stride;
  int64_t R, N, D;
  float scale;
};
hipError_t launch_lookup(rlscan_format f, const LookupArgs& a, hipStream_t st);

// How the gradient's tokens are sorted, or added up without (all zero: by one launch, which needs no
// workspace); a function of R, N and D alone.
struct Plan {
  int64_t blocks, per;     // of the sort (or shares of the tokens), and tokens to each
  int passes, bits[2];     // digits, lowest first
  int64_t chunks;          // of kChunk sorted tokens
  // workspace, in bytes, each a multiple of 16
  int64_t keys, hist, present, part;
  int64_t bytes;
};
constexpr int kChunk = 32;
Plan make_plan(int64_t R, int64_t N, int64_t D);

struct GradArgs {
  const void* d_out;       // [R, D], rows o_stride apart
  int64_t o_stride;
  const int64_t* tokens;   // [R]
  void* d_table;           // [N, D], rows t_stride apart
  int64_t t_stride;
  void* workspace;
  int64_t R, N, D;
  float scale;
};
hipError_t launch_backward(rlscan_format f, const GradArgs& a, hipStream_t st);

}  // namespace embed
}  // namespace rlscan

#endif
