// rlscan_nr.hpp -- normalised and rotated heads: arguments and launchers.
#ifndef RLSCAN_NR_HPP
#define RLSCAN_NR_HPP

#include "rlscan_la.hpp"
#include "rlscan_logits.hpp"

namespace rlscan {
namespace nr {

using la::View;

struct Args {
  View in[2], out[2];        // queries and keys; backward: out are the inputs' gradients
  View grad[2];              // backward: of the outputs
  int64_t heads[2];
  const float* weight[2];    // [D] or NULL: ones
  const int32_t* pos;        // by strides; not read where R is 0
  int64_t p_se, p_st;
  int64_t E, T;
  int D, R;                  // R of the D are rotated, in R / 2 pairs
  int interleaved;           // pairs 2j, 2j + 1, else j, j + R / 2
  float eps;
  double base;
  float* part;               // backward: workspace [blocks, 2 D]
  float* d_weight[2];        // [D] or NULL
};

// What is taken at once: a function of sizes, strides and alignment alone.
struct Plan {
  int V;           // pairs to a lane
  int vec;         // side by side, in loads of V elements
  int log_lanes;   // lanes to a head
  int64_t split;   // units that share a token's heads
  int64_t blocks;
};
Plan make_plan(rlscan_format f, const Args& a, bool backward);
int64_t backward_blocks(int64_t tokens, int64_t heads, int D);  // at most, whatever the strides

hipError_t launch_forward(rlscan_format f, const Args& a, hipStream_t st);
hipError_t launch_backward(rlscan_format f, const Args& a, hipStream_t st);

}  // namespace nr
}  // namespace rlscan

#endif
