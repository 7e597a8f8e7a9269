// rlscan_gr.hpp -- the gated recurrence: arguments, launch plan and the arithmetic that its
// kernels share.
//
// Per row and channel, with s_t = rate * sigmoid(r_t),
//   h_t = a_t h_{t-1} + m_t u_t,   a_t = exp(-s_t),  m_t = sqrt(1 - a_t^2),  u_t = sigmoid(i_t) x_t,
// and a_t = 0 where step t-1 ended an episode.  A chunk of steps takes the value c that
// enters it to A c + y, A = exp(-sum s) and y what leaves it for c = 0; such pairs are
// joined over waves (through LDS) and over segments of a row (through the workspace).
//
// Numbers.  Everything is float32.  The decay is held as a - 1 (expm1), whose relative
// error stays at a few 2^-24 however near a is to 1: h + (a - 1) h keeps memories of thousands
// of steps exact, and 1 - a^2 = (1 - a)(1 + a) does not cancel.  A product of decays
// is the exponential of a sum.
#ifndef RLSCAN_GR_HPP
#define RLSCAN_GR_HPP

#include "rlscan_la.hpp"
#include "rlscan_logits.hpp"

namespace rlscan {
namespace gr {

using la::View;
using logits::LBf16;
using logits::LF16;
using logits::LF32;

constexpr int kMark = RLSCAN_MARK_STEPS;  // steps from one marked state to the next

struct Args {
  View x, ig, dg;         // values and the two gates' logits (heads unused)
  View dout;              // backward
  View out, dx, dig, ddg; // outputs
  const float* rate;      // [D]
  const uint8_t* done;    // [E, T] or [T, E] by strides, or NULL
  int64_t d_se, d_st;
  const float* init;      // [E, D] or NULL
  const float* d_final;   // [E, D] or NULL
  float* final_state;     // [E, D] or NULL
  float* d_init;          // [E, D] or NULL
  float* marks;           // [E, ceil(T / kMark), D]: the state before every kMark-th step, or NULL
  float* seg_a;           // workspace [E, nseg, D]: each segment's pair
  float* seg_y;
  float* d_rate;          // [D]
  float* rate_part;       // workspace [groups * nseg, D]
  int64_t E, T, D;
  int64_t nseg, seg_steps;  // steps of a segment, a multiple of what a block takes at once
  int64_t groups;           // backward: blocks take the rows e, e + groups, ...
};

struct Plan {
  int waves;           // of a block, each with kMark steps
  int64_t nseg, seg_steps, groups;
  int64_t seg, part;   // floats of one array
  int64_t floats;      // workspace in all
};
Plan make_plan(rlscan_format f, int64_t E, int64_t T, int64_t D, bool backward);

hipError_t launch_forward(rlscan_format f, const Args& a, const Plan& p, hipStream_t st);
hipError_t launch_backward(rlscan_format f, const Args& a, const Plan& p, hipStream_t st);

// One step of E rows on pooled states.
struct StepArgs {
  const void *x, *ig, *dg;  // [E, D], rows by strides (elements)
  int64_t x_se, ig_se, dg_se, o_se;
  const float* rate;
  const uint8_t* reset;     // [E] or NULL
  const int32_t* slots;     // [E] or NULL
  float* state;             // [S, D]
  void* out;
  int64_t E, S, D;
};
hipError_t launch_step(rlscan_format f, const StepArgs& a, hipStream_t st);

constexpr float kLog2E = 1.44269504088896340736f;

__device__ __forceinline__ float exp2_fast(float x) { return __builtin_amdgcn_exp2f(x); }
__device__ __forceinline__ float sigmoid(float z) {
  return __builtin_amdgcn_rcpf(1.0f + exp2_fast(-kLog2E * z));
}

// exp(-s) - 1 for s >= 0: below a quarter the series (its next term is 2^-24 of the
// value), above it 1 - exp(-s) >= 0.22 loses at most two bits.
__device__ __forceinline__ float decay_less_1(float s) {
  const float far = exp2_fast(-kLog2E * s) - 1.0f;
  float p = __builtin_fmaf(s, 1.0f / 720.0f, -1.0f / 120.0f);
  p = __builtin_fmaf(s, p, 1.0f / 24.0f);
  p = __builtin_fmaf(s, p, -1.0f / 6.0f);
  p = __builtin_fmaf(s, p, 0.5f);
  p = __builtin_fmaf(s, p, -1.0f);
  return s < 0.25f ? s * p : far;
}
// 1 - a^2 from a - 1
__device__ __forceinline__ float one_less_square(float em1) { return -em1 * (2.0f + em1); }

// a h from a - 1
__device__ __forceinline__ float decayed(float em1, float h) { return __builtin_fmaf(em1, h, h); }

// The pair of a chunk as the waves and segments exchange it: A is kDropped where the chunk
// holds a cut, which takes any c, inf and NaN too, to y.
constexpr float kDropped = -1.0f;
__device__ __forceinline__ float enter(float A, float y, float c) { return A < 0.0f ? y : __builtin_fmaf(A, c, y); }

}  // namespace gr
}  // namespace rlscan

#endif
