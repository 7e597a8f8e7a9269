// rlscan_la_launch.hpp -- shape plan and launchers of the linear-attention kernels.
#ifndef RLSCAN_LA_LAUNCH_HPP
#define RLSCAN_LA_LAUNCH_HPP

#include "rlscan_la.hpp"

namespace rlscan {
namespace la {

constexpr int64_t kFillBlocks = 512;  // two blocks for each of the card's 256 compute units
constexpr int64_t kMaxBlocks = ((int64_t)1 << 24) - 1;  // of 256 threads: below 2^32 work-items

// How a call is cut up; a function of its sizes and storage format alone.
struct Plan {
  int KP;              // K and V padded to the kernels' tiles
  int64_t VP;
  int64_t C;           // steps of a chunk
  int64_t chunks;
  int64_t nseg, seg_chunks;
  // workspace, in floats
  int64_t seg_state, seg_decay;          // one direction's segment values
  int64_t states;                        // one direction's chunk values (backward)
  int64_t dg;                            // per-step decay gradients behind a [H] gradient
  int64_t floats;                        // total
};

// Segments per row: enough to give kFillBlocks blocks, none shorter than `least`
// chunks (a segment costs one more pass over its k and v, and a state).
inline void cut_segments(Plan& p, int64_t blocks, int64_t least) {
  int64_t want = blocks > 0 ? (kFillBlocks + blocks - 1) / blocks : 1;
  const int64_t most = p.chunks / least;
  if (want > most) want = most;
  if (want < 1) want = 1;
  p.seg_chunks = (p.chunks + want - 1) / want;
  if (p.seg_chunks < 1) p.seg_chunks = 1;
  p.nseg = p.chunks > 0 ? (p.chunks + p.seg_chunks - 1) / p.seg_chunks : 1;
}

inline Plan make_plan(rlscan_format f, int64_t E, int64_t T, int64_t H, int64_t K, int64_t V, bool backward,
                      bool per_head) {
  Plan p{};
  p.KP = K <= 64 ? 64 : 128;
  p.VP = V <= 64 ? 64 : 128;
  p.C = backward && f != RLSCAN_FORMAT_BF16 ? 32 : 64;
  p.chunks = (T + p.C - 1) / p.C;
  cut_segments(p, E * H * (p.VP / 64) * (backward ? 2 : 1), 4);
  const int64_t state = E * H * p.KP * p.VP;
  if (p.nseg > 1) {
    p.seg_state = state * p.nseg;
    p.seg_decay = (E * H * p.nseg + 3) / 4 * 4;
  }
  p.floats = (p.seg_state + p.seg_decay) * (backward ? 2 : 1);
  if (backward) {
    p.states = state * p.chunks;
    p.dg = per_head ? (E * T * H + 3) / 4 * 4 : 0;
    p.floats += 2 * p.states + p.dg;
  }
  return p;
}

hipError_t launch_forward(rlscan_format f, const Args& a, const Plan& pl, hipStream_t st);
// dg_head: [H] gradient of one log-decay for each head, summed from a.dg, or NULL.
hipError_t launch_backward(rlscan_format f, const Args& a, const Plan& pl, float* dg_head, hipStream_t st);

// One step of E rows on pooled states.
struct StepArgs {
  const void *q, *k, *v;       // [E, heads, D] by strides (elements)
  int64_t q_se, q_sh, k_se, k_sh, v_se, v_sh;
  const float* g;              // log-decays, strides 0 where broadcast
  int64_t g_se, g_sh;
  const uint8_t* reset;        // [E] or NULL
  const int32_t* slots;        // [E] or NULL
  float* state;                // [S, H, K, V]
  void* out;                   // [E, H, V]
  int64_t o_se, o_sh;
  int64_t E, H, G, S;
  int K, V;
  float scale;
};
hipError_t launch_step(rlscan_format f, const StepArgs& a, hipStream_t st);

}  // namespace la
}  // namespace rlscan

#endif
