// rlscan_la_launch.hpp -- shape plan and launchers of the linear-attention kernels.
#ifndef RLSCAN_LA_LAUNCH_HPP
#define RLSCAN_LA_LAUNCH_HPP

#include "rlscan_la.hpp"

namespace rlscan {
namespace la {

constexpr int64_t kMaxBlocks = ((int64_t)1 << 24) - 1;  // of 256 threads: below 2^32 work-items

// How a call is cut up; a function of its sizes and storage format alone.
struct Plan {
  int KP;              // K and V padded to the kernels' tiles
  int64_t VP;
  int64_t C;           // steps of a chunk
  int64_t chunks;
  int64_t nseg, seg_chunks;
  // workspace, in floats (each a multiple of 4)
  int64_t seg_state, seg_decay;  // one direction's segment values
  int64_t dots;                  // backward: u or w, in float64
  int64_t heads;                 // backward: one float for each row and head
  int64_t dk, dv;                // backward: gradients before heads are added up
  int64_t mark_chunks, nmarks;   // backward: marked boundaries (la_backward.hip)
  int64_t marks;                 // one direction's states there
  int64_t floats;                // total
};

inline int64_t round4(int64_t n) { return (n + 3) / 4 * 4; }

// Segments per row: enough to give `fill` blocks, none shorter than `least` chunks (a
// segment costs one more pass over its k and v, and a state).  Calls without segments, with
// half of `fill`, with it and with twice it, us:
//   heads  steps  forward, bfloat16 128     forward, bfloat16 64     gradients, bfloat16 128
//     1     8192   457   45   45   45        398   40   40   39       919  109  109  110
//    16     8192   470  109   80  103        406   59   50   50       972  532  362  327
//    64     4096   253  202  138  154        208   97   70   72       535  534  676  572
//    96     4096   256  211  244  225        215  140   99   96       778  779  778  836
//   160     2048   139  138  203  191        112  112   82   84       541  540  541  643
//   300     2048   271  272  271  318        139  139  140  133       935  934  935  937
// float32 goes the same way.  The count of blocks says nothing of how full their last round on
// the card is: just below `fill` (96 and 160 heads of 128 forward, 64 in the gradients) rows in one
// piece, or in fewer, are up to a third faster.
inline void cut_segments(Plan& p, int64_t blocks, int64_t fill, int64_t least) {
  int64_t want = blocks > 0 ? (fill + blocks - 1) / blocks : 1;
  const int64_t most = p.chunks / least;
  if (want > most) want = most;
  if (want < 1) want = 1;
  p.seg_chunks = (p.chunks + want - 1) / want;
  if (p.seg_chunks < 1) p.seg_chunks = 1;
  p.nseg = p.chunks > 0 ? (p.chunks + p.seg_chunks - 1) / p.seg_chunks : 1;
}

inline Plan make_plan(rlscan_format f, int64_t E, int64_t T, int64_t H, int64_t G, int64_t K, int64_t V, bool backward) {
  Plan p{};
  // K and V share one padded size: 64 or 128.  Chunks of 64 steps where their tiles leave
  // room for it: bfloat16 at 128 (forward, 32768 steps of 16 heads: 164 us against 182 with 32);
  // at 64 and in the formats of two and three terms more blocks of 32 fit a compute
  // unit (bfloat16, 256 rows of 256 steps, 8 heads: 85 us against 98 with 64).
  p.KP = K <= 64 && V <= 64 ? 64 : 128;
  p.VP = p.KP;
  p.C = f == RLSCAN_FORMAT_BF16 && p.KP == 128 ? 64 : 32;
  p.chunks = (T + p.C - 1) / p.C;
  if (backward) cut_segments(p, E * H * 3, 256, 256 / p.C);
  else cut_segments(p, E * H, p.KP == 128 ? 256 : 512, 256 / p.C);
  if (p.nseg > 1) {
    p.seg_state = E * H * p.KP * p.VP * p.nseg;
    p.seg_decay = round4(E * H * p.nseg);
  }
  p.floats = (p.seg_state + p.seg_decay) * (backward ? 2 : 1);
  if (backward) {
    p.dots = round4(2 * E * H * T);
    p.heads = round4(E * H);
    p.dk = G > 1 ? round4(E * T * H * K) : 0;
    p.dv = G > 1 ? round4(E * T * H * V) : 0;
    // The decay's gradient is summed from one marked boundary to the next: 64 steps in
    // formats whose other errors are smaller than what a longer sum adds, 512 in bfloat16.
    p.mark_chunks = (f == RLSCAN_FORMAT_BF16 ? 512 : 64) / p.C;
    p.nmarks = p.chunks > 0 ? (p.chunks - 1) / p.mark_chunks : 0;
    p.marks = E * H * p.nmarks * p.KP * p.VP;
    p.floats += 2 * p.dots + 3 * p.heads + p.dk + p.dv + 2 * p.marks + round4(2 * E * H * p.nmarks);
  }
  return p;
}

hipError_t launch_forward(rlscan_format f, const Args& a, const Plan& pl, hipStream_t st);
hipError_t launch_backward(rlscan_format f, const Args& a, const Backward& b, const Plan& pl, hipStream_t st);

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
