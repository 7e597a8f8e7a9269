// Linear attention over whole rows (rlscan_linear_attention).
//
// One chunk walk for each head (rlscan_la_attend.hpp).  Where the heads are too few to
// fill the card, rows are cut into segments: a first pass (rlscan_la_walk.hpp) computes what
// each segment adds to the state, a second joins these along the row, and the segments are
// walked side by side from the states so found; k and v are read twice.
//
// Measured (bfloat16, kernels in a run of 300 calls; in the first dozen of a process they take
// a tenth to a third longer): 256 rows of 256 steps, 8 heads of 64, gates for each step: 87
// us, 3.9 TB/s of its 338 MB; reading and writing them by a copy takes 64.  One row of 32768
// steps, 16 heads of 128 in groups of 4: 73 us for the segments' states, 8 to join them, 145
// for the walk.  What bounds the walk is the chain within a chunk (products, decays and masks
// on a C x C tile, products again), not memory.  At 128 a compute unit holds one block: eight
// waves of 255 or 256 registers.  The walk without care needs 199 to 247 and spills none; the
// one with care spills up to 51, and up to 87 where rows cannot be read 16 bytes at a time (the
// walk without care up to 3 there).  At 64 three blocks of bfloat16 fit: 2048 blocks are 2.67
// rounds of the card.
#include "rlscan_la_attend.hpp"
#include "rlscan_la_launch.hpp"
#include "rlscan_la_walk.hpp"

namespace rlscan {
namespace la {

struct ForwardArgs {
  Args a;
  Attend t;
  int64_t nvs;
};

// A block: one head, CD columns of V, one segment.
template <class F, int AD, int CD, int C, int NWV, int MINW, bool VEC>
__global__ void __launch_bounds__(64 * NWV, MINW) forward_kernel(const ForwardArgs p) {
  __shared__ AttendLds<F, AD, CD, C, NWV, false> s;
  const int64_t EH = p.a.E * p.a.H;
  const int64_t eh = blockIdx.x % EH, rest = blockIdx.x / EH;
  attend<F, F, AD, CD, C, NWV, false, false, F::NW, VEC>(s, p, &ForwardArgs::t, eh, rest / p.nvs,
                                                         (int)(rest % p.nvs) * CD);
}

template <class F, int KP, int CD, int C, int NWV, int MINW, bool VEC>
hipError_t launch_forward_as(const Args& a, const Plan& pl, hipStream_t st) {
  enter_segments<F, KP, C, false, VEC>(a, pl.VP, a.init, a.seg_state, a.seg_decay, st);
  Attend t{};
  t.a = a.q;
  t.b = a.k;
  t.c = a.v;
  t.out = a.out;
  t.ga = 1;
  t.gb = t.gc = a.G;
  t.A = a.K;
  t.D = a.V;
  if (pl.nseg > 1) t.enter = StateView{a.seg_state, pl.nseg * KP * pl.VP, KP * pl.VP, pl.VP, 1};
  else t.enter = StateView{const_cast<float*>(a.init), (int64_t)a.K * a.V, 0, a.V, 1};
  t.leave = StateView{a.final_state, (int64_t)a.K * a.V, 0, a.V, 1};
  t.leave_closed = 1;
  const int64_t nvs = pl.VP / CD;
  forward_kernel<F, KP, CD, C, NWV, MINW, VEC><<<dim3((unsigned)(a.E * a.H * nvs * pl.nseg)), 64 * NWV, 0, st>>>(ForwardArgs{a, t, nvs});
  return hipGetLastError();
}

template <class F, bool VEC>
hipError_t launch_forward_fmt(const Args& a, const Plan& pl, hipStream_t st) {
  if (pl.KP == 64) return launch_forward_as<F, 64, 64, 32, 4, F::NT == 1 ? 3 : 2, VEC>(a, pl, st);
  return launch_forward_as<F, 128, 128, F::NT == 1 ? 64 : 32, 8, 2, VEC>(a, pl, st);
}

template <class F>
hipError_t launch_forward_vec(const Args& a, const Plan& pl, hipStream_t st) {
  return a.q.vec && a.k.vec && a.v.vec && a.out.vec ? launch_forward_fmt<F, true>(a, pl, st) : launch_forward_fmt<F, false>(a, pl, st);
}

hipError_t launch_forward(rlscan_format f, const Args& a, const Plan& pl, hipStream_t st) {
  switch (f) {
    case RLSCAN_FORMAT_BF16: return launch_forward_vec<TBf16>(a, pl, st);
    case RLSCAN_FORMAT_F16: return launch_forward_vec<TF16>(a, pl, st);
    default: return launch_forward_vec<TF32>(a, pl, st);
  }
}

}  // namespace la
}  // namespace rlscan
