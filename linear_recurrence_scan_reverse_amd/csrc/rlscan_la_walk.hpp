// rlscan_la_walk.hpp -- the states of linear attention at chunk or segment ends.
//
// walk_kernel carries one head's state over the chunks of a segment, a 64-column
// slice of V per block: forward with S = across S + sum_j leave_j k_j v_j^T, and
// backward in time with the gradient of the state, the same recurrence reversed:
// dS = across dS + sum_i entry_i q_i dout_i^T.  combine_kernel joins segments.
#ifndef RLSCAN_LA_WALK_HPP
#define RLSCAN_LA_WALK_HPP

#include "rlscan_la.hpp"

namespace rlscan {
namespace la {

// What one walk reads and writes.
struct WalkArgs {
  Args a;
  int64_t VP;          // columns of a state in the workspace
  const float* enter;  // [E, H, nseg, KP, VP] value entering each segment, or NULL: zeros
  const float* given;  // [E, H, K, V] value entering the whole row if enter is NULL, or NULL
  float* each;         // [E, H, chunks, KP, VP] value before each chunk in walking order, or NULL
  float* seg_end;      // [E, H, nseg, KP, VP]: value after segment s goes to s + 1, or NULL
  float* seg_decay;    // [E, H, nseg] with seg_end
  float* end;          // [E, H, K, V] value after the row's last chunk, or NULL
};

// Whether the row's last step ends an episode, so that nothing leaves the row.
__device__ __forceinline__ bool row_closed(const Args& a, int64_t e) {
  return a.T > 0 && a.done && a.done[e * a.d_se + (a.T - 1) * a.d_st] != 0;
}

// A block: head eh = e*H + h, 64 columns of V, one segment.  Wave w holds the 16
// columns w*16 ... of the slice for all KP rows: accumulator tile kt, lane l holds
// S[kt*16 + l%16][w*16 + (l/16)*4 + r].
template <class F, int KP, int C, bool REV>
__global__ void __launch_bounds__(kThreads) walk_kernel(const WalkArgs p) {
  constexpr int NT = F::NT, NW = F::NW, KT = KP / 16;
  __shared__ Tile<NT, C, KP> xs;
  __shared__ Tile<NT, C, 64> ys;
  __shared__ Decay<C> dec;
  const Args& a = p.a;
  const int tid = threadIdx.x, lane = tid & 63, w = tid >> 6, col = lane & 15, grp = lane >> 4;
  const int64_t EH = a.E * a.H, nvs = p.VP / 64;
  const int64_t eh = blockIdx.x % EH, rest = blockIdx.x / EH;
  const int64_t vs = rest % nvs, seg = rest / nvs;
  const int64_t e = eh / a.H, h = eh % a.H;
  const View& X = REV ? a.q : a.k;
  const View& Y = REV ? a.dout : a.v;
  const int64_t hx = REV ? h : h / a.G, hy = hx;
  const int v0 = (int)vs * 64;
  const int vc = v0 + w * 16 + grp * 4;  // this lane's four columns

  f32x4 S[KT];
  const int64_t state = (int64_t)KP * p.VP;
#pragma unroll
  for (int kt = 0; kt < KT; ++kt) {
    const int k = kt * 16 + col;
    S[kt] = f32x4{0, 0, 0, 0};
    if (p.enter) {
      S[kt] = *reinterpret_cast<const f32x4*>(p.enter + (eh * a.nseg + seg) * state + (int64_t)k * p.VP + vc);
    } else if (p.given && k < a.K && !(REV && row_closed(a, e))) {
#pragma unroll
      for (int r = 0; r < 4; ++r)
        if (vc + r < a.V) S[kt][r] = p.given[(eh * a.K + k) * a.V + vc + r];
    }
  }

  const int64_t p0 = seg * a.seg_chunks;
  const int64_t p1 = p0 + a.seg_chunks < a.chunks ? p0 + a.seg_chunks : a.chunks;
  auto chunk_t0 = [&](int64_t n) { return (REV ? a.chunks - 1 - n : n) * C; };
  Piece<F> rx[Share<C, KP>::n], ry[Share<C, 64>::n];
  StepDecay sd{0.0f, false};
  float decay = 1.0f;
  if (p0 < p1) {
    fetch<F, C, KP>(X, e, hx, chunk_t0(p0), a.T, 0, a.K, tid, rx);
    fetch<F, C, 64>(Y, e, hy, chunk_t0(p0), a.T, v0, a.V, tid, ry);
    if (w == 0) sd = load_decay<C>(a, e, h, chunk_t0(p0), lane);
  }
  for (int64_t n = p0; n < p1; ++n) {
    stage<F, C, KP>(xs, rx, tid);
    stage<F, C, 64>(ys, ry, tid);
    if (w == 0) fill_decay<C>(dec, sd, a.scale, lane);
    __syncthreads();
    if (n + 1 < p1) {
      fetch<F, C, KP>(X, e, hx, chunk_t0(n + 1), a.T, 0, a.K, tid, rx);
      fetch<F, C, 64>(Y, e, hy, chunk_t0(n + 1), a.T, v0, a.V, tid, ry);
      if (w == 0) sd = load_decay<C>(a, e, h, chunk_t0(n + 1), lane);
    }
    if (p.each) {
      float* to = p.each + (eh * a.chunks + (REV ? a.chunks - 1 - n : n)) * state;
#pragma unroll
      for (int kt = 0; kt < KT; ++kt)
        *reinterpret_cast<f32x4*>(to + (int64_t)(kt * 16 + col) * p.VP + vc) = S[kt];
    }
    const float across = dec.across;
    decay *= across;
#pragma unroll
    for (int kt = 0; kt < KT; ++kt) S[kt] *= across;
#pragma unroll
    for (int jj = 0; jj < C / 32; ++jj) {
      float y[8];
      join<NT>(frag_col<NT, C, 64>(ys, w * 16, jj, lane), y);
      const float* weight = (REV ? dec.entry : dec.leave) + jj * 32 + grp * 8;
#pragma unroll
      for (int s = 0; s < 8; ++s) y[s] *= weight[s];
      const Frag<NW> fy = split<NW>(y);
#pragma unroll
      for (int kt = 0; kt < KT; ++kt) S[kt] = mma(fy, frag_col<NT, C, KP>(xs, kt * 16, jj, lane), S[kt]);
    }
    __syncthreads();
  }

  if (p.seg_end && seg + 1 < a.nseg) {
    float* to = p.seg_end + (eh * a.nseg + seg + 1) * state;
#pragma unroll
    for (int kt = 0; kt < KT; ++kt) *reinterpret_cast<f32x4*>(to + (int64_t)(kt * 16 + col) * p.VP + vc) = S[kt];
    if (tid == 0 && vs == 0) p.seg_decay[eh * a.nseg + seg + 1] = decay;
  }
  if (p.end && seg == a.nseg - 1) {
#pragma unroll
    for (int kt = 0; kt < KT; ++kt) {
      const int k = kt * 16 + col;
#pragma unroll
      for (int r = 0; r < 4; ++r)
        if (k < a.K && vc + r < a.V) p.end[(eh * a.K + k) * a.V + vc + r] = S[kt][r];
    }
  }
}

// Turns the segments' own contributions into the values entering them, in place:
// slot 0 gets the row's entering value, slot s + 1 becomes decay * slot s + slot s + 1.
struct CombineArgs {
  float* seg;          // [E, H, nseg, KP, VP]
  const float* decay;  // [E, H, nseg]
  const float* given;  // [E, H, K, V] or NULL
  const uint8_t* done; // with closed: rows whose last step ends an episode take nothing from given
  int64_t d_se, d_st;
  int64_t H, T, nseg, KP, VP, K, V;
  int closed;
};

static __global__ void __launch_bounds__(256) combine_kernel(const CombineArgs p) {
  const int64_t state = p.KP * p.VP;
  const int64_t per = (state + 255) / 256;
  const int64_t eh = blockIdx.x / per;
  const int64_t i = (blockIdx.x % per) * 256 + threadIdx.x;
  if (i >= state) return;
  const int64_t k = i / p.VP, v = i % p.VP, e = eh / p.H;
  float x = 0.0f;
  if (p.given && k < p.K && v < p.V &&
      !(p.closed && p.T > 0 && p.done && p.done[e * p.d_se + (p.T - 1) * p.d_st] != 0))
    x = p.given[(eh * p.K + k) * p.V + v];
  float* s = p.seg + eh * p.nseg * state + i;
  s[0] = x;
  for (int64_t n = 1; n < p.nseg; ++n) {
    x = p.decay[eh * p.nseg + n] * x + s[n * state];
    s[n * state] = x;
  }
}

}  // namespace la
}  // namespace rlscan

#endif
