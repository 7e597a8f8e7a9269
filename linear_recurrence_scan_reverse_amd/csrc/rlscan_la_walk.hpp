// rlscan_la_walk.hpp -- joining the segments of long rows of linear attention.
//
// Where the heads do not fill the card, rows are cut into segments that run side
// by side.  walk_kernel first carries a state that starts from zero over each segment:
// forward, S = across S + sum_j leave_j k_j v_j^T; backward in time the gradient of the
// state, which is the same recurrence reversed, dS = across dS + sum_i entry_i q_i do_i^T.
// combine_kernel turns these into the states that enter the segments.
#ifndef RLSCAN_LA_WALK_HPP
#define RLSCAN_LA_WALK_HPP

#include "rlscan_la.hpp"

namespace rlscan {
namespace la {

// A block: head eh = e*H + h, 64 columns of V, one segment but the last (in walking
// order).  Wave w holds the 16 columns w*16 ... of the slice for all KP rows: accumulator
// tile kt, lane l holds S[kt*16 + l%16][w*16 + (l/16)*4 + r].  What segment s adds goes
// to slot s + 1 of seg_state [E, H, nseg, KP, VP], its decay to seg_decay [E, H, nseg].
// CARE as in rlscan_la_attend.hpp: without, it returns false before the segment's values if
// they are not finite.
template <class F, int KP, int C>
struct WalkLds {
  MixTile<F::NT, C, KP> xs;
  MixTile<F::NT, C, 64> ys;
  Decay<C> dec;
  Odd<C, KP, 64, kThreads> odd;
};

struct WalkArgs {
  Args a;
  int64_t VP;
  float *seg_state, *seg_decay;
};

template <class F, int KP, int C, bool REV, bool VEC, bool CARE>
__device__ __forceinline__ bool walk_as(WalkLds<F, KP, C>& lds, const WalkArgs& p, int64_t block) {
  constexpr int NT = F::NT, NW = F::NW, KT = KP / 16;
  const Args& a = p.a;
  const int64_t VP = p.VP;
  auto& xs = lds.xs;
  auto& ys = lds.ys;
  auto& dec = lds.dec;
  auto& odd = lds.odd;
  const int tid = threadIdx.x, lane = tid & 63, w = tid >> 6, col = lane & 15, grp = lane >> 4;
  const int64_t EH = a.E * a.H, nvs = VP / 64;
  const int64_t eh = block % EH, rest = block / EH;
  const int64_t vs = rest % nvs, seg = rest / nvs;
  const int64_t e = eh / a.H, h = eh % a.H;
  const View& X = REV ? a.q : a.k;
  const View& Y = REV ? a.dout : a.v;
  const int64_t hx = REV ? h : h / a.G, hy = hx;
  const int v0 = (int)vs * 64;

  f32x4 S[KT];
#pragma unroll
  for (int kt = 0; kt < KT; ++kt) S[kt] = f32x4{0, 0, 0, 0};

  const int64_t p0 = seg * a.seg_chunks, p1 = p0 + a.seg_chunks;  // not the last segment: all its chunks exist
  auto chunk_t0 = [&](int64_t n) { return (REV ? a.chunks - 1 - n : n) * (int64_t)C; };
  // two chunks ahead: a chunk's work is shorter than a request's way to memory
  Piece<F> rx[2][Share<C, KP>::n], ry[2][Share<C, 64>::n];
  StepDecay sd[2] = {{0.0f, 0}, {0.0f, 0}};
  float decay = 1.0f;
  auto request = [&](int64_t n, int b) __attribute__((always_inline)) {
    fetch<F, C, KP, kThreads, REV, VEC>(TileRows<F>(X, e, hx, chunk_t0(n), a.T, C), 0, a.K, tid, rx[b]);
    fetch<F, C, 64, kThreads, REV, VEC>(TileRows<F>(Y, e, hy, chunk_t0(n), a.T, C), v0, a.V, tid, ry[b]);
    if (w == 0) sd[b] = load_decay<C>(a, e, h, chunk_t0(n), lane);
  };
  request(p0, 0);
  if (p0 + 1 < p1) request(p0 + 1, 1);
  auto chunk = [&](int64_t n, int b) __attribute__((always_inline)) {
    stage<F, kThreads>(xs, rx[b], tid);
    stage<F, kThreads>(ys, ry[b], tid);
    if (w == 0) put_decay<C, REV>(dec, scan_decay<C, REV>(sd[b], a.scale, lane), lane);
    __syncthreads();
    uint32_t bits = 0;
    if constexpr (CARE) {
      sweep_odd(odd, xs, ys, dec, tid);
      bits = take_odd(S);
      __syncthreads();
    }
    if (n + 2 < p1) request(n + 2, b);
    const float across = dec.across;
    decay *= across;
#pragma unroll
    for (int kt = 0; kt < KT; ++kt) S[kt] *= across;
#pragma unroll
    for (int jj = 0; jj < C / 32; ++jj) {
      float y[8];
      join<NT>(frag_col(ys, w, jj, lane), y);
      const float* weight = dec.out + jj * 32 + grp * 8;
#pragma unroll
      for (int s = 0; s < 8; ++s) y[s] *= weight[s];
      const Frag<NW> fy = split<NW>(y);
#pragma unroll
      for (int kt = 0; kt < KT; ++kt) S[kt] = mma(fy, frag_col(xs, kt, jj, lane), S[kt]);
    }
    if constexpr (CARE) {  // what was taken out
      if (across == 0.0f) bits = 0;
#pragma unroll
      for (int kt = 0; kt < KT; ++kt)
#pragma unroll
        for (int r = 0; r < 4; ++r)
          if (((odd.b[kt * 16 + col] | odd.c[w * 16 + grp * 4 + r]) & odd.leaving) != 0 ||
              (bits >> (kt * 4 + r) & 1) != 0)
            S[kt][r] = __builtin_nanf("");
    }
    __syncthreads();
  };
  for (int64_t n = p0; n < p1; n += 2) {
    chunk(n, 0);
    if (n + 1 < p1) chunk(n + 1, 1);
  }
  if (!CARE && any_of_block<kThreads>(odd.wave, any_odd(S), tid)) return false;

  float* to = p.seg_state + (eh * a.nseg + seg + 1) * KP * VP;
#pragma unroll
  for (int kt = 0; kt < KT; ++kt)
    *reinterpret_cast<f32x4*>(to + (kt * 16 + col) * VP + v0 + w * 16 + grp * 4) = S[kt];
  if (tid == 0 && vs == 0) p.seg_decay[eh * a.nseg + seg + 1] = decay;
  return true;
}

// At least as many waves as the walk without care leaves room for.
template <class F, int KP, int C, bool REV, bool VEC>
__global__ void __launch_bounds__(kThreads, KP == 128 ? 2 : F::NT < 3 && VEC ? 4 : 3) walk_kernel(const WalkArgs p) {
  __shared__ WalkLds<F, KP, C> lds;
  int block = (int)blockIdx.x;
  if (walk_as<F, KP, C, REV, VEC, false>(lds, p, block)) return;
  const WalkArgs again = argument_again<WalkArgs>();
  asm volatile("" : "+s"(block));
  walk_as<F, KP, C, REV, VEC, true>(lds, again, block);
}

// In place: slot 0 gets the row's entering value, slot s + 1 becomes decay * slot s + slot s + 1.
struct CombineArgs {
  float* seg;          // [E, H, nseg, KP, VP]
  const float* decay;  // [E, H, nseg]
  const float* given;  // [E, H, K, V] or NULL
  int64_t nseg, KP, VP;
  int closed;          // rows whose last step ends an episode take nothing from given
};

static __global__ void __launch_bounds__(256) combine_kernel(const Args a, const CombineArgs p) {
  const int64_t state = p.KP * p.VP, per = state / 256;
  const int64_t eh = blockIdx.x / per;
  const int64_t i = blockIdx.x % per * 256 + threadIdx.x;
  const int64_t k = i / p.VP, v = i % p.VP;
  float x = 0.0f;
  if (p.given && k < a.K && v < a.V && !(p.closed && row_closed(a, eh / a.H))) x = p.given[(eh * a.K + k) * a.V + v];
  float* s = p.seg + eh * p.nseg * state + i;
  const float* decay = p.decay + eh * p.nseg;
  s[0] = x;
  for (int64_t n0 = 1; n0 < p.nseg; n0 += 8) {  // eight requests at a time
    float add[8];
#pragma unroll
    for (int k = 0; k < 8; ++k) add[k] = n0 + k < p.nseg ? s[(n0 + k) * state] : 0.0f;
#pragma unroll
    for (int k = 0; k < 8; ++k)
      if (n0 + k < p.nseg) {
        x = gated(decay[n0 + k], x) + add[k];
        s[(n0 + k) * state] = x;
      }
  }
}

// The states entering every segment, in walking order (given: the row's own).
template <class F, int KP, int C, bool REV, bool VEC>
void enter_segments(const Args& a, int64_t VP, const float* given, float* seg_state, float* seg_decay, hipStream_t st) {
  if (a.nseg < 2) return;
  const int64_t heads = a.E * a.H;
  walk_kernel<F, KP, C, REV, VEC>
      <<<dim3((unsigned)(heads * (VP / 64) * (a.nseg - 1))), kThreads, 0, st>>>(WalkArgs{a, VP, seg_state, seg_decay});
  CombineArgs c{seg_state, seg_decay, given, a.nseg, KP, VP, REV};
  combine_kernel<<<dim3((unsigned)(heads * (KP * VP / 256))), 256, 0, st>>>(a, c);
}

}  // namespace la
}  // namespace rlscan

#endif
