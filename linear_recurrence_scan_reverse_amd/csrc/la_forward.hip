// Linear attention over whole rows (rlscan_linear_attention).
//
// A block walks one head's chunks of 64 steps for a slice of V with the state in
// registers, so q, k, v are read and the output is written once per slice (slices
// of a head share q and k through the L2 of one XCD).  Rows whose heads do not
// fill the card are cut into segments: walk_kernel leaves each segment's own
// contribution to the state, combine_kernel joins them, and the segments then run
// side by side.
#include "rlscan_la_walk.hpp"
#include "rlscan_la_launch.hpp"

namespace rlscan {
namespace la {

template <class F, int KP, int CT>
struct ForwardLds {
  Tile<F::NT, 64, KP> q, k;
  Tile<F::NT, 64, 64 * CT> v;
  Tile<F::NP, 64, 64> p;
  Decay<64> dec[2];
};

// Wave w owns 16*CT columns of V.  Its state tile kt holds
// S[kt*16 + (l/16)*4 + r][column l%16], which is the layout of an MFMA operand with
// the steps k in accumulator order (frag_row_acc), so S^T q needs no exchange.
template <class F, int KP, int CT>
__global__ void __launch_bounds__(kThreads) forward_kernel(const Args a, int64_t nvs) {
  constexpr int NT = F::NT, NP = F::NP, NW = F::NW, C = 64, VB = 64 * CT, KT = KP / 16;
  __shared__ ForwardLds<F, KP, CT> s;
  const int tid = threadIdx.x, lane = tid & 63, w = tid >> 6, col = lane & 15, grp = lane >> 4;
  const int64_t EH = a.E * a.H;
  const int64_t eh = blockIdx.x % EH, rest = blockIdx.x / EH;
  const int64_t vs = rest % nvs, seg = rest / nvs;
  const int64_t e = eh / a.H, h = eh % a.H, hk = h / a.G;
  const int v0 = (int)vs * VB;
  const int64_t VP = nvs * VB;

  f32x4 S[CT][KT];
#pragma unroll
  for (int ct = 0; ct < CT; ++ct) {
    const int v = v0 + (w * CT + ct) * 16 + col;
#pragma unroll
    for (int kt = 0; kt < KT; ++kt)
#pragma unroll
      for (int r = 0; r < 4; ++r) {
        const int k = kt * 16 + grp * 4 + r;
        float x = 0.0f;
        if (a.nseg > 1) x = a.seg_state[((eh * a.nseg + seg) * KP + k) * VP + v];
        else if (a.init && k < a.K && v < a.V) x = a.init[(eh * a.K + k) * a.V + v];
        S[ct][kt][r] = x;
      }
  }

  const int64_t c0 = seg * a.seg_chunks;
  const int64_t c1 = c0 + a.seg_chunks < a.chunks ? c0 + a.seg_chunks : a.chunks;
  Piece<F> rq[Share<C, KP>::n], rk[Share<C, KP>::n], rv[Share<C, VB>::n];
  StepDecay sd{0.0f, false};
  auto request = [&](int64_t c) __attribute__((always_inline)) {
    fetch<F, C, KP>(a.q, e, h, c * C, a.T, 0, a.K, tid, rq);
    fetch<F, C, KP>(a.k, e, hk, c * C, a.T, 0, a.K, tid, rk);
    fetch<F, C, VB>(a.v, e, hk, c * C, a.T, v0, a.V, tid, rv);
  };
  if (c0 < c1) {
    request(c0);
    if (w == 0) {
      fill_decay<C>(s.dec[c0 & 1], load_decay<C>(a, e, h, c0 * C, lane), a.scale, lane);
      sd = load_decay<C>(a, e, h, (c0 + 1) * C, lane);
    }
  }
  for (int64_t c = c0; c < c1; ++c) {
    const Decay<C>& d = s.dec[c & 1];
    stage<F, C, KP>(s.q, rq, tid);
    stage<F, C, KP>(s.k, rk, tid);
    stage<F, C, VB>(s.v, rv, tid);
    __syncthreads();
    if (c + 1 < c1) request(c + 1);

    // P: wave w takes the 16 queries w*16 ... against the keys up to them.  The
    // products are formed transposed (rows j, columns i), which leaves four
    // consecutive j of one query in a lane.
    {
      const int i = w * 16 + col;
      const float hi_i = d.hi[i], lo_i = d.lo[i];
      const int seg_i = d.seg[i];
      Frag<NT> fq[KP / 32];
#pragma unroll
      for (int kk = 0; kk < KP / 32; ++kk) fq[kk] = frag_row<NT, C, KP>(s.q, w * 16, kk, lane);
#pragma unroll
      for (int jt = 0; jt < C / 16; ++jt) {
        if (jt > (w | 1)) continue;  // not read
        float x[4] = {0.0f, 0.0f, 0.0f, 0.0f};
        if (jt <= w) {
          f32x4 acc{0, 0, 0, 0};
#pragma unroll
          for (int kk = 0; kk < KP / 32; ++kk) acc = mma(frag_row<NT, C, KP>(s.k, jt * 16, kk, lane), fq[kk], acc);
#pragma unroll
          for (int r = 0; r < 4; ++r) {
            const int j = jt * 16 + grp * 4 + r;
            x[r] = acc[r] * (a.scale * between<C>(d, hi_i, lo_i, seg_i, i, j));
          }
        }
        put4<NP, C, C>(s.p, i, jt * 16 + grp * 4, x);
      }
    }
    if (w == 0 && c + 1 < c1) {  // the wave with the fewest keys prepares the next chunk's decays
      fill_decay<C>(s.dec[(c + 1) & 1], sd, a.scale, lane);
      sd = load_decay<C>(a, e, h, (c + 2) * C, lane);
    }
    __syncthreads();

#pragma unroll
    for (int ct = 0; ct < CT; ++ct) {
      const int vt = (w * CT + ct) * 16;  // column of the slice
      Frag<NT> fv[C / 32];
#pragma unroll
      for (int jj = 0; jj < C / 32; ++jj) fv[jj] = frag_col<NT, C, VB>(s.v, vt, jj, lane);
      // o^T: rows v, columns i
      f32x4 o[C / 16];
#pragma unroll
      for (int it = 0; it < C / 16; ++it) o[it] = f32x4{0, 0, 0, 0};
#pragma unroll
      for (int kk = 0; kk < KP / 32; ++kk) {
        float x[8];
#pragma unroll
        for (int r = 0; r < 4; ++r) {
          x[r] = S[ct][2 * kk][r];
          x[4 + r] = S[ct][2 * kk + 1][r];
        }
        const Frag<NP> fs = split<NP>(x);  // a copy, to the output's precision
#pragma unroll
        for (int it = 0; it < C / 16; ++it) o[it] = mma(fs, frag_row_acc<NT, C, KP>(s.q, it * 16, kk, lane), o[it]);
      }
#pragma unroll
      for (int it = 0; it < C / 16; ++it) {
        o[it] *= d.entry[it * 16 + col];
#pragma unroll
        for (int jj = 0; jj <= it / 2; ++jj) o[it] = mma(fv[jj], frag_row<NP, C, C>(s.p, it * 16, jj, lane), o[it]);
        const int64_t t = c * C + it * 16 + col;
        if (t < a.T) {
          const float x[4] = {o[it][0], o[it][1], o[it][2], o[it][3]};
          store4<F>(static_cast<typename F::E*>(const_cast<void*>(a.out.p)) + e * a.out.se + h * a.out.sh + t * a.out.st,
                    v0 + vt + grp * 4, a.V, a.out.vec, x);
        }
      }
      // S = across S + sum_j k_j (leave_j v_j)^T
      const float across = d.across;
#pragma unroll
      for (int kt = 0; kt < KT; ++kt) S[ct][kt] *= across;
#pragma unroll
      for (int jj = 0; jj < C / 32; ++jj) {
        float y[8];
        join<NT>(fv[jj], y);
#pragma unroll
        for (int x = 0; x < 8; ++x) y[x] *= d.leave[jj * 32 + grp * 8 + x];
        const Frag<NW> fy = split<NW>(y);
#pragma unroll
        for (int kt = 0; kt < KT; ++kt)
          S[ct][kt] = mma(frag_col<NT, C, KP>(s.k, kt * 16, jj, lane), fy, S[ct][kt]);
      }
    }
    __syncthreads();
  }

  if (a.final_state && seg == a.nseg - 1) {
    const bool closed = row_closed(a, e);
#pragma unroll
    for (int ct = 0; ct < CT; ++ct) {
      const int v = v0 + (w * CT + ct) * 16 + col;
#pragma unroll
      for (int kt = 0; kt < KT; ++kt)
#pragma unroll
        for (int r = 0; r < 4; ++r) {
          const int k = kt * 16 + grp * 4 + r;
          if (k < a.K && v < a.V) a.final_state[(eh * a.K + k) * a.V + v] = closed ? 0.0f : S[ct][kt][r];
        }
    }
  }
}

template <class F, int KP, int CT>
hipError_t launch_forward_as(const Args& a, const Plan& pl, hipStream_t st) {
  if (pl.nseg > 1) {
    WalkArgs w{};
    w.a = a;
    w.VP = pl.VP;
    w.seg_end = a.seg_state;
    w.seg_decay = a.seg_decay;
    walk_kernel<F, KP, 64, false><<<dim3((unsigned)(a.E * a.H * (pl.VP / 64) * pl.nseg)), kThreads, 0, st>>>(w);
    CombineArgs c{};
    c.seg = a.seg_state;
    c.decay = a.seg_decay;
    c.given = a.init;
    c.H = a.H;
    c.T = a.T;
    c.nseg = pl.nseg;
    c.KP = KP;
    c.VP = pl.VP;
    c.K = a.K;
    c.V = a.V;
    combine_kernel<<<dim3((unsigned)(a.E * a.H * ((KP * pl.VP + 255) / 256))), 256, 0, st>>>(c);
  }
  const int64_t nvs = pl.VP / (64 * CT);
  forward_kernel<F, KP, CT><<<dim3((unsigned)(a.E * a.H * nvs * pl.nseg)), kThreads, 0, st>>>(a, nvs);
  return hipGetLastError();
}

template <class F>
hipError_t launch_forward_fmt(const Args& a, const Plan& pl, hipStream_t st) {
  return pl.KP == 64 ? launch_forward_as<F, 64, 1>(a, pl, st) : launch_forward_as<F, 128, 1>(a, pl, st);
}

hipError_t launch_forward(rlscan_format f, const Args& a, const Plan& pl, hipStream_t st) {
  switch (f) {
    case RLSCAN_FORMAT_BF16: return launch_forward_fmt<TBf16>(a, pl, st);
    case RLSCAN_FORMAT_F16: return launch_forward_fmt<TF16>(a, pl, st);
    default: return launch_forward_fmt<TF32>(a, pl, st);
  }
}

}  // namespace la
}  // namespace rlscan
