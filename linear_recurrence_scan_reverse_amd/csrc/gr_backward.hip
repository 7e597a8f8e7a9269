// Gradients of the gated recurrence (rlscan_gated_recurrence_backward).
//
// With g_t the gradient of h_t and e_t = a_t g_t what step t passes to the one before it,
//   g_t  = do_t + e_{t+1},
//   dx   = sigmoid(i) m g,   di = u m g (1 - sigmoid(i)),
//   dlog_a = g (a h_{t-1} - u a^2 / m),   dr = -rate sigmoid(r) (1 - sigmoid(r)) dlog_a,
//   drate = -sum sigmoid(r) dlog_a,
// and dlog_a = e = 0 at a step that starts anew.  e runs backward like h runs forward, in
// pairs of A and y.  The states h_{t-1} are computed again from the marks that the forward
// call left every kMark steps.
//
// Bound by memory like the forward pass: four values read and three written a step.  A wave holds the 16
// steps behind a mark.  What the decays are made of is read a round ahead, the rest (x, the input gate,
// the mark) in the round that uses it, behind the barrier: all of it ahead would leave one wave to a SIMD.
// Measured: 64 x 333 x 768 float32 92 us (5.0 TB/s), 8 x 4096 x 2048 bfloat16 217 (4.3).
#include "rlscan_gr.hpp"
#include "rlscan_sums.hpp"

namespace rlscan {
namespace gr {

// What the decays of a chunk are made of; the rest is asked for when these are at hand, and used
// behind the barrier.
template <class F, int S>
struct Chunk {
  typename F::E g[S], dg[S];
  uint8_t flag;
};
template <class F, int S>
struct Rest {
  typename F::E x[S], ig[S];
  float mark;
};

// sigmoid(r) and a - 1 of every step, the sum of y (logarithms of the decays) and what leaves
// the chunk to the steps before it for an entering e of 0.
template <int S>
struct Decays {
  float sr[S], em1[S];
  float L, out;
};

// CARE: some steps start anew (cut) or lie past the end (not live).
template <class F, int S, bool CARE>
__device__ __forceinline__ void decays(Decays<S>& c, const Chunk<F, S>& in, float rate2, uint32_t cut, uint32_t live) {
  c.L = c.out = 0.0f;
#pragma unroll
  for (int k = S - 1; k >= 0; --k) {
    const float dg = F::get(CARE ? apart(in.dg[k]) : in.dg[k]);
    float g = F::get(CARE ? apart(in.g[k]) : in.g[k]);
    float sr = sigmoid(dg), y = rate2 * sr, em1 = decay_less_1(y);
    if (CARE) {
      sr = keep(sr, spread(live & ~cut, k));  // the gate of a step that starts anew is not looked at: it may be NaN
      em1 = keep(pick(spread(cut, k), -1.0f, em1), spread(live, k));
      y = keep(y, spread(live, k));
      g = keep(g, spread(live, k));
    }
    c.sr[k] = sr;
    c.em1[k] = em1;
    c.L += y;
    c.out = decayed(em1, c.out + g);
    if (CARE) c.out = keep(c.out, ~spread(cut, k));
  }
}

// What a block's waves read and write: 64 channels of a row.
template <class F, int S, bool NEAR>
struct Tensors {
  Stream<F, S, NEAR> g, dg, x, ig, dx, dig, ddg;
  // bytes from a step to the next
  int64_t g_st, dg_st, x_st, ig_st, dx_st, dig_st, ddg_st;
  const uint8_t* done;
  int64_t done_step, mark_step;
  const float* marks;
  int lane;
  uint32_t at;  // byte of the lane's column

  __device__ __forceinline__ Tensors(const Args& p, int64_t e, int64_t d0, int lane_, uint32_t col)
      : g(p.dout, e, d0), dg(p.dg, e, d0), x(p.x, e, d0), ig(p.ig, e, d0), dx(p.dx, e, d0), dig(p.dig, e, d0),
        ddg(p.ddg, e, d0), done(p.done ? p.done + e * p.d_se : nullptr), done_step(p.d_st), mark_step(p.D),
        marks(p.marks + e * ((p.T + kMark - 1) / kMark) * p.D + d0 + col), lane(lane_),
        at(col * (uint32_t)sizeof(typename F::E)) {
    constexpr int64_t es = sizeof(typename F::E);
    g_st = p.dout.st * es;
    dg_st = p.dg.st * es;
    dx_st = p.dx.st * es;
    x_st = p.x.st * es;
    ig_st = p.ig.st * es;
    dig_st = p.dig.st * es;
    ddg_st = p.ddg.st * es;
  }
  __device__ __forceinline__ void load(Chunk<F, S>& c, int t, int end) const {
    dg.load(c.dg, t, end, Steps<S, NEAR>(dg_st, t, end), at);
    g.load(c.g, t, end, Steps<S, NEAR>(g_st, t, end), at);
    c.flag = load_flag<S>(done, done_step, t, end, lane);
  }
  __device__ __forceinline__ void load(Rest<F, S>& c, int t, int end) const {
    c.mark = marks[(t < end ? t : end - 1) / kMark * mark_step];
    ig.load(c.ig, t, end, Steps<S, NEAR>(ig_st, t, end), at);
    x.load(c.x, t, end, Steps<S, NEAR>(x_st, t, end), at);
  }
};

// The gradients of a chunk, from the e that enters it, to memory; returns the e that leaves it.
template <class F, int S, bool NEAR, bool CARE>
__device__ __forceinline__ float gradients(const Decays<S>& c, const Chunk<F, S>& in, const Rest<F, S>& rest, float e,
                                           float rate, float& d_rate, const Tensors<F, S, NEAR>& to, int t,
                                           uint32_t out_at, uint32_t cut, uint32_t live) {
  float before[S], u[S], si[S];
  float h = rest.mark;
#pragma unroll
  for (int k = 0; k < S; ++k) {
    si[k] = sigmoid(F::get(CARE ? apart(rest.ig[k]) : rest.ig[k]));
    u[k] = si[k] * F::get(CARE ? apart(rest.x[k]) : rest.x[k]);
    if (CARE) h = keep(h, ~spread(cut, k));
    before[k] = h;
    h = decayed(c.em1[k], h) + __builtin_amdgcn_sqrtf(one_less_square(c.em1[k])) * u[k];
  }
#pragma unroll
  for (int k = S - 1; k >= 0; --k) {
    float g = F::get(CARE ? apart(in.g[k]) : in.g[k]);
    if (CARE) g = keep(g, spread(live, k));
    g += e;
    const float m2 = one_less_square(c.em1[k]);
    const float over_m = m2 >= 1.1754944e-38f ? __builtin_amdgcn_rsqf(m2) : 0.0f;  // a held state has no part in u
    const float du = m2 * over_m * g, ud = u[k] * du;
    e = decayed(c.em1[k], g);
    if (CARE) e = keep(e, ~spread(cut, k));
    // a g (h - u a / m): the gradient of log a
    const float a = 1.0f + c.em1[k];
    float part = c.sr[k] * (e * (before[k] - u[k] * over_m * a));
    if (CARE) part = keep(part, spread(live & ~cut, k));
    d_rate -= part;
    if (!CARE || (live >> k) & 1) {
      to.dx.store(F::put(si[k] * du), t, k, to.dx_st, out_at);
      to.dig.store(F::put(ud - ud * si[k]), t, k, to.dig_st, out_at);
      to.ddg.store(F::put((rate * c.sr[k] - rate) * part), t, k, to.ddg_st, out_at);
    }
  }
  return e;
}

// The pair of each segment but the first: a wave takes a share of it, chunk after chunk, from the end.
template <class F, int S, int W, bool NEAR>
__global__ void __launch_bounds__(64 * W) fold_back_kernel(const Args p, uint32_t tiles) {
  __shared__ float s_a[W][64], s_y[W][64];
  const int lane = threadIdx.x & 63;
  const int w = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const uint32_t tile = blockIdx.x % tiles, es = blockIdx.x / tiles, nseg = (uint32_t)p.nseg;
  const int64_t seg = es % (nseg - 1) + 1, e = es / (nseg - 1), d0 = tile * 64;
  const bool column = d0 + lane < p.D;
  const uint32_t col = column ? lane : (uint32_t)(p.D - 1 - d0);  // loads stay inside the row
  const float rate2 = kLog2E * p.rate[d0 + col];
  const Tensors<F, S, NEAR> in(p, e, d0, lane, col);
  const int share = (int)p.seg_steps / W, begin = (int)seg * (int)p.seg_steps + w * share;
  const int end = (int)p.T < begin + share ? (int)p.T : begin + share;  // the last segment may be short
  float total = 0.0f, y = 0.0f;
  bool dropped = false;
  auto fold = [&](const Chunk<F, S>& c, uint32_t live) __attribute__((always_inline)) {
    const uint32_t cut = flag_word(c.flag, 1, 0);  // never the row's first step
    Decays<S> k;
    if (cut == 0 && live == (1u << S) - 1) decays<F, S, false>(k, c, rate2, 0, 0);
    else decays<F, S, true>(k, c, rate2, cut, live);
    total += k.L;
    dropped |= cut != 0;
    y = enter(cut ? kDropped : exp2_fast(-k.L), k.out, y);
  };
  if (begin < end) {
    Chunk<F, S> one, two;
    int t = begin + (end - begin - 1) / S * S;
    in.load(one, t, end);
    for (;;) {
      in.load(two, t > begin ? t - S : begin, end);
      fold(one, live_word<S>(t, end));
      if (t == begin) break;
      t -= S;
      in.load(one, t > begin ? t - S : begin, end);
      fold(two, (1u << S) - 1);
      if (t == begin) break;
      t -= S;
    }
  }
  s_a[w][lane] = dropped ? kDropped : exp2_fast(-total);
  s_y[w][lane] = y;
  __syncthreads();
  if (w == 0 && column) {
    float A = 1.0f, out = 0.0f;
    for (int v = W - 1; v >= 0; --v) {
      out = enter(s_a[v][lane], s_y[v][lane], out);
      A = A < 0.0f || s_a[v][lane] < 0.0f ? kDropped : A * s_a[v][lane];
    }
    const int64_t at = (e * p.nseg + seg) * p.D + d0 + lane;
    p.seg_a[at] = A;
    p.seg_y[at] = out;
  }
}

// One block: 64 channels of the rows e, e + groups, ... (or of one segment of them), W waves of
// S steps each at a time, from the end, the next ones' loads in flight meanwhile.
template <class F, int S, int W, bool NEAR>
__global__ void __launch_bounds__(64 * W) backward_kernel(const Args p, uint32_t tiles) {
  static_assert(S == kMark, "a chunk begins at a marked state");
  __shared__ Exchange<W> s;
  const int lane = threadIdx.x & 63;
  const int w = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const uint32_t tile = blockIdx.x % tiles, es = blockIdx.x / tiles, nseg = (uint32_t)p.nseg;
  const int64_t seg = es % nseg, group = es / nseg, d0 = tile * 64;
  const bool column = d0 + lane < p.D;
  const uint32_t col = column ? lane : (uint32_t)(p.D - 1 - d0);  // loads stay inside the row
  const float rate = p.rate[d0 + col], rate2 = kLog2E * rate;
  const int begin = (int)seg * (int)p.seg_steps;
  const int end = (int)(p.T < begin + p.seg_steps ? p.T : begin + p.seg_steps);
  constexpr int kStep = W * S;
  const int ahead = w * S;
  float d_rate = 0.0f;
  int buf = 0;
  for (int64_t e = group; e < p.E; e += p.groups) {
    const Tensors<F, S, NEAR> in(p, e, d0, lane, col);
    const uint32_t out_at = column ? in.at : kNoColumn;
    const uint32_t first = first_flag(p, e);
    float carry = 0.0f;  // e entering the W chunks at hand from the steps behind them
    if (p.d_final && !(in.done && p.T > 0 && in.done[(p.T - 1) * p.d_st] != 0)) carry = p.d_final[e * p.D + d0 + col];
    for (int64_t v = p.nseg - 1; v > seg; --v) {
      const int64_t at = (e * p.nseg + v) * p.D + d0 + col;
      carry = enter(p.seg_a[at], p.seg_y[at], carry);
    }
    if (W > 1) {
      meet();  // the row before has been read
      s.carry[buf][lane] = carry;  // the same from every wave
    }
    auto take = [&](const Chunk<F, S>& c, const Rest<F, S>& rest, int t) __attribute__((always_inline)) {
      const uint32_t cut = flag_word(c.flag, t, first), live = live_word<S>(t, end);
      const bool care = cut != 0 || live != (1u << S) - 1;
      Decays<S> k;
      if (!care) decays<F, S, false>(k, c, rate2, 0, 0);
      else decays<F, S, true>(k, c, rate2, cut, live);
      float g = carry;  // e entering this wave's chunk
      if constexpr (W > 1) {
        s.put(buf, w, lane, exp2_fast(-k.L), k.out, cut);
        meet();
        g = s.template entering<-1>(buf, w, lane);
      }
      if (!care) g = gradients<F, S, NEAR, false>(k, c, rest, g, rate, d_rate, in, t, out_at, 0, 0);
      else g = gradients<F, S, NEAR, true>(k, c, rest, g, rate, d_rate, in, t, out_at, cut, live);
      carry = g;
      if constexpr (W > 1) {  // what leaves the first wave enters the chunks before
        buf ^= 1;
        if (w == 0) s.carry[buf][lane] = g;
      }
    };
    if (begin < end) {
      Chunk<F, S> one, two;
      Rest<F, S> rest;
      int t = begin + (end - begin - 1) / kStep * kStep;
      in.load(one, t + ahead, end);
      for (;;) {
        in.load(rest, t + ahead, end);
        in.load(two, (t > begin ? t - kStep : begin) + ahead, end);
        take(one, rest, t + ahead);
        if (t == begin) break;
        t -= kStep;
        in.load(rest, t + ahead, end);
        in.load(one, (t > begin ? t - kStep : begin) + ahead, end);
        take(two, rest, t + ahead);
        if (t == begin) break;
        t -= kStep;
      }
    }
    if (w == 0 && column && seg == 0 && p.d_init) p.d_init[e * p.D + d0 + lane] = carry;
  }
  if constexpr (W > 1) {
    __syncthreads();
    s.a[0][w][lane] = d_rate;
    __syncthreads();
    d_rate = 0.0f;
    for (int v = 0; v < W; ++v) d_rate += s.a[0][v][lane];
  }
  if (w == 0 && column) (p.rate_part ? p.rate_part : p.d_rate)[(group * p.nseg + seg) * p.D + d0 + lane] = d_rate;
}

template <class F, int S, int W, bool NEAR>
static hipError_t backward_waves(const Args& a, hipStream_t st) {
  const int64_t tiles = (a.D + 63) / 64;
  hipError_t e = hipSuccess;
  if (a.nseg > 1) {
    fold_back_kernel<F, S, W, NEAR><<<dim3((unsigned)(a.E * (a.nseg - 1) * tiles)), 64 * W, 0, st>>>(a, (uint32_t)tiles);
    e = hipGetLastError();
    if (e != hipSuccess) return e;
  }
  backward_kernel<F, S, W, NEAR><<<dim3((unsigned)(a.groups * a.nseg * tiles)), 64 * W, 0, st>>>(a, (uint32_t)tiles);
  e = hipGetLastError();
  if (e != hipSuccess || !a.rate_part) return e;
  return sums::launch_columns(a.rate_part, a.groups * a.nseg, a.d_rate, a.D, nullptr, 0, st);
}

template <class F>
static hipError_t backward_fmt(const Args& a, const Plan& p, hipStream_t st) {
  constexpr int64_t es = sizeof(typename F::E);
  const View* const v[] = {&a.dout, &a.x, &a.ig, &a.dg, &a.dx, &a.dig, &a.ddg};
  if (!all_near(v, 7, es)) return backward_waves<F, kMark, 1, false>(a, st);  // as the forward pass
  switch (p.waves) {
    case 1: return backward_waves<F, kMark, 1, true>(a, st);
    case 4: return backward_waves<F, kMark, 4, true>(a, st);
    default: return backward_waves<F, kMark, kBackWaves, true>(a, st);
  }
}

hipError_t launch_backward(rlscan_format f, const Args& a, const Plan& p, hipStream_t st) {
  switch (f) {
    case RLSCAN_FORMAT_BF16: return backward_fmt<LBf16>(a, p, st);
    case RLSCAN_FORMAT_F16: return backward_fmt<LF16>(a, p, st);
    default: return backward_fmt<LF32>(a, p, st);
  }
}

}  // namespace gr
}  // namespace rlscan
