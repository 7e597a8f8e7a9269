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
// Measured: 64 x 333 x 768 float32 93 us (4.9 TB/s), 8 x 4096 x 2048 bfloat16 214 (4.4).
#include "rlscan_gr.hpp"
#include "rlscan_sums.hpp"

namespace rlscan {
namespace gr {

// What the decays of a chunk are made of; the rest is asked for when these are at hand, and used
// behind the barrier.
template <class F, int S>
struct Ahead {
  typename F::E g[S], dg[S];
  uint8_t flag;
};
template <class F, int S>
struct Rest {
  typename F::E x[S], ig[S];
  float mark;
};

// sigmoid(r) and the decay (decay_of) of every step, the sum of y (logarithms of the decays) and what leaves
// the chunk to the steps before it for an entering e of 0.
template <int S>
struct Decays {
  float sr[S], a[S];
  float L, out;
};

// less: see decay_of, for kEvery.
template <class F, int S, Form FORM>
__device__ __forceinline__ void decays(Decays<S>& c, const Ahead<F, S>& in, float rate2, float less, uint32_t cut,
                                       uint32_t live) {
#pragma clang fp contract(off)
  c.L = c.out = 0.0f;
#pragma unroll
  for (int k = S - 1; k >= 0; --k) {
    const float dg = F::get(FORM != kPlain ? apart(in.dg[k]) : in.dg[k]);
    float g = F::get(FORM != kPlain ? apart(in.g[k]) : in.g[k]);
    float sr = sigmoid(dg), a = decay_of<FORM>(rate2 * sr, FORM == kEvery ? less : 1.0f);
    if (FORM != kPlain) {
      sr = keep(sr, spread(live & ~cut, k));  // the gate of a step that starts anew is not looked at: it may be NaN
      a = decay_before<FORM>(decay_behind<FORM>(a, spread(cut, k)), spread(live, k));
      g = keep(g, spread(live, k));
    }
    c.sr[k] = sr;
    c.a[k] = a;
    c.L = __builtin_fmaf(rate2, sr, c.L);
    c.out = decayed<FORM>(a, c.out + g);
    if (FORM != kPlain) c.out = keep(c.out, ~spread(cut, k));
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
  __device__ __forceinline__ void load(Ahead<F, S>& c, int t, int end) const {
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
template <class F, int S, bool NEAR, Form FORM>
__device__ __forceinline__ float gradients(Decays<S>& c, const Ahead<F, S>& in, const Rest<F, S>& rest, float e,
                                           float& odd, float rate, float& d_rate, const Tensors<F, S, NEAR>& to, int t,
                                           uint32_t out_at, uint32_t cut, uint32_t live) {
#pragma clang fp contract(off)
  float before[S], u[S], si[S];
  float h = rest.mark;
#pragma unroll
  for (int k = 0; k < S; ++k) {
    si[k] = sigmoid(F::get(FORM != kPlain ? apart(rest.ig[k]) : rest.ig[k]));
    u[k] = si[k] * F::get(FORM != kPlain ? apart(rest.x[k]) : rest.x[k]);
    if (FORM != kPlain) h = keep(h, ~spread(cut, k));
    before[k] = h;
    if (FORM == kCut && k % 2 == 1) odd = seen(odd, before[k - 1], h);  // what each step takes: the next cut may hide it
    if (FORM == kEvery) c.a[k] = apart(c.a[k]);  // 16 masks of which is held as a - 1 would lie in scalars for long
    h = __builtin_fmaf(__builtin_amdgcn_sqrtf(one_less_square<FORM>(c.a[k])), u[k], decayed<FORM>(c.a[k], h));
  }
  if (FORM != kEvery) odd = seen(odd, h);
  float after = 0.0f;
#pragma unroll
  for (int k = S - 1; k >= 0; --k) {
    float g = F::get(FORM != kPlain ? apart(in.g[k]) : in.g[k]);
    if (FORM != kPlain) g = keep(g, spread(live, k));
    g += e;
    if (FORM == kCut && k % 2 == 0) odd = seen(odd, after, g);
    after = g;
    if (FORM == kEvery) c.a[k] = apart(c.a[k]);
    const float m2 = one_less_square<FORM>(c.a[k]);
    const float over_m = m2 >= 1.1754944e-38f ? __builtin_amdgcn_rsqf(m2) : 0.0f;  // a held state has no part in u
    const float du = m2 * over_m * g, ud = u[k] * du;
    e = decayed<FORM>(c.a[k], g);
    if (FORM != kPlain) e = keep(e, ~spread(cut, k));
    // a g (h - u a / m): the gradient of log a
    const float a = decayed<FORM>(c.a[k], 1.0f);
    float part = c.sr[k] * (e * __builtin_fmaf(-(u[k] * over_m), a, before[k]));
    if (FORM != kPlain) part = keep(part, spread(live & ~cut, k));
    d_rate -= part;
    if (FORM == kPlain || (live >> k) & 1) {
      to.dx.store(F::put(si[k] * du), t, k, to.dx_st, out_at);
      to.dig.store(F::put(ud * (1.0f - si[k])), t, k, to.dig_st, out_at);
      to.ddg.store(F::put(__builtin_fmaf(rate, c.sr[k], -rate) * part), t, k, to.ddg_st, out_at);
    }
  }
  if (FORM != kEvery) odd = seen(odd, e);
  return e;
}

// The pair of each segment but the first: a wave takes a share of it, chunk after chunk, from the end.
// Returns whether the share is for the walk that looks at everything (EVERY).
template <class F, int S, int W, bool NEAR, bool EVERY>
__device__ __forceinline__ bool fold_back_walk(const Args& p, uint32_t tile, uint32_t es, int w, int lane, float& A,
                                               float& y) {
  const uint32_t nseg = (uint32_t)p.nseg;
  const int64_t seg = es % (nseg - 1) + 1, e = es / (nseg - 1), d0 = tile * 64;
  const uint32_t col = d0 + lane < p.D ? lane : (uint32_t)(p.D - 1 - d0);  // loads stay inside the row
  const float rate = rate_of(p.rate[d0 + col]), rate2 = kLog2E * rate;
  const Tensors<F, S, NEAR> in(p, e, d0, lane, col);
  const int share = (int)p.seg_steps / W, begin = (int)seg * (int)p.seg_steps + w * share;
  const int end = (int)p.T < begin + share ? (int)p.T : begin + share;  // the last segment may be short
  float total = 0.0f;
  bool dropped = false;
  A = 1.0f;
  y = 0.0f;
  if (begin >= end) return false;
  if (!EVERY && __builtin_expect(any_quick(rate), false)) return true;
  Ahead<F, S> one, two;
  int t = begin + (end - begin - 1) / S * S;
  in.load(one, t, end);
  const float less = EVERY ? less_of(rate) : 1.0f;
  auto fold = [&](const Ahead<F, S>& c, uint32_t live) __attribute__((always_inline)) {
    const uint32_t cut = flag_word(c.flag, 1, 0);  // never the row's first step
    Decays<S> k;
    by_form<EVERY>(cut == 0 && live == (1u << S) - 1, [&](auto form) __attribute__((always_inline)) {
      decays<F, S, form>(k, c, rate2, less, cut, live);
    });
    total += k.L;
    dropped |= cut != 0;
    y = enter<EVERY>(cut ? kDropped : exp2_fast(-k.L), k.out, y);
  };
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
  A = dropped ? kDropped : exp2_fast(-total);
  return any_odd(seen(0.0f, y));
}

template <class F, int S, int W, bool NEAR>
__global__ void __launch_bounds__(64 * W) fold_back_kernel(const Args p, uint32_t tiles) {
  __shared__ float s_a[W][64], s_y[W][64];
  const int lane = threadIdx.x & 63;
  const int w = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const uint32_t tile = blockIdx.x % tiles, es = blockIdx.x / tiles;
  float A, y;
  if (__builtin_expect(fold_back_walk<F, S, W, NEAR, false>(p, tile, es, w, lane, A, y), false))
    fold_back_walk<F, S, W, NEAR, true>(arguments_again(), again(tile), again(es), again(w), la::rarely(lane), A,
                                        y);
  s_a[w][lane] = A;
  s_y[w][lane] = y;
  __syncthreads();
  const int64_t column = (int64_t)tile * 64 + lane;
  if (w == 0 && column < p.D) {
    float A;
    const float out = joined_shares<W, -1>(s_a, s_y, lane, A);
    const uint32_t nseg = (uint32_t)p.nseg;
    const int64_t at = ((int64_t)(es / (nseg - 1)) * nseg + es % (nseg - 1) + 1) * p.D + column;
    p.seg_a[at] = A;
    p.seg_y[at] = out;
  }
}

// 64 channels of the rows group, group + groups, ... (or of one segment of them), W waves of S steps each at a
// time, from the end, the next ones' loads in flight meanwhile; d_rate: their share of the rates' gradient.
// Returns whether they are for the walk that looks at everything (EVERY).
template <class F, int S, int W, bool NEAR, bool EVERY>
__device__ __forceinline__ bool backward_walk(const Args& p, Exchange<W>& s, uint32_t tile, uint32_t es, int w, int lane,
                                              float& d_rate) {
  const uint32_t nseg = (uint32_t)p.nseg;
  const int64_t seg = es % nseg, group = es / nseg, d0 = tile * 64;
  const bool column = d0 + lane < p.D;
  const uint32_t col = column ? lane : (uint32_t)(p.D - 1 - d0);  // loads stay inside the row
  const float rate = rate_of(p.rate[d0 + col]), rate2 = kLog2E * rate;
  d_rate = 0.0f;
  if (!EVERY && __builtin_expect(any_quick(rate), false)) return true;
  const float less = EVERY ? less_of(rate) : 1.0f;
  const int begin = (int)seg * (int)p.seg_steps;
  const int end = (int)(p.T < begin + p.seg_steps ? p.T : begin + p.seg_steps);
  constexpr int kStep = W * S;
  const int ahead = w * S;
  float odd = 0.0f;
  int buf = 0;
  for (int64_t e = group; e < p.E; e += p.groups) {
    const Tensors<F, S, NEAR> in(p, e, d0, lane, col);
    const uint32_t out_at = column ? in.at : kNoColumn;
    const uint32_t first = first_flag(p, e);
    float start = 0.0f;
    if (p.d_final && !(in.done && p.T > 0 && in.done[(p.T - 1) * p.d_st] != 0)) start = p.d_final[e * p.D + d0 + col];
    float carry = start;  // e entering the W chunks at hand from the steps behind them
    if (seg < p.nseg - 1) {
      carry = joined([&](auto every) __attribute__((always_inline)) {
        float c = start;
        for (int64_t v = p.nseg - 1; v > seg; --v) {
          const int64_t at = (e * p.nseg + v) * p.D + d0 + col;
          c = enter<every>(p.seg_a[at], p.seg_y[at], c);
        }
        return c;
      });
    }
    if (W > 1) {
      meet();  // the row before has been read
      s.carry[buf][lane] = carry;  // the same from every wave
    }
    auto take = [&](const Ahead<F, S>& c, const Rest<F, S>& rest, int t) __attribute__((always_inline)) {
      const uint32_t cut = flag_word(c.flag, t, first), live = live_word<S>(t, end);
      const bool whole = cut == 0 && live == (1u << S) - 1;
      Decays<S> k;
      by_form<EVERY>(whole, [&](auto form) __attribute__((always_inline)) {
        decays<F, S, form>(k, c, rate2, less, cut, live);
      });
      float g = carry;  // e entering this wave's chunk
      if constexpr (W > 1) {
        s.put(buf, w, lane, exp2_fast(-k.L), k.out, cut);
        meet();
        g = s.template entering<-1, EVERY>(buf, w, lane);
      }
      by_form<EVERY>(whole, [&](auto form) __attribute__((always_inline)) {
        g = gradients<F, S, NEAR, form>(k, c, rest, g, odd, rate, d_rate, in, t, out_at, cut, live);
      });
      carry = g;
      if constexpr (W > 1) {  // what leaves the first wave enters the chunks before
        buf ^= 1;
        if (w == 0) s.carry[buf][lane] = g;
      }
    };
    if (begin < end) {
      Ahead<F, S> one, two;
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
  return any_odd(odd);
}

// One block for a tile of channels and a group of rows (or one segment of them).
template <class F, int S, int W, bool NEAR>
__global__ void __launch_bounds__(64 * W) backward_kernel(const Args p, uint32_t tiles) {
  static_assert(S == kMark, "a chunk begins at a marked state");
  __shared__ Exchange<W> s;
  const int lane = threadIdx.x & 63;
  const int w = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const uint32_t tile = blockIdx.x % tiles, es = blockIdx.x / tiles;
  float d_rate;
  if (__builtin_expect(s.any(w, lane, backward_walk<F, S, W, NEAR, false>(p, s, tile, es, w, lane, d_rate)), false))
    backward_walk<F, S, W, NEAR, true>(arguments_again(), s, again(tile), again(es), again(w), la::rarely(lane), d_rate);
  if constexpr (W > 1) {
    __syncthreads();
    s.a[0][w][lane] = d_rate;
    __syncthreads();
    d_rate = 0.0f;
    for (int v = 0; v < W; ++v) d_rate += s.a[0][v][lane];
  }
  const int64_t column = (int64_t)tile * 64 + lane;
  if (w == 0 && column < p.D) (p.rate_part ? p.rate_part : p.d_rate)[(int64_t)es * p.D + column] = d_rate;
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
