// The gated recurrence over whole rows (rlscan_gated_recurrence).
//
// Bound by memory: three values read and one written a step, against about 30 vector instructions, seven of
// them transcendental.  A lane holds a channel, so that rows of 64 channels are read whole; a wave holds
// eight steps, whose coefficients stay in registers between the two uses of them: the pair that the block's
// other waves need, and the states once the one that enters is known.  One barrier for every W chunks, and the
// next ones' loads in flight across it.
//
// Measured (bytes read and written once): 64 x 333 x 768 float32 54 us (4.8 TB/s), 8 x 4096 x 2048 bfloat16 134
// (4.0), 1 x 32768 x 1280 bfloat16 in 12 segments 55 for their pairs and 84 for the states (2.4 in all).  Rows
// of 64 bfloat16 are 128 bytes, and loads and stores of that size alone, four streams, take 110 us of the 134.
#include "rlscan_gr.hpp"

namespace rlscan {
namespace gr {

template <class F, int S>
struct Chunk {
  typename F::E x[S], ig[S], dg[S];
  uint8_t flag;
};

// The decay (decay_of) and the term of every step, the sum of y (logarithms of the decays) and what leaves
// the chunk for a state of 0.
template <int S>
struct Coefficients {
  float a[S], b[S];
  float L, out;
};

// less: see decay_of, for kEvery.
template <class F, int S, Form FORM>
__device__ __forceinline__ void coefficients(Coefficients<S>& c, const Chunk<F, S>& in, float rate2, float less,
                                             uint32_t cut, uint32_t live) {
#pragma clang fp contract(off)
  c.L = c.out = 0.0f;
#pragma unroll
  for (int k = 0; k < S; ++k) {
    const float dg = F::get(FORM != kPlain ? apart(in.dg[k]) : in.dg[k]);
    const float ig = F::get(FORM != kPlain ? apart(in.ig[k]) : in.ig[k]);
    const float x = F::get(FORM != kPlain ? apart(in.x[k]) : in.x[k]);
    float sr = sigmoid(dg);
    float a = decay_of<FORM>(rate2 * sr, FORM == kEvery ? less : 1.0f);
    if (FORM != kPlain) a = decay_behind<FORM>(a, spread(cut, k));
    float m = __builtin_amdgcn_sqrtf(one_less_square<FORM>(a)), u = sigmoid(ig) * x;
    if (FORM != kPlain) {
      a = decay_before<FORM>(a, spread(live, k));
      m = keep(m, spread(live, k));
      u = keep(u, spread(live, k));
      sr = keep(sr, spread(live, k));
      c.out = keep(c.out, ~spread(cut, k));
    }
    c.a[k] = a;
    c.b[k] = m * u;
    c.L = __builtin_fmaf(rate2, sr, c.L);
    c.out = __builtin_fmaf(m, u, decayed<FORM>(a, c.out));
  }
}

// The states of a chunk, from the one that enters it, to memory.  Returns the last.
template <class F, int S, bool NEAR, Form FORM>
__device__ __forceinline__ float states(const Coefficients<S>& c, float h, float& odd, const Stream<F, S, NEAR>& out,
                                        int t, int64_t st, uint32_t lane, uint32_t cut, uint32_t live) {
#pragma clang fp contract(off)
  float before = 0.0f;
#pragma unroll
  for (int k = 0; k < S; ++k) {
    if (FORM != kPlain) h = keep(h, ~spread(cut, k));
    if (FORM == kCut && k % 2 == 1) odd = seen(odd, before, h);  // what each step takes: the next cut may hide it
    before = h;
    h = decayed<FORM>(c.a[k], h) + c.b[k];
    if (FORM == kPlain || (live >> k) & 1) out.store(F::put(h), t, k, st, lane);
  }
  if (FORM != kEvery) odd = seen(odd, h);
  return h;
}

// What a block's waves read: the three inputs of 64 channels of a row.  ALIKE: by one stride.
template <class F, int S, bool NEAR, bool ALIKE>
struct Inputs {
  Stream<F, S, NEAR> x, ig, dg;
  int64_t st[3];  // bytes from a step to the next
  const uint8_t* done;
  int64_t done_step;
  int lane;
  uint32_t at;  // byte of the lane's column

  __device__ __forceinline__ Inputs(const Args& p, int64_t e, int64_t d0, int lane_, uint32_t col)
      : x(p.x, e, d0), ig(p.ig, e, d0), dg(p.dg, e, d0), done(p.done ? p.done + e * p.d_se : nullptr),
        done_step(p.d_st), lane(lane_), at(col * (uint32_t)sizeof(typename F::E)) {
    st[0] = p.dg.st * (int64_t)sizeof(typename F::E);
    st[1] = p.ig.st * (int64_t)sizeof(typename F::E);
    st[2] = p.x.st * (int64_t)sizeof(typename F::E);
  }
  __device__ __forceinline__ void load(Chunk<F, S>& c, int t, int end) const {
    using At = Steps<S, NEAR>;
    dg.load(c.dg, t, end, At(st[0], t, end), at);
    ig.load(c.ig, t, end, At(st[ALIKE ? 0 : 1], t, end), at);
    x.load(c.x, t, end, At(st[ALIKE ? 0 : 2], t, end), at);
    c.flag = load_flag<S>(done, done_step, t, end, lane);
  }
};

// The pair of each segment but the last: a wave takes a share of it, chunk after chunk.
// Returns whether the share is for the walk that looks at everything (EVERY).
template <class F, int S, int W, bool NEAR, bool ALIKE, bool EVERY>
__device__ __forceinline__ bool fold_walk(const Args& p, uint32_t tile, uint32_t es, int w, int lane, float& A,
                                          float& y) {
  const uint32_t nseg = (uint32_t)p.nseg;
  const int64_t seg = es % (nseg - 1), e = es / (nseg - 1), d0 = tile * 64;
  const uint32_t col = d0 + lane < p.D ? lane : (uint32_t)(p.D - 1 - d0);  // loads stay inside the row
  const float rate = rate_of(p.rate[d0 + col]), rate2 = kLog2E * rate;
  const Inputs<F, S, NEAR, ALIKE> in(p, e, d0, lane, col);
  const int share = (int)p.seg_steps / W, begin = (int)seg * (int)p.seg_steps + w * share, end = begin + share;
  const uint32_t first = first_flag(p, e);
  if (!EVERY && __builtin_expect(any_quick(rate), false)) return true;
  Chunk<F, S> one, two;
  in.load(one, begin, end);
  const float less = EVERY ? less_of(rate) : 1.0f;
  float total = 0.0f;
  bool dropped = false;
  y = 0.0f;
  auto fold = [&](const Chunk<F, S>& c, int t) __attribute__((always_inline)) {
    const uint32_t cut = flag_word(c.flag, t, first);
    Coefficients<S> k;
    by_form<EVERY>(cut == 0, [&](auto form) __attribute__((always_inline)) {
      coefficients<F, S, form>(k, c, rate2, less, cut, (1u << S) - 1);
    });
    total += k.L;
    dropped |= cut != 0;
    y = enter<EVERY>(cut ? kDropped : exp2_fast(-k.L), k.out, y);
  };
  for (int t = begin;;) {  // a share holds whole chunks
    in.load(two, t + S, end);
    fold(one, t);
    t += S;
    if (t >= end) break;
    in.load(one, t + S, end);
    fold(two, t);
    t += S;
    if (t >= end) break;
  }
  A = dropped ? kDropped : exp2_fast(-total);
  return any_odd(seen(0.0f, y));
}

template <class F, int S, int W, bool NEAR, bool ALIKE>
__global__ void __launch_bounds__(64 * W) fold_kernel(const Args p, uint32_t tiles) {
  __shared__ float s_a[W][64], s_y[W][64];
  const int lane = threadIdx.x & 63;
  const int w = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const uint32_t tile = blockIdx.x % tiles, es = blockIdx.x / tiles;
  float A, y;
  if (__builtin_expect(fold_walk<F, S, W, NEAR, ALIKE, false>(p, tile, es, w, lane, A, y), false))
    fold_walk<F, S, W, NEAR, ALIKE, true>(arguments_again(), again(tile), again(es), again(w), la::rarely(lane), A, y);
  s_a[w][lane] = A;
  s_y[w][lane] = y;
  __syncthreads();
  const int64_t column = (int64_t)tile * 64 + lane;
  if (w == 0 && column < p.D) {
    float A;
    const float out = joined_shares<W, 1>(s_a, s_y, lane, A);
    const uint32_t nseg = (uint32_t)p.nseg;
    const int64_t at = ((int64_t)(es / (nseg - 1)) * nseg + es % (nseg - 1)) * p.D + column;
    p.seg_a[at] = A;
    p.seg_y[at] = out;
  }
}

// One block: 64 channels of one row (or of one segment of it), W waves of S steps each at a
// time, the next ones' loads in flight meanwhile.
// Returns whether the segment is for the walk that looks at everything (EVERY).
template <class F, int S, int W, bool NEAR, bool ALIKE, bool EVERY>
__device__ __forceinline__ bool forward_walk(const Args& p, Exchange<W>& s, uint32_t tile, uint32_t es, int w,
                                             int lane) {
  const uint32_t nseg = (uint32_t)p.nseg;
  const int64_t seg = nseg - 1 - es % nseg, e = es / nseg, d0 = tile * 64;
  const bool column = d0 + lane < p.D;
  const uint32_t col = column ? lane : (uint32_t)(p.D - 1 - d0);  // loads stay inside the row
  const float rate = rate_of(p.rate[d0 + col]), rate2 = kLog2E * rate;
  const Inputs<F, S, NEAR, ALIKE> in(p, e, d0, lane, col);
  const Stream<F, S, NEAR> out(p.out, e, d0);
  const int64_t out_st = p.out.st * (int64_t)sizeof(typename F::E);
  const uint32_t out_at = column ? in.at : kNoColumn;
  const int begin = (int)seg * (int)p.seg_steps;
  const int end = (int)(p.T < begin + p.seg_steps ? p.T : begin + p.seg_steps);
  float* marks = p.marks ? p.marks + (e * ((p.T + kMark - 1) / kMark)) * p.D + d0 + lane : nullptr;
  constexpr int kStep = W * S;
  const int ahead = w * S;
  const uint32_t first = first_flag(p, e);
  Chunk<F, S> one, two;
  if (begin < end) in.load(one, begin + ahead, end);

  const float start = p.init ? p.init[e * p.D + d0 + col] : 0.0f;
  float carry = start;  // the state entering the W chunks at hand
  if (seg > 0) {
    carry = joined([&](auto every) __attribute__((always_inline)) {
      float c = start;
      for (int64_t u = 0; u < seg; ++u) {
        const int64_t at = (e * p.nseg + u) * p.D + d0 + col;
        c = enter<every>(p.seg_a[at], p.seg_y[at], c);
      }
      return c;
    });
  }
  if (!EVERY && __builtin_expect(any_quick(rate), false)) return true;
  const float less = EVERY ? less_of(rate) : 1.0f;
  float odd = 0.0f;
  if (W > 1) s.carry[0][lane] = carry;  // the same from every wave
  int buf = 0;
  auto take = [&](const Chunk<F, S>& c, int t) __attribute__((always_inline)) {
    const uint32_t cut = flag_word(c.flag, t, first), live = live_word<S>(t, end);
    const bool whole = cut == 0 && live == (1u << S) - 1;
    Coefficients<S> k;
    by_form<EVERY>(whole, [&](auto form) __attribute__((always_inline)) {
      coefficients<F, S, form>(k, c, rate2, less, cut, live);
    });
    float h = carry;  // the state entering this wave's chunk
    if constexpr (W > 1) {
      s.put(buf, w, lane, exp2_fast(-k.L), k.out, cut);
      meet();
      h = s.template entering<1, EVERY>(buf, w, lane);
    }
    if (marks && column && live && t % kMark == 0) marks[(int64_t)(t / kMark) * p.D] = h;
    by_form<EVERY>(whole, [&](auto form) __attribute__((always_inline)) {
      h = states<F, S, NEAR, form>(k, h, odd, out, t, out_st, out_at, cut, live);
    });
    carry = h;
    if constexpr (W > 1) {  // the last wave's state is what enters the chunks behind
      buf ^= 1;
      if (w == W - 1) s.carry[buf][lane] = h;
    }
  };
  if (begin < end) {
    for (int t = begin;;) {
      in.load(two, t + kStep + ahead, end);
      take(one, t + ahead);
      t += kStep;
      if (t >= end) break;
      in.load(one, t + kStep + ahead, end);
      take(two, t + ahead);
      t += kStep;
      if (t >= end) break;
    }
  }
  // The state behind the row is the last wave's: its steps, or those past the end, which change nothing.
  if (w == W - 1 && column && seg == nseg - 1 && p.final_state) {
    const bool ended = in.done && p.T > 0 && in.done[(p.T - 1) * p.d_st] != 0;
    p.final_state[e * p.D + d0 + lane] = ended ? 0.0f : carry;
  }
  return any_odd(odd);
}

template <class F, int S, int W, bool NEAR, bool ALIKE>
__global__ void __launch_bounds__(64 * W) forward_kernel(const Args p, uint32_t tiles) {
  __shared__ Exchange<W> s;
  const int lane = threadIdx.x & 63;
  const int w = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const uint32_t tile = blockIdx.x % tiles, es = blockIdx.x / tiles;
  if (__builtin_expect(s.any(w, lane, forward_walk<F, S, W, NEAR, ALIKE, false>(p, s, tile, es, w, lane)), false))
    forward_walk<F, S, W, NEAR, ALIKE, true>(arguments_again(), s, again(tile), again(es), again(w),
                                             la::rarely(lane));
}

template <class F, int S, int W, bool NEAR, bool ALIKE>
static hipError_t forward_waves(const Args& a, hipStream_t st) {
  const int64_t tiles = (a.D + 63) / 64;
  if (a.nseg > 1) {
    fold_kernel<F, S, W, NEAR, ALIKE><<<dim3((unsigned)(a.E * (a.nseg - 1) * tiles)), 64 * W, 0, st>>>(a, (uint32_t)tiles);
    const hipError_t e = hipGetLastError();
    if (e != hipSuccess) return e;
  }
  forward_kernel<F, S, W, NEAR, ALIKE><<<dim3((unsigned)(a.E * a.nseg * tiles)), 64 * W, 0, st>>>(a, (uint32_t)tiles);
  return hipGetLastError();
}

template <class F, bool ALIKE>
static hipError_t forward_near(const Args& a, const Plan& p, hipStream_t st) {
  switch (p.waves) {
    case 1: return forward_waves<F, 8, 1, true, ALIKE>(a, st);
    case 4: return forward_waves<F, 8, 4, true, ALIKE>(a, st);
    default: return forward_waves<F, 8, kMaxWaves, true, ALIKE>(a, st);
  }
}

template <class F>
static hipError_t forward_fmt(const Args& a, const Plan& p, hipStream_t st) {
  constexpr int64_t es = sizeof(typename F::E);
  const View* const v[] = {&a.x, &a.ig, &a.dg, &a.out};
  // Steps 2^27 bytes apart or more are those of time-major windows of a million tiles and more, for which a
  // wave by itself is enough; 32-bit offsets take 13 and 23 us where 64-bit ones and blocks of 16 waves took 124
  // and 383 (512 x 16 x 512, bfloat16).
  if (!all_near(v, 4, es)) return forward_waves<F, 8, 1, false, false>(a, st);
  // Inputs by one stride share their offsets: one row of 32768 x 1280, bfloat16, 135 us against 141
  const bool alike = a.x.st == a.dg.st && a.ig.st == a.dg.st;
  return alike ? forward_near<F, true>(a, p, st) : forward_near<F, false>(a, p, st);
}

hipError_t launch_forward(rlscan_format f, const Args& a, const Plan& p, hipStream_t st) {
  switch (f) {
    case RLSCAN_FORMAT_BF16: return forward_fmt<LBf16>(a, p, st);
    case RLSCAN_FORMAT_F16: return forward_fmt<LF16>(a, p, st);
    default: return forward_fmt<LF32>(a, p, st);
  }
}

// Waves of a block.  Sixteen walk a row in the fewest rounds, where there is no more than one tile for a
// compute unit; of blocks of four a compute unit takes several, which fill each other's waits, and short
// rows waste less of them.  A wave by itself waits for no other: for rows of one chunk, and where there are
// many tiles and the last round of four would waste much.  Measured, bfloat16, us forward and backward:
//   256 tiles of 4096 steps   16 waves 144 and 225   4 waves 179 and 251
//   264 tiles of 4096                  245     397           264     364  (in segments 210 and 297, see below)
//   384 tiles of 333                    30      53            27      46
//   800 tiles of 128                    27      47            18      36   1 wave 21 and 36
//   3200 tiles of 64                                          27      67          25     55
//   3200 tiles of 16                                          18      65          10     27
//   8000 tiles of 128                                        114     229         107    199
//   8192 tiles of 256                                        213     406         216    388
static int waves_of(int64_t tiles, int64_t T, bool backward) {
  if (T <= kMark || (tiles >= 2048 && T < (backward ? 256 : 128))) return 1;
  return T <= 4 * kMark || tiles > 256 ? 4 : kMaxWaves;
}

// Segments of a row.  Where a call's tiles do not fill the card, or leave some compute units one more than the
// others, rows are cut into segments: their pairs take a pass over the inputs of their own, about 0.6 (0.35)
// of the time of the walk.  A compute unit takes its blocks one after another if they are of sixteen waves,
// and if they are of four each adds about 0.6 of the time of the first.  The count that is done first by that
// reckoning.  Measured, bfloat16, us forward and backward with them and without: 20 tiles of 32768 steps 149
// and 193 against 919 and 1505, 64 tiles of 4096 63 and 81 against 119 and 199, 264 tiles of 4096 210 and 297
// against 265 and 367; and where the reckoning takes none, 384 tiles of 4096 in two 265 and 363 against 267 and 378.
// Float32 is nearer to what memory gives, and more of its time is the second pass.  In two and whole: 264 tiles of
// 4096 363 and 542 against 307 and 540, 264 of 1024 85 and 136 against 79 and 141, 300 of 8192 744 and 1112 against
// 626 and 1111, 384 of 4096 441 and 647 against 334 and 592, 520 of 2048 323 and 474 against 259 and 470.
Plan make_plan(rlscan_format f, int64_t E, int64_t T, int64_t D, bool backward) {
  Plan p{};
  const int64_t tiles = E * ((D + 63) / 64);
  p.waves = waves_of(tiles, T, backward);
  // segments: whole super-tiles of the widest block, whatever the block is
  const int64_t unit = (int64_t)kMaxWaves * kMark, units = (T + unit - 1) / unit;
  const double pass = backward ? 0.35 : 0.6;
  auto time = [&](int64_t blocks) {
    const double each = (double)((blocks + 255) / 256);
    return p.waves == kMaxWaves ? each : 0.4 + 0.6 * each;
  };
  int64_t want = 1;
  double least = 0.0;
  const int64_t most = f == RLSCAN_FORMAT_F32 ? 256 : 1023;  // tiles
  for (int64_t n = 1; tiles > 0 && tiles <= most && n <= 64 && (n == 1 || n <= units / 2); ++n) {
    const int64_t per = (units + n - 1) / n;
    const double before = n > 1 ? pass * time(tiles * (n - 1)) : 0.0;
    const double cost = (time(tiles * n) + before) * (double)(per + 1);  // one more: a block's start and end
    if (n == 1 || cost < 0.95 * least) {
      want = n;
      least = cost;
    }
  }
  const int64_t per = units > 0 ? (units + want - 1) / want : 1;
  p.seg_steps = per * unit;
  p.nseg = units > 0 ? (units + per - 1) / per : 1;
  p.seg = p.nseg > 1 ? (E * p.nseg * D + 3) / 4 * 4 : 0;
  p.groups = E;
  if (backward) {
    const int64_t columns = (D + 63) / 64, most = 4096 / (columns * p.nseg) + 1;  // about: blocks
    if (p.groups > most) p.groups = most;
    p.part = p.groups * p.nseg > 1 ? (p.groups * p.nseg * D + 3) / 4 * 4 : 0;
  }
  p.floats = 2 * p.seg + p.part;
  return p;
}

}  // namespace gr
}  // namespace rlscan
