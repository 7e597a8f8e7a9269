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
// of steps exact, and 1 - a^2 = (1 - a)(1 + a) does not cancel.  What a fast decay leaves of a state
// or a gradient would lose its bits that way (all of them for s > 17), and an infinite one would be
// inf - inf.  Blocks with a rate of kQuick or more therefore hold a itself where s is above 0.17, and blocks
// that met a value that is not finite walk their rows once more, looking at every value (kEvery): an infinite one
// stays until its episode ends, however little its decays would leave of it.  A product of decays is the
// exponential of a sum.
#ifndef RLSCAN_GR_HPP
#define RLSCAN_GR_HPP

#include <type_traits>

#include "rlscan_la.hpp"
#include "rlscan_logits.hpp"

namespace rlscan {
namespace gr {

using la::View;
using logits::LBf16;
using logits::LF16;
using logits::LF32;

constexpr int kMark = RLSCAN_MARK_STEPS;  // steps from one marked state to the next
constexpr int kMaxWaves = 16;              // of a block
constexpr int kBackWaves = 128 / kMark;    // the same, of the gradients

struct Args {
  View x, ig, dg;         // values and the two gates' logits (heads unused)
  View dout;              // backward
  View out, dx, dig, ddg; // outputs
  const float* rate;      // [D]
  const uint8_t* done;    // [E, T] or [T, E] by strides, or NULL
  int64_t d_se, d_st;
  const uint8_t* reset;   // [E] or NULL: whether step 0 starts anew
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
  int waves;           // of a block
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

// Bit k of a chunk's words, as a mask of 32 bits.  An AND with it takes inf and NaN to 0 too.
__device__ __forceinline__ uint32_t spread(uint32_t word, int k) { return (uint32_t)((int32_t)(word << (31 - k)) >> 31); }
__device__ __forceinline__ float keep(float x, uint32_t mask) {
  return __builtin_bit_cast(float, __builtin_bit_cast(uint32_t, x) & mask);
}
// x where the mask is set, else y
__device__ __forceinline__ float pick(uint32_t mask, float x, float y) {
  return __builtin_bit_cast(float, (__builtin_bit_cast(uint32_t, x) & mask) | (__builtin_bit_cast(uint32_t, y) & ~mask));
}

// A rate as the kernels take it: NaN below 0, and -0 as 0.
__device__ __forceinline__ float rate_of(float rate) {
  return rate >= 0.0f ? __builtin_fabsf(rate) : __builtin_nanf("");
}

// What a chunk's arithmetic looks at: nothing but its steps; which of them start anew (cut) or lie past the end
// (not live); and besides these how each decay is held and whether what it is multiplied with is infinite.
// Finite values come out the same of each, to the last bit: sums and products are contracted by hand.
enum Form { kPlain, kCut, kEvery };

// f(form): the form that a chunk takes.  EVERY is known for a whole walk, so that each walk has its own forms alone.
template <bool EVERY, class Call>
__device__ __forceinline__ void by_form(bool whole, const Call& f) {
  if constexpr (EVERY) f(std::integral_constant<Form, kEvery>());
  else if (whole) f(std::integral_constant<Form, kPlain>());
  else f(std::integral_constant<Form, kCut>());
}

// Rates from which on a block holds fast decays as a: below, a > 0.135 and a - 1 keeps it to 4 of 2^-24.  Measured,
// us, forward and gradients by the first two forms and by kEvery: 8 x 4096 x 2048 bfloat16 351 and 484, 64 x 333 x 768
// float32 152 and 171, 8000 x 128 x 64 bfloat16 300 and 431.
constexpr float kQuick = 2.0f;
__device__ __forceinline__ bool any_quick(float rate) { return __builtin_amdgcn_ballot_w64(rate >= kQuick) != 0; }
// 1 in the sum a - less that is held for such a, 0 in blocks with a quick rate.
__device__ __forceinline__ float less_of(float rate) {
  return __builtin_bit_cast(float, __builtin_amdgcn_readfirstlane(any_quick(rate) ? 0 : 0x3f800000));
}
// The same number, unknown to the compiler, and the kernel's argument read from memory once more: what the second
// walk computes from them stays there, and the first walk's registers are its own.
__device__ __forceinline__ uint32_t again(uint32_t x) {
  asm volatile("" : "+s"(x));
  return x;
}
__device__ __forceinline__ Args arguments_again() {
  auto* p = __builtin_amdgcn_kernarg_segment_ptr();
  asm volatile("" : "+s"(p));
  return *(const Args*)p;
}

// `odd` once it has seen an x that is not finite, or an x or a y that is infinite, is infinite.
__device__ __forceinline__ float seen(float odd, float x) {
  return __builtin_fabsf(x) < __builtin_inff() ? odd : __builtin_inff();
}
__device__ __forceinline__ float seen(float odd, float x, float y) {
  return __builtin_fmaxf(__builtin_fmaxf(odd, __builtin_fabsf(x)), __builtin_fabsf(y));
}
__device__ __forceinline__ bool any_odd(float odd) {
  return __builtin_amdgcn_ballot_w64(odd == __builtin_inff()) != 0;
}

// A decay a = 2^-y for y >= 0 (y: s in units of log 2): a - 1, with the sign bit set (a = 1: -0).  For y below a
// quarter a cubic times y, fitted to (1 - 2^-y) / y by least largest relative error, 2^-24 of the value; above it
// 1 - a >= 0.16 loses at most three bits.  With less = 0 a itself is held there, with the sign bit clear; below
// the normal numbers the smallest of these, so that an infinite value stays.
template <Form FORM>
__device__ __forceinline__ float decay_of(float y, float less) {
  const float a = exp2_fast(-y), far = (FORM == kEvery && y == y ? __builtin_fmaxf(a, 1.17549435e-38f) : a) - less;
  float p = __builtin_fmaf(y, 0.008974975906f, -0.055404357612f);
  p = __builtin_fmaf(y, p, 0.240221500397f);
  p = __builtin_fmaf(y, p, -0.693147122860f);
  return y < 0.25f ? y * p : far;
}

// Whether a decay is held as a - 1, as a mask of 32 bits.
__device__ __forceinline__ uint32_t near_one(float decay) {
  return (uint32_t)(__builtin_bit_cast(int32_t, decay) >> 31);
}
// The decay of a step that starts anew (a = 0) or not, and that lies before the end or (a = 1) not.
template <Form FORM>
__device__ __forceinline__ float decay_behind(float decay, uint32_t cut) {
  return FORM == kEvery ? keep(decay, ~cut) : pick(cut, -1.0f, decay);
}
template <Form FORM>
__device__ __forceinline__ float decay_before(float decay, uint32_t live) {
  return FORM == kEvery ? pick(live, decay, -0.0f) : keep(decay, live);
}
// 1 - a^2
template <Form FORM>
__device__ __forceinline__ float one_less_square(float decay) {
  const float twice = -2.0f * decay;
  return __builtin_fmaf(-decay, decay, FORM == kEvery ? pick(near_one(decay), twice, 1.0f) : twice);
}
// a h
template <Form FORM>
__device__ __forceinline__ float decayed(float decay, float h) {
  if (FORM != kEvery) return __builtin_fmaf(decay, h, h);
  // h + (a - 1) h is inf - inf for an infinite h, so the largest number stands for it in the product
  const uint32_t near = near_one(decay);
  const float most = __builtin_amdgcn_fmed3f(h, -3.40282347e38f, 3.40282347e38f);
  return __builtin_fmaf(decay, pick(near, most, h), keep(h, near));
}

// A segment's pair in the workspace: A is kDropped where it holds a cut, which takes any c, inf
// and NaN too, to y.
constexpr float kDropped = -1.0f;
// EVERY: c may be infinite, and stays so where A is too little for float32.
template <bool EVERY>
__device__ __forceinline__ float enter(float A, float y, float c) {
  return A < 0.0f ? y : EVERY && __builtin_isinf(c) ? c + y : __builtin_fmaf(A, c, y);
}
// join(every): pairs joined one after the other; once more with care where the result is not finite.
template <class Join>
__device__ __forceinline__ float joined(const Join& join) {
  float c = join(std::false_type());
  if (__builtin_expect(any_odd(seen(0.0f, c)), false)) c = join(std::true_type());
  return c;
}
// The pair of a block's shares, of which STEP 1: the lowest wave's, -1: the highest one's comes first.
template <int W, int STEP>
__device__ __forceinline__ float joined_shares(const float (&s_a)[W][64], const float (&s_y)[W][64], int lane, float& A) {
  float a[W], y[W];  // asked for all at once, and no branches between
#pragma unroll
  for (int u = 0; u < W; ++u) {
    a[u] = s_a[STEP > 0 ? u : W - 1 - u][lane];
    y[u] = s_y[STEP > 0 ? u : W - 1 - u][lane];
  }
  bool dropped = false;
  A = 1.0f;
#pragma unroll
  for (int u = 0; u < W; ++u) {
    dropped |= a[u] < 0.0f;
    A *= a[u];
  }
  if (dropped) A = kDropped;
  return joined([&](auto every) __attribute__((always_inline)) {
    float c = 0.0f;
#pragma unroll
    for (int u = 0; u < W; ++u) c = enter<every>(a[u], y[u], c);
    return c;
  });
}

// The same value, of which the compiler knows nothing: keeps it from doing the work that both
// forms of a branch begin with before the branch, where its results lie in registers for long.
__device__ __forceinline__ float apart(float x) {
  asm("" : "+v"(x));
  return x;
}
__device__ __forceinline__ uint16_t apart(uint16_t x) {
  uint32_t y = x;
  asm("" : "+v"(y));
  return (uint16_t)y;
}

// The steps of a chunk as offsets from its first: t + k, or the row's last step where that is past
// the end.  NEAR: 32-bit offsets of buffer instructions.
template <int S, bool NEAR>
struct Steps {
  int64_t st;  // bytes from a step to the next
  int last;
  __device__ __forceinline__ Steps(int64_t st_, int t, int end)
      : st(st_), last(end - t < S ? (end > t ? end - t - 1 : 0) : S - 1) {}
  __device__ __forceinline__ int64_t far(int k) const { return (k < last ? k : last) * st; }
  __device__ __forceinline__ int near(int k) const { return (k < last ? k : last) * (int)st; }
};

// One [E, T, D] tensor at a row and a tile of columns.
constexpr uint32_t kNoColumn = 0x80000000u;
template <class F, int S, bool NEAR>
struct Stream {
  using E = typename F::E;
  static constexpr int kNonTemporal = 2;
  char* p;

  __device__ __forceinline__ Stream(const View& v, int64_t e, int64_t column)
      : p(static_cast<char*>(const_cast<void*>(v.p)) + (e * v.se + column) * (int64_t)sizeof(E)) {}
  static __device__ __forceinline__ __amdgpu_buffer_rsrc_t resource(char* q, bool some = true) {
    return __builtin_amdgcn_make_buffer_rsrc(q, 0, some ? 0x7fffffff : 0, 0x00020000);
  }
  // Steps [t, t + S) of the lane whose column is `lane` bytes behind the tile's first.  A chunk that
  // lies past the end altogether is asked for out of range, which reads no memory.
  __device__ __forceinline__ void load(E (&x)[S], int t, int end, const Steps<S, NEAR>& steps, uint32_t lane) const {
    char* const q = p + (t < end ? t : end - 1) * steps.st;
#pragma unroll
    for (int k = 0; k < S; ++k) {
      if constexpr (!NEAR) x[k] = *reinterpret_cast<const E*>(q + steps.far(k) + lane);
      else if constexpr (sizeof(E) == 4)
        x[k] = __builtin_bit_cast(float, __builtin_amdgcn_raw_buffer_load_b32(resource(q, t < end), lane, steps.near(k), 0));
      else x[k] = __builtin_amdgcn_raw_buffer_load_b16(resource(q, t < end), lane, steps.near(k), 0);
    }
  }
  // Step t + k; lane: kNoColumn for one that has none, which a buffer instruction drops as out of range.
  __device__ __forceinline__ void store(E v, int t, int k, int64_t st, uint32_t lane) const {
    char* const q = p + t * st;
    if constexpr (!NEAR) {
      if (lane != kNoColumn) *reinterpret_cast<E*>(q + k * st + lane) = v;
    } else if constexpr (sizeof(E) == 4) {
      __builtin_amdgcn_raw_buffer_store_b32(__builtin_bit_cast(uint32_t, v), resource(q), lane, k * (int)st, kNonTemporal);
    } else {
      __builtin_amdgcn_raw_buffer_store_b16(v, resource(q), lane, k * (int)st, kNonTemporal);
    }
  }
};

// Whether a chunk of each tensor lies within 2^31 bytes.
inline bool all_near(const View* const* v, int n, int64_t es) {
  for (int i = 0; i < n; ++i)
    if (v[i]->st * es >= (int64_t)1 << 27) return false;
  return true;
}

// Bit k: step t + k starts anew; the lane's byte of `done` is loaded ahead.  Out of range, which reads
// as 0, is what lies outside the row, and everything where there are no flags: the load is always made,
// since behind one that may not have been made the compiler waits for all of them.
template <int S>
__device__ __forceinline__ uint8_t load_flag(const uint8_t* done, int64_t step, int t, int end, int lane) {
  const auto rs = __builtin_amdgcn_make_buffer_rsrc(const_cast<uint8_t*>(done) + (t - 1) * step, 0,
                                                    done ? 0x7fffffff : 0, 0x00020000);
  const bool in = lane < S && t + lane > 0 && t + lane < end;  // a row's steps lie at most 2^22 bytes apart
  return __builtin_amdgcn_raw_buffer_load_b8(rs, in ? lane * (int)step : (int)kNoColumn, 0, 0);
}
// first: bit 0 if the row's first step starts anew.
__device__ __forceinline__ uint32_t flag_word(uint8_t flag, int t, uint32_t first) {
  return (uint32_t)__builtin_amdgcn_ballot_w64(flag != 0) | (t == 0 ? first : 0);
}
__device__ __forceinline__ uint32_t first_flag(const Args& p, int64_t e) {
  return __builtin_amdgcn_readfirstlane(p.reset && p.reset[e] != 0 ? 1 : 0);
}

// Bit k: step t + k lies before the end.
template <int S>
__device__ __forceinline__ uint32_t live_word(int t, int end) {
  const int n = end - t;
  return n >= S ? (1u << S) - 1 : n > 0 ? (1u << n) - 1 : 0;
}

// The block's barrier: LDS writes are done, loads and stores to memory stay in flight.
__device__ __forceinline__ void meet() {
  __builtin_amdgcn_fence(__ATOMIC_RELEASE, "workgroup", "local");
  __builtin_amdgcn_s_barrier();
  __builtin_amdgcn_fence(__ATOMIC_ACQUIRE, "workgroup", "local");
}

// What the waves of a block tell each other of their chunks, twice: one set is written
// while the other is read.
template <int W>
struct Exchange {
  float a[2][W][64], y[2][W][64], carry[2][64];
  uint32_t cut[2][W], odd[W];

  __device__ __forceinline__ void put(int buf, int w, int lane, float A, float out, uint32_t cut_word) {
    a[buf][w][lane] = A;
    y[buf][w][lane] = out;
    if (lane == 0) cut[buf][w] = cut_word;
  }
  // Whether a wave of the block says so; all of them are done with the walk behind them.
  __device__ __forceinline__ bool any(int w, int lane, bool mine) {
    if constexpr (W == 1) return mine;
    if (lane == 0) odd[w] = mine;
    meet();
    return __builtin_amdgcn_ballot_w64(lane < W && odd[lane < W ? lane : 0] != 0) != 0;
  }
  // What enters wave w's chunk from the chunks `before` it (STEP 1: lower waves, -1: higher ones).
  // A wave with a cut takes anything to its y, so the walk begins behind the nearest of these.
  // EVERY: what enters may be infinite.
  template <int STEP, bool EVERY>
  __device__ __forceinline__ float entering(int buf, int w, int lane) const {
    const uint32_t cuts = (uint32_t)__builtin_amdgcn_ballot_w64(lane < W && cut[buf][lane < W ? lane : 0] != 0);
    float c = carry[buf][lane];
    const uint32_t mine = STEP > 0 ? cuts & ((1u << w) - 1) : cuts & ~((2u << w) - 1);
    const int near = STEP > 0 ? 31 - __builtin_clz(mine | 1) : __builtin_ctz(mine | (1u << (W - 1)));
    const int from = mine ? near : STEP > 0 ? 0 : W - 1;
    // Eight pairs are asked for at once: one after the other their latencies would add up.
    constexpr int B = W < 8 ? W : 8;
#pragma unroll
    for (int half = 0; half < W / B; ++half) {
      const int base = STEP > 0 ? half * B : W - B - half * B;
      if (STEP > 0 ? base + B <= from || base >= w : base > from || base + B - 1 <= w) continue;
      float A[B], Y[B];
#pragma unroll
      for (int i = 0; i < B; ++i) {
        A[i] = a[buf][base + i][lane];
        Y[i] = y[buf][base + i][lane];
      }
#pragma unroll
      for (int j = 0; j < B; ++j) {
        const int i = STEP > 0 ? j : B - 1 - j, u = base + i;
        if (mine && u == from) c = Y[i];
        else if (STEP > 0 ? u >= from && u < w : u <= from && u > w)
          c = EVERY ? enter<true>(A[i], Y[i], c) : __builtin_fmaf(A[i], c, Y[i]);
      }
    }
    return c;
  }
};

}  // namespace gr
}  // namespace rlscan

#endif
