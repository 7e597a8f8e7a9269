// rlscan_checks.hpp -- what the entries of the policy operators check on the host before
// any HIP call: strides, alignment, and memory that a call would both read and write.
#ifndef RLSCAN_CHECKS_HPP
#define RLSCAN_CHECKS_HPP

#include <cstdint>

#include "rlscan.h"
#include "rlscan_la.hpp"

namespace rlscan {
namespace checks {

using la::View;

constexpr int64_t kMaxElems = (int64_t)1 << 46;  // keeps every byte offset far inside int64

inline rlscan_status launched(hipError_t e) { return e == hipSuccess ? RLSCAN_OK : RLSCAN_ERR_HIP; }

inline int elem_size(rlscan_format f) {
  switch (f) {
    case RLSCAN_FORMAT_F32: return 4;
    case RLSCAN_FORMAT_BF16: return 2;
    case RLSCAN_FORMAT_F16: return 2;
  }
  return 0;
}

// Memory that a call reads or writes.  `step` and `row` are 0 for plain arrays; a
// strided tensor has its step's own bytes [lo, lo + row) repeated every `step`.
struct Span {
  uintptr_t lo, hi;
  int64_t step, env, row;
};

inline Span plain(const void* p, int64_t bytes) {
  const uintptr_t b = (uintptr_t)p;
  return Span{b, b + (uintptr_t)(p ? bytes : 0), 0, 0, 0};
}

// Whether two spans can share a byte.  Slices of one buffer with equal strides (the
// parts of one fused projection) lie side by side in every step.
inline bool overlap(const Span& x, const Span& y) {
  if (!(x.lo < y.hi && y.lo < x.hi)) return false;
  if (x.row > 0 && y.row > 0 && x.step == y.step && x.env == y.env) {
    // The smaller of the two strides repeats the pattern; rows that fit side by
    // side in one period, with the other stride a multiple of it, never meet.
    const int64_t lo = x.step < x.env ? x.step : x.env, hi = x.step < x.env ? x.env : x.step;
    if (lo > 0 && hi % lo == 0) {
      const int64_t d = (int64_t)(((y.lo > x.lo ? y.lo - x.lo : x.lo - y.lo)) % (uintptr_t)lo);
      const Span& first = y.lo > x.lo ? x : y;
      const Span& second = y.lo > x.lo ? y : x;
      if (first.row <= d && d + second.row <= lo) return false;
    }
  }
  return true;
}

struct Spans {
  Span in[16], out[8];
  int n_in = 0, n_out = 0;
  void add_in(const Span& s) {
    if (s.hi > s.lo) in[n_in++] = s;
  }
  void add_out(const Span& s) {
    if (s.hi > s.lo) out[n_out++] = s;
  }
  bool clash() const {
    for (int i = 0; i < n_out; ++i) {
      for (int j = 0; j < n_in; ++j)
        if (overlap(out[i], in[j])) return true;
      for (int j = 0; j < i; ++j)
        if (overlap(out[i], out[j])) return true;
    }
    return false;
  }
};

inline bool aligned(const void* p, int es) { return (uintptr_t)p % (uintptr_t)es == 0; }

// One [E, T, heads, D] tensor: strides in range, and for outputs no element twice.
struct HeadsCheck {
  int64_t E, T, es;
  rlscan_status st = RLSCAN_OK;

  View view(const rlscan_heads* x, int64_t heads, int64_t D, bool output, Spans& spans) {
    View v{};
    if (st != RLSCAN_OK) return v;
    if (!x || !x->data) {
      st = RLSCAN_ERR_NULL;
      return v;
    }
    if (!aligned(x->data, (int)es)) {
      st = RLSCAN_ERR_ALIGN;
      return v;
    }
    const int64_t n[3] = {E, T, heads}, s[3] = {x->env, x->step, x->head};
    int64_t extent = D;
    for (int i = 0; i < 3; ++i) {
      if (s[i] < 0 || (n[i] > 1 && s[i] > kMaxElems / n[i])) {
        st = RLSCAN_ERR_SHAPE;
        return v;
      }
      extent += (n[i] - 1) * s[i];
    }
    if (output) {  // from the smallest stride up, each has to pass what lies inside it
      bool used[3] = {false, false, false};
      int64_t inner = D;
      for (int round = 0; round < 3; ++round) {
        int best = -1;
        for (int i = 0; i < 3; ++i)
          if (!used[i] && (best < 0 || s[i] < s[best])) best = i;
        used[best] = true;
        if (n[best] > 1) {
          if (s[best] < inner) {
            st = RLSCAN_ERR_ALIAS;
            return v;
          }
          inner += (n[best] - 1) * s[best];
        }
      }
    }
    v.p = x->data;
    v.se = E > 1 ? s[0] : 0;
    v.st = T > 1 ? s[1] : D;  // D: one step's end is the next one's start
    v.sh = heads > 1 ? s[2] : 0;
    const int64_t unit = 16 / es;
    v.vec = D % 8 == 0 && aligned(x->data, 16) && v.se % unit == 0 && v.st % unit == 0 && v.sh % unit == 0 &&
            v.st >= D && v.st * es <= ((int64_t)1 << 25);
    Span sp = plain(x->data, extent * es);
    sp.row = (D + (heads - 1) * s[2]) * es;
    const int64_t period = T > 1 ? s[1] : (E > 1 ? s[0] : 0);  // 0: one step, a plain range
    sp.step = period * es;
    sp.env = (E > 1 ? s[0] : period) * es;
    if (output) spans.add_out(sp);
    else spans.add_in(sp);
    return v;
  }
};

}  // namespace checks
}  // namespace rlscan

#endif
