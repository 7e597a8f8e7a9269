// rlscan_la_attend.hpp -- the chunk walk that computes linear attention's output and
// each of its gradients.
//
// All four are one recurrence with the parts exchanged.  Along the walk, with rows x and y of
// a chunk (y before or at x),
//   out_x = sum_{y <= x} D_xy scale (a_x . b_y) c_y + in_x S^T a_x
//   S     = across S + sum_y out_y b_y c_y^T
// where D_xy is the decay between the rows:
//   o:  a, b, c = q, k, v    forward in time
//   dq: a, b, c = do, v, k   forward in time
//   dk: a, b, c = v, do, q   backward in time
//   dv: a, b, c = k, q, do   backward in time
// A block walks one head's chunks with S in registers: a, b and c are read and out is
// written once, and no state goes to memory.
#ifndef RLSCAN_LA_ATTEND_HPP
#define RLSCAN_LA_ATTEND_HPP

#include "rlscan_la.hpp"

namespace rlscan {
namespace la {

// Asks the compiler for N matrix instructions with V others after each.
template <int N, int V>
__device__ __forceinline__ void interleave() {
#pragma unroll
  for (int i = 0; i < N; ++i) {
    __builtin_amdgcn_sched_group_barrier(0x008, 1, 0);  // MFMA
    __builtin_amdgcn_sched_group_barrier(0x002, V, 0);  // VALU
  }
}

// Matrix instructions of one mma.
template <int NA, int NB>
constexpr int products() {
  const int top = (NA > NB ? NA : NB) - 1;
  int n = 0;
  for (int i = 0; i < NA; ++i)
    for (int j = 0; j < NB; ++j) n += i + j <= top;
  return n;
}

__device__ __forceinline__ double sum_groups(double x) {  // over the 4 lane groups of a column
  x += __shfl_xor(x, 16);
  x += __shfl_xor(x, 32);
  return x;
}

// A state in memory: element (row of S, column of S) of head eh and segment s.
struct StateView {
  float* p;
  int64_t head, seg, row, col;
  __device__ __forceinline__ float* at(int64_t eh, int64_t s, int64_t r, int64_t c) const {
    return p + eh * head + s * seg + r * row + c * col;
  }
};

struct Attend {
  View a, b, c, out;
  int64_t ga, gb, gc;  // heads that share one of a, b, c (1 or G)
  int A, D;            // sizes of a and b, of c and out
  StateView enter;     // value entering a segment, or p = NULL: zeros
  int enter_closed;    // nothing enters rows whose last step ends an episode
  StateView leave;     // value after the last chunk, or p = NULL
  int leave_closed;    // ... is 0 in rows whose last step ends an episode
  // the dot products that the decay's gradient is made of (DOT)
  View m;              // [E, T, heads, D], dotted with out (without its y = x term)
  int64_t gm;
  double* dot;         // [E, H, T]
  StateView end;       // dotted with the value after the last chunk without the row's last
                       // step's own part (which holds no decay either), or p = NULL
  float* end_dot;      // [E, H]; then S leaves that part out
  float* marks;        // [E, H, nmarks, AD * CD] S at the boundaries between chunks b * mark_chunks - 1
  int64_t nmarks;      // and b * mark_chunks, b = 1 ... nmarks, in the order of registers
};

template <class F, int AD, int CD, int C, int NWV, bool DOT>
struct AttendLds {
  static constexpr int NP = DOT ? F::NW : F::NP;  // terms of P and S
  RowTile<F::NT, C, AD> a;
  MixTile<F::NT, C, AD> b;
  MixTile<F::NT, C, CD> c;
  RowTile<NP, C, C> p;
  Decay<C> dec;
  Odd<C, AD, CD, 64 * NWV> odd;
  float diag[DOT ? C : 1];
  double more[DOT ? (NWV - 2) * C : 1];
  // the waves' dot products: two in the place of decays that are no longer read
  __device__ __forceinline__ double* dots(int w) {
    return w < 2 ? reinterpret_cast<double*>(&dec.hi[0]) + w * C : more + (w - 2) * C;
  }
};

// NWV waves; CD columns of c and out from c0.  FO: the format of out (float32 scratch where
// heads of a group are added up later).  UPD: terms of the rows that go into S.  VEC: View::vec
// of all tensors.
//
// Wave w owns 16*CT columns.  Its tile at of S holds S[at*16 + (l/16)*4 + r][column l%16],
// the layout of an MFMA operand whose steps are in accumulator order (frag_row_acc),
// so S^T a needs no exchange.  Outputs are formed transposed (rows: columns of c,
// columns: x), which leaves four consecutive elements of one row in a lane.
//
// CARE: what is not finite reaches what the recurrence lets it reach and nothing else.
// Without, the walk leaves before its last values and returns false if it met any; all
// that it has written is written again.
template <class F, class FO, int AD, int CD, int C, int NWV, bool REV, bool DOT, int UPD, bool VEC, bool CARE>
__device__ __forceinline__ bool attend_as(AttendLds<F, AD, CD, C, NWV, DOT>& s, const Args& g, const Attend& t, int64_t eh,
                                          int64_t seg, int c0) {
  constexpr int NT = F::NT, NTHR = 64 * NWV, CT = CD / 16 / NWV, AT = AD / 16, XT = C / 16, XX = C / 32;
  constexpr int NP = AttendLds<F, AD, CD, C, NWV, DOT>::NP;
  static_assert(CT * 16 * NWV == CD, "waves share the columns evenly");
  const int tid = threadIdx.x, lane = tid & 63, col = lane & 15, grp = lane >> 4;
  const int w = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int64_t e = eh / g.H, h = eh % g.H;
  const int64_t ha = h / t.ga, hb = h / t.gb, hc = h / t.gc;

  f32x4 S[CT][AT];
  const bool enters = t.enter.p && !(t.enter_closed && row_closed(g, e));
  const int l = rarely(lane), x0 = (l >> 4) * 4, y0 = c0 + (l & 15);
#pragma unroll
  for (int ct = 0; ct < CT; ++ct)
#pragma unroll
    for (int at = 0; at < AT; ++at) {
#pragma unroll
      for (int r = 0; r < 4; ++r) {
        const int x = at * 16 + x0 + r, y = (w * CT + ct) * 16 + y0;
        S[ct][at][r] = enters && x < t.A && y < t.D ? *t.enter.at(eh, seg, x, y) : 0.0f;
      }
      hold_schedule();
    }

  const int64_t p0 = seg * g.seg_chunks;
  const int64_t p1 = p0 + g.seg_chunks < g.chunks ? p0 + g.seg_chunks : g.chunks;
  auto first_step = [&](int64_t n) __attribute__((always_inline)) { return (REV ? g.chunks - 1 - n : n) * (int64_t)C; };
  Piece<F> ra[Share<C, AD, NTHR>::n], rb[Share<C, AD, NTHR>::n], rc[Share<C, CD, NTHR>::n];
  // the tiles that are requested next
  const int64_t step = REV ? -1 : 1;
  TileRows<F> na(t.a, e, ha, first_step(p0), g.T, C), nb(t.b, e, hb, first_step(p0), g.T, C),
      nc(t.c, e, hc, first_step(p0), g.T, C);
  auto request = [&](int64_t n) __attribute__((always_inline)) {
    fetch<F, C, AD, NTHR, REV, VEC>(na, 0, t.A, tid, ra);
    fetch<F, C, AD, NTHR, REV, VEC>(nb, 0, t.A, tid, rb);
    fetch<F, C, CD, NTHR, REV, VEC>(nc, c0, t.D, tid, rc);
    const int64_t t0 = first_step(n + 1);
    na.move(step, t0, g.T, C);
    nb.move(step, t0, g.T, C);
    nc.move(step, t0, g.T, C);
  };
  StepDecay sd{0.0f, 0};
  LaneDecay ld{};
  auto scan = [&](const StepDecay& step, int64_t n) __attribute__((always_inline)) {
    LaneDecay d = scan_decay<C, REV>(step, g.scale, lane);
    if constexpr (DOT)
      if (t.end_dot && first_step(n) + lane == g.T - 1) d.out = 0.0f;
    return d;
  };
  constexpr int DW = NWV - 1;  // the wave that prepares the decays: it has the fewest tiles of P
  if (p0 < p1) {
    if (w == DW) {
      ld = scan(load_decay<C>(g, e, h, first_step(p0), lane), p0);
      if (p0 + 1 < p1) sd = load_decay<C>(g, e, h, first_step(p0 + 1), lane);
    }
    request(p0);
  }
  TileRows<FO> out(t.out, e, h, first_step(p0), g.T, C);
  // S to memory, if chunk c is the first behind a marked boundary
  auto mark = [&](int64_t c) __attribute__((always_inline)) {
    if constexpr (DOT) {
      if (c == 0 || c % g.mark_chunks != 0) return;
      float* to = t.marks + (eh * t.nmarks + c / g.mark_chunks - 1) * (AD * CD) + (w * CT * AT * 64 + lane) * 4;
#pragma unroll
      for (int ct = 0; ct < CT; ++ct)
#pragma unroll
        for (int at = 0; at < AT; ++at) *reinterpret_cast<f32x4*>(to + (ct * AT + at) * 256) = S[ct][at];
    }
  };
  for (int64_t n = p0; n < p1; ++n) {
    const int64_t t0 = first_step(n);
    if (!REV) mark(n);
    out.left = g.T - t0 < C ? (int)(g.T - t0) : C;
    const Decay<C>& d = s.dec;
    stage<F, NTHR>(s.a, ra, tid);
    stage<F, NTHR>(s.b, rb, tid);
    stage<F, NTHR>(s.c, rc, tid);
    // the next decays' inputs arrived before these tiles: kept from the wait for later requests
    StepDecay now = sd;
    if (w == DW) {
      asm volatile("" : "+v"(now.g), "+v"(now.done));
      put_decay<C, REV>(s.dec, ld, lane);
    }
    __syncthreads();
    if (w == DW && n + 2 < p1) sd = load_decay<C>(g, e, h, first_step(n + 2), lane);

    // step, from t0, of tile row it*16 + col
    auto step_of = [&](int it) __attribute__((always_inline)) {
      const int x = it * 16 + col;
      return REV ? C - 1 - x : x;
    };
    Quad<F> m[CT][XT];
    if constexpr (DOT) {
      const TileRows<F> rows(t.m, e, h / t.gm, t0, g.T, C);
#pragma unroll
      for (int ct = 0; ct < CT; ++ct)
#pragma unroll
        for (int it = 0; it < XT; ++it)
          m[ct][it] = load4<F, VEC>(rows, step_of(it), c0 + (w * CT + ct) * 16 + grp * 4, t.D);
    }
    if (n + 1 < p1) request(n + 1);

    // ---- P, as transposed tiles (rows y, columns x): those with y <= x, and for
    // even tiles of x the one behind, which is read with it, as zeros
    constexpr int kTiles = C == 64 ? 12 : 4, kMine = (kTiles + NWV - 1) / NWV, KK = AD / 32;
    auto tile_x = [&](int i) __attribute__((always_inline)) {
      const int idx = i * NWV + w;
      return idx < 4 ? idx >> 1 : 2 + ((idx - 4) >> 2);
    };
    auto tile_y = [&](int i) __attribute__((always_inline)) {
      const int idx = i * NWV + w;
      return idx < 4 ? idx & 1 : (idx - 4) & 3;
    };
#pragma unroll(DOT ? 1 : kMine)
    for (int i = 0; i < kMine; ++i) {
      if (kTiles % NWV != 0 && i * NWV + w >= kTiles) break;
      const int it = tile_x(i), jt = tile_y(i);
      float v[4] = {0.0f, 0.0f, 0.0f, 0.0f};
      const int x = it * 16 + col;
      if (jt <= it) {
        Frag<NT> fa[KK], fb[KK];
#pragma unroll
        for (int kk = 0; kk < KK; ++kk) {
          fb[kk] = frag_row(s.b, jt * 16, kk, lane);
          fa[kk] = frag_row(s.a, it * 16, kk, lane);
        }
        between4<C>(d, g.scale, x, jt * 16 + grp * 4, v);
        f32x4 acc{0, 0, 0, 0};
#pragma unroll
        for (int kk = 0; kk < KK; ++kk) acc = mma<NT, NT, DOT && NT == 2 ? 2 : NT - 1>(fb[kk], fa[kk], acc);
#pragma unroll
        for (int r = 0; r < 4; ++r) v[r] = gated(v[r], acc[r]);
        if constexpr (DOT) {  // the y = x term has no decay: kept apart, in float32
          if (jt == it && grp == col >> 2) {
            s.diag[x] = col & 2 ? (col & 1 ? v[3] : v[2]) : (col & 1 ? v[1] : v[0]);
#pragma unroll
            for (int r = 0; r < 4; ++r) v[r] = r == (col & 3) ? 0.0f : v[r];
          }
        }
      }
      put4(s.p, x, jt * 16 + grp * 4, v);
      hold_schedule();
    }
    if (w == DW && n + 1 < p1) ld = scan(now, n + 1);
    __syncthreads();
    if constexpr (CARE) {
      sweep_odd(s.odd, s.b, s.c, d, rarely(tid));
#pragma unroll
      for (int ct = 0; ct < CT; ++ct) {
        const uint32_t bits = take_odd(S[ct]);
        s.odd.bits[ct][rarely(tid)] = bits;
        const uint64_t who = __ballot(bits != 0);
        if (lane < 16) s.odd.state[(w * CT + ct) * 16 + lane] = (who >> lane & 0x0001000100010001ull) != 0;
      }
      __syncthreads();
    }

    // ---- out and S.  Matrix instructions leave room for others between them, within one
    // wave too: each region below multiplies what the regions before it requested
    // and split, and meanwhile requests and splits for the next.
    const float across = d.across;
    double dot[XT];  // float64: their differences are summed over the row
    float in[XT];
#pragma unroll
    for (int it = 0; it < XT; ++it) {
      dot[it] = 0.0;
      in[it] = d.in[it * 16 + col];
    }
#pragma unroll
    for (int ct = 0; ct < CT; ++ct) {
      const int vt = (w * CT + ct) * 16;
      f32x4 o[XT];
      constexpr bool kTight = DOT && AD == 128 && C == 64;  // no registers to request or split ahead
      Frag<NT> fa[kTight ? 1 : 2][XT], fc[XX];
      Frag<NP> fp[DOT ? 1 : 2][XX];
      auto split_state = [&](int kk) __attribute__((always_inline)) {
        float x[8];
#pragma unroll
        for (int r = 0; r < 4; ++r) {
          x[r] = S[ct][2 * kk][r];
          x[4 + r] = S[ct][2 * kk + 1][r];
        }
        return split<NP>(x);
      };
      auto load_p = [&](int it) __attribute__((always_inline)) {
#pragma unroll
        for (int jj = 0; jj <= it / 2; ++jj) fp[DOT ? 0 : it & 1][jj] = frag_row(s.p, it * 16, jj, lane);
      };
#pragma unroll
      for (int it = 0; it < XT; ++it) {
        o[it] = f32x4{0, 0, 0, 0};
        fa[0][it] = frag_row(s.a, it * 16, 0, lane);
      }
      Frag<NP> fs;
      if (!kTight) fs = split_state(0);
      hold_schedule();
#pragma unroll
      for (int kk = 0; kk < KK; ++kk) {
        Frag<NP> next = fs;
        if constexpr (kTight) {
          fs = split_state(kk);
        } else if (kk + 1 < KK) {
#pragma unroll
          for (int it = 0; it < XT; ++it) fa[(kk + 1) & 1][it] = frag_row(s.a, it * 16, kk + 1, lane);
          next = split_state(kk + 1);
        }
        if (kk + 1 == KK) {
#pragma unroll
          for (int jj = 0; jj < XX; ++jj) fc[jj] = frag_col(s.c, w * CT + ct, jj, lane);
          load_p(0);
        }
#pragma unroll
        for (int it = 0; it < XT; ++it) {
          o[it] = mma(fs, fa[kTight ? 0 : kk & 1][it], o[it]);
          if (kTight && kk + 1 < KK) fa[0][it] = frag_row(s.a, it * 16, kk + 1, lane);
        }
        S[ct][2 * kk] *= across;
        S[ct][2 * kk + 1] *= across;
        interleave<XT * products<NP, NT>(), 4>();
        if (!kTight) fs = next;
        hold_schedule();
      }
      constexpr int GB = DOT ? 2 : 4, kGroups = AT / GB;  // operands of b requested together
      Frag<NT> fb[2][GB];
      Frag<UPD> fy;
      auto split_rows = [&](int jj) __attribute__((always_inline)) {
        float y[8];
        join<NT>(fc[jj], y);
#pragma unroll
        for (int i = 0; i < 8; ++i) y[i] *= d.out[jj * 32 + grp * 8 + i];
        return split<UPD>(y);
      };
      auto load_b = [&](int group) __attribute__((always_inline)) {
#pragma unroll
        for (int i = 0; i < GB; ++i) fb[group & 1][i] = frag_col(s.b, group % kGroups * GB + i, group / kGroups, lane);
      };
#pragma unroll
      for (int it = 0; it < XT; ++it) {
        if constexpr (DOT) {  // no registers to request ahead
          if (it > 0) load_p(it);
          if (it + 1 == XT) load_b(0);
        } else if (it + 1 < XT) {
          load_p(it + 1);
        } else {
          load_b(0);
          fy = split_rows(0);
        }
        o[it] *= in[it];
#pragma unroll
        for (int jj = 0; jj <= it / 2; ++jj) o[it] = mma(fc[jj], fp[DOT ? 0 : it & 1][jj], o[it]);
        hold_schedule();
      }
#pragma unroll
      for (int group = 0; group < XX * kGroups; ++group) {
        const int jj = group / kGroups, at0 = group % kGroups * GB;
        if (DOT && at0 == 0) fy = split_rows(jj);
        Frag<UPD> next = fy;
        if (group + 1 < XX * kGroups) load_b(group + 1);
        if (!DOT && at0 + GB == AT && jj + 1 < XX) next = split_rows(jj + 1);
#pragma unroll
        for (int i = 0; i < GB; ++i) S[ct][at0 + i] = mma(fb[group & 1][i], fy, S[ct][at0 + i]);
        if (group == 0) {
#pragma unroll
          for (int it = 0; it < XT; ++it) {
            if constexpr (DOT) {
              float cx[4];
              get4(s.c, it * 16 + col, vt + grp * 4, cx);
              const float diag = s.diag[it * 16 + col];
#pragma unroll
              for (int r = 0; r < 4; ++r) {
                dot[it] += (double)quad_float<F>(m[ct][it], r) * (double)o[it][r];
                o[it][r] += diag * cx[r];
              }
            }
            const float x[4] = {o[it][0], o[it][1], o[it][2], o[it][3]};
            store4<FO, VEC>(out, step_of(it), c0 + vt + grp * 4, t.D, x);
          }
        }
        interleave<GB * products<NT, UPD>(), 4>();
        fy = next;
        hold_schedule();
      }
    }
    if constexpr (CARE) {  // what was taken out, in the output and the state
      const float nan = __builtin_nanf("");
      const int l = rarely(lane), x0 = l & 15, y0 = (l >> 4) * 4;
      const uint64_t leaving = s.odd.leaving;
#pragma unroll
      for (int ct = 0; ct < CT; ++ct) {
        const int vt = (w * CT + ct) * 16;
#pragma unroll
        for (int it = 0; it < XT; ++it) {
          const int x = it * 16 + x0;
          const uint64_t before = s.odd.before[x];
          const bool enters = d.in[x] != 0.0f;
#pragma unroll 1
          for (int r = 0; r < 4; ++r) {
            const int y = vt + y0 + r;
            if ((s.odd.c[y] & before) == 0 && !(enters && s.odd.state[y] != 0)) continue;
            store_nan<FO, VEC>(out, REV ? C - 1 - x : x, c0 + y, t.D);
            dot[it] = nan;
          }
        }
        const uint64_t c = s.odd.c[vt + x0];
        const uint32_t bits = across != 0.0f ? s.odd.bits[ct][w * 64 + l] : 0;
#pragma unroll
        for (int at = 0; at < AT; ++at)
#pragma unroll
          for (int r = 0; r < 4; ++r) {
            if (((s.odd.b[at * 16 + y0 + r] | c) & leaving) != 0 || (bits >> (at * 4 + r) & 1) != 0) S[ct][at][r] = nan;
            hold_schedule();
          }
      }
    }
    out.p += step * C * out.st;
    if constexpr (DOT) {
#pragma unroll
      for (int it = 0; it < XT; ++it) {
        const double v = sum_groups(dot[it]);
        if (grp == 0) s.dots(w)[it * 16 + col] = v;
      }
    }
    __syncthreads();
    if (REV) mark(g.chunks - 1 - n);
    if constexpr (DOT) {
      if (w == DW && lane < C) {  // by the wave that writes the next decays in their place
        double v = 0.0;
#pragma unroll
        for (int i = 0; i < NWV; ++i) v += s.dots(i)[lane];
        const int64_t st = t0 + (REV ? C - 1 - lane : lane);
        if (st < g.T) t.dot[eh * g.T + st] = v;
      }
    }
  }
  if constexpr (!CARE) {
    bool odd = false;
#pragma unroll
    for (int ct = 0; ct < CT; ++ct) odd |= any_odd(S[ct]);
    if (any_of_block<NTHR>(s.odd.wave, odd, tid)) return false;
  }

  if (seg != g.nseg - 1) return true;
  if (t.leave.p) {
    const bool closed = t.leave_closed && row_closed(g, e);
#pragma unroll
    for (int ct = 0; ct < CT; ++ct)
#pragma unroll
      for (int at = 0; at < AT; ++at) {
#pragma unroll
        for (int r = 0; r < 4; ++r) {
          const int x = at * 16 + grp * 4 + r, y = c0 + (w * CT + ct) * 16 + col;
          if (x < t.A && y < t.D) *t.leave.at(eh, 0, x, y) = closed ? 0.0f : S[ct][at][r];
        }
        hold_schedule();
      }
  }
  if constexpr (DOT) {
    if (t.end_dot) {
      float v = 0.0f;
      if (t.end.p && !row_closed(g, e)) {
#pragma unroll
        for (int ct = 0; ct < CT; ++ct)
#pragma unroll
          for (int at = 0; at < AT; ++at) {
#pragma unroll
            for (int r = 0; r < 4; ++r) {
              const int x = at * 16 + grp * 4 + r, y = c0 + (w * CT + ct) * 16 + col;
              if (x < t.A && y < t.D) v += S[ct][at][r] * *t.end.at(eh, 0, x, y);
            }
            hold_schedule();
          }
      }
#pragma unroll
      for (int o = 1; o < 64; o <<= 1) v += __shfl_xor(v, o);
      if (lane == 0) s.diag[w] = v;
      __syncthreads();
      if (tid == 0) {
        for (int i = 1; i < NWV; ++i) v += s.diag[i];
        t.end_dot[eh] = v;
      }
    }
  }
  return true;
}

// P: the kernel's argument, a struct with Args a and the Attend at T.
template <class F, class FO, int AD, int CD, int C, int NWV, bool REV, bool DOT, int UPD, bool VEC, class P>
__device__ __forceinline__ void attend(AttendLds<F, AD, CD, C, NWV, DOT>& s, const P& p, Attend P::*t, int64_t eh,
                                       int64_t seg, int c0) {
  if (attend_as<F, FO, AD, CD, C, NWV, REV, DOT, UPD, VEC, false>(s, p.a, p.*t, eh, seg, c0)) return;
  const P again = argument_again<P>();
  asm volatile("" : "+s"(eh), "+s"(seg), "+s"(c0));
  attend_as<F, FO, AD, CD, C, NWV, REV, DOT, UPD, VEC, true>(s, again.a, again.*t, eh, seg, c0);
}

}  // namespace la
}  // namespace rlscan

#endif
