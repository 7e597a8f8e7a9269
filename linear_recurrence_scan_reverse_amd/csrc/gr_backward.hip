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
#include "rlscan_gr.hpp"
#include "rlscan_sums.hpp"

namespace rlscan {
namespace gr {

// One block: 64 channels of the rows e, e + groups, ... (or of one segment of them), W waves of
// kMark steps each at a time.  FOLD: the pair of the segment alone.
template <class F, int W, bool FOLD>
__global__ void __launch_bounds__(64 * W) backward_kernel(const Args p, int64_t tiles) {
  using E = typename F::E;
  constexpr int S = kMark;
  __shared__ float s_a[2][W][64], s_y[2][W][64];
  const int lane = threadIdx.x & 63;
  const int w = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int64_t nseg = FOLD ? p.nseg - 1 : p.nseg;  // nothing comes before the first segment
  const int64_t tile = blockIdx.x % tiles, es = blockIdx.x / tiles;
  const int64_t seg = es % nseg + (FOLD ? 1 : 0), group = es / nseg;
  const int64_t d = tile * 64 + lane;
  const bool col_ok = d < p.D;
  const int64_t dc = col_ok ? d : p.D - 1;  // loads stay inside the row
  const float rate = p.rate[dc];
  const int64_t begin = seg * p.seg_steps;
  const int64_t end = p.T < begin + p.seg_steps ? p.T : begin + p.seg_steps;
  const int64_t nmarks = (p.T + S - 1) / S;
  float d_rate = 0.0f;
  int buf = 0;
  for (int64_t e = group; e < p.E; e += p.groups) {
    const E* px = static_cast<const E*>(p.x.p) + e * p.x.se + dc;
    const E* pi = static_cast<const E*>(p.ig.p) + e * p.ig.se + dc;
    const E* pr = static_cast<const E*>(p.dg.p) + e * p.dg.se + dc;
    const E* pg = static_cast<const E*>(p.dout.p) + e * p.dout.se + dc;
    E* ox = static_cast<E*>(const_cast<void*>(p.dx.p)) + e * p.dx.se + d;
    E* oi = static_cast<E*>(const_cast<void*>(p.dig.p)) + e * p.dig.se + d;
    E* od = static_cast<E*>(const_cast<void*>(p.ddg.p)) + e * p.ddg.se + d;
    const uint8_t* done = p.done ? p.done + e * p.d_se : nullptr;
    float carry = 0.0f;  // e entering the super-tile from the steps behind it
    if (!FOLD) {
      if (p.d_final && !(done && p.T > 0 && done[(p.T - 1) * p.d_st] != 0)) carry = p.d_final[e * p.D + dc];
      for (int64_t u = nseg - 1; u > seg; --u) {
        const int64_t at = (e * p.nseg + u) * p.D + dc;
        carry = enter(p.seg_a[at], p.seg_y[at], carry);
      }
    }
    float total = 0.0f;  // FOLD: sum of s over the segment
    bool dropped = false;
    const int64_t units = (end - begin + W * S - 1) / (W * S);
    for (int64_t n = units - 1; n >= 0; --n) {
      const int64_t c0 = begin + (n * W + w) * S;
      E gr[S], x[S], gi[S], gd[S];
#pragma unroll
      for (int k = 0; k < S; ++k) {
        const int64_t t = c0 + k < end ? c0 + k : end - 1;
        gd[k] = pr[t * p.dg.st];
        gr[k] = pg[t * p.dout.st];
        if (!FOLD) {
          x[k] = px[t * p.x.st];
          gi[k] = pi[t * p.ig.st];
        }
      }
      float h = 0.0f;
      if (!FOLD && c0 < end) h = p.marks[(e * nmarks + c0 / S) * p.D + dc];
      bool dn = false;  // lane k: whether step c0 + k starts anew
      if (done && lane < S) {
        const int64_t t = c0 + lane;
        if (t > 0 && t < end) dn = done[(t - 1) * p.d_st] != 0;
      }
      const uint32_t cut = (uint32_t)__builtin_amdgcn_ballot_w64(dn);
      float em1[S], sr[S], L = 0.0f, y = 0.0f;
#pragma unroll
      for (int k = S - 1; k >= 0; --k) {
        const bool live = c0 + k < end, fresh = (cut >> k) & 1;
        sr[k] = fresh ? 0.0f : sigmoid(F::get(gd[k]));  // not looked at: it may be NaN
        const float s = rate * sr[k];
        em1[k] = live ? decay_less_1(s) : 0.0f;
        L += live ? s : 0.0f;
        const float g = y + (live ? F::get(gr[k]) : 0.0f);
        y = fresh ? 0.0f : decayed(em1[k], g);
      }
      const float A = cut ? kDropped : exp2_fast(-kLog2E * L);
      s_a[buf][w][lane] = A;
      s_y[buf][w][lane] = y;
      __syncthreads();
      float c = carry;  // e entering this wave's chunk
      for (int u = W - 1; u > w; --u) c = enter(s_a[buf][u][lane], s_y[buf][u][lane], c);
      float next = c;
      for (int u = w; u >= 0; --u) next = enter(s_a[buf][u][lane], s_y[buf][u][lane], next);
      carry = next;
      buf ^= 1;
      if (FOLD) {
        total += L;
        dropped |= cut != 0;
        continue;
      }
      float before[S], u_[S], si[S];
#pragma unroll
      for (int k = 0; k < S; ++k) {
        const bool fresh = (cut >> k) & 1;
        si[k] = sigmoid(F::get(gi[k]));
        u_[k] = si[k] * F::get(x[k]);
        before[k] = fresh ? 0.0f : h;
        const float step = fresh ? -1.0f : em1[k];
        h = decayed(step, before[k]) + __builtin_amdgcn_sqrtf(one_less_square(step)) * u_[k];
      }
#pragma unroll
      for (int k = S - 1; k >= 0; --k) {
        const bool live = c0 + k < end, fresh = (cut >> k) & 1;
        const float g = c + (live ? F::get(gr[k]) : 0.0f);
        const float m2 = fresh ? 1.0f : one_less_square(em1[k]);
        const float over_m = m2 >= 1.1754944e-38f ? __builtin_amdgcn_rsqf(m2) : 0.0f;  // a held state has no part in u
        const float du = m2 * over_m * g;
        const float dx = si[k] * du;
        const float a = 1.0f + em1[k];
        const float dlog = g * (a * (before[k] - u_[k] * a * over_m));
        const float t_ = fresh || !live ? 0.0f : sr[k] * dlog;
        d_rate -= t_;
        if (col_ok && live) {
          const int64_t t = c0 + k;
          ox[t * p.dx.st] = F::put(dx);
          oi[t * p.dig.st] = F::put(u_[k] * du * (1.0f - si[k]));
          od[t * p.ddg.st] = F::put(-(rate * (1.0f - sr[k])) * t_);
        }
        c = fresh ? 0.0f : decayed(em1[k], g);
      }
    }
    if (FOLD) {
      __syncthreads();
      s_a[0][w][lane] = total;
      s_y[0][w][lane] = dropped ? 1.0f : 0.0f;
      __syncthreads();
      if (w == 0 && col_ok) {
        float sum = 0.0f, any = 0.0f;
        for (int u = 0; u < W; ++u) {
          sum += s_a[0][u][lane];
          any += s_y[0][u][lane];
        }
        const int64_t at = (e * p.nseg + seg) * p.D + d;
        p.seg_a[at] = any > 0.0f ? kDropped : exp2_fast(-kLog2E * sum);
        p.seg_y[at] = carry;
      }
      __syncthreads();
    } else if (w == 0 && col_ok && seg == 0 && p.d_init) {
      p.d_init[e * p.D + d] = carry;
    }
  }
  if (FOLD) return;
  __syncthreads();
  s_a[0][w][lane] = d_rate;
  __syncthreads();
  if (w == 0 && col_ok) {
    float sum = 0.0f;
    for (int u = 0; u < W; ++u) sum += s_a[0][u][lane];
    (p.rate_part ? p.rate_part : p.d_rate)[(group * nseg + seg) * p.D + d] = sum;
  }
}

template <class F, int W>
static hipError_t backward_waves(const Args& a, hipStream_t st) {
  const int64_t tiles = (a.D + 63) / 64;
  hipError_t e = hipSuccess;
  if (a.nseg > 1) {
    backward_kernel<F, W, true><<<dim3((unsigned)(a.groups * (a.nseg - 1) * tiles)), 64 * W, 0, st>>>(a, tiles);
    e = hipGetLastError();
    if (e != hipSuccess) return e;
  }
  backward_kernel<F, W, false><<<dim3((unsigned)(a.groups * a.nseg * tiles)), 64 * W, 0, st>>>(a, tiles);
  e = hipGetLastError();
  if (e != hipSuccess || !a.rate_part) return e;
  return sums::launch_columns(a.rate_part, a.groups * a.nseg, a.d_rate, a.D, nullptr, 0, st);
}

template <class F>
static hipError_t backward_fmt(const Args& a, const Plan& p, hipStream_t st) {
  switch (p.waves) {
    case 1: return backward_waves<F, 1>(a, st);
    case 4: return backward_waves<F, 4>(a, st);
    default: return backward_waves<F, 8>(a, st);
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
