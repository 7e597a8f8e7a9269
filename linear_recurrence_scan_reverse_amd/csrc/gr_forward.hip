// The gated recurrence over whole rows (rlscan_gated_recurrence).
#include "rlscan_gr.hpp"

namespace rlscan {
namespace gr {

// One block: 64 channels of one row (or of one segment of it), W waves of kMark steps each
// at a time.  FOLD: the pair of the segment alone, for the blocks that follow it.
template <class F, int W, bool FOLD>
__global__ void __launch_bounds__(64 * W) forward_kernel(const Args p, int64_t tiles) {
  using E = typename F::E;
  constexpr int S = kMark;
  __shared__ float s_a[2][W][64], s_y[2][W][64];
  const int lane = threadIdx.x & 63;
  const int w = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int64_t nseg = FOLD ? p.nseg - 1 : p.nseg;  // nothing follows the last segment
  const int64_t tile = blockIdx.x % tiles, es = blockIdx.x / tiles, seg = es % nseg, e = es / nseg;
  const int64_t d = tile * 64 + lane;
  const bool col_ok = d < p.D;
  const int64_t dc = col_ok ? d : p.D - 1;  // loads stay inside the row
  const float rate = p.rate[dc];
  const E* px = static_cast<const E*>(p.x.p) + e * p.x.se + dc;
  const E* pi = static_cast<const E*>(p.ig.p) + e * p.ig.se + dc;
  const E* pr = static_cast<const E*>(p.dg.p) + e * p.dg.se + dc;
  E* po = FOLD ? nullptr : static_cast<E*>(const_cast<void*>(p.out.p)) + e * p.out.se + d;
  const uint8_t* done = p.done ? p.done + e * p.d_se : nullptr;
  const int64_t begin = seg * p.seg_steps;
  const int64_t end = p.T < begin + p.seg_steps ? p.T : begin + p.seg_steps;

  float carry = 0.0f;  // the state entering the super-tile
  if (!FOLD) {
    if (p.init) carry = p.init[e * p.D + dc];
    for (int64_t u = 0; u < seg; ++u) {
      const int64_t at = (e * p.nseg + u) * p.D + dc;
      carry = enter(p.seg_a[at], p.seg_y[at], carry);
    }
  }
  float total = 0.0f;   // FOLD: sum of s over the segment
  bool dropped = false;
  int buf = 0;
  for (int64_t t0 = begin; t0 < end; t0 += W * S) {
    const int64_t c0 = t0 + w * S;
    E x[S], gi[S], gd[S];
#pragma unroll
    for (int k = 0; k < S; ++k) {
      const int64_t t = c0 + k < end ? c0 + k : end - 1;
      x[k] = px[t * p.x.st];
      gi[k] = pi[t * p.ig.st];
      gd[k] = pr[t * p.dg.st];
    }
    bool dn = false;  // lane k: whether step c0 + k starts anew
    if (done && lane < S) {
      const int64_t t = c0 + lane;
      if (t > 0 && t < end) dn = done[(t - 1) * p.d_st] != 0;
    }
    const uint32_t cut = (uint32_t)__builtin_amdgcn_ballot_w64(dn);
    float em1[S], b[S], L = 0.0f, y = 0.0f;
#pragma unroll
    for (int k = 0; k < S; ++k) {
      const bool live = c0 + k < end, fresh = (cut >> k) & 1;
      const float s = rate * sigmoid(F::get(gd[k]));
      em1[k] = fresh ? -1.0f : decay_less_1(s);
      b[k] = __builtin_amdgcn_sqrtf(one_less_square(em1[k])) * (sigmoid(F::get(gi[k])) * F::get(x[k]));
      if (!live) em1[k] = b[k] = 0.0f;
      L += live ? s : 0.0f;
      y = decayed(em1[k], fresh ? 0.0f : y) + b[k];
    }
    const float A = cut ? kDropped : exp2_fast(-kLog2E * L);
    s_a[buf][w][lane] = A;
    s_y[buf][w][lane] = y;
    __syncthreads();
    float h = carry;  // the state entering this wave's chunk
    for (int u = 0; u < w; ++u) h = enter(s_a[buf][u][lane], s_y[buf][u][lane], h);
    float next = h;
    for (int u = w; u < W; ++u) next = enter(s_a[buf][u][lane], s_y[buf][u][lane], next);
    carry = next;
    buf ^= 1;
    if (FOLD) {
      total += L;
      dropped |= cut != 0;
      continue;
    }
    if (p.marks && col_ok && c0 < end) p.marks[(e * ((p.T + S - 1) / S) + c0 / S) * p.D + d] = h;
#pragma unroll
    for (int k = 0; k < S; ++k) {
      h = decayed(em1[k], (cut >> k) & 1 ? 0.0f : h) + b[k];
      if (col_ok && c0 + k < end) po[(c0 + k) * p.out.st] = F::put(h);
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
  } else if (w == 0 && col_ok && seg == nseg - 1 && p.final_state) {
    const bool ended = done && p.T > 0 && done[(p.T - 1) * p.d_st] != 0;
    p.final_state[e * p.D + d] = ended ? 0.0f : carry;
  }
}

template <class F, int W>
static hipError_t forward_waves(const Args& a, hipStream_t st) {
  const int64_t tiles = (a.D + 63) / 64;
  if (a.nseg > 1) {
    forward_kernel<F, W, true><<<dim3((unsigned)(a.E * (a.nseg - 1) * tiles)), 64 * W, 0, st>>>(a, tiles);
    const hipError_t e = hipGetLastError();
    if (e != hipSuccess) return e;
  }
  forward_kernel<F, W, false><<<dim3((unsigned)(a.E * a.nseg * tiles)), 64 * W, 0, st>>>(a, tiles);
  return hipGetLastError();
}

template <class F>
static hipError_t forward_fmt(const Args& a, const Plan& p, hipStream_t st) {
  switch (p.waves) {
    case 1: return forward_waves<F, 1>(a, st);
    case 4: return forward_waves<F, 4>(a, st);
    default: return forward_waves<F, 16>(a, st);
  }
}

hipError_t launch_forward(rlscan_format f, const Args& a, const Plan& p, hipStream_t st) {
  switch (f) {
    case RLSCAN_FORMAT_BF16: return forward_fmt<LBf16>(a, p, st);
    case RLSCAN_FORMAT_F16: return forward_fmt<LF16>(a, p, st);
    default: return forward_fmt<LF32>(a, p, st);
  }
}

// Waves of a block and segments of a row.
Plan make_plan(rlscan_format, int64_t E, int64_t T, int64_t D, bool backward) {
  Plan p{};
  const int64_t tiles = E * ((D + 63) / 64);
  p.waves = T <= kMark || tiles >= 4096 ? 1 : T <= 4 * kMark || tiles >= 1024 ? 4 : 16;
  if (backward && p.waves == 16) p.waves = 8;
  const int64_t unit = (int64_t)p.waves * kMark, units = (T + unit - 1) / unit;
  int64_t want = tiles > 0 && tiles < 512 ? (512 + tiles - 1) / tiles : 1;
  if (want > units / 4) want = units / 4;  // a segment costs one more pass over its inputs
  if (want < 1) want = 1;
  const int64_t per = units > 0 ? (units + want - 1) / want : 1;
  p.seg_steps = per * unit;
  p.nseg = units > 0 ? (units + per - 1) / per : 1;
  p.seg = p.nseg > 1 ? (E * p.nseg * D + 3) / 4 * 4 : 0;
  p.groups = E;
  if (backward) {
    const int64_t columns = (D + 63) / 64, most = 8192 / (columns * p.nseg) + 1;
    if (p.groups > most) p.groups = most;
    p.part = p.groups * p.nseg > 1 ? (p.groups * p.nseg * D + 3) / 4 * 4 : 0;
  }
  p.floats = 2 * p.seg + p.part;
  return p;
}

}  // namespace gr
}  // namespace rlscan
