// Gradients of linear attention (rlscan_linear_attention_backward).
//
// With dS the gradient of the state leaving a chunk and S the state entering it,
// a chunk's gradients need nothing else from the rest of the row:
//   dP_ij = scale exp(b_i - b_j) (do_i . v_j)
//   dq_i  = sum_j dP_ij k_j + entry_i S do_i
//   dk_j  = sum_i dP_ij q_i + leave_j dS v_j
//   dv_j  = sum_i P_ij do_i + leave_j dS^T k_j
// and for the log-decay of step t, every product of decays that holds a_t:
//   dg_t  = sum_{j<t<=i} (q_i . k_j) dP_ij + sum_{i>=t} X_i + sum_{j<t} Y_j + across <S, dS>,
//   X_i   = q_i . (entry_i S do_i),  Y_j = k_j . (leave_j dS v_j).
// The textbook running sum of q.dq - k.dk over the rest of the row gives the same
// number, but cancels over the row's length; this form only ever sums over one chunk.
//
// walk_kernel first leaves S and dS of every chunk in the workspace (both
// directions), then every chunk runs by itself: one block per row, key/value head and chunk, which
// adds up dk and dv over the heads of the group in registers, in a fixed order.
#include "rlscan_la_walk.hpp"
#include "rlscan_la_launch.hpp"

namespace rlscan {
namespace la {

template <class F, int KP, int VP, int C>
struct BackwardLds {
  Tile<F::NT, C, KP> q, k;
  Tile<F::NT, C, VP> v, dout;
  Tile<F::NP, C, C> p, dp;    // row i, column j
  Decay<C> dec;
  float row[C / 16][C];       // sum over the j of one tile of pair_ij, j < i
  float column[C / 16][C];    // sum over the i of one tile of pair_ij
  float x[kWaves][C];         // parts of X and Y
  float y[kWaves][C];
  float z[kWaves];            // parts of <S, dS>
};

__device__ __forceinline__ float sum_groups(float x) {  // over the 4 lane groups of a column
  x += __shfl_xor(x, 16);
  x += __shfl_xor(x, 32);
  return x;
}

__device__ __forceinline__ float sum_columns(float x) {  // over the 16 lanes of a group
#pragma unroll
  for (int o = 1; o < 16; o <<= 1) x += __shfl_xor(x, o);
  return x;
}

// 8 consecutive floats.
__device__ __forceinline__ void load8(const float* p, float (&x)[8]) {
  const f32x4 a = *reinterpret_cast<const f32x4*>(p);
  const f32x4 b = *reinterpret_cast<const f32x4*>(p + 4);
#pragma unroll
  for (int s = 0; s < 4; ++s) {
    x[s] = a[s];
    x[4 + s] = b[s];
  }
}

// Four consecutive columns of an LDS row, as floats.
template <int N, int R, int D>
__device__ __forceinline__ void get4(const Tile<N, R, D>& t, int row, int col, float (&x)[4]) {
  const int o = row * Tile<N, R, D>::LD + col;
#pragma unroll
  for (int r = 0; r < 4; ++r) x[r] = 0.0f;
#pragma unroll
  for (int n = N - 1; n >= 0; --n) {
    const bf16x4 w = *reinterpret_cast<const bf16x4*>(&t.p[n][o]);
#pragma unroll
    for (int r = 0; r < 4; ++r) x[r] += (float)w[r];
  }
}

template <class F, int KP, int VP, int C>
__global__ void __launch_bounds__(kThreads) backward_kernel(const Args a) {
  constexpr int NT = F::NT, NP = F::NP, NW = F::NW, CT = C / 16, CC = C / 32;
  constexpr int KW = (KP / 16 + kWaves - 1) / kWaves, VW = (VP / 16 + kWaves - 1) / kWaves;
  constexpr bool kWhole = C == 64;  // a wave has a whole row of P tiles, or one tile of four
  __shared__ BackwardLds<F, KP, VP, C> s;
  const int tid = threadIdx.x, lane = tid & 63, w = tid >> 6, col = lane & 15, grp = lane >> 4;
  const int64_t Hkv = a.H / a.G;
  const int64_t ehk = blockIdx.x / a.chunks, c = blockIdx.x % a.chunks;
  const int64_t e = ehk / Hkv, hk = ehk % Hkv;
  const int64_t t0 = c * C;
  using El = typename F::E;

  {
    Piece<F> rk[Share<C, KP>::n], rv[Share<C, VP>::n];
    fetch<F, C, KP>(a.k, e, hk, t0, a.T, 0, a.K, tid, rk);
    fetch<F, C, VP>(a.v, e, hk, t0, a.T, 0, a.V, tid, rv);
    stage<F, C, KP>(s.k, rk, tid);
    stage<F, C, VP>(s.v, rv, tid);
  }
  f32x4 dk[KW][CT], dv[VW][CT];
#pragma unroll
  for (int n = 0; n < KW; ++n)
#pragma unroll
    for (int jt = 0; jt < CT; ++jt) dk[n][jt] = f32x4{0, 0, 0, 0};
#pragma unroll
  for (int n = 0; n < VW; ++n)
#pragma unroll
    for (int jt = 0; jt < CT; ++jt) dv[n][jt] = f32x4{0, 0, 0, 0};

  for (int64_t u = 0; u < a.G; ++u) {
    const int64_t h = hk * a.G + u, eh = e * a.H + h;
    {
      Piece<F> rq[Share<C, KP>::n], rd[Share<C, VP>::n];
      fetch<F, C, KP>(a.q, e, h, t0, a.T, 0, a.K, tid, rq);
      fetch<F, C, VP>(a.dout, e, h, t0, a.T, 0, a.V, tid, rd);
      stage<F, C, KP>(s.q, rq, tid);
      stage<F, C, VP>(s.dout, rd, tid);
    }
    if (w == 0) fill_decay<C>(s.dec, load_decay<C>(a, e, h, t0, lane), a.scale, lane);
    __syncthreads();

    // ---- P, dP and their part of dg, as transposed tiles (rows j, columns i)
    {
      const int it = kWhole ? w : w >> 1;
      const int i = it * 16 + col;
      const float hi_i = s.dec.hi[i], lo_i = s.dec.lo[i];
      const int seg_i = s.dec.seg[i];
#pragma unroll
      for (int m = 0; m < (kWhole ? CT : 1); ++m) {
        const int jt = kWhole ? m : w & 1;
        float p[4] = {0, 0, 0, 0}, dp[4] = {0, 0, 0, 0}, pair[4] = {0, 0, 0, 0};
        if (jt <= it) {
          f32x4 qk{0, 0, 0, 0}, dov{0, 0, 0, 0};
#pragma unroll
          for (int kk = 0; kk < KP / 32; ++kk)
            qk = mma(frag_row<NT, C, KP>(s.k, jt * 16, kk, lane), frag_row<NT, C, KP>(s.q, it * 16, kk, lane), qk);
#pragma unroll
          for (int vv = 0; vv < VP / 32; ++vv)
            dov = mma(frag_row<NT, C, VP>(s.v, jt * 16, vv, lane), frag_row<NT, C, VP>(s.dout, it * 16, vv, lane), dov);
#pragma unroll
          for (int r = 0; r < 4; ++r) {
            const int j = jt * 16 + grp * 4 + r;
            const float d = a.scale * between<C>(s.dec, hi_i, lo_i, seg_i, i, j);
            p[r] = qk[r] * d;
            dp[r] = dov[r] * d;
            pair[r] = j < i ? qk[r] * dp[r] : 0.0f;
          }
        }
        put4<NP, C, C>(s.p, i, jt * 16 + grp * 4, p);
        put4<NP, C, C>(s.dp, i, jt * 16 + grp * 4, dp);
        const float row = sum_groups((pair[0] + pair[1]) + (pair[2] + pair[3]));
        if (grp == 0) s.row[jt][i] = row;
#pragma unroll
        for (int r = 0; r < 4; ++r) {
          const float column = sum_columns(pair[r]);
          if (col == 0) s.column[it][jt * 16 + grp * 4 + r] = column;
        }
      }
    }
    __syncthreads();

    const float* S = a.states + (eh * a.chunks + c) * (int64_t)(KP * VP);
    const float* dS = a.grads + (eh * a.chunks + c) * (int64_t)(KP * VP);

    // ---- dq and dk: wave w has the tiles w, w + 4 of K.  Transposed: rows k, columns i or j
    float xs[CT], ys[CT], z = 0.0f;
#pragma unroll
    for (int n = 0; n < CT; ++n) xs[n] = ys[n] = 0.0f;
#pragma unroll
    for (int n = 0; n < KW; ++n) {
      const int kt = n * kWaves + w;
      if (kt >= KP / 16) break;
      f32x4 dq[CT], in[CT];
#pragma unroll
      for (int it = 0; it < CT; ++it) dq[it] = in[it] = f32x4{0, 0, 0, 0};
#pragma unroll
      for (int vv = 0; vv < VP / 32; ++vv) {
        float x[8], y[8];
        load8(S + (kt * 16 + col) * VP + vv * 32 + grp * 8, x);
        load8(dS + (kt * 16 + col) * VP + vv * 32 + grp * 8, y);
#pragma unroll
        for (int i = 0; i < 8; ++i) z += x[i] * y[i];
        const Frag<NW> fs = split<NW>(x), fd = split<NW>(y);
#pragma unroll
        for (int it = 0; it < CT; ++it) {
          dq[it] = mma(fs, frag_row<NT, C, VP>(s.dout, it * 16, vv, lane), dq[it]);
          in[it] = mma(fd, frag_row<NT, C, VP>(s.v, it * 16, vv, lane), in[it]);
        }
      }
#pragma unroll
      for (int it = 0; it < CT; ++it) {
        const int row = it * 16 + col;
        float q[4], k[4];
        get4<NT, C, KP>(s.q, row, kt * 16 + grp * 4, q);
        get4<NT, C, KP>(s.k, row, kt * 16 + grp * 4, k);
        dq[it] *= s.dec.entry[row];
        in[it] *= s.dec.leave[row];
#pragma unroll
        for (int r = 0; r < 4; ++r) {
          xs[it] += q[r] * dq[it][r];
          ys[it] += k[r] * in[it][r];
        }
        dk[n][it] += in[it];
      }
#pragma unroll
      for (int jj = 0; jj < CC; ++jj) {
        const Frag<NT> fk = frag_col<NT, C, KP>(s.k, kt * 16, jj, lane);
        const Frag<NT> fq = frag_col<NT, C, KP>(s.q, kt * 16, jj, lane);
#pragma unroll
        for (int it = 0; it < CT; ++it) {
          if (jj <= it / 2) dq[it] = mma(fk, frag_row<NP, C, C>(s.dp, it * 16, jj, lane), dq[it]);
          if (jj >= it / 2) dk[n][it] = mma(fq, frag_col<NP, C, C>(s.dp, it * 16, jj, lane), dk[n][it]);
        }
      }
#pragma unroll
      for (int it = 0; it < CT; ++it) {
        const int64_t t = t0 + it * 16 + col;
        if (t < a.T) {
          const float x[4] = {dq[it][0], dq[it][1], dq[it][2], dq[it][3]};
          store4<F>(static_cast<El*>(const_cast<void*>(a.dq.p)) + e * a.dq.se + h * a.dq.sh + t * a.dq.st,
                    kt * 16 + grp * 4, a.K, a.dq.vec, x);
        }
      }
    }
#pragma unroll
    for (int it = 0; it < CT; ++it) {
      xs[it] = sum_groups(xs[it]);
      ys[it] = sum_groups(ys[it]);
      if (grp == 0) {
        s.x[w][it * 16 + col] = xs[it];
        s.y[w][it * 16 + col] = ys[it];
      }
    }
    z = sum_columns(sum_groups(z));
    if (lane == 0) s.z[w] = z;

    // ---- dv: wave w has the tiles w, w + 4 of V.  Transposed: rows v, columns j
#pragma unroll
    for (int n = 0; n < VW; ++n) {
      const int vt = n * kWaves + w;
      if (vt >= VP / 16) break;
      f32x4 in[CT];
#pragma unroll
      for (int jt = 0; jt < CT; ++jt) in[jt] = f32x4{0, 0, 0, 0};
#pragma unroll
      for (int kk = 0; kk < KP / 32; ++kk) {
        float y[8];
#pragma unroll
        for (int i = 0; i < 8; ++i) y[i] = dS[(kk * 32 + grp * 8 + i) * VP + vt * 16 + col];
        const Frag<NP> fd = split<NP>(y);  // feeds dv alone: that output's precision
#pragma unroll
        for (int jt = 0; jt < CT; ++jt) in[jt] = mma(fd, frag_row<NT, C, KP>(s.k, jt * 16, kk, lane), in[jt]);
      }
#pragma unroll
      for (int jt = 0; jt < CT; ++jt) {
        const float leave = s.dec.leave[jt * 16 + col];
        dv[n][jt] += in[jt] * leave;
      }
#pragma unroll
      for (int ii = 0; ii < CC; ++ii) {
        const Frag<NT> fo = frag_col<NT, C, VP>(s.dout, vt * 16, ii, lane);
#pragma unroll
        for (int jt = 0; jt < CT; ++jt)
          if (ii >= jt / 2) dv[n][jt] = mma(fo, frag_col<NP, C, C>(s.p, jt * 16, ii, lane), dv[n][jt]);
      }
    }
    __syncthreads();

    // ---- dg: the first wave adds up the chunk's parts, in float64
    if (w == 0) {
      double back = 0.0, y = 0.0;  // summed over i >= t, and over j < t
      if (lane < C) {
#pragma unroll
        for (int n = 0; n < CT; ++n) back += (double)s.row[n][lane] - (double)s.column[n][lane];
#pragma unroll
        for (int n = 0; n < kWaves; ++n) {
          if (n < KP / 16) {
            back += (double)s.x[n][lane];
            y += (double)s.y[n][lane];
          }
        }
      }
      const double own = y;
#pragma unroll
      for (int o = 1; o < 64; o <<= 1) {
        const double b = __shfl_down(back, o), f = __shfl_up(y, o);
        if (lane + o < 64) back += b;
        if (lane >= o) y += f;
      }
      double zz = 0.0;
#pragma unroll
      for (int n = 0; n < kWaves; ++n) zz += (double)s.z[n];
      const double g = back + (y - own) + (double)s.dec.across * zz;
      const int64_t t = t0 + lane;
      if (lane < C && t < a.T)
        a.dg[e * a.dg_se + t * a.dg_st + h * a.dg_sh] = (s.dec.cuts >> lane & 1) ? 0.0f : (float)g;
    }
    __syncthreads();
  }

#pragma unroll
  for (int n = 0; n < KW; ++n) {
    const int kt = n * kWaves + w;
    if (kt >= KP / 16) break;
#pragma unroll
    for (int jt = 0; jt < CT; ++jt) {
      const int64_t t = t0 + jt * 16 + col;
      if (t >= a.T) continue;
      const float x[4] = {dk[n][jt][0], dk[n][jt][1], dk[n][jt][2], dk[n][jt][3]};
      store4<F>(static_cast<El*>(const_cast<void*>(a.dk.p)) + e * a.dk.se + hk * a.dk.sh + t * a.dk.st,
                kt * 16 + grp * 4, a.K, a.dk.vec, x);
    }
  }
#pragma unroll
  for (int n = 0; n < VW; ++n) {
    const int vt = n * kWaves + w;
    if (vt >= VP / 16) break;
#pragma unroll
    for (int jt = 0; jt < CT; ++jt) {
      const int64_t t = t0 + jt * 16 + col;
      if (t >= a.T) continue;
      const float x[4] = {dv[n][jt][0], dv[n][jt][1], dv[n][jt][2], dv[n][jt][3]};
      store4<F>(static_cast<El*>(const_cast<void*>(a.dv.p)) + e * a.dv.se + hk * a.dv.sh + t * a.dv.st,
                vt * 16 + grp * 4, a.V, a.dv.vec, x);
    }
  }
}

// The gradient of one log-decay for each head: the sum over rows and steps, in
// float64 and in a fixed order.
__global__ void __launch_bounds__(256) head_sum_kernel(const float* dg, float* out, int64_t rows, int64_t H) {
  __shared__ double part[256];
  const int64_t h = blockIdx.x;
  double x = 0.0;
  for (int64_t i = threadIdx.x; i < rows; i += 256) x += (double)dg[i * H + h];
  part[threadIdx.x] = x;
  __syncthreads();
  for (int o = 128; o > 0; o >>= 1) {
    if ((int)threadIdx.x < o) part[threadIdx.x] += part[threadIdx.x + o];
    __syncthreads();
  }
  if (threadIdx.x == 0) out[h] = (float)part[0];
}

template <class F, int KP, int C, bool REV>
void walk(const Args& a, const Plan& pl, hipStream_t st) {
  const int64_t heads = a.E * a.H * (pl.VP / 64);
  if (heads == 0) return;
  WalkArgs w{};
  w.a = a;
  w.VP = pl.VP;
  float* seg = REV ? a.seg_grad : a.seg_state;
  float* decay = REV ? a.seg_gdecay : a.seg_decay;
  const float* given = REV ? a.d_final : a.init;
  if (pl.nseg > 1) {
    w.seg_end = seg;
    w.seg_decay = decay;
    walk_kernel<F, KP, C, REV><<<dim3((unsigned)(heads * pl.nseg)), kThreads, 0, st>>>(w);
    CombineArgs c{};
    c.seg = seg;
    c.decay = decay;
    c.given = given;
    c.done = a.done;
    c.d_se = a.d_se;
    c.d_st = a.d_st;
    c.H = a.H;
    c.T = a.T;
    c.nseg = pl.nseg;
    c.KP = KP;
    c.VP = pl.VP;
    c.K = a.K;
    c.V = a.V;
    c.closed = REV;
    combine_kernel<<<dim3((unsigned)(a.E * a.H * ((KP * pl.VP + 255) / 256))), 256, 0, st>>>(c);
    w.seg_end = nullptr;
    w.seg_decay = nullptr;
    w.enter = seg;
  }
  w.given = given;
  w.each = REV ? a.grads : a.states;
  w.end = REV ? a.d_init : nullptr;
  walk_kernel<F, KP, C, REV><<<dim3((unsigned)(heads * pl.nseg)), kThreads, 0, st>>>(w);
}

template <class F, int KP, int C>
hipError_t launch_backward_as(Args a, const Plan& pl, float* dg_head, hipStream_t st) {
  walk<F, KP, C, false>(a, pl, st);
  walk<F, KP, C, true>(a, pl, st);
  const int64_t blocks = a.E * (a.H / a.G) * a.chunks;
  if (blocks > 0) {
    if (pl.VP == 64) backward_kernel<F, KP, 64, C><<<dim3((unsigned)blocks), kThreads, 0, st>>>(a);
    else backward_kernel<F, KP, 128, C><<<dim3((unsigned)blocks), kThreads, 0, st>>>(a);
  }
  if (dg_head && a.H > 0) head_sum_kernel<<<dim3((unsigned)a.H), 256, 0, st>>>(a.dg, dg_head, a.E * a.T, a.H);
  return hipGetLastError();
}

template <class F, int C>
hipError_t launch_backward_fmt(const Args& a, const Plan& pl, float* dg_head, hipStream_t st) {
  return pl.KP == 64 ? launch_backward_as<F, 64, C>(a, pl, dg_head, st) : launch_backward_as<F, 128, C>(a, pl, dg_head, st);
}

hipError_t launch_backward(rlscan_format f, const Args& a, const Plan& pl, float* dg_head, hipStream_t st) {
  switch (f) {
    case RLSCAN_FORMAT_BF16: return launch_backward_fmt<TBf16, 64>(a, pl, dg_head, st);
    case RLSCAN_FORMAT_F16: return launch_backward_fmt<TF16, 32>(a, pl, dg_head, st);
    default: return launch_backward_fmt<TF32, 32>(a, pl, dg_head, st);
  }
}

}  // namespace la
}  // namespace rlscan
