// Gradients of linear attention (rlscan_linear_attention_backward).
//
// dq, dk and dv are each a chunk walk of their own (rlscan_la_attend.hpp) with the state or
// its gradient in registers; the three run side by side in one launch, the blocks of one
// head next to each other on one XCD, whose L2 they share.  The log-decay's gradient follows from
// b_t, the running sum of g up to t: every product of decays is exp(b_i - b_j), so
//   dL/db_i = q_i . dq_i - k_i . dk_i  (without the i = j terms, which hold no decay),
//   dg_t    = sum of dL/db_i over the i >= t of t's episode, plus <S, dS> behind the last one
//             (of both, the part of k and v at T-1 holds no decay and is left out).
// Both dot products are taken from the float32 sums before dq and dk are rounded, from
// operands of float32 precision, in float64: their differences are small against them.
// So that their rounding does not add up over a row, some boundaries between chunks are
// marked: there the walks leave S and dS, and the sum starts anew from dg = <S, dS>.
//
// Measured (kernels in a run of 300 calls): 8 rows of 4096 steps, 16 heads of 128 in bfloat16,
// gates for each step: 981 us for the three walks, 24 for the marked boundaries and 18 for the
// sums of dg; 944 MB and 103 Gflop, 180 us of a copy.  A block takes 87,872 bytes of LDS, so a
// compute unit holds one: 128 heads times three walks are 384 blocks on 256 places, two rounds
// of which the second is half empty.  Within a block the chain of products is what takes time:
// dq and dk carry two terms for intermediates and three for the float32 sums that dg needs,
// 3 to 6 matrix instructions where an output in bfloat16 alone would need one.  The 128-wide
// walks without care need 203 (float16) to 253 registers and spill none, those with care 81 to 254;
// where rows cannot be read 16 bytes at a time 0 to 45 and 91 to 388.  64 rows of 333 steps, 4 heads
// of 64 in float32, keys and values shared by two: 120 us for the walks (245 registers, two blocks
// on a compute unit: 768 blocks on 512 places), 24 to add up the shared heads' gradients, 19 for dg.
#include "rlscan_la_attend.hpp"
#include "rlscan_la_launch.hpp"
#include "rlscan_la_walk.hpp"

namespace rlscan {
namespace la {

template <class F, int KP, int VP, int C, int NWV>
struct BackwardLds {
  union {
    AttendLds<F, VP, KP, C, NWV, true> k;   // dq and dk
    AttendLds<F, KP, VP, C, NWV, false> v;  // dv
  };
};

struct BackwardArgs {
  Args a;
  Attend q, k, v;
};

// FO: the format that dk and dv are left in (float32 scratch where heads share them).
template <class F, class FO, int KP, int VP, int C, int NWV, int MINW, bool VEC>
__global__ void __launch_bounds__(64 * NWV, MINW) backward_kernel(const BackwardArgs p) {
  __shared__ char lds[sizeof(BackwardLds<F, KP, VP, C, NWV>)] __attribute__((aligned(16)));
  auto& s = *reinterpret_cast<BackwardLds<F, KP, VP, C, NWV>*>(lds);
  const Args& a = p.a;
  const int64_t items = a.E * a.H * a.nseg;
  const int64_t item = blockIdx.x / 24 * 8 + blockIdx.x % 8;
  if (item >= items) return;
  const int64_t eh = item % (a.E * a.H), seg = item / (a.E * a.H);
  switch (blockIdx.x % 24 / 8) {
    case 0: attend<F, F, VP, KP, C, NWV, false, true, F::NW, VEC>(s.k, p, &BackwardArgs::q, eh, seg, 0); break;
    case 1: attend<F, FO, VP, KP, C, NWV, true, true, F::NW, VEC>(s.k, p, &BackwardArgs::k, eh, seg, 0); break;
    default: attend<F, FO, KP, VP, C, NWV, true, false, F::NP, VEC>(s.v, p, &BackwardArgs::v, eh, seg, 0); break;
  }
}

// dg of one row and head: x_t = u_t - w_t summed from the end, afresh at each episode's last step.
// A thread takes four steps; the sums of those behind it pass through the wave and the block.
// Rows past 1024 steps take blocks of 1024 threads: a tile's chain of sums and trips to
// memory is paid once for 4096 steps.  256 threads against 1024, us, rows of 1100, 2048, 4096 and 8192
// steps: one head 7.7, 7.9, 14.2, 26.9 and 6.1, 6.6, 7.2, 13.1; 128 heads 10.6, 13.0, 22.7, 44.9
// and 9.0, 11.2, 16.9, 32.2.  1024 heads fill the card by themselves: 29, 43, 96 (4096) and 34, 49, 90.
template <int NTHR>
__global__ void __launch_bounds__(NTHR) decay_grad_kernel(const Args a, const double* u, const double* w,
                                                          const float* end, const double* mark_dots, int64_t nmarks,
                                                          int64_t mark_steps, double* total) {
  constexpr int kWaves = NTHR / 64;
  __shared__ double sum[kWaves];
  __shared__ int open[kWaves];
  const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
  const int64_t eh = blockIdx.x, e = eh / a.H, h = eh % a.H;
  u += eh * a.T;
  w += eh * a.T;
  mark_dots += eh * nmarks;
  double carry = (double)end[eh];  // what comes from behind the tile
  double all = 0.0;
  const int64_t tiles = (a.T + NTHR * 4 - 1) / (NTHR * 4);
  for (int64_t n = tiles - 1; n >= 0; --n) {
    const int64_t t0 = n * (NTHR * 4) + (int64_t)(NTHR - 1 - tid) * 4;  // later steps in earlier lanes
    // this thread's steps from the last: R = x_t + (step t+1 starts afresh ? 0 : R)
    double x[4];
    bool cut[4];  // step t starts afresh: its own gradient is 0 and nothing passes to t-1
    bool mark[4];
    double anew[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const int64_t t = t0 + i;
      x[i] = t < a.T ? u[t] - (t < a.T - 1 ? w[t] : 0.0) : 0.0;
      cut[i] = false;
      mark[i] = t > 0 && t < a.T && t % mark_steps == 0;
      anew[i] = mark[i] ? mark_dots[t / mark_steps - 1] : 0.0;
      if (t < a.T)
        cut[i] = a.g[e * a.g_se + t * a.g_st + h * a.g_sh] < kCutBelow ||
                 (t > 0 && a.done && a.done[e * a.d_se + (t - 1) * a.d_st] != 0);
    }
    double own = 0.0;  // sum that leaves towards t0 - 1
    bool passes = true;
#pragma unroll
    for (int i = 3; i >= 0; --i) {
      own = mark[i] ? anew[i] : own + x[i];
      if (cut[i]) own = 0.0;
      passes &= !(cut[i] || mark[i]);
    }
    // inclusive over lanes: (own, passes) of this lane and those before it (later steps)
    double run = own;
    int through = passes;
#pragma unroll
    for (int o = 1; o < 64; o <<= 1) {
      const double b = __shfl_up(run, o);
      const int p = __shfl_up(through, o);
      if (lane >= o) {
        run += through ? b : 0.0;
        through &= p;
      }
    }
    if (lane == 63) {
      sum[wave] = run;
      open[wave] = through;
    }
    __syncthreads();
    double in = carry;
    for (int i = 0; i < wave; ++i) in = sum[i] + (open[i] ? in : 0.0);
    const double before = __shfl_up(run, 1);
    const int before_through = __shfl_up(through, 1);
    double r = lane == 0 ? in : before + (before_through ? in : 0.0);
    for (int i = wave; i < kWaves; ++i) in = sum[i] + (open[i] ? in : 0.0);
    carry = in;
    __syncthreads();
#pragma unroll
    for (int i = 3; i >= 0; --i) {
      r = mark[i] ? anew[i] : r + x[i];
      const double g = cut[i] ? 0.0 : r;
      if (cut[i]) r = 0.0;
      const int64_t t = t0 + i;
      if (t < a.T) {
        all += g;
        if (!total) a.dg[e * a.dg_se + t * a.dg_st + h * a.dg_sh] = (float)g;
      }
    }
  }
  if (!total) return;
#pragma unroll
  for (int o = 1; o < 64; o <<= 1) all += __shfl_xor(all, o);
  if (lane == 0) sum[wave] = all;
  __syncthreads();
  if (tid == 0) {
    for (int i = 1; i < kWaves; ++i) all += sum[i];
    total[eh] = all;
  }
}

// <S, dS> at one marked boundary, in float64 and in a fixed order.
__global__ void __launch_bounds__(256) mark_dot_kernel(const float* s, const float* ds, double* out, int64_t n) {
  __shared__ double part[4];
  const int64_t base = (int64_t)blockIdx.x * n;
  double x = 0.0;
  for (int64_t i = threadIdx.x * 4; i < n; i += 1024) {
    const f32x4 p = *reinterpret_cast<const f32x4*>(s + base + i), q = *reinterpret_cast<const f32x4*>(ds + base + i);
#pragma unroll
    for (int k = 0; k < 4; ++k) x += (double)p[k] * (double)q[k];
  }
#pragma unroll
  for (int o = 1; o < 64; o <<= 1) x += __shfl_xor(x, o);
  if ((threadIdx.x & 63) == 0) part[threadIdx.x >> 6] = x;
  __syncthreads();
  if (threadIdx.x == 0) out[blockIdx.x] = (part[0] + part[1]) + (part[2] + part[3]);
}

// One log-decay for each head: its gradient is the sum over the rows.
__global__ void __launch_bounds__(64) head_sum_kernel(const double* total, float* out, int64_t E, int64_t H) {
  double x = 0.0;
  for (int64_t e = threadIdx.x; e < E; e += 64) x += total[e * H + blockIdx.x];
#pragma unroll
  for (int o = 1; o < 64; o <<= 1) x += __shfl_xor(x, o);
  if (threadIdx.x == 0) out[blockIdx.x] = (float)x;
}

// Adds up the heads of a group, in order: from [E, T, H, D] float32 to out's [E, T, H / G, D].
template <class F>
__global__ void __launch_bounds__(256) group_sum_kernel(const Args a, const float* from, const View out, int D) {
  const int64_t Hkv = a.H / a.G;
  const int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x;
  const int64_t d = i % D, hk = i / D % Hkv, et = i / D / Hkv;
  if (et >= a.E * a.T) return;
  const float* p = from + (et * a.H + hk * a.G) * D + d;
  float x = p[0];
  for (int64_t n = 1; n < a.G; ++n) x += p[n * D];
  const int64_t e = et / a.T, t = et % a.T;
  auto* to = static_cast<typename F::E*>(const_cast<void*>(out.p)) + e * out.se + t * out.st + hk * out.sh + d;
  if constexpr (sizeof(*to) == 4) *to = x;
  else if constexpr (F::NT == 1) *to = __builtin_bit_cast(uint16_t, (__bf16)x);
  else *to = __builtin_bit_cast(uint16_t, (_Float16)x);
}

template <class F, class FO, int KP, int VP, int C, int NWV, int MINW, bool VEC>
void launch_walks(const Args& a, const Backward& b, const Plan& pl, hipStream_t st) {
  enter_segments<F, KP, C, false, VEC>(a, VP, a.init, b.seg_state, b.seg_decay, st);
  enter_segments<F, KP, C, true, VEC>(a, VP, b.d_final, b.seg_grad, b.seg_gdecay, st);
  const int64_t kv = (int64_t)a.K * a.V, pad = KP * VP;
  // states as [K][V] in memory, and as the walks with v first take them
  auto rows_k = [&](const float* p) { return StateView{const_cast<float*>(p), kv, 0, a.V, 1}; };
  auto rows_v = [&](const float* p) { return StateView{const_cast<float*>(p), kv, 0, 1, a.V}; };
  Attend q{}, k{}, v{};
  q.a = a.dout;
  q.b = a.v;
  q.c = a.k;
  q.out = a.dq;
  q.ga = 1;
  q.gb = q.gc = a.G;
  q.A = a.V;
  q.D = a.K;
  q.m = a.q;
  q.gm = 1;
  q.dot = b.u;
  q.enter = pl.nseg > 1 ? StateView{b.seg_state, pl.nseg * pad, pad, 1, VP} : rows_v(a.init);
  q.end = rows_v(b.d_final);
  q.end_dot = b.end;
  q.marks = b.marks;
  q.nmarks = k.nmarks = b.nmarks;
  k.marks = b.mark_grads;
  k.a = a.v;
  k.b = a.dout;
  k.c = a.q;
  k.out = b.dk;
  k.ga = a.G;
  k.gb = k.gc = 1;
  k.A = a.V;
  k.D = a.K;
  k.m = a.k;
  k.gm = a.G;
  k.dot = b.w;
  k.enter = pl.nseg > 1 ? StateView{b.seg_grad, pl.nseg * pad, pad, 1, VP} : rows_v(b.d_final);
  k.enter_closed = pl.nseg == 1;  // segments have it from combine_kernel
  k.leave = rows_v(b.d_init);
  v.a = a.k;
  v.b = a.q;
  v.c = a.dout;
  v.out = b.dv;
  v.ga = a.G;
  v.gb = v.gc = 1;
  v.A = a.K;
  v.D = a.V;
  v.enter = pl.nseg > 1 ? StateView{b.seg_grad, pl.nseg * pad, pad, VP, 1} : rows_k(b.d_final);
  v.enter_closed = pl.nseg == 1;
  const int64_t items = a.E * a.H * pl.nseg;
  backward_kernel<F, FO, KP, VP, C, NWV, MINW, VEC><<<dim3((unsigned)((items + 7) / 8 * 24)), 64 * NWV, 0, st>>>(BackwardArgs{a, q, k, v});
}

template <class F, class FO, bool VEC>
void launch_sizes(const Args& a, const Backward& b, const Plan& pl, hipStream_t st) {
  if (pl.KP == 64) launch_walks<F, FO, 64, 64, 32, 4, 2, VEC>(a, b, pl, st);
  else launch_walks<F, FO, 128, 128, F::NT == 1 ? 64 : 32, 8, 2, VEC>(a, b, pl, st);
}

template <class F>
hipError_t launch_backward_fmt(const Args& a, const Backward& b, const Plan& pl, hipStream_t st) {
  if (a.E * a.H > 0) {
    const bool vec = a.q.vec && a.k.vec && a.v.vec && a.dout.vec && a.dq.vec && b.dk.vec && b.dv.vec;
    if (a.G > 1) {
      if (vec) launch_sizes<F, TF32, true>(a, b, pl, st);
      else launch_sizes<F, TF32, false>(a, b, pl, st);
    } else {
      if (vec) launch_sizes<F, F, true>(a, b, pl, st);
      else launch_sizes<F, F, false>(a, b, pl, st);
    }
    if (b.nmarks > 0)
      mark_dot_kernel<<<dim3((unsigned)(a.E * a.H * b.nmarks)), 256, 0, st>>>(b.marks, b.mark_grads, b.mark_dots, pl.KP * pl.VP);
    auto decay_grad = a.T > 1024 ? decay_grad_kernel<1024> : decay_grad_kernel<256>;
    decay_grad<<<dim3((unsigned)(a.E * a.H)), a.T > 1024 ? 1024 : 256, 0, st>>>(
        a, b.u, b.w, b.end, b.mark_dots, b.nmarks, a.mark_chunks * pl.C, b.dg_head ? b.total : nullptr);
    if (a.G > 1 && a.T > 0) {
      const int64_t rows = a.E * a.T * (a.H / a.G);
      group_sum_kernel<F><<<dim3((unsigned)((rows * a.K + 255) / 256)), 256, 0, st>>>(a, static_cast<const float*>(b.dk.p), a.dk, a.K);
      group_sum_kernel<F><<<dim3((unsigned)((rows * a.V + 255) / 256)), 256, 0, st>>>(a, static_cast<const float*>(b.dv.p), a.dv, a.V);
    }
  }
  if (b.dg_head) head_sum_kernel<<<dim3((unsigned)a.H), 64, 0, st>>>(b.total, b.dg_head, a.E, a.H);
  return hipGetLastError();
}

hipError_t launch_backward(rlscan_format f, const Args& a, const Backward& b, const Plan& pl, hipStream_t st) {
  switch (f) {
    case RLSCAN_FORMAT_BF16: return launch_backward_fmt<TBf16>(a, b, pl, st);
    case RLSCAN_FORMAT_F16: return launch_backward_fmt<TF16>(a, b, pl, st);
    default: return launch_backward_fmt<TF32>(a, b, pl, st);
  }
}

}  // namespace la
}  // namespace rlscan
