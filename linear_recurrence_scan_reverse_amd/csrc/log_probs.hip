// Log-probability of the taken action and entropy of every row of logits, and the
// gradient of both (rlscan_action_log_probs, rlscan_action_log_probs_backward).
//
// With z = x / temperature over the legal actions,
//   lse = m + log sum exp(z - m),  log_prob = z_a - lse,
//   entropy = log s - t / s,  s = sum e^(z-m), t = sum e^(z-m) (z-m),
//   dx_j = [d_lp (1[j = a] - p_j) - d_H p_j (log p_j + entropy)] / temperature.
// One read of the logits forward, one read and one write backward: both are bound
// by memory.  The forward pass keeps a running maximum with s and t relative to it
// in each thread (float32), joined over the block; few long rows are split over
// blocks, whose sums a second kernel joins.
//
// Measured: 4096 rows of 64007 bfloat16 logits: 140 us forward (3.7 TB/s) and 192 backward
// (5.4 TB/s).  16384 rows of 18 float32 logits with a mask: 5.5 us, 8 lanes
// for a row (rows up to 64 logits); a wave for each took 15.3.
#include "rlscan_logits.hpp"

namespace rlscan {
namespace logits {

constexpr float kLog2E = 1.44269504088896340736f;
constexpr double kLn2 = 0.693147180559945309417;

__device__ __forceinline__ float exp2_fast(float x) { return __builtin_amdgcn_exp2f(x); }

// z = x / temperature in float64, rounded by itself and never fused into what
// follows, so that the same x gives the same z in both directions and differences
// of equal ones are 0.
__device__ __forceinline__ double scaled(float x, double inv_t) {
#pragma clang fp contract(off)
  const double z = (double)x * inv_t;
  return z;
}

__device__ __forceinline__ double minus(double a, double b) {
#pragma clang fp contract(off)
  return a - b;
}

// m: the largest logit; n: how many have it; r = sum 2^y and t = sum 2^y y over the
// others, y = (x - m) c, c = log2 e / temperature.  Keeping the largest apart keeps the
// bits of r: a nearly certain action has log-probability -r and entropy near r, far
// below the rounding of 1 + r.
struct Sums {
  float m, n, r, t;
};

__device__ __forceinline__ Sums none() { return Sums{kNegInf, 0.0f, 0.0f, 0.0f}; }

// Moves a (with a.n != 0) to a larger maximum.
__device__ __forceinline__ void raise(Sums& a, float m, float c) {
  const float s = a.n + a.r;
  float d = (a.m - m) * c;
  d = d < -200.0f ? -200.0f : d;  // 2^-200 is 0 in float32; keeps 0 * inf out of t
  const float f = exp2_fast(d);
  a = Sums{m, 0.0f, f * s, f * (a.t + s * d)};
}

__device__ __forceinline__ Sums join(Sums a, Sums b, float c) {
  if (a.n == 0.0f && a.r == 0.0f) return b;  // nothing in it
  if (b.n == 0.0f && b.r == 0.0f) return a;
  if (a.m < b.m) raise(a, b.m, c);
  else if (b.m < a.m) raise(b, a.m, c);
  return Sums{a.m, a.n + b.n, a.r + b.r, a.t + b.t};
}

// Adds logits; -inf stands for one that is not legal.  A NaN makes r and t NaN.
template <int N>
__device__ __forceinline__ void add(Sums& a, const float (&x)[N], float c) {
  float top = a.m;  // fmaxf passes a NaN over; as a difference below it reaches r and t
#pragma unroll
  for (int i = 0; i < N; ++i) top = fmaxf(top, x[i]);
  if (top == kNegInf) {
#pragma unroll
    for (int i = 0; i < N; ++i)
      if (x[i] != x[i]) a = Sums{0.0f, 1.0f, x[i], x[i]};
    return;
  }
  if (top > a.m) {
    if (a.n != 0.0f) raise(a, top, c);
    a.m = top;
  }
#pragma unroll
  for (int i = 0; i < N; ++i) {
    float d = (x[i] - a.m) * c;
    d = d < -200.0f ? -200.0f : d;
    const float p = exp2_fast(d);
    const bool is_top = x[i] == a.m;
    a.n += is_top ? 1.0f : 0.0f;
    a.r += is_top ? 0.0f : p;
    a.t += p * d;
  }
}

__device__ __forceinline__ Sums shuffle(const Sums& a, int o) {
  return Sums{__shfl_xor(a.m, o), __shfl_xor(a.n, o), __shfl_xor(a.r, o), __shfl_xor(a.t, o)};
}

// The results of a row from its joined sums; a row without a legal action has
// log-probability 0 and entropy 0, and lse -inf.
template <class F>
__device__ __forceinline__ void finish(const LogProbArgs& p, int64_t r, const Sums& a) {
  const bool any = a.n != 0.0f || a.r != 0.0f;
  const double log_s = any ? log1p((double)(a.n - 1.0f) + (double)a.r) : 0.0;
  double lp = 0.0;
  const int64_t act = p.action[r];
  if (any && act >= 0 && act < p.N) {
    const bool legal = !p.mask || p.mask[r * p.N + act] != 0;
    const float x = F::get(static_cast<const typename F::E*>(p.x)[r * p.stride + act]);
    lp = legal ? ((double)x - (double)a.m) * p.inv_t - log_s : (double)kNegInf;
  }
  p.log_prob[r] = (float)lp;
  p.entropy[r] = any ? (float)(log_s - kLn2 * (double)a.t / ((double)a.n + (double)a.r)) : 0.0f;
  p.lse[r] = any ? minus(scaled(a.m, p.inv_t), -log_s) : (double)kNegInf;
}

// NTHR threads take one row (below 256: several rows a block), or with SPLIT a share of one.
template <class F, int NTHR, bool SPLIT>
__global__ void __launch_bounds__(NTHR < 256 ? 256 : NTHR) log_probs_kernel(const LogProbArgs p) {
  constexpr int W = F::W, kRows = NTHR < 256 ? 256 / NTHR : 1;
  __shared__ Sums part[16];
  const int tid = threadIdx.x % NTHR;
  const int64_t split = SPLIT ? p.split : 1;
  const int64_t r = SPLIT ? blockIdx.x / split : (int64_t)blockIdx.x * kRows + threadIdx.x / NTHR;
  const int64_t piece = SPLIT ? blockIdx.x % split : 0;
  if (kRows > 1 && r >= p.R) return;  // whole groups of lanes: such rows meet no barrier
  const auto* row = static_cast<const typename F::E*>(p.x) + r * p.stride;
  const uint8_t* mask = p.mask ? p.mask + r * p.N : nullptr;
  int64_t lo = 0, hi = p.N;
  if (SPLIT) {
    const int64_t per = ((p.N + split - 1) / split + 63) / 64 * 64;
    lo = piece * per < p.N ? piece * per : p.N;
    hi = lo + per < p.N ? lo + per : p.N;
  }
  const float c = (float)(p.inv_t * (double)kLog2E);
  Sums a = none();
  // elements before the first 16-byte boundary, whole 16-byte loads, the rest
  const int64_t off = (int64_t)(((uintptr_t)(row + lo) / sizeof(typename F::E)) % W);
  const int64_t i0 = off && lo + (W - off) < hi ? lo + (W - off) : (off ? hi : lo);
  const int64_t i1 = i0 + (hi - i0) / W * W;
  auto one = [&](int64_t i) __attribute__((always_inline)) {
    const float x[1] = {(!mask || mask[i] != 0) ? F::get(row[i]) : kNegInf};
    add<1>(a, x, c);
  };
  for (int64_t i = lo + tid; i < i0; i += NTHR) one(i);
  auto group = [&](const Vec<F>& x, int64_t i) __attribute__((always_inline)) {
    float y[W];
#pragma unroll
    for (int k = 0; k < W; ++k) y[k] = F::get(x.e[k]);
    if (mask) {
#pragma unroll
      for (int k = 0; k < W; ++k)
        if (mask[i + k] == 0) y[k] = kNegInf;
    }
    add<W>(a, y, c);
  };
  constexpr int64_t kStep = (int64_t)NTHR * W;
  int64_t i = i0 + (int64_t)tid * W;
  for (; i + 3 * kStep < i1; i += 4 * kStep) {  // four requests at a time
    Vec<F> x[4];
#pragma unroll
    for (int k = 0; k < 4; ++k) x[k].w = *reinterpret_cast<const u32x4*>(row + i + k * kStep);
#pragma unroll
    for (int k = 0; k < 4; ++k) group(x[k], i + k * kStep);
  }
  for (; i < i1; i += kStep) {
    Vec<F> x;
    x.w = *reinterpret_cast<const u32x4*>(row + i);
    group(x, i);
  }
  for (int64_t j = i1 + tid; j < hi; j += NTHR) one(j);
#pragma unroll
  for (int o = 1; o < (NTHR < 64 ? NTHR : 64); o <<= 1) a = join(a, shuffle(a, o), c);
  if constexpr (NTHR > 64) {
    if ((tid & 63) == 0) part[tid >> 6] = a;
    __syncthreads();
    a = part[0];
    for (int n = 1; n < NTHR / 64; ++n) a = join(a, part[n], c);
  }
  if (tid == 0) {
    if constexpr (SPLIT) {
      float* to = p.part + (r * split + piece) * 4;
      to[0] = a.m;
      to[1] = a.n;
      to[2] = a.r;
      to[3] = a.t;
    } else {
      finish<F>(p, r, a);
    }
  }
}

template <class F>
__global__ void __launch_bounds__(64) log_probs_join_kernel(const LogProbArgs p) {
  const int64_t r = blockIdx.x;
  const float c = (float)(p.inv_t * (double)kLog2E);
  Sums a = none();
  for (int64_t n = threadIdx.x; n < p.split; n += 64) {
    const float* q = p.part + (r * p.split + n) * 4;
    a = join(a, Sums{q[0], q[1], q[2], q[3]}, c);
  }
#pragma unroll
  for (int o = 1; o < 64; o <<= 1) a = join(a, shuffle(a, o), c);
  if (threadIdx.x == 0) finish<F>(p, r, a);
}

// One block takes `per` groups of W logits of one row.  Groups lie on the 16-byte
// boundaries of the row, wherever it begins, if the logits and their gradient lie alike (vec).
template <class F>
__global__ void __launch_bounds__(256) log_probs_backward_kernel(const LogProbArgs p, int64_t pieces, int64_t per, int vec) {
  constexpr int W = F::W;
  const int64_t r = blockIdx.x / pieces;
  const auto* row = static_cast<const typename F::E*>(p.x) + r * p.stride;
  auto* out = static_cast<typename F::E*>(p.dx) + r * p.dx_stride;
  const int64_t shift = vec ? (int64_t)(((uintptr_t)row / sizeof(typename F::E)) % W) : 0;
  const uint8_t* mask = p.mask ? p.mask + r * p.N : nullptr;
  const double lse = p.lse[r];  // float64: log p keeps its bits where it is near 0
  const float ent = p.entropy[r], inv_t = (float)p.inv_t;
  const bool empty = lse == (double)kNegInf;
  const float dlp = p.d_log_prob ? p.d_log_prob[r] : 0.0f, dent = p.d_entropy ? p.d_entropy[r] : 0.0f;
  const int64_t act = p.action[r];
  const bool acts = act >= 0 && act < p.N;
  const float base = acts ? dlp : 0.0f;  // no taken action: only the entropy has a gradient
  auto grad = [&](float x, bool legal, bool taken) __attribute__((always_inline)) {
    float l = (float)minus(scaled(x, p.inv_t), lse);
    l = l < -150.0f ? -150.0f : l;  // e^-150 is 0 in float32; keeps 0 * inf out
    const float pr = exp2_fast(l * kLog2E);
    const float d = (taken ? dlp : 0.0f) - pr * (base + dent * (l + ent));
    return legal && x != kNegInf ? d * inv_t : 0.0f;  // -inf is not legal either, if it was taken
  };
  const int64_t g1 = (blockIdx.x % pieces + 1) * per;
  for (int64_t g = blockIdx.x % pieces * per + threadIdx.x; g < g1; g += 256) {
    const int64_t i = g * W - shift;
    if (i >= p.N) break;
    if (vec && i >= 0 && i + W <= p.N) {
      Vec<F> x, y;
      x.w = *reinterpret_cast<const u32x4*>(row + i);
#pragma unroll
      for (int k = 0; k < W; ++k) {
        const bool legal = !empty && (!mask || mask[i + k] != 0);
        y.e[k] = F::put(grad(F::get(x.e[k]), legal, i + k == act));
      }
      *reinterpret_cast<u32x4*>(out + i) = y.w;
    } else {
      for (int k = 0; k < W; ++k) {
        if (i + k < 0 || i + k >= p.N) continue;
        const bool legal = !empty && (!mask || mask[i + k] != 0);
        out[i + k] = F::put(grad(F::get(row[i + k]), legal, i + k == act));
      }
    }
  }
}

template <class F>
hipError_t forward_fmt(const LogProbArgs& a, hipStream_t st) {
  if (a.split > 1) {
    log_probs_kernel<F, 256, true><<<dim3((unsigned)(a.R * a.split)), 256, 0, st>>>(a);
    log_probs_join_kernel<F><<<dim3((unsigned)a.R), 64, 0, st>>>(a);
  } else if (a.N <= 64) {  // 16384 rows of 18: 15.3 us with a wave for each, 5.5 with 8 lanes
    log_probs_kernel<F, 8, false><<<dim3((unsigned)((a.R + 31) / 32)), 256, 0, st>>>(a);
  } else if (a.N <= 2048) {
    log_probs_kernel<F, 64, false><<<dim3((unsigned)((a.R + 3) / 4)), 256, 0, st>>>(a);
  } else {
    log_probs_kernel<F, 256, false><<<dim3((unsigned)a.R), 256, 0, st>>>(a);
  }
  return hipGetLastError();
}

template <class F>
hipError_t backward_fmt(const LogProbArgs& a, hipStream_t st) {
  const int64_t es = sizeof(typename F::E);
  const int vec = (uintptr_t)a.x % 16 == (uintptr_t)a.dx % 16 && (a.stride - a.dx_stride) * es % 16 == 0;
  const int64_t groups = (a.N + F::W - 1) / F::W + 1;  // a row may begin inside its first group
  const int64_t per = groups < 2048 ? (groups + 255) / 256 * 256 : 2048;
  const int64_t pieces = (groups + per - 1) / per;
  log_probs_backward_kernel<F><<<dim3((unsigned)(a.R * pieces)), 256, 0, st>>>(a, pieces, per, vec);
  return hipGetLastError();
}

hipError_t launch_log_probs(rlscan_format f, const LogProbArgs& a, hipStream_t st) {
  switch (f) {
    case RLSCAN_FORMAT_BF16: return forward_fmt<LBf16>(a, st);
    case RLSCAN_FORMAT_F16: return forward_fmt<LF16>(a, st);
    default: return forward_fmt<LF32>(a, st);
  }
}

hipError_t launch_log_probs_backward(rlscan_format f, const LogProbArgs& a, hipStream_t st) {
  switch (f) {
    case RLSCAN_FORMAT_BF16: return backward_fmt<LBf16>(a, st);
    case RLSCAN_FORMAT_F16: return backward_fmt<LF16>(a, st);
    default: return backward_fmt<LF32>(a, st);
  }
}

}  // namespace logits
}  // namespace rlscan
