// Queries and keys normalised by head and rotated by position (rlscan_norm_rotate_heads and
// its backward).
//
//   n = x / sqrt(mean(x^2) + eps),  z = w n,  y = z turned pair by pair by p base^(-2j / R)
//   dz = dy turned back,  dw = sum dz n,  dx = (w dz - n mean(w dz n)) / sqrt(mean(x^2) + eps)
//
// Bound by memory: one read and one write of every head forward, two and one backward.  A
// head lies on a group of lanes, V pairs to a lane: both members of a pair in one lane, so that
// a rotation moves nothing between lanes.  A group takes a token's
// heads one after another with its angles, which are made once for each token: in quarter
// turns, in float64 (a position times a frequency keeps 2^-52 of itself, so far positions turn
// like near ones), of which the part behind the point goes to a float32 sine and cosine.
//
// Measured: 32768 tokens of 16 and 4 heads of 128, bfloat16, forward 68 us (4.9 TB/s of those read and
// written), gradients 120 (4.2) with 5 for the sums of the weights' gradients over blocks; 21312 tokens of 4
// and 2 heads of 80, float32, 21 (4.0) and 35 (3.5): 10 of 16 lanes have a pair there, and one round of blocks is
// short; a token for 16 environments 4 us, latency.
#include <cmath>
#include <type_traits>

#include "rlscan_nr.hpp"
#include "rlscan_sums.hpp"

namespace rlscan {
namespace nr {

using logits::LBf16;
using logits::LF16;
using logits::LF32;

constexpr int kThreads = 256;
// Blocks of the gradients, each with its share of the weights' sums: as many as run at once (three to a
// compute unit).  Measured, us, the bfloat16 case above: 256 blocks 160, 512 118, 768 115, 1024 129.
constexpr int64_t kBackBlocks = 768;

struct Turns {      // frequencies in quarter turns, as products of powers
  double first;     // 2 / pi
  double bit[6];    // factor of a lane's bit b
  double step;      // from a lane's pair to its next
};

struct KernelArgs {
  Args a;
  Turns t;
  int log_lanes;
  int64_t split, units;
};

// V elements as they lie in memory.
template <int kBytes>
struct WordOf {
  using T = uint64_t;
};
template <>
struct WordOf<4> {
  using T = uint32_t;
};
template <class F, int V>
struct Raw {
  typename F::E e[V];
};
template <class F, int V>
__device__ __forceinline__ Raw<F, V> load_vec(const typename F::E* p) {
  constexpr int kBytes = V * (int)sizeof(typename F::E);
  Raw<F, V> r;
  if constexpr (kBytes % 16 == 0) {
    typedef uint32_t u32x4 __attribute__((ext_vector_type(4)));
#pragma unroll
    for (int i = 0; i < kBytes / 16; ++i) {
      const u32x4 v = reinterpret_cast<const u32x4*>(p)[i];
      __builtin_memcpy(reinterpret_cast<char*>(&r) + 16 * i, &v, 16);
    }
  } else {
    using Word = typename WordOf<kBytes>::T;
    const Word v = *reinterpret_cast<const Word*>(p);
    __builtin_memcpy(&r, &v, kBytes);
  }
  return r;
}
template <class F, int V>
__device__ __forceinline__ void store_vec(typename F::E* p, const Raw<F, V>& r) {
  constexpr int kBytes = V * (int)sizeof(typename F::E);
  if constexpr (kBytes % 16 == 0) {
    typedef uint32_t u32x4 __attribute__((ext_vector_type(4)));
#pragma unroll
    for (int i = 0; i < kBytes / 16; ++i) {
      u32x4 v;
      __builtin_memcpy(&v, reinterpret_cast<const char*>(&r) + 16 * i, 16);
      reinterpret_cast<u32x4*>(p)[i] = v;
    }
  } else {
    typename WordOf<kBytes>::T v;
    __builtin_memcpy(&v, &r, kBytes);
    *reinterpret_cast<typename WordOf<kBytes>::T*>(p) = v;
  }
}

// Where a lane's pairs lie.  VEC: a and b are V elements side by side each (INTER: the
// pairs lie within a and within b); else pair i is one element at oa[i] and one at ob[i], -1
// where the head has none.
template <int V, bool VEC, bool INTER>
struct Place {
  int oa[VEC ? 1 : V], ob[VEC ? 1 : V];
  bool some;  // the lane has any

  __device__ __forceinline__ Place(int lane, int lanes, int D, int R) {
    if constexpr (VEC) {
      const int j = lane * V;
      some = 2 * j < D;
      if (INTER || j >= R / 2) {
        oa[0] = 2 * j;
        ob[0] = 2 * j + V;
      } else {
        oa[0] = j;
        ob[0] = j + R / 2;
      }
    } else {
      some = 2 * lane < D;
#pragma unroll
      for (int i = 0; i < V; ++i) {
        const int j = lane + i * lanes;
        const bool turned = !INTER && j < R / 2;
        oa[i] = turned ? j : 2 * j;
        ob[i] = turned ? j + R / 2 : 2 * j + 1;
        if (oa[i] >= D) oa[i] = -1;
        if (ob[i] >= D) ob[i] = -1;
      }
    }
  }
  // The number of the pair behind angle i.
  static __device__ __forceinline__ int pair(int i, int lane, int lanes) {
    return VEC ? lane * V + i : lane + i * lanes;
  }
};

template <class F, int V, bool VEC, bool INTER>
struct Head {
  Raw<F, V> a, b;

  __device__ __forceinline__ void load(const typename F::E* p, const Place<V, VEC, INTER>& at) {
    if constexpr (VEC) {
      if (!at.some) return;
      a = load_vec<F, V>(p + at.oa[0]);
      b = load_vec<F, V>(p + at.ob[0]);
    } else {
#pragma unroll
      for (int i = 0; i < V; ++i) {
        a.e[i] = at.oa[i] >= 0 ? p[at.oa[i]] : F::put(0.0f);
        b.e[i] = at.ob[i] >= 0 ? p[at.ob[i]] : F::put(0.0f);
      }
    }
  }
  __device__ __forceinline__ void get(float (&x)[V], float (&y)[V], const Place<V, VEC, INTER>& at) const {
#pragma unroll
    for (int i = 0; i < V; ++i) {
      x[i] = at.some ? F::get(a.e[i]) : 0.0f;
      y[i] = at.some ? F::get(b.e[i]) : 0.0f;
    }
  }
  static __device__ __forceinline__ void store(typename F::E* p, const float (&x)[V], const float (&y)[V],
                                               const Place<V, VEC, INTER>& at) {
    if constexpr (VEC) {
      if (!at.some) return;
      Raw<F, V> r, s;
#pragma unroll
      for (int i = 0; i < V; ++i) {
        r.e[i] = F::put(x[i]);
        s.e[i] = F::put(y[i]);
      }
      store_vec<F, V>(p + at.oa[0], r);
      store_vec<F, V>(p + at.ob[0], s);
    } else {
#pragma unroll
      for (int i = 0; i < V; ++i) {
        if (at.oa[i] >= 0) p[at.oa[i]] = F::put(x[i]);
        if (at.ob[i] >= 0) p[at.ob[i]] = F::put(y[i]);
      }
    }
  }
};

// Turns the pairs of a lane.
template <int V, bool WITHIN>
__device__ __forceinline__ void turn(float (&x)[V], float (&y)[V], const float (&cs)[V], const float (&sn)[V]) {
  if constexpr (WITHIN) {  // pairs 2i, 2i + 1 of x, then of y
#pragma unroll
    for (int i = 0; i < V / 2; ++i) {
      const float a = x[2 * i], b = x[2 * i + 1], c = y[2 * i], d = y[2 * i + 1];
      x[2 * i] = a * cs[i] - b * sn[i];
      x[2 * i + 1] = b * cs[i] + a * sn[i];
      y[2 * i] = c * cs[V / 2 + i] - d * sn[V / 2 + i];
      y[2 * i + 1] = d * cs[V / 2 + i] + c * sn[V / 2 + i];
    }
  } else {
#pragma unroll
    for (int i = 0; i < V; ++i) {
      const float a = x[i], b = y[i];
      x[i] = a * cs[i] - b * sn[i];
      y[i] = b * cs[i] + a * sn[i];
    }
  }
}

// cos and sin of an angle given in quarter turns: the whole ones by exchange and sign, the rest,
// at most pi / 4, by the series (next terms below 2^-25).
__device__ __forceinline__ void angle(double quarters, float& cs, float& sn) {
  const double whole = __builtin_rint(quarters);
  const int q = (int)(whole - 4.0 * __builtin_floor(whole * 0.25));
  const float x = (float)(quarters - whole) * 1.57079632679489662f, x2 = x * x;
  float s = __builtin_fmaf(x2, 1.0f / 362880.0f, -1.0f / 5040.0f);
  s = __builtin_fmaf(x2, s, 1.0f / 120.0f);
  s = __builtin_fmaf(x2, s, -1.0f / 6.0f);
  s = __builtin_fmaf(x * x2, s, x);
  float c = __builtin_fmaf(x2, -1.0f / 3628800.0f, 1.0f / 40320.0f);
  c = __builtin_fmaf(x2, c, -1.0f / 720.0f);
  c = __builtin_fmaf(x2, c, 1.0f / 24.0f);
  c = __builtin_fmaf(x2, c, -0.5f);
  c = __builtin_fmaf(x2, c, 1.0f);
  cs = q & 1 ? s : c;
  sn = q & 1 ? c : s;
  if (q == 1 || q == 2) cs = -cs;
  if (q >= 2) sn = -sn;
}

// The sum over a group of 2^log_lanes lanes, in every one of them: up to 16 by lane moves within a
// row of 16, which take no trip through LDS.
__device__ __forceinline__ float group_sum(float v, int log_lanes) {
  auto moved = [](float x, auto control) __attribute__((always_inline)) {
    return __builtin_bit_cast(float, __builtin_amdgcn_update_dpp(0, __builtin_bit_cast(int, x), decltype(control)::value,
                                                                 0xf, 0xf, true));
  };
  if (log_lanes > 0) v += moved(v, std::integral_constant<int, 0xb1>{});   // lanes 1 0 3 2 of four
  if (log_lanes > 1) v += moved(v, std::integral_constant<int, 0x4e>{});   // lanes 2 3 0 1
  if (log_lanes > 2) v += moved(v, std::integral_constant<int, 0x141>{});  // eight reversed
  if (log_lanes > 3) v += moved(v, std::integral_constant<int, 0x140>{});  // sixteen reversed
  if (log_lanes > 4) v += __shfl_xor(v, 16);
  if (log_lanes > 5) v += __shfl_xor(v, 32);
  return v;
}

// A unit is a token's heads s, s + split, ...; a group of lanes takes units in turn.  The heads' loads
// go out ahead (RING of them), always, and ahead of the stores: behind one that may not have been
// made, a wait for one would wait for all.
template <class F, int V, bool VEC, bool INTER, bool BWD, int RING>
__global__ void __launch_bounds__(kThreads) __attribute__((amdgpu_waves_per_eu(BWD ? 3 : 4))) heads_kernel(const KernelArgs k) {
  using E = typename F::E;
  using At = Place<V, VEC, INTER>;
  using H = Head<F, V, VEC, INTER>;
  __shared__ float s_w[BWD ? kThreads * 2 * V : 1];
  const Args& p = k.a;
  const int lanes = 1 << k.log_lanes, lane = threadIdx.x & (lanes - 1), group = threadIdx.x >> k.log_lanes;
  const int groups = kThreads >> k.log_lanes;
  const At at(lane, lanes, p.D, p.R);
  const float over_d = 1.0f / (float)p.D;
  float dwa[2][BWD ? V : 1], dwb[2][BWD ? V : 1];
  if constexpr (BWD) {
#pragma unroll
    for (int i = 0; i < V; ++i) dwa[0][i] = dwb[0][i] = dwa[1][i] = dwb[1][i] = 0.0f;
  }
  // Groups leave the loop together with their wave: shuffles stay within a group, whose lanes
  // all have the same unit.
  for (int64_t u = (int64_t)blockIdx.x * groups + group; u < k.units; u += (int64_t)gridDim.x * groups) {
    const int64_t token = k.split == 1 ? u : u / k.split;
    int h = (int)(u - token * k.split);
    const int64_t e = p.E == 1 ? 0 : token / p.T, t = token - e * p.T;
    float cs[V], sn[V];
    {
      const double pos = p.R > 0 ? (double)p.pos[e * p.p_se + t * p.p_st] : 0.0;
      double f = k.t.first;
#pragma unroll
      for (int b = 0; b < 6; ++b) f *= (lane >> b) & 1 ? k.t.bit[b] : 1.0;
#pragma unroll
      for (int i = 0; i < V; ++i) {
        angle(At::pair(i, lane, lanes) < p.R / 2 ? pos * f : 0.0, cs[i], sn[i]);
        if (BWD) sn[i] = -sn[i];
        f *= k.t.step;
      }
    }
#pragma unroll
    for (int which = 0; which < 2; ++which) {
      const int heads = (int)p.heads[which], split = (int)k.split;
      if (h < heads) {
        const int64_t sh = p.in[which].sh, gh = BWD ? p.grad[which].sh : 0, oh = p.out[which].sh;
        const E* const px = static_cast<const E*>(p.in[which].p) + e * p.in[which].se + t * p.in[which].st;
        const E* const pg = BWD ? static_cast<const E*>(p.grad[which].p) + e * p.grad[which].se + t * p.grad[which].st : nullptr;
        E* const po = static_cast<E*>(const_cast<void*>(p.out[which].p)) + e * p.out[which].se + t * p.out[which].st;
        float wa[V], wb[V];
#pragma unroll
        for (int i = 0; i < V; ++i) {
          const int oa = VEC ? at.oa[0] + i : at.oa[VEC ? 0 : i], ob = VEC ? at.ob[0] + i : at.ob[VEC ? 0 : i];
          const bool ok = p.weight[which] != nullptr && at.some;
          wa[i] = ok && oa >= 0 ? p.weight[which][oa] : 1.0f;
          wb[i] = ok && ob >= 0 ? p.weight[which][ob] : 1.0f;
        }
        const int last = h + (heads - 1 - h) / split * split;
        H raw[RING], raw_g[RING];
#pragma unroll
        for (int r = 0; r < RING; ++r) {
          const int hr = h + r * split < last ? h + r * split : last;
          raw[r].load(px + hr * sh, at);
          if constexpr (BWD) raw_g[r].load(pg + hr * gh, at);
        }
        auto take = [&](H& now, H& now_g, int h) __attribute__((always_inline)) {
          float x[V], y[V], gx[V], gy[V];
          now.get(x, y, at);
          if constexpr (BWD) now_g.get(gx, gy, at);
          const int then = h + RING * split < last ? h + RING * split : last;
          now.load(px + then * sh, at);
          if constexpr (BWD) now_g.load(pg + then * gh, at);
          float sq = 0.0f;
#pragma unroll
          for (int i = 0; i < V; ++i) sq += x[i] * x[i] + y[i] * y[i];
          const float inv = __builtin_amdgcn_rsqf(group_sum(sq, k.log_lanes) * over_d + p.eps);
          if constexpr (!BWD) {
#pragma unroll
            for (int i = 0; i < V; ++i) {
              x[i] = x[i] * inv * wa[i];
              y[i] = y[i] * inv * wb[i];
            }
            turn<V, VEC && INTER>(x, y, cs, sn);
          } else {
            turn<V, VEC && INTER>(gx, gy, cs, sn);
            float dot = 0.0f;
#pragma unroll
            for (int i = 0; i < V; ++i) {
              x[i] *= inv;
              y[i] *= inv;
              dwa[which][i] += gx[i] * x[i];
              dwb[which][i] += gy[i] * y[i];
              gx[i] *= wa[i];
              gy[i] *= wb[i];
              dot += gx[i] * x[i] + gy[i] * y[i];
            }
            dot = group_sum(dot, k.log_lanes) * over_d;
#pragma unroll
            for (int i = 0; i < V; ++i) {
              x[i] = inv * (gx[i] - x[i] * dot);
              y[i] = inv * (gy[i] - y[i] * dot);
            }
          }
          H::store(po + h * oh, x, y, at);
        };
        for (; h + (RING - 1) * split <= last; h += RING * split) {
#pragma unroll
          for (int r = 0; r < RING; ++r) take(raw[r], raw_g[r], h + r * split);
        }
#pragma unroll
        for (int r = 0; r < RING - 1; ++r) {
          if (h <= last) {
            take(raw[r], raw_g[r], h);
            h += split;
          }
        }
      }
      h -= heads;
    }
  }
  if constexpr (BWD) {
#pragma unroll
    for (int which = 0; which < 2; ++which) {
      __syncthreads();
#pragma unroll
      for (int i = 0; i < V; ++i) {
        s_w[i * kThreads + threadIdx.x] = dwa[which][i];
        s_w[(V + i) * kThreads + threadIdx.x] = dwb[which][i];
      }
      __syncthreads();
      if (group == 0) {
#pragma unroll
        for (int i = 0; i < V; ++i) {
          float a = 0.0f, b = 0.0f;
          for (int g = 0; g < groups; ++g) {
            a += s_w[i * kThreads + g * lanes + lane];
            b += s_w[(V + i) * kThreads + g * lanes + lane];
          }
          const int oa = VEC ? at.oa[0] + i : at.oa[VEC ? 0 : i], ob = VEC ? at.ob[0] + i : at.ob[VEC ? 0 : i];
          float* part = p.part + ((int64_t)blockIdx.x * 2 + which) * p.D;
          if (at.some && oa >= 0) part[oa] = a;
          if (at.some && ob >= 0) part[ob] = b;
        }
      }
    }
  }
}

// Pairs to a lane, side by side: pieces of 8 bytes, 16 for float32's gradients.  Measured, us forward and
// backward, 32768 tokens of 16 and 4 heads of 128, bfloat16: four pairs 75 and 115, eight 78 and (with fewer
// waves to a compute unit) 150; 65536 tokens of 8 and 8 heads of 64, float32: two 97 and 165, four 100 and 165.
// Pairs one by one, where addresses or sizes do not fit, take 109 and 168, and 155 and 194; as many heads in flight
// as of pieces are more than their registers hold there, and some go through memory.
static constexpr int widest(int es, bool backward) { return es == 4 && !backward ? 2 : 4; }

static int log2_up(int64_t n) {
  int b = 0;
  while (((int64_t)1 << b) < n) ++b;
  return b;
}

int64_t backward_blocks(int64_t tokens, int64_t heads, int D) {
  const int64_t pairs = (D + 1) / 2, units = tokens * heads;
  const int64_t lanes = (int64_t)1 << log2_up((pairs + 3) / 4);
  const int64_t want = (units * lanes + kThreads - 1) / kThreads;
  return want < 1 ? 1 : want < kBackBlocks ? want : kBackBlocks;
}

Plan make_plan(rlscan_format f, const Args& a, bool backward) {
  Plan p{};
  const int es = f == RLSCAN_FORMAT_F32 ? 4 : 2;
  auto fits = [&](int V) {
    if (a.D % (2 * V) != 0 || (!a.interleaved && (a.R / 2) % V != 0)) return false;
    const int64_t bytes = V * es < 16 ? V * es : 16;
    for (int w = 0; w < 2; ++w) {
      if (a.heads[w] == 0) continue;
      const View* v[3] = {&a.in[w], &a.out[w], backward ? &a.grad[w] : &a.in[w]};
      for (const View* x : v)
        if ((uintptr_t)x->p % bytes || x->se * es % bytes || x->st * es % bytes || x->sh * es % bytes) return false;
    }
    return true;
  };
  p.V = 4;
  for (int V = widest(es, backward); V >= 2 && !p.vec; V /= 2) {
    if (!fits(V)) continue;
    p.V = V;
    p.vec = 1;
  }
  const int64_t pairs = (a.D + 1) / 2;
  p.log_lanes = log2_up((pairs + p.V - 1) / p.V);
  const int64_t tokens = a.E * a.T, heads = a.heads[0] + a.heads[1], groups = kThreads >> p.log_lanes;
  // Few tokens: their heads go to several groups, until there are 512 blocks, though each makes the angles
  // again.  Measured, us: one token of 20 heads by one group 15, by four 12.3, by eight 12.8; 21312 tokens by
  // one 20, by two 26
  p.split = tokens > 0 ? (512 * groups + tokens - 1) / tokens : 1;
  if (p.split > heads) p.split = heads;
  if (p.split < 1) p.split = 1;
  p.blocks = (tokens * p.split + groups - 1) / groups;
  const int64_t most = backward ? backward_blocks(tokens, heads, a.D) : (int64_t)1 << 20;
  if (p.blocks > most) p.blocks = most;
  if (p.blocks < 1) p.blocks = 1;
  return p;
}

template <class F, int V, bool VEC, bool BWD>
static void run_heads(const KernelArgs& k, int64_t blocks, hipStream_t st) {
  // Heads in flight, us: forward bfloat16 (32768 tokens of 20 heads) four 71, two 74; float32 (21312 of 6) two 18,
  // four 19; backward bfloat16 two, float32, which keeps twice the registers of each, one (21312 of 6 37.4, two 37.7;
  // 32768 of 20 204, two 203).
  constexpr int kRing = (BWD ? 2 : 4) / (sizeof(typename F::E) == 4 ? 2 : 1);
  if (k.a.interleaved) heads_kernel<F, V, VEC, true, BWD, kRing><<<dim3((unsigned)blocks), kThreads, 0, st>>>(k);
  else heads_kernel<F, V, VEC, false, BWD, kRing><<<dim3((unsigned)blocks), kThreads, 0, st>>>(k);
}

template <class F, bool BWD>
static hipError_t run_fmt(rlscan_format f, const Args& a, hipStream_t st) {
  const Plan p = make_plan(f, a, BWD);
  KernelArgs k{};
  k.a = a;
  k.log_lanes = p.log_lanes;
  k.split = p.split;
  k.units = a.E * a.T * p.split;
  // pair j turns by base^(-2j / R) for a step
  const double log_ratio = a.R > 0 ? -2.0 / a.R * std::log2(a.base) : 0.0;
  const int stride = p.vec ? p.V : 1;
  k.t.first = 0.63661977236758134308;
  for (int b = 0; b < 6; ++b) k.t.bit[b] = std::exp2(log_ratio * (double)(stride << b));
  k.t.step = std::exp2(log_ratio * (double)(p.vec ? 1 : 1 << p.log_lanes));
  constexpr int kV = widest(sizeof(typename F::E), BWD);
  if (p.vec && p.V == kV) run_heads<F, kV, true, BWD>(k, p.blocks, st);
  else if (p.vec) run_heads<F, 2, true, BWD>(k, p.blocks, st);
  else run_heads<F, 4, false, BWD>(k, p.blocks, st);
  hipError_t e = hipGetLastError();
  if (!BWD || e != hipSuccess || (!a.d_weight[0] && !a.d_weight[1])) return e;
  // the sums of a weight that is not asked for are left unread
  const int64_t D = a.D;
  return sums::launch_columns(a.part, p.blocks, a.d_weight[0], D, a.d_weight[1], D, st);
}

hipError_t launch_forward(rlscan_format f, const Args& a, hipStream_t st) {
  switch (f) {
    case RLSCAN_FORMAT_BF16: return run_fmt<LBf16, false>(f, a, st);
    case RLSCAN_FORMAT_F16: return run_fmt<LF16, false>(f, a, st);
    default: return run_fmt<LF32, false>(f, a, st);
  }
}

hipError_t launch_backward(rlscan_format f, const Args& a, hipStream_t st) {
  switch (f) {
    case RLSCAN_FORMAT_BF16: return run_fmt<LBf16, true>(f, a, st);
    case RLSCAN_FORMAT_F16: return run_fmt<LF16, true>(f, a, st);
    default: return run_fmt<LF32, true>(f, a, st);
  }
}

}  // namespace nr
}  // namespace rlscan
