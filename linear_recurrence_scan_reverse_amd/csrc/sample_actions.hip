// Sampling one action from each row of logits with given uniform numbers
// (rlscan_sample_actions).
//
// Legal logits x_i (mask set, above -inf) get the weights w_i = e^((x_i - max) / temperature).
// In the order of falling logits (equal ones: lower index first) the row keeps its
// first top_k, of those the shortest prefix with top_p of their weight, and of
// those the ones with w_i >= min_p.  The action is the first index, in the order
// of the indices, whose running weight passes u times the kept weight; its
// log-probability is that under the kept distribution.
//
// Which action comes out turns on sums of up to a million weights next to a
// border, so weights are exact functions of a logit: computed in float64 (about
// 2e-16) and rounded once to whole multiples of 2^-43.  Sums of them are whole
// numbers below 2^63 and do not depend on any order: neither atomics nor the way
// a row is shared changes an action.
//
// A kept set is a prefix of the falling order: all logits above a threshold and
// the first `quota` of those equal to it.  A block finds it for one row: a pass
// for the maximum; for long rows a pass that sorts logits into coarse bins of
// (max - x) with their counts and weights, which leaves one bin to look into; that
// bin's logits, collected in LDS, are searched by 8-bit digits of their
// order-preserving keys.  A last pass sums the kept weights of tiles of the row, and
// one wave finds the tile and in it the action.
#include "rlscan_logits.hpp"

namespace rlscan {
namespace logits {

constexpr int kBins = 1024;     // coarse bins over 32 temperatures below the maximum
constexpr int kSmall = 1024;    // rows up to here go to one wave
constexpr int kMiddle = 4096;   // and up to here to four
constexpr double kUnit = 8796093022208.0;  // 2^43
constexpr float kMaxFloat = 3.4028234663852886e38f;

__device__ __forceinline__ uint32_t key_of(float x) {  // larger logit, larger key
  const uint32_t b = __builtin_bit_cast(uint32_t, x + 0.0f);  // -0 and 0 are equal
  return b & 0x80000000u ? ~b : b | 0x80000000u;
}

__device__ __forceinline__ float value_of(uint32_t k) {
  return __builtin_bit_cast(float, k & 0x80000000u ? k & 0x7fffffffu : ~k);
}

// e^y for y <= 0, to about 2e-16: 2^(n/64) from a table, and the Taylor series of
// the rest, |r| <= ln 2 / 128, to the fifth power.
__device__ __forceinline__ double exp_table(double y, const double* table) {
  const double n = __builtin_rint(y * (64.0 / 0.693147180559945309417));
  double r = __builtin_fma(n, -0x1.62e42fefap-7, y);  // the leading 37 bits of ln 2 / 64: n * it is exact
  r = __builtin_fma(n, -(0x1.62e42fefa39efp-7 - 0x1.62e42fefap-7) - 0x1.abc9e3b39803fp-62, r);
  double p = __builtin_fma(r, 1.0 / 120.0, 1.0 / 24.0);
  p = __builtin_fma(p, r, 1.0 / 6.0);
  p = __builtin_fma(p, r, 0.5);
  p = __builtin_fma(p, r, 1.0);
  p = __builtin_fma(p, r, 1.0);
  const int i = (int)n;
  return __builtin_ldexp(p * table[i & 63], i >> 6);
}

struct Weigh {
  double max, inv_t;
  const double* table;
  __device__ __forceinline__ double log_weight(float x) const { return ((double)x - max) * inv_t; }
  // A weight as a float64, 0 where it rounds to no unit.
  __device__ __forceinline__ double weight(float x) const {
    const double y = log_weight(x);
    return y < -31.0 ? 0.0 : exp_table(y, table);
  }
  static __device__ __forceinline__ uint64_t units(double w) {
    const double m = __builtin_fma(w, kUnit, 4503599627370496.0);  // + 2^52: rounds to a whole number
    return __builtin_bit_cast(uint64_t, m) & 0xfffffffffffffull;
  }
};

// NTHR threads; rows up to kSmall, kMiddle or kMaxActions logits.  Rows of the first
// two sizes go to the list whole and need no coarse bins.
template <int NTHR>
struct SampleLds {
  static constexpr bool kCoarse = NTHR == 1024;
  static constexpr int kList = NTHR == 64 ? kSmall : kMiddle;  // keys held
  static constexpr int kTiles = (int)((kCoarse ? kMaxActions : kList) / 256) + 2;
  double table[64];
  uint64_t hist[256];
  uint64_t coarse_w[kCoarse ? kBins : 1];
  uint32_t coarse_n[kCoarse ? kBins : 1];
  uint32_t list[kList];
  uint64_t tile_w[kTiles];
  uint32_t tile_n[kTiles];
  uint64_t red[NTHR / 64];
  float redf[NTHR / 64];
  uint32_t count;
  // a search's result
  int bin;
  uint64_t before;
  uint64_t inside;
};

template <int NTHR>
__device__ __forceinline__ uint64_t block_sum(uint64_t v, uint64_t* red) {
#pragma unroll
  for (int o = 1; o < 64; o <<= 1) v += __shfl_xor(v, o);
  __syncthreads();
  if ((threadIdx.x & 63) == 0) red[threadIdx.x >> 6] = v;
  __syncthreads();
  uint64_t s = 0;
#pragma unroll
  for (int n = 0; n < NTHR / 64; ++n) s += red[n];
  return s;
}

// The first of n bins whose running sum reaches `target` (at least one unit), by the
// first wave; the last bin with anything in it if none does.  Results in s.bin,
// s.before (sum before the bin, with `base`) and s.inside (its own).
template <class S, class V>
__device__ __forceinline__ void search_bins(S& s, const V* bins, int n, uint64_t base, double target, bool falling) {
  __syncthreads();
  if (threadIdx.x < 64) {
    const int lane = threadIdx.x;
    const int per = n / 64;
    uint64_t own = 0;
    for (int i = 0; i < per; ++i) {
      const int b = lane * per + i;
      own += bins[falling ? n - 1 - b : b];
    }
    uint64_t upto = own;
#pragma unroll
    for (int o = 1; o < 64; o <<= 1) {
      const uint64_t up = __shfl_up(upto, o);
      if (lane >= o) upto += up;
    }
    const uint64_t reached = __ballot((double)(base + upto) >= target && own > 0);
    const uint64_t filled = __ballot(own > 0);
    // running sums grow, so the first lane that reaches the target holds the bin
    const int who = reached ? __ffsll((unsigned long long)reached) - 1 : (filled ? 63 - __clzll((long long)filled) : 0);
    if (lane == who) {
      uint64_t sum = base + upto - own;
      int found = 0;
      uint64_t before = sum, inside = 0;
      for (int i = 0; i < per; ++i) {
        const int b = falling ? n - 1 - (lane * per + i) : lane * per + i;
        const uint64_t v = bins[b];
        if (v == 0) continue;
        found = b;
        before = sum;
        inside = v;
        sum += v;
        if ((double)sum >= target) break;
      }
      s.bin = found;
      s.before = before;
      s.inside = inside;
    }
  }
  __syncthreads();
}

template <class F, int NTHR>
__global__ void __launch_bounds__(NTHR) sample_kernel(const SampleArgs a) {
  constexpr int W = F::W;
  __shared__ SampleLds<NTHR> s;
  const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
  const int64_t r = blockIdx.x;
  const auto* row = static_cast<const typename F::E*>(a.x) + r * a.stride;
  const uint8_t* mask = a.mask ? a.mask + r * a.N : nullptr;
  const int N = (int)a.N;
  // groups of W logits on the row's 16-byte boundaries; the row begins `shift` into the first
  const int shift = (int)(((uintptr_t)row / sizeof(typename F::E)) % W);
  const int groups = (N + shift + W - 1) / W;

  float temperature = a.temperature ? a.temperature[r] : a.temperature1;
  int top_k = a.top_k ? a.top_k[r] : a.top_k1;
  const float top_p = a.top_p ? a.top_p[r] : a.top_p1;
  float min_p = a.min_p ? a.min_p[r] : a.min_p1;
  if (!(temperature > 0.0f)) {  // greedy: the largest logit, lowest index first
    temperature = 1.0f;
    top_k = 1;
  }
  min_p = min_p > 0.0f ? fminf(min_p, 1.0f) : 0.0f;

  // fn(x) for each legal logit of group g
  auto group = [&](int g, float (&x)[W]) __attribute__((always_inline)) {
    const int i = g * W - shift;
    if (i >= 0 && i + W <= N) {
      Vec<F> v;
      v.w = *reinterpret_cast<const u32x4*>(row + i);
#pragma unroll
      for (int k = 0; k < W; ++k) x[k] = F::get(v.e[k]);
    } else {
#pragma unroll
      for (int k = 0; k < W; ++k) x[k] = i + k >= 0 && i + k < N ? F::get(row[i + k]) : kNegInf;
    }
#pragma unroll
    for (int k = 0; k < W; ++k) {
      // NaN is not legal; +inf counts as the largest float
      if (mask && i + k >= 0 && i + k < N && mask[i + k] == 0) x[k] = kNegInf;
      x[k] = x[k] > kNegInf ? fminf(x[k], kMaxFloat) : kNegInf;
    }
  };

  // ---- maximum
  float top = kNegInf;
  for (int g = tid; g < groups; g += NTHR) {
    float x[W];
    group(g, x);
#pragma unroll
    for (int k = 0; k < W; ++k) top = fmaxf(top, x[k]);
  }
#pragma unroll
  for (int o = 1; o < 64; o <<= 1) top = fmaxf(top, __shfl_xor(top, o));
  if (lane == 0) s.redf[wave] = top;
  if (tid < 64) s.table[tid] = exp2((double)tid / 64.0);
  __syncthreads();
#pragma unroll
  for (int n = 0; n < NTHR / 64; ++n) top = fmaxf(top, s.redf[n]);
  if (top == kNegInf) {  // no legal action: the whole block leaves
    if (tid == 0) {
      a.action[r] = -1;
      if (a.log_prob) a.log_prob[r] = 0.0f;
    }
    return;
  }
  const Weigh weigh{(double)top, 1.0 / (double)temperature, s.table};

  // ---- the threshold: keys above it, and `quota` of those equal to it, are kept
  bool need_k = top_k > 0 && top_k < N;
  const bool need_p = top_p < 1.0f;
  uint32_t thr = 0;
  uint64_t quota = ~0ull;
  if (need_k || need_p) {
    constexpr bool coarse = SampleLds<NTHR>::kCoarse;
    constexpr int kList = SampleLds<NTHR>::kList;
    const float per = fminf((float)kBins / (32.0f * temperature), 1e30f);
    auto bin_of = [&](float x) __attribute__((always_inline)) { return (int)fminf((top - x) * per, (float)(kBins - 1)); };
    if (coarse) {
      for (int i = tid; i < kBins; i += NTHR) {
        s.coarse_n[i] = 0;
        s.coarse_w[i] = 0;
      }
      __syncthreads();
      for (int g = tid; g < groups; g += NTHR) {
        float x[W];
        group(g, x);
#pragma unroll
        for (int k = 0; k < W; ++k) {
          if (x[k] == kNegInf) continue;
          const int b = bin_of(x[k]);
          if (need_k) atomicAdd(&s.coarse_n[b], 1u);
          if (need_p) {
            const uint64_t u = Weigh::units(weigh.weight(x[k]));
            if (u) atomicAdd((unsigned long long*)&s.coarse_w[b], (unsigned long long)u);
          }
        }
      }
      __syncthreads();
    }

    int held = -2;  // the bin whose keys are in the list; -1: the whole row
    bool in_list = false;
    // Calls fn(key) for each logit of a bin (-1: of the row).
    auto collect = [&](int bin) __attribute__((always_inline)) {
      if (held == bin) return;
      __syncthreads();
      if (tid == 0) s.count = 0;
      __syncthreads();
      for (int g = tid; g < groups; g += NTHR) {
        float x[W];
        group(g, x);
#pragma unroll
        for (int k = 0; k < W; ++k) {
          if (x[k] == kNegInf || (bin >= 0 && bin_of(x[k]) != bin)) continue;
          const uint32_t at = atomicAdd(&s.count, 1u);
          if (at < (uint32_t)kList) s.list[at] = key_of(x[k]);
        }
      }
      __syncthreads();
      held = bin;
      in_list = s.count <= (uint32_t)kList;
    };
    auto each = [&](auto fn) __attribute__((always_inline)) {
      if (in_list) {
        const int n = (int)s.count;
        for (int i = tid; i < n; i += NTHR) fn(s.list[i]);
      } else {
        for (int g = tid; g < groups; g += NTHR) {
          float x[W];
          group(g, x);
#pragma unroll
          for (int k = 0; k < W; ++k)
            if (x[k] != kNegInf && (held < 0 || bin_of(x[k]) == held)) fn(key_of(x[k]));
        }
      }
    };
    // Within the held bin: the key at which the running sum (of 1 for each logit, or
    // of its weight) reaches target, from `base`; leaves the sum before that key in
    // s.before and that of all logits equal to it in s.inside.
    auto descend = [&](bool weights, uint64_t base, double target) __attribute__((always_inline)) {
      uint32_t prefix = 0, known = 0;
#pragma unroll 1
      for (int d = 24; d + 8 > F::kLow; d -= 8) {
        for (int i = tid; i < 256; i += NTHR) s.hist[i] = 0;
        __syncthreads();
        each([&](uint32_t key) __attribute__((always_inline)) {
          if ((key & known) != prefix) return;
          const uint64_t v = weights ? Weigh::units(weigh.weight(value_of(key))) : 1;
          if (v) atomicAdd((unsigned long long*)&s.hist[key >> d & 255], (unsigned long long)v);
        });
        search_bins(s, s.hist, 256, base, target, true);
        prefix |= (uint32_t)s.bin << d;
        known |= 255u << d;
        base = s.before;
      }
      // bits below the last digit: zero in a value, so ones in a negative one's key
      if (!(prefix & 0x80000000u)) prefix |= ~known;
      return prefix;
    };

    uint64_t kept_before = 0;  // weight of whole bins before the one that top_k cuts
    uint64_t kept = 0;         // weight that top_k keeps
    int bin_k = kBins;         // the bin that top_k cuts
    if (need_k) {
      uint64_t before = 0;
      int bin = -1;
      if (coarse) {
        search_bins(s, s.coarse_n, kBins, 0, (double)top_k, false);
        before = s.before;
        bin = bin_k = s.bin;
        need_k = s.before + s.inside >= (uint64_t)top_k;
      }
      if (need_k) {
        collect(bin);
        if (!coarse) need_k = s.count > (uint32_t)top_k;
      }
      if (need_k) {
        thr = descend(false, before, (double)top_k);
        quota = (uint64_t)top_k - s.before;
        if (need_p) {
          uint64_t mine = 0;
          each([&](uint32_t key) __attribute__((always_inline)) {
            if (key > thr) mine += Weigh::units(weigh.weight(value_of(key)));
          });
          kept = block_sum<NTHR>(mine, s.red) + quota * Weigh::units(weigh.weight(value_of(thr)));
          if (coarse) {
            uint64_t w = 0;
            for (int i = tid; i < bin_k; i += NTHR) w += s.coarse_w[i];
            kept_before = block_sum<NTHR>(w, s.red);
            kept += kept_before;
          }
        }
      }
    }
    if (need_p) {
      int bin = -1;
      uint64_t base = 0;
      if (!need_k) {
        uint64_t w = 0;
        if (coarse) {
          for (int i = tid; i < kBins; i += NTHR) w += s.coarse_w[i];
        } else {
          collect(-1);
          each([&](uint32_t key) __attribute__((always_inline)) { w += Weigh::units(weigh.weight(value_of(key))); });
        }
        kept = block_sum<NTHR>(w, s.red);
      }
      double target = (double)top_p * (double)kept;
      if (!(target >= 1.0)) target = 1.0;  // the largest is always kept
      if (coarse) {
        if (need_k && (double)kept_before < target) {
          bin = bin_k;
          base = kept_before;
        } else {
          search_bins(s, s.coarse_w, kBins, 0, target, false);
          bin = s.bin;
          base = s.before;
        }
      }
      collect(bin);
      const uint32_t key = descend(true, base, target);
      const uint64_t one = Weigh::units(weigh.weight(value_of(key)));
      uint64_t n = 1;  // as many of the equal ones as reach the target
      if (one > 0 && (double)(s.before + one) < target) {
        n = (uint64_t)ceil((target - (double)s.before) / (double)one);
        // the division may be off by one unit in the last place
        while (n > 1 && (double)(s.before + (n - 1) * one) >= target) --n;
        while ((double)(s.before + n * one) < target && n * one < s.inside) ++n;
      }
      if (!need_k || key > thr || (key == thr && n < quota)) {
        thr = key;
        quota = n;
      }
    }
  }
  if (thr != 0 && weigh.weight(value_of(thr)) < (double)min_p) quota = 0;

  // ---- kept weight of each tile of 64 groups, above the threshold and equal to it
  const uint64_t thr_units = thr != 0 ? Weigh::units(weigh.weight(value_of(thr))) : 0;
  const int tiles = (groups + 63) / 64;
  auto lane_part = [&](int t, uint64_t (&u)[W], bool (&tie)[W]) __attribute__((always_inline)) {
    const int g = t * 64 + lane;
    float x[W];
    if (g < groups) {
      group(g, x);
    } else {
#pragma unroll
      for (int k = 0; k < W; ++k) x[k] = kNegInf;
    }
#pragma unroll
    for (int k = 0; k < W; ++k) {
      u[k] = 0;
      tie[k] = false;
      if (x[k] == kNegInf) continue;
      const uint32_t key = key_of(x[k]);
      tie[k] = key == thr;
      if (key > thr) {
        const double w = weigh.weight(x[k]);
        if (w >= (double)min_p) u[k] = Weigh::units(w);
      }
    }
  };
  for (int t = wave; t < tiles; t += NTHR / 64) {
    uint64_t u[W], sum = 0;
    bool tie[W];
    uint32_t n = 0;
    lane_part(t, u, tie);
#pragma unroll
    for (int k = 0; k < W; ++k) {
      sum += u[k];
      n += tie[k];
    }
    if (__ballot(sum != 0 || n != 0)) {
#pragma unroll
      for (int o = 1; o < 64; o <<= 1) {
        sum += __shfl_xor(sum, o);
        n += __shfl_xor(n, o);
      }
    }
    if (lane == 0) {
      s.tile_w[t] = sum;
      s.tile_n[t] = n;
    }
  }
  __syncthreads();
  if (wave != 0) return;

  // ---- the tile, then the action: lanes hold consecutive tiles
  const int per = (tiles + 63) / 64;
  const int t0 = lane * per < tiles ? lane * per : tiles;
  const int t1 = t0 + per < tiles ? t0 + per : tiles;
  uint64_t ties = 0;
  for (int t = t0; t < t1; ++t) ties += s.tile_n[t];
  uint64_t ties_upto = ties;
#pragma unroll
  for (int o = 1; o < 64; o <<= 1) {
    const uint64_t up = __shfl_up(ties_upto, o);
    if (lane >= o) ties_upto += up;
  }
  // how many of `n` equal ones are kept when `before` lie in front of them
  auto granted = [&](uint64_t before, uint64_t n) __attribute__((always_inline)) {
    const uint64_t left = quota > before ? quota - before : 0;
    return left < n ? left : n;
  };
  uint64_t own = 0, seen = ties_upto - ties;
  for (int t = t0; t < t1; ++t) {
    own += s.tile_w[t] + granted(seen, s.tile_n[t]) * thr_units;
    seen += s.tile_n[t];
  }
  uint64_t upto = own;
#pragma unroll
  for (int o = 1; o < 64; o <<= 1) {
    const uint64_t up = __shfl_up(upto, o);
    if (lane >= o) upto += up;
  }
  const uint64_t total = __shfl(upto, 63);
  const double goal = (double)a.u[r] * (double)total;
  const uint64_t passed = __ballot((double)upto > goal && own > 0);
  const uint64_t filled = __ballot(own > 0);
  const int who = passed ? __ffsll((unsigned long long)passed) - 1 : 63 - __clzll((long long)filled);
  int tile = 0;
  uint64_t sum = upto - own;
  seen = ties_upto - ties;
  if (lane == who) {
    uint64_t at = sum, at_ties = seen;
    for (int t = t0; t < t1; ++t) {
      const uint64_t w = s.tile_w[t] + granted(at_ties, s.tile_n[t]) * thr_units;
      if (w > 0) {
        tile = t;
        sum = at;
        seen = at_ties;
        if ((double)(at + w) > goal) break;
      }
      at += w;
      at_ties += s.tile_n[t];
    }
  }
  tile = __shfl(tile, who);
  sum = __shfl(sum, who);
  seen = __shfl(seen, who);

  uint64_t u[W];
  bool tie[W];
  lane_part(tile, u, tie);
  uint64_t n = 0;
#pragma unroll
  for (int k = 0; k < W; ++k) n += tie[k];
  uint64_t n_upto = n;
#pragma unroll
  for (int o = 1; o < 64; o <<= 1) {
    const uint64_t up = __shfl_up(n_upto, o);
    if (lane >= o) n_upto += up;
  }
  uint64_t before = seen + n_upto - n;
  own = 0;
#pragma unroll
  for (int k = 0; k < W; ++k) {
    if (tie[k]) {
      u[k] = before < quota ? thr_units : 0;
      ++before;
    }
    own += u[k];
  }
  upto = own;
#pragma unroll
  for (int o = 1; o < 64; o <<= 1) {
    const uint64_t up = __shfl_up(upto, o);
    if (lane >= o) upto += up;
  }
  const uint64_t here = __ballot((double)(sum + upto) > goal && own > 0);
  const uint64_t any = __ballot(own > 0);
  const int last = here ? __ffsll((unsigned long long)here) - 1 : 63 - __clzll((long long)any);
  if (lane == last) {
    uint64_t at = sum + upto - own;
    int k_found = 0;
    bool done = false;
#pragma unroll
    for (int k = 0; k < W; ++k) {
      if (done || u[k] == 0) continue;
      k_found = k;
      at += u[k];
      done = (double)at > goal;
    }
    const int i = (tile * 64 + lane) * W - shift + k_found;
    a.action[r] = i;
    if (a.log_prob) {
      const float x = fminf(F::get(row[i]), kMaxFloat);
      a.log_prob[r] = (float)(weigh.log_weight(x) - log((double)total / kUnit));
    }
  }
}

template <class F>
hipError_t sample_fmt(const SampleArgs& a, hipStream_t st) {
  if (a.N <= kSmall) sample_kernel<F, 64><<<dim3((unsigned)a.R), 64, 0, st>>>(a);
  else if (a.N <= kMiddle) sample_kernel<F, 256><<<dim3((unsigned)a.R), 256, 0, st>>>(a);
  else sample_kernel<F, 1024><<<dim3((unsigned)a.R), 1024, 0, st>>>(a);
  return hipGetLastError();
}

hipError_t launch_sample(rlscan_format f, const SampleArgs& a, hipStream_t st) {
  switch (f) {
    case RLSCAN_FORMAT_BF16: return sample_fmt<LBf16>(a, st);
    case RLSCAN_FORMAT_F16: return sample_fmt<LF16>(a, st);
    default: return sample_fmt<LF32>(a, st);
  }
}

}  // namespace logits
}  // namespace rlscan
