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
// the first `quota` of those equal to it.  Long rows go by bins of max - x, which
// spread the LDS atomics (bins of the keys' leading bits put most logits into some fifty:
// twice the time).  A pass after the one for the maximum counts each bin's logits, for
// top_k, which leaves a few hundred that it can keep.  They are collected in LDS, ranked
// against each other, and the rest of the work is on them alone.  Without top_k, or where
// it leaves more, the threshold is searched instead: by the bins' weights, then in the
// one bin that it falls into, each logit against all or by 8-bit digits of the keys; a last
// pass sums the kept weights of tiles of the row, and one wave finds the tile and in it
// the action.  One block takes a row; where rows are few and long, blocks share the passes
// (slice_kernel) and one block for each row makes the choice.
//
// 256 rows of 64007 bfloat16 logits with top_k up to 100: 78 us, of which reading them
// takes 6 and the few rows without a top_k nearly all: two passes with some 40 instructions
// a logit for the float64 exponential, by one compute unit.  One row of 131072 float32
// logits with top_p alone: 3.2, 6.6 and 11.3 us for the three shared passes and 10.7 for the
// choice; a chain of four kernels that each wait for memory a few times (122 us on one
// compute unit).
#include "rlscan_logits.hpp"

namespace rlscan {
namespace logits {

constexpr int kBins = 4096;     // bins of long rows, over 32 temperatures below the maximum
constexpr int kFew = 512;       // logits that are ranked against each other: work grows with the square
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

// e^y for -31 <= y <= 0, to about 2e-16: 2^(n/64) from a table, and the Taylor series
// of the rest, |r| <= ln 2 / 128, to the fifth power.  The whole number n is read from
// a sum's low bits and 2^(n/64)'s exponent added to as an integer.
__device__ __forceinline__ double exp_table(double y, const double* table) {
  constexpr double kWhole = 6755399441055744.0;  // 1.5 * 2^52: sums with it are whole numbers
  const double t = __builtin_fma(y, 64.0 / 0.693147180559945309417, kWhole);
  const double n = t - kWhole;
  double r = __builtin_fma(n, -0x1.62e42fefap-7, y);  // the leading 37 bits of ln 2 / 64: n * it is exact
  r = __builtin_fma(n, -(0x1.62e42fefa39efp-7 - 0x1.62e42fefap-7) - 0x1.abc9e3b39803fp-62, r);
  double p = __builtin_fma(r, 1.0 / 120.0, 1.0 / 24.0);
  p = __builtin_fma(p, r, 1.0 / 6.0);
  p = __builtin_fma(p, r, 0.5);
  p = __builtin_fma(p, r, 1.0);
  p = __builtin_fma(p, r, 1.0);
  const int i = (int)(uint32_t)__builtin_bit_cast(uint64_t, t);
  const uint64_t scale = __builtin_bit_cast(uint64_t, table[i & 63]) + ((uint64_t)(uint32_t)(i >> 6) << 52);
  return p * __builtin_bit_cast(double, scale);
}

struct Weigh {
  double max, inv_t;
  const double* table;
  __device__ __forceinline__ double log_weight(float x) const { return ((double)x - max) * inv_t; }
  // A weight as a float64, 0 where it rounds to no unit.  No branch: the weights of a
  // group are computed side by side (131072 of them by one CU with their sums by bins:
  // 84 thousand clocks; 92 with a branch around each).
  __device__ __forceinline__ double weight(float x) const {
    const double y = log_weight(x);
    const double w = exp_table(fmax(y, -31.0), table);
    return y < -31.0 ? 0.0 : w;
  }
  // in units
  static __device__ __forceinline__ double whole(double w) {
    return __builtin_fma(w, kUnit, 4503599627370496.0) - 4503599627370496.0;
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
  uint64_t few[kFew];    // key << 32 | ~index: falling order is that of these numbers
  uint64_t sorted[kFew];
  uint64_t kept[kFew];   // units, in falling order
  uint32_t rank[kFew];
  int last;              // how many are kept
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

// The wave's sum, in lane 63.
template <int CTRL, int ROWS>
__device__ __forceinline__ double add_from(double v) {
  const uint64_t b = __builtin_bit_cast(uint64_t, v);
  const uint32_t lo = __builtin_amdgcn_update_dpp(0, (int)(uint32_t)b, CTRL, ROWS, 0xf, false);
  const uint32_t hi = __builtin_amdgcn_update_dpp(0, (int)(uint32_t)(b >> 32), CTRL, ROWS, 0xf, false);
  return v + __builtin_bit_cast(double, (uint64_t)hi << 32 | lo);
}
__device__ __forceinline__ double wave_sum_last(double v) {
  v = add_from<0x111, 0xf>(v);  // row_shr:1
  v = add_from<0x112, 0xf>(v);
  v = add_from<0x114, 0xf>(v);
  v = add_from<0x118, 0xf>(v);
  v = add_from<0x142, 0xa>(v);  // row_bcast:15
  return add_from<0x143, 0xc>(v);  // row_bcast:31
}

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
// whole block, n / PER threads with PER bins each; the last bin with anything in it if none
// does.  Results in s.bin, s.before (sum before the bin, with `base`) and s.inside (its own).
template <int NTHR, int PER, class V>
__device__ __forceinline__ void search_bins(SampleLds<NTHR>& s, const V* bins, int n, uint64_t base, double target,
                                            bool falling) {
  const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
  const bool has = tid * PER < n;
  __syncthreads();  // the bins are filled
  V v[PER];
  uint64_t own = 0;
#pragma unroll
  for (int i = 0; i < PER; ++i) {
    const int b = tid * PER + i;
    v[i] = 0;
    if (has) v[i] = bins[falling ? n - 1 - b : b];
    own += v[i];
  }
  uint64_t upto = own;
#pragma unroll
  for (int o = 1; o < 64; o <<= 1) {
    const uint64_t up = __shfl_up(upto, o);
    if (lane >= o) upto += up;
  }
  if (lane == 63) s.red[wave] = upto;
  if (tid == 0) s.bin = -1;
  __syncthreads();
  uint64_t before = base, total = base;
  int last_wave = 0;  // with anything in it
#pragma unroll
  for (int i = 0; i < NTHR / 64; ++i) {
    if (i < wave) before += s.red[i];
    total += s.red[i];
    if (s.red[i] > 0) last_wave = i;
  }
  before += upto - own;
  const uint64_t filled = __ballot(own > 0);
  const bool reaches = (double)total >= target;
  const bool here = reaches ? (double)before < target && (double)(before + own) >= target
                            : wave == last_wave && filled && lane == 63 - __clzll((long long)filled);
  if (here) {
    uint64_t sum = before;
#pragma unroll
    for (int i = 0; i < PER; ++i) {
      if (v[i] == 0 || (s.bin >= 0 && (double)sum >= target)) continue;
      s.bin = falling ? n - 1 - (tid * PER + i) : tid * PER + i;
      s.before = sum;
      s.inside = v[i];
      sum += v[i];
    }
  }
  __syncthreads();
}

// What a prefix must reach to have top_p of the weight.
__device__ __forceinline__ double weight_target(uint64_t kept, float top_p) {
  const double target = (double)top_p * (double)kept;
  return target >= 1.0 ? target : 1.0;  // the largest is always kept
}

// Searches the bins' weights for the bin in which the target is reached.
__device__ __forceinline__ void cut_weight(SampleLds<1024>& s, uint64_t kept, float top_p) {
  search_bins<1024, 4>(s, s.coarse_w, kBins, 0, weight_target(kept, top_p), false);
}

// The rest of a row's work on the n <= kFew logits in s.few, by the whole block.
template <class F, int NTHR>
__device__ __forceinline__ void take_few(SampleLds<NTHR>& s, const SampleArgs& a, int64_t r, const Weigh& weigh, int n,
                                         int top_k, float top_p, float min_p) {
  const int tid = threadIdx.x, lane = tid & 63;
  // each logit's place in falling order: how many come before it.  `share` threads compare one.
  int share = 1;
  while (share * 2 * n <= NTHR && share < 64) share *= 2;
  for (int i = tid; i < n; i += NTHR) s.rank[i] = 0;
  __syncthreads();
  for (int i = tid / share; i < n; i += NTHR / share) {
    const uint64_t mine = s.few[i];
    uint32_t before = 0;
    for (int j = tid % share; j < n; j += share) before += s.few[j] > mine;
    if (before) atomicAdd(&s.rank[i], before);
  }
  __syncthreads();
  for (int i = tid; i < n; i += NTHR) s.sorted[s.rank[i]] = s.few[i];
  __syncthreads();
  if (tid < 64) {  // one wave: consecutive places per lane
    const int per = (n + 63) / 64, i0 = lane * per < n ? lane * per : n, i1 = i0 + per < n ? i0 + per : n;
    uint64_t own = 0;
    for (int i = i0; i < i1; ++i) {
      const double w = i < top_k ? weigh.weight(value_of((uint32_t)(s.sorted[i] >> 32))) : 0.0;
      s.kept[i] = Weigh::units(w);
      own += s.kept[i];
    }
    uint64_t upto = own;
#pragma unroll
    for (int o = 1; o < 64; o <<= 1) {
      const uint64_t up = __shfl_up(upto, o);
      if (lane >= o) upto += up;
    }
    const uint64_t total = __shfl(upto, 63);
    double target = top_p < 1.0f ? (double)top_p * (double)total : (double)total;
    if (!(target >= 1.0)) target = 1.0;  // the largest is always kept
    uint64_t before = upto - own;
    int last = 0;
    for (int i = i0; i < i1; ++i) {
      const uint64_t u = s.kept[i];
      const bool keep = i < top_k && (double)before < target &&
                        weigh.weight(value_of((uint32_t)(s.sorted[i] >> 32))) >= (double)min_p;
      before += u;
      if (keep) last = i + 1;  // what is kept is a prefix
    }
#pragma unroll
    for (int o = 1; o < 64; o <<= 1) {
      const int other = __shfl_xor(last, o);
      last = other > last ? other : last;
    }
    if (lane == 0) s.last = last;
  }
  __syncthreads();
  // the running weight in the order of the indices, of each that is kept
  const int m = s.last;
  uint64_t total = 0;
  for (int j = 0; j < m; ++j) total += s.kept[j];
  const double goal = (double)a.u[r] * (double)total;
  for (int i = tid; i < m; i += NTHR) {
    const uint32_t mine = ~(uint32_t)s.sorted[i];
    uint64_t before = 0;
    bool none_after = true;
    for (int j = 0; j < m; ++j) {
      const uint32_t other = ~(uint32_t)s.sorted[j];
      if (other < mine) before += s.kept[j];
      none_after &= !(other > mine && s.kept[j] > 0);
    }
    const uint64_t own = s.kept[i];
    // the first that passes the goal; the last with any weight if none does (u >= 1)
    const bool reached = own > 0 && (double)(before + own) > goal;
    const bool first = !((double)before > goal) || before == 0;
    if ((reached && first) || (own > 0 && !reached && none_after)) {
      a.action[r] = (int64_t)mine;
      if (a.log_prob)
        a.log_prob[r] = (float)(weigh.log_weight(value_of((uint32_t)(s.sorted[i] >> 32))) - log((double)total / kUnit));
    }
  }
}

// A row of logits and its settings.
template <class F>
struct Row {
  static constexpr int W = F::W;
  const typename F::E* row;
  const uint8_t* mask;
  int N, shift, groups;  // groups of W logits on 16-byte boundaries; the row begins `shift` into the first
  float temperature, top_p, min_p;
  int top_k;
  __device__ __forceinline__ Row(const SampleArgs& a, int64_t r) {
    row = static_cast<const typename F::E*>(a.x) + r * a.stride;
    mask = a.mask ? a.mask + r * a.N : nullptr;
    N = (int)a.N;
    shift = (int)(((uintptr_t)row / sizeof(typename F::E)) % W);
    groups = (N + shift + W - 1) / W;
    temperature = a.temperature ? a.temperature[r] : a.temperature1;
    top_k = a.top_k ? a.top_k[r] : a.top_k1;
    top_p = a.top_p ? a.top_p[r] : a.top_p1;
    min_p = a.min_p ? a.min_p[r] : a.min_p1;
    if (!(temperature > 0.0f)) {  // greedy: the largest logit, lowest index first
      temperature = 1.0f;
      top_k = 1;
    }
    min_p = min_p > 0.0f ? fminf(min_p, 1.0f) : 0.0f;
  }
  // NaN is not legal; +inf counts as the largest float
  static __device__ __forceinline__ float legal(float x) { return x > kNegInf ? fminf(x, kMaxFloat) : kNegInf; }
  // the logits of group g, -inf where not legal or outside the row
  __device__ __forceinline__ void group(int g, float (&x)[W]) const {
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
      if (mask && i + k >= 0 && i + k < N && mask[i + k] == 0) x[k] = kNegInf;
      x[k] = legal(x[k]);
    }
  }
  // bins of 32 temperatures below the maximum; lower logits share the last
  __device__ __forceinline__ float per_bin() const { return fminf((float)kBins / (32.0f * temperature), 1e30f); }
  static __device__ __forceinline__ int bin(float top, float per, float x) {
    return (int)fminf((top - x) * per, (float)(kBins - 1));
  }
};

// What the blocks of a shared row leave in the workspace for each other.
struct Shared {
  uint64_t* w;       // [kBins] the bins' weight, where top_p is on and top_k is not
  uint64_t* list;    // [kMiddle] key << 32 | ~index
  uint32_t* n;       // [kBins] logits in each bin, where top_k is on
  uint64_t* tile;    // [tiles] kept weight, without what is in the list
  float* top;        // [slices] largest logit
  uint32_t* listed;  // [1] logits that belong in the list
  uint64_t* cut;     // [3] top_k: candidates, 0 if the list does not hold them; else the bin that
                     // top_p cuts, the weight before it and the row's
  static int64_t words(int64_t tiles, int64_t slices) {  // of 8 bytes, for one row
    return kBins + kMiddle + kBins / 2 + 3 + tiles + (slices + 2) / 2;
  }
  __device__ __forceinline__ Shared(const SampleArgs& a, int64_t r) {
    w = static_cast<uint64_t*>(a.shared) + r * a.shared_words;
    list = w + kBins;
    n = reinterpret_cast<uint32_t*>(list + kMiddle);
    cut = reinterpret_cast<uint64_t*>(n + kBins);
    tile = cut + 3;
    top = reinterpret_cast<float*>(tile + a.tiles);
    listed = reinterpret_cast<uint32_t*>(top + a.slices);
  }
};

// The passes over a shared row, `slices` blocks a row, each over a.slice_tiles tiles:
// 0, the maximum; 1, the bins; 2, the kept weight of tiles and the logits of the bin
// that is cut (with a top_k, the logits down to that bin).
template <class F, int STAGE>
__global__ void __launch_bounds__(1024) slice_kernel(const SampleArgs a) {
  constexpr int W = F::W, NTHR = 1024;
  __shared__ SampleLds<NTHR> s;
  const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
  const int64_t r = blockIdx.x / a.slices;
  const int slice = (int)(blockIdx.x % a.slices);
  const Row<F> in(a, r);
  const Shared sh(a, r);
  const int tiles = (in.groups + 63) / 64, t0 = slice * a.slice_tiles;
  const int t1 = t0 + a.slice_tiles < tiles ? t0 + a.slice_tiles : tiles;
  float top = kNegInf;
  if constexpr (STAGE == 0) {
    for (int i = slice * NTHR + tid; i < kBins; i += a.slices * NTHR) {
      sh.w[i] = 0;
      sh.n[i] = 0;
    }
    if (slice == 0 && tid == 0) *sh.listed = 0;
    for (int t = t0 + wave; t < t1; t += NTHR / 64) {
      const int g = t * 64 + lane;
      if (g >= in.groups) break;
      float x[W];
      in.group(g, x);
#pragma unroll
      for (int k = 0; k < W; ++k) top = fmaxf(top, x[k]);
    }
#pragma unroll
    for (int o = 1; o < 64; o <<= 1) top = fmaxf(top, __shfl_xor(top, o));
    if (lane == 0) s.redf[wave] = top;
    __syncthreads();
    for (int n = 0; n < NTHR / 64; ++n) top = fmaxf(top, s.redf[n]);
    if (tid == 0) sh.top[slice] = top;
  } else {
    for (int i = 0; i < a.slices; ++i) top = fmaxf(top, sh.top[i]);
    if (top == kNegInf) return;  // no legal action: the whole block leaves
    const bool need_k = in.top_k > 0 && in.top_k < in.N, need_p = in.top_p < 1.0f;
    if (tid < 64) s.table[tid] = exp2((double)tid / 64.0);
    const Weigh weigh{(double)top, 1.0 / (double)in.temperature, s.table};
    const float per = in.per_bin();
    if constexpr (STAGE == 1) {
      if (!need_k && !need_p) return;
      for (int i = tid; i < kBins; i += NTHR) {
        s.coarse_n[i] = 0;
        s.coarse_w[i] = 0;
      }
      __syncthreads();
      for (int t = t0 + wave; t < t1; t += NTHR / 64) {
        const int g = t * 64 + lane;
        if (g >= in.groups) break;
        float x[W];
        in.group(g, x);
        if (need_k) {
#pragma unroll
          for (int k = 0; k < W; ++k)
            if (x[k] != kNegInf) atomicAdd(&s.coarse_n[Row<F>::bin(top, per, x[k])], 1u);
        } else {
          uint64_t u[W];
#pragma unroll
          for (int k = 0; k < W; ++k) u[k] = Weigh::units(weigh.weight(x[k]));
#pragma unroll
          for (int k = 0; k < W; ++k)
            if (u[k]) atomicAdd((unsigned long long*)&s.coarse_w[Row<F>::bin(top, per, x[k])], (unsigned long long)u[k]);
        }
      }
      __syncthreads();
      for (int i = tid; i < kBins; i += NTHR) {
        if (s.coarse_n[i]) atomicAdd(&sh.n[i], s.coarse_n[i]);
        if (s.coarse_w[i]) atomicAdd((unsigned long long*)&sh.w[i], (unsigned long long)s.coarse_w[i]);
      }
    } else {
      int cut = kBins;
      if (need_k) {
        for (int i = tid; i < kBins; i += NTHR) s.coarse_n[i] = sh.n[i];
        search_bins<NTHR, 4>(s, s.coarse_n, kBins, 0, (double)in.top_k, false);
        const uint64_t candidates = s.before + s.inside;
        const bool listed = candidates >= (uint64_t)in.top_k && candidates <= (uint64_t)kFew;
        if (slice == 0 && tid == 0) sh.cut[0] = listed ? candidates : 0;
        if (!listed) return;  // passed over again
        cut = s.bin;
      } else if (need_p) {
        uint64_t w = 0;
        for (int i = tid; i < kBins; i += NTHR) w += s.coarse_w[i] = sh.w[i];
        const uint64_t kept = block_sum<NTHR>(w, s.red);
        cut_weight(s, kept, in.top_p);
        cut = s.bin;
        if (slice == 0 && tid == 0) {
          sh.cut[0] = (uint64_t)cut;
          sh.cut[1] = s.before;
          sh.cut[2] = kept;
        }
      }
      __syncthreads();
      for (int t = t0 + wave; t < t1; t += NTHR / 64) {
        const int g = t * 64 + lane;
        float x[W];
        if (g < in.groups) {
          in.group(g, x);
        } else {
#pragma unroll
          for (int k = 0; k < W; ++k) x[k] = kNegInf;
        }
        double sum = 0.0;  // in units, below 2^53 for a tile: a whole number
#pragma unroll
        for (int k = 0; k < W; ++k) {
          const int b = Row<F>::bin(top, per, x[k]);
          const bool valid = x[k] != kNegInf;
          if (need_k || need_p) {
            if (valid && (need_k ? b <= cut : b == cut)) {
              const uint32_t at = atomicAdd(sh.listed, 1u);
              if (at < (uint32_t)kMiddle) sh.list[at] = (uint64_t)key_of(x[k]) << 32 | (uint32_t)~(g * W - in.shift + k);
            }
          }
          const double w = weigh.weight(x[k]);
          sum += valid && b < cut && w >= (double)in.min_p ? Weigh::whole(w) : 0.0;
        }
        if (!need_k) {
          sum = wave_sum_last(sum);
          if (lane == 63) sh.tile[t] = (uint64_t)sum;
        }
      }
    }
  }
}

// SHARED: slice_kernel has passed over the row, and what it left in the workspace is
// taken; where that is not enough (a list that does not hold a bin, more than kFew
// candidates of a top_k) the row is passed over again as without.
template <class F, int NTHR, bool SHARED>
__global__ void __launch_bounds__(NTHR) sample_kernel(const SampleArgs a) {
  constexpr int W = F::W;
  __shared__ SampleLds<NTHR> s;
  const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
  const int64_t r = blockIdx.x;
  const Row<F> in(a, r);
  const auto* row = in.row;
  const bool mask = in.mask != nullptr;
  const int N = in.N, shift = in.shift, groups = in.groups;
  const float temperature = in.temperature, top_p = in.top_p, min_p = in.min_p;
  const int top_k = in.top_k;
  auto legal = [](float x) __attribute__((always_inline)) { return Row<F>::legal(x); };
  auto group = [&](int g, float (&x)[W]) __attribute__((always_inline)) { in.group(g, x); };
  // Calls fn(g, x) for each of the thread's groups.  Unmasked long rows ask for 64 bytes
  // at a time (one row of 131072 float32 logits: 121 us; 134 with 16 bytes).
  auto each_group = [&](auto fn) __attribute__((always_inline)) {
    constexpr int kAhead = 16 / W;
    int g = tid;
    if (NTHR == 1024 && !mask) {
      if (g == 0) {  // it may begin before the row
        float x[W];
        group(g, x);
        fn(g, x);
        g += NTHR;
      }
      const int inside = (N + shift) / W;  // groups that end within the row
      for (; g + (kAhead - 1) * NTHR < inside; g += kAhead * NTHR) {
        Vec<F> v[kAhead];
#pragma unroll
        for (int j = 0; j < kAhead; ++j) v[j].w = *reinterpret_cast<const u32x4*>(row + ((g + j * NTHR) * W - shift));
#pragma unroll
        for (int j = 0; j < kAhead; ++j) {
          float x[W];
#pragma unroll
          for (int k = 0; k < W; ++k) x[k] = legal(F::get(v[j].e[k]));
          fn(g + j * NTHR, x);
        }
      }
    }
    for (; g < groups; g += NTHR) {
      float x[W];
      group(g, x);
      fn(g, x);
    }
  };

  constexpr bool coarse = SampleLds<NTHR>::kCoarse;
  constexpr int kList = SampleLds<NTHR>::kList;
  bool need_k = top_k > 0 && top_k < N;
  const bool need_p = top_p < 1.0f;

  // ---- maximum
  float top = kNegInf;
  const Shared sh(a, r);
  bool taken = SHARED && !need_k;  // the tiles' weights, and the list, are in the workspace
  if (SHARED) {
    for (int i = tid; i < a.slices; i += NTHR) top = fmaxf(top, sh.top[i]);
  } else {
    each_group([&](int, float (&x)[W]) __attribute__((always_inline)) {
#pragma unroll
      for (int k = 0; k < W; ++k) top = fmaxf(top, x[k]);
    });
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
  uint32_t thr = 0;
  uint64_t quota = ~0ull;
  if (need_k || need_p) {
    uint64_t before_k = 0;  // logits in the bins before the one that top_k cuts
    int bin_k = kBins;
    const float per = in.per_bin();
    auto bin_of = [&](float x) __attribute__((always_inline)) { return Row<F>::bin(top, per, x); };
    const uint64_t shared_few = SHARED && need_k ? sh.cut[0] : 0;
    if (coarse && need_k && shared_few == 0) {
      for (int i = tid; i < kBins; i += NTHR) s.coarse_n[i] = SHARED ? sh.n[i] : 0;
      __syncthreads();
      if (!SHARED) {
        each_group([&](int, float (&x)[W]) __attribute__((always_inline)) {
#pragma unroll
          for (int k = 0; k < W; ++k)
            if (x[k] != kNegInf) atomicAdd(&s.coarse_n[bin_of(x[k])], 1u);
        });
      }
      search_bins<NTHR, 4>(s, s.coarse_n, kBins, 0, (double)top_k, false);
      before_k = s.before;
      bin_k = s.bin;
      need_k = s.before + s.inside >= (uint64_t)top_k;
    }
    const uint64_t candidates = shared_few ? shared_few : coarse && need_k ? before_k + s.inside : (uint64_t)N;
    if (candidates <= (uint64_t)kFew) {
      __syncthreads();
      if (tid == 0) s.count = 0;
      __syncthreads();
      if (SHARED) {
        if (tid == 0) s.count = (uint32_t)candidates;
        for (int i = tid; i < (int)candidates; i += NTHR) s.few[i] = sh.list[i];
      } else {
        each_group([&](int g, float (&x)[W]) __attribute__((always_inline)) {
#pragma unroll
          for (int k = 0; k < W; ++k) {
            if (x[k] == kNegInf || (coarse && need_k && bin_of(x[k]) > bin_k)) continue;
            const uint32_t at = atomicAdd(&s.count, 1u);  // at most kFew: the bins were counted
            if (at < (uint32_t)kFew) s.few[at] = (uint64_t)key_of(x[k]) << 32 | (uint32_t)~(g * W - shift + k);
          }
        });
      }
      __syncthreads();
      const int n = (int)s.count < kFew ? (int)s.count : kFew;
      take_few<F, NTHR>(s, a, r, weigh, n, need_k ? top_k : n, top_p, min_p);
      return;
    }
    if (coarse && need_p && !taken) {
      for (int i = tid; i < kBins; i += NTHR) s.coarse_w[i] = 0;
      __syncthreads();
      each_group([&](int, float (&x)[W]) __attribute__((always_inline)) {
        uint64_t u[W];
#pragma unroll
        for (int k = 0; k < W; ++k) u[k] = Weigh::units(weigh.weight(x[k]));
#pragma unroll
        for (int k = 0; k < W; ++k) {
          if (u[k]) atomicAdd((unsigned long long*)&s.coarse_w[bin_of(x[k])], (unsigned long long)u[k]);
        }
      });
      __syncthreads();
    }

    int held = -2;  // the bin whose keys are in the list; -1: the whole row
    bool in_list = false;
    // Calls fn(key) for each logit of a bin (-1: of the row).
    auto collect = [&](int bin) __attribute__((always_inline)) {
      if (held == bin) return;
      __syncthreads();
      if (SHARED && taken) {
        taken = *sh.listed <= (uint32_t)kList;
        if (taken) {
          if (tid == 0) s.count = *sh.listed;
          for (int i = tid; i < (int)*sh.listed; i += NTHR) s.list[i] = (uint32_t)(sh.list[i] >> 32);
          __syncthreads();
          held = bin;
          in_list = true;
          return;
        }
      }
      if (tid == 0) s.count = 0;
      __syncthreads();
      each_group([&](int, float (&x)[W]) __attribute__((always_inline)) {
#pragma unroll
        for (int k = 0; k < W; ++k) {
          if (x[k] == kNegInf || (bin >= 0 && bin_of(x[k]) != bin)) continue;
          const uint32_t at = atomicAdd(&s.count, 1u);
          if (at < (uint32_t)kList) s.list[at] = key_of(x[k]);
        }
      });
      __syncthreads();
      held = bin;
      in_list = s.count <= (uint32_t)kList;
    };
    auto each = [&](auto fn) __attribute__((always_inline)) {
      if (in_list) {
        const int n = (int)s.count;
        for (int i = tid; i < n; i += NTHR) fn(s.list[i]);
      } else {
        each_group([&](int, float (&x)[W]) __attribute__((always_inline)) {
#pragma unroll
          for (int k = 0; k < W; ++k)
            if (x[k] != kNegInf && (held < 0 || bin_of(x[k]) == held)) fn(key_of(x[k]));
        });
      }
    };
    // Within the held bin: the key at which the running sum (of 1 for each logit, or
    // of its weight) reaches target, from `base`; leaves the sum before that key in
    // s.before and that of all logits equal to it in s.inside.
    auto descend = [&](bool weights, uint64_t base, double target) __attribute__((always_inline)) {
      if (in_list && s.count <= (uint32_t)kFew) {  // each against all, at once
        const int n = (int)s.count;
        for (int i = tid; i < n; i += NTHR) s.kept[i] = weights ? Weigh::units(weigh.weight(value_of(s.list[i]))) : 1;
        __syncthreads();
        for (int i = tid; i < n; i += NTHR) {
          const uint32_t mine = s.list[i];
          uint64_t above = base, same = 0, below = 0;
          for (int j = 0; j < n; ++j) {
            const uint32_t key = s.list[j];
            const uint64_t v = s.kept[j];
            above += key > mine ? v : 0;
            same += key == mine ? v : 0;
            below += key < mine ? v : 0;
          }
          // the last key with anything if none reaches it
          const bool reaches = (double)above < target && (double)(above + same) >= target;
          if (reaches || (same > 0 && below == 0 && (double)(above + same) < target)) {
            s.rank[0] = mine;
            s.before = above;
            s.inside = same;
          }
        }
        __syncthreads();
        return s.rank[0];
      }
      uint32_t prefix = 0, known = 0;
      // the bits below the format's own are equal in all keys, but for what +inf counts as
      const uint32_t infinite = key_of(kMaxFloat);
#pragma unroll 1
      for (int d = 24; d >= 0 && (d + 8 > F::kLow || prefix == (infinite & known)); d -= 8) {
        for (int i = tid; i < 256; i += NTHR) s.hist[i] = 0;
        __syncthreads();
        each([&](uint32_t key) __attribute__((always_inline)) {
          if ((key & known) != prefix) return;
          const uint64_t v = weights ? Weigh::units(weigh.weight(value_of(key))) : 1;
          if (v) atomicAdd((unsigned long long*)&s.hist[key >> d & 255], (unsigned long long)v);
        });
        search_bins<NTHR, NTHR < 256 ? 256 / NTHR : 1>(s, s.hist, 256, base, target, true);
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
    if (need_k) {
      collect(coarse ? bin_k : -1);
      if (!coarse) need_k = s.count > (uint32_t)top_k;
      if (need_k) {
        thr = descend(false, before_k, (double)top_k);
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
      if (SHARED && taken) {
        kept = sh.cut[2];
      } else if (!need_k) {
        uint64_t w = 0;
        if (coarse) {
          for (int i = tid; i < kBins; i += NTHR) w += s.coarse_w[i];
        } else {
          collect(-1);
          each([&](uint32_t key) __attribute__((always_inline)) { w += Weigh::units(weigh.weight(value_of(key))); });
        }
        kept = block_sum<NTHR>(w, s.red);
      }
      const double target = weight_target(kept, top_p);
      if constexpr (coarse) {
        if (SHARED && taken) {
          bin = (int)sh.cut[0];
          base = sh.cut[1];
        } else if (need_k && (double)kept_before < target) {
          bin = bin_k;
          base = kept_before;
        } else {
          cut_weight(s, kept, top_p);
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
      const bool valid = x[k] != kNegInf;
      const uint32_t key = key_of(x[k]);
      tie[k] = valid && key == thr;
      const double w = weigh.weight(x[k]);
      if (valid && key > thr && w >= (double)min_p) u[k] = Weigh::units(w);
    }
  };
  if (SHARED && taken) {
    for (int t = tid; t < tiles; t += NTHR) {
      s.tile_w[t] = sh.tile[t];
      s.tile_n[t] = 0;
    }
    __syncthreads();
    const int listed = need_p ? (int)*sh.listed : 0;
    for (int i = tid; i < listed; i += NTHR) {
      const uint32_t key = (uint32_t)(sh.list[i] >> 32);
      const int t = ((int)~(uint32_t)sh.list[i] + shift) / W / 64;
      const double w = weigh.weight(value_of(key));
      if (key > thr && w >= (double)min_p) atomicAdd((unsigned long long*)&s.tile_w[t], (unsigned long long)Weigh::units(w));
      if (key == thr) atomicAdd(&s.tile_n[t], 1u);
    }
  } else {
    Vec<F> ahead;  // of the next tile, where it lies within an unmasked row
    auto inside = [&](int t) __attribute__((always_inline)) { return !mask && t > 0 && (t + 1) * 64 * W - shift <= N; };
    auto ask = [&](int t) __attribute__((always_inline)) {
      if (inside(t)) ahead.w = *reinterpret_cast<const u32x4*>(row + ((t * 64 + lane) * W - shift));
    };
    ask(wave);
    for (int t = wave; t < tiles; t += NTHR / 64) {
      const int g = t * 64 + lane;
      float x[W];
      if (inside(t)) {
#pragma unroll
        for (int k = 0; k < W; ++k) x[k] = legal(F::get(ahead.e[k]));
      } else if (g < groups) {
        group(g, x);
      } else {
#pragma unroll
        for (int k = 0; k < W; ++k) x[k] = kNegInf;
      }
      ask(t + NTHR / 64);
      uint32_t ties = 0;
      bool above[W], some = false;
#pragma unroll
      for (int k = 0; k < W; ++k) {
        const uint32_t key = key_of(x[k]);
        const bool valid = x[k] != kNegInf;
        above[k] = valid && key > thr;
        some |= above[k];
        ties += __popcll(__ballot(valid && key == thr));
      }
      double sum = 0.0;  // in units, below 2^53 for a tile: a whole number
      if (__ballot(some)) {
#pragma unroll
        for (int k = 0; k < W; ++k) {
          const double w = weigh.weight(x[k]);
          sum += above[k] && w >= (double)min_p ? Weigh::whole(w) : 0.0;
        }
        sum = wave_sum_last(sum);
      }
      if (lane == 63) {
        s.tile_w[t] = (uint64_t)sum;
        s.tile_n[t] = ties;
      }
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

// Blocks that share a row.  Where rows are few and long, the compute units that they leave
// idle pay for three more launches.  One block a row against shared, us: one row of
// 131072 float32, top_p 0.9: 122, 36.  Bfloat16, top_p 0.9, then top_k 50: 64 rows of
// 64007: 74, 45 and 35, 35; 128 rows: 76, 99 and 36, 75; 64 rows of 32768: 43, 38 and
// 24, 33 (which settings a row has is known on the device only); of 8192: 26, 40 and 19, 33.
// Every pass holds the whole of SampleLds, 131,832 bytes, so one block to a compute unit,
// and rows with a top_k are shared too.
int64_t sample_slices(int64_t R, int64_t N) {
  return R < 1 || R > 64 || N < 32768 ? 1 : 256 / R < N / 4096 ? 256 / R : N / 4096;
}

// Groups of a row that begins anywhere, in tiles of 64.
static int64_t tiles_of(int64_t N, int W) { return (((N + 2 * (W - 1)) / W) + 63) / 64; }

int64_t sample_workspace(int64_t R, int64_t N) {
  const int64_t slices = sample_slices(R, N);
  return slices > 1 ? R * Shared::words(tiles_of(N, 4), slices) * 8 : 0;
}

template <class F>
hipError_t sample_fmt(const SampleArgs& given, hipStream_t st) {
  SampleArgs a = given;
  a.slices = a.shared ? (int)sample_slices(a.R, a.N) : 1;
  if (a.slices > 1) {
    a.tiles = (int)tiles_of(a.N, F::W);
    a.slice_tiles = (a.tiles + a.slices - 1) / a.slices;
    a.shared_words = Shared::words(a.tiles, a.slices);
    const dim3 grid((unsigned)(a.R * a.slices));
    slice_kernel<F, 0><<<grid, 1024, 0, st>>>(a);
    slice_kernel<F, 1><<<grid, 1024, 0, st>>>(a);
    slice_kernel<F, 2><<<grid, 1024, 0, st>>>(a);
    sample_kernel<F, 1024, true><<<dim3((unsigned)a.R), 1024, 0, st>>>(a);
  } else if (a.N <= kSmall) {
    sample_kernel<F, 64, false><<<dim3((unsigned)a.R), 64, 0, st>>>(a);
  } else if (a.N <= kMiddle) {
    sample_kernel<F, 256, false><<<dim3((unsigned)a.R), 256, 0, st>>>(a);
  } else {
    sample_kernel<F, 1024, false><<<dim3((unsigned)a.R), 1024, 0, st>>>(a);
  }
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
