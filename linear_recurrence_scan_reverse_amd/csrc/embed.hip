// Rows of a table by token (rlscan_embed_tokens) and the table's gradient
// (rlscan_embed_tokens_backward).
//
//   out_r = scale table[token_r],   d_table_n = scale sum over token_r = n of d_out_r
//
// Both are bound by memory.  For the gradient the tokens are sorted (stable, by one or two
// digits of up to ten bits), so that a row's terms follow one another in the order of the
// tokens: chunks of sorted tokens are summed by a wave each, and what passes a chunk's border is
// joined afterwards, in order.  No atomics on values: results do not vary from run to run.
#include "rlscan_embed.hpp"

namespace rlscan {
namespace embed {

using logits::LBf16;
using logits::LF16;
using logits::LF32;

// V elements as they lie in memory: 16 bytes, or one element.
template <class F, int V>
struct Piece {
  typename F::E e[V];
};
template <class F, int V>
__device__ __forceinline__ Piece<F, V> load_piece(const typename F::E* p) {
  Piece<F, V> r;
  if constexpr (V == 1) {
    r.e[0] = *p;
  } else {
    const logits::u32x4 v = *reinterpret_cast<const logits::u32x4*>(p);
    __builtin_memcpy(&r, &v, 16);
  }
  return r;
}
template <class F, int V>
__device__ __forceinline__ void store_piece(typename F::E* p, const float (&x)[V]) {
  Piece<F, V> r;
#pragma unroll
  for (int i = 0; i < V; ++i) r.e[i] = F::put(x[i]);
  if constexpr (V == 1) {
    *p = r.e[0];
  } else {
    logits::u32x4 v;
    __builtin_memcpy(&v, &r, 16);
    *reinterpret_cast<logits::u32x4*>(p) = v;
  }
}

// A wave takes 64 V columns of one token.
template <class F, int V>
__global__ void __launch_bounds__(256) lookup_kernel(const LookupArgs p, int64_t tiles) {
  using E = typename F::E;
  const int64_t u = (int64_t)blockIdx.x * 4 + (threadIdx.x >> 6);
  const int64_t r = u / tiles, d = (u - r * tiles) * 64 * V + (threadIdx.x & 63) * V;
  if (r >= p.R || d >= p.D) return;
  const int64_t n = p.tokens[r];
  float x[V];
#pragma unroll
  for (int i = 0; i < V; ++i) x[i] = 0.0f;
  if (n >= 0 && n < p.N) {
    const Piece<F, V> w = load_piece<F, V>(static_cast<const E*>(p.table) + n * p.t_stride + d);
#pragma unroll
    for (int i = 0; i < V; ++i) x[i] = p.scale * F::get(w.e[i]);
  }
  store_piece<F, V>(static_cast<E*>(p.out) + r * p.o_stride + d, x);
}

static bool wide(const void* a, int64_t sa, const void* b, int64_t sb, int64_t D, int V, int es) {
  return D % V == 0 && (uintptr_t)a % 16 == 0 && (uintptr_t)b % 16 == 0 && sa * es % 16 == 0 && sb * es % 16 == 0;
}

template <class F>
static hipError_t lookup_fmt(const LookupArgs& a, hipStream_t st) {
  constexpr int V = F::W, es = sizeof(typename F::E);
  if (wide(a.table, a.t_stride, a.out, a.o_stride, a.D, V, es)) {
    const int64_t tiles = (a.D + 64 * V - 1) / (64 * V);
    lookup_kernel<F, V><<<dim3((unsigned)((a.R * tiles + 3) / 4)), 256, 0, st>>>(a, tiles);
  } else {
    const int64_t tiles = (a.D + 63) / 64;
    lookup_kernel<F, 1><<<dim3((unsigned)((a.R * tiles + 3) / 4)), 256, 0, st>>>(a, tiles);
  }
  return hipGetLastError();
}

hipError_t launch_lookup(rlscan_format f, const LookupArgs& a, hipStream_t st) {
  switch (f) {
    case RLSCAN_FORMAT_BF16: return lookup_fmt<LBf16>(a, st);
    case RLSCAN_FORMAT_F16: return lookup_fmt<LF16>(a, st);
    default: return lookup_fmt<LF32>(a, st);
  }
}

// ------------------------------------------------------------------ sorting the tokens
constexpr int kBins = 1024;
constexpr int kSortThreads = 1024, kSortWaves = kSortThreads / 64;

struct SortArgs {
  const int64_t* tokens;
  int32_t *key_a, *at_a, *key_b, *at_b;  // by the first digit, and by both
  int32_t* hist;      // [blocks, kBins], of the pass at hand
  int32_t* valid;     // how many tokens are in range
  uint8_t* present;   // [N]: whether a row has a token
  int64_t R, N, per;
  int blocks, shift, bits;
};

// The token at place i of a pass's input, or -1.
template <bool FIRST>
__device__ __forceinline__ int32_t key_at(const SortArgs& p, int64_t i, int64_t end) {
  if (i >= end) return -1;
  if (!FIRST) return p.key_a[i];
  const int64_t t = p.tokens[i];
  return t >= 0 && t < p.N ? (int32_t)t : -1;
}

// How often each digit stands in a block's share; the first pass also clears `present`.
template <bool FIRST>
__global__ void __launch_bounds__(kSortThreads) count_kernel(const SortArgs p) {
  __shared__ int32_t bins[kBins];
  const int tid = threadIdx.x;
  bins[tid] = 0;
  if (FIRST) {
    for (int64_t n = (int64_t)blockIdx.x * kSortThreads + tid; n < p.N; n += (int64_t)p.blocks * kSortThreads)
      p.present[n] = 0;
  }
  __syncthreads();
  const int64_t n = FIRST ? p.R : (int64_t)*p.valid;
  const int64_t lo = blockIdx.x * p.per, hi = lo + p.per < n ? lo + p.per : n;
  for (int64_t i = lo + tid; i < hi; i += kSortThreads) {
    const int32_t key = key_at<FIRST>(p, i, hi);
    if (key >= 0) atomicAdd(&bins[(key >> p.shift) & (kBins - 1) & ((1 << p.bits) - 1)], 1);
  }
  __syncthreads();
  p.hist[blockIdx.x * kBins + tid] = bins[tid];
}

// Places a block's share by its digit: behind the smaller digits, behind the same digit in
// earlier blocks and waves, and in the order of the share.
template <bool FIRST>
__global__ void __launch_bounds__(kSortThreads) place_kernel(const SortArgs p) {
  __shared__ int32_t at[kSortWaves][kBins];
  __shared__ int32_t sums[kSortWaves];
  const int tid = threadIdx.x, lane = tid & 63, w = tid >> 6;
  const int64_t n = FIRST ? p.R : (int64_t)*p.valid;
  int32_t before = 0, total = 0;
  for (int b = 0; b < p.blocks; ++b) {
    const int32_t c = p.hist[b * kBins + tid];
    before += b < (int)blockIdx.x ? c : 0;
    total += c;
  }
  int32_t run = total;  // inclusive sums over the bins: in the wave, then over the waves
  for (int o = 1; o < 64; o *= 2) {
    const int32_t v = __shfl_up(run, o);
    run += lane >= o ? v : 0;
  }
  if (lane == 63) sums[w] = run;
  for (int v = 0; v < kSortWaves; ++v) at[v][tid] = 0;
  __syncthreads();
  int32_t base = run - total + before;
  for (int v = 0; v < w; ++v) base += sums[v];
  if (FIRST && blockIdx.x == 0 && tid == 0) {
    int32_t all = 0;
    for (int v = 0; v < kSortWaves; ++v) all += sums[v];
    *p.valid = all;
  }
  const int64_t share = p.per / kSortWaves;  // a multiple of 64
  const int64_t first = blockIdx.x * p.per + w * share;
  const int64_t end = first + share < n ? first + share : n;
  const int32_t mask = (1 << p.bits) - 1;
  for (int64_t i = first; i < end; i += 64) {
    const int32_t key = key_at<FIRST>(p, i + lane, end);
    if (key >= 0) atomicAdd(&at[w][(key >> p.shift) & mask], 1);
  }
  __syncthreads();
  for (int v = 0; v < kSortWaves; ++v) {
    const int32_t c = at[v][tid];
    at[v][tid] = base;
    base += c;
  }
  __syncthreads();
  for (int64_t i = first; i < end; i += 64) {
    const int32_t key = key_at<FIRST>(p, i + lane, end);
    const int32_t digit = (key >> p.shift) & mask;
    uint64_t same = __ballot(key >= 0);
    for (int b = 0; b < p.bits; ++b) {
      const uint64_t set = __ballot((digit >> b) & 1);
      same &= (digit >> b) & 1 ? set : ~set;
    }
    if (key >= 0) {
      const int leader = __ffsll((unsigned long long)same) - 1;
      int32_t start = 0;
      if (lane == leader) start = atomicAdd(&at[w][digit], __popcll(same));
      start = __shfl(start, leader);
      const int32_t to = start + __popcll(same & ((1ull << lane) - 1));
      (FIRST ? p.key_a : p.key_b)[to] = key;
      (FIRST ? p.at_a : p.at_b)[to] = FIRST ? (int32_t)(i + lane) : p.at_a[i + lane];
      if (FIRST) p.present[key] = 1;
    }
  }
}

// ------------------------------------------------------------------ adding up
struct SumArgs {
  GradArgs g;
  const int32_t *key, *at;  // sorted tokens and their places in d_out
  const int32_t* valid;
  const uint8_t* present;
  float* part;              // [chunks, 2, D]: what came from the chunk before, and what goes on in the next
  int64_t chunks, tiles;
};

constexpr int kAhead = 8;  // rows of d_out in flight in a wave

// Waves take one chunk and 64 V columns each; behind them, the rows without a token, 16 to a wave.
template <class F, int V>
__global__ void __launch_bounds__(256) sum_kernel(const SumArgs p) {
  using E = typename F::E;
  const int lane = threadIdx.x & 63;
  const int64_t u = (int64_t)blockIdx.x * 4 + __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int64_t c = u / p.tiles, d = (u - c * p.tiles) * 64 * V + lane * V;
  const bool some = d < p.g.D;
  E* table = static_cast<E*>(p.g.d_table) + d;
  float acc[V];
#pragma unroll
  for (int i = 0; i < V; ++i) acc[i] = 0.0f;
  if (c >= p.chunks) {
    const int64_t n0 = (c - p.chunks) * 16;
    for (int64_t n = n0; n < n0 + 16 && n < p.g.N; ++n)
      if (p.present[n] == 0 && some) store_piece<F, V>(table + n * p.g.t_stride, acc);
    return;
  }
  const int64_t valid = *p.valid, i0 = c * kChunk;
  if (i0 >= valid) return;
  const int count = valid - i0 < kChunk ? (int)(valid - i0) : kChunk;
  // lane l: token and place of entry l, and behind the chunk the next token (-1: none)
  const int32_t key = i0 + lane < valid ? p.key[i0 + lane] : -1;
  const int32_t at = i0 + lane < valid ? p.at[i0 + lane] : 0;
  const int32_t last = i0 > 0 ? p.key[i0 - 1] : -1;
  const E* rows = static_cast<const E*>(p.g.d_out) + (some ? d : 0);
  bool open = __builtin_amdgcn_readlane(key, 0) == last;  // the sum at hand began in an earlier chunk
  for (int j0 = 0; j0 < count; j0 += kAhead) {
    Piece<F, V> x[kAhead];
#pragma unroll
    for (int j = 0; j < kAhead; ++j) {
      const int l = j0 + j < count ? j0 + j : count - 1;
      x[j] = load_piece<F, V>(rows + (int64_t)__builtin_amdgcn_readlane(at, l) * p.g.o_stride);
    }
#pragma unroll
    for (int j = 0; j < kAhead; ++j) {
      if (j0 + j < count) {
#pragma unroll
        for (int i = 0; i < V; ++i) acc[i] += F::get(x[j].e[i]);
        const int32_t k = __builtin_amdgcn_readlane(key, j0 + j), next = __builtin_amdgcn_readlane(key, j0 + j + 1);
        const bool ends = k != next, border = j0 + j + 1 == count;
        if (ends || border) {
          if (ends && !open) {
#pragma unroll
            for (int i = 0; i < V; ++i) acc[i] *= p.g.scale;
            if (some) store_piece<F, V>(table + k * p.g.t_stride, acc);
          } else if (some) {
            float* part = p.part + (2 * c + (open ? 0 : 1)) * p.g.D + d;
#pragma unroll
            for (int i = 0; i < V; ++i) part[i] = acc[i];
          }
#pragma unroll
          for (int i = 0; i < V; ++i) acc[i] = 0.0f;
          open = false;
        }
      }
    }
  }
}

// The sums that pass a border: the block of the chunk in which one begins adds its parts up,
// a wave a run of chunks, and joins those in order.
template <class F, int V>
__global__ void __launch_bounds__(512) join_kernel(const SumArgs p) {
  using E = typename F::E;
  __shared__ float s[8][64 * V];
  const int lane = threadIdx.x & 63, w = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int64_t c = blockIdx.x / p.tiles, d = (blockIdx.x - c * p.tiles) * 64 * V + lane * V;
  const int64_t valid = *p.valid, i0 = c * kChunk, i1 = i0 + kChunk;
  if (i1 >= valid) return;
  const int32_t k = p.key[i1 - 1];
  if (p.key[i1] != k || (p.key[i0] == k && i0 > 0 && p.key[i0 - 1] == k)) return;  // none begins here and goes on
  // the last chunk it reaches: chunks lo hold its first token beyond doubt, chunks hi do not
  int64_t lo = c + 1, hi = (valid + kChunk - 1) / kChunk;
  while (hi - lo > 1) {
    const int64_t step = (hi - lo + 63) / 64, m = lo + lane * step;
    const bool in = m < hi && p.key[m * kChunk] == k;  // sorted: these hold for the first lanes
    const int n = __popcll(__ballot(in));
    const int64_t to = lo + n * step;
    lo = lo + (n - 1) * step;
    hi = to < hi ? to : hi;
  }
  const int64_t n = lo - c;  // chunks after c
  const int64_t share = (n + 7) / 8, from = c + 1 + w * share;
  const int64_t to = from + share < lo + 1 ? from + share : lo + 1;
  const bool some = d < p.g.D;
  float acc[V];
#pragma unroll
  for (int i = 0; i < V; ++i) acc[i] = w == 0 && some ? p.part[(2 * c + 1) * p.g.D + d + i] : 0.0f;
#pragma unroll 4
  for (int64_t m = from; m < to; ++m) {
#pragma unroll
    for (int i = 0; i < V; ++i) acc[i] += some ? p.part[2 * m * p.g.D + d + i] : 0.0f;
  }
#pragma unroll
  for (int i = 0; i < V; ++i) s[w][lane * V + i] = acc[i];
  __syncthreads();
  if (w == 0 && some) {
    for (int v = 1; v < 8; ++v) {
#pragma unroll
      for (int i = 0; i < V; ++i) acc[i] += s[v][lane * V + i];
    }
#pragma unroll
    for (int i = 0; i < V; ++i) acc[i] *= p.g.scale;
    store_piece<F, V>(static_cast<E*>(p.g.d_table) + k * p.g.t_stride + d, acc);
  }
}

static int64_t round16(int64_t n) { return (n + 15) / 16 * 16; }

Plan make_plan(int64_t R, int64_t N, int64_t D) {
  Plan p{};
  int bits = 1;
  while (((int64_t)1 << bits) < N) ++bits;
  p.passes = bits <= 10 ? 1 : 2;
  p.bits[0] = p.passes == 1 ? bits : (bits + 1) / 2;
  p.bits[1] = bits - p.bits[0];
  // a block of 16 waves for each 1024 tokens, 64 blocks at most (each reads all others' counts)
  int64_t per = (R + 63) / 64;
  p.per = (per + kSortThreads - 1) / kSortThreads * kSortThreads;
  if (p.per < kSortThreads) p.per = kSortThreads;
  p.blocks = R > 0 ? (R + p.per - 1) / p.per : 1;
  p.chunks = (R + kChunk - 1) / kChunk;
  p.keys = round16(4 * R);
  p.hist = 4 * p.blocks * kBins;
  p.present = round16(N);
  p.part = round16(p.chunks * 2 * D * 4);
  p.bytes = 4 * p.keys + 2 * p.hist + p.present + p.part + 16;
  return p;
}

template <class F, int V>
static hipError_t sums_of(const SumArgs& a, hipStream_t st) {
  SumArgs s = a;
  s.tiles = (a.g.D + 64 * V - 1) / (64 * V);
  const int64_t units = (s.chunks + (a.g.N + 15) / 16) * s.tiles;
  sum_kernel<F, V><<<dim3((unsigned)((units + 3) / 4)), 256, 0, st>>>(s);
  hipError_t e = hipGetLastError();
  if (e != hipSuccess || s.chunks < 2) return e;
  join_kernel<F, V><<<dim3((unsigned)(s.chunks * s.tiles)), 512, 0, st>>>(s);
  return hipGetLastError();
}

template <class F>
static hipError_t sums_fmt(const SumArgs& a, hipStream_t st) {
  constexpr int V = F::W, es = sizeof(typename F::E);
  const bool w = wide(a.g.d_out, a.g.o_stride, a.g.d_table, a.g.t_stride, a.g.D, V, es);
  return w ? sums_of<F, V>(a, st) : sums_of<F, 1>(a, st);
}

hipError_t launch_backward(rlscan_format f, const GradArgs& g, hipStream_t st) {
  const Plan p = make_plan(g.R, g.N, g.D);
  char* ws = static_cast<char*>(g.workspace);
  auto take = [&](int64_t bytes) {
    char* at = ws;
    ws += bytes;
    return at;
  };
  SortArgs s{};
  s.tokens = g.tokens;
  s.key_a = reinterpret_cast<int32_t*>(take(p.keys));
  s.at_a = reinterpret_cast<int32_t*>(take(p.keys));
  s.key_b = reinterpret_cast<int32_t*>(take(p.keys));
  s.at_b = reinterpret_cast<int32_t*>(take(p.keys));
  int32_t* hist[2];
  hist[0] = reinterpret_cast<int32_t*>(take(p.hist));
  hist[1] = reinterpret_cast<int32_t*>(take(p.hist));
  s.valid = reinterpret_cast<int32_t*>(take(16));
  s.present = reinterpret_cast<uint8_t*>(take(p.present));
  s.R = g.R;
  s.N = g.N;
  s.per = p.per;
  s.blocks = (int)p.blocks;
  s.hist = hist[0];
  s.bits = p.bits[0];
  const dim3 grid((unsigned)p.blocks);
  count_kernel<true><<<grid, kSortThreads, 0, st>>>(s);
  place_kernel<true><<<grid, kSortThreads, 0, st>>>(s);
  if (p.passes == 2) {
    s.hist = hist[1];
    s.shift = p.bits[0];
    s.bits = p.bits[1];
    count_kernel<false><<<grid, kSortThreads, 0, st>>>(s);
    place_kernel<false><<<grid, kSortThreads, 0, st>>>(s);
  }
  hipError_t e = hipGetLastError();
  if (e != hipSuccess) return e;
  SumArgs a{};
  a.g = g;
  a.key = p.passes == 2 ? s.key_b : s.key_a;
  a.at = p.passes == 2 ? s.at_b : s.at_a;
  a.valid = s.valid;
  a.present = s.present;
  a.part = reinterpret_cast<float*>(take(p.part));
  a.chunks = p.chunks;
  switch (f) {
    case RLSCAN_FORMAT_BF16: return sums_fmt<LBf16>(a, st);
    case RLSCAN_FORMAT_F16: return sums_fmt<LF16>(a, st);
    default: return sums_fmt<LF32>(a, st);
  }
}

}  // namespace embed
}  // namespace rlscan
