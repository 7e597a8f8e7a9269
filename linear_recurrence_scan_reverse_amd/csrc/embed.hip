// Rows of a table by token (rlscan_embed_tokens) and the table's gradient
// (rlscan_embed_tokens_backward).
//
//   out_r = scale table[token_r],   d_table_n = scale sum over token_r = n of d_out_r
//
// Both are bound by memory: the lookup of 32768 rows of 1024 of a table of 64007, bfloat16, takes 21 us
// (6.4 TB/s, some rows from the caches), pieces of 16 bytes 26 us where those of 4 take 34 (65536 x 512,
// float32).  For the gradient of many tokens of more than a few kinds the tokens are sorted
// (stable, by one or two digits of up to ten bits), so that a row's terms follow one another in the
// order of the tokens: chunks of sorted tokens are summed by a wave each, and what passes a chunk's border
// is joined afterwards, in order.  No atomics on values: results do not vary from run to run.
#include "rlscan_embed.hpp"

namespace rlscan {
namespace embed {

using logits::LBf16;
using logits::LF16;
using logits::LF32;

// V elements as they lie in memory: 16, 8 or 4 bytes, or one element of 2.
template <int kBytes>
struct WordOf;
template <>
struct WordOf<16> {
  using T = logits::u32x4;
};
template <>
struct WordOf<8> {
  using T = uint64_t;
};
template <>
struct WordOf<4> {
  using T = uint32_t;
};
template <>
struct WordOf<2> {
  using T = uint16_t;
};
template <class F, int V>
struct Piece {
  using Word = typename WordOf<V * (int)sizeof(typename F::E)>::T;
  typename F::E e[V];
};
template <class F, int V>
__device__ __forceinline__ Piece<F, V> load_piece(const typename F::E* p) {
  Piece<F, V> r;
  const typename Piece<F, V>::Word v = *reinterpret_cast<const typename Piece<F, V>::Word*>(p);
  __builtin_memcpy(&r, &v, sizeof(v));
  return r;
}
template <class F, int V>
__device__ __forceinline__ void store_piece(typename F::E* p, const float (&x)[V]) {
  Piece<F, V> r;
#pragma unroll
  for (int i = 0; i < V; ++i) r.e[i] = F::put(x[i]);
  typename Piece<F, V>::Word v;
  __builtin_memcpy(&v, &r, sizeof(v));
  *reinterpret_cast<typename Piece<F, V>::Word*>(p) = v;
}
// The widest piece, of at most 16 bytes, that rows of D elements at these addresses and strides are made of.
static int piece_of(const void* a, int64_t sa, const void* b, int64_t sb, int64_t D, int es) {
  int v = 16 / es;
  while (v > 1 && (D % v || (uintptr_t)a % (uintptr_t)(v * es) || (uintptr_t)b % (uintptr_t)(v * es) || sa % v || sb % v))
    v /= 2;
  return v;
}

constexpr int kLookups = 4;  // tokens to a wave, whose rows are asked for together

// A wave takes 64 V columns of kLookups tokens.
template <class F, int V>
__global__ void __launch_bounds__(256) lookup_kernel(const LookupArgs p, uint32_t tiles) {
  using E = typename F::E;
  const uint32_t u = blockIdx.x * 4 + (threadIdx.x >> 6);
  const int64_t r0 = (int64_t)(u / tiles) * kLookups, d = (int64_t)(u % tiles) * 64 * V + (threadIdx.x & 63) * V;
  if (r0 >= p.R || d >= p.D) return;
  int64_t n[kLookups];
  Piece<F, V> w[kLookups];
#pragma unroll
  for (int i = 0; i < kLookups; ++i) n[i] = r0 + i < p.R ? p.tokens[r0 + i] : -1;
#pragma unroll
  for (int i = 0; i < kLookups; ++i) {
    const bool in = n[i] >= 0 && n[i] < p.N;
    w[i] = load_piece<F, V>(static_cast<const E*>(p.table) + (in ? n[i] : 0) * p.t_stride + d);
    if (!in) w[i] = Piece<F, V>{};
  }
#pragma unroll
  for (int i = 0; i < kLookups; ++i) {
    float x[V];
#pragma unroll
    for (int j = 0; j < V; ++j) x[j] = p.scale * F::get(w[i].e[j]);
    if (r0 + i < p.R) store_piece<F, V>(static_cast<E*>(p.out) + (r0 + i) * p.o_stride + d, x);
  }
}

template <class F, int V>
static hipError_t lookup_of(const LookupArgs& a, hipStream_t st) {
  const int64_t tiles = (a.D + 64 * V - 1) / (64 * V), units = (a.R + kLookups - 1) / kLookups * tiles;
  lookup_kernel<F, V><<<dim3((unsigned)((units + 3) / 4)), 256, 0, st>>>(a, (uint32_t)tiles);
  return hipGetLastError();
}

template <class F>
static hipError_t lookup_fmt(const LookupArgs& a, hipStream_t st) {
  switch (piece_of(a.table, a.t_stride, a.out, a.o_stride, a.D, sizeof(typename F::E))) {
    case 8:
      if constexpr (F::W == 8) return lookup_of<F, 8>(a, st);
      break;
    case 4: return lookup_of<F, 4>(a, st);
    case 2: return lookup_of<F, 2>(a, st);
  }
  return lookup_of<F, 1>(a, st);
}

hipError_t launch_lookup(rlscan_format f, const LookupArgs& a, hipStream_t st) {
  switch (f) {
    case RLSCAN_FORMAT_BF16: return lookup_fmt<LBf16>(a, st);
    case RLSCAN_FORMAT_F16: return lookup_fmt<LF16>(a, st);
    default: return lookup_fmt<LF32>(a, st);
  }
}

// ------------------------------------------------------------------ sorting the tokens
// 32768 tokens of 64007 kinds: count 3, place 14 and 6 us, latency; then 33 us to add up (x 1024, bfloat16,
// 6 TB/s of those read and written) and 6 to join.  2^20 tokens x 256 of the same kinds, the first the most frequent:
// 11, 144 and 35, then 126 and 93, of which the most is one block that joins the first kind's 2000 chunks.
constexpr int kBins = 1024;
constexpr int kSortThreads = 1024, kSortWaves = kSortThreads / 64;

struct SortArgs {
  const int64_t* tokens;
  int32_t *key_a, *at_a, *key_b, *at_b;  // by the first digit, and by both
  int32_t *hist_a, *hist_b;              // [blocks, kBins], of either pass
  int32_t* valid;     // how many tokens are in range
  uint8_t* present;   // [N]: whether a row has a token
  int64_t R, N, per;
  int blocks, passes, bits[2];
};

// The token at place i of a pass's input, or -1.
template <bool FIRST>
__device__ __forceinline__ int32_t key_at(const SortArgs& p, int64_t i, int64_t end) {
  if (i >= end) return -1;
  if (!FIRST) return p.key_a[i];
  const int64_t t = p.tokens[i];
  return t >= 0 && t < p.N ? (int32_t)t : -1;
}

// The lanes whose key has the same bits [from, from + bits); only those with a key.
__device__ __forceinline__ uint64_t alike(uint64_t among, int32_t key, int from, int bits) {
  for (int b = from; b < from + bits; ++b) {
    const uint64_t set = __ballot((key >> b) & 1);
    among &= (key >> b) & 1 ? set : ~set;
  }
  return among;
}

// How often each first digit stands in a block's share; also clears `present` and the second pass's counts.
__global__ void __launch_bounds__(kSortThreads) count_kernel(const SortArgs p) {
  __shared__ int32_t bins[kBins];
  const int tid = threadIdx.x;
  bins[tid] = 0;
  p.hist_b[blockIdx.x * kBins + tid] = 0;
  for (int64_t n = (int64_t)blockIdx.x * kSortThreads + tid; n < p.N; n += (int64_t)p.blocks * kSortThreads)
    p.present[n] = 0;
  __syncthreads();
  const int64_t lo = blockIdx.x * p.per, hi = lo + p.per < p.R ? lo + p.per : p.R;
  for (int64_t i = lo + tid; i < hi; i += kSortThreads) {
    const int32_t key = key_at<true>(p, i, hi);
    if (key >= 0) atomicAdd(&bins[key & ((1 << p.bits[0]) - 1)], 1);
  }
  __syncthreads();
  p.hist_a[blockIdx.x * kBins + tid] = bins[tid];
}

// Places a block's share by its digit: behind the smaller digits, behind the same digit in
// earlier blocks and waves, and in the order of the share.  The first pass counts, where its tokens go,
// the second's digits: whole numbers, whose sums do not depend on their order.
template <bool FIRST>
__global__ void __launch_bounds__(kSortThreads) place_kernel(const SortArgs p) {
  __shared__ int32_t at[kSortWaves][kBins];
  __shared__ int32_t sums[kSortWaves];
  const int tid = threadIdx.x, lane = tid & 63, w = tid >> 6;
  const int shift = FIRST ? 0 : p.bits[0], bits = p.bits[FIRST ? 0 : 1];
  const int32_t* const hist = FIRST ? p.hist_a : p.hist_b;
  const int64_t n = FIRST ? p.R : (int64_t)*p.valid;
  int32_t before = 0, total = 0;
  if (tid < 1 << bits) {
#pragma unroll 16
    for (int b = 0; b < p.blocks; ++b) {
      const int32_t c = hist[b * kBins + tid];
      before += b < (int)blockIdx.x ? c : 0;
      total += c;
    }
  }
  int32_t run = total;  // inclusive sums over the bins: in the wave, then over the waves
  for (int o = 1; o < 64; o *= 2) {
    const int32_t v = __shfl_up(run, o);
    run += lane >= o ? v : 0;
  }
  if (lane == 63) sums[w] = run;
#pragma unroll
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
  const int32_t mask = (1 << bits) - 1;
  for (int64_t i = first; i < end; i += 64) {
    const int32_t key = key_at<FIRST>(p, i + lane, end);
    if (key >= 0) atomicAdd(&at[w][(key >> shift) & mask], 1);
  }
  __syncthreads();
#pragma unroll
  for (int v = 0; v < kSortWaves; ++v) {
    const int32_t c = at[v][tid];
    at[v][tid] = base;
    base += c;
  }
  __syncthreads();
  for (int64_t i = first; i < end; i += 64) {
    const int32_t key = key_at<FIRST>(p, i + lane, end);
    const int32_t source = !FIRST && key >= 0 ? p.at_a[i + lane] : (int32_t)(i + lane);
    const int32_t digit = (key >> shift) & mask;
    const uint64_t same = alike(__ballot(key >= 0), key, shift, bits);
    // those of them that are the same token stand side by side in their block of the second pass, but for a border
    const uint64_t twins = FIRST && p.passes == 2 ? alike(same, key, p.bits[0], p.bits[1]) : 0;
    if (key >= 0) {
      const int leader = __ffsll((unsigned long long)same) - 1;
      int32_t start = 0;
      if (lane == leader) start = atomicAdd(&at[w][digit], __popcll(same));
      start = __shfl(start, leader);
      const int32_t to = start + __popcll(same & ((1ull << lane) - 1));
      (FIRST ? p.key_a : p.key_b)[to] = key;
      (FIRST ? p.at_a : p.at_b)[to] = source;
      if (FIRST) {
        p.present[key] = 1;
        if (p.passes == 2) {
          // one lane counts for all twins that go to the same block of the second pass
          const int32_t block = to / (int32_t)p.per;
          const int32_t before_me = lane > 0 ? 63 - __builtin_clzll((twins & ((1ull << lane) - 1)) | 1) : 0;
          const bool has = (twins & ((1ull << lane) - 1)) != 0;
          const int32_t block_before = __shfl(block, has ? before_me : lane);
          const bool heads = !has || block_before != block;
          const uint64_t ends = __ballot(heads);
          if (heads) {
            // twins from here to the next that begins anew
            const uint64_t behind = lane == 63 ? 0 : twins & ~((2ull << lane) - 1);
            const uint64_t stop = behind & ends;
            const uint64_t mine = stop ? behind & ((1ull << (__ffsll((unsigned long long)stop) - 1)) - 1) : behind;
            atomicAdd(&p.hist_b[(int64_t)block * kBins + ((key >> p.bits[0]) & ((1 << p.bits[1]) - 1))],
                      1 + __popcll(mine));
          }
        }
      }
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

constexpr int kJoinWaves = 4;

// The sums that pass a border: the block of the chunk in which one begins adds its parts up,
// a wave a run of chunks, and joins those in order.
template <class F, int V>
__global__ void __launch_bounds__(64 * kJoinWaves) join_kernel(const SumArgs p) {
  using E = typename F::E;
  __shared__ float s[kJoinWaves][64 * V];
  const int lane = threadIdx.x & 63, w = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const uint32_t chunk = blockIdx.x / (uint32_t)p.tiles;
  const int64_t c = chunk, d = (int64_t)(blockIdx.x - chunk * (uint32_t)p.tiles) * 64 * V + lane * V;
  const int64_t valid = *p.valid, i0 = c * kChunk, i1 = i0 + kChunk;
  if (i1 >= valid) return;
  const int64_t chunks = (valid + kChunk - 1) / kChunk;
  // all at once: the borders of the chunk, and the first tokens of the 64 behind it
  const int32_t first = p.key[i0], k = p.key[i1 - 1], next = p.key[i1], last = p.key[i0 > 0 ? i0 - 1 : 0];
  const int32_t probe = c + 1 + lane < chunks ? p.key[(c + 1 + lane) * kChunk] : -1;
  if (next != k || (first == k && i0 > 0 && last == k)) return;  // none begins here and goes on
  // the last chunk it reaches: chunk lo holds it beyond doubt, chunk hi does not
  int64_t n = __popcll(__ballot(probe == k));  // sorted: these hold for the first lanes
  int64_t lo = c + n, hi = n < 64 ? lo + 1 : chunks;
  while (hi - lo > 1) {
    const int64_t step = (hi - lo + 63) / 64, m = lo + lane * step;
    n = __popcll(__ballot(m < hi && p.key[m < hi ? m * kChunk : 0] == k));
    const int64_t to = lo + n * step;
    lo = lo + (n - 1) * step;
    hi = to < hi ? to : hi;
  }
  const int64_t share = (lo - c + kJoinWaves - 1) / kJoinWaves, from = c + 1 + w * share;
  const int64_t to = from + share < lo + 1 ? from + share : lo + 1;
  const bool some = d < p.g.D;
  const float* const part = p.part + (some ? d : 0);
  float acc[V];
#pragma unroll
  for (int i = 0; i < V; ++i) acc[i] = w == 0 ? part[(2 * c + 1) * p.g.D + i] : 0.0f;
#pragma unroll 4
  for (int64_t m = from; m < to; ++m) {
#pragma unroll
    for (int i = 0; i < V; ++i) acc[i] += part[2 * m * p.g.D + i];
  }
#pragma unroll
  for (int i = 0; i < V; ++i) s[w][i * 64 + lane] = acc[i];
  __syncthreads();
  if (w == 0 && some) {
    for (int v = 1; v < kJoinWaves; ++v) {
#pragma unroll
      for (int i = 0; i < V; ++i) acc[i] += s[v][i * 64 + lane];
    }
#pragma unroll
    for (int i = 0; i < V; ++i) acc[i] *= p.g.scale;
    store_piece<F, V>(static_cast<E*>(p.g.d_table) + k * p.g.t_stride + d, acc);
  }
}

// ------------------------------------------------------------------ few kinds of token
// A wave adds its tokens' rows up in a table of its own in LDS, a block's waves in order to a share, and
// the shares in order to the gradient: two launches and one pass over d_out, no sort.  Bound by memory
// where there are many tokens (262144 x 256 float32: 53 us, 5.1 TB/s), by the latencies of two short kernels
// where there are few (16384 x 250 of 18 kinds, float32: 7.7 and 2.9 us).
// Up to 31 kinds and one for tokens out of range, pieces of two elements: four tables take 64 KiB at most, so
// that two blocks share a compute unit.  Measured against the sort, us: 16384 x 250 float32, 18 kinds, 12
// against 18; 262144 x 256 bfloat16, 4 kinds 36 against 95, 31 kinds 37 against 62, 64 kinds (one element a
// lane) 80 against 58.  Pieces of four elements leave fewer waves to a compute unit: 8 kinds 58 against 44.
constexpr int64_t kFewKinds = 31;
constexpr int kFewWaves = 4, kFewAhead = 16;
struct FewArgs {
  GradArgs g;
  float* part;  // [rows, N, D]
  int64_t per;  // tokens of a share
  int64_t rows;
  uint32_t tiles;
};

template <class F, int V>
__global__ void __launch_bounds__(64 * kFewWaves) few_kernel(const FewArgs p) {
  using E = typename F::E;
  extern __shared__ __align__(16) float few_table[];  // [kFewWaves, N + 1, 64 V]: the last for tokens out of range
  const int lane = threadIdx.x & 63, w = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6), N = (int)p.g.N;
  const int size = (N + 1) * 64 * V;  // of a wave's table
  const uint32_t row = blockIdx.x / p.tiles, tile = blockIdx.x % p.tiles;
  const int64_t d = (int64_t)tile * 64 * V + lane * V;
  const bool some = d < p.g.D;
  float* const mine = few_table + w * size + lane * V;
  for (int n = 0; n < N; ++n) {
#pragma unroll
    for (int i = 0; i < V; ++i) mine[n * 64 * V + i] = 0.0f;
  }
  const int64_t share = p.per / kFewWaves, first = row * p.per + w * share;
  const int64_t end = first + share < p.g.R ? first + share : p.g.R;
  const E* const rows = static_cast<const E*>(p.g.d_out) + (some ? d : 0);
  for (int64_t i0 = first; i0 < end; i0 += 64) {
    const int64_t t = i0 + lane < end ? p.g.tokens[i0 + lane] : -1;
    const int32_t key = t >= 0 && t < p.g.N ? (int32_t)t : N;
    const int count = end - i0 < 64 ? (int)(end - i0) : 64;
    for (int j0 = 0; j0 < count; j0 += kFewAhead) {
      Piece<F, V> x[kFewAhead];
#pragma unroll
      for (int j = 0; j < kFewAhead; ++j)
        x[j] = load_piece<F, V>(rows + (i0 + (j0 + j < count ? j0 + j : count - 1)) * p.g.o_stride);
#pragma unroll
      for (int j = 0; j < kFewAhead; ++j) {
        // Every row is added, those past the end to the last table too: loads under a condition would go out
        // one by one
        float* const at = mine + __builtin_amdgcn_readlane(key, j0 + j) * 64 * V;
#pragma unroll
        for (int i = 0; i < V; ++i) at[i] += F::get(x[j].e[i]);
      }
    }
  }
  __syncthreads();
  for (int i = threadIdx.x; i < N * 64 * V; i += 64 * kFewWaves) {
    float sum = few_table[i];
#pragma unroll
    for (int v = 1; v < kFewWaves; ++v) sum += few_table[v * size + i];
    const int64_t column = (int64_t)tile * 64 * V + i % (64 * V);
    if (column < p.g.D) p.part[(row * p.g.N + i / (64 * V)) * p.g.D + column] = sum;
  }
}

constexpr int kFewGroups = 16;
template <class F>
__global__ void __launch_bounds__(64 * kFewGroups) few_join_kernel(const FewArgs p) {
  __shared__ float s[kFewGroups][64];
  const int lane = threadIdx.x & 63, group = threadIdx.x >> 6;
  const int64_t columns = p.g.N * p.g.D, c = (int64_t)blockIdx.x * 64 + lane;
  const int64_t share = (p.rows + kFewGroups - 1) / kFewGroups, from = group * share;
  const int64_t to = from + share < p.rows ? from + share : p.rows;
  float sum = 0.0f;
  if (c < columns) {
#pragma unroll 8
    for (int64_t r = from; r < to; ++r) sum += p.part[r * columns + c];
  }
  s[group][lane] = sum;
  __syncthreads();
  if (group != 0 || c >= columns) return;
#pragma unroll
  for (int v = 1; v < kFewGroups; ++v) sum += s[v][lane];
  const int64_t n = c / p.g.D;
  static_cast<typename F::E*>(p.g.d_table)[n * p.g.t_stride + (c - n * p.g.D)] = F::put(p.g.scale * sum);
}

// ------------------------------------------------------------------ few tokens
// One launch: a block for each token and tile of columns looks the tokens over; the first of its kind adds up
// all of its kind, each wave those of a quarter of the tokens, and the quarters in order.  Behind these blocks,
// waves that write zeros where a row has no token, 64 rows each.  Bound by latency, and where the table is
// large by its zeros (100000 x 1024 float32: 85 us, 4.8 TB/s).
// Up to 1024 tokens.  Measured against the other two ways, us, float32: 64 tokens x 128 of 64 kinds 7.3 against
// 16.6, 1024 x 1024 of 18 kinds 7.3 against 11.4, of 64 9.7 against 16.6, of 1000 12 against 18; the nearest,
// 1024 x 2048 of 1000, 17.4 against 18.7, and 1024 x 1024 of 2 kinds, bfloat16, 14.8 against 11.5.
constexpr int64_t kFewTokens = 1024;
constexpr int kEachWaves = 4, kEachWords = (int)kFewTokens / 64 / kEachWaves;

template <class F, int V>
__global__ void __launch_bounds__(64 * kEachWaves) each_kernel(const GradArgs g, uint32_t tiles, uint32_t sums) {
  using E = typename F::E;
  __shared__ float s[kEachWaves][64 * V];
  __shared__ int32_t seen[kEachWaves];
  const int lane = threadIdx.x & 63, w = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6), R = (int)g.R;
  if (blockIdx.x >= sums) {
    const uint32_t u = (blockIdx.x - sums) * kEachWaves + w, tile = u % tiles;
    const int64_t n0 = (int64_t)(u / tiles) * 64, d = (int64_t)tile * 64 * V + lane * V;
    uint64_t has = 0;
    for (int i = lane; i < R; i += 64) {
      const int64_t k = g.tokens[i] - n0;
      has |= k >= 0 && k < 64 ? 1ull << k : 0;
    }
    for (int o = 32; o > 0; o /= 2) has |= __shfl_xor((unsigned long long)has, o);
    float zero[V];
#pragma unroll
    for (int i = 0; i < V; ++i) zero[i] = 0.0f;
    for (int k = 0; k < 64 && n0 + k < g.N; ++k)
      if (((has >> k) & 1) == 0 && d < g.D) store_piece<F, V>(static_cast<E*>(g.d_table) + (n0 + k) * g.t_stride + d, zero);
    return;
  }
  const int r = (int)(blockIdx.x / tiles);
  const int64_t d = (int64_t)(blockIdx.x % tiles) * 64 * V + lane * V, token = g.tokens[r];
  if (token < 0 || token >= g.N) return;
  const bool some = d < g.D;
  const int share = (R + 64 * kEachWaves - 1) / (64 * kEachWaves) * 64, from = w * share;
  uint64_t alike[kEachWords];  // which of the wave's quarter are the same
  bool earlier = false;
#pragma unroll
  for (int b = 0; b < kEachWords; ++b) {
    const int i = from + 64 * b + lane;
    const bool same = 64 * b < share && i < R && g.tokens[i < R ? i : 0] == token;
    earlier |= same && i < r;
    alike[b] = __ballot(same);
  }
  const uint64_t any = __ballot(earlier);
  if (lane == 0) seen[w] = any != 0;
  __syncthreads();
  if (seen[0] | seen[1] | seen[2] | seen[3]) return;
  const E* const rows = static_cast<const E*>(g.d_out) + (some ? d : 0);
  float acc[V];
#pragma unroll
  for (int i = 0; i < V; ++i) acc[i] = 0.0f;
#pragma unroll
  for (int b = 0; b < kEachWords; ++b) {
    for (uint64_t left = alike[b]; left != 0;) {
      Piece<F, V> x[kAhead];
      bool is[kAhead];
#pragma unroll
      for (int j = 0; j < kAhead; ++j) {
        is[j] = left != 0;
        const int at = is[j] ? from + 64 * b + __ffsll((unsigned long long)left) - 1 : r;
        left &= left - 1;
        x[j] = load_piece<F, V>(rows + (int64_t)at * g.o_stride);
      }
#pragma unroll
      for (int j = 0; j < kAhead; ++j) {
#pragma unroll
        for (int i = 0; i < V; ++i) acc[i] += is[j] ? F::get(x[j].e[i]) : 0.0f;
      }
    }
  }
#pragma unroll
  for (int i = 0; i < V; ++i) s[w][i * 64 + lane] = acc[i];
  __syncthreads();
  if (w != 0 || !some) return;
#pragma unroll
  for (int i = 0; i < V; ++i) {
#pragma unroll
    for (int v = 1; v < kEachWaves; ++v) acc[i] += s[v][i * 64 + lane];
    acc[i] *= g.scale;
  }
  store_piece<F, V>(static_cast<E*>(g.d_table) + token * g.t_stride + d, acc);
}

static int64_t round16(int64_t n) { return (n + 15) / 16 * 16; }

Plan make_plan(int64_t R, int64_t N, int64_t D) {
  Plan p{};
  if (R <= kFewTokens) return p;
  if (N <= kFewKinds) {
    // shares of 128 tokens and more, as many as fill the card
    int64_t most = 65536 / D;
    most = most > 512 ? 512 : most < 8 ? 8 : most;
    const int64_t unit = 32 * kFewWaves, per = (R + most - 1) / most;
    p.per = (per + unit - 1) / unit * unit;
    if (p.per < unit) p.per = unit;
    p.blocks = R > 0 ? (R + p.per - 1) / p.per : 1;
    p.part = round16(p.blocks * N * D * 4);
    p.bytes = p.part;
    return p;
  }
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
static hipError_t each_of(const GradArgs& a, hipStream_t st) {
  const int64_t tiles = (a.D + 64 * V - 1) / (64 * V), sums = a.R * tiles, rest = (a.N + 63) / 64 * tiles;
  each_kernel<F, V><<<dim3((unsigned)(sums + (rest + kEachWaves - 1) / kEachWaves)), 64 * kEachWaves, 0, st>>>(
      a, (uint32_t)tiles, (uint32_t)sums);
  return hipGetLastError();
}

template <class F>
static hipError_t each_fmt(const GradArgs& a, hipStream_t st) {
  switch (piece_of(a.d_out, a.o_stride, a.d_table, a.t_stride, a.D, sizeof(typename F::E))) {
    case 8:
      if constexpr (F::W == 8) return each_of<F, 8>(a, st);
      break;
    case 4: return each_of<F, 4>(a, st);
    case 2: return each_of<F, 2>(a, st);
  }
  return each_of<F, 1>(a, st);
}

template <class F, int V>
static hipError_t sums_of(const SumArgs& a, hipStream_t st) {
  SumArgs s = a;
  s.tiles = (a.g.D + 64 * V - 1) / (64 * V);
  const int64_t units = (s.chunks + (a.g.N + 15) / 16) * s.tiles;
  sum_kernel<F, V><<<dim3((unsigned)((units + 3) / 4)), 256, 0, st>>>(s);
  hipError_t e = hipGetLastError();
  if (e != hipSuccess || s.chunks < 2) return e;
  join_kernel<F, V><<<dim3((unsigned)(s.chunks * s.tiles)), 64 * kJoinWaves, 0, st>>>(s);
  return hipGetLastError();
}

template <class F, int V>
static hipError_t few_of(FewArgs a, hipStream_t st) {
  a.tiles = (uint32_t)((a.g.D + 64 * V - 1) / (64 * V));
  few_kernel<F, V><<<dim3((unsigned)(a.rows * a.tiles)), 64 * kFewWaves, kFewWaves * (a.g.N + 1) * 64 * V * 4, st>>>(a);
  const hipError_t e = hipGetLastError();
  if (e != hipSuccess) return e;
  few_join_kernel<F><<<dim3((unsigned)((a.g.N * a.g.D + 63) / 64)), 64 * kFewGroups, 0, st>>>(a);
  return hipGetLastError();
}

template <class F>
static hipError_t few_fmt(const FewArgs& a, hipStream_t st) {
  const bool pairs = piece_of(a.g.d_out, a.g.o_stride, a.g.d_out, a.g.o_stride, a.g.D, sizeof(typename F::E)) > 1;
  return pairs ? few_of<F, 2>(a, st) : few_of<F, 1>(a, st);
}

template <class F>
static hipError_t sums_fmt(const SumArgs& a, hipStream_t st) {
  switch (piece_of(a.g.d_out, a.g.o_stride, a.g.d_table, a.g.t_stride, a.g.D, sizeof(typename F::E))) {
    case 8:
      if constexpr (F::W == 8) return sums_of<F, 8>(a, st);
      break;
    case 4: return sums_of<F, 4>(a, st);
    case 2: return sums_of<F, 2>(a, st);
  }
  return sums_of<F, 1>(a, st);
}

hipError_t launch_backward(rlscan_format f, const GradArgs& g, hipStream_t st) {
  const Plan p = make_plan(g.R, g.N, g.D);
  if (g.R <= kFewTokens) {
    switch (f) {
      case RLSCAN_FORMAT_BF16: return each_fmt<LBf16>(g, st);
      case RLSCAN_FORMAT_F16: return each_fmt<LF16>(g, st);
      default: return each_fmt<LF32>(g, st);
    }
  }
  if (g.N <= kFewKinds) {
    const FewArgs a{g, static_cast<float*>(g.workspace), p.per, p.blocks, 0};
    switch (f) {
      case RLSCAN_FORMAT_BF16: return few_fmt<LBf16>(a, st);
      case RLSCAN_FORMAT_F16: return few_fmt<LF16>(a, st);
      default: return few_fmt<LF32>(a, st);
    }
  }
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
  s.hist_a = reinterpret_cast<int32_t*>(take(p.hist));
  s.hist_b = reinterpret_cast<int32_t*>(take(p.hist));
  s.valid = reinterpret_cast<int32_t*>(take(16));
  s.present = reinterpret_cast<uint8_t*>(take(p.present));
  s.R = g.R;
  s.N = g.N;
  s.per = p.per;
  s.blocks = (int)p.blocks;
  s.passes = p.passes;
  s.bits[0] = p.bits[0];
  s.bits[1] = p.bits[1];
  const dim3 grid((unsigned)p.blocks);
  count_kernel<<<grid, kSortThreads, 0, st>>>(s);
  place_kernel<true><<<grid, kSortThreads, 0, st>>>(s);
  if (p.passes == 2) place_kernel<false><<<grid, kSortThreads, 0, st>>>(s);
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
