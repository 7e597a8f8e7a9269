// rlscan_la.hpp -- linear attention with a decay for each head: what its kernels share.
//
// Per row e and head h, with k and v of the head's group,
//   S_t = a_t S_{t-1} + k_t v_t^T,   o_t = scale * S_t^T q_t,   a_t = exp(g_t),
// and a_t = 0 where step t-1 ended an episode (done[t-1]) or exp(g_t) is 0 in
// float32.  A row is walked in chunks of C steps.  With b the running sum of g
// inside a chunk and "same" saying that no cut lies between two steps,
//   P_ij  = scale * (q_i . k_j) * exp(b_i - b_j)            j <= i, same
//   o_i   = sum_j P_ij v_j + entry_i S_in^T q_i             entry_i = scale * exp(b_i)
//   S_out = across S_in + sum_j leave_j k_j v_j^T           leave_j = exp(b_last - b_j)
// so that a chunk is five matrix products on MFMA and no step waits for the one
// before it.
//
// Numbers.  Every product runs on bfloat16 MFMA with float32 sums.  An operand
// is held as a sum of bfloat16 terms, largest first: one for bfloat16 storage
// and two for float16 (both exact), three for float32 (24 bits).  A product
// keeps the pairs of terms that reach its precision (1, 3 and 6 of them); six
// bfloat16 products cost less than one product on the float32 matrix
// instructions (16 times slower on this card).  Decays are summed in float64 in units
// of log2 and held as two floats, so differences far from the row's start keep
// their bits.  States stay in float32 registers and are split only to be multiplied.
#ifndef RLSCAN_LA_HPP
#define RLSCAN_LA_HPP

#include <hip/hip_runtime.h>

#include <cstdint>

#include "rlscan.h"

namespace rlscan {
namespace la {

typedef __bf16 bf16x8 __attribute__((ext_vector_type(8)));
typedef __bf16 bf16x4 __attribute__((ext_vector_type(4)));
typedef short s16x4 __attribute__((ext_vector_type(4)));
typedef float f32x4 __attribute__((ext_vector_type(4)));
typedef uint32_t u32x4 __attribute__((ext_vector_type(4)));

constexpr int kWaves = 4;
constexpr int kThreads = 64 * kWaves;
constexpr int kPad = 8;  // elements behind each LDS row: rows 16 bytes apart in the banks

// A strided [E, T, heads, D] tensor (strides in elements, D contiguous).
struct View {
  const void* p;
  int64_t se, st, sh;
  int vec;  // rows can be read and written 16 bytes at a time
};

struct Args {
  View q, k, v, dout;     // inputs (dout: backward)
  View out, dq, dk, dv;   // outputs
  const float* g;         // log-decays, with strides (0 where a dimension is broadcast)
  int64_t g_se, g_st, g_sh;
  const uint8_t* done;    // [E, T] or [T, E] by strides, or NULL
  int64_t d_se, d_st;
  const float* init;      // [E, H, K, V] or NULL
  float* final_state;     // [E, H, K, V] or NULL
  const float* d_final;   // [E, H, K, V] or NULL
  float* d_init;          // [E, H, K, V] or NULL
  float* dg;              // gradient of the log-decays
  int64_t dg_se, dg_st, dg_sh;
  int64_t E, T, H, G;     // G heads share a key/value head
  int K, V;
  float scale;
  // workspace
  float* seg_state;       // [E, H, nseg, KP, VP] states entering each segment
  float* seg_decay;       // [E, H, nseg]
  float* seg_grad;        // the same two for the backward direction
  float* seg_gdecay;
  float* states;          // [E, H, chunks, KP, VP] state entering each chunk
  float* grads;           // [E, H, chunks, KP, VP] gradient of the state leaving each chunk
  int64_t nseg, seg_chunks, chunks;
};

// ------------------------------------------------------------------ number formats
struct TBf16 {
  using E = uint16_t;
  static constexpr int NT = 1;  // bfloat16 terms that hold an element
  static constexpr int NP = 2;  // terms of a float32 intermediate that reaches an output of this type
  static constexpr int NW = 3;  // terms of a float32 intermediate that reaches a float32 output
};
struct TF16 {
  using E = uint16_t;
  static constexpr int NT = 2;
  static constexpr int NP = 2;
  static constexpr int NW = 3;
};
struct TF32 {
  using E = float;
  static constexpr int NT = 3;
  static constexpr int NP = 3;
  static constexpr int NW = 3;
};

template <int N>
struct Frag {
  bf16x8 t[N];  // 8 operand elements of a lane, as N terms
};

// acc += A B^T over 32 contraction steps: row (A) and column (B) l % 16, slot
// s of lane group l / 16 is step (l/16)*8 + s, the same for both.  Small terms first.
template <int NA, int NB>
__device__ __forceinline__ f32x4 mma(const Frag<NA>& a, const Frag<NB>& b, f32x4 acc) {
  constexpr int top = (NA > NB ? NA : NB) - 1;
#pragma unroll
  for (int order = top; order >= 0; --order)
#pragma unroll
    for (int i = 0; i < NA; ++i) {
      const int j = order - i;
      if (j >= 0 && j < NB) acc = __builtin_amdgcn_mfma_f32_16x16x32_bf16(a.t[i], b.t[j], acc, 0, 0, 0);
    }
  return acc;
}

template <int N>
__device__ __forceinline__ void split1(float x, __bf16 (&t)[N]) {
#pragma unroll
  for (int n = 0; n < N; ++n) {
    t[n] = (__bf16)x;
    x -= (float)t[n];
  }
}

template <int N>
__device__ __forceinline__ Frag<N> split(const float (&x)[8]) {
  Frag<N> f;
#pragma unroll
  for (int s = 0; s < 8; ++s) {
    __bf16 t[N];
    split1<N>(x[s], t);
#pragma unroll
    for (int n = 0; n < N; ++n) f.t[n][s] = t[n];
  }
  return f;
}

template <int N>
__device__ __forceinline__ void join(const Frag<N>& f, float (&x)[8]) {
#pragma unroll
  for (int s = 0; s < 8; ++s) {
    float v = (float)f.t[N - 1][s];
#pragma unroll
    for (int n = N - 2; n >= 0; --n) v += (float)f.t[n][s];
    x[s] = v;
  }
}

// ------------------------------------------------------------------ LDS tiles
// A matrix of R rows and D columns, as N planes of bfloat16 terms.
template <int N, int R, int D>
struct Tile {
  static constexpr int LD = D + kPad;
  __bf16 p[N][R * LD];
};

// Row `row0 + l%16`, columns kk*32 + (l/16)*8 ... +7.
template <int N, int R, int D>
__device__ __forceinline__ Frag<N> frag_row(const Tile<N, R, D>& t, int row0, int kk, int lane) {
  Frag<N> f;
  const int o = (row0 + (lane & 15)) * Tile<N, R, D>::LD + kk * 32 + (lane >> 4) * 8;
#pragma unroll
  for (int n = 0; n < N; ++n) f.t[n] = *reinterpret_cast<const bf16x8*>(&t.p[n][o]);
  return f;
}

// The same row in the order in which two accumulator tiles hold 32 steps: slots
// 0-3 are columns kk*32 + (l/16)*4 ..., slots 4-7 the columns 16 further on.
template <int N, int R, int D>
__device__ __forceinline__ Frag<N> frag_row_acc(const Tile<N, R, D>& t, int row0, int kk, int lane) {
  Frag<N> f;
  const int o = (row0 + (lane & 15)) * Tile<N, R, D>::LD + kk * 32 + (lane >> 4) * 4;
#pragma unroll
  for (int n = 0; n < N; ++n) {
    const bf16x4 a = *reinterpret_cast<const bf16x4*>(&t.p[n][o]);
    const bf16x4 b = *reinterpret_cast<const bf16x4*>(&t.p[n][o + 16]);
    f.t[n] = __builtin_shufflevector(a, b, 0, 1, 2, 3, 4, 5, 6, 7);
  }
  return f;
}

// Column `col0 + l%16`, rows kk*32 + (l/16)*8 ... +7, by the LDS transpose read: each
// 16 lanes fetch four rows of 16 columns and each gets one column of them.
template <int N, int R, int D>
__device__ __forceinline__ Frag<N> frag_col(const Tile<N, R, D>& t, int col0, int kk, int lane) {
  using lds_s16x4 = __attribute__((address_space(3))) s16x4;
  constexpr int LD = Tile<N, R, D>::LD;
  Frag<N> f;
  const int i = lane & 15;
  const int o = (kk * 32 + (lane >> 4) * 8 + (i >> 2)) * LD + col0 + (i & 3) * 4;
#pragma unroll
  for (int n = 0; n < N; ++n) {
    union {
      s16x4 h[2];
      bf16x8 v;
    } u;
    u.h[0] = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_s16x4*)(&t.p[n][o]));
    u.h[1] = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_s16x4*)(&t.p[n][o + 4 * LD]));
    f.t[n] = u.v;
  }
  return f;
}

// Four consecutive columns of one row, from the values of an accumulator.
template <int N, int R, int D>
__device__ __forceinline__ void put4(Tile<N, R, D>& t, int row, int col, const float (&x)[4]) {
  bf16x4 w[N];
#pragma unroll
  for (int r = 0; r < 4; ++r) {
    __bf16 s[N];
    split1<N>(x[r], s);
#pragma unroll
    for (int n = 0; n < N; ++n) w[n][r] = s[n];
  }
#pragma unroll
  for (int n = 0; n < N; ++n) *reinterpret_cast<bf16x4*>(&t.p[n][row * Tile<N, R, D>::LD + col]) = w[n];
}

// ------------------------------------------------------------------ global rows
__device__ __forceinline__ float f16_bits(uint16_t b) {
  union {
    uint16_t u;
    _Float16 h;
  } x;
  x.u = b;
  return (float)x.h;
}

// 8 consecutive elements of a row, as they lie in memory.
template <class F>
struct Piece {
  u32x4 w[sizeof(typename F::E) * 8 / 16];
};

// Elements col ... col+7 of a row of D; zeros past the row's end.
template <class F>
__device__ __forceinline__ Piece<F> load_piece(const typename F::E* row, int col, int D, bool row_ok, int vec) {
  Piece<F> x;
  constexpr int W = sizeof(x.w) / 16;
#pragma unroll
  for (int i = 0; i < W; ++i) x.w[i] = u32x4{0, 0, 0, 0};
  if (!row_ok || col >= D) return x;
  if (vec) {  // D is a multiple of 8 here
#pragma unroll
    for (int i = 0; i < W; ++i) x.w[i] = reinterpret_cast<const u32x4*>(row + col)[i];
    return x;
  }
  union {
    Piece<F> p;
    typename F::E e[8];
  } u;
  u.p = x;
#pragma unroll
  for (int s = 0; s < 8; ++s)
    if (col + s < D) u.e[s] = row[col + s];
  return u.p;
}

template <class F>
__device__ __forceinline__ void piece_floats(const Piece<F>& x, float (&v)[8]) {
  if constexpr (sizeof(typename F::E) == 4) {
#pragma unroll
    for (int s = 0; s < 8; ++s) {
      const uint32_t b = x.w[s / 4][s % 4];  // a copy: __builtin_bit_cast of a vector's element reads the vector's first
      v[s] = __builtin_bit_cast(float, b);
    }
  } else {
#pragma unroll
    for (int s = 0; s < 8; ++s) {
      const uint16_t b = (uint16_t)(x.w[0][s / 2] >> (16 * (s & 1)));
      if constexpr (F::NT == 1) v[s] = __builtin_bit_cast(float, (uint32_t)b << 16);
      else v[s] = f16_bits(b);
    }
  }
}

// How a block's threads share the pieces of an [R, D] tile.
template <int R, int D>
struct Share {
  static constexpr int per_row = D / 8;
  static constexpr int total = R * per_row;
  static constexpr int n = (total + kThreads - 1) / kThreads;
  static __device__ __forceinline__ bool mine(int i, int tid) { return total % kThreads == 0 || i * kThreads + tid < total; }
  static __device__ __forceinline__ int row(int i, int tid) { return (i * kThreads + tid) / per_row; }
  static __device__ __forceinline__ int col(int i, int tid) { return (i * kThreads + tid) % per_row * 8; }
};

// Requests rows t0 ... t0+R-1 (those below T) and columns c0 ... c0+D-1 (those below
// width) of one head into registers.
template <class F, int R, int D>
__device__ __forceinline__ void fetch(const View& x, int64_t e, int64_t h, int64_t t0, int64_t T, int c0, int width,
                                      int tid, Piece<F> (&reg)[Share<R, D>::n]) {
  using S = Share<R, D>;
  const auto* base = static_cast<const typename F::E*>(x.p) + e * x.se + h * x.sh;
#pragma unroll
  for (int i = 0; i < S::n; ++i) {
    const int64_t t = t0 + S::row(i, tid);
    reg[i] = load_piece<F>(base + t * x.st, c0 + S::col(i, tid), width, S::mine(i, tid) && t < T, x.vec);
  }
}

template <class F, int R, int D>
__device__ __forceinline__ void stage(Tile<F::NT, R, D>& tile, const Piece<F> (&reg)[Share<R, D>::n], int tid) {
  using S = Share<R, D>;
  constexpr int LD = Tile<F::NT, R, D>::LD;
#pragma unroll
  for (int i = 0; i < S::n; ++i) {
    if (!S::mine(i, tid)) continue;
    const int o = S::row(i, tid) * LD + S::col(i, tid);
    if constexpr (F::NT == 1) {
      *reinterpret_cast<u32x4*>(&tile.p[0][o]) = reg[i].w[0];
    } else {
      float v[8];
      piece_floats<F>(reg[i], v);
      const Frag<F::NT> f = split<F::NT>(v);
#pragma unroll
      for (int n = 0; n < F::NT; ++n) *reinterpret_cast<bf16x8*>(&tile.p[n][o]) = f.t[n];
    }
  }
}

// Four consecutive elements of an output row, rounded once to the storage format
// (nearest even); those past the row's end are dropped.
template <class F>
__device__ __forceinline__ void store4(typename F::E* row, int col, int D, int vec, const float (&x)[4]) {
  if (col >= D) return;
  if constexpr (sizeof(typename F::E) == 4) {
    if (vec) {
      *reinterpret_cast<f32x4*>(row + col) = f32x4{x[0], x[1], x[2], x[3]};
      return;
    }
#pragma unroll
    for (int r = 0; r < 4; ++r)
      if (col + r < D) row[col + r] = x[r];
  } else {
    uint16_t b[4];
#pragma unroll
    for (int r = 0; r < 4; ++r) {
      if constexpr (F::NT == 1) b[r] = __builtin_bit_cast(uint16_t, (__bf16)x[r]);
      else b[r] = __builtin_bit_cast(uint16_t, (_Float16)x[r]);
    }
    if (vec) {
      *reinterpret_cast<uint2*>(row + col) = make_uint2(b[0] | (uint32_t)b[1] << 16, b[2] | (uint32_t)b[3] << 16);
      return;
    }
#pragma unroll
    for (int r = 0; r < 4; ++r)
      if (col + r < D) row[col + r] = b[r];
  }
}

// ------------------------------------------------------------------ decays of a chunk
template <int C>
struct Decay {
  float hi[C], lo[C];  // running sum of log2 a, as two floats
  int seg[C];          // cuts up to and with a step
  float entry[C];      // scale * decay from the chunk's entry, 0 behind a cut
  float leave[C];      // decay to the chunk's end, 0 before a cut
  float across;        // decay over the chunk, 0 if it has a cut
  uint64_t cuts;       // bit i: step i starts afresh
};

constexpr double kLog2E = 1.4426950408889634;
constexpr float kCutBelow = -104.0f;  // exp below this is 0 in float32

__device__ __forceinline__ float exp2_fast(float x) { return __builtin_amdgcn_exp2f(x); }

// One step's log-decay and whether it starts afresh; steps past T have neither.
struct StepDecay {
  float g;
  bool cut;
};

// Lane i's step t0 + i (i < C) of row e, head h.
template <int C>
__device__ __forceinline__ StepDecay load_decay(const Args& a, int64_t e, int64_t h, int64_t t0, int lane) {
  StepDecay s{0.0f, false};
  const int64_t t = t0 + lane;
  if (lane < C && t < a.T) {
    s.g = a.g[e * a.g_se + t * a.g_st + h * a.g_sh];
    s.cut = s.g < kCutBelow || (t > 0 && a.done && a.done[e * a.d_se + (t - 1) * a.d_st] != 0);
    if (s.cut) s.g = 0.0f;
  }
  return s;
}

// One wave fills a chunk's decays.
template <int C>
__device__ __forceinline__ void fill_decay(Decay<C>& d, const StepDecay& s, float scale, int lane) {
  double b = (double)s.g * kLog2E;
#pragma unroll
  for (int o = 1; o < C; o <<= 1) {
    const double up = __shfl_up(b, o);
    if (lane >= o) b += up;
  }
  const double last = __shfl(b, C - 1);
  const uint64_t cuts = __ballot(s.cut);
  const int seg = __popcll(cuts & (~0ull >> (63 - lane)));
  const int total = __popcll(cuts);
  if (lane < C) {
    const float hi = (float)b;
    d.hi[lane] = hi;
    d.lo[lane] = (float)(b - (double)hi);
    d.seg[lane] = seg;
    d.entry[lane] = seg == 0 ? scale * exp2_fast((float)b) : 0.0f;
    d.leave[lane] = seg == total ? exp2_fast((float)(last - b)) : 0.0f;
  }
  if (lane == 0) {
    d.across = total == 0 ? exp2_fast((float)last) : 0.0f;
    d.cuts = cuts;
  }
}

// Decay from step j to step i of a chunk (0 unless j <= i with no cut between).
template <int C>
__device__ __forceinline__ float between(const Decay<C>& d, float hi_i, float lo_i, int seg_i, int i, int j) {
  const float x = (hi_i - d.hi[j]) + (lo_i - d.lo[j]);
  return (j <= i && d.seg[j] == seg_i) ? exp2_fast(x) : 0.0f;
}

}  // namespace la
}  // namespace rlscan

#endif
