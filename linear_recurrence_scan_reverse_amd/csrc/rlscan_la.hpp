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
//
// What is not finite.  A cut or a mask is a weight of 0, and 0 times inf or NaN is NaN; a
// matrix product mixes all rows of a chunk.  So one such element of the rows that reach
// others (k and v, backward also q and do) spoils the state, which stays so to the walk's end.
// There the state is looked at, once; if it is not finite the block walks again with care:
// such elements are taken out of the tiles and of the state before the products, and what
// the recurrence makes of them is written behind the products (Odd).
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

constexpr int kThreads = 256;  // of the walking and the joining kernels

// A strided [E, T, heads, D] tensor (strides in elements, D contiguous).
struct View {
  const void* p;
  int64_t se, st, sh;
  int vec;  // rows can be read and written 16 bytes at a time, at 32-bit offsets within a chunk
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
  float* dg;              // gradient of the log-decays
  int64_t dg_se, dg_st, dg_sh;
  int64_t E, T, H, G;     // G heads share a key/value head
  int K, V;
  float scale;
  float* seg_state;       // workspace [E, H, nseg, KP, VP]: states entering each segment
  float* seg_decay;       // [E, H, nseg]
  int64_t nseg, seg_chunks, chunks;
  int64_t mark_chunks;    // backward: chunks from one marked boundary to the next
};

// What the backward call has besides.
struct Backward {
  const float* d_final;  // [E, H, K, V] or NULL
  float* d_init;         // [E, H, K, V] or NULL
  float* dg_head;        // [H] gradient of one log-decay for each head, or NULL: Args::dg
  View dk, dv;           // Args::dk and dv, or float32 scratch [E, T, H, D] where heads share them
  // workspace
  float *seg_state, *seg_decay;  // as Args'
  float *seg_grad, *seg_gdecay;  // the same for the gradient of the state
  double *u, *w;                 // [E, H, T] q . dq and k . dk
  float* end;                    // [E, H] <S_T, dS_T>
  double* total;                 // [E, H] sums of dg over a row
  float *marks, *mark_grads;     // [E, H, marks, KP * VP] S and dS at the marked boundaries
  double* mark_dots;             // [E, H, marks] <S, dS>
  int64_t nmarks;
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
// TOP: the smallest pairs kept, by the sum of their terms' numbers.
template <int NA, int NB, int TOP = (NA > NB ? NA : NB) - 1>
__device__ __forceinline__ f32x4 mma(const Frag<NA>& a, const Frag<NB>& b, f32x4 acc) {
#pragma unroll
  for (int order = TOP; order >= 0; --order)
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
// A matrix of R rows and D columns, as N planes of bfloat16 terms.  Two layouts,
// each free of bank conflicts in the ways that it is read:
//
// RowTile: rows read 16 bytes at a time by 16 lanes; each row begins 16 bytes further on in the banks.
template <int N, int R, int D>
struct RowTile {
  static constexpr int LD = D + 8;
  __bf16 p[N][R * LD];
};

// MixTile: 8-byte units, the unit's index exchanged with bits of the row (XOR). 32 lanes
// that read 4 neighbouring units of the rows 0-3 and 8-11 (the transpose read), or
// two of each of 16 rows, fall on all 32 places of the banks.
template <int N, int R, int D>
struct MixTile {
  static constexpr int LD = D;
  __bf16 p[N][R * D];
  static __device__ __forceinline__ int swap(int row) {
    const int far = row >> 3 & 1;  // bits 0-1 of the row: the quad of units; 2 and 3: the unit in it
    return ((row & 3) << 2 | (row >> 2 & 1) << 1 | far) ^ (D == 64 ? far << 2 : far << 4);
  }
  static __device__ __forceinline__ int at(int row, int unit) { return row * D + (unit ^ swap(row)) * 4; }
};

// Row `row0 + l%16`, columns kk*32 + (l/16)*8 ... +7.
template <int N, int R, int D>
__device__ __forceinline__ Frag<N> frag_row(const RowTile<N, R, D>& t, int row0, int kk, int lane) {
  Frag<N> f;
  const int o = (row0 + (lane & 15)) * RowTile<N, R, D>::LD + kk * 32 + (lane >> 4) * 8;
#pragma unroll
  for (int n = 0; n < N; ++n) f.t[n] = *reinterpret_cast<const bf16x8*>(&t.p[n][o]);
  return f;
}

// The same row in the order in which two accumulator tiles hold 32 steps: slots
// 0-3 are columns kk*32 + (l/16)*4 ..., slots 4-7 the columns 16 further on.  row0 % 16 == 0.
template <int N, int R, int D>
__device__ __forceinline__ Frag<N> frag_row(const MixTile<N, R, D>& t, int row0, int kk, int lane) {
  using M = MixTile<N, R, D>;
  Frag<N> f;
  const int r = lane & 15, g = lane >> 4;
  const int lo = M::at(r, kk * 8 + g), hi = M::at(r, kk * 8 + 4 + g), far = row0 * D;  // swap repeats every 16 rows
#pragma unroll
  for (int n = 0; n < N; ++n) {
    const bf16x4 x = *reinterpret_cast<const bf16x4*>(&t.p[n][lo + far]);
    const bf16x4 y = *reinterpret_cast<const bf16x4*>(&t.p[n][hi + far]);
    f.t[n] = __builtin_shufflevector(x, y, 0, 1, 2, 3, 4, 5, 6, 7);
  }
  return f;
}

// Column `16 tile + l%16`, rows kk*32 + (l/16)*8 ... +7, by the LDS transpose read: each
// 16 lanes fetch four rows of 16 columns and each gets one column of them.
template <int N, int R, int D>
__device__ __forceinline__ Frag<N> frag_col(const MixTile<N, R, D>& t, int tile, int kk, int lane) {
  using lds_s16x4 = __attribute__((address_space(3))) s16x4;
  Frag<N> f;
  const int i = lane & 15, r = (lane >> 4) * 8 + (i >> 2);
  const int first = MixTile<N, R, D>::at(r, tile * 4 + (i & 3)), second = MixTile<N, R, D>::at(r + 4, tile * 4 + (i & 3));
  const int far = kk * 32 * D;
#pragma unroll
  for (int n = 0; n < N; ++n) {
    union {
      s16x4 h[2];
      bf16x8 v;
    } u;
    u.h[0] = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_s16x4*)(&t.p[n][first + far]));
    u.h[1] = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_s16x4*)(&t.p[n][second + far]));
    f.t[n] = u.v;
  }
  return f;
}

// Four consecutive columns of one row, from the values of an accumulator.
template <int N, int R, int D>
__device__ __forceinline__ void put4(RowTile<N, R, D>& t, int row, int col, const float (&x)[4]) {
  bf16x4 w[N];
#pragma unroll
  for (int r = 0; r < 4; ++r) {
    __bf16 s[N];
    split1<N>(x[r], s);
#pragma unroll
    for (int n = 0; n < N; ++n) w[n][r] = s[n];
  }
#pragma unroll
  for (int n = 0; n < N; ++n) *reinterpret_cast<bf16x4*>(&t.p[n][row * RowTile<N, R, D>::LD + col]) = w[n];
}

// Four consecutive columns of one row, as floats.
template <int N, int R, int D>
__device__ __forceinline__ void get4(const MixTile<N, R, D>& t, int row, int col, float (&x)[4]) {
  const int o = MixTile<N, R, D>::at(row, col / 4);
#pragma unroll
  for (int r = 0; r < 4; ++r) x[r] = 0.0f;
#pragma unroll
  for (int n = N - 1; n >= 0; --n) {
    const bf16x4 w = *reinterpret_cast<const bf16x4*>(&t.p[n][o]);
#pragma unroll
    for (int r = 0; r < 4; ++r) x[r] += (float)w[r];
  }
}

// x, unknown to the compiler: what a rare branch computes from it stays in the branch.
__device__ __forceinline__ int rarely(int x) {
  asm volatile("" : "+v"(x));
  return x;
}

// The kernel's argument, a struct of type T, read from memory once more: a rare branch that
// takes it keeps no register of the ones before busy.
template <class T>
__device__ __forceinline__ T argument_again() {
  auto* p = __builtin_amdgcn_kernarg_segment_ptr();
  asm volatile("" : "+s"(p));
  T t;
  __builtin_memcpy(&t, (const void*)p, sizeof t);
  return t;
}

// Whether one of n values is not finite: 0 times them adds up to NaN.
template <int N>
__device__ __forceinline__ bool any_odd(const f32x4 (&x)[N]) {
  float sum = 0.0f;
#pragma unroll
  for (int i = 0; i < N; ++i)
#pragma unroll
    for (int r = 0; r < 4; ++r) sum = __builtin_fmaf(0.0f, x[i][r], sum);
  return sum != sum;
}

// Takes what is not finite out of a thread's part of the state; returns which it was.
template <int N>
__device__ __forceinline__ uint32_t take_odd(f32x4 (&x)[N]) {
  static_assert(N <= 8, "a bit for each");
  uint32_t bits = 0;
#pragma unroll
  for (int i = 0; i < N; ++i)
#pragma unroll
    for (int r = 0; r < 4; ++r) {
      const float v = x[i][r];
      if (0.0f * v == 0.0f) continue;
      bits |= 1u << (i * 4 + r);
      x[i][r] = 0.0f;
    }
  return bits;
}

// The elements of a chunk that are not finite, in a careful walk: bit y of a mask is row y of
// the tiles.
template <int C, int AD, int CD, int NTHR>
struct Odd {
  uint32_t wave[NTHR / 64];  // whether a wave's state is not finite at the end
  uint32_t bits[CD / 16 / (NTHR / 64)][NTHR];  // take_odd of each thread's states
  uint32_t state[CD];        // for each column, whether it has one in the state entering the chunk
  uint64_t b[AD], c[CD];     // for each column of the tiles, the rows in which it has one
  uint64_t before[C];        // for each row, those that reach it: at or before it, no cut between
  uint64_t leaving;          // rows that reach the state behind the chunk
};

// Whether any thread of the block says so.
template <int NTHR>
__device__ __forceinline__ bool any_of_block(uint32_t (&wave)[NTHR / 64], bool mine, int tid) {
  const bool any = __ballot(mine) != 0;
  if ((tid & 63) == 0) wave[tid >> 6] = any;
  __syncthreads();
  return __ballot(wave[(tid & 63) % (NTHR / 64)] != 0) != 0;
}

// Sets every element of column `col` that is not finite to 0; returns their rows.
template <int N, int R, int D>
__device__ __forceinline__ uint64_t take_odd(MixTile<N, R, D>& t, int col) {
  uint64_t rows = 0;
#pragma unroll 1
  for (int r = 0; r < R; ++r) {
    const int o = MixTile<N, R, D>::at(r, col / 4) + col % 4;
    if ((__builtin_bit_cast(uint16_t, t.p[0][o]) & 0x7f80) != 0x7f80) continue;
    rows |= 1ull << r;
#pragma unroll
    for (int n = 0; n < N; ++n) t.p[n][o] = (__bf16)0.0f;
  }
  return rows;
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

// w x, and 0 where w is 0 whatever x is (the instruction v_mul_legacy_f32).
extern "C" __device__ float rlscan_la_gated(float w, float x) __asm("llvm.amdgcn.fmul.legacy");
__device__ __forceinline__ float gated(float w, float x) { return rlscan_la_gated(w, x); }

// Nothing moves across in the compiler's schedule: keeps it from requesting the operands of
// all products at once, which costs twice the registers and half the waves.
__device__ __forceinline__ void hold_schedule() { __builtin_amdgcn_sched_barrier(0); }

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

// How a block's NTHR threads share the pieces of an [R, D] tile.
template <int R, int D, int NTHR = kThreads>
struct Share {
  static constexpr int per_row = D / 8;
  static constexpr int total = R * per_row;
  static constexpr int n = (total + NTHR - 1) / NTHR;
  static __device__ __forceinline__ bool mine(int i, int tid) { return total % NTHR == 0 || i * NTHR + tid < total; }
  static __device__ __forceinline__ int row(int i, int tid) { return (i * NTHR + tid) / per_row; }
  static __device__ __forceinline__ int col(int i, int tid) { return (i * NTHR + tid) % per_row * 8; }
};

constexpr uint32_t kNowhere = 0x80000000u;  // an offset past every tile: reads 0, writes nothing

// One head's rows of up to R steps from t0, as a buffer resource over exactly those
// below T: rows behind the end read as 0 and drop what is written to them.
template <class F>
struct TileRows {
  const typename F::E* p;  // row 0
  int64_t st;              // elements between rows
  int left;                // rows below T
  __device__ __forceinline__ TileRows(const View& x, int64_t e, int64_t h, int64_t t0, int64_t T, int R)
      : p(static_cast<const typename F::E*>(x.p) + e * x.se + h * x.sh + t0 * x.st),
        st(x.st),
        left(T - t0 < R ? (int)(T - t0) : R) {}
  // The tile `chunks` of R rows further on.
  __device__ __forceinline__ void move(int64_t chunks, int64_t t0, int64_t T, int R) {
    p += chunks * R * st;
    left = T - t0 < R ? (int)(T - t0) : R;
  }
  __device__ __forceinline__ __amdgpu_buffer_rsrc_t resource(int D) const {
    const int n = left > 0 ? (int)(((left - 1) * st + D) * (int64_t)sizeof(typename F::E)) : 0;
    return __builtin_amdgcn_make_buffer_rsrc(const_cast<typename F::E*>(p), 0, n, 0x00020000);
  }
  __device__ __forceinline__ uint32_t offset(int r, int col, int D) const {
    return col < D ? (uint32_t)(r * (int)st + col) * (uint32_t)sizeof(typename F::E) : kNowhere;
  }
};

// Requests the columns c0 ... c0+D-1 (those below width) of R steps of one head into
// registers; REV: tile row r is step R-1 - r.  VEC: rows can be read 16 bytes at a time
// (View::vec), else element by element.
template <class F, int R, int D, int NTHR, bool REV, bool VEC>
__device__ __forceinline__ void fetch(const TileRows<F>& rows, int c0, int width, int tid,
                                      Piece<F> (&reg)[Share<R, D, NTHR>::n]) {
  using S = Share<R, D, NTHR>;
  if constexpr (VEC) {
    const auto rs = rows.resource(width);
#pragma unroll
    for (int i = 0; i < S::n; ++i) {
      const int r = REV ? R - 1 - S::row(i, tid) : S::row(i, tid);
      const uint32_t o = S::mine(i, tid) ? rows.offset(r, c0 + S::col(i, tid), width) : kNowhere;
#pragma unroll
      for (int k = 0; k < (int)(sizeof(reg[i].w) / 16); ++k)
        reg[i].w[k] = __builtin_bit_cast(u32x4, __builtin_amdgcn_raw_buffer_load_b128(rs, o + 16 * k, 0, 0));
    }
  } else {
#pragma unroll
    for (int i = 0; i < S::n; ++i) {
      const int r = REV ? R - 1 - S::row(i, tid) : S::row(i, tid);
      union {
        Piece<F> p;
        typename F::E e[8];
      } u;
#pragma unroll
      for (int k = 0; k < 8; ++k) {
        const int col = c0 + S::col(i, tid) + k;
        u.e[k] = 0;
        if (S::mine(i, tid) && r < rows.left && col < width) u.e[k] = rows.p[r * rows.st + col];
      }
      reg[i] = u.p;
      hold_schedule();
    }
  }
}

// Writes a thread's pieces to LDS.  Where a RowTile is multiplied with MixTiles its columns
// lie in their order (frag_row): of every 32, units 0 4 1 5 2 6 3 7.
template <class F, int NTHR, class T, int R, int D>
__device__ __forceinline__ void stage_pieces(T& tile, const Piece<F> (&reg)[Share<R, D, NTHR>::n], int tid) {
  using S = Share<R, D, NTHR>;
#pragma unroll
  for (int i = 0; i < S::n; ++i) {
    if (!S::mine(i, tid)) continue;
    const int row = S::row(i, tid), col = S::col(i, tid);
    int first, second;
    if constexpr (__is_same(T, MixTile<F::NT, R, D>)) {
      first = T::at(row, col / 4);
      second = T::at(row, col / 4 + 1);
    } else {
      first = row * T::LD + (col & ~31) + (col >> 3 & 1) * 16 + (col >> 4 & 1) * 4;
      second = first + 8;
    }
    if constexpr (F::NT == 1) {
      const bf16x8 w = __builtin_bit_cast(bf16x8, reg[i]);
      *reinterpret_cast<bf16x4*>(&tile.p[0][first]) = __builtin_shufflevector(w, w, 0, 1, 2, 3);
      *reinterpret_cast<bf16x4*>(&tile.p[0][second]) = __builtin_shufflevector(w, w, 4, 5, 6, 7);
    } else {
      float v[8];
      piece_floats<F>(reg[i], v);
      const Frag<F::NT> f = split<F::NT>(v);
#pragma unroll
      for (int n = 0; n < F::NT; ++n) {
        *reinterpret_cast<bf16x4*>(&tile.p[n][first]) = __builtin_shufflevector(f.t[n], f.t[n], 0, 1, 2, 3);
        *reinterpret_cast<bf16x4*>(&tile.p[n][second]) = __builtin_shufflevector(f.t[n], f.t[n], 4, 5, 6, 7);
      }
    }
  }
}

template <class F, int NTHR, int R, int D>
__device__ __forceinline__ void stage(RowTile<F::NT, R, D>& tile, const Piece<F> (&reg)[Share<R, D, NTHR>::n], int tid) {
  stage_pieces<F, NTHR, RowTile<F::NT, R, D>, R, D>(tile, reg, tid);
}

template <class F, int NTHR, int R, int D>
__device__ __forceinline__ void stage(MixTile<F::NT, R, D>& tile, const Piece<F> (&reg)[Share<R, D, NTHR>::n], int tid) {
  stage_pieces<F, NTHR, MixTile<F::NT, R, D>, R, D>(tile, reg, tid);
}

// Columns col ... col+3 of row r, as they lie in memory; zeros past the end.
template <class F>
struct Quad {
  uint32_t w[sizeof(typename F::E)];
};

template <class F, bool VEC>
__device__ __forceinline__ Quad<F> load4(const TileRows<F>& rows, int r, int col, int D) {
  typedef uint32_t u32x2 __attribute__((ext_vector_type(2)));
  Quad<F> q;
  if constexpr (VEC) {
    const auto rs = rows.resource(D);
    const uint32_t o = rows.offset(r, col, D);
    if constexpr (sizeof(typename F::E) == 4) {
      const u32x4 w = __builtin_bit_cast(u32x4, __builtin_amdgcn_raw_buffer_load_b128(rs, o, 0, 0));
      __builtin_memcpy(&q, &w, sizeof q);
    } else {
      const u32x2 w = __builtin_bit_cast(u32x2, __builtin_amdgcn_raw_buffer_load_b64(rs, o, 0, 0));
      __builtin_memcpy(&q, &w, sizeof q);
    }
  } else {
    typename F::E b[4] = {0, 0, 0, 0};
#pragma unroll
    for (int k = 0; k < 4; ++k)
      if (r < rows.left && col + k < D) b[k] = rows.p[r * rows.st + col + k];
    __builtin_memcpy(&q, b, sizeof q);
  }
  return q;
}

template <class F>
__device__ __forceinline__ float quad_float(const Quad<F>& q, int k) {
  if constexpr (sizeof(typename F::E) == 4) return __builtin_bit_cast(float, q.w[k]);
  const uint16_t b = (uint16_t)(q.w[k / 2] >> (16 * (k & 1)));
  if constexpr (F::NT == 1) return __builtin_bit_cast(float, (uint32_t)b << 16);
  else return f16_bits(b);
}

// Columns col ... col+3 of row r, rounded once to the storage format (nearest even);
// what lies past the end is dropped.
template <class F, bool VEC>
__device__ __forceinline__ void store4(const TileRows<F>& rows, int r, int col, int D, const float (&x)[4]) {
  typedef uint32_t u32x2 __attribute__((ext_vector_type(2)));
  typename F::E b[4];
#pragma unroll
  for (int k = 0; k < 4; ++k) {
    if constexpr (sizeof(b[0]) == 4) b[k] = x[k];
    else if constexpr (F::NT == 1) b[k] = __builtin_bit_cast(uint16_t, (__bf16)x[k]);
    else b[k] = __builtin_bit_cast(uint16_t, (_Float16)x[k]);
  }
  if constexpr (VEC) {
    const auto rs = rows.resource(D);
    const uint32_t o = rows.offset(r, col, D);
    if constexpr (sizeof(b[0]) == 4) {
      u32x4 w;
      __builtin_memcpy(&w, b, sizeof w);
      __builtin_amdgcn_raw_buffer_store_b128(w, rs, o, 0, 0);
    } else {
      u32x2 w;
      __builtin_memcpy(&w, b, sizeof w);
      __builtin_amdgcn_raw_buffer_store_b64(w, rs, o, 0, 0);
    }
  } else {
    auto* p = const_cast<typename F::E*>(rows.p) + r * rows.st + col;
#pragma unroll
    for (int k = 0; k < 4; ++k)
      if (r < rows.left && col + k < D) p[k] = b[k];
  }
}

// A NaN to column col of row r.
template <class F, bool VEC>
__device__ __forceinline__ void store_nan(const TileRows<F>& rows, int r, int col, int D) {
  constexpr auto bits = sizeof(typename F::E) == 4 ? 0x7fc00000u : F::NT == 1 ? 0x7fc0u : 0x7e00u;
  if constexpr (VEC) {
    const auto rs = rows.resource(D);
    const uint32_t o = rows.offset(r, col, D);
    if constexpr (sizeof(typename F::E) == 4) __builtin_amdgcn_raw_buffer_store_b32(bits, rs, o, 0, 0);
    else __builtin_amdgcn_raw_buffer_store_b16((uint16_t)bits, rs, o, 0, 0);
  } else if (r < rows.left && col < D) {
    auto* p = const_cast<typename F::E*>(rows.p) + r * rows.st + col;
    if constexpr (sizeof(typename F::E) == 4) *p = __builtin_bit_cast(float, bits);
    else *p = (uint16_t)bits;
  }
}

// ------------------------------------------------------------------ decays of a chunk
// Tile row r is step t0 + r, or with REV step t0 + C-1 - r: rows follow the walk.
template <int C>
struct alignas(16) Decay {
  float hi[C], lo[C];  // running sum of log2 a (REV: its negative), as two floats
  int seg[C];          // number of the row's episode within the chunk
  float more[C];       // not a decay: hi ... more are free once P is formed, 4*C floats
  float in[C];         // weight of the state entering the chunk (in walking order)
  float out[C];        // weight of a row in the state leaving it
  float across;        // decay over the chunk, 0 if it has a cut
};

constexpr double kLog2E = 1.4426950408889634;
constexpr float kCutBelow = -104.0f;  // exp below this is 0 in float32

__device__ __forceinline__ float exp2_fast(float x) { return __builtin_amdgcn_exp2f(x); }

// What one step's decay is made of, as it lies in memory: requested early, looked at late.
struct StepDecay {
  float g;        // 0 past the row's end
  uint32_t done;  // of the step before
};

// Lane i's step t0 + i (i < C) of row e, head h.
template <int C>
__device__ __forceinline__ StepDecay load_decay(const Args& a, int64_t e, int64_t h, int64_t t0, int lane) {
  StepDecay s{0.0f, 0};
  const int64_t t = t0 + lane;
  if (lane < C && t >= 0 && t < a.T) {
    s.g = a.g[e * a.g_se + t * a.g_st + h * a.g_sh];
    if (a.done && t > 0) s.done = a.done[e * a.d_se + (t - 1) * a.d_st];
  }
  return s;
}

// A DPP move of a double; 0 where the pattern has no source or the row is masked off.
template <int CTRL, int ROWS>
__device__ __forceinline__ double lane_shift(double x) {
  const uint64_t b = __builtin_bit_cast(uint64_t, x);
  const uint32_t lo = (uint32_t)__builtin_amdgcn_update_dpp(0, (int)(uint32_t)b, CTRL, ROWS, 0xf, true);
  const uint32_t hi = (uint32_t)__builtin_amdgcn_update_dpp(0, (int)(uint32_t)(b >> 32), CTRL, ROWS, 0xf, true);
  return __builtin_bit_cast(double, (uint64_t)hi << 32 | lo);
}

__device__ __forceinline__ double read_lane(double x, int lane) {
  const uint64_t b = __builtin_bit_cast(uint64_t, x);
  const uint32_t lo = (uint32_t)__builtin_amdgcn_readlane((int)(uint32_t)b, lane);
  const uint32_t hi = (uint32_t)__builtin_amdgcn_readlane((int)(uint32_t)(b >> 32), lane);
  return __builtin_bit_cast(double, (uint64_t)hi << 32 | lo);
}

// A lane's share of a chunk's decays.
struct LaneDecay {
  float hi, lo, in, out, across;
  int seg;
};

// One wave computes them.  Forward, the entering state is read through scale * decay from the
// entry, and rows leave through the decay to the end; backward in time it is the
// other way round.
template <int C, bool REV>
__device__ __forceinline__ LaneDecay scan_decay(const StepDecay& s, float scale, int lane) {
  const bool cut = s.done != 0 || s.g < kCutBelow;  // the step starts afresh
  double b = cut ? 0.0 : (double)s.g * kLog2E;
  b += lane_shift<0x111, 0xf>(b);  // row_shr 1, 2, 4, 8: sums within 16 lanes
  b += lane_shift<0x112, 0xf>(b);
  b += lane_shift<0x114, 0xf>(b);
  b += lane_shift<0x118, 0xf>(b);
  b += lane_shift<0x142, 0xa>(b);  // row_bcast 15 and 31: the sums of the rows before
  b += lane_shift<0x143, 0xc>(b);
  const double last = read_lane(b, 63);  // lanes past C added 0
  const uint64_t cuts = __ballot(cut);
  const int total = __popcll(cuts);
  LaneDecay d;
  d.seg = __popcll(cuts & (~0ull >> (63 - lane)));
  const double sum = REV ? -b : b;
  d.hi = (float)sum;
  d.lo = (float)(sum - (double)d.hi);
  const float entry = d.seg == 0 ? scale * exp2_fast((float)b) : 0.0f;
  const float leave = d.seg == total ? exp2_fast((float)(last - b)) : 0.0f;
  d.in = REV ? leave : entry;
  d.out = REV ? entry : leave;
  d.across = total == 0 ? exp2_fast((float)last) : 0.0f;
  return d;
}

template <int C, bool REV>
__device__ __forceinline__ void put_decay(Decay<C>& t, const LaneDecay& d, int lane) {
  if (lane < C) {
    const int r = REV ? C - 1 - lane : lane;
    t.hi[r] = d.hi;
    t.lo[r] = d.lo;
    t.seg[r] = d.seg;
    t.in[r] = d.in;
    t.out[r] = d.out;
  }
  if (lane == 0) t.across = d.across;
}

// By the whole block, between barriers: takes what is not finite out of the tiles and says
// which rows it reaches.
template <int N, int C, int AD, int CD, int NTHR>
__device__ __forceinline__ void sweep_odd(Odd<C, AD, CD, NTHR>& odd, MixTile<N, C, AD>& b, MixTile<N, C, CD>& c,
                                          const Decay<C>& d, int tid) {
  for (int i = tid; i < AD + CD; i += NTHR) {
    if (i < AD) odd.b[i] = take_odd(b, i);
    else odd.c[i - AD] = take_odd(c, i - AD);
  }
  if (tid < C) {
    uint64_t rows = 0;
    const int seg = d.seg[tid];
#pragma unroll 1
    for (int y = 0; y <= tid; ++y) rows |= (uint64_t)(d.seg[y] == seg) << y;
    odd.before[tid] = rows;
  }
  if (tid < 64) {
    const uint64_t rows = __ballot(tid < C && d.out[tid < C ? tid : 0] != 0.0f);
    if (tid == 0) odd.leaving = rows;
  }
}

// scale * decay between row x and the rows y ... y+3 of a chunk (0 unless y + r <= x with
// no cut between).
template <int C>
__device__ __forceinline__ void between4(const Decay<C>& d, float scale, int x, int y, float (&v)[4]) {
  typedef int i32x4 __attribute__((ext_vector_type(4)));
  const float hi_x = d.hi[x], lo_x = d.lo[x];
  const int seg_x = d.seg[x];
  const f32x4 hi = *reinterpret_cast<const f32x4*>(&d.hi[y]);
  const f32x4 lo = *reinterpret_cast<const f32x4*>(&d.lo[y]);
  const i32x4 seg = *reinterpret_cast<const i32x4*>(&d.seg[y]);
#pragma unroll
  for (int r = 0; r < 4; ++r) {
    const float w = scale * exp2_fast((hi_x - hi[r]) + (lo_x - lo[r]));
    v[r] = (y + r <= x) & (seg[r] == seg_x) ? w : 0.0f;
  }
}

// Whether the row's last step ends an episode, so that nothing leaves the row.
__device__ __forceinline__ bool row_closed(const Args& a, int64_t e) {
  return a.T > 0 && a.done && a.done[e * a.d_se + (a.T - 1) * a.d_st] != 0;
}

}  // namespace la
}  // namespace rlscan

#endif
