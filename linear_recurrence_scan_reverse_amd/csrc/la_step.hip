// Linear attention for one step of many environments (rlscan_linear_attention_step).
//
//   S = a S + k v^T (in place, a = 0 where reset), o = scale * S^T q
//
// Bound by reading and writing the states (K*V floats for each row and head); all
// else is small.  A block takes VB columns of one state: a thread holds four
// columns of RPT rows, requests them all at once, updates, stores, and the block
// sums its rows' products with q through LDS.
//
// Measured: 256 rows of 16 heads of 128 x 128 in float16, states in one of three pools in
// turn: 109 to 117 us, 4.6 to 4.9 TB/s of its 539 MB (a copy: 5.25).  One pool of 315 MB called again and
// again takes 87: the last-level cache keeps part of it.  One row: 5.6 us, a launch and
// two trips to memory.
#include "rlscan_la_launch.hpp"

namespace rlscan {
namespace la {

template <class F>
__device__ __forceinline__ float element(const void* p, int64_t i) {
  if constexpr (sizeof(typename F::E) == 4) return static_cast<const float*>(p)[i];
  else if constexpr (F::NT == 1) return __builtin_bit_cast(float, (uint32_t)static_cast<const uint16_t*>(p)[i] << 16);
  else return f16_bits(static_cast<const uint16_t*>(p)[i]);
}

template <class F, int VB>
__global__ void __launch_bounds__(256) step_kernel(const StepArgs a, int64_t nvs, int vec) {
  constexpr int CG = VB / 4, RG = 256 / CG, RPT = 128 / RG;  // column groups, row groups, rows per thread
  __shared__ float sq[128], sk[128];
  __shared__ f32x4 part[RG][CG];
  const int tid = threadIdx.x, cg = tid % CG, rg = tid / CG;
  const int64_t eh = blockIdx.x / nvs, vs = blockIdx.x % nvs;
  const int64_t e = eh / a.H, h = eh % a.H, hk = h / a.G;
  const int64_t slot = a.slots ? (int64_t)a.slots[e] : e;
  const int v = (int)vs * VB + cg * 4;
  const TileRows<F> out(View{a.out, a.o_se, 0, a.o_sh, 0}, e, h, 0, 1, 1);  // one row
  if (slot < 0 || slot >= a.S) {  // no state: the whole block leaves with a zero output
    const float zero[4] = {0, 0, 0, 0};
    if (rg == 0) store4<F, false>(out, 0, v, a.V, zero);
    return;
  }
  float decay = 0.0f;
  if (!(a.reset && a.reset[e] != 0)) {
    const float g = a.g[e * a.g_se + h * a.g_sh];
    decay = g < kCutBelow ? 0.0f : expf(g);
  }
  float* S = a.state + (slot * a.H + h) * a.K * (int64_t)a.V;
  f32x4 x[RPT];
#pragma unroll
  for (int n = 0; n < RPT; ++n) {
    const int k = n * RG + rg;
    x[n] = f32x4{0, 0, 0, 0};
    if (decay == 0.0f || k >= a.K) continue;  // a state that is dropped is not read
    if (vec) {
      if (v < a.V) x[n] = *reinterpret_cast<const f32x4*>(S + k * a.V + v);
    } else {
#pragma unroll
      for (int r = 0; r < 4; ++r)
        if (v + r < a.V) x[n][r] = S[k * a.V + v + r];
    }
  }
  for (int k = tid; k < 128; k += 256) {
    sq[k] = k < a.K ? a.scale * element<F>(a.q, e * a.q_se + h * a.q_sh + k) : 0.0f;
    sk[k] = k < a.K ? element<F>(a.k, e * a.k_se + hk * a.k_sh + k) : 0.0f;
  }
  f32x4 vv{0, 0, 0, 0};
#pragma unroll
  for (int r = 0; r < 4; ++r)
    if (v + r < a.V) vv[r] = element<F>(a.v, e * a.v_se + hk * a.v_sh + v + r);
  __syncthreads();
  f32x4 o{0, 0, 0, 0};
#pragma unroll
  for (int n = 0; n < RPT; ++n) {
    const int k = n * RG + rg;
    if (k >= a.K) continue;
    x[n] = x[n] * decay + vv * sk[k];
    o += x[n] * sq[k];
    if (vec) {
      if (v < a.V) *reinterpret_cast<f32x4*>(S + k * a.V + v) = x[n];
    } else {
#pragma unroll
      for (int r = 0; r < 4; ++r)
        if (v + r < a.V) S[k * a.V + v + r] = x[n][r];
    }
  }
  part[rg][cg] = o;
  __syncthreads();
  if (rg == 0) {
#pragma unroll
    for (int n = 1; n < RG; ++n) o += part[n][cg];
    const float y[4] = {o[0], o[1], o[2], o[3]};
    store4<F, false>(out, 0, v, a.V, y);
  }
}

template <class F>
hipError_t launch_step_fmt(const StepArgs& a, hipStream_t st) {
  const int vec = a.V % 4 == 0 && (uintptr_t)a.state % 16 == 0;
  // few states: 32 columns a block, so that more compute units share the reads
  if (a.E * a.H * ((a.V + 127) / 128) < 1024) {
    const int64_t nvs = (a.V + 31) / 32;
    step_kernel<F, 32><<<dim3((unsigned)(a.E * a.H * nvs)), 256, 0, st>>>(a, nvs, vec);
  } else {
    const int64_t nvs = (a.V + 127) / 128;
    step_kernel<F, 128><<<dim3((unsigned)(a.E * a.H * nvs)), 256, 0, st>>>(a, nvs, vec);
  }
  return hipGetLastError();
}

hipError_t launch_step(rlscan_format f, const StepArgs& a, hipStream_t st) {
  switch (f) {
    case RLSCAN_FORMAT_BF16: return launch_step_fmt<TBf16>(a, st);
    case RLSCAN_FORMAT_F16: return launch_step_fmt<TF16>(a, st);
    default: return launch_step_fmt<TF32>(a, st);
  }
}

}  // namespace la
}  // namespace rlscan
