// The gated recurrence for one step of many environments (rlscan_gated_recurrence_step):
// the state of each row's slot is updated in place.  A lane for a channel: nothing is shared, and the
// time is latency (256 rows of 2048, float16, in a pool 4.5 us, of which 1.6 would be their bytes; one row of
// 2048 2.8).
#include "rlscan_gr.hpp"

namespace rlscan {
namespace gr {

template <class F>
__global__ void __launch_bounds__(256) step_kernel(const StepArgs p, int64_t tiles) {
  using E = typename F::E;
  const int64_t e = blockIdx.x / tiles, d = blockIdx.x % tiles * 256 + threadIdx.x;
  if (d >= p.D) return;
  E* out = static_cast<E*>(p.out) + e * p.o_se + d;
  const int64_t slot = p.slots ? (int64_t)p.slots[e] : e;
  if (slot < 0 || slot >= p.S) {
    *out = F::put(0.0f);
    return;
  }
  const bool fresh = p.reset && p.reset[e] != 0;
  float* state = p.state + slot * p.D + d;
  const float x = F::get(static_cast<const E*>(p.x)[e * p.x_se + d]);
  const float gi = F::get(static_cast<const E*>(p.ig)[e * p.ig_se + d]);
  const float gd = F::get(static_cast<const E*>(p.dg)[e * p.dg_se + d]);
  const float a = fresh ? 0.0f : decay_of<kEvery>(kLog2E * rate_of(p.rate[d]) * sigmoid(gd), 0.0f);
  const float b = __builtin_amdgcn_sqrtf(one_less_square<kEvery>(a)) * (sigmoid(gi) * x);
  const float h = decayed<kEvery>(a, fresh ? 0.0f : *state) + b;
  *state = h;
  *out = F::put(h);
}

hipError_t launch_step(rlscan_format f, const StepArgs& a, hipStream_t st) {
  const int64_t tiles = (a.D + 255) / 256;
  const dim3 grid((unsigned)(a.E * tiles));
  switch (f) {
    case RLSCAN_FORMAT_BF16: step_kernel<LBf16><<<grid, 256, 0, st>>>(a, tiles); break;
    case RLSCAN_FORMAT_F16: step_kernel<LF16><<<grid, 256, 0, st>>>(a, tiles); break;
    default: step_kernel<LF32><<<grid, 256, 0, st>>>(a, tiles); break;
  }
  return hipGetLastError();
}

}  // namespace gr
}  // namespace rlscan
