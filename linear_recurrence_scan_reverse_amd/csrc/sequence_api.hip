// sequence_api.hip -- the C ABI of what a policy over token sequences has besides attention
// and sampling (declared in include/rlscan.h): the gated recurrence.  Every entry validates
// on the host before any HIP call and enqueues its kernels on the caller's stream; scratch
// memory comes from the caller.
#include <cmath>
#include <cstdint>

#include "rlscan.h"
#include "rlscan_checks.hpp"
#include "rlscan_gr.hpp"

namespace {

using namespace rlscan::checks;

constexpr int64_t kMaxBlocks = ((int64_t)1 << 22) - 1;  // of up to 1024 threads: below 2^32 work-items

bool layout_ok(rlscan_layout l) { return l == RLSCAN_LAYOUT_ENV_MAJOR || l == RLSCAN_LAYOUT_TIME_MAJOR; }

// Sizes that the entries of the gated recurrence take.
rlscan_status check_recurrence(rlscan_format f, int64_t E, int64_t T, int64_t D) {
  if (E < 0 || T < 0 || T >= RLSCAN_MAX_T || D < 0) return RLSCAN_ERR_SHAPE;
  if (D > 0 && E > kMaxElems / D) return RLSCAN_ERR_SHAPE;
  if (E * D > 0 && T > kMaxElems / (E * D)) return RLSCAN_ERR_SHAPE;
  if (elem_size(f) == 0) return RLSCAN_ERR_PARAM;
  if (E > 0 && (D + 63) / 64 > kMaxBlocks / E) return RLSCAN_ERR_SHAPE;
  return RLSCAN_OK;
}

int64_t marks_bytes(int64_t E, int64_t T, int64_t D) {
  return E * ((T + rlscan::gr::kMark - 1) / rlscan::gr::kMark) * D * 4;
}

void fill_recurrence(rlscan::gr::Args& a, const rlscan::gr::Plan& p, rlscan_layout l, const float* rate,
                     const uint8_t* done, int64_t E, int64_t T, int64_t D, void* workspace) {
  const bool tm = l == RLSCAN_LAYOUT_TIME_MAJOR;
  a.rate = rate;
  a.done = done;
  a.d_se = tm ? 1 : T;
  a.d_st = tm ? E : 1;
  a.E = E;
  a.T = T;
  a.D = D;
  a.nseg = p.nseg;
  a.seg_steps = p.seg_steps;
  a.groups = p.groups;
  float* ws = static_cast<float*>(workspace);
  a.seg_a = ws;
  a.seg_y = ws + p.seg;
  a.rate_part = p.part > 0 ? ws + 2 * p.seg : nullptr;
}

}  // namespace

extern "C" {

int64_t rlscan_gated_recurrence_workspace(rlscan_format fmt, int64_t E, int64_t T, int64_t D, int backward) {
  if (check_recurrence(fmt, E, T, D) != RLSCAN_OK) return -1;
  if (E * D == 0) return 0;
  return rlscan::gr::make_plan(fmt, E, T, D, backward != 0).floats * (int64_t)sizeof(float);
}

rlscan_status rlscan_gated_recurrence(rlscan_format fmt, rlscan_layout layout, const rlscan_heads* x,
                                      const rlscan_heads* input_gate, const rlscan_heads* decay_gate,
                                      const float* rate, const uint8_t* done, const float* init_state,
                                      const rlscan_heads* out, float* final_state, float* marks, void* workspace,
                                      int64_t workspace_bytes, int64_t E, int64_t T, int64_t D, hipStream_t stream) {
  rlscan_status st = check_recurrence(fmt, E, T, D);
  if (st != RLSCAN_OK) return st;
  if (!layout_ok(layout)) return RLSCAN_ERR_PARAM;
  if (E * D == 0 || (T == 0 && !final_state)) return RLSCAN_OK;
  const rlscan::gr::Plan p = rlscan::gr::make_plan(fmt, E, T, D, false);
  const int64_t need = p.floats * (int64_t)sizeof(float);
  rlscan::gr::Args a{};
  Spans io;
  if (!rate) return RLSCAN_ERR_NULL;
  if (T > 0) {
    HeadsCheck c{E, T, elem_size(fmt)};
    a.x = c.view(x, 1, D, false, io);
    a.ig = c.view(input_gate, 1, D, false, io);
    a.dg = c.view(decay_gate, 1, D, false, io);
    a.out = c.view(out, 1, D, true, io);
    if (c.st != RLSCAN_OK) return c.st;
  }
  if (need > 0 && !workspace) return RLSCAN_ERR_NULL;
  if (workspace_bytes < need) return RLSCAN_ERR_WORKSPACE;
  if (!aligned(rate, 4) || !aligned(init_state, 4) || !aligned(final_state, 4) || !aligned(marks, 4) ||
      !aligned(workspace, 16))
    return RLSCAN_ERR_ALIGN;
  io.add_in(plain(rate, D * 4));
  io.add_in(plain(done, E * T));
  io.add_in(plain(init_state, E * D * 4));
  io.add_out(plain(final_state, E * D * 4));
  io.add_out(plain(marks, marks_bytes(E, T, D)));
  io.add_out(plain(workspace, need));
  if (io.clash()) return RLSCAN_ERR_ALIAS;
  fill_recurrence(a, p, layout, rate, done, E, T, D, workspace);
  a.init = init_state;
  a.final_state = final_state;
  a.marks = marks;
  return launched(rlscan::gr::launch_forward(fmt, a, p, stream));
}

rlscan_status rlscan_gated_recurrence_backward(
    rlscan_format fmt, rlscan_layout layout, const rlscan_heads* d_out, const rlscan_heads* x,
    const rlscan_heads* input_gate, const rlscan_heads* decay_gate, const float* rate, const float* marks,
    const uint8_t* done, const float* d_final_state, const rlscan_heads* dx, const rlscan_heads* d_input_gate,
    const rlscan_heads* d_decay_gate, float* d_rate, float* d_init_state, void* workspace, int64_t workspace_bytes,
    int64_t E, int64_t T, int64_t D, hipStream_t stream) {
  rlscan_status st = check_recurrence(fmt, E, T, D);
  if (st != RLSCAN_OK) return st;
  if (!layout_ok(layout)) return RLSCAN_ERR_PARAM;
  if (D == 0) return RLSCAN_OK;
  if (!rate || !d_rate) return RLSCAN_ERR_NULL;
  const rlscan::gr::Plan p = rlscan::gr::make_plan(fmt, E, T, D, true);
  const int64_t need = E > 0 ? p.floats * (int64_t)sizeof(float) : 0;
  rlscan::gr::Args a{};
  Spans io;
  if (E * T > 0) {
    if (!marks) return RLSCAN_ERR_NULL;
    HeadsCheck c{E, T, elem_size(fmt)};
    a.dout = c.view(d_out, 1, D, false, io);
    a.x = c.view(x, 1, D, false, io);
    a.ig = c.view(input_gate, 1, D, false, io);
    a.dg = c.view(decay_gate, 1, D, false, io);
    a.dx = c.view(dx, 1, D, true, io);
    a.dig = c.view(d_input_gate, 1, D, true, io);
    a.ddg = c.view(d_decay_gate, 1, D, true, io);
    if (c.st != RLSCAN_OK) return c.st;
  }
  if (need > 0 && !workspace) return RLSCAN_ERR_NULL;
  if (workspace_bytes < need) return RLSCAN_ERR_WORKSPACE;
  if (!aligned(rate, 4) || !aligned(marks, 4) || !aligned(d_final_state, 4) || !aligned(d_rate, 4) ||
      !aligned(d_init_state, 4) || !aligned(workspace, 16))
    return RLSCAN_ERR_ALIGN;
  io.add_in(plain(rate, D * 4));
  io.add_in(plain(marks, marks_bytes(E, T, D)));
  io.add_in(plain(done, E * T));
  io.add_in(plain(d_final_state, E * D * 4));
  io.add_out(plain(d_rate, D * 4));
  io.add_out(plain(d_init_state, E * D * 4));
  io.add_out(plain(workspace, need));
  if (io.clash()) return RLSCAN_ERR_ALIAS;
  fill_recurrence(a, p, layout, rate, done, E, T, D, workspace);
  if (E == 0) a.groups = 1;  // one block a tile, which writes zeros
  a.marks = const_cast<float*>(marks);
  a.d_final = d_final_state;
  a.d_rate = d_rate;
  a.d_init = d_init_state;
  return launched(rlscan::gr::launch_backward(fmt, a, p, stream));
}

rlscan_status rlscan_gated_recurrence_step(rlscan_format fmt, const rlscan_heads* x, const rlscan_heads* input_gate,
                                           const rlscan_heads* decay_gate, const float* rate, const uint8_t* reset,
                                           const int32_t* slots, float* state, const rlscan_heads* out, int64_t E,
                                           int64_t S, int64_t D, hipStream_t stream) {
  rlscan_status st = check_recurrence(fmt, E, 1, D);
  if (st != RLSCAN_OK) return st;
  if (S < 0 || (D > 0 && S > kMaxElems / D) || (!slots && S < E)) return RLSCAN_ERR_SHAPE;
  if (E * D == 0) return RLSCAN_OK;
  if (!rate || (!state && S > 0)) return RLSCAN_ERR_NULL;
  Spans io;
  HeadsCheck c{E, 1, elem_size(fmt)};
  const View vx = c.view(x, 1, D, false, io);
  const View vi = c.view(input_gate, 1, D, false, io);
  const View vd = c.view(decay_gate, 1, D, false, io);
  const View vo = c.view(out, 1, D, true, io);
  if (c.st != RLSCAN_OK) return c.st;
  if (!aligned(rate, 4) || !aligned(slots, 4) || !aligned(state, 4)) return RLSCAN_ERR_ALIGN;
  io.add_in(plain(rate, D * 4));
  io.add_in(plain(reset, E));
  io.add_in(plain(slots, E * 4));
  io.add_out(plain(state, S * D * 4));
  if (io.clash()) return RLSCAN_ERR_ALIAS;
  rlscan::gr::StepArgs a{};
  a.x = vx.p;
  a.x_se = vx.se;
  a.ig = vi.p;
  a.ig_se = vi.se;
  a.dg = vd.p;
  a.dg_se = vd.se;
  a.out = const_cast<void*>(vo.p);
  a.o_se = vo.se;
  a.rate = rate;
  a.reset = reset;
  a.slots = slots;
  a.state = state;
  a.E = E;
  a.S = S;
  a.D = D;
  return launched(rlscan::gr::launch_step(fmt, a, stream));
}

}  // extern "C"
