// sequence_api.hip -- the C ABI of what a policy over token sequences has besides attention
// and sampling (declared in include/rlscan.h): the gated recurrence, normalised and rotated heads,
// and rows of a table by token.  Every entry validates
// on the host before any HIP call and enqueues its kernels on the caller's stream; scratch
// memory comes from the caller.
#include <cmath>
#include <cstdint>

#include "rlscan.h"
#include "rlscan_checks.hpp"
#include "rlscan_embed.hpp"
#include "rlscan_gr.hpp"
#include "rlscan_nr.hpp"

namespace {

using namespace rlscan::checks;

constexpr int64_t kMaxBlocks = ((int64_t)1 << 22) - 1;  // of up to 1024 threads: below 2^32 work-items
constexpr int64_t kMaxHeads = (int64_t)1 << 20;

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
                     const uint8_t* done, const uint8_t* reset, int64_t E, int64_t T, int64_t D, void* workspace) {
  const bool tm = l == RLSCAN_LAYOUT_TIME_MAJOR;
  a.rate = rate;
  a.done = done;
  a.reset = reset;
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

// Sizes that the entries of the heads take.
rlscan_status check_heads(rlscan_format f, int64_t E, int64_t T, int64_t H, int64_t Hk, int64_t D, int64_t rotate,
                          float base, float eps) {
  if (E < 0 || T < 0 || T >= RLSCAN_MAX_T || H < 0 || Hk < 0) return RLSCAN_ERR_SHAPE;
  if (D < 1 || D > RLSCAN_MAX_NORM_DIM || rotate < 0 || rotate > D || rotate % 2 != 0) return RLSCAN_ERR_SHAPE;
  if (E > 0 && T > kMaxElems / E) return RLSCAN_ERR_SHAPE;  // tokens are counted where there are no heads too
  if (H > kMaxHeads || H + Hk > kMaxHeads || (E > 0 && H + Hk > kMaxElems / D / E)) return RLSCAN_ERR_SHAPE;
  if (E * (H + Hk) > 0 && T > kMaxElems / D / (E * (H + Hk))) return RLSCAN_ERR_SHAPE;
  if (elem_size(f) == 0) return RLSCAN_ERR_PARAM;
  if (!(base > 0.0f && std::isfinite(base)) || !(eps >= 0.0f && std::isfinite(eps))) return RLSCAN_ERR_PARAM;
  return RLSCAN_OK;
}

void fill_heads(rlscan::nr::Args& a, rlscan_layout l, const float* q_weight, const float* k_weight,
                const int32_t* positions, int64_t E, int64_t T, int64_t H, int64_t Hk, int64_t D, int64_t rotate,
                float base, int interleaved, float eps) {
  const bool tm = l == RLSCAN_LAYOUT_TIME_MAJOR;
  a.heads[0] = H;
  a.heads[1] = Hk;
  a.weight[0] = q_weight;
  a.weight[1] = k_weight;
  a.pos = positions;
  a.p_se = tm ? 1 : T;
  a.p_st = tm ? E : 1;
  a.E = E;
  a.T = T;
  a.D = (int)D;
  a.R = (int)rotate;
  a.interleaved = interleaved != 0;
  a.eps = eps;
  a.base = base;
}

// Sizes that the entries of the table take: rows on one grid of waves, and of the gradient
// also what its sums take.
rlscan_status check_table(rlscan_format f, int64_t R, int64_t N, int64_t D) {
  if (R < 0 || R > rlscan::embed::kMaxTokens || N < 1 || N > rlscan::embed::kMaxKinds) return RLSCAN_ERR_SHAPE;
  if (D < 1 || D > RLSCAN_MAX_TABLE_DIM || R * ((D + 63) / 64) >= (int64_t)1 << 26) return RLSCAN_ERR_SHAPE;
  return elem_size(f) == 0 ? RLSCAN_ERR_PARAM : RLSCAN_OK;
}

bool stride_ok(int64_t rows, int64_t stride, int64_t D) {
  return rows <= 1 || (stride >= D && stride <= kMaxElems / rows);
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
                                      const float* rate, const uint8_t* done, const uint8_t* reset, const float* init_state,
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
  io.add_in(plain(reset, E));
  io.add_in(plain(init_state, E * D * 4));
  io.add_out(plain(final_state, E * D * 4));
  io.add_out(plain(marks, marks_bytes(E, T, D)));
  io.add_out(plain(workspace, need));
  if (io.clash()) return RLSCAN_ERR_ALIAS;
  fill_recurrence(a, p, layout, rate, done, reset, E, T, D, workspace);
  a.init = init_state;
  a.final_state = final_state;
  a.marks = marks;
  return launched(rlscan::gr::launch_forward(fmt, a, p, stream));
}

rlscan_status rlscan_gated_recurrence_backward(
    rlscan_format fmt, rlscan_layout layout, const rlscan_heads* d_out, const rlscan_heads* x,
    const rlscan_heads* input_gate, const rlscan_heads* decay_gate, const float* rate, const float* marks,
    const uint8_t* done, const uint8_t* reset, const float* d_final_state, const rlscan_heads* dx, const rlscan_heads* d_input_gate,
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
  io.add_in(plain(reset, E));
  io.add_in(plain(d_final_state, E * D * 4));
  io.add_out(plain(d_rate, D * 4));
  io.add_out(plain(d_init_state, E * D * 4));
  io.add_out(plain(workspace, need));
  if (io.clash()) return RLSCAN_ERR_ALIAS;
  fill_recurrence(a, p, layout, rate, done, reset, E, T, D, workspace);
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

rlscan_status rlscan_norm_rotate_heads(rlscan_format fmt, rlscan_layout layout, const rlscan_heads* q,
                                       const rlscan_heads* k, const float* q_weight, const float* k_weight,
                                       const int32_t* positions, const rlscan_heads* q_out, const rlscan_heads* k_out,
                                       int64_t E, int64_t T, int64_t H, int64_t Hk, int64_t D, int64_t rotate,
                                       float base, int interleaved, float eps, hipStream_t stream) {
  rlscan_status st = check_heads(fmt, E, T, H, Hk, D, rotate, base, eps);
  if (st != RLSCAN_OK) return st;
  if (!layout_ok(layout)) return RLSCAN_ERR_PARAM;
  if (E * T * (H + Hk) == 0) return RLSCAN_OK;
  if (rotate > 0 && !positions) return RLSCAN_ERR_NULL;
  rlscan::nr::Args a{};
  Spans io;
  HeadsCheck c{E, T, elem_size(fmt)};
  if (H > 0) {
    a.in[0] = c.view(q, H, D, false, io);
    a.out[0] = c.view(q_out, H, D, true, io);
  }
  if (Hk > 0) {
    a.in[1] = c.view(k, Hk, D, false, io);
    a.out[1] = c.view(k_out, Hk, D, true, io);
  }
  if (c.st != RLSCAN_OK) return c.st;
  if (!aligned(q_weight, 4) || !aligned(k_weight, 4) || !aligned(positions, 4)) return RLSCAN_ERR_ALIGN;
  io.add_in(plain(q_weight, D * 4));
  io.add_in(plain(k_weight, D * 4));
  if (rotate > 0) io.add_in(plain(positions, E * T * 4));
  if (io.clash()) return RLSCAN_ERR_ALIAS;
  fill_heads(a, layout, q_weight, k_weight, positions, E, T, H, Hk, D, rotate, base, interleaved, eps);
  return launched(rlscan::nr::launch_forward(fmt, a, stream));
}

int64_t rlscan_norm_rotate_heads_workspace(int64_t E, int64_t T, int64_t H, int64_t Hk, int64_t D) {
  if (check_heads(RLSCAN_FORMAT_F32, E, T, H, Hk, D, 0, 1.0f, 0.0f) != RLSCAN_OK) return -1;
  return rlscan::nr::backward_blocks(E * T, H + Hk, (int)D) * 2 * D * (int64_t)sizeof(float);
}

rlscan_status rlscan_norm_rotate_heads_backward(
    rlscan_format fmt, rlscan_layout layout, const rlscan_heads* d_q_out, const rlscan_heads* d_k_out,
    const rlscan_heads* q, const rlscan_heads* k, const float* q_weight, const float* k_weight,
    const int32_t* positions, const rlscan_heads* dq, const rlscan_heads* dk, float* d_q_weight, float* d_k_weight,
    void* workspace, int64_t workspace_bytes, int64_t E, int64_t T, int64_t H, int64_t Hk, int64_t D, int64_t rotate,
    float base, int interleaved, float eps, hipStream_t stream) {
  rlscan_status st = check_heads(fmt, E, T, H, Hk, D, rotate, base, eps);
  if (st != RLSCAN_OK) return st;
  if (!layout_ok(layout)) return RLSCAN_ERR_PARAM;
  const bool some = E * T * (H + Hk) > 0;
  if (!some && !d_q_weight && !d_k_weight) return RLSCAN_OK;
  const int64_t need = rlscan_norm_rotate_heads_workspace(E, T, H, Hk, D);
  rlscan::nr::Args a{};
  Spans io;
  HeadsCheck c{E, T, elem_size(fmt)};
  if (some) {
    if (rotate > 0 && !positions) return RLSCAN_ERR_NULL;
    if (H > 0) {
      a.grad[0] = c.view(d_q_out, H, D, false, io);
      a.in[0] = c.view(q, H, D, false, io);
      a.out[0] = c.view(dq, H, D, true, io);
    }
    if (Hk > 0) {
      a.grad[1] = c.view(d_k_out, Hk, D, false, io);
      a.in[1] = c.view(k, Hk, D, false, io);
      a.out[1] = c.view(dk, Hk, D, true, io);
    }
    if (c.st != RLSCAN_OK) return c.st;
  }
  if (!workspace) return RLSCAN_ERR_NULL;
  if (workspace_bytes < need) return RLSCAN_ERR_WORKSPACE;
  if (!aligned(q_weight, 4) || !aligned(k_weight, 4) || !aligned(positions, 4) || !aligned(d_q_weight, 4) ||
      !aligned(d_k_weight, 4) || !aligned(workspace, 16))
    return RLSCAN_ERR_ALIGN;
  io.add_in(plain(q_weight, D * 4));
  io.add_in(plain(k_weight, D * 4));
  if (some && rotate > 0) io.add_in(plain(positions, E * T * 4));
  io.add_out(plain(d_q_weight, D * 4));
  io.add_out(plain(d_k_weight, D * 4));
  io.add_out(plain(workspace, need));
  if (io.clash()) return RLSCAN_ERR_ALIAS;
  // Without heads there are no tokens either: their positions may be NULL, and only zeros are written.
  fill_heads(a, layout, q_weight, k_weight, positions, some ? E : 0, T, some ? H : 0, some ? Hk : 0, D, rotate, base,
             interleaved, eps);
  a.part = static_cast<float*>(workspace);
  a.d_weight[0] = d_q_weight;
  a.d_weight[1] = d_k_weight;
  return launched(rlscan::nr::launch_backward(fmt, a, stream));
}

rlscan_status rlscan_embed_tokens(rlscan_format fmt, const void* table, int64_t table_stride, const int64_t* tokens,
                                  void* out, int64_t out_stride, int64_t R, int64_t N, int64_t D, float scale,
                                  hipStream_t stream) {
  rlscan_status st = check_table(fmt, R, N, D);
  if (st != RLSCAN_OK) return st;
  const int es = elem_size(fmt);
  if (!stride_ok(N, table_stride, D) || !stride_ok(R, out_stride, D)) return RLSCAN_ERR_SHAPE;
  if (!std::isfinite(scale)) return RLSCAN_ERR_PARAM;
  if (R == 0) return RLSCAN_OK;
  if (!table || !tokens || !out) return RLSCAN_ERR_NULL;
  if (!aligned(table, es) || !aligned(tokens, 8) || !aligned(out, es)) return RLSCAN_ERR_ALIGN;
  Spans io;
  io.add_in(plain(table, ((N - 1) * table_stride + D) * es));
  io.add_in(plain(tokens, R * 8));
  io.add_out(plain(out, ((R - 1) * out_stride + D) * es));
  if (io.clash()) return RLSCAN_ERR_ALIAS;
  rlscan::embed::LookupArgs a{table, table_stride, tokens, out, out_stride, R, N, D, scale};
  return launched(rlscan::embed::launch_lookup(fmt, a, stream));
}

int64_t rlscan_embed_tokens_workspace(int64_t R, int64_t N, int64_t D) {
  if (check_table(RLSCAN_FORMAT_F32, R, N, D) != RLSCAN_OK) return -1;
  return rlscan::embed::make_plan(R, N, D).bytes;
}

rlscan_status rlscan_embed_tokens_backward(rlscan_format fmt, const void* d_out, int64_t out_stride,
                                           const int64_t* tokens, void* d_table, int64_t table_stride, void* workspace,
                                           int64_t workspace_bytes, int64_t R, int64_t N, int64_t D, float scale,
                                           hipStream_t stream) {
  rlscan_status st = check_table(fmt, R, N, D);
  if (st != RLSCAN_OK) return st;
  const int es = elem_size(fmt);
  if (!stride_ok(N, table_stride, D) || !stride_ok(R, out_stride, D)) return RLSCAN_ERR_SHAPE;
  if (!std::isfinite(scale)) return RLSCAN_ERR_PARAM;
  const int64_t need = rlscan_embed_tokens_workspace(R, N, D);
  if (!d_table || (need > 0 && !workspace) || (R > 0 && (!d_out || !tokens))) return RLSCAN_ERR_NULL;
  if (workspace_bytes < need) return RLSCAN_ERR_WORKSPACE;
  if (!aligned(d_table, es) || !aligned(tokens, 8) || !aligned(d_out, es) || !aligned(workspace, 16))
    return RLSCAN_ERR_ALIGN;
  Spans io;
  if (R > 0) io.add_in(plain(d_out, ((R - 1) * out_stride + D) * es));
  io.add_in(plain(tokens, R * 8));
  io.add_out(plain(d_table, ((N - 1) * table_stride + D) * es));
  io.add_out(plain(workspace, need));
  if (io.clash()) return RLSCAN_ERR_ALIAS;
  rlscan::embed::GradArgs a{d_out, out_stride, tokens, d_table, table_stride, workspace, R, N, D, scale};
  return launched(rlscan::embed::launch_backward(fmt, a, stream));
}

}  // extern "C"
