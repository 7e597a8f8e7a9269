// policy_api.hip -- the C ABI of the policy operators (declared in include/rlscan.h):
// linear attention, action sampling and action log-probabilities.  Every entry
// validates on the host before any HIP call and enqueues its kernels on the
// caller's stream; scratch memory comes from the caller.
#include <cmath>
#include <cstdint>

#include "rlscan.h"
#include "rlscan_checks.hpp"
#include "rlscan_la_launch.hpp"
#include "rlscan_logits.hpp"

namespace {

using rlscan::la::Args;
using rlscan::la::Plan;
using namespace rlscan::checks;

// Sizes that every linear-attention entry takes.
rlscan_status check_sizes(rlscan_format f, int64_t E, int64_t T, int64_t H, int64_t Hkv, int64_t K, int64_t V) {
  if (E < 0 || T < 0 || T >= RLSCAN_MAX_T || H < 0 || Hkv < 0) return RLSCAN_ERR_SHAPE;
  if (K < 1 || V < 1 || K > RLSCAN_MAX_HEAD_DIM || V > RLSCAN_MAX_HEAD_DIM) return RLSCAN_ERR_SHAPE;
  if (H > 0 && (Hkv < 1 || H % Hkv != 0)) return RLSCAN_ERR_SHAPE;
  if (H > 0 && E > kMaxElems / 128 / H) return RLSCAN_ERR_SHAPE;
  if (E * H > 0 && T > kMaxElems / 128 / (E * H)) return RLSCAN_ERR_SHAPE;
  if (elem_size(f) == 0) return RLSCAN_ERR_PARAM;
  return RLSCAN_OK;
}

// Whether every launch stays below the block limit.
bool grid_ok(const Plan& p, int64_t E, int64_t T, int64_t H, int64_t Hkv, int64_t K, int64_t V, bool backward) {
  const int64_t most = rlscan::la::kMaxBlocks;
  const int64_t heads = E * H;
  if (heads > most / 64 || H > most) return false;  // combine: up to 64 blocks a head; the sum over rows: one
  const int64_t per = (p.VP / 64 > 3 || !backward ? p.VP / 64 : 3) * p.nseg;
  if (heads > (most - 24) / per) return false;
  if (backward && p.nmarks > 0 && heads > most / p.nmarks) return false;
  // group sums: one block for 256 elements
  if (backward && Hkv != H && E * T * Hkv > (most - 1) * 256 / (K > V ? K : V)) return false;
  return true;
}

rlscan_status fill_common(Args& a, rlscan_layout l, const float* log_decay, int per_step, const uint8_t* done,
                          int64_t E, int64_t T, int64_t H, int64_t Hkv, int64_t K, int64_t V, float scale) {
  const bool tm = l == RLSCAN_LAYOUT_TIME_MAJOR;
  a.g = log_decay;
  a.g_sh = 1;
  a.g_se = per_step ? (tm ? H : T * H) : 0;
  a.g_st = per_step ? (tm ? E * H : H) : 0;
  a.done = done;
  a.d_se = tm ? 1 : T;
  a.d_st = tm ? E : 1;
  a.E = E;
  a.T = T;
  a.H = H;
  a.G = H / Hkv;
  a.K = (int)K;
  a.V = (int)V;
  a.scale = scale;
  return RLSCAN_OK;
}

bool layout_ok(rlscan_layout l) { return l == RLSCAN_LAYOUT_ENV_MAJOR || l == RLSCAN_LAYOUT_TIME_MAJOR; }

void fill_plan(Args& a, const Plan& p) {
  a.nseg = p.nseg;
  a.seg_chunks = p.seg_chunks;
  a.chunks = p.chunks;
}

}  // namespace

extern "C" {

int64_t rlscan_linear_attention_workspace(rlscan_format fmt, int64_t E, int64_t T, int64_t H, int64_t Hkv, int64_t K,
                                          int64_t V, int backward) {
  if (check_sizes(fmt, E, T, H, Hkv, K, V) != RLSCAN_OK) return -1;
  if (E * H == 0) return 0;
  const Plan p = rlscan::la::make_plan(fmt, E, T, H, H / Hkv, K, V, backward != 0);
  if (!grid_ok(p, E, T, H, Hkv, K, V, backward != 0)) return -1;
  return p.floats * (int64_t)sizeof(float);
}

rlscan_status rlscan_linear_attention(rlscan_format fmt, rlscan_layout layout, const rlscan_heads* q,
                                      const rlscan_heads* k, const rlscan_heads* v, const float* log_decay,
                                      int per_step, const uint8_t* done, const float* init_state,
                                      const rlscan_heads* out, float* final_state, void* workspace,
                                      int64_t workspace_bytes, int64_t E, int64_t T, int64_t H, int64_t Hkv,
                                      int64_t K, int64_t V, float scale, hipStream_t stream) {
  rlscan_status st = check_sizes(fmt, E, T, H, Hkv, K, V);
  if (st != RLSCAN_OK) return st;
  if (!layout_ok(layout) || !std::isfinite(scale)) return RLSCAN_ERR_PARAM;
  if (E * H == 0 || (T == 0 && !final_state)) return RLSCAN_OK;
  const Plan p = rlscan::la::make_plan(fmt, E, T, H, H / Hkv, K, V, false);
  if (!grid_ok(p, E, T, H, Hkv, K, V, false)) return RLSCAN_ERR_SHAPE;
  const int64_t need = p.floats * (int64_t)sizeof(float);
  Args a{};
  fill_common(a, layout, log_decay, per_step, done, E, T, H, Hkv, K, V, scale);
  Spans io;
  if (T > 0) {
    if (!log_decay) return RLSCAN_ERR_NULL;
    HeadsCheck c{E, T, elem_size(fmt)};
    a.q = c.view(q, H, K, false, io);
    a.k = c.view(k, Hkv, K, false, io);
    a.v = c.view(v, Hkv, V, false, io);
    a.out = c.view(out, H, V, true, io);
    if (c.st != RLSCAN_OK) return c.st;
  }
  if (need > 0 && !workspace) return RLSCAN_ERR_NULL;
  if (workspace_bytes < need) return RLSCAN_ERR_WORKSPACE;
  if (!aligned(log_decay, 4) || !aligned(init_state, 4) || !aligned(final_state, 4) || !aligned(workspace, 16))
    return RLSCAN_ERR_ALIGN;
  const int64_t state = E * H * K * V * 4;
  io.add_in(plain(log_decay, (per_step ? E * T * H : H) * 4));
  io.add_in(plain(done, E * T));
  io.add_in(plain(init_state, state));
  io.add_out(plain(final_state, state));
  io.add_out(plain(workspace, need));
  if (io.clash()) return RLSCAN_ERR_ALIAS;
  a.init = init_state;
  a.final_state = final_state;
  fill_plan(a, p);
  float* ws = static_cast<float*>(workspace);
  a.seg_state = ws;
  a.seg_decay = ws + p.seg_state;
  return launched(rlscan::la::launch_forward(fmt, a, p, stream));
}

rlscan_status rlscan_linear_attention_backward(
    rlscan_format fmt, rlscan_layout layout, const rlscan_heads* d_out, const rlscan_heads* q, const rlscan_heads* k,
    const rlscan_heads* v, const float* log_decay, int per_step, const uint8_t* done, const float* init_state,
    const float* d_final_state, const rlscan_heads* dq, const rlscan_heads* dk, const rlscan_heads* dv,
    float* d_log_decay, float* d_init_state, void* workspace, int64_t workspace_bytes, int64_t E, int64_t T, int64_t H,
    int64_t Hkv, int64_t K, int64_t V, float scale, hipStream_t stream) {
  rlscan_status st = check_sizes(fmt, E, T, H, Hkv, K, V);
  if (st != RLSCAN_OK) return st;
  if (!layout_ok(layout) || !std::isfinite(scale)) return RLSCAN_ERR_PARAM;
  if (H == 0 || (E == 0 && per_step)) return RLSCAN_OK;
  if (!d_log_decay && (!per_step || T > 0)) return RLSCAN_ERR_NULL;
  const Plan p = rlscan::la::make_plan(fmt, E, T, H, H / Hkv, K, V, true);
  if (!grid_ok(p, E, T, H, Hkv, K, V, true)) return RLSCAN_ERR_SHAPE;
  const int64_t need = p.floats * (int64_t)sizeof(float);
  Args a{};
  fill_common(a, layout, log_decay, per_step, done, E, T, H, Hkv, K, V, scale);
  Spans io;
  if (E * T > 0) {
    if (!log_decay) return RLSCAN_ERR_NULL;
    HeadsCheck c{E, T, elem_size(fmt)};
    a.dout = c.view(d_out, H, V, false, io);
    a.q = c.view(q, H, K, false, io);
    a.k = c.view(k, Hkv, K, false, io);
    a.v = c.view(v, Hkv, V, false, io);
    a.dq = c.view(dq, H, K, true, io);
    a.dk = c.view(dk, Hkv, K, true, io);
    a.dv = c.view(dv, Hkv, V, true, io);
    if (c.st != RLSCAN_OK) return c.st;
  }
  if (need > 0 && !workspace) return RLSCAN_ERR_NULL;
  if (workspace_bytes < need) return RLSCAN_ERR_WORKSPACE;
  if (!aligned(log_decay, 4) || !aligned(init_state, 4) || !aligned(d_final_state, 4) || !aligned(d_log_decay, 4) ||
      !aligned(d_init_state, 4) || !aligned(workspace, 16))
    return RLSCAN_ERR_ALIGN;
  const int64_t state = E * H * K * V * 4, gates = (per_step ? E * T * H : H) * 4;
  io.add_in(plain(log_decay, gates));
  io.add_in(plain(done, E * T));
  io.add_in(plain(init_state, state));
  io.add_in(plain(d_final_state, state));
  io.add_out(plain(d_log_decay, gates));
  io.add_out(plain(d_init_state, state));
  io.add_out(plain(workspace, need));
  if (io.clash()) return RLSCAN_ERR_ALIAS;
  a.init = init_state;
  fill_plan(a, p);
  if (per_step) {
    a.dg = d_log_decay;
    a.dg_se = a.g_se;
    a.dg_st = a.g_st;
    a.dg_sh = 1;
  }
  rlscan::la::Backward b{};
  b.d_final = d_final_state;
  b.d_init = d_init_state;
  b.dg_head = per_step ? nullptr : d_log_decay;
  float* ws = static_cast<float*>(workspace);
  auto take = [&](int64_t floats) {
    float* at = ws;
    ws += floats;
    return at;
  };
  b.total = reinterpret_cast<double*>(take(2 * p.heads));
  b.end = take(p.heads);
  b.seg_state = take(p.seg_state);
  b.seg_decay = take(p.seg_decay);
  b.seg_grad = take(p.seg_state);
  b.seg_gdecay = take(p.seg_decay);
  b.u = reinterpret_cast<double*>(take(p.dots));
  b.w = reinterpret_cast<double*>(take(p.dots));
  b.marks = take(p.marks);
  b.mark_grads = take(p.marks);
  b.mark_dots = reinterpret_cast<double*>(take((2 * E * H * p.nmarks + 3) / 4 * 4));
  b.nmarks = p.nmarks;
  a.mark_chunks = p.mark_chunks;
  b.dk = a.dk;
  b.dv = a.dv;
  if (a.G > 1) {
    auto scratch = [&](float* at, int64_t D) {
      return View{at, T * H * D, H * D, D, D % 8 == 0 && H * D <= ((int64_t)1 << 23)};
    };
    b.dk = scratch(take(p.dk), K);
    b.dv = scratch(take(p.dv), V);
  }
  return launched(rlscan::la::launch_backward(fmt, a, b, p, stream));
}

rlscan_status rlscan_linear_attention_step(rlscan_format fmt, const rlscan_heads* q, const rlscan_heads* k,
                                           const rlscan_heads* v, const float* log_decay, int per_row,
                                           const uint8_t* reset, const int32_t* slots, float* state,
                                           const rlscan_heads* out, int64_t E, int64_t S, int64_t H, int64_t Hkv,
                                           int64_t K, int64_t V, float scale, hipStream_t stream) {
  rlscan_status st = check_sizes(fmt, E, 1, H, Hkv, K, V);
  if (st != RLSCAN_OK) return st;
  if (S < 0 || (H > 0 && S > kMaxElems / 16384 / H) || (!slots && S < E)) return RLSCAN_ERR_SHAPE;
  if (!std::isfinite(scale)) return RLSCAN_ERR_PARAM;
  if (E * H == 0) return RLSCAN_OK;
  if (E * H > rlscan::la::kMaxBlocks / 4) return RLSCAN_ERR_SHAPE;
  if (!log_decay || (!state && S > 0)) return RLSCAN_ERR_NULL;
  Spans io;
  HeadsCheck c{E, 1, elem_size(fmt)};
  const View vq = c.view(q, H, K, false, io);
  const View vk = c.view(k, Hkv, K, false, io);
  const View vv = c.view(v, Hkv, V, false, io);
  const View vo = c.view(out, H, V, true, io);
  if (c.st != RLSCAN_OK) return c.st;
  if (!aligned(log_decay, 4) || !aligned(slots, 4) || !aligned(state, 4)) return RLSCAN_ERR_ALIGN;
  io.add_in(plain(log_decay, (per_row ? E * H : H) * 4));
  io.add_in(plain(reset, E));
  io.add_in(plain(slots, E * 4));
  io.add_out(plain(state, S * H * K * V * 4));
  if (io.clash()) return RLSCAN_ERR_ALIAS;
  rlscan::la::StepArgs a{};
  a.q = vq.p;
  a.q_se = vq.se;
  a.q_sh = vq.sh;
  a.k = vk.p;
  a.k_se = vk.se;
  a.k_sh = vk.sh;
  a.v = vv.p;
  a.v_se = vv.se;
  a.v_sh = vv.sh;
  a.out = const_cast<void*>(vo.p);
  a.o_se = vo.se;
  a.o_sh = vo.sh;
  a.g = log_decay;
  a.g_se = per_row ? H : 0;
  a.g_sh = 1;
  a.reset = reset;
  a.slots = slots;
  a.state = state;
  a.E = E;
  a.H = H;
  a.G = H / Hkv;
  a.S = S;
  a.K = (int)K;
  a.V = (int)V;
  a.scale = scale;
  return launched(rlscan::la::launch_step(fmt, a, stream));
}

int64_t rlscan_sample_actions_workspace(int64_t R, int64_t N) {
  if (R < 0 || R > rlscan::logits::kMaxSampleRows || N < 1 || N > rlscan::logits::kMaxActions) return -1;
  return rlscan::logits::sample_workspace(R, N);
}

rlscan_status rlscan_sample_actions(rlscan_format fmt, const void* logits, int64_t stride, const uint8_t* mask,
                                    const float* uniforms, const float* temperatures, const int32_t* top_ks,
                                    const float* top_ps, const float* min_ps, float temperature, int32_t top_k,
                                    float top_p, float min_p, int64_t* actions, float* log_probs, int64_t R, int64_t N,
                                    hipStream_t stream) {
  return rlscan_sample_actions_shared(fmt, logits, stride, mask, uniforms, temperatures, top_ks, top_ps, min_ps,
                                      temperature, top_k, top_p, min_p, actions, log_probs, nullptr, 0, R, N, stream);
}

rlscan_status rlscan_sample_actions_shared(rlscan_format fmt, const void* logits, int64_t stride, const uint8_t* mask,
                                    const float* uniforms, const float* temperatures, const int32_t* top_ks,
                                    const float* top_ps, const float* min_ps, float temperature, int32_t top_k,
                                    float top_p, float min_p, int64_t* actions, float* log_probs, void* workspace,
                                    int64_t workspace_bytes, int64_t R, int64_t N,
                                    hipStream_t stream) {
  const int es = elem_size(fmt);
  if (R < 0 || R > rlscan::logits::kMaxSampleRows || N < 1 || N > rlscan::logits::kMaxActions) return RLSCAN_ERR_SHAPE;
  if (R > 1 && (stride < N || stride > kMaxElems / R)) return RLSCAN_ERR_SHAPE;
  if (es == 0) return RLSCAN_ERR_PARAM;
  if (!temperatures && !(temperature >= 0.0f && std::isfinite(temperature))) return RLSCAN_ERR_PARAM;
  if (!top_ps && !(top_p > 0.0f && std::isfinite(top_p))) return RLSCAN_ERR_PARAM;
  if (!min_ps && !(min_p >= 0.0f && min_p <= 1.0f)) return RLSCAN_ERR_PARAM;
  if (!top_ks && top_k < 0) return RLSCAN_ERR_PARAM;
  if (R == 0) return RLSCAN_OK;
  if (workspace && workspace_bytes < rlscan_sample_actions_workspace(R, N)) return RLSCAN_ERR_WORKSPACE;
  if (!logits || !uniforms || !actions) return RLSCAN_ERR_NULL;
  if (!aligned(logits, es) || !aligned(uniforms, 4) || !aligned(temperatures, 4) || !aligned(top_ks, 4) ||
      !aligned(top_ps, 4) || !aligned(min_ps, 4) || !aligned(actions, 8) || !aligned(log_probs, 4) ||
      !aligned(workspace, 8))
    return RLSCAN_ERR_ALIGN;
  Spans io;
  io.add_in(plain(logits, ((R - 1) * stride + N) * es));
  io.add_in(plain(mask, R * N));
  io.add_in(plain(uniforms, R * 4));
  io.add_in(plain(temperatures, R * 4));
  io.add_in(plain(top_ks, R * 4));
  io.add_in(plain(top_ps, R * 4));
  io.add_in(plain(min_ps, R * 4));
  io.add_out(plain(actions, R * 8));
  io.add_out(plain(log_probs, R * 4));
  io.add_out(plain(workspace, rlscan_sample_actions_workspace(R, N)));
  if (io.clash()) return RLSCAN_ERR_ALIAS;
  rlscan::logits::SampleArgs a{};
  a.x = logits;
  a.stride = stride;
  a.mask = mask;
  a.u = uniforms;
  a.temperature = temperatures;
  a.top_k = top_ks;
  a.top_p = top_ps;
  a.min_p = min_ps;
  a.temperature1 = temperature;
  a.top_k1 = top_k;
  a.top_p1 = top_p;
  a.min_p1 = min_p;
  a.shared = workspace;
  a.action = actions;
  a.log_prob = log_probs;
  a.R = R;
  a.N = N;
  return launched(rlscan::logits::launch_sample(fmt, a, stream));
}

int64_t rlscan_action_log_probs_workspace(int64_t R, int64_t N) {
  if (R < 0 || R > rlscan::la::kMaxBlocks || N < 1 || N >= RLSCAN_MAX_T) return -1;
  const int64_t split = rlscan::logits::log_probs_split(R, N);
  return split > 1 ? R * split * 4 * (int64_t)sizeof(float) : 0;
}

rlscan_status rlscan_action_log_probs(rlscan_format fmt, const void* logits, int64_t stride, const uint8_t* mask,
                                      const int64_t* actions, float temperature, float* log_probs, float* entropies,
                                      double* lse, void* workspace, int64_t workspace_bytes, int64_t R, int64_t N,
                                      hipStream_t stream) {
  const int es = elem_size(fmt);
  const int64_t need = rlscan_action_log_probs_workspace(R, N);
  if (need < 0) return RLSCAN_ERR_SHAPE;
  if (R > 1 && (stride < N || stride > kMaxElems / R)) return RLSCAN_ERR_SHAPE;
  if (es == 0 || !(temperature > 0.0f && std::isfinite(temperature) && std::isfinite(1.0f / temperature)))
    return RLSCAN_ERR_PARAM;
  if (R == 0) return RLSCAN_OK;
  if (!logits || !actions || !log_probs || !entropies || !lse || (need > 0 && !workspace)) return RLSCAN_ERR_NULL;
  if (workspace_bytes < need) return RLSCAN_ERR_WORKSPACE;
  if (!aligned(logits, es) || !aligned(actions, 8) || !aligned(log_probs, 4) || !aligned(entropies, 4) ||
      !aligned(lse, 8) || !aligned(workspace, 4))
    return RLSCAN_ERR_ALIGN;
  Spans io;
  io.add_in(plain(logits, ((R - 1) * stride + N) * es));
  io.add_in(plain(mask, R * N));
  io.add_in(plain(actions, R * 8));
  io.add_out(plain(log_probs, R * 4));
  io.add_out(plain(entropies, R * 4));
  io.add_out(plain(lse, R * 8));
  io.add_out(plain(workspace, need));
  if (io.clash()) return RLSCAN_ERR_ALIAS;
  rlscan::logits::LogProbArgs a{};
  a.x = logits;
  a.stride = stride;
  a.mask = mask;
  a.action = actions;
  a.inv_t = 1.0 / (double)temperature;
  a.log_prob = log_probs;
  a.entropy = entropies;
  a.lse = lse;
  a.part = static_cast<float*>(workspace);
  a.R = R;
  a.N = N;
  a.split = rlscan::logits::log_probs_split(R, N);
  return launched(rlscan::logits::launch_log_probs(fmt, a, stream));
}

rlscan_status rlscan_action_log_probs_backward(rlscan_format fmt, const float* d_log_probs, const float* d_entropies,
                                               const void* logits, int64_t stride, const uint8_t* mask,
                                               const int64_t* actions, float temperature, const double* lse,
                                               const float* entropies, void* d_logits, int64_t d_stride, int64_t R,
                                               int64_t N, hipStream_t stream) {
  const int es = elem_size(fmt);
  if (rlscan_action_log_probs_workspace(R, N) < 0) return RLSCAN_ERR_SHAPE;
  if (R > 1 && (stride < N || d_stride < N || stride > kMaxElems / R || d_stride > kMaxElems / R))
    return RLSCAN_ERR_SHAPE;
  // one block for each 2048 groups of a row
  if (R > 0 && N / 8192 + 2 > (int64_t)0xffffff / R) return RLSCAN_ERR_SHAPE;
  if (es == 0 || !(temperature > 0.0f && std::isfinite(temperature) && std::isfinite(1.0f / temperature)))
    return RLSCAN_ERR_PARAM;
  if (R == 0) return RLSCAN_OK;
  if (!logits || !actions || !lse || !entropies || !d_logits) return RLSCAN_ERR_NULL;
  if (!aligned(logits, es) || !aligned(d_logits, es) || !aligned(actions, 8) || !aligned(lse, 8) ||
      !aligned(entropies, 4) || !aligned(d_log_probs, 4) || !aligned(d_entropies, 4))
    return RLSCAN_ERR_ALIGN;
  Spans io;
  io.add_in(plain(logits, ((R - 1) * stride + N) * es));
  io.add_in(plain(mask, R * N));
  io.add_in(plain(actions, R * 8));
  io.add_in(plain(lse, R * 8));
  io.add_in(plain(entropies, R * 4));
  io.add_in(plain(d_log_probs, R * 4));
  io.add_in(plain(d_entropies, R * 4));
  io.add_out(plain(d_logits, ((R - 1) * d_stride + N) * es));
  if (io.clash()) return RLSCAN_ERR_ALIAS;
  rlscan::logits::LogProbArgs a{};
  a.x = logits;
  a.stride = stride;
  a.mask = mask;
  a.action = actions;
  a.inv_t = 1.0 / (double)temperature;
  a.lse = const_cast<double*>(lse);
  a.entropy = const_cast<float*>(entropies);
  a.d_log_prob = d_log_probs;
  a.d_entropy = d_entropies;
  a.dx = d_logits;
  a.dx_stride = d_stride;
  a.R = R;
  a.N = N;
  return launched(rlscan::logits::launch_log_probs_backward(fmt, a, stream));
}

}  // extern "C"
