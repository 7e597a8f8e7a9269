"""The gated recurrence where its decays are fast: what is left of a state and of a gradient keeps its
bits relative to its own size, however little it is."""
from __future__ import annotations

import math

import pytest

torch = pytest.importorskip("torch")

import linear_recurrence_scan_reverse_amd as rl  # noqa: E402
from tests.sequence_oracle import U, close, logistic  # noqa: E402
from tests.test_gpu_gated_recurrence import both, draw, on_gpu  # noqa: E402

pytestmark = pytest.mark.gpu

# A sigmoid is off by 20 of U (see GATE in the oracle), s and its logarithm's factor by 3 more; a sum of 16
# such logarithms by 16 roundings; exp by what its argument is off, and 2.
GATE = 60.0
SMALL = 2.0 ** -118  # decays below the normal numbers are 0, times values of a few hundred at most


def relative_error(s, a):
    """Of a decay: by its own size, held as a itself or (s up to 0.18) as a - 1, and of a product of 16."""
    return U * torch.where(s < 0.18, 26 * (1 - a) / a + 16 * s, 40 * s) + 8 * U


class Oracle:
    """Values and gradients in float64, step by step, and what each may be off by: terms' errors are relative to
    themselves, so that a sum's bound is small where all its terms are."""

    def __init__(self, d):
        x, ig, dg, rate, init, d_out, d_final = (d[n].double() for n in
                                                 ("x", "ig", "dg", "rate", "init", "d_out", "d_final"))
        E, T, D = x.shape
        si, sr = logistic(ig), logistic(dg)
        s = rate * sr
        fresh = torch.zeros(E, T, 1, dtype=torch.bool)
        if d["done"] is not None:
            fresh[:, 1:, 0] = d["done"][:, :-1]
        a = torch.where(fresh, torch.zeros_like(s), torch.exp(-s))
        m2 = torch.where(fresh, torch.ones_like(s), -torch.expm1(-2.0 * s))
        m, u = m2.sqrt(), si * x
        R = torch.where(fresh, torch.zeros_like(s), relative_error(s, torch.exp(-s)))
        Rm = 26 * U * (s < 0.18) + a * a / m2 * R  # of m, about half of that of 1 - a^2
        h, habs, hb = [init], [init.abs()], [torch.zeros_like(init)]
        for t in range(T):
            h.append(a[:, t] * h[t] + m[:, t] * u[:, t])
            term = m[:, t] * u[:, t].abs()
            habs.append(a[:, t] * habs[t] + term)
            hb.append(a[:, t] * (hb[t] + R[:, t] * habs[t]) + term * (GATE * U + Rm[:, t]) + 3 * U * habs[-1] + SMALL)
        self.out, self.out_b = torch.stack(h[1:], 1), torch.stack(hb[1:], 1)
        ended = torch.zeros(E, 1, dtype=torch.bool) if d["done"] is None else d["done"][:, -1:]
        e = torch.where(ended, torch.zeros_like(init), d_final)
        eabs, eb = e.abs(), torch.zeros_like(e)
        self.dr, self.dr_b = torch.zeros_like(x), torch.zeros_like(x)
        self.d_rate, self.d_rate_b = torch.zeros_like(rate), torch.zeros_like(rate)
        for t in reversed(range(T)):
            g, gabs = e + d_out[:, t], eabs + d_out[:, t].abs()
            gb = eb + 2 * U * gabs
            over = a[:, t] ** 2 / m[:, t]
            inner, inner_abs = a[:, t] * h[t] - u[:, t] * over, a[:, t] * habs[t] + u[:, t].abs() * over
            dlog = g * inner
            size = gabs * inner_abs
            dlog_b = gb * inner_abs + gabs * a[:, t] * hb[t] + (2 * R[:, t] + Rm[:, t] + 2 * GATE * U) * size
            rest = 1 - sr[:, t]
            self.dr[:, t] = -s[:, t] * rest * dlog
            self.dr_b[:, t] = s[:, t] * (rest * (dlog_b + GATE * U * size) + GATE * U * sr[:, t] * size) + SMALL
            self.d_rate -= (sr[:, t] * dlog).sum(0)
            self.d_rate_b += (sr[:, t] * (dlog_b + (GATE + E * T) * U * size)).sum(0) + SMALL
            e, eabs, eb = a[:, t] * g, a[:, t] * gabs, a[:, t] * (gb + (R[:, t] + 2 * U) * gabs) + SMALL
        self.d_init, self.d_init_b = e, eb


RATES = [(0.1, 3.0), (5.0, 10.0), (10.0, 20.0), (20.0, 40.0), (40.0, 80.0)]


@pytest.mark.parametrize("E,T,D,p_done", [(3, 70, 40, 0.0), (2, 1, 64, 0.0), (2, 90, 33, 0.1), (1, 1100, 64, 0.0)])
@pytest.mark.parametrize("low,high", RATES)
def test_fast_decays(low, high, E, T, D, p_done):
    d = draw(E, T, D, torch.float32, seed=40, p_done=p_done, low=low, high=high)
    got, grads = both(on_gpu(d))
    want = Oracle(d)
    close(got[0], want.out, want.out_b, "out")
    close(grads[2], want.dr, want.dr_b, "d_decay_gate")
    close(grads[3], want.d_rate, want.d_rate_b, "d_rate")
    close(grads[4], want.d_init, want.d_init_b, "d_init_state")


@pytest.mark.parametrize("low,high", RATES)
def test_nothing_but_the_state(low, high):
    # closed input gates (a sigmoid of 0 in float32): every state is the decayed initial one alone
    d = draw(2, 8, 50, torch.float32, seed=41, p_done=0.0, low=low, high=high / 8)
    d["ig"].fill_(-200.0)
    got, grads = both(on_gpu(d))
    want = Oracle(d)
    relative = (got[0].cpu().double() / want.out - 1).abs()
    assert (relative <= want.out_b / want.out.abs()).all()
    # eight decays of exp(-12) each may leave float32: what their product leaves of a value is 0 there
    for g, w, b in ((got[0], want.out, want.out_b), (grads[2], want.dr, want.dr_b), (grads[4], want.d_init, want.d_init_b)):
        assert (g.cpu()[w.abs() > b] != 0).all() and (w.abs() > b).sum() > w.numel() // 4
        close(g, w, b, "of the state alone")


@pytest.mark.parametrize("low,high", RATES)
def test_fast_steps(low, high):
    d = draw(3, 6, 70, torch.float32, seed=42, p_done=0.0, low=low, high=high)
    c, want = on_gpu(d), Oracle(d)
    state = c["init"].clone()
    for t in range(6):
        out = rl.gated_recurrence_step(c["x"][:, t], c["ig"][:, t], c["dg"][:, t], c["rate"], state)
        close(out, want.out[:, t], want.out_b[:, t], "step %d" % t)
        assert torch.equal(out, state)


def test_rates_at_and_below_zero():
    # 0 of either sign holds the state; below, as with NaN, the channel is NaN
    d = draw(2, 40, 4, torch.float32, seed=43, p_done=0.0)
    d["rate"] = torch.tensor([0.0, -0.0, -1.0, math.nan])
    c = on_gpu(d)
    got, grads = both(c)
    held = c["init"][:, None, :2].expand(2, 40, 2)
    assert torch.equal(got[0][..., :2], held) and torch.equal(got[1][:, :2], c["init"][:, :2])
    assert torch.isnan(got[0][..., 2:]).all() and torch.isnan(grads[3][2:]).all() and torch.isfinite(grads[3][:2]).all()
    state = c["init"].clone()
    rl.gated_recurrence_step(c["x"][:, 0], c["ig"][:, 0], c["dg"][:, 0], c["rate"], state)
    assert torch.equal(state[:, :2], c["init"][:, :2]) and torch.isnan(state[:, 2:]).all()
