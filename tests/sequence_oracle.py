"""Float64 oracles of the operators of policies over token sequences, and what their float32
arithmetic may be off by.

Every oracle works step by step or token by token on CPU tensors.  The bounds count float32
roundings (U each, half a step) against sums of absolute values, worst case."""
from __future__ import annotations

import math

import torch

U = 2.0 ** -24
# half a step of a rounding to the storage type, and half its smallest step below the normal numbers
HALF = {torch.float32: 2.0 ** -24, torch.bfloat16: 2.0 ** -8, torch.float16: 2.0 ** -11}
TINY = {torch.float32: 2.0 ** -126, torch.bfloat16: 2.0 ** -126, torch.float16: 2.0 ** -25}
assert all(HALF[t] == torch.finfo(t).eps / 2 for t in HALF)


def stored(value, bound, dtype):
    """The bound after the result has been rounded to its storage type."""
    return bound * (1 + HALF[dtype]) + HALF[dtype] * value.abs() + TINY[dtype]


def close(got, want, bound, what):
    """|got - want| <= bound everywhere; inf and NaN in the same places."""
    got, want, bound = got.detach().cpu().double(), want.double(), bound.double()
    assert got.shape == want.shape, what
    fine = torch.isfinite(want)
    assert torch.equal(torch.isfinite(got), fine), "%s: inf or NaN in other places" % what
    off = ((got - want).abs() / bound)[fine]
    worst = off.max().item() if off.numel() else 0.0
    assert worst <= 1.0, "%s: %.3g times its bound" % (what, worst)
    return worst


# ------------------------------------------------------------------ gated recurrence
# A sigmoid: exponent's product (|z| log2 e roundings in the worst case, |z| <= 8 here: 12), exp2, sum,
# reciprocal (2 each for the hardware's): 20 of U.  s = rate sigmoid: 21.  sqrt(1 - a^2): that, 5 for
# 1 - a and 3; u: a sigmoid and 2.  Their product: 52 at most, 56 with those that follow.
GATE = 56.0


def decay_error(s, a):
    """Of a as the kernels hold it, a - 1: relative to 1 - a, s's 21 and 5 for the series of s below a
    quarter; above it exp(-s)'s error, 21 s exp(-s) <= 21 / e < 8 of U, and one rounding of a - 1."""
    return U * (26 * (1 - a) + 9 * (s >= 0.25).double())


def logistic(z):
    return 1.0 / (1.0 + torch.exp(-z))


class Recurrence:
    """Forward values and, given d_out, gradients of [E, T, D] inputs (env-major, any storage type),
    each with its bound before storage: attributes name and name + '_b'."""

    def __init__(self, x, ig, dg, rate, done=None, init=None, d_out=None, d_final=None,
                 reset=None):
        x, ig, dg, rate = x.cpu().double(), ig.cpu().double(), dg.cpu().double(), rate.cpu().double()
        E, T, D = x.shape
        live = torch.ones(E, T + 1, 1, dtype=torch.float64)
        if done is not None:
            live[:, 1:, 0] = (done.cpu() == 0).double()
        if reset is not None:
            live[:, 0, 0] = (reset.cpu() == 0).double()
        si, sr = logistic(ig), logistic(dg)
        s = rate * sr
        fresh = live[:, :T] == 0
        a = torch.where(fresh, torch.zeros_like(s), torch.exp(-s))
        m = torch.where(fresh, torch.ones_like(s), torch.sqrt(-torch.expm1(-2.0 * s)))
        u = si * x
        h0 = torch.zeros(E, D, dtype=torch.float64) if init is None else init.cpu().double()
        zero = torch.zeros_like(h0)
        err = decay_error(s, a)
        hs, habs, hb = [h0], [h0.abs()], [zero]  # states, the same with absolute terms, and their bounds
        for t in range(T):
            drop = fresh[:, t]

            def keep(v):
                return torch.where(drop, zero, v)

            hs.append(a[:, t] * keep(hs[-1]) + m[:, t] * u[:, t])
            habs.append(a[:, t] * keep(habs[-1]) + m[:, t] * u[:, t].abs())
            # the decay's error, the term's, and roundings of a h and of the sum
            hb.append(a[:, t] * keep(hb[-1]) + err[:, t] * keep(habs[-2]) + GATE * U * m[:, t] * u[:, t].abs()
                      + 3 * U * habs[-1])
        self.states = torch.stack(hs, 1)  # [E, T + 1, D], from the initial one on
        self.habs = torch.stack(habs, 1)
        self.states_b = torch.stack(hb, 1)
        self.out, self.out_b = self.states[:, 1:], self.states_b[:, 1:]
        ended = live[:, T] == 0
        self.final = torch.where(ended, zero, hs[-1])
        self.final_b = torch.where(ended, zero, self.states_b[:, T]) + TINY[torch.float32]
        if d_out is None:
            return
        d_out = d_out.cpu().double()
        e = zero if d_final is None else torch.where(ended, zero, d_final.cpu().double())
        eabs, eb = e.abs(), zero
        names = ("dx", "di", "dr")
        grads = {n: torch.empty_like(x) for n in names}
        bounds = {n: torch.empty_like(x) for n in names}
        d_rate, d_rate_b = torch.zeros_like(rate), torch.zeros_like(rate)
        for t in reversed(range(T)):
            drop = fresh[:, t]
            g, gabs = e + d_out[:, t], eabs + d_out[:, t].abs()
            gb = eb + 2 * U * gabs
            before = torch.where(drop, zero, self.states[:, t])
            babs, bb = torch.where(drop, zero, self.habs[:, t]), torch.where(drop, zero, self.states_b[:, t])
            at, mt, ut, si_t, sr_t, s_t = a[:, t], m[:, t], u[:, t], si[:, t], sr[:, t], s[:, t]
            over = torch.where(mt > 0, at * at / mt, zero)  # a^2 / m; the limit where the state is held
            inner = at * before - ut * over
            inner_abs = at * babs + ut.abs() * over
            grads["dx"][:, t] = si_t * mt * g
            bounds["dx"][:, t] = si_t * mt * (gb + GATE * U * gabs)
            grads["di"][:, t] = ut * mt * g * (1 - si_t)
            # 1 - sigmoid is off by sigmoid's error, which need not be small next to it
            bounds["di"][:, t] = ut.abs() * mt * ((1 - si_t) * (gb + GATE * U * gabs) + GATE * U * gabs * si_t)
            dlog = torch.where(drop, zero, g * inner)
            dlog_b = torch.where(drop, zero, gb * inner_abs
                                 + gabs * (at * bb + err[:, t] * babs + 2 * GATE * U * inner_abs))
            grads["dr"][:, t] = -s_t * (1 - sr_t) * dlog
            bounds["dr"][:, t] = s_t * ((1 - sr_t) * (dlog_b + GATE * U * gabs * inner_abs)
                                        + GATE * U * sr_t * gabs * inner_abs)
            d_rate -= (sr_t * dlog).sum(0)
            # its own errors, and the float32 sum's: no more than E T additions
            d_rate_b += (sr_t * (dlog_b + (GATE + E * T) * U * gabs * inner_abs)).sum(0)
            e = torch.where(drop, zero, at * g)
            eabs = torch.where(drop, zero, at * gabs)
            eb = torch.where(drop, zero, at * gb + err[:, t] * gabs + 2 * U * eabs)
        for n in names:
            setattr(self, n, grads[n])
            setattr(self, n + "_b", bounds[n])
        self.d_rate, self.d_rate_b = d_rate, d_rate_b + TINY[torch.float32]
        self.d_init = e
        self.d_init_b = eb + TINY[torch.float32]


# ------------------------------------------------------------------ normalised and rotated heads
class Heads:
    """y and, given dy, dx and dw of [..., H, D] heads with positions [...], each with its bound
    before storage.

    Bounds: a mean of squares is off by a few roundings for each of the 16 terms that a lane adds, the
    6 steps over lanes and the division: 26 of U at most, its root's reciprocal by 13 and 2; x inv w by
    2 more.  A sine or cosine by 4 of U: the angle's two roundings and the series'.  A turned pair
    by its members' errors, its angle's and two roundings: 26 of U of |a| + |b|; 32 here."""

    def __init__(self, x, weight, positions, rotate, base=10000.0, interleaved=False, eps=1e-6, dy=None):
        x = x.cpu().double()
        D = x.shape[-1]
        w = torch.ones(D, dtype=torch.float64) if weight is None else weight.cpu().double()
        a = torch.arange(0, rotate, 2) if interleaved else torch.arange(rotate // 2)
        b = a + 1 if interleaved else a + rotate // 2
        freq = base ** (-2.0 * torch.arange(rotate // 2, dtype=torch.float64) / max(1, rotate))
        pos = torch.zeros(x.shape[:-2]) if positions is None else positions.cpu()
        angle = (pos.double()[..., None] * freq).unsqueeze(-2)  # the same for a token's heads

        def turn(z, back=False):
            sin = -angle.sin() if back else angle.sin()
            za, zb = z[..., a], z[..., b]
            out, size = z.clone(), z.abs()
            out[..., a], out[..., b] = za * angle.cos() - zb * sin, zb * angle.cos() + za * sin
            size[..., a] = size[..., b] = za.abs() + zb.abs()
            return out, size

        inv = 1.0 / torch.sqrt((x * x).mean(-1, keepdim=True) + eps)
        n = x * inv
        self.y, size = turn(n * w)
        self.y_b = 32 * U * size
        if dy is None:
            return
        dz, size = turn(dy.cpu().double(), back=True)
        lead = tuple(range(x.dim() - 1))
        count = x.numel() // D
        self.dw = (dz * n).sum(lead)
        self.dw_b = (32 + count) * U * (size * n.abs()).sum(lead) + TINY[torch.float32]
        g, gabs = dz * w, size * w.abs()
        self.dx = inv * (g - n * (g * n).mean(-1, keepdim=True))
        # dz 8 of U, inv 15, n 16, the mean 26 and its factors' 24: under 100 in all, twice n's for its square
        self.dx_b = 100 * U * inv * (gabs + n.abs() * (gabs * n.abs()).mean(-1, keepdim=True))


# ------------------------------------------------------------------ rows of a table
def lookup(table, tokens, scale):
    t = tokens.cpu()
    ok = (t >= 0) & (t < table.shape[0])
    out = table.cpu().double()[t.clamp(0, table.shape[0] - 1)] * scale
    return torch.where(ok[..., None], out, torch.zeros_like(out))


def table_gradient(d_out, tokens, N, scale):
    """(gradient, bound before storage): a row of c terms takes c additions and the scale."""
    D = d_out.shape[-1]
    t, d = tokens.cpu().reshape(-1), d_out.cpu().double().reshape(-1, D)
    total, size, count = torch.zeros(N, D, dtype=torch.float64), torch.zeros(N, D, dtype=torch.float64), torch.zeros(N)
    for r in range(t.numel()):
        n = int(t[r])
        if 0 <= n < N:
            total[n] += d[r]
            size[n] += d[r].abs()
            count[n] += 1
    return total * scale, (count.double()[:, None] + 2) * U * size * abs(scale)
