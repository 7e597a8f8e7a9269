"""Plain float64 forms of the policy operators, written from their definitions.

Linear attention runs step by step, its gradient as the recursion backward in
time; sampling sorts; nothing here is chunked.  Inputs are torch tensors of any
dtype on the CPU; everything is widened to float64 first (exactly).

``magnitude=True`` replaces every input by its absolute value: the result is the sum of
the absolute values of the terms that make up each element, against which the
rounding of those terms is bounded.
"""
from __future__ import annotations

import math

import numpy as np
import torch

CUT_BELOW = -104.0  # log-decays below this start afresh: exp is 0 in float32


def _wide(x, magnitude):
    x = x.double()
    return x.abs() if magnitude else x


def _decays(log_decay, done, E, T, H):
    """a [E, T, H], 0 where a step starts afresh, and that mask."""
    g = log_decay.double().expand(E, T, H)
    cut = g < CUT_BELOW
    if done is not None and T:
        before = torch.zeros(E, T, dtype=torch.bool)
        before[:, 1:] = done[:, :-1] != 0
        cut = cut | before.unsqueeze(2)
    return torch.where(cut, torch.zeros((), dtype=torch.float64), g.exp()), cut


def _group(x, H):
    return x.repeat_interleave(H // x.shape[2], dim=2) if x.shape[2] != H else x


def linear_attention(q, k, v, log_decay, done=None, init=None, scale=None, magnitude=False, states=False):
    """(out [E, T, H, V], final [E, H, K, V]); with states also S before and after each step."""
    E, T, H, K = q.shape
    scale = K ** -0.5 if scale is None else scale
    scale = abs(scale) if magnitude else scale
    a, _ = _decays(log_decay, done, E, T, H)
    q, k, v = _wide(q, magnitude), _group(_wide(k, magnitude), H), _group(_wide(v, magnitude), H)
    V = v.shape[3]
    S = torch.zeros(E, H, K, V, dtype=torch.float64) if init is None else _wide(init, magnitude)
    out = torch.zeros(E, T, H, V, dtype=torch.float64)
    kept = [S]
    for t in range(T):
        S = a[:, t, :, None, None] * S + k[:, t, :, :, None] * v[:, t, :, None, :]
        out[:, t] = scale * (q[:, t, :, :, None] * S).sum(2)
        kept.append(S)
    final = S
    if done is not None and T:
        final = S * (done[:, -1] == 0).double().view(E, 1, 1, 1)
    return (out, final, kept) if states else (out, final)


def linear_attention_backward(d_out, q, k, v, log_decay, done=None, init=None, d_final=None, scale=None,
                              magnitude=False):
    """(dq, dk, dv, dg, d_init): dg like log_decay."""
    E, T, H, K = q.shape
    Hkv, V = k.shape[2], v.shape[3]
    scale = K ** -0.5 if scale is None else scale
    scale = abs(scale) if magnitude else scale
    _, _, S = linear_attention(q, k, v, log_decay, done, init, scale, magnitude, states=True)
    a, cut = _decays(log_decay, done, E, T, H)
    do, q, k, v = (_wide(x, magnitude) for x in (d_out, q, k, v))
    k, v = _group(k, H), _group(v, H)
    dS = torch.zeros(E, H, K, V, dtype=torch.float64)
    if d_final is not None:
        dS = _wide(d_final, magnitude)
        if done is not None and T:
            dS = dS * (done[:, -1] == 0).double().view(E, 1, 1, 1)
    dq, dk, dv = torch.zeros_like(q), torch.zeros_like(k), torch.zeros_like(v)
    dg = torch.zeros(E, T, H, dtype=torch.float64)
    for t in reversed(range(T)):
        dq[:, t] = scale * (S[t + 1] * do[:, t, :, None, :]).sum(3)
        dS = dS + scale * q[:, t, :, :, None] * do[:, t, :, None, :]
        dk[:, t] = (dS * v[:, t, :, None, :]).sum(3)
        dv[:, t] = (dS * k[:, t, :, :, None]).sum(2)
        dS = dS * a[:, t, :, None, None]
        dg[:, t] = (S[t] * dS).sum((2, 3))
    G = H // Hkv
    dk = dk.view(E, T, Hkv, G, K).sum(3)
    dv = dv.view(E, T, Hkv, G, V).sum(3)
    dg = dg if log_decay.dim() == 3 else dg.sum((0, 1))
    return dq, dk, dv, dg, dS


def sample_row(x, u, temperature, top_k, top_p, min_p, mask=None):
    """(action, log_prob, gap) of one row; gap: how near the choice came to another
    (relative distance of u * total from the nearest border of the running sum, and of the
    top_p and min_p borders)."""
    x = np.asarray(x, np.float64).copy()
    legal = x > -np.inf  # false for NaN
    if mask is not None:
        legal &= np.asarray(mask) != 0
    index = np.flatnonzero(legal)
    if not index.size:
        return -1, 0.0, 1.0
    if not temperature > 0:
        temperature, top_k = 1.0, 1
    z = np.minimum(x[index], float(np.finfo(np.float32).max))
    z = (z - z.max()) / temperature
    order = np.argsort(-z, kind="stable")
    if top_k > 0:
        order = order[:top_k]
    gap = 1.0
    if top_p < 1:
        w = np.exp(z[order])
        c = np.cumsum(w)
        n = min(int(np.searchsorted(c, top_p * c[-1], side="left")), order.size - 1)
        gap = min(gap, np.abs(c - top_p * c[-1]).min() / c[-1])
        order = order[:n + 1]
    w = np.exp(z[order])
    m = min(max(min_p, 0.0), 1.0)
    if 0 < m < 1:
        gap = min(gap, np.abs(w - m).min())
    order = np.sort(order[w >= m])
    w = np.exp(z[order])
    c = np.cumsum(w)
    i = min(int(np.searchsorted(c, u * c[-1], side="right")), order.size - 1)
    gap = min(gap, np.abs(c - u * c[-1]).min() / c[-1]) if u > 0 else gap
    return int(index[order[i]]), float(z[order[i]] - math.log(c[-1])), float(gap)


def log_probs(logits, actions, temperature=1.0, mask=None):
    """(log_prob, entropy, lse) of [R, N] logits in float64."""
    x = logits.double() / temperature
    if mask is not None:
        x = torch.where(mask != 0, x, torch.full_like(x, -math.inf))
    R, N = x.shape
    empty = ~(x > -math.inf).any(1) & ~torch.isnan(x).any(1)
    lse = torch.logsumexp(x, 1)
    logp = x - torch.where(empty, torch.zeros_like(lse), lse).unsqueeze(1)
    p = logp.exp()
    ent = -torch.where(p == 0, torch.zeros_like(p), p * logp).sum(1)
    taken = (actions >= 0) & (actions < N)
    lp = logp.gather(1, actions.clamp(0, N - 1).unsqueeze(1)).squeeze(1)
    lp = torch.where(taken & ~empty, lp, torch.zeros_like(lp))
    ent = torch.where(empty, torch.zeros_like(ent), ent)
    return lp, ent, lse


def log_probs_backward(d_lp, d_ent, logits, actions, temperature=1.0, mask=None):
    """d_logits in float64, and the magnitude of its terms."""
    x = logits.double() / temperature
    if mask is not None:
        x = torch.where(mask != 0, x, torch.full_like(x, -math.inf))
    R, N = x.shape
    empty = ~(x > -math.inf).any(1)
    lse = torch.logsumexp(x, 1)
    logp = x - torch.where(empty, torch.zeros_like(lse), lse).unsqueeze(1)
    p = logp.exp()
    p = torch.where(empty.unsqueeze(1), torch.zeros_like(p), p)
    safe = torch.where(p == 0, torch.zeros_like(logp), logp)
    ent = -(p * safe).sum(1, keepdim=True)
    taken = ((actions >= 0) & (actions < N) & ~empty).double().unsqueeze(1)
    one = torch.zeros_like(p).scatter_(1, actions.clamp(0, N - 1).unsqueeze(1), 1.0) * taken
    if mask is not None:
        one = one * (mask != 0).double()
    d_lp = torch.zeros(R, 1, dtype=torch.float64) if d_lp is None else d_lp.double().unsqueeze(1)
    d_ent = torch.zeros(R, 1, dtype=torch.float64) if d_ent is None else d_ent.double().unsqueeze(1)
    d = d_lp * (one - taken * p) - d_ent * p * (safe + ent)
    size = d_lp.abs() * (one + p) + d_ent.abs() * p * (safe.abs() + ent.abs())
    return d / temperature, size / temperature
