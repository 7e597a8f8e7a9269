"""The policy operators and the sizes at which they are timed and compared.

A policy with a linear-attention memory acts one step at a time and learns from
whole rollouts or token sequences.  Its operators:

* ``linear_attention``: per head, S_t = a_t S_{t-1} + k_t v_t^T and
  o_t = scale * S_t^T q_t with the decay a_t = exp(log_decay_t); a step flagged
  in ``done`` ends an episode (or one of several sequences packed into a row),
  so the next step starts from a zero state;
* ``linear_attention_backward``: the gradients of q, k, v, the decay and the
  initial state;
* ``linear_attention_step``: the same recurrence for one step of every
  environment, on states kept in a pool;
* ``sample_actions``: temperature, top-k, top-p and min-p, with given uniform
  numbers;
* ``action_log_probs`` and its backward: log-probability of the taken action
  and entropy, over a whole row of logits.

``run`` computes them from elementary torch operations, or with ``own`` set
through the package.
"""
import math

import numpy as np
import torch

own = False

_DTYPES = {"f32": torch.float32, "bf16": torch.bfloat16, "f16": torch.float16}
_SIZE = {"f32": 4, "bf16": 2, "f16": 2}


# ------------------------------------------------------------------------ cases
def _la(name, op, E, T, H, G, K, V, dtype, gate, p_done, init):
    """E rows of T steps, H heads of which G share a key/value head; gate: a log-decay
    for every step (True) or one for each head; p_done: rate of episode ends;
    init: the rows start from a given state."""
    return {"name": name, "op": op, "E": E, "T": T, "H": H, "G": G, "K": K, "V": V, "dtype": dtype,
            "gate": gate, "p_done": p_done, "init": init}


def _step(name, E, H, G, K, V, dtype, gate, pool):
    """One step of E environments whose states lie in a pool of `pool` slots (0: row e is slot e)."""
    return {"name": name, "op": "la_step", "E": E, "H": H, "G": G, "K": K, "V": V, "dtype": dtype,
            "gate": gate, "pool": pool}


def _sample(name, R, N, dtype, top_k, top_p, min_p, mask, per_row):
    """R rows of N logits; top_k 0, top_p 1 and min_p 0 are off; per_row: the
    parameters are tensors that vary from row to row, around the given ones."""
    return {"name": name, "op": "sample", "R": R, "N": N, "dtype": dtype, "top_k": top_k, "top_p": top_p,
            "min_p": min_p, "mask": mask, "per_row": per_row}


def _logp(name, op, R, N, dtype, mask):
    return {"name": name, "op": op, "R": R, "N": N, "dtype": dtype, "mask": mask}


def listed():
    return [
        # a short episode fragment of one environment, evaluated between two others: latency
        _la("la_fragment_f32", "la", 1, 37, 4, 1, 32, 32, "f32", True, 0.0, False),
        # the rollouts of many environments, with episode ends, continued from the last window
        _la("la_rollout_bf16", "la", 256, 256, 8, 1, 64, 64, "bf16", True, 0.01, True),
        # one long row of packed sequences, heads sharing keys and values, a fixed decay for each head
        _la("la_packed_bf16", "la", 1, 32768, 16, 4, 128, 128, "bf16", False, 0.0005, False),
        # learner on rollouts in full precision: odd length, shared heads, learned fixed decays
        _la("la_backward_f32", "la_bwd", 64, 333, 4, 2, 64, 64, "f32", False, 0.005, True),
        # learner on long sequences
        _la("la_backward_bf16", "la_bwd", 8, 4096, 16, 1, 128, 128, "bf16", True, 0.0005, False),
        # one environment acting: latency
        _step("la_step_one_bf16", 1, 16, 1, 128, 128, "bf16", True, 0),
        # a server's batch of environments with their states in a pool
        _step("la_step_pool_f16", 256, 16, 4, 128, 128, "f16", True, 300),
        # a small discrete action space with illegal moves masked: latency
        _sample("sample_actions_f32", 64, 18, "f32", 0, 1.0, 0.0, True, False),
        # one stream of tokens: latency over a large vocabulary
        _sample("sample_one_f32", 1, 131072, "f32", 0, 0.9, 0.0, False, False),
        # a batch of streams, each with settings of its own, over a vocabulary of odd size
        _sample("sample_batch_bf16", 256, 64007, "bf16", 50, 0.95, 0.02, False, True),
        # the learner's log-probabilities over rollouts of a small action space, with legal-move masks
        _logp("logp_actions_f32", "logp", 16384, 18, "f32", True),
        # the learner's log-probabilities and entropies over a vocabulary, and their gradient
        _logp("logp_train_bf16", "logp_train", 4096, 64007, "bf16", False),
    ]


def _log_uniform(rng, lo, hi):
    return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["la", "la", "la_bwd", "la_bwd", "la_step", "sample", "sample", "logp", "logp_train"])
    dtype = rng.choice(["f32", "bf16", "f16"])
    if op in ("la", "la_bwd"):
        top = 2 ** 15 if op == "la_bwd" or dtype != "f32" else 2 ** 14
        G = rng.choice([1, 1, 2, 4])
        H = G * rng.choice([1, 2, 3, 4])
        dims = [16, 24, 32, 40, 64, 64, 80, 96, 128, 128]
        T = _log_uniform(rng, 1, top if op == "la" else 4096)
        E = _log_uniform(rng, 1, max(1, min(256, top // T)))
        return _la("", op, E, T, H, G, rng.choice(dims), rng.choice(dims), dtype, rng.random() < 0.6,
                   rng.choice([0.0, 0.002, 0.05]), rng.random() < 0.5)
    if op == "la_step":
        E = _log_uniform(rng, 1, 256)
        G = rng.choice([1, 2, 4])
        return _step("", E, G * rng.choice([1, 2, 4]), G, rng.choice([32, 64, 80, 128]), rng.choice([32, 64, 96, 128]),
                     dtype, rng.random() < 0.6, E + rng.randrange(1, 40) if rng.random() < 0.5 else 0)
    if op == "sample":
        N = _log_uniform(rng, 2, 131072)
        R = _log_uniform(rng, 1, max(1, min(1024, 2 ** 23 // N)))
        return _sample("", R, N, dtype, rng.choice([0, 0, 1, 20, 50, 400]), rng.choice([1.0, 0.9, 0.95, 0.5]),
                       rng.choice([0.0, 0.0, 0.02, 0.1]), rng.random() < 0.3, rng.random() < 0.5)
    N = _log_uniform(rng, 2, 131072)
    R = _log_uniform(rng, 1, max(1, min(16384, 2 ** 25 // N)))
    return _logp("", op, R, N, dtype, rng.random() < 0.3)


# ------------------------------------------------------------------------ inputs
def prepare(case, seed):
    dev = "cuda"
    g = torch.Generator(device=dev).manual_seed(seed * 7919 + 11)
    dt = _DTYPES[case["dtype"]]

    def normal(*shape, scale=1.0, dtype=dt):
        return (torch.randn(shape, generator=g, device=dev) * scale).to(dtype)

    def uniform(*shape):
        return torch.rand(shape, generator=g, device=dev)

    st = {"case": case}
    if case["op"] in ("la", "la_bwd", "la_step"):
        E, H, K, V = case["E"], case["H"], case["K"], case["V"]
        Hkv = H // case["G"]
        rows = (E, case["T"]) if case["op"] != "la_step" else (E,)
        # decays as policies have them: memories of some ten to some thousand steps
        if case["gate"]:
            st["log_decay"] = torch.nn.functional.logsigmoid(normal(*rows, H, dtype=torch.float32) + 2.0) / 16.0
        else:
            st["log_decay"] = torch.log1p(-torch.exp2(-5.0 - 5.0 * torch.arange(H, device=dev) / max(1, H - 1)
                                                      - 0.1 * uniform(H)))
        st["q"] = normal(*rows, H, K)
        st["k"] = normal(*rows, Hkv, K, scale=K ** -0.5)
        st["v"] = normal(*rows, Hkv, V)
        if case["op"] == "la_step":
            pool = case["pool"] or E
            st["state"] = normal(pool, H, K, V, dtype=torch.float32)
            st["reset"] = (uniform(E) < 0.02).to(torch.uint8)
            st["slots"] = torch.randperm(pool, generator=g, device=dev)[:E].to(torch.int32) if case["pool"] else None
        else:
            st["done"] = (uniform(*rows) < case["p_done"]).to(torch.uint8) if case["p_done"] else None
            st["init"] = normal(E, H, K, V, scale=0.5, dtype=torch.float32) if case["init"] else None
            if case["op"] == "la_bwd":
                st["d_out"] = normal(*rows, H, V)
                st["d_final"] = normal(E, H, K, V, scale=0.1, dtype=torch.float32) if case["init"] else None
        return st
    R, N = case["R"], case["N"]
    st["logits"] = normal(R, N, scale=2.5)
    if case["mask"]:
        st["mask"] = (uniform(R, N) < 0.7).to(torch.uint8)
        if R > 3:
            st["mask"][R // 2] = 0  # a row without a legal action (a finished game)
    else:
        st["mask"] = None
    if case["op"] == "sample":
        st["uniforms"] = uniform(R)
        if case["per_row"]:
            st["temperature"] = 0.5 + uniform(R)
            st["top_k"] = torch.randint(0, 2 * case["top_k"] + 1, (R,), generator=g, device=dev, dtype=torch.int32)
            st["top_p"] = 1.0 - (1.0 - case["top_p"]) * 2.0 * uniform(R)
            st["min_p"] = case["min_p"] * 2.0 * uniform(R)
        else:
            st["temperature"], st["top_k"], st["top_p"], st["min_p"] = 0.8, case["top_k"], case["top_p"], case["min_p"]
        return st
    legal = st["mask"] if st["mask"] is not None else torch.ones_like(st["logits"], dtype=torch.uint8)
    st["actions"] = torch.argmax(uniform(R, N) * legal + (legal - 1.0), dim=1)
    st["temperature"] = 0.875
    if case["op"] == "logp_train":
        st["d_log_probs"] = normal(R, dtype=torch.float32)
        st["d_entropy"] = torch.full((R,), 0.01, device=dev)
    return st


def work(case):
    b = _SIZE[case["dtype"]]
    if case["op"] in ("la", "la_bwd"):
        E, T, H, K, V = case["E"], case["T"], case["H"], case["K"], case["V"]
        Hkv = H // case["G"]
        qkv = E * T * (H * K + Hkv * (K + V)) * b
        extra = (E * T * H if case["gate"] else H) * 4 + (E * T if case["p_done"] else 0)
        state = E * H * K * V * 4
        step = E * T * H * K * V * 2  # one product with a K x V matrix for each step and head
        if case["op"] == "la":
            return {"bytes": qkv + E * T * H * V * b + extra + state * (2 if case["init"] else 1), "flops": 2 * step}
        return {"bytes": 2 * qkv + E * T * H * V * b + 2 * extra + state * (3 if case["init"] else 0), "flops": 6 * step}
    if case["op"] == "la_step":
        E, H, K, V = case["E"], case["H"], case["K"], case["V"]
        Hkv = H // case["G"]
        return {"bytes": 2 * E * H * K * V * 4 + E * (H * (K + V) + Hkv * (K + V)) * b, "flops": 5 * E * H * K * V}
    R, N = case["R"], case["N"]
    row = R * N * (b + (1 if case["mask"] else 0))
    if case["op"] == "sample":
        return {"bytes": row + R * 16, "flops": 4 * R * N}
    if case["op"] == "logp":
        return {"bytes": row + R * 20, "flops": 5 * R * N}
    return {"bytes": 2 * row + R * N * b + R * 44, "flops": 12 * R * N}


# ------------------------------------------------------------------------ plain forms
def run(state):
    case = state["case"]
    if own:
        return _run_own(state, case)
    if case["op"] == "la":
        return _plain_forward(state, case)
    if case["op"] == "la_bwd":
        return _plain_backward(state, case)
    if case["op"] == "la_step":
        return _plain_step(state, case)
    if case["op"] == "sample":
        return _plain_sample(state, case)
    return _plain_logp(state, case)


def _run_own(st, case):
    import linear_recurrence_scan_reverse_amd as rl

    if case["op"] == "la":
        return rl.linear_attention(st["q"], st["k"], st["v"], st["log_decay"], st["done"], st["init"], with_state=True)
    if case["op"] == "la_bwd":
        return rl.linear_attention_backward(st["d_out"], st["q"], st["k"], st["v"], st["log_decay"], st["done"],
                                            st["init"], st["d_final"])
    if case["op"] == "la_step":
        out = rl.linear_attention_step(st["q"], st["k"], st["v"], st["log_decay"], st["state"], st["reset"], st["slots"])
        return out, st["state"]
    if case["op"] == "sample":
        return rl.sample_actions(st["logits"], st["uniforms"], temperature=st["temperature"], top_k=st["top_k"],
                                 top_p=st["top_p"], min_p=st["min_p"], mask=st["mask"])
    lp, ent, lse = rl.action_log_probs(st["logits"], st["actions"], temperature=st["temperature"], mask=st["mask"])
    if case["op"] == "logp":
        return lp, ent
    d = rl.action_log_probs_backward(st["d_log_probs"], st["d_entropy"], st["logits"], st["actions"], lse, ent,
                                     temperature=st["temperature"], mask=st["mask"])
    return lp, ent, d


_CHUNK = 128  # steps that the plain forms take at once


def _heads(x, G):
    """[E, T, h, D] as float32 [E, h*G, T, D]."""
    x = x.float().permute(0, 2, 1, 3)
    return x.repeat_interleave(G, dim=1) if G > 1 else x.contiguous()


def _chunks(st, case):
    """Per chunk: its slice, the decay between its steps [E, H, c, c] (row i, column j <= i),
    from its entry to its steps [E, H, c, 1], from its steps to its end [E, H, c, 1], across it [E, H, 1, 1]."""
    E, T, H = case["E"], case["T"], case["H"]
    g = st["log_decay"].double()
    g = g.permute(0, 2, 1) if case["gate"] else g.view(1, H, 1).expand(E, H, T)
    done = st["done"]
    cut = torch.zeros(E, 1, T, dtype=torch.int64, device=g.device) if done is None else (done != 0).long().view(E, 1, T)
    for t0 in range(0, T, _CHUNK):
        s = slice(t0, min(T, t0 + _CHUNK))
        b = g[:, :, s].cumsum(2)
        after = cut[:, :, s].cumsum(2)       # episode ends up to and with a step
        before = after - cut[:, :, s]        # and before it
        i, j = b.unsqueeze(3), b.unsqueeze(2)
        same = (before.unsqueeze(3) == before.unsqueeze(2)).tril()
        inner = torch.where(same, (i - j).clamp(max=0).exp(), torch.zeros_like(i)).float()
        entry = torch.where(before == 0, b.exp(), torch.zeros_like(b)).float().unsqueeze(3)
        last = b[:, :, -1:]
        ends = after[:, :, -1:]
        leave = torch.where(before == ends, (last - b).exp(), torch.zeros_like(b)).float().unsqueeze(3)
        across = torch.where(ends == 0, last.exp(), torch.zeros_like(last)).float().unsqueeze(3)
        yield s, inner, entry, leave, across


def _plain_forward(st, case, keep=None):
    E, H, K, V, G = case["E"], case["H"], case["K"], case["V"], case["G"]
    q, k, v = _heads(st["q"], 1) * K ** -0.5, _heads(st["k"], G), _heads(st["v"], G)
    S = torch.zeros(E, H, K, V, device=q.device) if st["init"] is None else st["init"]
    outs = []
    for s, inner, entry, leave, across in _chunks(st, case):
        if keep is not None:
            keep.append(S)
        qs, ks, vs = q[:, :, s], k[:, :, s], v[:, :, s]
        if keep is None:
            outs.append((qs @ ks.transpose(2, 3) * inner) @ vs + (qs * entry) @ S)
        S = S * across + (ks * leave).transpose(2, 3) @ vs
    if keep is None:
        return torch.cat(outs, 2).permute(0, 2, 1, 3).contiguous().to(st["q"].dtype), S


def _plain_backward(st, case):
    E, T, H, K, V, G = (case[n] for n in ("E", "T", "H", "K", "V", "G"))
    scale = K ** -0.5
    q, k, v = _heads(st["q"], 1) * scale, _heads(st["k"], G), _heads(st["v"], G)
    do = _heads(st["d_out"], 1)
    states = []
    _plain_forward(st, case, states)
    dS = torch.zeros(E, H, K, V, device=q.device) if st["d_final"] is None else st["d_final"]
    dq, dk, dv = torch.empty_like(q), torch.empty_like(k), torch.empty_like(v)
    dg = torch.empty(E, H, T, device=q.device)
    for (s, inner, entry, leave, across), S in reversed(list(zip(_chunks(st, case), states))):
        qs, ks, vs, ds = q[:, :, s], k[:, :, s], v[:, :, s], do[:, :, s]
        p = qs @ ks.transpose(2, 3) * inner
        dp = ds @ vs.transpose(2, 3) * inner
        q_in = ds @ S.transpose(2, 3) * entry
        k_out = vs @ dS.transpose(2, 3) * leave
        dq[:, :, s] = (dp @ ks + q_in) * scale
        dk[:, :, s] = dp.transpose(2, 3) @ qs + k_out
        dv[:, :, s] = p.transpose(2, 3) @ ds + (ks * leave) @ dS
        # every product of decays that holds a_t: steps j < t <= i, entry to i >= t, j < t to the end, entry to end
        pair = (qs @ ks.transpose(2, 3) * dp).tril(-1)
        n = pair.shape[2]
        upto = torch.ones(n, n, device=q.device).tril(-1)  # [t, j]: j < t
        to_i = (upto @ pair.transpose(2, 3)).transpose(2, 3)  # [i, t]: sum over j < t
        dgs = to_i.tril().sum(2)
        dgs = dgs + (qs * q_in).sum(3).flip(2).cumsum(2).flip(2)
        ky = (ks * k_out).sum(3)
        dgs = dgs + ky.cumsum(2) - ky + (S * dS).sum((2, 3)).unsqueeze(2) * across.squeeze(3)
        dg[:, :, s] = dgs
        dS = dS * across + (qs * entry).transpose(2, 3) @ ds
    dt = st["q"].dtype
    back = lambda x: x.permute(0, 2, 1, 3).contiguous().to(dt)
    dk = dk.view(E, H // G, G, T, K).sum(2)
    dv = dv.view(E, H // G, G, T, V).sum(2)
    dg = dg.permute(0, 2, 1).contiguous() if case["gate"] else dg.double().sum((0, 2)).float()
    return back(dq), back(dk), back(dv), dg, (dS if st["init"] is not None else None)


def _plain_step(st, case):
    K, G = case["K"], case["G"]
    q, k, v = st["q"].float() * K ** -0.5, st["k"].float(), st["v"].float()
    if G > 1:
        k, v = k.repeat_interleave(G, 1), v.repeat_interleave(G, 1)
    a = st["log_decay"].exp().expand(q.shape[0], q.shape[1])
    a = torch.where(st["reset"].view(-1, 1) != 0, torch.zeros_like(a), a)
    S = st["state"] if st["slots"] is None else st["state"][st["slots"].long()]
    S = S * a[:, :, None, None] + k.unsqueeze(3) * v.unsqueeze(2)
    out = (S * q.unsqueeze(3)).sum(2).to(st["q"].dtype)
    if st["slots"] is None:
        st["state"].copy_(S)
    else:
        st["state"][st["slots"].long()] = S
    return out, st["state"]


def _column(x, R, device):
    return (x if torch.is_tensor(x) else torch.full((R,), float(x), device=device).float()).double().view(R, 1)


def _plain_sample(st, case):
    # in 64 bits: whether a token is kept, and which one is taken, turns on values next to a border
    R, N = case["R"], case["N"]
    x = st["logits"].double()
    dev = x.device
    if st["mask"] is not None:
        x = torch.where(st["mask"] != 0, x, torch.full_like(x, -math.inf))
    top_k, top_p, min_p = (_column(st[n], R, dev) for n in ("top_k", "top_p", "min_p"))
    x, order = torch.sort(x, dim=1, descending=True, stable=True)
    legal = x > -math.inf
    x = torch.where(legal, (x - x[:, :1]) / _column(st["temperature"], R, dev), torch.full_like(x, -math.inf))
    rank = torch.arange(N, device=dev).view(1, N)
    keep = legal & ((top_k <= 0) | (rank < top_k))
    w = torch.where(keep, x.exp(), torch.zeros_like(x))
    before = w.cumsum(1) - w
    keep &= (top_p >= 1) | (before < top_p * w.sum(1, keepdim=True))
    keep &= w >= min_p
    w = torch.zeros_like(w).scatter_(1, order, torch.where(keep, w, torch.zeros_like(w)))  # in the order of the indices
    c = w.cumsum(1)
    total = w.sum(1, keepdim=True)
    hit = (c > st["uniforms"].double().view(R, 1) * total) & (w > 0)
    a = torch.where(hit.any(1), hit.to(torch.uint8).argmax(1), torch.full((R,), -1, device=dev))
    lp = torch.log(w.gather(1, a.clamp(min=0).view(R, 1)) / total).view(R)
    return a, torch.where(a >= 0, lp, torch.zeros_like(lp)).float()


def _plain_logp(st, case):
    R = case["R"]
    T = st["temperature"]
    x = st["logits"].float() / T
    if st["mask"] is not None:
        x = torch.where(st["mask"] != 0, x, torch.full_like(x, -math.inf))
    m = x.max(1, keepdim=True).values
    empty = m == -math.inf
    m = torch.where(empty, torch.zeros_like(m), m)
    e = (x - m).exp()
    total = torch.where(empty, torch.ones_like(m), e.sum(1, keepdim=True))
    lse = m + total.log()
    p = e / total
    ll = torch.where(e > 0, x - lse, torch.zeros_like(x))
    ent = -(p * ll).sum(1)
    a = st["actions"].view(R, 1)
    lp = torch.where(empty, torch.zeros_like(m), x.gather(1, a) - lse).view(R)
    if case["op"] == "logp":
        return lp, ent
    d = -p * (st["d_log_probs"].view(R, 1) + st["d_entropy"].view(R, 1) * (ll + ent.view(R, 1)))
    d.scatter_add_(1, a, torch.where(empty, torch.zeros_like(m), st["d_log_probs"].view(R, 1)))
    return lp, ent, (d / T).to(st["logits"].dtype)


# ------------------------------------------------------------------------ 64-bit values
def exact(case, seed):
    """Step by step and row by row, from the definitions."""
    st = prepare(case, seed)
    if case["op"] == "sample":
        return _exact_sample(st, case)
    if case["op"] in ("logp", "logp_train"):
        return _exact_logp(st, case)
    G, K, E, H = case["G"], case["K"], case["E"], case["H"]
    rep = lambda x: x.double().repeat_interleave(G, dim=-2)
    q, k, v = st["q"].double() / math.sqrt(K), rep(st["k"]), rep(st["v"])
    if case["op"] == "la_step":
        out = torch.empty(E, H, case["V"], dtype=torch.float64, device=q.device)
        state = st["state"].double()
        where = st["slots"].tolist() if st["slots"] is not None else list(range(E))
        a = torch.exp(st["log_decay"].double()).expand(E, H) * (st["reset"] == 0).double().view(E, 1)
        for e, s in enumerate(where):
            state[s] = a[e].view(H, 1, 1) * state[s] + torch.einsum("hk,hv->hkv", k[e], v[e])
            out[e] = torch.einsum("hk,hkv->hv", q[e], state[s])
        return out, state
    T = case["T"]
    a = torch.exp(st["log_decay"].double()).expand(E, T, H)
    if st["done"] is not None:  # a_t is 0 where step t - 1 ended an episode
        a = a.clone()
        a[:, 1:] *= (st["done"][:, :-1] == 0).double().unsqueeze(2)
    S = torch.zeros(E, H, K, case["V"], dtype=torch.float64, device=q.device) if st["init"] is None else st["init"].double()

    def advance(S, t):
        return a[:, t, :, None, None] * S + k[:, t].unsqueeze(3) * v[:, t].unsqueeze(2)

    last = torch.ones(E, 1, 1, 1, dtype=torch.float64, device=q.device)
    if st["done"] is not None:  # nothing leaves a row whose last step ended an episode
        last = (st["done"][:, -1] == 0).double().view(E, 1, 1, 1)
    if case["op"] == "la":
        out = torch.empty(E, T, H, case["V"], dtype=torch.float64, device=q.device)
        for t in range(T):
            S = advance(S, t)
            out[:, t] = (q[:, t].unsqueeze(2) @ S).squeeze(2)
        return out, S * last
    every = 64
    marks = []  # the state before every 64th step
    for t in range(T):
        if t % every == 0:
            marks.append(S)
        S = advance(S, t)
    do = st["d_out"].double()
    dS = torch.zeros_like(S) if st["d_final"] is None else st["d_final"].double() * last
    dq, dk, dv = torch.empty_like(q), torch.empty_like(k), torch.empty_like(v)
    dg = torch.empty(E, T, H, dtype=torch.float64, device=q.device)
    for m in reversed(range(len(marks))):
        before = [marks[m]]
        steps = list(range(m * every, min(T, (m + 1) * every)))
        for t in steps:
            before.append(advance(before[-1], t))
        for t in reversed(steps):
            St = before[t - steps[0] + 1]
            dq[:, t] = (St @ do[:, t].unsqueeze(3)).squeeze(3) / math.sqrt(K)
            dS = dS + q[:, t].unsqueeze(3) * do[:, t].unsqueeze(2)
            dk[:, t] = (dS @ v[:, t].unsqueeze(3)).squeeze(3)
            dv[:, t] = (k[:, t].unsqueeze(2) @ dS).squeeze(2)
            dS = dS * a[:, t, :, None, None]
            dg[:, t] = (before[t - steps[0]] * dS).sum((2, 3))
    fold = lambda x: x.view(E, T, H // G, G, x.shape[3]).sum(3)
    return (dq, fold(dk), fold(dv), dg if case["gate"] else dg.sum((0, 1)), dS if st["init"] is not None else None)


def _exact_sample(st, case):
    host = lambda x: x.double().cpu().numpy() if torch.is_tensor(x) else np.full(case["R"], np.float64(np.float32(x)))
    x, u = host(st["logits"]), host(st["uniforms"])
    temp, top_k, top_p, min_p = (host(st[n]) for n in ("temperature", "top_k", "top_p", "min_p"))
    mask = None if st["mask"] is None else st["mask"].cpu().numpy() != 0
    actions, lps = np.full(case["R"], -1, np.int64), np.zeros(case["R"])
    for r in range(case["R"]):
        legal = np.arange(case["N"]) if mask is None else np.flatnonzero(mask[r])
        if not legal.size:
            continue
        z = (x[r, legal] - x[r, legal].max()) / temp[r]
        order = np.argsort(-z, kind="stable")
        if top_k[r] > 0:
            order = order[:int(top_k[r])]
        w = np.exp(z[order])
        if top_p[r] < 1:
            kept = 1 + np.searchsorted(np.cumsum(w), top_p[r] * w.sum(), side="left")
            order, w = order[:kept], w[:kept]
        order = np.sort(order[w >= min_p[r]])
        w = np.exp(z[order])
        c = np.cumsum(w)
        i = order[np.searchsorted(c, u[r] * c[-1], side="right")]
        actions[r], lps[r] = legal[i], z[i] - np.log(c[-1])
    return torch.from_numpy(actions), torch.from_numpy(lps)


def _exact_logp(st, case):
    R, T = case["R"], st["temperature"]
    parts = ([], [], [])
    for r0 in range(0, R, 512):
        rows = slice(r0, min(R, r0 + 512))
        x = st["logits"][rows].double() / T
        if st["mask"] is not None:
            x = x.masked_fill(st["mask"][rows] == 0, -math.inf)
        some = (x > -math.inf).any(1)
        logp = torch.where(some.view(-1, 1), x - torch.logsumexp(x, 1, keepdim=True), torch.full_like(x, -math.inf))
        p = logp.exp()
        ent = -torch.where(p > 0, p * logp, torch.zeros_like(p)).sum(1)
        a = st["actions"][rows]
        index = torch.arange(a.numel(), device=a.device)
        parts[0].append(torch.where(some, logp[index, a], torch.zeros_like(ent)))
        parts[1].append(ent)
        if case["op"] == "logp_train":
            dlp = st["d_log_probs"][rows].double().view(-1, 1)
            den = st["d_entropy"][rows].double().view(-1, 1)
            d = -dlp * p - den * torch.where(p > 0, p * (logp + ent.view(-1, 1)), torch.zeros_like(p))
            d[index, a] += torch.where(some, dlp.view(-1), torch.zeros_like(ent))
            parts[2].append(d / T)
    return tuple(torch.cat(x) for x in parts if x)
