"""Operators of a policy over token sequences, and the sizes at which they are timed and compared.

A policy whose steps are tokens looks its inputs up in a table, normalises and rotates the
queries and keys of its attention, and may keep a vector in place of a matrix as its memory:

* ``gated_recurrence``: h_t = a_t h_{t-1} + sqrt(1 - a_t^2) sigmoid(i_t) x_t for every channel,
  a_t = exp(-rate sigmoid(r_t)); the step after one flagged in ``done`` has a_t = 0;
* ``gated_recurrence_backward``: the gradients of x, both gates, the rate and the initial state;
* ``gated_recurrence_step``: one step of every environment, on states kept in a pool;
* ``norm_rotate_heads`` and its backward: queries and keys divided by their root mean square,
  times a learned weight, and rotated by their position's angles;
* ``embed_tokens`` and its backward: rows of a table times a scale, and the sum of the
  gradients of every row's tokens.

``run`` computes them from elementary torch operations, or with ``own`` set through the package.
"""
import math

import torch

own = False

_DTYPES = {"f32": torch.float32, "bf16": torch.bfloat16, "f16": torch.float16}
_SIZE = {"f32": 4, "bf16": 2, "f16": 2}
_EPS = 1e-6


# ------------------------------------------------------------------------ cases
def _gr(name, op, E, T, D, dtype, p_done, init):
    """E rows of T steps with D channels; p_done: rate of episode ends; init: the rows
    start from a given state (and its end has a gradient)."""
    return {"name": name, "op": op, "E": E, "T": T, "D": D, "dtype": dtype, "p_done": p_done, "init": init}


def _gr_step(name, E, D, dtype, pool):
    """One step of E environments whose states lie in a pool of `pool` slots (0: row e is slot e)."""
    return {"name": name, "op": "gr_step", "E": E, "D": D, "dtype": dtype, "pool": pool}


def _heads(name, op, E, T, H, G, D, R, dtype, interleaved, first):
    """H query heads, H / G key heads of D, the first R rotated; positions start anew in each
    episode of about 500 steps, the row's first one at up to `first`."""
    return {"name": name, "op": op, "E": E, "T": T, "H": H, "G": G, "D": D, "R": R, "dtype": dtype,
            "interleaved": interleaved, "first": first}


def _embed(name, op, R, N, D, dtype, padded):
    """R tokens of N kinds, the first ones the most frequent; padded: a share of them is padding."""
    return {"name": name, "op": op, "R": R, "N": N, "D": D, "dtype": dtype, "padded": padded}


def listed():
    return [
        # a short episode fragment of one environment, evaluated between two others: latency
        _gr("gr_fragment_f32", "gr", 1, 37, 256, "f32", 0.0, False),
        # one long row of packed sequences
        _gr("gr_packed_bf16", "gr", 1, 32768, 1280, "bf16", 0.0005, False),
        # learner on rollouts in full precision: odd length, episode ends, continued from the last window
        _gr("gr_train_f32", "gr_train", 64, 333, 768, "f32", 0.005, True),
        # learner on long sequences
        _gr("gr_train_bf16", "gr_train", 8, 4096, 2048, "bf16", 0.0005, False),
        # one environment acting: latency
        _gr_step("gr_step_one_bf16", 1, 2048, "bf16", 0),
        # a server's batch of environments with their states in a pool
        _gr_step("gr_step_pool_f16", 256, 2048, "f16", 300),
        # one environment's next token, far into its episode: latency
        _heads("heads_step_bf16", "heads", 1, 1, 16, 4, 128, 128, "bf16", False, 100000),
        # learner on rollouts in full precision: odd length, a part of each head rotated, pairs side by side
        _heads("heads_train_f32", "heads_train", 64, 333, 4, 2, 80, 40, "f32", True, 500),
        # learner on long sequences
        _heads("heads_train_bf16", "heads_train", 8, 4096, 16, 4, 128, 128, "bf16", False, 0),
        # the tokens that a server's streams have just drawn: latency
        _embed("embed_step_bf16", "embed", 64, 131072, 1024, "bf16", False),
        # rollouts of a small world: few kinds of observations, each seen a thousand times
        _embed("embed_train_f32", "embed_train", 16384, 18, 250, "f32", False),
        # learner on padded token sequences, over a vocabulary of odd size
        _embed("embed_train_bf16", "embed_train", 32768, 64007, 1024, "bf16", True),
    ]


def _log_uniform(rng, lo, hi):
    return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["gr", "gr", "gr_train", "gr_train", "gr_step", "heads", "heads_train", "heads_train", "embed",
                     "embed_train", "embed_train"])
    dtype = rng.choice(["f32", "bf16", "f16"])
    wide = 2 if dtype == "f32" else 1
    if op in ("gr", "gr_train"):
        most = 2 ** 25 // wide  # values of x
        D = _log_uniform(rng, 1, 2048)
        T = _log_uniform(rng, 1, min(32768, most // D))
        E = _log_uniform(rng, 1, max(1, min(1024, most // (D * T))))
        return _gr("", op, E, T, D, dtype, rng.choice([0.0, 0.002, 0.05]), rng.random() < 0.5)
    if op == "gr_step":
        E = _log_uniform(rng, 1, 512)
        return _gr_step("", E, _log_uniform(rng, 8, 4096), dtype, E + rng.randrange(1, 40) if rng.random() < 0.5 else 0)
    if op in ("heads", "heads_train"):
        D = rng.choice([16, 32, 40, 64, 64, 72, 80, 96, 128, 128, 160, 192, 256])
        R = rng.choice([D, D, D // 2, D // 4 * 2, 0])
        G = rng.choice([1, 1, 2, 4])
        H = G * rng.choice([1, 2, 3, 4])
        most = 2 ** 25 // wide // (D * H)
        T = _log_uniform(rng, 1, min(8192, most))
        E = _log_uniform(rng, 1, max(1, min(512, most // T)))
        return _heads("", op, E, T, H, G, D, R, dtype, rng.random() < 0.5, rng.choice([0, 1000, 1000000]))
    D = _log_uniform(rng, 8, 2048)
    N = _log_uniform(rng, 2, min(131072, 2 ** 26 // wide // D))
    R = _log_uniform(rng, 1, min(65536, 2 ** 26 // wide // D))
    return _embed("", op, R, N, D, dtype, rng.random() < 0.5)


# ------------------------------------------------------------------------ inputs
def prepare(case, seed):
    dev = "cuda"
    g = torch.Generator(device=dev).manual_seed(seed * 7919 + 23)
    dt = _DTYPES[case["dtype"]]

    def normal(*shape, scale=1.0, dtype=dt):
        return (torch.randn(shape, generator=g, device=dev) * scale).to(dtype)

    def uniform(*shape):
        return torch.rand(shape, generator=g, device=dev)

    st = {"case": case}
    if case["op"].startswith("gr"):
        E, D = case["E"], case["D"]
        rows = (E,) if case["op"] == "gr_step" else (E, case["T"])
        st["x"] = normal(*rows, D)
        st["input_gate"], st["decay_gate"] = normal(*rows, D), normal(*rows, D)
        # decays as such memories start out: of some steps to some thousand
        st["rate"] = torch.exp(math.log(0.008) + (math.log(0.84) - math.log(0.008)) * uniform(D))
        if case["op"] == "gr_step":
            pool = case["pool"] or E
            st["state"] = normal(pool, D, dtype=torch.float32)
            st["reset"] = (uniform(E) < 0.02).to(torch.uint8)
            st["slots"] = torch.randperm(pool, generator=g, device=dev)[:E].to(torch.int32) if case["pool"] else None
            return st
        st["done"] = (uniform(*rows) < case["p_done"]).to(torch.uint8) if case["p_done"] else None
        st["init"] = normal(E, D, dtype=torch.float32) if case["init"] else None
        if case["op"] == "gr_train":
            st["d_out"] = normal(*rows, D)
            st["d_final"] = normal(E, D, dtype=torch.float32) if case["init"] else None
        return st
    if case["op"].startswith("heads"):
        E, T, H, D = case["E"], case["T"], case["H"], case["D"]
        st["q"], st["k"] = normal(E, T, H, D, scale=3.0), normal(E, T, H // case["G"], D, scale=3.0)
        st["q_weight"], st["k_weight"] = 1.0 + normal(D, scale=0.2, dtype=torch.float32), 1.0 + normal(
            D, scale=0.2, dtype=torch.float32)
        steps = torch.arange(T, device=dev).view(1, T)
        first = (uniform(E, 1) * (case["first"] + 1)).long()
        cut = (uniform(E, T) < 0.002) & (steps > 0)
        start = torch.where(cut, steps, torch.zeros_like(steps)).cummax(1).values
        st["positions"] = torch.where(start > 0, steps - start, first + steps).to(torch.int32)
        if case["op"] == "heads_train":
            st["dq"], st["dk"] = normal(*st["q"].shape), normal(*st["k"].shape)
        return st
    R, N, D = case["R"], case["N"], case["D"]
    st["table"] = normal(N, D, scale=D ** -0.5)
    st["tokens"] = (torch.exp(uniform(R).double() * math.log(N + 1)).long() - 1).clamp(0, N - 1)
    if case["padded"]:
        st["tokens"] = torch.where(uniform(R) < 0.06, torch.full_like(st["tokens"], -1), st["tokens"])
    st["scale"] = D ** 0.5
    if case["op"] == "embed_train":
        st["d_out"] = normal(R, D)
    return st


def work(case):
    b = _SIZE[case["dtype"]]
    if case["op"] == "gr_step":
        n = case["E"] * case["D"]
        return {"bytes": n * (4 * b + 8) + case["D"] * 4, "flops": 20 * n}
    if case["op"] in ("gr", "gr_train"):
        n, state = case["E"] * case["T"] * case["D"], case["E"] * case["D"] * 4
        flags = case["E"] * case["T"] if case["p_done"] else 0
        forward = 4 * n * b + flags + case["D"] * 4 + state * (2 if case["init"] else 1)
        if case["op"] == "gr":
            return {"bytes": forward, "flops": 20 * n}
        return {"bytes": forward + 7 * n * b + flags + case["D"] * 8 + state * (2 if case["init"] else 1),
                "flops": 60 * n}
    if case["op"] in ("heads", "heads_train"):
        n = case["E"] * case["T"] * (case["H"] + case["H"] // case["G"]) * case["D"]
        extra = case["E"] * case["T"] * 4 + case["D"] * 8
        if case["op"] == "heads":
            return {"bytes": 2 * n * b + extra, "flops": 7 * n}
        return {"bytes": 5 * n * b + 2 * extra + case["D"] * 8, "flops": 20 * n}
    R, N, D = case["R"], case["N"], case["D"]
    kinds = N * (1.0 - math.exp(-R / N)) if R < 64 * N else N  # rows that are read at most
    lookup = int(min(R, kinds)) * D * b + R * 8 + R * D * b
    if case["op"] == "embed":
        return {"bytes": lookup, "flops": R * D}
    return {"bytes": lookup + R * D * b + N * D * b + R * 8, "flops": 3 * R * D}


# ------------------------------------------------------------------------ passes
def run(state):
    case = state["case"]
    if own:
        return _run_own(state, case)
    if case["op"] == "gr_step":
        return _plain_step(state, case)
    if case["op"] in ("gr", "gr_train"):
        return _plain_recurrence(state, case)
    if case["op"] in ("heads", "heads_train"):
        return _plain_heads(state, case)
    return _plain_embed(state, case)


def _run_own(st, case):
    import linear_recurrence_scan_reverse_amd as rl

    if case["op"] == "gr_step":
        out = rl.gated_recurrence_step(st["x"], st["input_gate"], st["decay_gate"], st["rate"], st["state"],
                                       st["reset"], st["slots"])
        return out, st["state"]
    if case["op"] == "gr":
        return rl.gated_recurrence(st["x"], st["input_gate"], st["decay_gate"], st["rate"], st["done"], st["init"],
                                   with_state=True)
    if case["op"] == "gr_train":
        out, last, marks = rl.gated_recurrence(st["x"], st["input_gate"], st["decay_gate"], st["rate"], st["done"],
                                               st["init"], with_state=True, with_marks=True)
        return (out, last) + rl.gated_recurrence_backward(st["d_out"], st["x"], st["input_gate"], st["decay_gate"],
                                                          st["rate"], marks, st["done"], st["d_final"])
    if case["op"] in ("heads", "heads_train"):
        how = dict(rotate=case["R"], interleaved=case["interleaved"], eps=_EPS)
        outs = rl.norm_rotate_heads(st["q"], st["k"], st["q_weight"], st["k_weight"], st["positions"], **how)
        if case["op"] == "heads":
            return outs
        return outs + rl.norm_rotate_heads_backward(st["dq"], st["dk"], st["q"], st["k"], st["q_weight"],
                                                    st["k_weight"], st["positions"], **how)
    out = rl.embed_tokens(st["table"], st["tokens"], scale=st["scale"])
    if case["op"] == "embed":
        return out
    return out, rl.embed_tokens_backward(st["d_out"], st["tokens"], case["N"], scale=st["scale"])


# ------------------------------------------------------------------------ plain forms
def _scan(log_a, b):
    """x_t = exp(log_a_t) x_{t-1} + b_t along dim 1, in steps of 1, 2, 4, ..."""
    k = 1
    while k < b.shape[1]:
        b = torch.cat([b[:, :k], b[:, k:] + log_a[:, k:].exp() * b[:, :-k]], 1)
        log_a = torch.cat([log_a[:, :k], log_a[:, k:] + log_a[:, :-k]], 1)
        k *= 2
    return b


def _gates(st, cut):
    """sigmoid of both gates, log a, a and sqrt(1 - a^2); cut: steps with a = 0, or None."""
    si, sr = st["input_gate"].float().sigmoid(), st["decay_gate"].float().sigmoid()
    log_a = -st["rate"] * sr
    if cut is not None:
        log_a = log_a.masked_fill(cut, -math.inf)
    return si, sr, log_a, log_a.exp(), (-torch.expm1(2.0 * log_a)).sqrt()


def _plain_step(st, case):
    si, _, _, a, m = _gates(st, (st["reset"] != 0).unsqueeze(1))
    where = slice(None) if st["slots"] is None else st["slots"].long()
    h = a * st["state"][where] + m * si * st["x"].float()
    st["state"][where] = h
    return h.to(st["x"].dtype), st["state"]


def _plain_recurrence(st, case):
    E, T, D = case["E"], case["T"], case["D"]
    dt = st["x"].dtype
    done = None if st["done"] is None else (st["done"] != 0).unsqueeze(2)
    cut = None if done is None else torch.cat([torch.zeros_like(done[:, :1]), done[:, :-1]], 1)
    si, sr, log_a, a, m = _gates(st, cut)
    x = st["x"].float()
    u = si * x
    b = m * u
    init = torch.zeros(E, D, device=x.device) if st["init"] is None else st["init"]
    b[:, 0] += a[:, 0] * init
    h = _scan(log_a, b)
    last = h[:, -1].clone() if done is None else h[:, -1].masked_fill(done[:, -1], 0.0)
    if case["op"] == "gr":
        return h.to(dt), last
    d = st["d_out"].float().clone()
    if st["d_final"] is not None:
        d[:, -1] += st["d_final"] if done is None else st["d_final"].masked_fill(done[:, -1], 0.0)
    later = torch.cat([log_a[:, 1:], torch.zeros_like(log_a[:, :1])], 1)
    g = _scan(later.flip(1), d.flip(1)).flip(1)
    before = torch.cat([init.unsqueeze(1), h[:, :-1]], 1)
    d_log_a = g * (a * before - u * a * a / m)
    du = m * g
    dx = si * du
    d_input = x * dx * (1.0 - si)
    d_decay = -st["rate"] * sr * (1.0 - sr) * d_log_a
    d_rate = -(sr * d_log_a).sum((0, 1), dtype=torch.float64).float()
    return h.to(dt), last, dx.to(dt), d_input.to(dt), d_decay.to(dt), d_rate, a[:, 0] * g[:, 0]


def _angles(st, case):
    """cos and sin [E, T, 1, R / 2]; in 64 bits, where far positions keep their angles."""
    R = case["R"]
    j = torch.arange(0, R, 2, dtype=torch.float64, device=st["q"].device)
    angle = st["positions"].double()[:, :, None, None] * 10000.0 ** (-j / max(R, 1))
    return angle.cos().float(), angle.sin().float()


def _rotated(x, cos, sin, case):
    """The first R of the last dimension turned pair by pair."""
    R = case["R"]
    if R == 0:
        return x
    if case["interleaved"]:
        a, b = x[..., 0:R:2], x[..., 1:R:2]
        turned = torch.stack([a * cos - b * sin, b * cos + a * sin], -1).flatten(-2)
    else:
        a, b = x[..., :R // 2], x[..., R // 2:R]
        turned = torch.cat([a * cos - b * sin, b * cos + a * sin], -1)
    return torch.cat([turned, x[..., R:]], -1)


def _plain_heads(st, case):
    cos, sin = _angles(st, case)
    outs, grads, d_weights = [], [], []
    for name in ("q", "k"):
        x, w = st[name].float(), st[name + "_weight"]
        inv = (x.square().mean(-1, keepdim=True) + _EPS).rsqrt()
        n = x * inv
        outs.append(_rotated(n * w, cos, sin, case).to(st[name].dtype))
        if case["op"] == "heads_train":
            d = _rotated(st["d" + name].float(), cos, -sin, case)
            d_weights.append((d * n).sum((0, 1, 2), dtype=torch.float64).float())
            d = d * w
            grads.append((inv * (d - n * (d * n).mean(-1, keepdim=True))).to(st[name].dtype))
    return tuple(outs + grads + d_weights)


def _plain_embed(st, case):
    tokens, dt = st["tokens"], st["table"].dtype
    valid = ((tokens >= 0) & (tokens < case["N"])).unsqueeze(1)
    rows = tokens.clamp(0, case["N"] - 1)
    out = torch.where(valid, st["table"][rows].float() * st["scale"], torch.zeros((), device=tokens.device)).to(dt)
    if case["op"] == "embed":
        return out
    d = torch.where(valid, st["d_out"].float(), torch.zeros((), device=tokens.device))
    total = torch.zeros(case["N"], case["D"], device=tokens.device).index_add_(0, rows, d)
    return out, (total * st["scale"]).to(dt)


# ------------------------------------------------------------------------ 64-bit values
def exact(case, seed):
    """Step by step, token by token and as matrices, from the definitions."""
    st = prepare(case, seed)
    if case["op"] == "gr_step":
        return _exact_step(st, case)
    if case["op"] in ("gr", "gr_train"):
        return _exact_recurrence(st, case)
    if case["op"] in ("heads", "heads_train"):
        return _exact_heads(st, case)
    return _exact_embed(st, case)


def _logistic(z):
    return 1.0 / (1.0 + torch.exp(-z.double()))


def _exact_step(st, case):
    state = st["state"].double()
    outs = []
    slots = list(range(case["E"])) if st["slots"] is None else st["slots"].tolist()
    fresh = st["reset"].tolist()
    for e, s in enumerate(slots):
        p = st["rate"].double() * _logistic(st["decay_gate"][e])
        v = _logistic(st["input_gate"][e]) * st["x"][e].double()
        state[s] = v if fresh[e] else torch.exp(-p) * state[s] + torch.sqrt(-torch.expm1(-2.0 * p)) * v
        outs.append(state[s].clone())
    return torch.stack(outs), state


def _exact_recurrence(st, case):
    E, T, D = case["E"], case["T"], case["D"]
    x = st["x"].double()
    gate, keep = _logistic(st["input_gate"]), _logistic(st["decay_gate"])
    rate = st["rate"].double()
    p = rate * keep
    lives = torch.ones(E, T + 1, 1, dtype=torch.float64, device=x.device)  # whether a step sees the one before it
    if st["done"] is not None:
        lives[:, 1:, 0] = (st["done"] == 0).double()
    a = torch.exp(-p) * lives[:, :-1]
    m = torch.where(lives[:, :-1] > 0, torch.sqrt(-torch.expm1(-2.0 * p)), torch.ones_like(p))
    states = torch.empty(E, T + 1, D, dtype=torch.float64, device=x.device)
    states[:, 0] = 0.0 if st["init"] is None else st["init"].double()
    for t in range(T):
        states[:, t + 1] = a[:, t] * states[:, t] + m[:, t] * gate[:, t] * x[:, t]
    out, last = states[:, 1:], states[:, T] * lives[:, T]
    if case["op"] == "gr":
        return out, last
    d = torch.zeros(E, D, dtype=torch.float64, device=x.device)
    if st["d_final"] is not None:
        d = st["d_final"].double() * lives[:, T]
    dx, d_input, d_decay = torch.empty_like(x), torch.empty_like(x), torch.empty_like(x)
    d_rate = torch.zeros_like(rate)
    for t in reversed(range(T)):
        d = d + st["d_out"][:, t].double()
        v = gate[:, t] * x[:, t]
        dx[:, t] = d * m[:, t] * gate[:, t]
        d_input[:, t] = d * m[:, t] * v * (1.0 - gate[:, t])
        # d m / d p = exp(-2 p) / m
        dp = d * (v * a[:, t] * torch.exp(-p[:, t]) / m[:, t] - a[:, t] * states[:, t])
        d_decay[:, t] = dp * p[:, t] * (1.0 - keep[:, t])
        d_rate += (dp * keep[:, t]).sum(0)
        d = d * a[:, t]
    return out, last, dx, d_input, d_decay, d_rate, d


def _exact_heads(st, case):
    R, D = case["R"], case["D"]
    dev = st["q"].device
    if case["interleaved"]:
        first, second = torch.arange(0, R, 2, device=dev), torch.arange(1, R, 2, device=dev)
    else:
        first, second = torch.arange(0, R // 2, device=dev), torch.arange(R // 2, R, device=dev)
    freq = torch.pow(torch.tensor(10000.0, dtype=torch.float64, device=dev),
                     -2.0 * torch.arange(R // 2, dtype=torch.float64, device=dev) / max(1, R))
    parts = ([], [], [])
    for name in ("q", "k"):
        heads = st[name].shape[2]
        w = st[name + "_weight"].double()
        o = torch.empty(st[name].shape, dtype=torch.float64, device=dev)
        dx, dw = torch.empty_like(o), torch.zeros_like(w)
        for e in range(case["E"]):
            turn = torch.polar(torch.ones((), dtype=torch.float64, device=dev),
                               st["positions"][e].double()[:, None] * freq).unsqueeze(1).expand(-1, heads, -1)
            x = st[name][e].double()
            rms = torch.sqrt((x * x).sum(-1, keepdim=True) / D + _EPS)
            z = x / rms * w
            pair = torch.complex(z[..., first], z[..., second]) * turn
            o[e] = z
            o[e][..., first], o[e][..., second] = pair.real, pair.imag
            if case["op"] == "heads_train":
                dz = st["d" + name][e].double()
                pair = torch.complex(dz[..., first], dz[..., second]) * turn.conj()
                dz[..., first], dz[..., second] = pair.real, pair.imag
                dw += (dz * x / rms).sum((0, 1))
                dz = dz * w
                dx[e] = dz / rms - x * (dz * x).sum(-1, keepdim=True) / (D * rms ** 3)
        parts[0].append(o)
        parts[1].append(dx)
        parts[2].append(dw)
    return tuple(parts[0]) if case["op"] == "heads" else tuple(parts[0] + parts[1] + parts[2])


def _exact_embed(st, case):
    out = torch.zeros(case["R"], case["D"], dtype=torch.float64, device=st["table"].device)
    seen = (st["tokens"] >= 0).nonzero().view(-1)
    tokens = st["tokens"][seen]
    out[seen] = st["table"].double()[tokens] * st["scale"]
    if case["op"] == "embed":
        return out
    total = torch.zeros(case["N"], case["D"], dtype=torch.float64, device=out.device)
    order = torch.argsort(tokens, stable=True)
    kinds, counts = torch.unique_consecutive(tokens[order], return_counts=True)
    rows = st["d_out"][seen[order]].double()
    # the running sum of each run of equal tokens, from one running sum of everything in blocks of columns
    ends = counts.cumsum(0)
    for c in range(0, case["D"], 128):
        run_ = torch.nn.functional.pad(rows[:, c:c + 128].cumsum(0), (0, 0, 1, 0))
        total[kinds, c:c + 128] = run_[ends] - run_[ends - counts]
    return out, total * st["scale"]
