"""Linear attention on the GPU against the float64 oracle.

Tolerances, fixed before the first run.  Let A be the oracle's result for the absolute
values of all inputs: the sum of the absolute values of an element's terms.  A
result in bfloat16 or float16 is rounded once (half a step, eps/2 of its value); what
is rounded before that (P and the states, to two bfloat16 terms: 2^-8 * 2^-8 of each
term, for both factors of a product: 2^-15 A; the dropped products of two second terms: 2^-16 A)
stays within 2^-14 A.  float32 results (and all of float32 storage) come from three
terms (2^-24 each, dropped products 3 * 2^-24), float32 sums of up to 64 + 128 + T/64
terms in a tree of MFMA steps and exp2 of differences of up to about 30 (30 * 2^-24):
2^-18 A.  The decay's gradient is the difference of sums over a chunk, so its A is the
largest of the row and head.
"""
from __future__ import annotations

import pytest
import torch

import linear_recurrence_scan_reverse_amd as rl
from tests import policy_oracle as po

pytestmark = pytest.mark.gpu

DTYPES = {"f32": torch.float32, "bf16": torch.bfloat16, "f16": torch.float16}
TERMS = {torch.float32: 2.0 ** -18, torch.bfloat16: 2.0 ** -14, torch.float16: 2.0 ** -14}


def half_step(dtype):
    return torch.finfo(dtype).eps / 2


def make(seed, E, T, H, G, K, V, dtype="bf16", per_step=True, p_done=0.1, init=True, decay=0.1):
    gen = torch.Generator().manual_seed(seed)
    dt = DTYPES[dtype]
    n = lambda *s: torch.randn(*s, generator=gen)
    Hkv = H // G
    d = {"q": n(E, T, H, K).to(dt), "k": (n(E, T, Hkv, K) * K ** -0.5).to(dt), "v": n(E, T, Hkv, V).to(dt),
         "g": -decay * torch.rand((E, T, H) if per_step else (H,), generator=gen),
         "done": (torch.rand(E, T, generator=gen) < p_done).to(torch.uint8) if p_done else None,
         "init": n(E, H, K, V) if init else None, "do": n(E, T, H, V).to(dt),
         "df": n(E, H, K, V) if init else None}
    return d


def gpu(x):
    return None if x is None else x.cuda()


def near(got, want, size, dtype_terms, what):
    """got within half a step of its own type, plus the terms' rounding, of want."""
    assert got.shape == want.shape, what
    err = (got.double().cpu() - want).abs()
    tol = half_step(got.dtype) * want.abs() + dtype_terms * size + 1e-30
    if got.dtype == torch.float16:
        tol = tol + 2.0 ** -25  # half a step of its subnormals
    worst = (err / tol).max().item() if err.numel() else 0.0
    assert torch.isfinite(got).all(), what
    assert worst <= 1.0, "%s: %.3g times the tolerance" % (what, worst)


def check_forward(d, scale=None, **kw):
    out, final = rl.linear_attention(gpu(d["q"]), gpu(d["k"]), gpu(d["v"]), gpu(d["g"]), gpu(d["done"]),
                                     gpu(d["init"]), scale=scale, with_state=True, **kw)
    want, last = po.linear_attention(d["q"], d["k"], d["v"], d["g"], d["done"], d["init"], scale)
    size, lsize = po.linear_attention(d["q"], d["k"], d["v"], d["g"], d["done"], d["init"], scale, magnitude=True)
    dt = d["q"].dtype
    near(out, want, size, TERMS[dt], "out")
    near(final, last, lsize, TERMS[torch.float32], "final state")
    return out, final


def check_backward(d, scale=None):
    got = rl.linear_attention_backward(gpu(d["do"]), gpu(d["q"]), gpu(d["k"]), gpu(d["v"]), gpu(d["g"]),
                                       gpu(d["done"]), gpu(d["init"]), gpu(d["df"]), scale=scale)
    args = (d["do"], d["q"], d["k"], d["v"], d["g"], d["done"], d["init"], d["df"], scale)
    want = po.linear_attention_backward(*args)
    size = po.linear_attention_backward(*args, magnitude=True)
    dt = d["q"].dtype
    for i, name in enumerate(("dq", "dk", "dv")):
        near(got[i], want[i], size[i], TERMS[dt], name)
    if d["g"].dim() == 3:
        top = size[3].amax(1, keepdim=True).expand_as(size[3]) if size[3].shape[1] else size[3]
    else:
        top = size[3]
        per = po.linear_attention_backward(d["do"], d["q"], d["k"], d["v"],
                                           d["g"].expand(d["q"].shape[:3]).contiguous(), *args[5:], magnitude=True)[3]
        if per.shape[1]:
            top = torch.maximum(top, per.amax(1).sum(0) * d["q"].shape[1])
    near(got[3], want[3], top, TERMS[torch.float32], "dg")
    if d["init"] is None:
        assert got[4] is None
    else:
        near(got[4], want[4], size[4], TERMS[torch.float32], "d_init")
    return got


LENGTHS = [1, 2, 15, 16, 17, 31, 32, 33, 63, 64, 65, 96, 127, 128, 129, 200]


@pytest.mark.parametrize("dtype", ["f32", "bf16", "f16"])
@pytest.mark.parametrize("T", LENGTHS)
def test_lengths(dtype, T):
    check_forward(make(T, 2, T, 2, 1, 64, 64, dtype))
    check_backward(make(T, 2, T, 2, 1, 64, 64, dtype))


@pytest.mark.parametrize("dtype", ["f32", "bf16", "f16"])
@pytest.mark.parametrize("K,V", [(1, 1), (3, 5), (8, 16), (16, 8), (24, 40), (40, 100), (65, 64), (64, 65), (100, 72),
                                 (127, 129 - 2), (128, 128), (128, 32), (32, 128)])
def test_head_sizes(dtype, K, V):
    check_forward(make(K * 131 + V, 2, 70, 2, 1, K, V, dtype))
    check_backward(make(K * 131 + V, 2, 70, 2, 1, K, V, dtype))


@pytest.mark.parametrize("dtype", ["f32", "bf16", "f16"])
@pytest.mark.parametrize("H,G", [(1, 1), (4, 2), (6, 3), (8, 8), (5, 5)])
@pytest.mark.parametrize("per_step", [True, False])
def test_shared_heads_and_decays(dtype, H, G, per_step):
    check_forward(make(H * 10 + G, 3, 90, H, G, 48, 64, dtype, per_step=per_step))
    check_backward(make(H * 10 + G, 3, 90, H, G, 48, 64, dtype, per_step=per_step))


def cuts(kind, E, T):
    done = torch.zeros(E, T, dtype=torch.uint8)
    if kind == "all":
        done[:] = 255
    elif kind == "last":
        done[:, -1] = 1
    elif kind == "first":
        done[:, 0] = 1
    elif kind == "chunk ends":
        done[:, 31::32] = 1
    elif kind == "after chunk ends":
        done[:, 32::32] = 1
    elif kind == "all but one":
        done[:] = 1
        done[0, T // 2] = 0
    elif kind == "one row":
        done[0] = 1
    return done


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("kind", ["none", "all", "last", "first", "chunk ends", "after chunk ends", "all but one",
                                  "one row"])
def test_episode_ends(dtype, kind):
    d = make(9, 2, 160, 2, 1, 32, 64, dtype)
    d["done"] = cuts(kind, 2, 160)
    _, final = check_forward(d)
    got = check_backward(d)
    closed = d["done"][:, -1] != 0
    assert torch.all(final.cpu()[closed] == 0)
    # a decay across a cut has gradient 0, exactly
    cut = torch.zeros(2, 160, dtype=torch.bool)
    cut[:, 1:] = d["done"][:, :-1] != 0
    assert torch.all(got[3].cpu()[cut] == 0)


@pytest.mark.parametrize("dtype", ["f32", "bf16", "f16"])
@pytest.mark.parametrize("value", [0.0, -1e-9, -0.5, -3.0, -20.0, -103.0, -105.0, -1e4, float(torch.finfo(torch.float32).min),
                                   -float("inf")])
def test_decays(dtype, value):
    """One decay for all steps, from none to one that empties the state at once."""
    d = make(11, 2, 150, 2, 1, 32, 32, dtype, p_done=0.02)
    d["g"] = torch.full((2, 150, 2), value)
    check_forward(d)
    check_backward(d)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_decays_of_all_sizes_in_one_row(dtype):
    """Strong and weak decays mixed: a strong one must not cost the weak ones behind it their bits."""
    d = make(12, 2, 300, 3, 1, 32, 32, dtype, p_done=0.0)
    gen = torch.Generator().manual_seed(1)
    pick = torch.randint(0, 6, (2, 300, 3), generator=gen)
    d["g"] = torch.tensor([-1e-4, -1e-3, -0.01, -0.1, -30.0, -float("inf")])[pick]
    check_forward(d)
    check_backward(d)


def test_growing_decays():
    """exp(g) above 1 is the same recurrence."""
    d = make(13, 1, 100, 2, 1, 32, 32, "f32", p_done=0.0, decay=-0.02)
    check_forward(d)
    check_backward(d)


@pytest.mark.parametrize("dtype", ["f32", "bf16", "f16"])
@pytest.mark.parametrize("T", [513, 1000, 2049, 4100])
def test_long_rows_are_cut_into_segments(dtype, T):
    """One row, one head: segments joined through the workspace, cuts anywhere."""
    H, G = (2, 2) if T == 1000 else (1, 1)
    fmt = {"f32": 0, "bf16": 1, "f16": 2}[dtype]
    assert rl.lib().rlscan_linear_attention_workspace(fmt, 1, T, H, H // G, 32, 40, 0) > 0
    d = make(T, 1, T, H, G, 32, 40, dtype, p_done=0.002, decay=0.01)
    check_forward(d)
    if T < 3000:
        check_backward(d)


def test_a_given_scale_and_no_initial_state():
    d = make(21, 2, 100, 2, 1, 32, 32, "f32", init=False)
    check_forward(d, scale=-1.5)
    check_backward(d, scale=-1.5)
    check_forward(d, scale=0.0)


def test_empty_rows():
    d = make(22, 2, 0, 2, 1, 32, 16, "f32", p_done=0.0)
    out, final = check_forward(d)
    assert out.shape == (2, 0, 2, 16) and torch.equal(final.cpu(), d["init"])
    got = check_backward(d)
    assert torch.equal(got[4].cpu(), d["df"])
    d["g"] = torch.zeros(2)
    got = check_backward(d)
    assert torch.all(got[3] == 0)
    d = make(22, 0, 40, 2, 1, 32, 16, "f32")
    out, final = check_forward(d)
    assert out.shape == (0, 40, 2, 16) and final.shape == (0, 2, 32, 16)
    d["g"] = torch.zeros(2)
    assert torch.all(check_backward(d)[3] == 0)


def test_time_major_and_strides():
    """Time-major tensors, slices of a fused projection at odd offsets, heads before steps: the same bits."""
    E, T, H, G, K, V = 3, 130, 4, 2, 40, 24
    for dtype in ("bf16", "f32"):
        d = {n: gpu(x) for n, x in make(31, E, T, H, G, K, V, dtype).items()}
        base = rl.linear_attention(d["q"], d["k"], d["v"], d["g"], d["done"], d["init"], with_state=True)
        grads = rl.linear_attention_backward(d["do"], d["q"], d["k"], d["v"], d["g"], d["done"], d["init"], d["df"])

        tm = {n: (x.transpose(0, 1).contiguous() if n not in ("init", "df") else x) for n, x in d.items()}
        out, final = rl.linear_attention(tm["q"], tm["k"], tm["v"], tm["g"], tm["done"], tm["init"], with_state=True,
                                         time_major=True)
        assert torch.equal(out.transpose(0, 1), base[0]) and torch.equal(final, base[1])
        got = rl.linear_attention_backward(tm["do"], tm["q"], tm["k"], tm["v"], tm["g"], tm["done"], tm["init"],
                                           tm["df"], time_major=True)
        for i, (a, b) in enumerate(zip(got, grads)):
            assert torch.equal(a.transpose(0, 1) if i < 4 else a, b), i

        Hkv = H // G
        for lead in (0, 1, 3, 8):  # elements in front of q: with and without 16-byte alignment
            width = lead + H * K + Hkv * K + Hkv * V + 5
            fused = torch.randn(E, T, width, device="cuda").to(d["q"].dtype)
            cut = lambda buf: (buf[:, :, lead:lead + H * K].view(E, T, H, K),
                               buf[:, :, lead + H * K:lead + H * K + Hkv * K].view(E, T, Hkv, K),
                               buf[:, :, lead + H * K + Hkv * K:width - 5].view(E, T, Hkv, V))
            for part, x in zip(cut(fused), (d["q"], d["k"], d["v"])):
                part.copy_(x)
            q, k, v = cut(fused)
            out, final = rl.linear_attention(q, k, v, d["g"], d["done"], d["init"], with_state=True)
            assert torch.equal(out, base[0]) and torch.equal(final, base[1])
            dfused = torch.full_like(fused, 7.0)  # gradients side by side in one buffer
            dq, dk, dv = cut(dfused)
            got = rl.linear_attention_backward(d["do"], q, k, v, d["g"], d["done"], d["init"], d["df"], dq=dq, dk=dk,
                                               dv=dv)
            for a, b in zip(got, grads):
                assert torch.equal(a, b)
            assert torch.all(dfused[:, :, :lead] == 7) and torch.all(dfused[:, :, width - 5:] == 7)

        hb = {n: d[n].transpose(1, 2).contiguous().transpose(1, 2) for n in ("q", "k", "v", "do")}  # [E, H, T, D] memory
        out = rl.linear_attention(hb["q"], hb["k"], hb["v"], d["g"], d["done"], d["init"])
        assert torch.equal(out, base[0])
        # one key and value for all environments, broadcast with stride 0
        k1, v1 = d["k"][:1].expand(E, T, Hkv, K), d["v"][:1].expand(E, T, Hkv, V)
        out = rl.linear_attention(d["q"], k1, v1, d["g"], d["done"], d["init"])
        assert torch.equal(out, rl.linear_attention(d["q"], k1.contiguous(), v1.contiguous(), d["g"], d["done"],
                                                    d["init"]))


def test_windows_chain_through_the_state():
    d = make(41, 2, 192, 2, 1, 64, 64, "f32", p_done=0.03)
    want, last = po.linear_attention(d["q"], d["k"], d["v"], d["g"], d["done"], d["init"])
    size, lsize = po.linear_attention(d["q"], d["k"], d["v"], d["g"], d["done"], d["init"], magnitude=True)
    state, outs = gpu(d["init"]), []
    for lo, hi in ((0, 1), (1, 50), (50, 114), (114, 115), (115, 192)):
        out, state = rl.linear_attention(*(gpu(d[n][:, lo:hi].contiguous()) for n in ("q", "k", "v", "g")),
                                         gpu(d["done"][:, lo:hi].contiguous()), state, with_state=True)
        outs.append(out)
    near(torch.cat(outs, 1), want, size, TERMS[torch.float32], "out")
    near(state, last, lsize, TERMS[torch.float32], "state")


@pytest.mark.parametrize("dtype", ["f32", "bf16", "f16"])
@pytest.mark.parametrize("H,G,K,V", [(2, 1, 64, 64), (4, 2, 48, 40), (3, 3, 128, 128), (1, 1, 1, 3), (2, 1, 33, 65)])
@pytest.mark.parametrize("per_row", [True, False])
def test_steps_follow_the_recurrence(dtype, H, G, K, V, per_row):
    E, T = 3, 12
    d = make(K + V, E, T, H, G, K, V, dtype, per_step=per_row, p_done=0.2)
    want, last = po.linear_attention(d["q"], d["k"], d["v"], d["g"], d["done"], d["init"])
    size, lsize = po.linear_attention(d["q"], d["k"], d["v"], d["g"], d["done"], d["init"], magnitude=True)
    state = gpu(d["init"]).clone()
    reset = None
    for t in range(T):
        out = rl.linear_attention_step(gpu(d["q"][:, t].contiguous()), gpu(d["k"][:, t].contiguous()),
                                       gpu(d["v"][:, t].contiguous()),
                                       gpu(d["g"][:, t].contiguous() if per_row else d["g"]), state, reset)
        reset = gpu(d["done"][:, t].contiguous())
        near(out, want[:, t], size[:, t], TERMS[torch.float32], "step %d" % t)
    state = state * (reset == 0).view(E, 1, 1, 1)
    near(state, last, lsize, TERMS[torch.float32], "state")


@pytest.mark.parametrize("E", [5, 600])
def test_step_pool(E):
    """States in a pool, slots in any order; rows without a slot change nothing; dropped states may hold NaN."""
    H, K, V, S = 2, 64, 40, E + 7
    gen = torch.Generator().manual_seed(3)
    d = make(50, E, 1, H, 1, K, V, "bf16", p_done=0.0)
    pool = torch.randn(S, H, K, V, generator=gen)
    slots = torch.randperm(S, generator=gen)[:E].to(torch.int32)
    slots[1], slots[2] = -1, S
    slots[3] = -2 ** 31
    reset = torch.zeros(E, dtype=torch.uint8)
    reset[0] = 1
    d["g"][4] = -float("inf")
    state = pool.clone()
    state[slots[0].item()] = float("nan")
    state[slots[4].item()] = float("inf")
    state = state.cuda()
    before = state.clone()
    out = rl.linear_attention_step(gpu(d["q"][:, 0].contiguous()), gpu(d["k"][:, 0].contiguous()),
                                   gpu(d["v"][:, 0].contiguous()), gpu(d["g"][:, 0].contiguous()), state, gpu(reset),
                                   gpu(slots))
    good = [e for e in range(E) if 0 <= slots[e] < S]
    start = pool[slots[good].long()]
    start[0] = 0
    start[good.index(4)] = 0
    sub = lambda x: x[good]
    args = (sub(d["q"]), sub(d["k"]), sub(d["v"]), sub(d["g"]), None, start)
    want, last = po.linear_attention(*args)
    size, lsize = po.linear_attention(*args, magnitude=True)
    near(out[good], want[:, 0], size[:, 0], TERMS[torch.float32], "out")
    near(state[slots[good].long().cuda()], last, lsize, TERMS[torch.float32], "state")
    assert torch.all(out[[1, 2, 3]] == 0)
    other = [s for s in range(S) if s not in set(slots[good].tolist())]
    assert torch.equal(state[other], before[other])


def test_step_strides_and_unaligned_state():
    E, H, K, V = 4, 2, 32, 20
    d = {n: gpu(x) for n, x in make(51, E, 1, H, 1, K, V, "f16", p_done=0.0).items()}
    q, k, v, g = (d[n][:, 0].contiguous() for n in ("q", "k", "v", "g"))
    state = d["init"].clone()
    base = rl.linear_attention_step(q, k, v, g, state)
    raw = torch.zeros(state.numel() + 1, device="cuda")
    other = raw[1:].view_as(state).copy_(d["init"])
    fused = torch.zeros(E, H, 2 * K + V + 3, device="cuda", dtype=torch.float16)
    parts = fused[:, :, 3:3 + K], fused[:, :, 3 + K:3 + 2 * K], fused[:, :, 3 + 2 * K:]
    for p, x in zip(parts, (q, k, v)):
        p.copy_(x)
    out = torch.full((H, E, V + 1), 5.0, device="cuda", dtype=torch.float16)
    rl.linear_attention_step(*parts, g, other, out=out[:, :, :V].transpose(0, 1))
    assert torch.equal(out[:, :, :V].transpose(0, 1), base) and torch.all(out[:, :, V] == 5)
    assert torch.equal(other, state)


def test_gradient_is_the_difference_quotient():
    """The loss is linear in q, k, v and the initial state one at a time, so differences of any size are exact but for
    rounding: the float32 outputs' 2^-18 of their terms over the step h."""
    d = make(61, 2, 100, 4, 2, 32, 32, "f32", p_done=0.03)
    names = {"q": 0, "k": 1, "v": 2, "init": 4, "g": 3}
    grads = rl.linear_attention_backward(gpu(d["do"]), gpu(d["q"]), gpu(d["k"]), gpu(d["v"]), gpu(d["g"]),
                                         gpu(d["done"]), gpu(d["init"]), gpu(d["df"]))
    size, lsize = po.linear_attention(d["q"], d["k"], d["v"], d["g"], d["done"], d["init"], magnitude=True)
    terms = float((size * d["do"].double().abs()).sum() + (lsize * d["df"].double().abs()).sum())

    def loss(**kw):
        x = {n: gpu(y) for n, y in dict(d, **kw).items()}
        out, final = rl.linear_attention(x["q"], x["k"], x["v"], x["g"], x["done"], x["init"], with_state=True)
        return float((out.double() * x["do"].double()).sum() + (final.double() * x["df"].double()).sum())

    for name, i in names.items():
        gen = torch.Generator().manual_seed(i)
        way = torch.randn(d[name].shape, generator=gen)
        h = 0.5 if name != "g" else 2.0 ** -8
        x = d[name]
        up, down = x + h * way, x - h * way
        slope = (loss(**{name: up}) - loss(**{name: down}))
        want = float((grads[i].double().cpu() * (up.double() - down.double())).sum())
        tol = 4 * 2.0 ** -18 * terms
        if name == "g":  # third derivative: (h |way| T)^3 / 6 of the terms, over a memory of about 1 / 0.05 steps
            tol += (3 * h * 20) ** 3 / 6 * terms * 1e-2
        assert abs(slope - want) <= tol, (name, slope, want, tol)


def test_same_bits_every_time_and_on_another_stream():
    d = {n: gpu(x) for n, x in make(71, 3, 700, 4, 2, 64, 64, "bf16").items()}
    run = lambda **kw: (rl.linear_attention(d["q"], d["k"], d["v"], d["g"], d["done"], d["init"], with_state=True, **kw)
                        + rl.linear_attention_backward(d["do"], d["q"], d["k"], d["v"], d["g"], d["done"], d["init"],
                                                       d["df"], **kw))
    base = run()
    for _ in range(3):
        assert all(torch.equal(a, b) for a, b in zip(run(), base))
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    got = run(stream=side)
    side.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(got, base))


def test_captured_in_a_graph():
    d = {n: gpu(x) for n, x in make(72, 1, 1200, 2, 1, 64, 64, "bf16", p_done=0.01).items()}
    state = d["init"].clone()
    step_in = [d[n][:, 0].contiguous() for n in ("q", "k", "v", "g")]

    def work():
        return (rl.linear_attention(d["q"], d["k"], d["v"], d["g"], d["done"], d["init"], with_state=True)
                + rl.linear_attention_backward(d["do"], d["q"], d["k"], d["v"], d["g"], d["done"], d["init"], d["df"])
                + (rl.linear_attention_step(*step_in, state),))

    work()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        outs = work()
    for i in range(4):
        gen = torch.Generator(device="cuda").manual_seed(i)
        for n in ("q", "k", "v", "do"):
            d[n].copy_(torch.randn(d[n].shape, generator=gen, device="cuda"))
        for x, n in zip(step_in, ("q", "k", "v", "g")):
            x.copy_(d[n][:, 0])
        state.copy_(d["init"])
        graph.replay()
        torch.cuda.synchronize()
        got, after = [x.clone() for x in outs], state.clone()
        state.copy_(d["init"])
        for a, b in zip(got, work()):
            assert torch.equal(a, b)
        assert torch.equal(after, state)


def test_offsets_past_32_bits():
    """Steps 2^26 elements apart (the row spans 10 GB), and a pool whose last slot lies past 2^31 elements."""
    T, H, K = 75, 1, 64
    d = make(81, 1, T, H, 1, K, K, "bf16", p_done=0.0)
    far = torch.zeros(2 ** 26 * (T - 1) + 3 * K, dtype=torch.bfloat16, device="cuda")
    parts = [far[i * K:].as_strided((1, T, H, K), (0, 2 ** 26, K, 1), i * K) for i in range(3)]
    for p, n in zip(parts, ("q", "k", "v")):
        p.copy_(d[n])
    base = rl.linear_attention(gpu(d["q"]), gpu(d["k"]), gpu(d["v"]), gpu(d["g"]))
    assert torch.equal(rl.linear_attention(*parts, gpu(d["g"])), base)
    grads = rl.linear_attention_backward(gpu(d["do"]), gpu(d["q"]), gpu(d["k"]), gpu(d["v"]), gpu(d["g"]))
    got = rl.linear_attention_backward(gpu(d["do"]), *parts, gpu(d["g"]))
    assert all(torch.equal(a, b) for a, b in zip(got[:4], grads[:4]))
    del far, parts
    S, V = 2 ** 17 + 50, 128
    pool = torch.zeros(S, 1, 128, V, device="cuda")
    e = make(82, 2, 1, 1, 1, 128, V, "bf16", p_done=0.0)
    slots = torch.tensor([S - 1, 2 ** 17 + 3], dtype=torch.int32)
    pool[slots.long().cuda()] = gpu(e["init"])
    state = gpu(e["init"]).clone()
    ins = [gpu(e[n][:, 0].contiguous()) for n in ("q", "k", "v", "g")]
    base = rl.linear_attention_step(*ins, state)
    assert torch.equal(rl.linear_attention_step(*ins, pool, None, slots.cuda()), base)
    assert torch.equal(pool[slots.long().cuda()], state)
    assert float(pool[:100].abs().sum()) == 0.0


def test_refusals_on_the_gpu():
    d = {n: gpu(x) for n, x in make(91, 2, 10, 4, 2, 16, 16, "bf16").items()}
    call = lambda **kw: rl.linear_attention(*(kw.get(n, d[n]) for n in ("q", "k", "v", "g", "done", "init")))
    call()
    with pytest.raises(TypeError):
        call(k=d["k"].float())
    with pytest.raises(TypeError):
        call(g=d["g"].bfloat16())
    with pytest.raises(ValueError):
        call(k=d["k"][:, :, :, :15])
    with pytest.raises(ValueError):
        call(v=d["v"][:1])
    with pytest.raises(ValueError):
        call(g=d["g"][:, :, :3])
    with pytest.raises(ValueError):
        call(init=d["init"].transpose(2, 3))
    with pytest.raises(ValueError):
        call(q=d["q"].transpose(2, 3).contiguous().transpose(2, 3))
    with pytest.raises(ValueError):
        call(k=d["k"].repeat(1, 1, 2, 1)[:, :, :3], v=d["v"].repeat(1, 1, 2, 1)[:, :, :3])
    with pytest.raises(TypeError):
        call(done=d["done"].int())
    big = torch.zeros(1, 4, 1, 129, device="cuda")
    with pytest.raises(rl.RlscanError):
        rl.linear_attention(big, big, big, torch.zeros(1, device="cuda"))
    with pytest.raises(rl.RlscanError):  # output on an input
        rl.linear_attention(d["q"], d["k"], d["v"], d["g"], out=d["q"])
    with pytest.raises(ValueError):
        rl.linear_attention_step(d["q"][:, 0], d["k"][:, 0], d["v"][:, 0], d["g"][:, 0].contiguous(),
                                 d["init"][:1])
    with pytest.raises(TypeError):
        rl.linear_attention_step(d["q"][:, 0], d["k"][:, 0], d["v"][:, 0], d["g"][:, 0].contiguous(), d["init"],
                                 None, torch.zeros(2, dtype=torch.int64, device="cuda"))
