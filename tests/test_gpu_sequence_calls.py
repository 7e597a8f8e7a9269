"""The sequence operators called as programs call them: on two streams at once, from two captured
graphs, with other strides, at the ends of segments and at the largest and smallest sizes."""
from __future__ import annotations

import math

import pytest

torch = pytest.importorskip("torch")

import linear_recurrence_scan_reverse_amd as rl  # noqa: E402
from tests import sequence_oracle as so  # noqa: E402
from tests.test_gpu_gated_recurrence import both, check, draw, on_gpu  # noqa: E402

pytestmark = pytest.mark.gpu


def every_operator(seed, T=1500):
    """(call, inputs): a call that runs all operators on the inputs, on the current stream."""
    g = torch.Generator().manual_seed(seed)
    c = on_gpu(draw(2, T, 70, torch.bfloat16, seed=seed))
    c["q"] = torch.randn(2, T, 4, 32, generator=g).to(torch.bfloat16).cuda()
    c["k"] = torch.randn(2, T, 2, 32, generator=g).to(torch.bfloat16).cuda()
    c["w"] = torch.rand(32, generator=g).cuda()
    c["pos"] = torch.randint(0, 9000, (2, T), generator=g).to(torch.int32).cuda()
    c["table"] = torch.randn(300, 70, generator=g).to(torch.bfloat16).cuda()
    c["tokens"] = torch.randint(-1, 300, (2, T), generator=g).cuda()
    c["pool"] = torch.randn(6, 70, generator=g).cuda()
    c["slots"] = torch.tensor([4, 1], dtype=torch.int32).cuda()

    def call():
        forward, grads = both(c)
        heads = rl.norm_rotate_heads(c["q"], c["k"], c["w"], c["w"], c["pos"])
        head_grads = rl.norm_rotate_heads_backward(*heads, c["q"], c["k"], c["w"], c["w"], c["pos"])
        rows = rl.embed_tokens(c["table"], c["tokens"], scale=0.5)
        table = rl.embed_tokens_backward(c["d_out"], c["tokens"], 300, scale=0.5)
        pool = c["pool"].clone()
        step = rl.gated_recurrence_step(c["x"][:, 0], c["ig"][:, 0], c["dg"][:, 0], c["rate"], pool, None, c["slots"])
        return forward + grads + heads + head_grads + (rows, table, step, pool)

    return call, c


def test_two_streams_at_once():
    calls = [every_operator(s)[0] for s in (1, 2)]
    want = [call() for call in calls]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in calls]
    got = []
    for _ in range(3):
        for call, stream in zip(calls, streams):
            with torch.cuda.stream(stream):
                got.append(call())
    torch.cuda.synchronize()
    for i, outs in enumerate(got):
        assert all(torch.equal(x, y) for x, y in zip(outs, want[i % 2])), i


def test_two_graphs_of_one_memory_pool():
    made = [every_operator(s) for s in (3, 4)]
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        for call, _ in made:
            call()
    torch.cuda.current_stream().wait_stream(side)
    pool, graphs, outs = torch.cuda.graph_pool_handle(), [], []
    for call, _ in made:
        graphs.append(torch.cuda.CUDAGraph())
        with torch.cuda.graph(graphs[-1], pool=pool):
            outs.append(call())
    for seed in (5, 6, 7):
        for i in (0, 1):
            for name, value in every_operator(seed + 10 * i)[1].items():
                if torch.is_tensor(value):
                    made[i][1][name].copy_(value)
        for i in (1, 0, 1):
            graphs[i].replay()
            torch.cuda.synchronize()
            want = made[i][0]()
            assert all(torch.equal(x, y) for x, y in zip(outs[i], want)), (seed, i)


# ------------------------------------------------------------------ strides
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
def test_long_rows_of_unequal_strides(dtype):
    # every tensor by a stride of its own: pieces of buffers of other widths; long enough for segments
    E, T, D = 2, 2600, 70
    d = draw(E, T, D, dtype, seed=21, p_done=0.01)
    d["done"][0, 900] = True
    c = on_gpu(d)

    def wide(x, more, at):
        b = torch.full((E, T, D + more), 5.0, dtype=dtype, device="cuda")
        b[..., at:at + D].copy_(x)
        return b[..., at:at + D]

    def strided(c):
        s = dict(c, x=wide(c["x"], 3, 1), ig=wide(c["ig"], 10, 7), dg=wide(c["dg"], 1, 0), d_out=wide(c["d_out"], 6, 6))
        out, bufs = wide(c["x"] * 0, 5, 2), [wide(c["x"] * 0, n, 1) for n in (2, 4, 7)]
        got = rl.gated_recurrence(s["x"], s["ig"], s["dg"], s["rate"], s["done"], s["init"], with_state=True,
                                  with_marks=True, out=out)
        return got, rl.gated_recurrence_backward(s["d_out"], s["x"], s["ig"], s["dg"], s["rate"], got[2], s["done"],
                                                 s["d_final"], dx=bufs[0], d_input_gate=bufs[1], d_decay_gate=bufs[2])

    check(d, *strided(c))
    # what is not finite is so in the same places as where the strides are equal
    c["x"][0, 700, 3], c["init"][1, 5], c["d_out"][1, 2000, 6] = math.inf, math.nan, math.inf
    got, grads = strided(c)
    ref, ref_grads = both(c)
    for a, b in zip(got + grads, ref + ref_grads):
        assert torch.equal(torch.isfinite(a), torch.isfinite(b))
    assert torch.isfinite(got[0][0, 901:]).all() and not torch.isfinite(got[0][0, 700, 3])


def test_one_step_for_all():
    # a gate that all steps share, and a gradient that all rows share
    d = draw(3, 90, 40, torch.float32, seed=22)
    c = on_gpu(d)
    gate, grad = c["ig"][:, :1].expand(3, 90, 40), c["d_out"][:1].expand(3, 90, 40)
    d["ig"], d["d_out"] = gate.cpu(), grad.cpu()
    check(d, *both(dict(c, ig=gate, d_out=grad)))


def test_heads_and_rows_that_are_shared():
    g = torch.Generator().manual_seed(23)
    q = torch.randn(2, 5, 1, 64, generator=g).cuda().expand(2, 5, 3, 64)
    k = torch.randn(1, 5, 2, 64, generator=g).cuda().expand(2, 5, 2, 64)
    pos = torch.randint(0, 99, (2, 5), generator=g).to(torch.int32).cuda()
    dq = torch.randn(2, 1, 3, 64, generator=g).cuda().expand(2, 5, 3, 64)
    dk = torch.randn(2, 5, 2, 64, generator=g).cuda()
    outs = rl.norm_rotate_heads(q, k, None, None, pos)
    grads = rl.norm_rotate_heads_backward(dq, dk, q, k, None, None, pos)
    for x, dy, out, grad in ((q, dq, outs[0], grads[0]), (k, dk, outs[1], grads[1])):
        want = so.Heads(x, None, pos, 64, dy=dy.cpu())
        so.close(out, want.y, so.stored(want.y, want.y_b, torch.float32), "out")
        so.close(grad, want.dx, so.stored(want.dx, want.dx_b, torch.float32), "gradient")
    table = torch.randn(1, 24, generator=g).cuda().expand(7, 24)
    tokens = torch.tensor([6, 0, 9, -3]).cuda()
    with pytest.raises(rl.RlscanError):
        rl.embed_tokens(table, tokens)  # rows that are one row
    d_out = torch.randn(1, 24, generator=g).cuda().expand(4, 24)
    with pytest.raises(rl.RlscanError):
        rl.embed_tokens_backward(d_out, tokens, 7)


@pytest.mark.parametrize("T", [1, 17, 40])
def test_steps_far_apart(T):
    # steps 2^27 bytes and more from one another: offsets of 64 bits
    E, D, far = 2, 70, 2 ** 26 + 96
    d = draw(E, T, D, torch.bfloat16, seed=23)
    c = on_gpu(d)

    def wide(x):
        b = torch.empty((T - 1) * far + E * D, dtype=torch.bfloat16, device="cuda").as_strided((E, T, D), (D, far, 1))
        return b.copy_(x)

    s = dict(c, x=wide(c["x"]))
    got = rl.gated_recurrence(s["x"], s["ig"], s["dg"], s["rate"], s["done"], s["init"], with_state=True,
                              with_marks=True, out=wide(c["x"] * 0))
    grads = rl.gated_recurrence_backward(s["d_out"], s["x"], s["ig"], s["dg"], s["rate"], got[2], s["done"],
                                         s["d_final"], dx=wide(c["x"] * 0))
    check(d, got, grads)


# ------------------------------------------------------------------ rows in windows
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("T,cut", [(5, 1), (40, 16), (1300, 777), (2100, 1024)])
def test_windows_of_a_row(T, cut, dtype):
    # a row in two windows, its state, flags and gradients handed on, with and without an end at the border; a
    # state that is dropped may hold anything
    E, D = 4, 40
    d = draw(E, T, D, dtype, seed=30, p_done=0.01)
    d["done"][:, cut - 1] = torch.tensor([True, False, True, False])
    d["reset"] = torch.tensor([True, True, False, False])
    c = on_gpu(d)
    c["init"][0, 3] = math.nan
    d["init"][0, 3] = 0.0
    parts = []
    for a, b in ((0, cut), (cut, T)):
        p = {k: v[:, a:b] for k, v in c.items() if k in ("x", "ig", "dg", "d_out")}
        p["done"] = c["done"][:, a:b].contiguous()
        p["init"] = parts[0]["out"][1] if parts else c["init"]
        p["reset"] = parts[0]["done"][:, -1].contiguous() if parts else c["reset"]
        p["out"] = rl.gated_recurrence(p["x"], p["ig"], p["dg"], c["rate"], p["done"], p["init"], reset=p["reset"],
                                       with_state=True, with_marks=True)
        parts.append(p)
    d_final, grads = c["d_final"], []
    for p in reversed(parts):
        g = rl.gated_recurrence_backward(p["d_out"], p["x"], p["ig"], p["dg"], c["rate"], p["out"][2], p["done"], d_final,
                                         reset=p["reset"])
        d_final, grads = g[4], [g] + grads
    want = so.Recurrence(d["x"], d["ig"], d["dg"], d["rate"], d["done"], d["init"], d["d_out"], d["d_final"], d["reset"])
    out = torch.cat([p["out"][0] for p in parts], 1)
    so.close(out, want.out, so.stored(want.out, want.out_b, dtype), "out")
    so.close(parts[1]["out"][1], want.final, want.final_b, "final state")
    for i, name in enumerate(("dx", "di", "dr")):
        w = getattr(want, name)
        so.close(torch.cat([g[i] for g in grads], 1), w, so.stored(w, getattr(want, name + "_b"), dtype), name)
    so.close(grads[0][3] + grads[1][3], want.d_rate, want.d_rate_b + 3 * so.U * want.d_rate.abs(), "d_rate")
    so.close(grads[0][4], want.d_init, want.d_init_b, "d_init")
    assert not grads[0][4][:2].any() and not parts[1]["init"][[0, 2]].any()


# ------------------------------------------------------------------ ends of segments
@pytest.mark.parametrize("T", [511, 512, 513, 767, 768, 769, 1023, 1024, 1025, 2047, 2049])
def test_ends_of_segments(T):
    d = draw(1, T, 64, torch.float32, seed=24, p_done=0.004)
    d["done"][0, T - 1] = T % 2 == 0
    check(d, *both(on_gpu(d)))


def test_more_tiles_than_compute_units_and_long():
    # segments that are taken in more than one round, and the last one short
    d = draw(5, 1100, 64 * 60, torch.bfloat16, seed=25, p_done=0.002)
    check(d, *both(on_gpu(d)))


def test_many_shares_of_a_rate():
    # 2500 shares of d_rate and more: added up in two steps
    d = draw(2500, 3, 20, torch.float32, seed=26)
    check(d, *both(on_gpu(d)))


# ------------------------------------------------------------------ the largest and the smallest
def test_as_many_rows_as_a_launch_takes():
    E = 2 ** 22 - 1
    x = torch.linspace(-2, 2, E, device="cuda").view(E, 1, 1)
    rate = torch.full((1,), 0.5, device="cuda")
    out, final, marks = rl.gated_recurrence(x, x, x, rate, with_state=True, with_marks=True)
    dx, di, dd, dr, dh = rl.gated_recurrence_backward(x, x, x, x, rate, marks)
    pick = torch.tensor([0, 1, 12345, E // 2, E - 2, E - 1], device="cuda")
    some = x[pick].cpu()
    want = so.Recurrence(some, some, some, rate, d_out=some)
    so.close(out[pick], want.out, so.stored(want.out, want.out_b, torch.float32), "out")
    for name, got in (("dx", dx), ("di", di), ("dr", dd)):
        w = getattr(want, name)
        so.close(got[pick], w, so.stored(w, getattr(want, name + "_b"), torch.float32), name)
    assert torch.equal(final, out[:, 0]) and not marks.any()
    with pytest.raises(rl.RlscanError):
        big = torch.empty(1, 1, 1, device="cuda").expand(2 ** 22, 1, 1)
        rl.gated_recurrence(big, big, big, rate)


def test_one_token_of_no_dimension():
    table = torch.randn(9, 40, device="cuda")
    token = torch.tensor(4, device="cuda")
    assert torch.equal(rl.embed_tokens(table, token), table[4])
    d_out = torch.randn(40, device="cuda")
    got = rl.embed_tokens_backward(d_out, token, 9)
    assert torch.equal(got[4], d_out) and not got[[0, 1, 2, 3, 5, 6, 7, 8]].any()


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16, torch.float16])
@pytest.mark.parametrize("R,N,D", [
    (1, 1, 1), (3, 200, 64), (127, 31, 2), (256, 65, 130), (257, 64, 600), (1024, 33, 5), (1024, 3, 70),  # few tokens
    (1025, 31, 2), (1025, 1, 130), (1500, 31, 129), (5000, 2, 1), (70000, 3, 3),                          # few kinds
    (1025, 32, 130), (1500, 1000, 129), (1500, 1100, 3)])                                                 # sorted
def test_few_kinds_and_more(R, N, D, dtype):
    # both sides of the numbers of tokens and of kinds that are added up without a sort
    g = torch.Generator().manual_seed(R + N)
    tokens = torch.randint(-1, N + 1, (R,), generator=g)
    d_out = torch.randn(R, D + 2, generator=g).to(dtype)
    want, bound = so.table_gradient(d_out[:, :D], tokens, N, 0.7)
    on = d_out.cuda()[:, :D]
    for x in (on, on.contiguous()):
        big = torch.full((N, D + 3), 5.0, dtype=dtype, device="cuda")
        rl.embed_tokens_backward(x, tokens.cuda(), N, scale=0.7, d_table=big[:, 2:D + 2])
        so.close(big[:, 2:D + 2], want, so.stored(want, bound, dtype), "gradient")
        assert (big[:, :2] == 5).all() and (big[:, D + 2:] == 5).all()


@pytest.mark.parametrize("R,N", [(600, 6), (2000, 6), (2000, 40), (2000, 2000)])
def test_not_finite_stays_with_its_token(R, N):
    tokens = torch.arange(R).remainder(5).cuda()
    d_out = torch.randn(R, 40, device="cuda")
    want = rl.embed_tokens_backward(d_out, tokens, N)
    d_out[7, 3], d_out[11, 4], d_out[R - 1, 5] = math.inf, math.nan, -math.inf  # of tokens 2, 1 and 4
    got = rl.embed_tokens_backward(d_out, tokens, N)
    bad = torch.zeros(N, 40, dtype=torch.bool, device="cuda")
    bad[[2, 1, 4], [3, 4, 5]] = True
    assert torch.equal(torch.isfinite(got), ~bad) and torch.equal(got[~bad], want[~bad])


@pytest.mark.parametrize("R,N", [(1024, 5000), (1024, 2), (3000, 5000), (3000, 2)])
def test_one_token_many_times_and_padding_behind(R, N):
    # all tokens but some padding are one; whole numbers, so that sums are exact
    tokens = torch.full((R,), N - 1)
    tokens[::7] = -1
    tokens[-1] = N
    d_out = torch.randint(-8, 9, (R, 30)).float()
    want = d_out[tokens == N - 1].sum(0)
    got = rl.embed_tokens_backward(d_out.cuda(), tokens.cuda(), N).cpu()
    assert torch.equal(got[N - 1], want) and not got[:N - 1].any()


def test_no_tokens():
    table = torch.randn(9, 40, device="cuda")
    none = torch.empty(0, dtype=torch.int64, device="cuda")
    assert rl.embed_tokens(table, none).shape == (0, 40)
    assert not rl.embed_tokens_backward(torch.empty(0, 40, device="cuda"), none, 9).any()
    assert rl.embed_tokens(table, none.view(3, 0)).shape == (3, 0, 40)


def test_positions_of_either_end():
    # float64 angles: no more than 12 roundings of 2^-53 of an angle of 2^31 at most, 2^-18; of a pair's
    # two elements, each at most the largest (a turned pair is no longer than it was): 2^-17
    g = torch.Generator().manual_seed(27)
    q = torch.randn(4, 2, 64, generator=g)
    pos = torch.tensor([2 ** 31 - 1, -2 ** 31, 0, -1], dtype=torch.int32)
    out, _ = rl.norm_rotate_heads(q.cuda(), q.cuda(), positions=pos.cuda())
    want = so.Heads(q, None, pos, 64)
    largest = so.Heads(q, None, None, 0).y.abs().max()
    so.close(out, want.y, so.stored(want.y, want.y_b + 2.0 ** -17 * largest, torch.float32), "out")


def test_rows_longer_apart_than_32_bits():
    far = 2 ** 31 + 128
    table = torch.zeros(2 * far, dtype=torch.bfloat16, device="cuda").as_strided((2, 64), (far, 1))
    rows = torch.randn(2, 64, device="cuda").bfloat16()
    table.copy_(rows)
    tokens = torch.tensor([1, 0, 1, 5, -1], device="cuda")
    out = rl.embed_tokens(table, tokens)
    assert torch.equal(out[:3], rows[tokens[:3]]) and not out[3:].any()
    grad = torch.zeros(2 * far, dtype=torch.bfloat16, device="cuda").as_strided((2, 64), (far, 1))
    rl.embed_tokens_backward(out, tokens, 2, d_table=grad)
    want, bound = so.table_gradient(out, tokens, 2, 1.0)
    so.close(grad, want, so.stored(want, bound, torch.bfloat16), "gradient")
