"""Rows of a table by token and the table's gradient against the float64 oracle."""
from __future__ import annotations

import math

import pytest

torch = pytest.importorskip("torch")

import linear_recurrence_scan_reverse_amd as rl  # noqa: E402
from tests import sequence_oracle as so  # noqa: E402

pytestmark = pytest.mark.gpu
DTYPES = [torch.float32, torch.bfloat16, torch.float16]


def draw(R, N, D, dtype, seed=0, how="zipf"):
    g = torch.Generator().manual_seed(100 * seed + R + N + D)
    u = torch.rand(R, generator=g, dtype=torch.float64)
    tokens = {"zipf": lambda: torch.exp(u * math.log(N + 1)).long() - 1, "even": lambda: (u * N).long(),
              "one": lambda: torch.full((R,), N // 2), "rising": lambda: torch.sort((u * N).long()).values,
              "falling": lambda: torch.sort((u * N).long(), descending=True).values,
              "padding": lambda: torch.full((R,), -1)}[how]().clamp(max=N - 1)
    if how in ("zipf", "falling"):  # some out of range, on both sides and past 32 bits
        odd = torch.tensor([-1, N, -2 ** 63, 2 ** 63 - 1, 2 ** 32, 2 ** 40 + N - 1])
        at = torch.rand(R, generator=g) < 0.05
        tokens = torch.where(at, odd[torch.randint(0, 6, (R,), generator=g)], tokens)
    return {"table": torch.randn(N, D, generator=g).to(dtype), "tokens": tokens,
            "d": torch.randn(R, D, generator=g).to(dtype)}


def check(d, out, grad, scale, dtype):
    want = so.lookup(d["table"], d["tokens"], scale)
    so.close(out, want, so.stored(want, so.U * want.abs(), dtype), "rows")
    check_gradient(d, grad, scale, dtype)


def check_gradient(d, grad, scale, dtype):
    N = grad.shape[0]
    want, bound = so.table_gradient(d["d"], d["tokens"], N, scale)
    # float32's own last rounding is one of those counted
    so.close(grad, want, so.stored(want, bound, dtype), "table's gradient")
    seen = torch.zeros(N, dtype=torch.bool)
    t = d["tokens"].view(-1)
    seen[t[(t >= 0) & (t < N)]] = True
    assert not grad[~seen.to(grad.device)].any()


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("R,N,D", [
    (1, 1, 1), (1, 1, 8), (5, 3, 7), (31, 2, 64), (32, 40, 65), (33, 5, 250), (64, 18, 512), (65, 1024, 16), (300, 1025, 24),
    (1000, 1000, 72), (1024, 5000, 40), (1025, 3, 1000), (5000, 2000, 9), (33, 100000, 16), (4000, 64007, 8)])
def test_tokens(R, N, D, dtype):
    d = draw(R, N, D, dtype)
    scale = 1.7
    out = rl.embed_tokens(d["table"].cuda(), d["tokens"].cuda(), scale=scale)
    grad = rl.embed_tokens_backward(d["d"].cuda(), d["tokens"].cuda(), N, scale=scale)
    # the kernels' scale is a float32
    check(d, out, grad, torch.tensor(scale, dtype=torch.float32).item(), dtype)


@pytest.mark.parametrize("how", ["even", "one", "rising", "falling", "padding"])
@pytest.mark.parametrize("R,N", [(50, 7), (3000, 40), (7000, 3000), (70000, 5)])
def test_orders(R, N, how):
    d = draw(R, N, 12, torch.float32, seed=1, how=how)
    grad = rl.embed_tokens_backward(d["d"].cuda(), d["tokens"].cuda(), N)
    check_gradient(d, grad, 1.0, torch.float32)


def test_largest_table():
    N, D = 2 ** 20, 8
    d = draw(4096, N, D, torch.float16, seed=2, how="even")
    d["tokens"][:3] = torch.tensor([0, N - 1, N])
    out = rl.embed_tokens(d["table"].cuda(), d["tokens"].cuda())
    want = so.lookup(d["table"], d["tokens"], 1.0)
    assert torch.equal(out.cpu().double(), want)
    grad = rl.embed_tokens_backward(d["d"].cuda(), d["tokens"].cuda(), N)
    rows = torch.unique(d["tokens"][d["tokens"] < N])
    few = {"d": d["d"], "tokens": torch.where(d["tokens"] < N, torch.searchsorted(rows, d["tokens"]), -1)}
    check_gradient(few, grad[rows.cuda()], 1.0, torch.float16)
    empty = torch.ones(N, dtype=torch.bool, device="cuda")
    empty[rows.cuda()] = False
    assert not grad[empty].any()


def test_shapes_strides_and_buffers():
    N, D = 50, 40
    for dtype in DTYPES:
        d = draw(60, N, D, dtype, seed=3)
        for pad in (0, 8, 3):  # rows at 16 bytes and at odd places
            table = torch.nn.functional.pad(d["table"], (pad, pad)).cuda()[:, pad:pad + D]
            out = torch.full((4, 15, D + 2 * pad), 9.0, dtype=dtype, device="cuda")
            tokens = d["tokens"].view(4, 15).cuda()
            got = rl.embed_tokens(table, tokens, out=out[..., pad:pad + D])
            want = so.lookup(d["table"], d["tokens"], 1.0).view(4, 15, D)
            assert torch.equal(got.cpu().double(), want)
            assert (out[..., :pad] == 9).all() and (out[..., pad + D:] == 9).all()
            d_out = torch.nn.functional.pad(d["d"].view(4, 15, D), (pad, pad)).cuda()[..., pad:pad + D]
            to = torch.full((N, D + pad), 9.0, dtype=dtype, device="cuda")
            grad = rl.embed_tokens_backward(d_out, tokens, N, d_table=to[:, :D])
            check_gradient(d, grad, 1.0, dtype)
            assert (to[:, D:] == 9).all()
    # one token
    got = rl.embed_tokens(table, torch.tensor(3, device="cuda"))
    assert got.shape == (D,) and torch.equal(got, table[3])


def test_no_tokens():
    out = rl.embed_tokens(torch.ones(5, 8, device="cuda"), torch.empty(0, dtype=torch.int64, device="cuda"))
    assert out.shape == (0, 8)
    grad = rl.embed_tokens_backward(torch.empty(0, 8, device="cuda"), torch.empty(0, dtype=torch.int64, device="cuda"), 5,
                                    d_table=torch.ones(5, 8, device="cuda"))
    assert not grad.any()


def test_not_finite_stays_with_its_token():
    d = draw(2000, 30, 64, torch.float32, seed=4, how="even")
    ref = rl.embed_tokens_backward(d["d"].cuda(), d["tokens"].cuda(), 30)
    r = 700
    d["d"][r, 5] = math.inf
    d["tokens"][900] = -1
    d["d"][900] = math.nan  # padding is not read into any sum
    got = rl.embed_tokens_backward(d["d"].cuda(), d["tokens"].cuda(), 30)
    bad = torch.zeros(30, 64, dtype=torch.bool)
    bad[d["tokens"][r], 5] = True
    assert torch.isinf(got[bad.cuda()]).all() and torch.isfinite(got[~bad.cuda()]).all()
    rows = [n for n in range(30) if n not in (int(d["tokens"][r]), )]
    moved = draw(2000, 30, 64, torch.float32, seed=4, how="even")["tokens"][900]
    rows = [n for n in rows if n != int(moved)]
    same = (got[rows].cpu().double() - ref[rows].cpu().double()).abs()
    # the same terms in other chunks: no more than the additions' roundings apart
    _, bound = so.table_gradient(torch.nan_to_num(d["d"], posinf=0.0), d["tokens"], 30, 1.0)
    assert (same <= 2 * bound[rows]).all()


def test_same_every_time_streams_and_graphs():
    d = draw(20000, 3000, 96, torch.bfloat16, seed=5)
    d_out, tokens = d["d"].cuda(), d["tokens"].cuda()
    table = d["table"].cuda()
    ref = rl.embed_tokens_backward(d_out, tokens, 3000)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    for _ in range(3):
        assert torch.equal(rl.embed_tokens_backward(d_out, tokens, 3000), ref)
    other = rl.embed_tokens_backward(d_out, tokens, 3000, stream=side)
    torch.cuda.current_stream().wait_stream(side)
    assert torch.equal(other, ref)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = rl.embed_tokens(table, tokens, scale=2.0)
        grad = rl.embed_tokens_backward(d_out, tokens, 3000, scale=0.5)
    for seed in (6, 7, 8):
        n = draw(20000, 3000, 96, torch.bfloat16, seed=seed)
        d_out.copy_(n["d"])
        tokens.copy_(n["tokens"])
        want = rl.embed_tokens(table, tokens, scale=2.0), rl.embed_tokens_backward(d_out, tokens, 3000, scale=0.5)
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(out, want[0]) and torch.equal(grad, want[1])


def test_far_offsets():
    far = 2 ** 31 + 64
    table = torch.zeros(far + 4096, dtype=torch.bfloat16, device="cuda").as_strided((2, 64), (far, 1))
    table[1] = 3.0
    tokens = torch.tensor([0, 1, 1], device="cuda")
    out = torch.zeros(2 * far + 4096, dtype=torch.bfloat16, device="cuda").as_strided((3, 64), (far, 1))
    rl.embed_tokens(table, tokens, out=out)
    assert not out[0].any() and (out[1:] == 3).all()
    grad = rl.embed_tokens_backward(out, tokens, 2, d_table=table)
    assert not grad[0].any() and (grad[1] == 6).all()
